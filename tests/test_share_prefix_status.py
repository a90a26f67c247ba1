"""A wait of a shared decode step's attention that runs out is recorded where flashloop_sync_status finds it, like those of
every other kernel of a step.  (No input makes such a wait run out, so the wiring is read.)"""
import os
import re

from cross_loop_sparsity_b200 import build as fl_build


def source(name):
    with open(os.path.join(fl_build.CSRC, name)) as f:
        return f.read()


def test_waits_of_the_shared_attention_record_their_status():
    text = source("fl_prefix.cu")
    at = text.index("    k_prefix_split(")
    body = text[at:text.index("\n}\n", at)]
    waits = re.findall(r"mbar_wait\(.*?, ([\w.]+)\)[;)]", body)
    assert len(waits) == body.count("mbar_wait(") >= 2
    assert set(waits) == {"a.status"}


def test_the_step_hands_its_status_on():
    assert re.search(r"\ba\.status = L\.status;", source("fl_prefix.cu"))
    step = source("fl_runtime.cu")
    at = step.index("PrefixLaunch pl{};")
    assert "pl.status = ctx->status;" in step[at:step.index("launch_prefix(pl", at)]
