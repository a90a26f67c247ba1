"""A shared prefix's scratch while decode steps that use it still run on another stream."""
import pytest
import torch

from cross_loop_sparsity_b200 import flashloop as fl
from cross_loop_sparsity_b200 import synth

pytestmark = pytest.mark.gpu


def test_scratch_is_not_given_out_under_a_running_step():
    """The steps wait behind two tenths of a second of other work on their stream; sharing ends meanwhile, and the next
    buffers of the scratch's size lie elsewhere until the steps are done."""
    cfg = synth.config("c2").with_(n_layers=1, n_loops=2)
    w = synth.make_weights(cfg)
    lens, n = [300, 280], 256
    ctx = synth.make_context(cfg, w["rng"], lens)
    eng = fl.FlashLoop(cfg, fl.upload_weights(w), max_batch=2, max_ctx=310)
    eng.load_context(ctx, False)
    side, h0 = torch.cuda.Stream(), torch.randn((2, cfg.d_model), device="cuda")
    h = torch.empty_like(h0)
    eng.share_prefix(2, n)
    ptr, nbytes = eng._share_scratch.data_ptr(), eng._share_scratch.numel()
    eng.decode_step(h0, 2, h, stream=side)
    torch.cuda.synchronize()
    want = h.clone()
    eng.reset(lens)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)
    eng.decode_step(h0, 2, h, stream=side)
    eng.share_prefix(0, 0)
    with torch.cuda.stream(torch.cuda.default_stream()):
        others = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not side.query()                         # the step has not run yet
    assert all(x.data_ptr() + nbytes <= ptr or x.data_ptr() >= ptr + nbytes for x in others)
    torch.cuda.synchronize()
    assert torch.equal(h, want) and eng.sync_status() == 0
    eng.close()
