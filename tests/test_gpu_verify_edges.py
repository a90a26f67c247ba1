"""Draft verification at the ends of what it accepts."""
import pytest
import torch

from cross_loop_sparsity_b200 import flashloop as fl
from test_gpu_serving import ints

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
MAX = float(torch.finfo(torch.float32).max)


# ---------------------------------------------------------------------------- greedy
@pytest.mark.parametrize("V", [1, 17, 8188, 20000])
@pytest.mark.parametrize("fill", [NAN, -INF])
def test_greedy_rows_without_a_candidate(V, fill):
    """Only NaN, or nothing above -inf: token -1, and no draft is accepted there, whatever its token."""
    logits = torch.zeros((5, 3, V), device="cuda")
    logits[:, 0, V // 2] = 1.0
    logits[:4, 1] = fill          # the deciding row behind an accepted draft
    logits[4, 0] = fill           # the first row
    draft = ints([[V // 2, 2 ** 31 - 1], [V // 2, -1], [V // 2, 0], [V // 2, V - 1], [2 ** 31 - 1, 0]])
    tok, acc = fl.verify_draft(logits, None, draft, None, temperature=0.0)
    assert acc.tolist() == [1, 1, 1, 1, 0]
    assert tok.tolist() == [[V // 2, -1, -1]] * 4 + [[-1, -1, -1]]


def test_greedy_candidates_beside_nan_and_infinities():
    """A chunk of NaN beside one that holds a logit, the lowest finite value beside -inf, and +inf (the largest)."""
    logits = torch.full((4, 1, 20000), NAN, device="cuda")
    logits[0, 0, 19999] = -5.0
    logits[1, 0, :9000] = -INF
    logits[1, 0, 9001] = -MAX
    logits[2, 0, 12000:12002] = INF
    logits[3, 0, 3] = -INF
    tok, _ = fl.verify_draft(logits, None, None, None, temperature=0.0)
    assert tok[:, 0].tolist() == [19999, 9001, 12000, -1]
