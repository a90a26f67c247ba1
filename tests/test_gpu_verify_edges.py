"""Draft verification at the ends of what it accepts."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from cross_loop_sparsity_b200 import flashloop as fl
from test_gpu_serving import check_verify, gen, ints, verify_inputs

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


# ---------------------------------------------------------------------------- temperatures
@pytest.mark.parametrize("T", [1e-20, 1e-19, 1e-18, 1e-17, 1e-16, 1e-14, 1e-10])
@pytest.mark.parametrize("B,D,V", [(64, 0, 300), (16, 3, 900), (4, 2, 40000)])
def test_smallest_temperatures(B, D, V, T):
    """Everything at the maximum, as (x - max) / T says, and never a row given up for its scale."""
    logits, dl, draft, u = verify_inputs(int(-np.log10(T)) + V, B, D, V, 1.0)
    logits += 12.0
    if D:
        draft[::2] = logits[::2, :D].argmax(-1).to(torch.int32)
    wt, wa = check_verify(logits, dl, draft, u, None, T)
    assert all(wt[b, wa[b]] >= 0 for b in range(B) if wa[b] == D)
    check_verify(logits, None, draft, u, None, T)


def test_logits_near_the_ends_of_fp32():
    """A forced token, rows masked with the type's lowest value, all of one value, and both ends in one row."""
    B, V = 8, 5003
    logits, _, _, u = verify_inputs(3, B, 0, V, 1.0)
    logits[0, 0, 4321] = 1e30
    logits[1, 0] = -MAX
    logits[2, 0] = MAX
    logits[3, 0, 100:] = -MAX
    logits[4, 0, 7], logits[4, 0, 8] = MAX, -MAX
    logits[5, 0] += 1e20
    logits[6, 0] = -1e30
    logits[6, 0, 5000:] = -1e30 * (1 + 2.0 ** -20)
    logits[7, 0] += 1e9
    for T in (1.0, 0.3, 1e-6):
        check_verify(logits, None, torch.empty((B, 0), dtype=torch.int32, device="cuda"), u, None, T)


@pytest.mark.parametrize("T", [1e30, 1e35, 1e36, 1e38, 3e38])
def test_largest_temperatures(T):
    """Every token that is not masked alike; the masked ones (-inf) never."""
    logits, dl, draft, u = verify_inputs(8, 16, 2, 4001, 1.0)
    logits[:, :, ::3] = -INF
    dl[:, :, ::5] = -INF
    wt, wa = check_verify(logits, None, draft, u, None, T)
    assert all(wt[b, wa[b]] % 3 for b in range(16))
    check_verify(logits[:, :1].contiguous(), None, torch.empty((16, 0), dtype=torch.int32, device="cuda"), u[:, :1].contiguous(), None, T)


@pytest.mark.parametrize("top", [3.0, 20.0, -50.0, 1e20])
@pytest.mark.parametrize("part", [0.3, 0.55, 0.75, 0.97, 1.2])
def test_temperatures_at_the_spacing_of_the_logits(top, part):
    """The logit next to the maximum lies between 2^-800 and 2^-4000 of it: it counts as nothing, or as that little."""
    x = np.float32(top)
    below = np.nextafter(x, np.float32(-INF))
    T = part * float(x - below) / (1000 * np.log(2.0))
    logits = torch.full((4, 1, 900), float(below), device="cuda")
    logits[:, 0, 555] = float(x)
    tok, _ = fl.verify_draft(logits, None, None, torch.rand((4, 1), generator=gen(1), device="cuda"), temperature=T)
    assert tok[:, 0].tolist() == [555] * 4


@pytest.mark.parametrize("T", [5e37, 3e38])
def test_logits_further_apart_than_fp32_reaches(T):
    """The lowest and the largest value in one row, at a temperature where both have weight."""
    B, D, V = 64, 3, 900
    g = gen(2)
    kind = torch.randint(0, 3, (B, D + 1, V), generator=g, device="cuda")
    logits = torch.where(kind == 0, -MAX, torch.where(kind == 1, 0.0, MAX))
    dl = torch.where(torch.randint(0, 3, (B, D, V), generator=g, device="cuda") == 0, -MAX, 0.5 * MAX)
    draft = torch.randint(0, V, (B, D), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand((B, D + 1), generator=g, device="cuda")
    check_verify(logits, dl, draft, u, None, T)
    check_verify(logits, None, draft, (u / V).contiguous(), None, T)


# ---------------------------------------------------------------------------- targets next to the draft
def tokens_of_the_residual(logits, dl, u):
    """Token of max(p_0 - q_0, 0) at u in 64 bits, and whether u is further than 2e-6 of the total from a border: the
    64-bit sums are good to 4e-14 of p, and p - q is about 1e-7 of p at the least here."""
    def soft(x):
        e = np.exp(x.astype(np.float64) - x.max(-1, keepdims=True))
        return e / e.sum(-1, keepdims=True)

    w = np.maximum(soft(logits) - soft(dl), 0.0)
    cdf = np.cumsum(w, -1)
    target = u.astype(np.float64) * cdf[:, -1]
    y = (cdf <= target[:, None]).sum(-1)
    rows = np.arange(len(y))
    lo, hi = cdf[rows, y] - w[rows, y], cdf[rows, y]
    return y, np.minimum(target - lo, hi - target) > 2e-6 * cdf[:, -1]


@pytest.mark.parametrize("share", [1.0, 0.5, 0.02])
@pytest.mark.parametrize("V", [777, 20011])
def test_target_next_to_the_draft(V, share):
    """The draft's logits are the target's next fp32 value, up or down, for a share of the tokens (the others' the target's
    own, but for one in a hundred, where they differ by 1e-4): the residual's signs hang on the totals' last bits."""
    B, g = 64, gen(V)
    x = 3.0 * torch.randn((B, V), generator=g, device="cuda")
    up = torch.rand((B, V), generator=g, device="cuda") < 0.5
    q = torch.nextafter(x, torch.where(up, INF, -INF))
    kind = torch.rand((B, V), generator=g, device="cuda")
    q = torch.where(kind < share, q, torch.where(kind > 0.99, x + 1e-4 * torch.randn((B, V), generator=g, device="cuda"), x))
    draft = (q - x).argmax(-1).to(torch.int32)[:, None]     # the least p / q: rejected at the largest u
    u = torch.rand((B, 2), generator=g, device="cuda")
    u[:, 0] = 1.0 - 2.0 ** -24
    logits = torch.stack([x, x], 1)
    want, sure = tokens_of_the_residual(x.cpu().numpy(), q.cpu().numpy(), u[:, 1].cpu().numpy())
    tok, acc = fl.verify_draft(logits, q[:, None].contiguous(), draft, u)
    _, wa = ref.verify(logits.cpu().numpy(), q[:, None].cpu().numpy(), draft.cpu().numpy(), u.cpu().numpy(), None, 1.0)
    assert np.array_equal(acc.cpu().numpy(), wa)      # (a row's q may be below its p everywhere that it could be rejected)
    sure &= wa == 0
    assert sure.mean() >= 0.85
    assert np.array_equal(tok[:, 0].cpu().numpy()[sure], want[sure])
