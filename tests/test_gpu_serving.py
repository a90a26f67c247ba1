"""The serving operators on the GPU against plain 64-bit statements of them:
attention over a shared prefix, column weights, eviction, draft verification."""
import math

import numpy as np
import pytest
import torch

import serving_ref as ref
from cross_loop_sparsity_b200 import flashloop as fl

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------- shared-prefix attention
def check_attention(q, kp, vp, k, v, lens, q_lens, scale=None):
    B, Tq, H, hd = q.shape
    Hkv = kp.shape[0] if kp is not None else k.shape[1]
    out = torch.full((B, Tq, H, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Tq, H), 7.0, device="cuda")
    fl.prefix_attention(q, kp, vp, k, v, None if lens is None else ints(lens),
                        q_lens=None if q_lens is None else ints(q_lens), scale=scale, out=out, lse=lse)
    torch.cuda.synchronize()
    none3, none4 = np.zeros((Hkv, 0, hd)), np.zeros((B, Hkv, 0, hd))
    want, wlse, tol, ltol = ref.attention(
        ref.f64(q), none3 if kp is None else ref.f64(kp), none3 if vp is None else ref.f64(vp),
        none4 if k is None else ref.f64(k), none4 if v is None else ref.f64(v),
        [0] * B if lens is None else lens, [Tq] * B if q_lens is None else q_lens,
        hd ** -0.5 if scale is None else scale)
    got, glse = ref.f64(out), lse.double().cpu().numpy()
    qn = [Tq] * B if q_lens is None else [min(max(x, 0), Tq) for x in q_lens]
    for b in range(B):
        n = qn[b]
        assert np.all(np.abs(got[b, :n] - want[b, :n]) <= tol[b, :n]), (
            b, np.max(np.abs(got[b, :n] - want[b, :n]) / np.maximum(tol[b, :n], 1e-30)))
        empty = np.isneginf(wlse[b, :n])
        assert np.array_equal(np.isneginf(glse[b, :n]), empty)
        assert np.all(np.abs(glse[b, :n] - wlse[b, :n])[~empty] <= ltol[b, :n][~empty])
        assert np.all(got[b, n:] == 7.0) and np.all(glse[b, n:] == 7.0)   # rows that are no query: untouched
    return out, lse


ATT = [
    # B, Tq, H, Hkv, hd, P, S, lens, q_lens
    (1, 1, 1, 1, 64, 1, 1, [1], None),
    (1, 1, 1, 1, 128, 0, 1, [1], None),
    (2, 1, 4, 4, 64, 128, 32, [32, 5], None),
    (3, 1, 8, 2, 128, 33, 40, [40, 1, 17], None),
    (2, 2, 6, 2, 128, 31, 9, [9, 2], [2, 1]),
    (4, 3, 5, 1, 64, 65, 70, [70, 3, 0, 33], [3, 2, 1, 0]),
    (5, 1, 16, 4, 128, 1000, 0, None, None),
    (2, 5, 24, 3, 128, 257, 100, [100, 64], [5, 4]),
    (9, 4, 8, 1, 128, 640, 33, [33, 4, 5, 6, 7, 8, 20, 31, 32], [4, 1, 2, 3, 4, 4, 3, 2, 1]),
    (33, 1, 8, 1, 64, 515, 3, [3] * 33, None),
    (1, 64, 2, 1, 128, 7, 130, [130], [64]),
    (2, 64, 4, 2, 64, 0, 64, [64, 40], [64, 40]),
    (3, 7, 64, 1, 64, 300, 12, [12, 7, 9], [7, 7, 2]),
    (40, 8, 8, 2, 128, 400, 20, list(range(8, 20)) * 3 + [20] * 4, [1 + i % 8 for i in range(40)]),
    (2, 1, 2, 2, 128, 20011, 3000, [3000, 1501], None),
    (70, 2, 4, 1, 128, 2049, 5, [5] * 70, [2, 0] * 35),
    (40, 1, 1, 1, 128, 128, 0, None, None),
    (12, 3, 4, 1, 64, 129, 4, [4, 3, 2] * 4, [3, 1, 2] * 4),
    (65, 1, 6, 2, 128, 1407, 2, [2] * 65, None),
    (33, 4, 4, 2, 128, 5000, 6, [6, 5, 4] * 11, [4, 3, 2] * 11),
    (64, 8, 2, 1, 64, 3333, 9, [9] * 64, [i % 9 for i in range(64)]),
    (9, 4, 8, 2, 128, 300, 4, [4] * 9, [0] * 9),
    # many rows, few columns: a row block per warp
    (117, 6, 64, 8, 128, 2, 8, [i % 9 for i in range(117)], [i % 7 for i in range(117)]),
    (128, 1, 12, 4, 128, 100, 200, [200 - i for i in range(128)], None),
    (100, 7, 16, 4, 64, 103, 130, [130 - (7 * i) % 131 for i in range(100)], [i % 8 for i in range(100)]),
    (80, 3, 30, 6, 64, 0, 33, [33, 1, 0, 32] * 20, [3, 1, 0, 2] * 20),
    (128, 2, 8, 8, 64, 1500, 17, [17 - i % 18 for i in range(128)], [2, 1] * 64),
    # prefixes long enough for the tensor-core kernel: lengths off its 128-column tiles, one row tile and several blocks
    # of two, a last block with one, sequences without queries
    (40, 1, 4, 4, 128, 12007, 0, None, None),
    (12, 3, 4, 1, 64, 37633, 4, [4, 3, 2] * 4, [3, 1, 2] * 4),
    (65, 1, 6, 2, 128, 7041, 2, [2] * 65, None),
    (33, 1, 8, 1, 64, 21001, 3, [3] * 33, None),
    (33, 4, 4, 2, 128, 6000, 6, [6, 5, 4] * 11, [4, 3, 2] * 11),
    (64, 8, 2, 1, 64, 6145, 9, [9] * 64, [i % 9 for i in range(64)]),
    (70, 2, 4, 1, 128, 5249, 5, [5] * 70, [2, 0] * 35),
    (40, 8, 8, 2, 128, 1291, 20, list(range(8, 20)) * 3 + [20] * 4, [1 + i % 8 for i in range(40)]),
    (3, 7, 64, 1, 64, 4600, 12, [12, 7, 9], [7, 7, 2]),
    (9, 4, 8, 2, 128, 9500, 4, [4] * 9, [0] * 9),
    (9, 4, 8, 2, 128, 9473, 4, [4] * 9, [1] * 9),
]


@pytest.mark.parametrize("case", ATT, ids=[f"{c[0]}x{c[1]}h{c[2]}_{c[3]}d{c[4]}p{c[5]}s{c[6]}" for c in ATT])
def test_attention_against_64_bits(case):
    B, Tq, H, Hkv, hd, P, S, lens, q_lens = case
    g = gen(P + S + B)
    q = normal(g, B, Tq, H, hd, scale=2.0)
    kp, vp = (normal(g, Hkv, P, hd), normal(g, Hkv, P, hd)) if P else (None, None)
    k, v = (normal(g, B, Hkv, S, hd), normal(g, B, Hkv, S, hd)) if S else (None, None)
    check_attention(q, kp, vp, k, v, lens, q_lens)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3])
def test_attention_scales(scale):
    """Large scores (one column takes all the weight), none at all, and a negative scale."""
    g = gen(3)
    check_attention(normal(g, 2, 2, 4, 64), normal(g, 2, 99, 64), normal(g, 2, 99, 64), normal(g, 2, 2, 40, 64),
                    normal(g, 2, 2, 40, 64), [40, 11], [2, 2], scale=scale)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3])
@pytest.mark.parametrize("hd,B,P", [(64, 15, 700), (128, 40, 700), (64, 64, 16001), (128, 40, 12007)])
def test_attention_scales_many_rows(hd, B, P, scale):
    """The same with more than 32 rows per KV head (the longer prefixes on the tensor-core kernel), scores growing along the
    prefix so that the running maximum moves often, and one or two row tiles."""
    g = gen(31)
    kp, vp = normal(g, 2, P, hd), normal(g, 2, P, hd)
    kp = (kp.float() * torch.linspace(0.1, 3.0, P, device="cuda")[None, :, None]).to(torch.bfloat16)
    check_attention(normal(g, B, 2, 6, hd), kp, vp, normal(g, B, 2, 8, hd), normal(g, B, 2, 8, hd), [8, 3, 2] * (B // 3) +
                    [5] * (B % 3), None, scale=scale)


@pytest.mark.parametrize("P", [500, 24301])
def test_attention_non_finite_scores_many_rows(P):
    """More than 32 rows per KV head (the longer prefix on the tensor-core kernel): a visible NaN key makes the rows NaN,
    columns of -inf score weigh nothing, a +inf score gives NaN, and no finite score at all 0 and -inf."""
    g = gen(32)
    q = normal(g, 24, 1, 8, 64).abs()
    kp, vp = normal(g, 4, P, 64), normal(g, 4, P, 64)
    kp[0, 130] = NAN
    kp[1, 5:300] = -INF                  # q > 0: scores -inf, the first two tiles all of them
    kp[2, P - 1] = INF
    kp[3] = -INF
    out, lse = fl.prefix_attention(q, kp, vp, None, None, None)
    o = out.float()
    for h in (0, 1, 4, 5):
        assert bool(torch.isnan(o[:, 0, h]).all()) and bool(torch.isnan(lse[:, 0, h]).all())
    assert bool((o[:, 0, 6:] == 0).all()) and bool((lse[:, 0, 6:] == -INF).all())
    keep = [i for i in range(P) if not 5 <= i < 300]
    want, wl = fl.prefix_attention(q, kp[:, keep].contiguous(), vp[:, keep].contiguous(), None, None, None)
    # each side within its bound of 2^-8 of A + |out|, A the mean |v| under the weights (below 5 here)
    assert bool(((o - want.float())[:, 0, 2:4].abs() <= 2 * 2 ** -8 * 10).all())
    assert bool(((lse - wl)[:, 0, 2:4].abs() <= 1e-4).all())


@pytest.mark.parametrize("B,P", [(3, 150), (24, 8001)])
def test_attention_strided_layouts(B, P):
    """Queries inside a wider projection, caches as [B][S][Hkv][hd] and [P][Hkv][hd], a strided output."""
    g = gen(4)
    Tq, H, Hkv, hd, S = 2, 8, 2, 128, 70
    qkv = normal(g, B, Tq, (H + 2 * Hkv) * hd)
    q = qkv[..., :H * hd].view(B, Tq, H, hd)
    pre = normal(g, 2, P, Hkv, hd)
    own = normal(g, 2, B, S, Hkv, hd)
    kp, vp = (pre[i].transpose(0, 1) for i in (0, 1))
    k, v = (own[i].transpose(1, 2) for i in (0, 1))
    lens, qn = [70, 2, 33] * (B // 3), [2, 1, 2] * (B // 3)
    want, _ = check_attention(q, kp, vp, k, v, lens, qn)
    wide = torch.full((B, Tq, H, 2 * hd), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[..., :hd] = 7.0
    fl.prefix_attention(q, kp, vp, k, v, ints(lens), q_lens=ints(qn), out=wide[..., :hd])
    assert torch.equal(wide[..., :hd], want) and bool((wide[..., hd:] == 3.0).all())


@pytest.mark.parametrize("B,P", [(2, 70), (16, 12007)])
def test_attention_ignores_what_masked_rows_hold(B, P):
    """NaN and infinities past a sequence's length, and in tokens that only later queries see."""
    g = gen(5)
    Tq, H, Hkv, hd, S = 4, 4, 2, 128, 80
    q, kp, vp = normal(g, B, Tq, H, hd), normal(g, Hkv, P, hd), normal(g, Hkv, P, hd)
    k, v = normal(g, B, Hkv, S, hd), normal(g, B, Hkv, S, hd)
    lens, qn = [50, 33] * (B // 2), [4, 3] * (B // 2)
    clean, clse = check_attention(q, kp, vp, k, v, lens, qn)
    for b in range(B):
        k[b, :, lens[b]:] = NAN
        v[b, :, lens[b]:] = INF
        k[b, :, lens[b] - 1] = NAN      # the last token: the last query's alone
        v[b, :, lens[b] - 1] = -INF
    out, lse = fl.prefix_attention(q, kp, vp, k, v, ints(lens), q_lens=ints(qn))
    for b in range(B):
        n = qn[b]
        assert torch.equal(out[b, :n - 1], clean[b, :n - 1]) and torch.equal(lse[b, :n - 1], clse[b, :n - 1])
        assert bool(torch.isnan(out[b, n - 1].float()).all())


def test_attention_non_finite_scores():
    """A visible NaN makes its rows NaN; a column of -inf score weighs nothing; no finite score at all: 0 and -inf."""
    g = gen(6)
    q = normal(g, 1, 1, 2, 64).abs()
    kp, vp = normal(g, 2, 40, 64), normal(g, 2, 40, 64)
    kp[0, 7] = NAN
    kp[1, 5] = -INF                      # q > 0: score -inf
    out, lse = fl.prefix_attention(q, kp, vp, None, None, None)
    assert bool(torch.isnan(out[0, 0, 0].float()).all()) and math.isnan(float(lse[0, 0, 0]))
    keep = [i for i in range(40) if i != 5]
    want, wl = fl.prefix_attention(q, kp[:, keep].contiguous(), vp[:, keep].contiguous(), None, None, None)
    assert torch.allclose(out[0, 0, 1].float(), want[0, 0, 1].float(), rtol=2 ** -7, atol=2 ** -7)
    kp[1] = -INF
    out, lse = fl.prefix_attention(q, kp, vp, None, None, None)
    assert bool((out[0, 0, 1] == 0).all()) and float(lse[0, 0, 1]) == -INF


@pytest.mark.parametrize("B,P", [(3, 40), (24, 31007)])
def test_attention_clamps_bad_lengths(B, P):
    g = gen(7)
    q, kp, vp = normal(g, B, 2, 4, 64), normal(g, 2, P, 64), normal(g, 2, P, 64)
    k, v = normal(g, B, 2, 24, 64), normal(g, B, 2, 24, 64)
    n = B // 3
    a, al = fl.prefix_attention(q, kp, vp, k, v, ints([24, 0, 24] * n), q_lens=ints([2, 2, 0] * n))
    b, bl = fl.prefix_attention(q, kp, vp, k, v, ints([1000000, -5, 24] * n), q_lens=ints([77, 2, -3] * n))
    assert torch.equal(a, b) and torch.equal(al, bl)


@pytest.mark.parametrize("B,P", [(4, 3000), (24, 8001)])
def test_attention_streams_graphs_and_scratch(B, P):
    """The same bits on another stream, replayed from a graph with new inputs, and with a dirty scratch buffer."""
    g = gen(8)
    Tq, H, Hkv, hd, S = 2, 8, 2, 128, 500
    q, kp, vp = normal(g, B, Tq, H, hd), normal(g, Hkv, P, hd), normal(g, Hkv, P, hd)
    k, v, lens = normal(g, B, Hkv, S, hd), normal(g, B, Hkv, S, hd), ints([500, 2, 77, 300] * (B // 4))
    want, wl = fl.prefix_attention(q, kp, vp, k, v, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = fl.prefix_attention(q, kp, vp, k, v, lens, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    n = fl.prefix_attention_scratch_bytes(B, Tq, H, Hkv, hd, P, S)
    scratch = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    o2, l2 = torch.empty_like(want), torch.empty_like(wl)
    q2 = q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fl.prefix_attention(q2, kp, vp, k, v, lens, out=o2, lse=l2, scratch=scratch)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, want) and torch.equal(l2, wl)
    q2.copy_(normal(g, B, Tq, H, hd))
    lens.copy_(ints([3, 500, 9, 2] * (B // 4)))
    graph.replay()
    want, wl = fl.prefix_attention(q2, kp, vp, k, v, lens)
    torch.cuda.synchronize()
    assert torch.equal(o2, want) and torch.equal(l2, wl)


# ---------------------------------------------------------------------------- column weights
CW = [
    # B, Tq, H, Hkv, hd, S, lens, q_lens
    (1, 1, 1, 1, 64, 1, None, None),
    (2, 1, 4, 4, 64, 200, [200, 7], None),
    (3, 3, 10, 2, 128, 300, [300, 3, 129], [3, 1, 2]),
    (1, 37, 6, 2, 128, 257, None, None),
    (1, 70, 4, 1, 64, 500, [500], [70]),
    (2, 130, 8, 2, 128, 140, [130, 140], [130, 130]),
    (2, 20, 3, 1, 128, 128, [128, 0], [20, 20]),
    (1, 300, 8, 1, 128, 1025, None, None),
    (2, 600, 2, 1, 64, 900, [900, 650], [600, 599]),
    (1, 40, 5, 1, 128, 33, [33], [40]),
    (3, 9, 4, 1, 64, 131, [131, 60, 9], [9, 0, 9]),
    (1, 2, 64, 1, 128, 400, None, None),
    (1, 700, 3, 1, 64, 260, None, None),
    (5, 4, 4, 2, 128, 33, [33, 1, 0, 32, 7], [4, 4, 4, 2, 1]),
]


@pytest.mark.parametrize("case", CW, ids=[f"{c[0]}x{c[1]}h{c[2]}_{c[3]}d{c[4]}s{c[5]}" for c in CW])
def test_column_weights_against_64_bits(case):
    B, Tq, H, Hkv, hd, S, lens, q_lens = case
    g = gen(S + Tq)
    q, k = normal(g, B, Tq, H, hd, scale=2.0), normal(g, B, Hkv, S, hd)
    lse = math.log(S) + 1.0 + torch.rand((B, Tq, H), generator=g, device="cuda")
    lse[0, 0, 0] = -INF
    acc = torch.rand((B, Hkv, S), generator=g, device="cuda")
    ln, qn = None if lens is None else ints(lens), None if q_lens is None else ints(q_lens)
    out = fl.column_weights(q, k, lse, acc, lens=ln, q_lens=qn)
    want, tol = ref.column_weights(ref.f64(q), ref.f64(k), lse.double().cpu().numpy(), acc.double().cpu().numpy(), lens,
                                   q_lens, hd ** -0.5)
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
    inplace = acc.clone()
    assert fl.column_weights(q, k, lse, inplace, lens=ln, q_lens=qn, out=inplace) is inplace
    assert torch.equal(inplace, out)


def test_column_weights_ignore_masked_rows():
    g = gen(11)
    q, k = normal(g, 2, 3, 4, 128), normal(g, 2, 2, 150, 128)
    lse, acc = torch.full((2, 3, 4), 5.0, device="cuda"), torch.zeros((2, 2, 150), device="cuda")
    lens = ints([140, 60])
    want = fl.column_weights(q, k, lse, acc, lens=lens)
    for b, n in enumerate((140, 60)):
        k[b, :, n:] = NAN
    got = fl.column_weights(q, k, lse, acc, lens=lens)
    assert torch.equal(got, want) and bool((got[1, :, 60:] == 0).all())


def test_column_weights_nan_lse_reaches_every_column_it_weighs():
    """A query whose lse is NaN makes the columns it sees NaN, and no other: few rows and many."""
    for Tq in (3, 40):
        g = gen(13)
        q, k = normal(g, 1, Tq, 4, 64), normal(g, 1, 2, 100, 64)
        lse = torch.full((1, Tq, 4), 5.0, device="cuda")
        lse[0, 1, 2] = NAN                       # KV head 1; sees columns 0 .. 100 - Tq + 1
        lse[0, 0, 0] = -INF
        out = fl.column_weights(q, k, lse, torch.zeros((1, 2, 100), device="cuda"), lens=ints([100]))
        seen = 100 - Tq + 2
        assert bool(torch.isfinite(out[0, 0]).all())
        assert bool(torch.isnan(out[0, 1, :seen]).all()) and bool(torch.isfinite(out[0, 1, seen:]).all())


def test_column_weights_sum_to_the_queries():
    """With the attention's own lse the weights of all columns sum to the number of (query, head) pairs
    of the group: each row's weights sum to 1 within the fp32 error of lse and the weights."""
    g = gen(12)
    B, Tq, H, Hkv, hd, P, S = 3, 4, 8, 2, 128, 700, 90
    q, kp, vp = normal(g, B, Tq, H, hd), normal(g, Hkv, P, hd), normal(g, Hkv, P, hd)
    k, v, lens = normal(g, B, Hkv, S, hd), normal(g, B, Hkv, S, hd), ints([90, 4, 31])
    _, lse = fl.prefix_attention(q, kp, vp, k, v, lens)
    wp = fl.column_weights(q.view(1, B * Tq, H, hd), kp[None], lse.view(1, B * Tq, H),
                           torch.zeros((1, Hkv, P), device="cuda"))
    ws = fl.column_weights(q, k, lse, torch.zeros((B, Hkv, S), device="cuda"), lens=lens)
    total = wp.sum() + ws.sum()
    assert abs(float(total) - B * Tq * H) <= 1e-4 * B * Tq * H


# ---------------------------------------------------------------------------- eviction
def evict_inputs(g, B, Hkv, S, hd, ties):
    k, v = normal(g, B, Hkv, S, hd), normal(g, B, Hkv, S, hd)
    acc = torch.rand((B, Hkv, S), generator=g, device="cuda") ** 3
    if ties:
        acc = torch.floor(acc * 4)
    pos = torch.argsort(torch.rand((B, Hkv, S), generator=g, device="cuda"), dim=-1).to(torch.int32)
    return k, v, acc, pos


EV = [
    # B, Hkv, S, hd, lens, keep, recent, sinks, ties
    (1, 1, 1, 64, [1], 1, 0, 0, False),
    (1, 1, 2, 64, [2], 1, 0, 0, False),
    (2, 2, 40, 64, [40, 11], 10, 3, 2, False),
    (3, 2, 100, 128, [100, 0, 60], 60, 0, 0, True),
    (2, 1, 513, 128, [513, 512], 512, 64, 4, True),
    (2, 3, 5000, 128, [5000, 4097], 300, 200, 4, False),
    (1, 2, 9000, 64, [8999], 8000, 7000, 1000, True),
    (1, 1, 70001, 64, [70001], 1, 1, 0, True),
    (1, 1, 33000, 64, [33000], 32999, 5, 5, True),
    (2, 1, 64, 200, [64, 64], 100, 10, 0, False),
    (1, 1, 262144, 8, [262143], 5000, 10, 1, True),
]


@pytest.mark.parametrize("case", EV, ids=[f"{c[0]}x{c[1]}s{c[2]}k{c[5]}" for c in EV])
def test_evict_against_its_definition(case):
    B, Hkv, S, hd, lens, keep, recent, sinks, ties = case
    k, v, acc, pos = evict_inputs(gen(S + keep), B, Hkv, S, hd, ties)
    ln = ints(lens)
    want = ref.evict(acc.cpu().numpy(), pos.cpu().numpy(), lens, keep, recent, sinks)
    out = (torch.full((B, Hkv, keep, hd), 5.0, dtype=torch.bfloat16, device="cuda"),
           torch.full((B, Hkv, keep, hd), 5.0, dtype=torch.bfloat16, device="cuda"),
           torch.full((B, Hkv, keep), 5.0, device="cuda"), torch.full((B, Hkv, keep), 5, dtype=torch.int32, device="cuda"),
           torch.zeros(B, dtype=torch.int32, device="cuda"))
    fl.evict(k, v, acc, pos, ln, keep, recent=recent, sinks=sinks, out=out)
    held = [t.clone() for t in (k, v, acc, pos, ln)]
    fl.evict(*held, keep, recent=recent, sinks=sinks)
    torch.cuda.synchronize()
    assert out[4].tolist() == [min(n, keep) for n in lens] == held[4].tolist()
    for b in range(B):
        for h in range(Hkv):
            idx = torch.tensor(want[b][h], dtype=torch.long, device="cuda")
            n = len(idx)
            for got, kept, src in zip(out[:4], held[:4], (k, v, acc, pos)):
                assert torch.equal(got[b, h, :n], src[b, h][idx])
                assert bool((got[b, h, n:] == 5).all())            # slots from the new length on: untouched
                assert torch.equal(kept[b, h, :n], src[b, h][idx])
                assert torch.equal(kept[b, h, n:], src[b, h, n:])


def test_evict_protects_and_orders():
    """Protected tokens stay whatever their weight; equal weights keep the lower slot; inf and NaN weights
    rank by their bits (NaN above inf)."""
    k = torch.arange(8, dtype=torch.bfloat16, device="cuda").view(1, 1, 8, 1).expand(1, 1, 8, 8).contiguous()
    acc = torch.tensor([[[0.0, 1.0, 1.0, NAN, INF, 1.0, 0.5, 0.0]]], device="cuda")
    pos = ints([[[0, 6, 7, 8, 9, 10, 11, 12]]])
    o = fl.evict(k.clone(), k.clone(), acc.clone(), pos.clone(), ints([8]), 4, recent=1, sinks=1)
    # kept: slots 0 (pos < 1) and 7 (newest), then 3 (NaN), 4 (inf); holes 1, 2 take 4, 7
    assert o[3][0, 0, :4].tolist() == [0, 9, 12, 8] and o[4].tolist() == [4]
    o = fl.evict(k.clone(), k.clone(), torch.ones_like(acc), pos.clone(), ints([8]), 5)
    assert o[3][0, 0, :5].tolist() == [0, 6, 7, 8, 9]


def test_evict_strided_cache_and_graph():
    """A [B][S][Hkv][hd] cache compacted in place inside a graph, replayed after the lengths grew again."""
    g = gen(21)
    B, S, Hkv, hd, keep = 2, 300, 3, 64, 200
    kv = normal(g, 2, B, S, Hkv, hd)
    k, v = kv[0].transpose(1, 2), kv[1].transpose(1, 2)
    acc = torch.rand((B, Hkv, S), generator=g, device="cuda")
    pos = torch.arange(S, dtype=torch.int32, device="cuda").expand(B, Hkv, S).contiguous()
    lens = ints([300, 250])
    scratch = torch.full((fl.evict_scratch_bytes(B, Hkv, S, keep),), 77, dtype=torch.uint8, device="cuda")
    first = [t.clone() for t in (k, v, acc, pos)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fl.evict(k, v, acc, pos, lens, keep, recent=10, scratch=scratch)
    for step in range(2):
        before = [t.clone() for t in (k, v, acc, pos)]
        n = lens.tolist()
        graph.replay()
        torch.cuda.synchronize()
        want = ref.evict(before[2].cpu().numpy(), before[3].cpu().numpy(), n, keep, 10, 0)
        for b in range(B):
            for h in range(Hkv):
                idx = torch.tensor(want[b][h], dtype=torch.long, device="cuda")
                for now, was in zip((k, v, acc, pos), before):
                    assert torch.equal(now[b, h, :len(idx)], was[b, h][idx])
        lens += 60
        pos[:, :, 200:] += 1000
    assert not torch.equal(first[0], k)


# ---------------------------------------------------------------------------- draft verification
VD = [
    # B, D, V, temperature, n_draft, with draft logits
    (1, 1, 1, 1.0, None, True),
    (3, 2, 5, 1.0, [2, 1, 0], True),
    (4, 4, 1000, 0.7, [4, 3, 0, 1], True),
    (8, 3, 32000, 1.0, None, True),
    (2, 8, 32001, 1.3, [8, 5], True),
    (5, 3, 8189, 1.0, None, False),
    (3, 1, 131071, 0.5, None, True),
    (6, 5, 3001, 0.0, [5, 4, 3, 2, 1, 0], True),
    (16, 0, 700, 1.0, None, True),
    (2, 64, 300, 2.0, None, True),
    (32, 4, 50, 1.0, None, True),
    (2, 2, 300007, 1.0, None, True),
    (300, 1, 2100, 0.9, None, True),
    (24, 4, 100003, 1.0, [4, 3, 2, 1, 0, 4] * 4, True),
    (40, 5, 100001, 0.8, None, False),
    (6, 64, 30011, 1.0, None, True),
    (5, 2, 900, 1e-9, None, True),
]


def verify_inputs(seed, B, D, V, T):
    g = gen(seed)
    logits = 3.0 * torch.randn((B, D + 1, V), generator=g, device="cuda")
    dl = logits[:, :D] + 0.7 * torch.randn((B, D, V), generator=g, device="cuda")
    noise = -torch.log(-torch.log(torch.rand((B, D, V), generator=g, device="cuda").clamp(1e-6, 1 - 1e-6)))
    draft = (torch.argmax(dl / max(T, 1e-2) + noise, -1) if D else torch.zeros((B, 0), device="cuda")).to(torch.int32)
    return logits, dl, draft, torch.rand((B, D + 1), generator=g, device="cuda")


def check_verify(logits, dl, draft, u, n_draft, T):
    nd = None if n_draft is None else ints(n_draft)
    tok, acc = fl.verify_draft(logits, dl, draft, u, n_draft=nd, temperature=T)
    torch.cuda.synchronize()
    wt, wa = ref.verify(logits.cpu().numpy(), None if dl is None else dl.cpu().numpy(), draft.cpu().numpy(),
                        u.cpu().numpy(), n_draft, T)
    assert np.array_equal(acc.cpu().numpy(), wa) and np.array_equal(tok.cpu().numpy(), wt)
    return wt, wa


@pytest.mark.parametrize("case", VD, ids=[f"{c[0]}x{c[1]}v{c[2]}t{c[3]}" for c in VD])
def test_verify_against_64_bits(case):
    B, D, V, T, n_draft, with_draft = case
    for seed in range(4 if B * D * V < 10 ** 6 else 1):
        logits, dl, draft, u = verify_inputs(seed * 100 + V, B, D, V, T)
        check_verify(logits, dl if with_draft else None, draft, u, n_draft, T)


def test_verify_large_calls_skip_only_what_decides_nothing():
    """A call large enough to stop at rejections, repeated into a dirty scratch buffer and replayed: the same tokens each
    time; drafts taken from the target's own most likely tokens, so that long runs are accepted."""
    B, D, V = 32, 8, 40009
    logits, _, _, u = verify_inputs(31, B, D, V, 1.0)
    draft = logits[:, :D].argmax(-1).to(torch.int32)
    dl = logits[:, :D] - 0.2 * torch.rand((B, D, 1), generator=gen(3), device="cuda")
    dl.scatter_add_(2, draft.long()[..., None], torch.full((B, D, 1), 0.1, device="cuda"))
    wt, wa = check_verify(logits, dl, draft, u, None, 1.0)
    assert wa.max() == D and wa.min() < D
    scratch = torch.full((fl.verify_draft_scratch_bytes(B, D, V),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        tok, acc = fl.verify_draft(logits, dl, draft, u, scratch=scratch)
        assert np.array_equal(tok.cpu().numpy(), wt) and np.array_equal(acc.cpu().numpy(), wa)


def test_verify_large_calls_stop_at_rejections():
    """The same beyond the size from which rows behind a rejection are not read (350 MB of logits), with unequal draft
    counts, and without draft probabilities."""
    B, D, V = 24, 8, 230003
    g = gen(41)
    logits = 3.0 * torch.randn((B, D + 1, V), generator=g, device="cuda")
    draft = logits[:, :D].argmax(-1).to(torch.int32)
    dl = logits[:, :D] - 0.2 * torch.rand((B, D, 1), generator=g, device="cuda")
    dl.scatter_add_(2, draft.long()[..., None], torch.full((B, D, 1), 0.1, device="cuda"))
    u = torch.rand((B, D + 1), generator=g, device="cuda")
    n_draft = ints([D, 0, 3, 1] * (B // 4))
    scratch = torch.full((fl.verify_draft_scratch_bytes(B, D, V),), 255, dtype=torch.uint8, device="cuda")
    wt, wa = check_verify(logits, dl, draft, u, n_draft, 1.0)
    for _ in range(3):
        tok, acc = fl.verify_draft(logits, dl, draft, u, n_draft=n_draft, scratch=scratch)
        assert np.array_equal(tok.cpu().numpy(), wt) and np.array_equal(acc.cpu().numpy(), wa)
    logits = torch.cat([logits, logits], 1)[:, :D + 1 + 5].contiguous()   # 13 drafts of one row of logits each
    draft = torch.cat([draft, draft], 1)[:, :D + 5].contiguous()
    check_verify(logits, None, draft, torch.rand((B, D + 6), generator=g, device="cuda") ** 8, None, 0.3)


def test_verify_border_random_numbers():
    """u at 0 and at the largest fp32 below 1, for the decisions and for the sampled token."""
    for value in (0.0, 1.0 - 2.0 ** -24):
        logits, dl, draft, u = verify_inputs(5, 6, 3, 777, 1.0)
        check_verify(logits, dl, draft, torch.full_like(u, value), None, 1.0)


def test_verify_decisions_on_the_border():
    """u within a few fp32 steps of p / q: the 64-bit sums decide."""
    logits, dl, draft, u = verify_inputs(9, 32, 1, 4001, 1.0)
    p = torch.softmax(logits.double(), -1)[:, 0].gather(1, draft.long())
    q = torch.softmax(dl.double(), -1)[:, 0].gather(1, draft.long())
    ratio = (p / q).float().clamp(max=1 - 2.0 ** -24)
    steps = torch.arange(-16, 16, device="cuda")[:, None] * 2.0 ** -24
    u[:, :1] = (ratio * (1 + steps)).clamp(0, 1 - 2.0 ** -24)
    check_verify(logits, dl, draft, u, None, 1.0)


def test_verify_equal_distributions_accept_everything():
    logits, _, draft, u = verify_inputs(10, 8, 4, 500, 1.0)
    _, acc = check_verify(logits, logits[:, :4].contiguous(), draft, u, None, 1.0)
    assert (acc == 4).all()


def test_verify_masked_vocabulary_and_bad_tokens():
    """-inf logits are never sampled; a draft token out of range, or of probability 0, is rejected."""
    logits, dl, draft, u = verify_inputs(11, 8, 2, 600, 1.0)
    logits[:, :, 300:] = -INF
    dl[:, :, :10] = -INF
    draft[0, 0], draft[1, 0], draft[2, 0], draft[3, 1] = -1, 600, 450, 2 ** 31 - 1
    wt, wa = check_verify(logits, dl, draft, u, None, 1.0)
    assert wa[0] == wa[1] == wa[2] == 0 and wt.max() < 300
    check_verify(logits, None, draft, u, None, 1.0)


def test_verify_rows_without_a_distribution():
    """NaN, +inf or no finite logit in the deciding row: token -1, the count still right; a NaN in a row that
    decides nothing changes nothing."""
    logits, dl, draft, u = verify_inputs(12, 4, 2, 300, 1.0)
    clean_t, clean_a = fl.verify_draft(logits, dl, draft, u)
    bad = logits.clone()
    for b in range(4):
        bad[b, int(clean_a[b])] = NAN
    tok, acc = fl.verify_draft(bad, dl, draft, u)
    for b in range(4):
        m = int(clean_a[b])
        assert int(acc[b]) == m and int(tok[b, m]) == -1 and torch.equal(tok[b, :m], clean_t[b, :m])
    for fill in (INF, -INF):
        bad = logits[:, :1].clone()
        bad[0, 0, 3] = fill
        if fill < 0:
            bad[0] = fill
        tok, acc = fl.verify_draft(bad, None, torch.empty((4, 0), dtype=torch.int32, device="cuda"), u[:, :1].contiguous())
        assert int(tok[0, 0]) == -1 and bool((tok[1:] >= 0).all())
    late = logits.clone()
    late[:, 2] = NAN
    tok, acc = fl.verify_draft(late, dl, draft, u)
    for b in range(4):
        if int(clean_a[b]) < 2:
            assert torch.equal(tok[b], clean_t[b])


def test_verify_greedy_ties_and_nan():
    logits = torch.zeros((1, 2, 20000), device="cuda")
    logits[0, 0, [19000, 12000, 700]] = 4.0
    logits[0, 1, 5] = NAN
    logits[0, 1, [9000, 100]] = 1.0
    tok, acc = fl.verify_draft(logits, None, ints([[700]]), None, temperature=0.0)
    assert tok.tolist() == [[700, 100]] and acc.tolist() == [1]
    tok, acc = fl.verify_draft(logits, None, ints([[12000]]), None, temperature=0.0)
    assert tok.tolist() == [[700, -1]] and acc.tolist() == [0]


def test_verify_strided_logits_streams_and_graph():
    """Rows of a padded vocabulary (any alignment), another stream, and a replayed graph."""
    B, D, V = 3, 3, 1013
    logits, dl, draft, u = verify_inputs(13, B, D, V, 1.0)
    want = fl.verify_draft(logits, dl, draft, u)
    wide = torch.full((B, D + 1, V + 6), NAN, device="cuda")
    wide[..., 3:V + 3] = logits
    got = fl.verify_draft(wide[..., 3:V + 3], dl, draft, u)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fl.verify_draft(logits, dl, draft, u, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    scratch = torch.full((fl.verify_draft_scratch_bytes(B, D, V),), 255, dtype=torch.uint8, device="cuda")
    tok, acc = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fl.verify_draft(logits, dl, draft, u, tokens=tok, n_accepted=acc, scratch=scratch)
    for seed in (13, 14, 15):
        l2, d2, x2, u2 = verify_inputs(seed, B, D, V, 1.0)
        logits.copy_(l2), dl.copy_(d2), draft.copy_(x2), u.copy_(u2)
        graph.replay()
        torch.cuda.synchronize()
        wt, wa = ref.verify(l2.cpu().numpy(), d2.cpu().numpy(), x2.cpu().numpy(), u2.cpu().numpy(), None, 1.0)
        assert np.array_equal(tok.cpu().numpy(), wt) and np.array_equal(acc.cpu().numpy(), wa)


@pytest.mark.parametrize("V", [17, 4099, 40000])
def test_verify_writes_a_token_where_target_and_draft_differ_by_roundings(V):
    """A draft token outside the vocabulary is rejected; what is left of the target's row after the draft's is then
    nothing but roundings.  Whether that counts as empty (-1) or gives some token, one of the two is written."""
    B, D = 8, 2
    g = gen(V)
    x = torch.randn((B, D + 1, V), device="cuda", generator=g) * 3
    q = x[:, :D].clone()
    q[1::2] += 0.75   # the same distribution up to the rounding of the sums
    tokens = torch.full((B, D + 1), 12345678, dtype=torch.int32, device="cuda")
    draft = torch.full((B, D), V, dtype=torch.int32, device="cuda")
    got, n = fl.verify_draft(x, q, draft, torch.rand((B, D + 1), device="cuda", generator=g), tokens=tokens)
    assert (n == 0).all()
    assert ((got[:, 0] >= -1) & (got[:, 0] < V)).all() and (got[:, 1:] == -1).all()
    assert (got[0::2, 0] == -1).all()   # equal rows: exactly nothing is left


# ---------------------------------------------------------------------------- long strides
@pytest.fixture(scope="module")
def far():
    """A bf16 buffer whose second part starts past 2^31 elements (2^32 bytes)."""
    gap = 2 ** 31 + 4096
    buf = torch.empty(gap + 2 ** 22, dtype=torch.bfloat16, device="cuda")
    yield lambda x, dim: far_copy(buf, gap, x, dim)
    del buf
    torch.cuda.empty_cache()


def far_copy(buf, gap, x, dim):
    """x (two elements long in `dim`) with that dimension's stride past 2^31."""
    assert x.shape[dim] == 2
    strides = list(x.select(dim, 0).contiguous().stride())
    strides.insert(dim, gap)
    y = buf.as_strided(x.shape, strides)
    y.copy_(x)
    return y


@pytest.mark.parametrize("B,P", [(3, 200), (40, 9473)])
def test_attention_offsets_past_32_bits(far, B, P):
    """KV heads further apart than 2^31 elements, for either kernel of the prefix: the bits of adjacent ones."""
    g = gen(51)
    q, kp, vp = normal(g, B, 2, 8, 128), normal(g, 2, P, 128), normal(g, 2, P, 128)
    k, v, lens = normal(g, B, 2, 70, 128), normal(g, B, 2, 70, 128), ints([70 - 2 * (i % 30) for i in range(B)])
    want, wl = fl.prefix_attention(q, kp, vp, k, v, lens)
    for i, x in enumerate((kp, vp)):
        got, gl = fl.prefix_attention(q, *[far(y, 0) if j == i else y for j, y in enumerate((kp, vp))], k, v, lens)
        assert torch.equal(got, want) and torch.equal(gl, wl)
    for i in range(2):
        got, gl = fl.prefix_attention(q, kp, vp, *[far(y, 1) if j == i else y for j, y in enumerate((k, v))], lens)
        assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("Tq", [1, 40])
def test_column_weights_offsets_past_32_bits(far, Tq):
    g = gen(52)
    q, k = normal(g, 2, Tq, 8, 64), normal(g, 2, 2, 700, 64)
    lse, acc, lens = torch.full((2, Tq, 8), 7.0, device="cuda"), torch.rand((2, 2, 700), device="cuda"), ints([700, 333])
    want = fl.column_weights(q, k, lse, acc, lens=lens)
    assert torch.equal(fl.column_weights(q, far(k, 0), lse, acc, lens=lens), want)
    assert torch.equal(fl.column_weights(far(q, 0), k, lse, acc, lens=lens), want)


def test_evict_offsets_past_32_bits(far):
    g = gen(53)
    B, Hkv, S, hd, keep = 2, 2, 900, 64, 500
    k, v, acc, pos = evict_inputs(g, B, Hkv, S, hd, False)
    lens = ints([900, 777])
    want = fl.evict(*[x.clone() for x in (k, v, acc, pos, lens)], keep, recent=9, sinks=2)
    y = far(k, 0)
    got = fl.evict(y, v.clone(), acc.clone(), pos.clone(), lens.clone(), keep, recent=9, sinks=2)   # in place
    for a, b in zip(got, want):
        assert torch.equal(a[:, :, :keep] if a.dim() > 1 else a, b[:, :, :keep] if b.dim() > 1 else b)
    y = far(v, 0)
    out = (torch.empty_like(k[:, :, :keep].contiguous()), torch.empty_like(k[:, :, :keep].contiguous()),
           torch.empty((B, Hkv, keep), device="cuda"), torch.empty((B, Hkv, keep), dtype=torch.int32, device="cuda"),
           torch.empty_like(lens))
    for a, b in zip(fl.evict(k, y, acc, pos, lens, keep, recent=9, sinks=2, out=out), want):
        assert torch.equal(a, b[:, :, :keep] if b.dim() > 1 else b)


def test_verify_offsets_past_32_bits():
    gap = 2 ** 31 + 4097
    buf = torch.empty(gap + 10 ** 6, device="cuda")
    logits, dl, draft, u = verify_inputs(54, 2, 3, 5003, 1.0)
    want = fl.verify_draft(logits, dl, draft, u)
    for which in range(2):
        x = (logits, dl)[which]
        y = buf.as_strided(x.shape, (gap, 5003, 1))
        y.copy_(x)
        got = fl.verify_draft(y if which == 0 else logits, y if which == 1 else dl, draft, u)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = buf.as_strided(logits.shape, (gap, 5003, 1))
    y.copy_(logits)
    greedy = fl.verify_draft(logits, None, draft, None, temperature=0.0)
    assert all(torch.equal(a, b) for a, b in zip(fl.verify_draft(y, None, draft, None, temperature=0.0), greedy))


# ---------------------------------------------------------------------------- calls side by side
def operator_calls(seed):
    """One call of each operator as call(scratch) -> outputs, and its scratch bytes; sizes that take each kernel."""
    g = gen(seed)
    calls = []
    for B, P in ((5, 300), (40, 9473)):   # warp tiles; tensor cores
        q, kp, vp = normal(g, B, 1, 16, 128), normal(g, 2, P, 128), normal(g, 2, P, 128)
        k, v, lens = normal(g, B, 2, 90, 128), normal(g, B, 2, 90, 128), ints([90 - i for i in range(B)])
        calls.append((lambda s, x=(q, kp, vp, k, v, lens): fl.prefix_attention(*x, scratch=s),
                      fl.prefix_attention_scratch_bytes(B, 1, 16, 2, 128, P, 90)))
    for Tq in (1, 60):
        q, k = normal(g, 2, Tq, 8, 128), normal(g, 2, 2, 3001, 128)
        lse, acc = torch.full((2, Tq, 8), 8.0, device="cuda"), torch.rand((2, 2, 3001), device="cuda", generator=g)
        calls.append((lambda s, x=(q, k, lse, acc): (fl.column_weights(*x, scratch=s),),
                      fl.column_weights_scratch_bytes(2, Tq, 8, 2, 128, 3001)))
    for S, keep in ((700, 600), (20000, 3001)):   # one CTA, a cluster
        k, v, acc, pos = evict_inputs(g, 2, 2, S, 64, True)
        lens = ints([S, S - 90])

        def evict(s, x=(k, v, acc, pos, lens), keep=keep):
            out = tuple(torch.zeros_like(t[:, :, :keep]) if t.dim() > 1 else torch.zeros_like(t) for t in x)
            return fl.evict(*x, keep, recent=5, sinks=1, out=out, scratch=s)
        calls.append((evict, fl.evict_scratch_bytes(2, 2, S, keep)))
    for B, D, V in ((3, 4, 5003), (24, 6, 300007)):   # every row; up to the first rejection
        x = verify_inputs(seed, B, D, V, 1.0)
        calls.append((lambda s, x=x: fl.verify_draft(*x, scratch=s), fl.verify_draft_scratch_bytes(B, D, V)))
    return calls


def test_calls_on_two_streams_at_once():
    """Every operator on two streams at the same time, each with its own scratch: the bits of calls made alone."""
    one, two = operator_calls(61), operator_calls(62)
    alone = [[f(None) for f, _ in calls] for calls in (one, two)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i, calls in enumerate((one, two)):
            with torch.cuda.stream(streams[i]):
                got[i].append([f(torch.empty(n, dtype=torch.uint8, device="cuda")) for f, n in calls])
    torch.cuda.synchronize()
    for i in range(2):
        for rep in got[i]:
            for a, b in zip(rep, alone[i]):
                assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_graphs_share_a_scratch_buffer():
    """Two captured sequences of all operators with one scratch buffer, replayed in turn."""
    both = [operator_calls(63), operator_calls(64)]
    alone = [[f(None) for f, _ in calls] for calls in both]
    scratch = torch.full((max(n for calls in both for _, n in calls),), 170, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for calls in both:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append([f(scratch) for f, _ in calls])
        graphs.append(graph)
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, alone):
        for x, y in zip(a, b):
            assert all(torch.equal(s, t) for s, t in zip(x, y))

