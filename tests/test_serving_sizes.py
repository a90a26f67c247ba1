"""Sizes and temperatures that 32 bits would turn into others are refused by the binding, on the host."""
import pytest
import torch

from cross_loop_sparsity_b200 import build as fl_build
from cross_loop_sparsity_b200 import flashloop as fl


@pytest.fixture(scope="module", autouse=True)
def built():
    fl_build.build()


def cache(S):
    k = torch.empty((1, 1, S, 8), dtype=torch.bfloat16, device="meta")
    return (k, k, torch.empty((1, 1, S), device="meta"), torch.empty((1, 1, S), dtype=torch.int32, device="meta"),
            torch.empty(1, dtype=torch.int32, device="meta"))


@pytest.mark.parametrize("sizes", [dict(keep=2 ** 32 + 4), dict(keep=4, recent=2 ** 32), dict(keep=4, sinks=2 ** 32 + 1),
                                   dict(keep=-2 ** 31 - 1)])
def test_evict_counts(sizes):
    name = next(n for n, x in sizes.items() if not -2 ** 31 <= x < 2 ** 31)
    with pytest.raises(fl.FlashLoopError, match=f"{name} = .* out of range"):
        fl.evict(*cache(16), **sizes)


def test_lengths():
    n = 2 ** 32 + 5                # (meta tensors: no memory)
    with pytest.raises(fl.FlashLoopError, match="S = .* out of range"):
        fl.evict(*cache(n), 4)
    with pytest.raises(fl.FlashLoopError, match="V = .* out of range"):
        fl.verify_draft(torch.empty((1, 1, n), device="meta"), None, None, None)
    q, k = (torch.empty((1, 1, s, 64), dtype=torch.bfloat16, device="meta") for s in (1, n))
    x = torch.empty((1, 1, n), device="meta")
    with pytest.raises(fl.FlashLoopError, match="S = .* out of range"):
        fl.column_weights(q, k, torch.empty((1, 1, 1), device="meta"), x)
    with pytest.raises(fl.FlashLoopError, match="P = .* out of range"):
        fl.prefix_attention(q, k[0], k[0], None, None, None)


@pytest.mark.parametrize("T", [1e-46, 1e-30, -1e-46, -1.0, float("nan")])
def test_temperatures(T):
    """1e-46 is 0 in 32 bits: greedy, which nobody asked for."""
    with pytest.raises(fl.FlashLoopError, match="temperature"):
        fl.verify_draft(torch.empty((1, 1, 9), device="meta"), None, None, None, temperature=T)


def test_scratch_figures():
    big = 2 ** 32 + 64
    assert fl.prefix_attention_scratch_bytes(1, 1, 4, 4, 64, 0, big) == 0
    assert fl.column_weights_scratch_bytes(1, 1, 4, 4, 64, big) == 0
    assert fl.evict_scratch_bytes(1, 1, big, 4) == 0 and fl.evict_scratch_bytes(1, 1, 64, big) == 0
    assert fl.verify_draft_scratch_bytes(1, big, 100) == 0


@pytest.mark.parametrize("args", [(2, 2 ** 32), (2 ** 32 + 2, 5), (2, -2 ** 31 - 1)])
def test_shared_positions(args):
    """2^32 positions are 0 in 32 bits, which ends sharing."""
    eng = fl.FlashLoop.__new__(fl.FlashLoop)
    with pytest.raises(fl.FlashLoopError, match="out of range"):
        eng.share_prefix(*args)
