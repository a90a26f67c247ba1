"""The serving operators' refusals and scratch figures, on the host: a refused call launches
nothing, so made-up aligned addresses stand for device buffers."""
import ctypes

import pytest

from cross_loop_sparsity_b200 import build as fl_build
from cross_loop_sparsity_b200 import flashloop as fl

PTR = 1 << 20   # 256-byte aligned; never read
INVALID, WORKSPACE = 1, 3


@pytest.fixture(scope="module")
def L():
    fl_build.build()
    return fl.lib()


def prefix(**kw):
    a = fl.PrefixArgs(PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, None, 2, 3, 8, 2, 128, 100, 50, 0.1,
                      fl._I3(3 * 1024, 1024, 128), fl._I3(3 * 1024, 1024, 128), fl._I2(12800, 128),
                      fl._I2(12800, 128), fl._I3(12800, 6400, 128), fl._I3(12800, 6400, 128))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def weights(**kw):
    a = fl.WeightsArgs(PTR, PTR, PTR, PTR, PTR, PTR, None, 2, 3, 8, 2, 128, 50, 0.1, fl._I3(3 * 1024, 1024, 128),
                       fl._I3(12800, 6400, 128))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def evict(**kw):
    a = fl.EvictArgs(*[PTR * (i + 1) for i in range(10)], 2, 2, 50, 128, 20, 4, 2, fl._I3(12800, 6400, 128),
                     fl._I3(12800, 6400, 128), fl._I2(100, 50), fl._I2(100, 50), fl._I3(5120, 2560, 128),
                     fl._I3(5120, 2560, 128), fl._I2(40, 20), fl._I2(40, 20))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def verify(**kw):
    a = fl.VerifyArgs(PTR, PTR, PTR, PTR, None, PTR, PTR, 2, 3, 100, 1.0, fl._I2(400, 100), fl._I2(300, 100))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


NAN, INF = float("nan"), float("inf")
BAD = {
    "prefix_attention": (prefix, [
        dict(B=0), dict(Tq=0), dict(Tq=65), dict(H=9), dict(Hkv=0), dict(H=130, Hkv=2), dict(hd=96), dict(P=-1),
        dict(S=-1), dict(scale=NAN), dict(scale=INF), dict(q=None), dict(q=PTR + 8), dict(out=None), dict(out=PTR + 2),
        dict(lse=PTR + 1), dict(k_prefix=None), dict(v_prefix=PTR + 4), dict(k=None), dict(v=PTR + 8), dict(lens=None),
        dict(q_stride=fl._I3(3 * 1024, 1023, 128)), dict(q_stride=fl._I3(0, 1024, 128)),
        dict(out_stride=fl._I3(3 * 1024, 1024, -128)), dict(kp_stride=fl._I2(12800, 4)),
        dict(v_stride=fl._I3(12800, 6400, 0)), dict(q_stride=fl._I3(1 << 34, 1024, 128)), dict(B=1 << 20, Tq=64, H=64, Hkv=1), dict(P=(1 << 30) + 1),
        dict(S=(1 << 30) + 1)]),
    "column_weights": (weights, [
        dict(B=0), dict(Tq=0), dict(H=9), dict(hd=32), dict(S=-1), dict(scale=INF), dict(q=None), dict(k=PTR + 8),
        dict(lse=None), dict(acc=None), dict(out=PTR + 2), dict(lens=PTR + 1), dict(k_stride=fl._I3(12800, 6400, 100)),
        dict(q_stride=fl._I3(-8, 1024, 128)), dict(S=2 ** 31 - 1)]),
    "evict": (evict, [
        dict(B=0), dict(Hkv=0), dict(S=0), dict(S=262145), dict(keep=0), dict(hd=12), dict(hd=2048), dict(recent=-1),
        dict(sinks=-1), dict(recent=19, sinks=2), dict(recent=2 ** 31 - 1, sinks=2 ** 31 - 1), dict(k=None),
        dict(v_out=PTR + 8), dict(acc=None), dict(pos=PTR + 2), dict(lens_out=None), dict(k_out=PTR),
        dict(k_stride=fl._I3(12800, 6400, 0)), dict(acc_stride=fl._I2(0, 50)),
        dict(k_out=PTR, v_out=PTR * 2, acc_out=PTR * 3, pos_out=PTR * 4, lens_out=PTR * 5)]),
    "verify_draft": (verify, [
        dict(B=0), dict(D=-1), dict(D=65), dict(V=0), dict(temperature=-0.5), dict(temperature=1e-30), dict(temperature=NAN),
        dict(temperature=INF), dict(logits=None), dict(draft=None), dict(u=None), dict(tokens=None),
        dict(n_accepted=PTR + 2), dict(logits=PTR + 1), dict(logits_stride=fl._I2(-400, 100)),
        dict(draft_logits_stride=fl._I2(300, 0))]),
}
CASES = [(op, i) for op, (_, bad) in BAD.items() for i in range(len(bad))]


@pytest.mark.parametrize("op,i", CASES, ids=[f"{op}-{i}" for op, i in CASES])
def test_refused_before_any_launch(L, op, i):
    make, bad = BAD[op]
    st = getattr(L, "flashloop_" + op)(ctypes.byref(make(**bad[i])), PTR, 1 << 40, None)
    assert st == INVALID, bad[i]
    assert L.flashloop_last_cuda_error(None)


@pytest.mark.parametrize("op", sorted(BAD))
def test_scratch_is_checked(L, op):
    fn, make = getattr(L, "flashloop_" + op), BAD[op][0]
    assert fn(None, PTR, 1 << 40, None) == INVALID
    for ptr, size in ((None, 1 << 40), (PTR + 128, 1 << 40), (PTR, 0)):
        assert fn(ctypes.byref(make()), ptr, size, None) == WORKSPACE
        assert b"scratch" in L.flashloop_last_cuda_error(None)


def test_scratch_figures(L):
    assert fl.prefix_attention_scratch_bytes(8, 1, 16, 4, 128, 4096, 256) > 0
    assert fl.column_weights_scratch_bytes(8, 1, 16, 4, 128, 256) > 0
    assert fl.evict_scratch_bytes(8, 4, 4160, 4096) >= 8 * 4 * 4096 * 4
    assert fl.verify_draft_scratch_bytes(64, 8, 131072) > 0
    for n in (fl.prefix_attention_scratch_bytes(8, 1, 16, 4, 96, 4096, 256),
              fl.prefix_attention_scratch_bytes(8, 1, 16, 3, 128, 4096, 256),
              fl.column_weights_scratch_bytes(0, 1, 16, 4, 128, 256), fl.evict_scratch_bytes(1, 1, 1 << 20, 5),
              fl.verify_draft_scratch_bytes(1, 65, 100)):
        assert n == 0


def test_binding_refuses_wrong_tensors():
    """dtype, shape, layout and device are checked before the library is called."""
    import torch
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(fl.FlashLoopError):   # not a cuda tensor
        fl.prefix_attention(q, torch.zeros((2, 9, 64), dtype=torch.bfloat16),
                            torch.zeros((2, 9, 64), dtype=torch.bfloat16), None, None, None)
    with pytest.raises(fl.FlashLoopError):
        fl.prefix_attention(q, None, None, None, None, None)
    with pytest.raises(fl.FlashLoopError):   # fp32 queries
        fl.column_weights(q.float(), q, q, q)
    with pytest.raises(fl.FlashLoopError):
        fl.evict(torch.zeros((1, 1, 4, 8)), q, q, q, q, 2)
    with pytest.raises(fl.FlashLoopError):
        fl.verify_draft(torch.zeros((2, 8)), None, None, None)
