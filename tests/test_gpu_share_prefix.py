"""Decode steps of a batch whose sequences share a prefix: the context reads it once, and its
hidden states and logits stay within the oracle's tolerance; and the serving operators run
together as a sampling loop runs them."""
import numpy as np
import pytest
import torch

import e2e_common as E
import serving_ref as ref
from cross_loop_sparsity_b200 import flashloop as fl
from cross_loop_sparsity_b200 import synth

pytestmark = pytest.mark.gpu


def shared_context(cfg, rng, lens, n, dense):
    """A synthetic context whose sequences hold sequence 0's first n positions."""
    ctx = synth.make_dense_context(cfg, rng, lens) if dense else synth.make_context(cfg, rng, lens)
    for name, a in ctx.items():
        if name == "lens" or not isinstance(a, np.ndarray):
            continue
        seq = {"kv_k": 2, "kv_v": 2, "codes_k": 2, "codes_v": 2, "scales_k": 2, "scales_v": 2}.get(name, 1)
        a = np.moveaxis(a, (seq, seq + 2), (0, 1))      # [sequence][position]: a view
        a[1:, :n] = a[:1, :n]
    return ctx


def run(cfg, lens, n, dense, steps, share, forced=True, graph=1):
    from oracle import flashloop_oracle as orc
    if dense:
        cfg = cfg.with_(resid_bits=16)
    B = len(lens)
    w = synth.make_weights(cfg)
    rng = w["rng"]
    W = orc.prepare_weights(w)
    tmax = max(lens) + steps + 3
    ctx = shared_context(cfg, rng, lens, n, dense)
    cache = (orc.KVCache.from_dense_context if dense else orc.KVCache.from_context)(cfg, ctx, tmax)
    eng = fl.FlashLoop(cfg, fl.upload_weights(w), max_batch=B, max_ctx=tmax)
    eng.set_option(fl.FL_OPT_USE_GRAPH, graph)
    eng.load_context(ctx, dense)
    if share:
        eng.share_prefix(B, n)
    stream = torch.cuda.Stream()     # (steps on the legacy stream are not captured into graphs)
    out = []
    for _ in range(steps):
        h0 = synth.make_h0(cfg, rng, B)
        pos = cache.lens[:B].copy()
        r = orc.decode_step(cfg, W, cache, h0)
        if forced and not dense and cfg.n_loops > 1:
            eng.force_selection(*E.forced_arrays(cfg, r.trace, B), n_tiles=B)
            eng.force_codes(*E.forced_codes(cfg, cache, r.trace, np.arange(B), pos))
        h, lg = (torch.empty((B, k), dtype=torch.float32, device="cuda") for k in (cfg.d_model, cfg.vocab))
        x = torch.from_numpy(h0).cuda()
        torch.cuda.synchronize()
        eng.decode_step(x, B, h, lg, stream=stream)
        torch.cuda.synchronize()
        out.append((r, {"h": h.cpu().numpy(), "logits": lg.cpu().numpy(), "status": eng.sync_status(),
                        "launches": eng.kernels_per_call()}))
    return cfg, eng, out


CASES = [
    # block, head_dim-64 or 128, lengths, shared positions
    ("c1", [70, 65, 130], 65, False),
    ("c1", [70, 65, 130], 65, True),
    ("c2", [300, 257, 511, 256, 400], 256, False),
    ("c2", [300, 257, 511, 256, 400], 200, True),
]


@pytest.mark.parametrize("name,lens,n,dense", CASES)
def test_shared_decode_matches_the_oracle(name, lens, n, dense):
    cfg = synth.config(name).with_(n_layers=2, n_loops=3)
    _, eng, out = run(cfg, lens, n, dense, 3, True)
    E.check_all(out)
    eng.close()


def test_shared_decode_with_prelude_coda_and_last_loop():
    cfg = synth.config("c1").with_(n_layers=1, n_loops=2, n_prelude=1, n_coda=1)
    for c, dense in ((cfg, False), (cfg.with_(kv_mode=1), True)):
        _, eng, out = run(c, [90, 80], 70, dense, 2, True)
        E.check_all(out)
        eng.close()


def test_sharing_changes_only_the_order_of_sums_and_ends_when_told():
    """The dense baseline with and without sharing: within the order of fp32 sums of bf16 products (each side is within
    2e-2 of the oracle; the two differ far less).  Ending it restores the unshared bits."""
    cfg = synth.config("c2").with_(n_layers=1, n_loops=2)
    lens, n = [140, 133, 190], 130
    _, a, plain = run(cfg, lens, n, True, 1, False)
    _, b, shared = run(cfg, lens, n, True, 1, True)
    assert E.rel_err(shared[0][1]["h"], plain[0][1]["h"]) <= 4e-3
    assert shared[0][1]["launches"] > plain[0][1]["launches"]
    h0 = torch.randn((3, cfg.d_model), device="cuda")
    bufs = [torch.empty((3, cfg.d_model), device="cuda") for _ in range(2)]
    for eng, buf in ((a, bufs[0]), (b, bufs[1])):
        eng.reset(lens)
        if eng is b:
            eng.share_prefix(0, 0)
        eng.decode_step(h0, 3, buf)
        torch.cuda.synchronize()
    assert torch.equal(*bufs)
    # a reset below the shared length ends it too; a refused statement leaves things as they are
    b.reset(lens)
    b.share_prefix(3, n)
    b.reset([n - 1, n, n])
    b.reset(lens)
    b.decode_step(h0, 3, bufs[1])
    torch.cuda.synchronize()
    assert torch.equal(*bufs)
    for args in ((1, 5), (4, 5), (3, 10 ** 6), (3, 135), (3, -1)):   # (the second sequence holds 134 by now)
        with pytest.raises(fl.FlashLoopError):
            b.share_prefix(*args)
    b.reset(lens)
    b.decode_step(h0, 3, bufs[1])
    torch.cuda.synchronize()
    assert torch.equal(*bufs)


def test_shared_decode_replays_its_graph():
    """Direct launches and the captured graph (from the second step on) give the same bits, step after step."""
    cfg = synth.config("c2").with_(n_layers=1, n_loops=2)
    outs = []
    for graph in (1, 0):
        _, eng, out = run(cfg, [300, 280], 256, False, 4, True, forced=False, graph=graph)
        outs.append(out)
        eng.close()
    for (_, x), (_, y) in zip(*outs):
        assert x["status"] == y["status"] == 0
        assert np.array_equal(x["h"], y["h"]) and np.array_equal(x["logits"], y["logits"])


def test_operators_together():
    """Samples of one prompt: drafted tokens attend to the shared prefix and their own rows, every column's
    weight is summed, verification keeps some of the drafts, and caches over their budget are evicted,
    prefix included; each step against the 64-bit statements on the same state."""
    g = torch.Generator(device="cuda")
    g.manual_seed(77)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    B, D, H, Hkv, hd, V, P, S, keep_p, keep_s = 6, 3, 8, 2, 64, 500, 400, 48, 300, 32
    Tq = D + 1
    kp, vp = rnd(1, Hkv, P, hd).bfloat16(), rnd(1, Hkv, P, hd).bfloat16()
    acc_p = torch.zeros((1, Hkv, P), device="cuda")
    pos_p = torch.arange(P, dtype=torch.int32, device="cuda").expand(1, Hkv, P).contiguous()
    len_p = torch.tensor([P], dtype=torch.int32, device="cuda")
    k, v = torch.full((B, Hkv, S, hd), float("nan"), device="cuda").bfloat16(), torch.full((B, Hkv, S, hd), float("nan"), device="cuda").bfloat16()
    acc = torch.zeros((B, Hkv, S), device="cuda")
    pos = torch.zeros((B, Hkv, S), dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    seen = [0] * B
    out_w = rnd(H * hd, V) / 8
    for step in range(14):
        n_draft = torch.randint(0, D + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        q_lens = n_draft + 1
        q = (1.5 * rnd(B, Tq, H, hd)).bfloat16()
        for b in range(B):       # the new tokens' rows
            n, c = int(lens[b]), int(q_lens[b])
            k[b, :, n:n + c], v[b, :, n:n + c] = rnd(Hkv, c, hd).bfloat16(), rnd(Hkv, c, hd).bfloat16()
            acc[b, :, n:n + c] = 0
            pos[b, :, n:n + c] = torch.arange(seen[b], seen[b] + c, device="cuda")
        lens += q_lens
        np_now = int(len_p[0])
        kpn, vpn = kp[0, :, :np_now], vp[0, :, :np_now]
        out, lse = fl.prefix_attention(q, kpn, vpn, k, v, lens, q_lens=q_lens)
        clean = [ref.f64(torch.nan_to_num(t)) for t in (k, v)]
        want, wlse, tol, ltol = ref.attention(ref.f64(q), ref.f64(kpn), ref.f64(vpn), *clean, lens.tolist(),
                                              q_lens.tolist(), hd ** -0.5)
        for b in range(B):
            n = int(q_lens[b])
            assert np.all(np.abs(ref.f64(out)[b, :n] - want[b, :n]) <= tol[b, :n])
            assert np.all(np.abs(lse.double().cpu().numpy()[b, :n] - wlse[b, :n]) <= ltol[b, :n])
        before = acc.clone()
        fl.column_weights(q, k, lse, acc, lens=lens, q_lens=q_lens, out=acc)
        ww, wt = ref.column_weights(ref.f64(q), clean[0], lse.double().cpu().numpy(), before.double().cpu().numpy(),
                                    lens.tolist(), q_lens.tolist(), hd ** -0.5)
        assert np.all(np.abs(acc.double().cpu().numpy() - ww) <= wt)
        ap = acc_p[:, :, :np_now].contiguous()
        fl.column_weights(q.view(1, B * Tq, H, hd), kpn[None], lse.view(1, B * Tq, H), ap, out=ap)
        acc_p[:, :, :np_now] = ap
        logits = (out.float().reshape(B, Tq, H * hd) @ out_w).nan_to_num()
        dl = logits[:, :D] + 0.5 * rnd(B, D, V)
        draft = dl.argmax(-1).to(torch.int32)
        u = torch.rand((B, Tq), generator=g, device="cuda")
        tokens, n_acc = fl.verify_draft(logits, dl, draft, u, n_draft=n_draft)
        vt, va = ref.verify(logits.cpu().numpy(), dl.cpu().numpy(), draft.cpu().numpy(), u.cpu().numpy(),
                            n_draft.tolist(), 1.0)
        assert np.array_equal(tokens.cpu().numpy(), vt) and np.array_equal(n_acc.cpu().numpy(), va)
        lens -= n_draft - n_acc          # rejected drafts leave the cache
        for b in range(B):
            seen[b] += int(n_acc[b]) + 1
        if int(lens.max()) > keep_s:
            src = ref.evict(acc.cpu().numpy(), pos.cpu().numpy(), lens.tolist(), keep_s, 8, 2)
            old = [t.clone() for t in (k, v, acc, pos)]
            fl.evict(k, v, acc, pos, lens, keep_s, recent=8, sinks=2)
            for b in range(B):
                for h in range(Hkv):
                    idx = torch.tensor(src[b][h], device="cuda")
                    for now, was in zip((k, v, acc, pos), old):
                        assert torch.equal(now[b, h, :len(idx)], was[b, h][idx])
        if step == 6:                    # the shared prefix over its budget as well
            fl.evict(kp, vp, acc_p, pos_p, len_p, keep_p, sinks=4)
            assert int(len_p[0]) == keep_p
    assert int(lens.max()) <= S
