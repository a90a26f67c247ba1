"""The serving operators around a decode step, as timed cases: attention over a
prefix that the whole batch shares, the attention weight of every key column,
eviction from a cache by that weight, and the verification of drafted tokens.

``run`` computes an operator in elementary torch operations where ``own`` is
false, and calls the library's entry point where it is true.  Both return the
whole result.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # two sequences of the smallest block's heads over a short common prompt: launch latency
        dict(name="prefix-small", op="prefix", B=2, Tq=1, H=4, Hkv=4, hd=64, P=128, S=32, ragged=False),
        # the 8 x 4096 decode step's heads, one new token each, a common prompt
        dict(name="prefix-step", op="prefix", B=8, Tq=1, H=16, Hkv=4, hd=128, P=4096, S=257, ragged=True),
        # many samples of one prompt, the deep block's heads, unequal continuations
        dict(name="prefix-samples", op="prefix", B=64, Tq=1, H=32, Hkv=8, hd=128, P=8192, S=1000, ragged=True),
        # drafted tokens of 32 samples checked at once over a long, odd prompt length
        dict(name="prefix-drafts", op="prefix", B=32, Tq=5, H=32, Hkv=8, hd=128, P=65531, S=300, ragged=True),
        # column weights of one decode step over each sequence's own cache
        dict(name="weights-step", op="weights", B=8, Tq=1, H=16, Hkv=4, hd=128, S=4097, causal=True),
        # column weights of a prompt's last 512 tokens over the whole prompt
        dict(name="weights-prompt", op="weights", B=1, Tq=512, H=16, Hkv=4, hd=128, S=16384, causal=True),
        # a cache slightly over its budget after a few steps, into the other of two buffers
        dict(name="evict-step", op="evict", B=8, Hkv=4, hd=128, S=4160, keep=4096, recent=64, sinks=4, ragged=False),
        # long prompts cut down to a decode budget
        dict(name="evict-prompt", op="evict", B=4, Hkv=8, hd=128, S=65536, keep=8192, recent=256, sinks=4, ragged=True),
        # one sequence, four drafted tokens
        dict(name="verify-one", op="verify", B=1, D=4, V=32000, temp=1.0, ragged=False),
        # a decode batch with unequal draft counts
        dict(name="verify-batch", op="verify", B=32, D=5, V=32000, temp=0.8, ragged=True),
        # a large batch over a large vocabulary
        dict(name="verify-large", op="verify", B=64, D=8, V=131071, temp=1.0, ragged=False),
        # greedy verification: argmax of every row
        dict(name="verify-greedy", op="verify", B=16, D=4, V=50001, temp=0.0, ragged=True),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {op: [work(c) for c in listed() if c["op"] == op] for op in ("prefix", "weights", "evict", "verify")}
    while True:
        op = rng.choice(["prefix", "prefix", "weights", "evict", "verify"])
        hd, Hkv, G = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 4, 5, 8])
        if op == "prefix":
            c = dict(op=op, B=_logint(rng, 1, 128), Tq=_logint(rng, 1, 8), H=Hkv * G, Hkv=Hkv, hd=hd,
                     P=_logint(rng, 1, 131072), S=_logint(rng, 8, 4096), ragged=rng.random() < 0.7)
        elif op == "weights":
            c = dict(op=op, B=_logint(rng, 1, 32), Tq=_logint(rng, 1, 512), H=Hkv * G, Hkv=Hkv, hd=hd,
                     S=_logint(rng, 512, 65536), causal=rng.random() < 0.8)
        elif op == "evict":
            S = _logint(rng, 16, 65536)
            keep = max(8, int(S * rng.uniform(0.05, 1.0)))
            c = dict(op=op, B=_logint(rng, 1, 32), Hkv=Hkv, hd=hd, S=S, keep=keep, recent=keep // rng.choice([3, 8, 100]),
                     sinks=rng.choice([0, 1, 4]), ragged=rng.random() < 0.7)
        else:
            c = dict(op=op, B=_logint(rng, 1, 128), D=_logint(rng, 1, 8), V=_logint(rng, 1000, 200000),
                     temp=rng.choice([0.0, 0.6, 1.0, 1.0, 1.3]), ragged=rng.random() < 0.5)
        w = work(c)
        if all(w[k] <= max(t[k] for t in top[op]) for k in w):
            return c


def work(case):
    c = case
    if c["op"] == "prefix":
        rows = c["B"] * ((1 + c["Tq"]) / 2 if c["ragged"] else c["Tq"])   # mean of q_lens
        cols = c["S"] * (0.75 if c["ragged"] else 1.0)                    # mean suffix length
        kv = 4 * c["Hkv"] * c["hd"] * (c["P"] + c["B"] * cols)
        return {"bytes": kv + 4 * rows * c["H"] * c["hd"] + 4 * rows * c["H"],
                "flops": 4 * rows * c["H"] * c["hd"] * (c["P"] + cols)}
    if c["op"] == "weights":
        rows = c["B"] * c["Tq"]
        seen = c["B"] * c["S"]
        pairs = rows * (c["S"] - (c["Tq"] - 1) / 2 if c["causal"] else c["S"])
        return {"bytes": c["Hkv"] * seen * (2 * c["hd"] + 8) + rows * c["H"] * (2 * c["hd"] + 4),
                "flops": 2 * pairs * c["H"] * c["hd"]}
    if c["op"] == "evict":
        seg = c["B"] * c["Hkv"]
        cols = c["S"] * (0.75 if c["ragged"] else 1.0)
        return {"bytes": seg * (cols * 8 + min(c["keep"], cols) * (8 * c["hd"] + 8)), "flops": 0}
    rows = c["B"] * (c["D"] + 1 + (c["D"] if c["temp"] > 0 else 0))
    return {"bytes": 4 * rows * c["V"], "flops": 4 * rows * c["V"]}


# ---------------------------------------------------------------------------- inputs
def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * seed + 17)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int32)

    c = case
    if c["op"] == "prefix":
        B, Tq, S = c["B"], c["Tq"], c["S"]
        x = dict(q=normal(B, Tq, c["H"], c["hd"], scale=1.5), kp=normal(c["Hkv"], c["P"], c["hd"]),
                 vp=normal(c["Hkv"], c["P"], c["hd"]), k=normal(B, c["Hkv"], S, c["hd"]),
                 v=normal(B, c["Hkv"], S, c["hd"]))
        if c["ragged"]:
            x["lens"] = whole(min(S, max(Tq, S // 2)), S, B)
            x["q_lens"] = torch.minimum(whole(1, Tq, B), x["lens"])
        else:
            x["lens"] = torch.full((B,), S, dtype=torch.int32, device=DEV)
            x["q_lens"] = torch.full((B,), min(Tq, S), dtype=torch.int32, device=DEV)
        return x
    if c["op"] == "weights":
        B, Tq, S = c["B"], c["Tq"], c["S"]
        q = normal(B, Tq, c["H"], c["hd"], scale=1.5)
        # |scale q.k| has a standard deviation of 1.5: lse is near log(columns) + 1.5^2 / 2
        lse = math.log(S) + 1.125 + 0.1 * torch.randn((B, Tq, c["H"]), generator=g, device=DEV)
        x = dict(q=q, k=normal(B, c["Hkv"], S, c["hd"]), lse=lse, acc=4.0 * uniform(B, c["Hkv"], S) ** 4)
        if c["causal"]:
            x["lens"] = torch.full((B,), S, dtype=torch.int32, device=DEV)
        return x
    if c["op"] == "evict":
        B, Hkv, S, hd = c["B"], c["Hkv"], c["S"], c["hd"]
        # a few columns carry most of the weight, some none at all (ties)
        acc = torch.exp(2.0 * torch.randn((B, Hkv, S), generator=g, device=DEV))
        acc = torch.where(uniform(B, Hkv, S) < 0.1, torch.zeros_like(acc), acc)
        pos = torch.argsort(uniform(B, Hkv, S), dim=-1).to(torch.int32)
        lens = whole(max(1, S // 2), S, B) if c["ragged"] else torch.full((B,), S, dtype=torch.int32, device=DEV)
        return dict(k=normal(B, Hkv, S, hd), v=normal(B, Hkv, S, hd), acc=acc, pos=pos, lens=lens)
    B, D, V = c["B"], c["D"], c["V"]
    logits = 3.0 * torch.randn((B, D + 1, V), generator=g, device=DEV)
    draft_logits = logits[:, :D] + torch.randn((B, D, V), generator=g, device=DEV)
    # draft tokens sampled from the draft's own distribution (Gumbel noise)
    t = max(c["temp"], 1e-2)
    noise = -torch.log(-torch.log(uniform(B, D, V).clamp_(1e-7, 1 - 1e-7)))
    draft = torch.argmax(draft_logits / t + noise, dim=-1).to(torch.int32)
    n_draft = whole(0, D, B) if c["ragged"] else torch.full((B,), D, dtype=torch.int32, device=DEV)
    return dict(logits=logits, draft_logits=draft_logits, draft=draft, u=uniform(B, D + 1), n_draft=n_draft)


def prepare(case, seed):
    """Inputs, and the result buffers and scratch that a serving loop keeps from step to step."""
    x = _inputs(case, seed)
    c = case
    if c["op"] == "prefix":
        x["out"] = torch.zeros_like(x["q"])
        x["lse"] = torch.zeros((c["B"], c["Tq"], c["H"]), device=DEV)
    elif c["op"] == "weights":
        x["out"] = torch.zeros_like(x["acc"])
    elif c["op"] == "evict":
        B, Hkv, n, hd = c["B"], c["Hkv"], c["keep"], c["hd"]
        x["out"] = (torch.zeros((B, Hkv, n, hd), dtype=torch.bfloat16, device=DEV),
                    torch.zeros((B, Hkv, n, hd), dtype=torch.bfloat16, device=DEV),
                    torch.zeros((B, Hkv, n), device=DEV),
                    torch.zeros((B, Hkv, n), dtype=torch.int32, device=DEV),
                    torch.zeros((B,), dtype=torch.int32, device=DEV))
    else:
        x["tokens"] = torch.zeros((c["B"], c["D"] + 1), dtype=torch.int32, device=DEV)
        x["n_accepted"] = torch.zeros((c["B"],), dtype=torch.int32, device=DEV)
    x["scratch"] = {}
    return {"case": dict(case), "x": x}


# ---------------------------------------------------------------------------- one pass
def run(state):
    c, x = state["case"], state["x"]
    if own:
        return _call(c, x)
    if c["op"] == "prefix":
        return _plain_prefix(c, x)
    if c["op"] == "weights":
        return _plain_weights(c, x)
    if c["op"] == "evict":
        return _plain_evict(c, x)
    return _plain_verify(c, x)


def _scratch(x, nbytes):
    """The step's scratch buffer, kept by the caller from one call to the next."""
    buf = x["scratch"].get("buf")
    if buf is None or buf.numel() < nbytes:
        buf = x["scratch"]["buf"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    return buf


def _call(c, x):
    from cross_loop_sparsity_b200 import flashloop as fl
    if c["op"] == "prefix":
        n = fl.prefix_attention_scratch_bytes(c["B"], c["Tq"], c["H"], c["Hkv"], c["hd"], c["P"], c["S"])
        return fl.prefix_attention(x["q"], x["kp"], x["vp"], x["k"], x["v"], x["lens"], q_lens=x["q_lens"],
                                   out=x["out"], lse=x["lse"], scratch=_scratch(x, n))
    if c["op"] == "weights":
        n = fl.column_weights_scratch_bytes(c["B"], c["Tq"], c["H"], c["Hkv"], c["hd"], c["S"])
        return fl.column_weights(x["q"], x["k"], x["lse"], x["acc"], lens=x.get("lens"), out=x["out"],
                                 scratch=_scratch(x, n))
    if c["op"] == "evict":
        n = fl.evict_scratch_bytes(c["B"], c["Hkv"], c["S"], c["keep"])
        return fl.evict(x["k"], x["v"], x["acc"], x["pos"], x["lens"], c["keep"], recent=c["recent"],
                        sinks=c["sinks"], out=x["out"], scratch=_scratch(x, n))
    n = fl.verify_draft_scratch_bytes(c["B"], c["D"], c["V"])
    return fl.verify_draft(x["logits"], x["draft_logits"], x["draft"], x["u"], n_draft=x["n_draft"],
                           temperature=c["temp"], tokens=x["tokens"], n_accepted=x["n_accepted"],
                           scratch=_scratch(x, n))


def _visible(lens, q_lens, Tq, S):
    """[B, Tq, S]: query t of the last q_lens tokens sees column j <= lens - q_lens + t."""
    j = torch.arange(S, device=DEV)
    t = torch.arange(Tq, device=DEV)
    last = (lens - q_lens).long()[:, None] + t
    return j[None, None, :] <= last[:, :, None]


def _plain_prefix(c, x):
    B, Tq, H, Hkv, hd, P, S = (c[n] for n in ("B", "Tq", "H", "Hkv", "hd", "P", "S"))
    G = H // Hkv
    q = x["q"].float().view(B, Tq, Hkv, G, hd).permute(2, 0, 1, 3, 4)          # [Hkv, B, Tq, G, hd]
    sp = torch.matmul(q.reshape(Hkv, B * Tq * G, hd), x["kp"].float().transpose(1, 2)) / math.sqrt(hd)
    qs = q.permute(1, 0, 2, 3, 4).reshape(B, Hkv, Tq * G, hd)
    ss = torch.matmul(qs, x["k"].float().transpose(2, 3)) / math.sqrt(hd)
    see = _visible(x["lens"], x["q_lens"], Tq, S)[:, None, :, None, :].expand(B, Hkv, Tq, G, S)
    ss = ss.masked_fill(~see.reshape(B, Hkv, Tq * G, S), -math.inf)
    sp = sp.view(Hkv, B, Tq * G, P).transpose(0, 1)                               # [B, Hkv, Tq*G, P]
    m = torch.maximum(sp.amax(-1), ss.amax(-1))[..., None]
    ep, es = torch.exp(sp - m), torch.exp(ss - m)
    total = (ep.sum(-1) + es.sum(-1))[..., None]
    op = torch.matmul(ep.transpose(0, 1).reshape(Hkv, B * Tq * G, P), x["vp"].float())
    o = op.view(Hkv, B, Tq * G, hd).transpose(0, 1) + torch.matmul(es, x["v"].float())
    o = (o / total).view(B, Hkv, Tq, G, hd).permute(0, 2, 1, 3, 4).reshape(B, Tq, H, hd)
    lse = (m + torch.log(total)).view(B, Hkv, Tq, G).permute(0, 2, 1, 3).reshape(B, Tq, H)
    given = torch.arange(Tq, device=DEV)[None, :] < x["q_lens"][:, None]          # rows past q_lens stay as they were
    out = torch.where(given[:, :, None, None], o, x["out"].float())
    return out.to(torch.bfloat16), torch.where(given[:, :, None], lse, x["lse"])


def _plain_weights(c, x):
    B, Tq, H, Hkv, hd, S = (c[n] for n in ("B", "Tq", "H", "Hkv", "hd", "S"))
    G = H // Hkv
    q = x["q"].float().view(B, Tq, Hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Tq * G, hd)
    s = torch.matmul(q, x["k"].float().transpose(2, 3)) / math.sqrt(hd)
    lse = x["lse"].view(B, Tq, Hkv, G).permute(0, 2, 1, 3).reshape(B, Hkv, Tq * G, 1)
    w = torch.exp(s - lse)
    if c["causal"]:
        see = _visible(x["lens"], torch.full_like(x["lens"], Tq), Tq, S)
        w = w * see[:, None, :, None, :].expand(B, Hkv, Tq, G, S).reshape(B, Hkv, Tq * G, S)
    return x["acc"] + w.sum(2)


def _plain_evict(c, x):
    B, Hkv, S, keep, hd = c["B"], c["Hkv"], c["S"], c["keep"], c["hd"]
    lens = x["lens"].long()[:, None, None]
    slot = torch.arange(S, device=DEV).expand(B, Hkv, S)
    there = slot < lens
    pos = x["pos"].long()
    newest = torch.where(there, pos, -1).amax(-1, keepdim=True)
    safe = (pos < c["sinks"]) | (pos > newest - c["recent"])
    key = torch.where(there, torch.where(safe, math.inf, x["acc"]), -1.0)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    n = torch.minimum(lens, torch.full_like(lens, keep))
    kept = torch.zeros((B, Hkv, S), dtype=torch.bool, device=DEV)
    kept = kept.scatter(2, order, slot < n)
    late = torch.sort(torch.where(kept & (slot >= keep), slot, S), dim=-1).values   # kept slots past the budget
    to = torch.arange(keep, device=DEV).expand(B, Hkv, keep)
    hole = ~kept[:, :, :keep] & (to < n)
    fill = torch.gather(late, 2, (torch.cumsum(hole, -1) - 1).clamp_(0, S - 1))
    src = torch.where(hole, fill, to).clamp_(0, S - 1)
    used = to < n
    rows = src[..., None].expand(B, Hkv, keep, hd)
    ko, vo, ao, po, _ = x["out"]
    return (torch.where(used[..., None], torch.gather(x["k"], 2, rows), ko),
            torch.where(used[..., None], torch.gather(x["v"], 2, rows), vo),
            torch.where(used, torch.gather(x["acc"], 2, src), ao),
            torch.where(used, torch.gather(x["pos"], 2, src), po),
            torch.minimum(x["lens"], torch.full_like(x["lens"], keep)))


def _plain_verify(c, x):
    B, D, V = c["B"], c["D"], c["V"]
    n_draft, draft = x["n_draft"].long(), x["draft"].long()
    i = torch.arange(D, device=DEV)
    if c["temp"] == 0:
        best = torch.argmax((x["logits"] == x["logits"].amax(-1, keepdim=True)).to(torch.uint8), dim=-1)   # lowest index of a tie
        ok = (best[:, :D] == draft) & (i < n_draft[:, None])
        n = torch.cumprod(ok.long(), 1).sum(1)
        token = torch.gather(best, 1, n[:, None])[:, 0]
    else:
        p = torch.softmax(x["logits"].double() / c["temp"], -1)
        q = torch.softmax(x["draft_logits"].double() / c["temp"], -1)
        px = torch.gather(p[:, :D], 2, draft[..., None])[..., 0]
        qx = torch.gather(q, 2, draft[..., None])[..., 0]
        ok = (x["u"][:, :D].double() * qx < px) & (i < n_draft[:, None])
        n = torch.cumprod(ok.long(), 1).sum(1)
        row = n[:, None, None].expand(B, 1, V)
        pr = torch.gather(p, 1, row)[:, 0]
        qr = torch.gather(q, 1, row.clamp(max=D - 1))[:, 0] * (n < n_draft)[:, None]
        cdf = torch.cumsum((pr - qr).clamp_(min=0), -1)
        token = (cdf <= x["u"][:, D, None].double() * cdf[:, -1:]).sum(-1).clamp_(max=V - 1)
    j = torch.arange(D + 1, device=DEV)
    padded = torch.cat([draft, torch.zeros_like(draft[:, :1])], 1)
    tokens = torch.where(j < n[:, None], padded, torch.where(j == n[:, None], token[:, None], -1))
    return tokens.to(torch.int32), n.to(torch.int32)


# ---------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The definitions in 64 bits, one head or one row at a time."""
    c, x = case, _inputs(case, seed)
    if c["op"] == "prefix":
        G, scale = c["H"] // c["Hkv"], 1.0 / math.sqrt(c["hd"])
        out = torch.zeros(x["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros((c["B"], c["Tq"], c["H"]), dtype=torch.float64, device=DEV)
        lens, qn = x["lens"].tolist(), x["q_lens"].tolist()
        for h in range(c["H"]):
            kp, vp = x["kp"][h // G].double(), x["vp"][h // G].double()
            for b in range(c["B"]):
                n, L = qn[b], lens[b]
                s = x["q"][b, :n, h].double() @ torch.cat([kp, x["k"][b, h // G, :L].double()]).T * scale
                s[:, c["P"]:] += torch.triu(torch.full((n, L), -math.inf, dtype=torch.float64, device=DEV), L - n + 1)
                lse[b, :n, h] = torch.logsumexp(s, 1)
                out[b, :n, h] = torch.softmax(s, 1) @ torch.cat([vp, x["v"][b, h // G, :L].double()])
        return out, lse
    if c["op"] == "weights":
        G, scale = c["H"] // c["Hkv"], 1.0 / math.sqrt(c["hd"])
        out = x["acc"].double()
        for b in range(c["B"]):
            for h in range(c["H"]):
                s = x["k"][b, h // G].double() @ x["q"][b, :, h].double().T * scale     # [S, Tq]
                w = torch.exp(s - x["lse"][b, :, h].double())
                if c["causal"]:
                    w = torch.triu(w, -(c["S"] - c["Tq"]))
                out[b, h // G] += w.sum(1)
        return out
    if c["op"] == "evict":
        return None   # a choice of rows and their copies: no computed number
    return None       # whole numbers
