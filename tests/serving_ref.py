"""Plain 64-bit statements of the serving operators, for the tests (CPU numpy)."""
import numpy as np


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def score_error(q, k, scale, hd):
    """Bound on the error of a score formed in fp32 from exact bf16 products: each of the hd
    additions and the scaling rounds by at most 2^-24 of the running magnitude; the
    exponent's argument rounds twice more."""
    mag = np.abs(q) @ np.abs(k).T * abs(scale)
    return (hd + 6) * 2.0 ** -24 * (mag.max() if mag.size else 0.0)


def attention(q, kp, vp, k, v, lens, q_lens, scale):
    """q [B,Tq,H,hd], kp/vp [Hkv,P,hd], k/v [B,Hkv,S,hd] (float64).  Returns out, lse, and per output the
    bound on a bf16 kernel's error: probabilities and output each rounded to bf16 (half a step, 2^-8
    relative), scores off by ``score_error`` (twice: numerator and sum), fp32 sums (2^-18 relative)."""
    B, Tq, H, hd = q.shape
    Hkv, P = kp.shape[:2]
    S = k.shape[2]
    G = H // Hkv
    out = np.zeros(q.shape)
    tol = np.zeros(q.shape)
    lse = np.full((B, Tq, H), -np.inf)
    lse_tol = np.zeros((B, Tq, H))
    for b in range(B):
        ln, qn = min(max(int(lens[b]), 0), S), min(max(int(q_lens[b]), 0), Tq)
        for t in range(qn):
            vis = min(max(ln - qn + t + 1, 0), ln)
            for h in range(H):
                kk = np.concatenate([kp[h // G], k[b, h // G, :vis]])
                vv = np.concatenate([vp[h // G], v[b, h // G, :vis]])
                if len(kk) == 0:
                    continue
                s = kk @ q[b, t, h] * scale
                m = s.max()
                p = np.exp(s - m)
                L = p.sum()
                out[b, t, h] = p @ vv / L
                lse[b, t, h] = m + np.log(L)
                A = p @ np.abs(vv) / L
                ds = score_error(q[b, t, h][None], kk, scale, hd)
                tol[b, t, h] = 2.0 ** -8 * (A + np.abs(out[b, t, h])) * (1 + 2.0 ** -6) + (2 * ds + 2.0 ** -18) * A
                lse_tol[b, t, h] = ds + 2.0 ** -18 + 2.0 ** -22 * abs(lse[b, t, h])
    return out, lse, tol, lse_tol


def column_weights(q, k, lse, acc, lens, q_lens, scale):
    """Returns out and the bound on an fp32 kernel's error: each weight off by its score's error and the
    exponential's (2^-20 relative), the sum of n weights by n 2^-24."""
    B, Tq, H, hd = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    G = H // Hkv
    out = acc.astype(np.float64).copy()
    tol = np.abs(out) * 2.0 ** -23
    for b in range(B):
        ln = S if lens is None else min(max(int(lens[b]), 0), S)
        qn = Tq if q_lens is None else min(max(int(q_lens[b]), 0), Tq)
        for t in range(qn):
            vis = S if lens is None else min(max(ln - qn + t + 1, 0), ln)
            if vis == 0:
                continue
            for h in range(H):
                if lse[b, t, h] == -np.inf:
                    continue
                s = k[b, h // G, :vis] @ q[b, t, h] * scale
                w = np.exp(s - lse[b, t, h])
                out[b, h // G, :vis] += w
                ds = score_error(q[b, t, h][None], k[b, h // G, :vis], scale, hd) + 2.0 ** -22 * (
                    abs(lse[b, t, h]) + np.abs(s).max())
                tol[b, h // G, :vis] += w * (ds + 2.0 ** -20 + qn * H * 2.0 ** -24)
    return out, tol * 1.01


def evict(acc, pos, lens, keep, recent, sinks):
    """Source slot of every destination slot, per (sequence, head): [B][Hkv] lists."""
    B, Hkv, S = acc.shape
    src = []
    for b in range(B):
        n = min(max(int(lens[b]), 0), S)
        heads = []
        for g in range(Hkv):
            if n <= keep:
                heads.append(list(range(n)))
                continue
            newest = max(int(x) for x in pos[b, g, :n])
            bits = acc[b, g, :n].astype(np.float32).view(np.uint32)

            def key(i):
                p = int(pos[b, g, i])
                safe = p < sinks or p > newest - recent
                return (0 if safe else 1, -int(bits[i]) if not safe else 0, i)

            kept = sorted(sorted(range(n), key=key)[:keep])
            stay = set(i for i in kept if i < keep)
            late = [i for i in kept if i >= keep]
            row, it = [], iter(late)
            for i in range(keep):
                row.append(i if i in stay else next(it))
            heads.append(row)
        src.append(heads)
    return src


def verify(logits, draft_logits, draft, u, n_draft, temperature):
    """tokens [B, D+1], n_accepted [B] (float64 softmax, sequential inverse CDF)."""
    B, rows, V = logits.shape
    D = rows - 1
    tokens = np.full((B, D + 1), -1, np.int64)
    n_acc = np.zeros(B, np.int64)
    for b in range(B):
        n = D if n_draft is None else min(max(int(n_draft[b]), 0), D)
        if temperature == 0:
            m = 0
            while m < n and draft[b, m] == int(np.argmax(logits[b, m])):
                m += 1
            y = int(np.argmax(logits[b, m]))
        else:
            T = float(np.float32(temperature))

            def soft(x):
                x = x.astype(np.float64) / T
                e = np.exp(x - x.max())
                return e / e.sum()

            m, y = 0, -1
            while m < n:
                x = int(draft[b, m])
                if not 0 <= x < V:
                    break
                p = soft(logits[b, m])[x]
                q = 1.0 if draft_logits is None else soft(draft_logits[b, m])[x]
                if not float(u[b, m]) * q < p:
                    break
                m += 1
            w = soft(logits[b, m])
            if m < n:
                if draft_logits is None:
                    if 0 <= draft[b, m] < V:
                        w[int(draft[b, m])] = 0.0
                else:
                    w = np.maximum(w - soft(draft_logits[b, m]), 0.0)
            cdf = np.cumsum(w)
            if np.isfinite(cdf[-1]) and cdf[-1] > 0:
                y = int(np.searchsorted(cdf, float(u[b, D]) * cdf[-1], side="right"))
                y = min(y, int(np.nonzero(w)[0][-1]))
        tokens[b, :m] = draft[b, :m]
        tokens[b, m] = y
        n_acc[b] = m
    return tokens, n_acc
