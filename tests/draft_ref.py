"""Plain 64-bit forms of the drafter-side operators, and the tolerances their kernels are held to.

Tolerances.  A kernel's sum of exponentials has terms 2^x, x = c (z - m): the hardware exponential is within one unit
(2^-23 relative), x carries the roundings of c and of one fused multiply-add (2^-24 |x| each, times ln 2 in the result).
Terms that matter have |x| <= 25, so a term is within 25 * 2 * 2^-24 * 0.7 + 2^-23 < 2.3e-6.  A thread adds at most
about 100 terms in sequence after trees of five levels (2^-24 each: < 6.3e-6 in the worst case, one sign throughout).
The top-value pass takes terms up to 2^100 of its reference (100 * 1.5 * 2^-24 * 0.7 + 2^-23 < 6.4e-6) and no 32-bit sum of
more than a vector.  A shift c m that is rounded before it is taken off is below 64 then: 2^-25 * 64 * 0.7 < 1.4e-6,
whatever the logits' size.
So a sum is within SUM = 1e-5 of itself, and its logarithm within 1e-5.
"""
import math

import torch

SUM = 1e-5
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def in_32_bits(T):
    """The temperature as the entry points take it: at |z / T| = 1e7 its rounding shows."""
    return float(torch.tensor(T, dtype=torch.float32))


def teacher(z, k, T):
    """ids, vals, rest of [R, V] rows (any device) in 64 bits."""
    T = in_32_bits(T)
    z = z.double()
    R, V = z.shape
    n = min(k, V)
    v, i = z.sort(dim=-1, descending=True, stable=True)
    ids = torch.full((R, k), -1, dtype=torch.int64)
    vals = torch.full((R, k), -math.inf, dtype=torch.float64)
    ids[:, :n], vals[:, :n] = i[:, :n], v[:, :n]
    rest = (v[:, n:] / T).logsumexp(-1) if n < V else torch.full((R,), -math.inf, dtype=torch.float64)
    return ids, vals, rest


def distill(z, ids, vals, rest, T, g=None):
    """loss, stat, gradient, and |gradient|'s scale (g / T) (q + p) per element, from the formulas."""
    T = in_32_bits(T)
    z = z.double()
    R, V = z.shape
    ids, vals = ids.long(), vals.double()
    g = torch.ones(R, dtype=torch.float64) if g is None else g.double()
    loss, stat = torch.zeros(R, dtype=torch.float64), torch.zeros(R, 4, dtype=torch.float64)
    grad, size = torch.zeros(R, V, dtype=torch.float64), torch.zeros(R, V, dtype=torch.float64)
    for r in range(R):
        seen = {}
        for i, t in zip(ids[r].tolist(), vals[r].tolist()):
            if 0 <= i < V and i not in seen:
                seen[i] = t
        r0 = -math.inf if rest is None else float(rest[r])
        at = torch.tensor(sorted(seen), dtype=torch.int64)
        t = torch.tensor([seen[i] for i in sorted(seen)], dtype=torch.float64)
        top = max([r0] + [x / T for x in t.tolist()])
        if top == -math.inf or not bool((z[r] > -math.inf).any()):
            continue
        e = (t / T - top).exp()
        e0 = math.exp(r0 - top)
        Z = float(e.sum()) + e0
        p, p0 = e / Z, e0 / Z
        m = z[r].max()
        q = ((z[r] - m) / T).exp()
        s = q.sum()
        lq = (z[r] - m) / T - s.log()
        q = q / s
        out = torch.ones(V, dtype=torch.bool)
        out[at] = False
        zo = z[r][out]
        m0 = zo.max() if len(zo) else torch.tensor(-math.inf, dtype=torch.float64)
        s0 = ((zo - m0) / T).exp().sum() if float(m0) > -math.inf else torch.zeros((), dtype=torch.float64)
        lq0 = (m0 - m) / T + s0.log() - s.log()
        lp = p.log()
        x = torch.where(p > 0, p * (lp - lq[at]), torch.zeros_like(p)).sum()
        if p0 > 0:
            x = x + p0 * (math.log(p0) - lq0)
        loss[r] = x
        stat[r] = torch.stack([m, s, m0, s0])
        d, w = q.clone(), q.clone()
        if p0 > 0 and float(m0) > -math.inf:  # p_0 q_v / q_0 without q_0, which may underflow
            e = p0 * ((zo - m0) / T).exp() / s0
            d[out] = q[out] - e
            w[out] = q[out] + e
        d[at] = q[at] - p
        w[at] = q[at] + p
        grad[r], size[r] = d * g[r] / T, w * abs(float(g[r])) / T
    return loss, stat, grad, size


def beams(z, scores, N, T, finished=None, pad=0):
    """beam, tok, score [B, N + 1] (one more than asked: the next score) in 64 bits."""
    T = in_32_bits(T)
    B, W, V = z.shape
    beam = torch.full((B, N + 1), -1, dtype=torch.int64)
    tok, score = beam.clone(), torch.full((B, N + 1), -math.inf, dtype=torch.float64)
    for b in range(B):
        x = torch.full((W, V), -math.inf, dtype=torch.float64)
        fin = {}
        for w in range(W):
            s = float(scores[b, w])
            if s == -math.inf:
                continue
            if finished is not None and int(finished[b, w]):
                fin[w] = s
            else:
                zt = z[b, w].double() / T
                if bool((zt > -math.inf).any()):
                    x[w] = s + zt - zt.logsumexp(-1)
        v, i = x.flatten().sort(descending=True, stable=True)
        best = [(-float(v[j]), int(i[j]) // V, int(i[j]) % V) for j in range(min(N + 1, W * V))]
        best = [c for c in best + [(-s, w, pad) for w, s in fin.items()] if c[0] < math.inf]
        for n, (s, w, t) in enumerate(sorted(best)[: N + 1]):
            beam[b, n], tok[b, n], score[b, n] = w, t, -s
    return beam, tok, score


def reorder(src, dst, parent, lens):
    """dst after the reorder; src [L, B, W, H, S, D], dst [L, B, N, H, S, D]."""
    out = dst.clone()
    for b in range(parent.shape[0]):
        for n in range(parent.shape[1]):
            w = int(parent[b, n])
            if w >= 0:
                k = int(lens[b])
                out[:, b, n, :, :k] = src[:, b, w, :, :k]
    return out
