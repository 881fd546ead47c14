"""The verifier's pass in plain 64-bit torch on the CPU (formulas of specverify_pass.h), and how far the kernels may be off."""
import math

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
F64 = torch.float64


# ---------------------------------------------------------------------------
# the 4-bit format
# ---------------------------------------------------------------------------
def encode(x):
    """[..., D] of 16 or 32 bits -> codes [..., D] (sign 8, place in GRID), scale bytes [..., D/32]."""
    b = x.double().unflatten(-1, (-1, 32))
    a = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    m, e = torch.where(bad | (a == 0), torch.ones_like(a), a).frexp()  # a = m 2^e, 0.5 <= m < 1
    s = (e - 3 + (m >= 0.875).int()).clamp(-126, 125)
    s = torch.where(a == 0, -126, s)
    y = b.abs() * torch.exp2(-s.double())[..., None]
    y = torch.where(bad[..., None], torch.zeros_like(y), y)
    # between neighbours of the grid: the nearer, of two as near the one in an even place
    mid = (GRID[1:] + GRID[:-1]) / 2
    code = (y[..., None] > mid).sum(-1)
    tie = (y[..., None] == mid).any(-1) & (code % 2 == 1)
    code = code + tie.long()
    sign = torch.where(bad[..., None], torch.zeros_like(code), b.signbit().long())
    return (code + 8 * sign).flatten(-2).to(torch.uint8), torch.where(bad, 255, s + 127).to(torch.uint8)


def decode(codes, scales):
    v = GRID[(codes & 7).long()]
    v = torch.where(codes >= 8, -v, v)
    s = torch.where(scales == 255, math.nan, torch.exp2(scales.double() - 127))
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


class Cache:
    """A pool on the CPU, written and read by the layout that specverify_pass.h describes."""

    def __init__(self, B, H, D, P, max_pages, seed=0, layers=1, spare=3, fill=None):
        g = torch.Generator().manual_seed(seed)
        self.H, self.D, self.P = H, D, P
        self.n = B * max_pages + spare
        self.bytes = H * P * (D + D // 16)
        self.pool = torch.randint(0, 256, (layers, self.n, self.bytes), generator=g, dtype=torch.uint8)  # NaN scales too
        if fill is not None:
            self.pool.fill_(fill)
        self.pages = torch.randperm(self.n, generator=g)[:B * max_pages].view(B, max_pages).int()

    def _at(self, b, t, h):
        """Page, and the offsets of a token's key codes, key scales, value codes, value scales."""
        D, P = self.D, self.P
        page, s = int(self.pages[b, t // P]), t % P
        base = h * P * (D + D // 16)
        d, j = torch.arange(0, D, 2), torch.arange(D // 32)
        w = D // 32
        kc = base + s * (D // 2) + d // 2
        ks = base + P * D // 2 + s * w + j
        v0 = base + P * (D // 2 + w)
        byte = d // 2
        vc = v0 + ((s // 4 * 16 + byte // w) * 4 + s % 4) * w + byte % w
        vs = v0 + P * D // 2 + (s // 4 * w + j) * 4 + s % 4
        return page, kc, ks, vc, vs

    def put(self, b, t, k, v, layer=0):
        """One token's keys and values [H, D]."""
        for h in range(self.H):
            page, kc, ks, vc, vs = self._at(b, t, h)
            row = self.pool[layer, page]
            for x, c, s in ((k, kc, ks), (v, vc, vs)):
                code, scale = encode(x[h])
                row[c] = code[0::2] | (code[1::2] << 4)
                row[s] = scale

    def get(self, b, t, layer=0):
        """Keys and values [H, D] of one token in 64 bits."""
        out = []
        for h in range(self.H):
            page, kc, ks, vc, vs = self._at(b, t, h)
            row = self.pool[layer, page]
            out.append([decode(torch.stack([row[c] & 15, row[c] >> 4], -1).flatten(), row[s]) for c, s in ((kc, ks), (vc, vs))])
        return torch.stack([o[0] for o in out]), torch.stack([o[1] for o in out])

    def raw(self, b, t, layer=0):
        """The bytes of one token, heads and sections in a row."""
        got = []
        for h in range(self.H):
            page, *at = self._at(b, t, h)
            got += [self.pool[layer, page][a] for a in at]
        return torch.cat(got)

    def set_raw(self, b, t, x, layer=0):
        for h, part in enumerate(x.view(self.H, -1)):
            page, *at = self._at(b, t, h)
            self.pool[layer, page][torch.cat(at)] = part

    def tokens(self, b, n, layer=0):
        """Keys and values [n, H, D] of a sequence's first tokens, all at once (the same as get, token by token)."""
        D, P, H, w = self.D, self.P, self.H, self.D // 32
        at = torch.arange(n)
        raw = self.pool[layer][self.pages[b].long()[at // P]].view(n, H, -1)
        s = (at % P)[:, None]
        d, j = torch.arange(0, D, 2), torch.arange(w)
        byte = d // 2
        v0 = P * (D // 2 + w)
        idx = [s * (D // 2) + byte, P * D // 2 + s * w + j, v0 + ((s // 4 * 16 + byte // w) * 4 + s % 4) * w + byte % w,
               v0 + P * D // 2 + (s // 4 * w + j) * 4 + s % 4]
        kc, ks, vc, vs = (raw.gather(2, i[:, None].expand(n, H, -1)) for i in idx)
        return tuple(decode(torch.stack([c & 15, c >> 4], -1).flatten(-2), x) for c, x in ((kc, ks), (vc, vs)))


# ---------------------------------------------------------------------------
# windows
# ---------------------------------------------------------------------------
def ancestors(parent, n):
    """For each of n nodes the list from the root (or from where its parents stop being valid) to itself."""
    out = []
    for i in range(n):
        p = i - 1 if parent is None else int(parent[i])
        out.append((out[p] if i and 0 <= p < i else []) + [i])
    return out


def random_tree(n, seed, width=4):
    g = torch.Generator().manual_seed(seed)
    return torch.tensor([-1] + [max(0, i - 1 - int(torch.randint(0, width, (1,), generator=g))) for i in range(1, n)],
                        dtype=torch.int32)


def rope(x, at, freq, factor, interleaved, inverse):
    """x [N, heads, D], at [N] -> the turned rows in 64 bits, and what their error is measured by."""
    R = 2 * freq.shape[0]
    y, size = x.double().clone(), x.double().abs()
    a = at.double()[:, None] * freq
    c, s = factor * a.cos()[:, None], factor * a.sin()[:, None] * (-1 if inverse else 1)
    i = torch.arange(R // 2)
    i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    u, w = x[..., i].double(), x[..., j].double()
    y[..., i], y[..., j] = u * c - w * s, w * c + u * s
    size[..., i] = size[..., j] = abs(factor) * (u.abs() + w.abs())
    return y, size


# An angle is off by its rounding to 32 bits as a part of a turn (2^-26 turns, 2^-23.3), its sine and cosine by two units in
# the last place (2^-23), the factor, products and sum by half a unit each (2^-24): 2^-21 in all, of |x| + |y|
ROPE = 2.0 ** -21


def attention(q, k, v, n0, parent, scale, cap, slopes, reach, dtype):
    """q [n, Hq, D], k, v [n0 + n, H, D] in 64 bits -> out [n, Hq, D], lse [n, Hq] and how far the kernel's may be off.

    Scores: products and sums of 32 bits, each off by at most half a unit (2^-24) of the sum of magnitudes, at most D + 8 of them
    in a row.  The matrix instruction for 4 and 8 bits aligns 128 products to the largest and drops what lies 2^-17 below it:
    of products of random codes of every exponent its sums were off by 2^-10.4 of the largest at most, which is 128 times
    2^-17.4; so D 2^-17 of the largest product, once for each of up to three parts that a query is split into (each 2^-4 of
    the one before or less: 1.07 in all).  Queries of two parts leave 2^-22 of the row's largest value; what follows (scale, cap, bias, exponential) six
    roundings of the score, the cap's reciprocal and exponential 2^-21 of the cap.  A score's error counts twice, in its
    own weight and in the sum.  Weights are rounded to bf16 (2^-9), with fp16 to twice as many bits (2^-17), again twice.  Sums over
    T tokens lose T 2^-24 at most.  The result is rounded to half a step of its type."""
    n, Hq, D = q.shape
    H, T = k.shape[1], k.shape[0]
    G = Hq // H
    paths = ancestors(parent, n)
    depth = torch.tensor([len(p) - 1 for p in paths])
    pos = torch.cat([torch.arange(n0), n0 + depth])
    d = (n0 + depth)[:, None] - pos
    see = torch.zeros(n, T, dtype=torch.bool)
    see[:, :n0] = True
    for i, p in enumerate(paths):
        see[i, [n0 + j for j in p]] = True
    if reach:
        see &= d < reach
    qd = q.double().unflatten(1, (H, G))
    s = torch.einsum("nhgd,thd->nhgt", qd, k) * scale
    mag = torch.einsum("nhgd,thd->nhgt", qd.abs(), k.abs()) * abs(scale)
    most = qd.abs().amax(-1)[..., None] * k.abs().sum(-1).t()[None, :, None] * abs(scale)
    biggest = (qd.abs()[:, :, :, None] * k.abs().permute(1, 0, 2)[None, :, None]).amax(-1) * abs(scale)
    off = mag * (D + 8) * 2.0 ** -24 + most * 2.0 ** -22 + biggest * 1.07 * D * 2.0 ** -17
    if cap:
        s = cap * torch.tanh(s / cap)
        off = off + cap * 2.0 ** -21
    if slopes is not None:
        bias = slopes.double().view(H, G, 1) * d[:, None, None]
        s = s - bias
        off = off + bias.abs() * 2.0 ** -23
    off = off + s.abs() * 6 * 2.0 ** -24
    vis = see[:, None, None].expand_as(s)
    s = torch.where(vis, s, -math.inf)
    off = torch.where(vis, off, 0.0).amax(-1)
    none = ~see.any(-1)
    m = s.nan_to_num(-math.inf, math.inf, -math.inf).amax(-1, keepdim=True).clamp(min=-1e300)
    e = torch.where(vis, (s - m).exp(), 0.0)
    l = e.sum(-1, keepdim=True)
    w = e / torch.where(l == 0, 1.0, l)
    # what a row does not see counts for nothing, NaN or not
    pairs = torch.where(vis[..., None], v.permute(1, 0, 2)[None, :, None] * 1.0, 0.0) if not torch.isfinite(v).all() else None
    if pairs is None:
        out = torch.einsum("nhgt,thd->nhgd", w, v)
        size = torch.einsum("nhgt,thd->nhgd", w, v.abs())
    else:
        out, size = (w[..., None] * pairs).sum(3), (w[..., None] * pairs.abs()).sum(3)
    lse = torch.where(l[..., 0] == 0, -math.inf, m[..., 0] + l[..., 0].log())
    rounding = 2.0 ** -9 if dtype is torch.bfloat16 else 2.0 ** -17
    rel = (2 * (off.exp() - 1) + 2 * rounding + T * 2.0 ** -24)[..., None]
    tol = torch.finfo(dtype).eps / 2 * out.abs() + size * rel * (1 + 2.0 ** -7) + torch.finfo(dtype).tiny
    lse_tol = (off + 1.01 * rounding + T * 2.0 ** -24 + 2.0 ** -21 * (1 + lse.abs().nan_to_num(0, 0, 0)))
    return out.flatten(1, 2), lse.flatten(1, 2), tol.flatten(1, 2), lse_tol.flatten(1, 2), none
