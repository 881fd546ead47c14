"""The C ABI of the verifier's pass without a GPU: exported names, sizes, and refusals before any HIP call (pointers are fake
addresses that are never read); the format's plain form."""
import ctypes
import math
import os
import re

import pytest
import torch

from lossless_draft_verification_04_amd import specverify as svx
from tests import pass_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = svx._lib
P = ctypes.c_void_p
A, A2, A3, A4, WS = P(0x100000000), P(0x200000000), P(0x300000000), P(0x400000000), P(0x40000)
BIG = 1 << 34
INF, NAN = math.inf, math.nan


def st(*v):
    return (ctypes.c_int64 * 3)(*v) if v and v[0] is not None else None


def cache(**kw):
    c = dict(pool=0x500000000, pages=0x600000000, page_stride=4 * 64 * 136, layer_stride=0, num_pages=10, max_pages=4,
             page_tokens=64, H=4, D=128, layers=1)
    c.update(kw)
    return ctypes.byref(svx._CCache(*[c[n] for n, _ in svx._CCache._fields_]))


def test_every_declared_function_is_exported():
    text = open(os.path.join(ROOT, "include", "specverify_pass.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(sv_[a-z_]+)\s*\(", text))
    assert names == set(svx.PASS_EXPORTED)
    for n in names:
        assert hasattr(L, n)


def test_sizes():
    n = ctypes.c_size_t(0)
    size = lambda op, B=8, N=17, Hq=32, H=8, D=128: (  # noqa: E731
        L.sv_pass_workspace_size(op, B, N, Hq, H, D, ctypes.byref(n)), n.value)
    for op in range(5):
        s, b = size(op)
        assert s == svx.SV_OK and b % 256 == 0 and b >= 256 + 65536 * 4
    assert size(5)[0] == svx.SV_EINVAL and size(-1)[0] == svx.SV_EINVAL
    for kw in (dict(B=-1), dict(N=0), dict(Hq=0), dict(H=0), dict(Hq=30)):
        assert size(3, **kw)[0] == svx.SV_EINVAL, kw
    for kw in (dict(B=32769), dict(N=1025), dict(Hq=2048), dict(D=96), dict(D=0)):
        assert size(3, **kw)[0] == svx.SV_EUNSUPPORTED, kw
    assert size(3, B=32768, N=1024, Hq=1024, H=1, D=256)[0] == svx.SV_OK
    assert L.sv_pass_workspace_size(0, 0, 0, 0, 0, 0, None) == svx.SV_EINVAL
    assert svx.kv_page_bytes(8, 128, 64) == 8 * 64 * 136 and svx.kv_page_bytes(1, 64, 16) == 16 * 68
    for bad in ((0, 128, 64), (8, 96, 64), (8, 128, 48), (8, 128, 8), (1025, 128, 64), (8, 128, 1 << 21)):
        with pytest.raises(svx.SpecVerifyError):
            svx.kv_page_bytes(*bad)


def cache_refusals(f):
    """Common refusals of an entry point over a cache: f(c=, ws=, wsb=)."""
    assert f(c=ctypes.POINTER(svx._CCache)()) == svx.SV_EINVAL
    for kw in (dict(H=0), dict(page_tokens=0), dict(page_tokens=48), dict(page_tokens=8), dict(num_pages=0),
               dict(max_pages=0), dict(pool=None), dict(pages=None), dict(page_stride=4 * 64 * 136 - 16),
               dict(num_pages=2 ** 31 - 1, page_stride=1 << 40)):
        assert f(c=cache(**kw)) == svx.SV_EINVAL, kw
    for kw in (dict(D=96), dict(D=512), dict(page_tokens=1 << 21)):
        assert f(c=cache(**kw)) == svx.SV_EUNSUPPORTED, kw
    for kw in (dict(pool=0x500000008), dict(page_stride=4 * 64 * 136 + 8)):
        assert f(c=cache(**kw)) == svx.SV_EALIGN, kw
    assert f(ws=None) == svx.SV_EWORKSPACE and f(wsb=1024) == svx.SV_EWORKSPACE and f(ws=P(0x40010)) == svx.SV_EALIGN


KS = (5 * 512, 512, 128)  # [B, 5, 4, 128]


def test_write_and_read_argument_checks():
    def w(k=A, ks=KS, v=A2, vs=KS, dt=1, c=None, lens=A3, B=3, N=5, ws=WS, wsb=BIG):
        return L.sv_kv_write(k, st(*ks), v, st(*vs), dt, cache() if c is None else c, lens, None, B, N, ws, wsb, None)

    def r(k=A, ks=KS, v=A2, vs=KS, dt=1, c=None, lens=A3, B=3, N=5, ws=WS, wsb=BIG):
        return L.sv_kv_read(cache() if c is None else c, lens, None, B, N, dt, k, st(*ks), v, st(*vs), ws, wsb, None)

    for f in (w, r):
        cache_refusals(f)
        assert f(dt=3) == svx.SV_EDTYPE and f(dt=-1) == svx.SV_EDTYPE
        assert f(B=-1) == svx.SV_EINVAL and f(N=-1) == svx.SV_EINVAL and f(B=32769) == svx.SV_EUNSUPPORTED
        assert f(B=0) == svx.SV_OK and f(N=0) == svx.SV_OK
        for name in ("k", "v"):
            assert f(**{name: None}) == svx.SV_EINVAL and f(**{name: P(0x100000008)}) == svx.SV_EALIGN
        for name in ("ks", "vs"):
            assert f(**{name: (None,)}) == svx.SV_EINVAL
            assert f(**{name: (2560, -512, 128)}) == svx.SV_EINVAL and f(**{name: (2560, 516, 128)}) == svx.SV_EALIGN
            assert f(**{name: (1 << 62, 512, 128)}) == svx.SV_EINVAL
        assert f(B=32768, N=2 ** 31 - 1, ks=(1 << 44, 512, 128), vs=(1 << 44, 512, 128), v=P(1 << 62)) in (svx.SV_EUNSUPPORTED, svx.SV_EINVAL)
    assert w(lens=None) == svx.SV_EINVAL
    assert r(ks=(2560, 512, 64)) == svx.SV_EINVAL and r(vs=(2560, 0, 128)) == svx.SV_EINVAL  # rows on top of one another
    assert r(v=P(0x100000000 + 256)) == svx.SV_EINVAL


def test_attention_argument_checks():
    qs = (5 * 1024, 1024, 128)  # [B, 5, 8, 128]

    def f(q=A, qs=qs, dt=1, c=None, lens=A3, B=3, N=5, Hq=8, scale=0.1, cap=0.0, reach=0, out=A2, os=qs, lse=None, ws=WS,
          wsb=BIG):
        return L.sv_kv_attention(q, st(*qs), dt, cache() if c is None else c, lens, None, None, B, N, Hq, scale, cap, None, reach, out, st(*os),
                                 lse, ws, wsb, None)

    cache_refusals(f)
    assert f(lse=A) == svx.SV_EINVAL and f(lse=P(0x200000000 + 4)) == svx.SV_EINVAL and f(lse=P(0x500000002)) == svx.SV_EALIGN
    assert f(dt=0) == svx.SV_EDTYPE and f(dt=3) == svx.SV_EDTYPE
    assert f(B=-1) == svx.SV_EINVAL and f(N=0) == svx.SV_EINVAL and f(Hq=6) == svx.SV_EINVAL and f(Hq=0) == svx.SV_EINVAL
    assert f(B=32769) == svx.SV_EUNSUPPORTED and f(N=1025) == svx.SV_EUNSUPPORTED and f(Hq=1028) == svx.SV_EUNSUPPORTED
    for v in (INF, -INF, NAN, 3e38):
        assert f(scale=v) == svx.SV_EINVAL and f(cap=v) == svx.SV_EINVAL
    assert f(cap=-1.0) == svx.SV_EINVAL and f(cap=1e-45) == svx.SV_EINVAL and f(reach=-1) == svx.SV_EINVAL
    for name in ("q", "out", "lens"):
        assert f(**{name: None}) == svx.SV_EINVAL, name
    assert f(q=P(0x100000008)) == svx.SV_EALIGN and f(out=P(0x200000008)) == svx.SV_EALIGN
    assert f(qs=(5120, 1028, 128)) == svx.SV_EALIGN and f(os=(5120, 1028, 136)) == svx.SV_EALIGN
    assert f(os=(5120, 1024, 64)) == svx.SV_EINVAL and f(out=P(0x100000000 + 512)) == svx.SV_EINVAL and f(out=A) == svx.SV_EINVAL
    assert f(B=0) == svx.SV_OK


def test_commit_argument_checks():
    def f(c=None, lens=A, n=A2, path=A3, B=3, M=8, out=A4, ws=WS, wsb=BIG):
        return L.sv_kv_commit(cache() if c is None else c, lens, n, path, B, M, out, ws, wsb, None)

    cache_refusals(f)
    page = 4 * 64 * 136
    for kw in (dict(layers=0), dict(layers=-1), dict(layers=2, layer_stride=page - 16), dict(layers=2, layer_stride=9 * page),
               dict(layers=2, layer_stride=-page), dict(layers=3, page_stride=2 * page, layer_stride=page)):
        assert f(c=cache(**kw)) == svx.SV_EINVAL, kw
    assert f(c=cache(layers=2, layer_stride=10 * page + 8)) == svx.SV_EALIGN
    assert f(c=cache(layers=1 << 20), B=32768) == svx.SV_EINVAL  # no layer stride
    assert f(c=cache(layers=65537, layer_stride=1 << 30)) == svx.SV_EUNSUPPORTED
    for name in ("lens", "n", "out"):
        assert f(**{name: None}) == svx.SV_EINVAL, name
    assert f(out=A) == svx.SV_EINVAL and f(out=P(0x100000008)) == svx.SV_EINVAL
    assert f(out=A2) == svx.SV_EINVAL and f(out=P(0x200000008)) == svx.SV_EINVAL
    assert f(out=A3) == svx.SV_EINVAL and f(out=P(0x300000000 + 4 * 23)) == svx.SV_EINVAL
    assert f(c=cache(layers=65536, layer_stride=1 << 48)) == svx.SV_EINVAL
    assert f(B=-1) == svx.SV_EINVAL and f(M=-1) == svx.SV_EINVAL and f(M=1025) == svx.SV_EUNSUPPORTED
    assert f(B=0) == svx.SV_OK


def test_rope_argument_checks():
    qs = (5 * 512, 512, 128)  # [B, 5, 4, 128]

    def f(q=A, qs=qs, k=A2, ks=qs, dt=1, B=3, N=5, Hq=4, Hk=4, D=128, R=64, freq=P(0x700000000), factor=1.0, parent=None, oq=A3, oqs=qs,
          ok=A4, oks=qs, ws=WS, wsb=BIG):
        return L.sv_rope(q, st(*qs), k, st(*ks), dt, B, N, Hq, Hk, D, R, freq, factor, 0, 0, None, None, parent, oq, st(*oqs), ok,
                         st(*oks), ws, wsb, None)

    assert f(dt=3) == svx.SV_EDTYPE
    for kw in (dict(B=-1), dict(N=-1), dict(Hq=-1), dict(Hk=-1), dict(D=1), dict(R=0), dict(R=63), dict(R=130), dict(factor=INF),
               dict(factor=NAN), dict(q=None), dict(k=None), dict(oq=None), dict(ok=None), dict(freq=None), dict(qs=(None,)),
               dict(oks=(None,)), dict(qs=(2560, -512, 128)), dict(oqs=(2560, 512, 64)),
               dict(oq=P(0x100000100)), dict(ok=P(0x200000100)), dict(oq=A, oqs=(5120, 1024, 128)), dict(oq=A2), dict(ok=A3)):
        assert f(**kw) == svx.SV_EINVAL, kw
    for kw in (dict(D=8194), dict(Hq=1025), dict(Hk=1025), dict(B=1 << 20, N=1 << 20), dict(N=1025, parent=A)):
        assert f(**kw) == svx.SV_EUNSUPPORTED, kw
    assert f(q=P(0x100000001)) == svx.SV_EALIGN and f(freq=P(0x700000004)) == svx.SV_EALIGN
    assert f(ws=None) == svx.SV_EWORKSPACE and f(wsb=16) == svx.SV_EWORKSPACE and f(ws=P(0x40010)) == svx.SV_EALIGN
    assert f(B=0) == svx.SV_OK and f(N=0) == svx.SV_OK and f(Hq=0, Hk=0) == svx.SV_OK
    # q in place, k apart, where what is read as k is q itself, or one of its heads
    assert f(oq=A, k=A) == svx.SV_EINVAL and f(oq=A, k=P(0x100000000 + 128 * 2)) == svx.SV_EINVAL
    assert f(ok=A2, q=A2) == svx.SV_EINVAL and f(ok=A2, q=P(0x200000000 + 512 * 2)) == svx.SV_EINVAL
    # views of one projection whose heads lie across one another
    fused = (5 * 1024, 1024, 128)
    assert f(q=A, qs=fused, k=P(0x100000000 + 256 * 2), ks=fused, oq=A, oqs=fused, ok=P(0x100000000 + 256 * 2), oks=fused) == svx.SV_EINVAL


def test_rope_frequencies_refuse():
    out, s = (ctypes.c_double * 64)(), ctypes.c_float(0)

    def f(kind=0, R=64, theta=1e4, scale=1.0, orig=4096, fast=32.0, slow=1.0, o=out, s=ctypes.byref(s)):
        return L.sv_rope_frequencies(kind, R, theta, scale, orig, fast, slow, o, s)

    for kind in range(4):
        assert f(kind) == svx.SV_OK
    for kw in (dict(kind=4), dict(kind=-1), dict(R=0), dict(R=7), dict(R=8194), dict(theta=0.0), dict(theta=NAN), dict(scale=0.5),
               dict(scale=INF), dict(o=None), dict(s=None), dict(kind=3, orig=0), dict(kind=3, slow=0.0), dict(kind=3, fast=1.0),
               dict(kind=3, theta=1.0)):
        assert f(**kw) == svx.SV_EINVAL, kw


def test_rope_frequencies_by_parts_where_all_are_slow():
    """Angles of less than `slow` turns over `original` positions are divided by the scale, the first pair's among them."""
    for R, original, fast, slow in ((64, 4096, 2000.0, 1000.0), (64, 4, 32.0, 1.0), (2, 6, 2.0, 1.0), (128, 100, 40.0, 16.0)):
        plain, _ = svx.sv_rope_frequencies(R)
        assert float(original * plain[0]) / (2 * math.pi) < slow
        f, _ = svx.sv_rope_frequencies(R, kind="parts", scale=4.0, original=original, fast=fast, slow=slow)
        assert torch.allclose(f, plain / 4, rtol=1e-15, atol=0)
    for R, original, fast, slow in ((64, 4096, 600.0, 1.0), (64, 128, 32.0, 1.0), (64, 7, 32.0, 1.0)):  # the first pair turns more than that
        plain, _ = svx.sv_rope_frequencies(R)
        f, _ = svx.sv_rope_frequencies(R, kind="parts", scale=4.0, original=original, fast=fast, slow=slow)
        assert f[0] == 1.0 and f[-1] == plain[-1] / 4


def test_binding_refuses_layouts():
    B, H, D, N = 2, 2, 64, 3
    pool = torch.zeros(6, svx.kv_page_bytes(H, D, 16), dtype=torch.uint8)
    pages = torch.zeros(B, 2, dtype=torch.int32)
    c = svx.KvCache(pool, pages, H, D, 16)
    several = svx.KvCache(torch.zeros(2, 6, svx.kv_page_bytes(H, D, 16), dtype=torch.uint8), pages, H, D, 16)
    kv, q = torch.zeros(B, N, H, D), torch.zeros(B, N, 4, D, dtype=torch.bfloat16)
    lens, freq = torch.zeros(B, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    bad = [
        lambda: svx.KvCache(pool[:, :-1], pages, H, D, 16),
        lambda: svx.KvCache(pool.int(), pages, H, D, 16),
        lambda: svx.KvCache(pool, pages.long(), H, D, 16),
        lambda: svx.KvCache(pool, pages[0], H, D, 16),
        lambda: svx.KvCache(pool, pages, H, 48, 16),
        lambda: svx.sv_kv_write(c, kv, kv, lens),                                     # not on the GPU
        lambda: svx.sv_kv_write(c, kv.double(), kv.double(), lens),
        lambda: svx.sv_kv_write(c, kv, kv[:, :2], lens),
        lambda: svx.sv_kv_write(c, kv[:1], kv[:1], lens[:1]),
        lambda: svx.sv_kv_write(c, kv.transpose(2, 3), kv.transpose(2, 3), lens),
        lambda: svx.sv_kv_write(c, kv, kv, lens.long()),
        lambda: svx.sv_kv_write(c, kv, kv, lens, news=lens[:1]),
        lambda: svx.sv_kv_read(c, lens, lens, kv, kv[:, :, :1]),
        lambda: svx.sv_kv_attention(c, q.float(), lens),
        lambda: svx.sv_kv_attention(c, q[..., :32], lens),
        lambda: svx.sv_kv_attention(c, q, lens, parent=torch.zeros(B, N + 1, dtype=torch.int32)),
        lambda: svx.sv_kv_attention(c, q, lens, slopes=torch.zeros(3)),
        lambda: svx.sv_kv_attention(c, q, lens, out=q.half()),
        lambda: svx.sv_kv_commit(c, lens, lens, path=torch.zeros(B, dtype=torch.int32)),
        lambda: svx.sv_kv_commit(c, lens, lens, path=torch.zeros(B, 4)),
        lambda: svx.sv_rope(kv, freq.float()),
        lambda: svx.sv_rope(kv, freq, k=kv.half()),
        lambda: svx.sv_rope(kv, freq, positions=lens),
        lambda: svx.sv_rope(kv, freq, out_k=kv),
        lambda: svx.sv_rope(kv[0], freq),
        lambda: svx.sv_rope_frequencies(64, kind="other"),
        lambda: svx.sv_rope_frequencies(63),
        lambda: several._one("sv_kv_write"),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(svx.SpecVerifyError):
            f()
            print("not refused:", i)
    assert several.layer(1)._one("x") is not None and several._c.layers == 2 and several._c.layer_stride == 6 * pool.shape[1]


def test_format():
    """Every value of the grid is kept; each other goes to the nearest, ties to even codes; the reference's two ways of
    reading a pool agree."""
    scale = torch.exp2(torch.arange(-20, 20.0))
    x = torch.zeros(40, 32)
    x[:, :8] = ref.GRID.float() * scale[:, None]
    x[:, 8:16] = -x[:, :8]
    x[:, 16:23] = (ref.GRID[1:] + ref.GRID[:-1]).float() / 2 * scale[:, None]
    code, s = ref.encode(x)
    assert torch.equal(s.long() - 127, torch.arange(-20, 20)[:, None])
    y = ref.decode(code, s)
    assert torch.equal(y[:, :16], x[:, :16].double())
    assert torch.equal(code[0, 16:23].long(), torch.tensor([0, 2, 2, 4, 4, 6, 6]))
    big = torch.linspace(1, 2, 129)[:-1, None].repeat(1, 32).clone()
    _, s = ref.encode(big)
    assert torch.equal(s[:, 0].long() - 127, torch.where(big[:, 0] >= 1.75, -1, -2))
    for D in (64, 128, 256):
        c = ref.Cache(2, 3, D, 16, 3, seed=D)
        k, v = c.tokens(1, 40)
        for t in (0, 1, 5, 15, 16, 39):
            for a, b in zip(c.get(1, t), (k[t], v[t])):
                assert torch.equal(a.nan_to_num(-1), b.nan_to_num(-1))
        raw = c.raw(0, 17)
        assert raw.numel() == 3 * (D + D // 16)
        c.set_raw(1, 2, raw)
        assert torch.equal(c.raw(1, 2), raw)
