"""Attention over the 4-bit cache where scores are hard: one channel far above the others, queries of very different sizes
within a row, large scores whose references move along the tokens, caps near their ends.  Tolerances are those of sums in 32
bits, with nothing in them for products that a matrix unit drops."""
import math

import pytest
import torch

from lossless_draft_verification_04_amd import specverify as svx
from tests import pass_ref as ref
from tests.test_gpu_pass import BF16, DEV, F16, handle, i32, near, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_error():
    svx.sv_get_device_error(DEV)
    yield
    assert svx.sv_get_device_error(DEV) == 0


def attention(q, k, v, n0, scale, cap, dtype, exact=False, tokens=None):
    """A chain's q [n, Hq, D] over k, v [n0 + n, H, D] in 64 bits -> out, lse and how far off sums in 32 bits may be.

    A score is a sum of D exact products (8 bits by 3; fp16's two parts 2 D), each addition off by half a unit (2^-24) of the
    magnitudes' sum, or exact where `exact` says that all of them fit 24 bits.  Scale, cap and exponential are six roundings of
    the score; a cap multiplies what came before by its slope, at most 1 - tanh^2 at the error's inner end, and is itself off by
    2^-21 of the cap.  With scores off by e at most, weights are off by d = e^e (1 + u) - 1 of themselves, u = 2^-8 (bf16) or
    2^-16 (fp16: two parts) for their rounding, and sum w~ v / sum w~ by d / (1 - d) sum w |v - out| (weights are summed as
    rounded).  Sums over T tokens lose T 2^-24 of their magnitudes, twice.  The result is rounded to half a step."""
    n, Hq, D = q.shape
    H, T = k.shape[1], k.shape[0]
    qd = q.double().unflatten(1, (H, Hq // H))
    s = torch.einsum("nhgd,thd->nhgt", qd, k) * scale
    off = s.abs() * 2 * 2.0 ** -24
    if not exact:
        off = off + torch.einsum("nhgd,thd->nhgt", qd.abs(), k.abs()) * abs(scale) * (2 * D + 8) * 2.0 ** -24
    if cap:
        inner = ((s.abs() - off).clamp(min=0) / cap).tanh()
        off = off * (1 - inner ** 2) + cap * 2.0 ** -21
        s = cap * torch.tanh(s / cap)
    off = off + s.abs() * 4 * 2.0 ** -24
    see = torch.arange(T) <= (n0 + torch.arange(n))[:, None]
    if tokens is not None:
        see = see & tokens
    vis = see[:, None, None].expand_as(s)
    s = torch.where(vis, s, -math.inf)
    off = torch.where(vis, off, 0.0).amax(-1)
    w = s.softmax(-1)
    out = torch.einsum("nhgt,thd->nhgd", w, v)
    size = torch.einsum("nhgt,thd->nhgd", w, v.abs())
    apart = torch.zeros_like(out)
    for i in range(n):
        apart[i] = torch.einsum("hgt,thgd->hgd", w[i], (v[:, :, None] - out[i]).abs())
    u = 2.0 ** -8 if dtype is BF16 else 2.0 ** -16
    d = off.exp() * (1 + u) - 1
    assert float(d.max()) < 0.25, "the inputs leave no bound"
    tol = (d / (1 - d))[..., None] * apart + 2 * T * 2.0 ** -24 * size
    tol = (out.abs() + tol) * torch.finfo(dtype).eps / 2 + tol + torch.finfo(dtype).tiny
    lse = torch.logsumexp(s, -1)
    lse_tol = off + 1.01 * u + T * 2.0 ** -24 + 2.0 ** -22 * (1 + lse.abs())
    return out.flatten(1, 2), lse.flatten(1, 2), tol.flatten(1, 2), lse_tol.flatten(1, 2)


def check(k, v, q, P=64, scale=None, cap=0.0, exact=False):
    """k, v [n0 + n, H, D], q [n, Hq, D].  Also that the tolerance would tell: zeros, and the attention of every other token (the even
    ones or the odd ones), lie outside of it."""
    T, H, D = k.shape
    n = q.shape[0]
    scale = D ** -0.5 if scale is None else scale
    c = ref.Cache(1, H, D, P, -(-T // P), seed=1)
    h = handle(c)
    svx.sv_kv_write(h, k[None].to(DEV), v[None].to(DEV), i32(0))
    c.pool[0] = h.pool.cpu()
    kk, vv = c.tokens(0, T)
    if exact:
        assert torch.equal(kk, k.double())
    out, lse, tol, lse_tol = attention(q, kk, vv, T - n, scale, cap, q.dtype, exact)
    told = torch.zeros(n, q.shape[1], dtype=torch.bool)
    for odd in (0, 1):  # (a row that looks at one token alone misses only that one)
        other = attention(q, kk, vv, T - n, scale, cap, q.dtype, exact, torch.arange(T) % 2 == odd)[0]
        told |= ((out - other).abs() > tol).any(-1)
    assert bool(told.all())
    assert float((out.abs() > 2 * tol).double().mean()) > 0.8
    got = svx.sv_kv_attention(h, q[None].to(DEV), i32(T - n), scale=scale, cap=cap, want_lse=True)
    near(got["out"][0], out, tol, "out")
    near(got["lse"][0], lse, lse_tol, "lse")


def values(T, H, D, seed):
    return torch.randn(T, H, D, generator=torch.Generator().manual_seed(seed)) + 0.25


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(1, 1), (5, 4), (17, 8)])
def test_one_channel_far_above_the_others(n, G, D, dtype):
    """Keys and queries with a channel whose product is 2^17, the same for all tokens: it shifts all scores alike, and what the
    others say (products up to 6, multiples of 1/4) stays, those of its own block of 32 among them.  All sums have at most 24
    bits: 2^17 + 6 D and two places behind."""
    H, T = 2, 300 + n
    g = torch.Generator().manual_seed(D + n)
    k = torch.randint(-3, 4, (T, H, D), generator=g) * 0.5  # with a scale of an eighth or a quarter
    k[..., 32:64] *= 16  # with a scale of 16
    k[..., 37] = 64.0
    q = torch.randint(-4, 5, (n, H * G, D), generator=g) * 0.5
    q[..., 32:64] /= 8
    q[..., 37] = torch.where(torch.rand(n, H * G, generator=g) < 0.5, -1.0, 1.0) * 2048
    check(k, values(T, H, D, 1), q.to(dtype), exact=True)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_values_beside_large_ones_in_a_query(D, dtype):
    """A query's channel 2^20 (fp16: 2^15) times the others, where the keys are zero: the others make the scores."""
    H, G, n, T = 2, 3, 4, 200
    g = torch.Generator().manual_seed(D)
    k = torch.randn(T, H, D, generator=g)
    k[..., :32] = 0
    q = torch.randn(n, H * G, D, generator=g)
    q[..., 3] = 2.0 ** 20 if dtype is BF16 else 2.0 ** 15
    check(k, values(T, H, D, 2), q.to(dtype))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_large_scores_that_move_references(sign, rising, D, dtype):
    """Scores of hundreds, exact in 24 bits, rising (or falling) along the tokens by steps past which a reference moves, within a
    wave's tokens and from one block's to the next; the last ones, a few within e of one another, make the result."""
    H, G, n, T = 1, 4, 3, 2000
    g = torch.Generator().manual_seed(D)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    # channels 0 .. 31 climb by steps of 1/2 to 6 every (T / 12) tokens, beside queries of 64 in eight of them
    step = (torch.arange(T) * 8 // T) if rising else (7 - torch.arange(T) * 8 // T)
    k = torch.zeros(T, H, D)
    k[:, 0, :31] = grid[step][:, None]
    k[:, 0, 31] = 6.0  # the block's scale is 1 for every token
    small = torch.randint(-3, 4, (T, D - 32), generator=g) * 0.25
    k[:, 0, 32:] = small
    k[:, 0, 32::32] = 1.5  # and 1/4 for the others: 1.5 is 6 of them
    q = torch.zeros(n, G, D)
    q[..., :8] = 64.0 * torch.tensor([1.0, 2.0, 0.5, 1.5])[:, None]
    q[..., 32:] = torch.randint(-4, 5, (n, G, D - 32), generator=g) * 0.5
    for a in (1.0, 0.5):
        check(k, values(T, H, D, 3), (q * sign).to(dtype), P=16, scale=sign * a * D ** -0.5, exact=True)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("cap", [5.0, 30.0, 200.0])
def test_caps_at_their_ends(cap, dtype):
    """Scores from a tenth of a cap to several times it: tokens whose scores the cap makes alike count alike."""
    H, G, n, T, D = 2, 4, 4, 500, 128
    g = torch.Generator().manual_seed(int(cap))
    k = torch.randn(T, H, D, generator=g) * torch.exp2(torch.randint(-3, 4, (T, 1, 1), generator=g).float())
    q = torch.randn(n, H * G, D, generator=g) * cap / 8
    check(k, values(T, H, D, 4), q.to(dtype), cap=cap)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(1, 4), (40, 5)])
def test_ordinary_scores(n, G, D, dtype):
    """What the operator meets every day, against the tight bound; lengths that end inside a step."""
    H, T = 2, 777
    g = torch.Generator().manual_seed(D)
    k = torch.randn(T, H, D, generator=g)
    k[..., ::16] *= 4
    check(k, values(T, H, D, 5), queries(1, n, H * G, D, dtype, 5)[0], P=16)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(4, 1), (30, 4)])
def test_what_is_not_finite(n, G, D, dtype):
    """An infinity or NaN anywhere in a query makes its row NaN (also where all scores would be -inf, as beside keys of one sign),
    one in a key the rows that see its token, and no other row or head."""
    H, T, P = 2, 150 + n, 16
    g = torch.Generator().manual_seed(D + n)
    k, v = torch.rand(T, H, D, generator=g) + 0.5, values(T, H, D, 6)
    q = torch.randn(n, H * G, D, generator=g)
    c = ref.Cache(1, H, D, P, -(-T // P), seed=1)
    h = handle(c)
    for bad in (math.inf, -math.inf, math.nan):
        for at in (0, 1, 17, D // 2 + 7, D - 1):
            qq = q.clone()
            qq[n - 1, H * G - 1] = 0.0
            qq[n - 1, H * G - 1, at] = qq[0, 0, at] = bad
            svx.sv_kv_write(h, k[None].to(DEV), v[None].to(DEV), i32(0))
            got = svx.sv_kv_attention(h, qq[None].to(dtype).to(DEV), i32(T - n), want_lse=True)
            nan = torch.zeros(n, H * G, dtype=torch.bool)
            nan[n - 1, H * G - 1] = nan[0, 0] = True
            assert torch.equal(got["out"][0].cpu().isnan(), nan[..., None].expand(n, H * G, D)), (bad, at)
            assert torch.equal(got["lse"][0].cpu().isnan(), nan), (bad, at)
            # a key of the last head, of a node in the middle
            kk = k.clone()
            kk[T - n + n // 2, H - 1, at] = bad
            svx.sv_kv_write(h, kk[None].to(DEV), v[None].to(DEV), i32(0))
            got = svx.sv_kv_attention(h, q[None].to(dtype).to(DEV), i32(T - n), want_lse=True)
            nan = torch.zeros(n, H * G, dtype=torch.bool)
            nan[n // 2:, (H - 1) * G:] = True
            assert torch.equal(got["out"][0].cpu().isnan(), nan[..., None].expand(n, H * G, D)), (bad, at)
            assert torch.equal(got["lse"][0].cpu().isnan(), nan), (bad, at)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_least_and_largest_magnitudes(D, dtype):
    """Keys near the ends of the scales' range beside queries that bring their scores to ordinary size, and the type's least
    values beside large keys: nothing is flushed, nothing overflows."""
    H, G, n, T = 2, 2, 3, 100
    g = torch.Generator().manual_seed(D)
    for size in (2.0 ** -100, 2.0 ** 100) if dtype is BF16 else (2.0 ** -13, 2.0 ** 22):
        k = torch.randint(-3, 4, (T, H, D), generator=g) * size
        q = torch.randint(-4, 5, (n, H * G, D), generator=g) / size
        check(k.float(), values(T, H, D, 7), q.to(dtype), exact=True)
