"""Drafter-side operators where 64-bit scores no longer tell logits apart, where a thread adds up thousands of terms,
in place where a block walks several rows, and past 4 GiB of rows."""
import math

import pytest
import torch

from lossless_draft_verification_04_amd import specverify as svx
from tests import draft_ref as ref
from tests.test_gpu_draft import DEV, beam_scores, near, put, rows

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
INF = math.inf


@pytest.fixture(autouse=True)
def no_device_error():
    svx.sv_get_device_error(DEV)
    yield
    assert svx.sv_get_device_error(DEV) == 0


# ---------------------------------------------------------------------------
# beams whose score is a large finite number, as a stand-in for a dead beam
# ---------------------------------------------------------------------------
def far_beams(x, scores, N, finished, pad):
    """The N best of [W, V] rows: by 64-bit score, then beam; within a beam by logit, then token."""
    out = []
    for w in range(x.shape[0]):
        s = float(scores[w])
        if s == -INF:
            continue
        if finished[w]:
            out.append((-s, w, 0, pad))
            continue
        z = x[w].double()
        lse = float(z.logsumexp(-1))
        v, i = z.sort(descending=True, stable=True)
        out += [(-(s - lse + float(v[j])), w, j, int(i[j])) for j in range(min(N, int((v > -INF).sum())))]
    return sorted(out)[:N]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("far", [-1e30, torch.finfo(F32).min])
@pytest.mark.parametrize("Wd,V,N", [(4, 50, 8), (5, 20011, 64), (64, 515, 33), (3, 152064, 20)])
def test_beams_far_below_the_others(Wd, V, N, far, dtype):
    """Next to finished beams the far ones' continuations fill the places that are left: beam by beam, each in its own
    order."""
    B = 3
    x = rows(B * Wd, V, dtype, V + N).view(B, Wd, V)
    s = torch.full((B, Wd), far)
    fin = torch.zeros(B, Wd, dtype=torch.int32)
    s[0, Wd - 1], fin[0, Wd - 1] = -3.0, 1          # one finished beam
    s[1, 1], s[1, 2], fin[1, 2] = -2.0, -1.0, 1     # a living one that has few tokens, and a finished one
    x[1, 1, 5:] = -INF
    s[2, 0] = -INF                                  # nothing but far ones
    got = svx.sv_beam_select(put(x), s.to(DEV), N, 1.0, finished=fin.to(DEV), pad_tok=7)
    for b in range(B):
        want = far_beams(x[b], s[b], N, fin[b].tolist(), 7)
        want += [(INF, -1, 0, -1)] * (N - len(want))
        assert got["beam"][b].tolist() == [c[1] for c in want], b
        assert got["tok"][b].tolist() == [c[3] for c in want], b
        near(got["score"][b], torch.tensor([-c[0] for c in want], dtype=torch.float64),
             ref.SUM + 2.0 ** -24 * torch.tensor([abs(c[0]) if c[0] < INF else 0.0 for c in want]), "score")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("far", [1e14, 1e16, 1e18])
def test_beams_whose_scores_tie_in_part(far, dtype):
    """Scores a few steps apart: the list falls, and every beam's tokens come in the order of its logits."""
    B, Wd, V, N = 4, 6, 20011, 50
    x = rows(B * Wd, V, dtype, 77).view(B, Wd, V)
    s = -far * (1 + torch.rand(B, Wd, generator=torch.Generator().manual_seed(78)).mul_(2.0 ** -20))
    got = {k: v.cpu() for k, v in svx.sv_beam_select(put(x), s.to(DEV), N, 1.0).items()}
    for b in range(B):
        assert bool((got["score"][b][1:] <= got["score"][b][:-1]).all()) and int(got["beam"][b].min()) >= 0
        for w in range(Wd):
            mine = got["tok"][b][got["beam"][b] == w].tolist()
            assert mine == x[b, w].double().sort(descending=True, stable=True)[1][: len(mine)].tolist(), (b, w)


# ---------------------------------------------------------------------------
# rows whose parts are read a second time, thousands of vectors a thread
# ---------------------------------------------------------------------------
def second_read(V, threads, parts, bulk):
    """fp32 logits whose mass outside the listed values has to be summed again: a thread of every wave owns two listed
    values, in different vectors, that outweigh all the rest by e^40.  Returns the row and the number of listed values."""
    x = bulk.clone()
    per = V // 4 // parts  # vectors of a part
    n = 0
    for p in range(parts):
        for w in range(threads // 64):
            for j in (100, 900):
                v = p * per + w * 64 + 5 + j * threads
                x[4 * v + j % 4] = 60.0 + 0.25 * (n % 4)
                n += 1
    return x, n


def one_above(V, threads, parts, above):
    """Zeros, and one value above them in every thread's first vector, against which the thread's sum is formed."""
    x = torch.zeros(V)
    per = V // 4 // parts
    for p in range(parts):
        x[4 * p * per: 4 * (p * per + threads): 4] = above
    return x


BULKS = [2.8, 4.95, 3.31, 1.4, "rising", "falling", "normal", "steps"]


def bulk_of(kind, V, threads, parts):
    if kind == "rising":
        return torch.linspace(0, 3, V)
    if kind == "falling":
        return torch.linspace(3, 0, V)
    if kind == "normal":
        return torch.randn(V, generator=torch.Generator().manual_seed(3))
    if kind == "steps":  # from 2^-170 to the largest in jumps of 2^1 to 2^80
        at = torch.tensor([-118.0, -80.0, -79.0, -40.0, -38.0, -16.0, 0.0, 5.0])
        return at[torch.arange(V) // (V // 4) % 4 * 2 + torch.arange(V) // (V // 8) % 2]
    return one_above(V, threads, parts, kind)


@pytest.mark.parametrize("kind", BULKS)
def test_long_row_read_twice(kind):
    """2^24 logits in 4 parts of 512 threads: 2048 vectors a thread."""
    V, k = 1 << 24, 64
    x, n = second_read(V, 512, 4, bulk_of(kind, V, 512, 4))
    assert n == k
    got = svx.sv_teacher_topk(x[None].to(DEV), k, 1.0)
    ids, vals, rest = ref.teacher(x[None], k, 1.0)
    assert torch.equal(got["ids"].cpu().long(), ids)
    near(got["rest"], rest, ref.SUM + 2.0 ** -24 * rest.abs(), "rest")


@pytest.mark.parametrize("kind", BULKS)
def test_long_rows_read_twice(kind):
    """257 rows of 2^21 logits, a block of 256 threads each: 2048 vectors a thread; and beams of such rows."""
    V, R = 1 << 21, 257
    x, k = second_read(V, 256, 1, bulk_of(kind, V, 256, 1))
    z = x.to(DEV).expand(R, V).contiguous()
    got = svx.sv_teacher_topk(z, k, 1.0)
    ids, vals, rest = ref.teacher(x[None], k, 1.0)
    assert torch.equal(got["ids"].cpu().long(), ids.expand(R, k))
    near(got["rest"], rest.expand(R), ref.SUM + 2.0 ** -24 * rest.abs().expand(R), "rest")
    out = svx.sv_beam_select(z[:, None], torch.zeros(R, 1, device=DEV), k)
    assert torch.equal(out["tok"].cpu().long(), ids.expand(R, k))
    score = vals - x.double().logsumexp(-1)
    near(out["score"], score.expand(R, k), ref.SUM + 2.0 ** -24 * score.abs().expand(R, k), "score")


# ---------------------------------------------------------------------------
# loss and gradient in place where a block walks several rows, and rows past 4 GiB
# ---------------------------------------------------------------------------
def teacher_of(z, k, seed):
    """k distinct tokens of every row, some rows without a target."""
    R, V = z.shape
    g = torch.Generator(device=DEV).manual_seed(seed)
    ids = ((torch.randint(0, V, (R, 1), generator=g, device=DEV) + torch.arange(k, device=DEV) * (V // k)) % V).int()
    vals = torch.randn(R, k, generator=g, device=DEV) + 9
    rest = torch.rand(R, generator=g, device=DEV) * 4 + math.log(V)
    ids[5::7], rest[5::7] = -1, -INF
    return ids, vals, rest, torch.rand(R, generator=g, device=DEV)


@pytest.mark.parametrize("dtype,R,V", [(BF16, 3000, 1031), (F32, 1700, 8003), (BF16, 1300, 30011), (BF16, 600, 128256),
                                       (F32, 600, 60001), (BF16, 600, 147456), (BF16, 600, 160003), (BF16, 600, 180003),
                                       (BF16, 600, 196608), (F32, 600, 98304)])
def test_in_place_gives_the_bits_of_apart(dtype, R, V):
    g = torch.Generator(device=DEV).manual_seed(V)
    z = put(torch.randn(R, V, generator=g, device=DEV).mul_(2).to(dtype))
    ids, vals, rest, w = teacher_of(z, 24, R)
    apart = svx.sv_distill_topk(z, ids, vals, 1.0, rest=rest, grad_loss=w, want_grad=True)
    want = apart["grad"].clone()
    got = svx.sv_distill_topk(z, ids, vals, 1.0, rest=rest, grad_loss=w, grad=z)
    assert got["grad"] is z and torch.equal(z, want)
    assert torch.equal(got["loss"], apart["loss"]) and torch.equal(got["stat"], apart["stat"])
    assert float(want.abs().amax()) > 0


@pytest.mark.parametrize("dtype,R,V", [(BF16, 18001, 128256), (F32, 600, 1 << 21)])
def test_rows_past_4_gib(dtype, R, V):
    """The last rows, in every entry point over rows; by a block a row that holds it, and in two launches."""
    z = torch.zeros(R, V, dtype=dtype, device=DEV)
    assert z.numel() * z.element_size() > 1 << 32
    last = rows(3, V, dtype, 5)
    z[-3:] = last.to(DEV)
    k, T = 16, 1.0
    got = svx.sv_teacher_topk(z, k, T)
    ids, vals, rest = ref.teacher(last, k, T)
    assert torch.equal(got["ids"][-3:].cpu().long(), ids)
    near(got["rest"][-3:], rest, ref.SUM + 2.0 ** -24 * rest.abs(), "rest")
    out = svx.sv_beam_select(z[:, None], torch.zeros(R, 1, device=DEV), k)
    assert torch.equal(out["tok"][-3:].cpu().long(), ids)
    target = got["ids"], got["vals"] + 0.25 * torch.arange(k, device=DEV), got["rest"]
    loss, stat, grad, size = ref.distill(last, *(t[-3:].cpu() for t in target), T)
    tol = 3e-5 * size + ref.HALF[dtype] * grad.abs() + 1e-37
    fwd = svx.sv_distill_topk(z, *target[:2], T, rest=target[2])
    near(fwd["loss"][-3:], loss, 2 * ref.SUM + 2.0 ** -23 * loss.abs(), "loss")
    near(svx.sv_distill_topk_backward(z, *target[:2], fwd["stat"], T, rest=target[2])[-3:], grad, tol, "backward")
    both = svx.sv_distill_topk(z, *target[:2], T, rest=target[2], grad=z)
    near(both["loss"][-3:], loss, 2 * ref.SUM + 2.0 ** -23 * loss.abs(), "loss")
    near(z[-3:], grad, tol, "in place")
