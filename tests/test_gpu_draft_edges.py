"""Drafter-side operators where 64-bit scores no longer tell logits apart, and where a thread adds up thousands of
terms."""
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
