"""The bindings' default workspace beside captured graphs: captured before any eager call, and replaced after a capture."""
import pytest
import torch

from lossless_draft_verification_04_amd import specverify as svx

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture
def fresh(monkeypatch):
    """As in a process that has made no call yet."""
    torch.cuda.synchronize()
    monkeypatch.setattr(svx.Workspace, "_cache", {})
    monkeypatch.setattr(svx.Workspace, "_replaced", {})
    yield
    torch.cuda.synchronize()


def rows(R, V, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(R, -(-V // 8) * 8, generator=g, device=DEV).bfloat16()[:, :V]


def bits(out):
    return {k: v.clone().view(torch.uint8) for k, v in out.items()}


def same(a, b):
    return a.keys() == b.keys() and all(torch.equal(a[k], b[k]) for k in a)


def test_captured_before_any_call(fresh):
    """A drafter-side call is refused there; the next eager one, whose rows are split over blocks, is whole."""
    z = rows(3, 150011, 1)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(svx.SpecVerifyError) as e:
        with torch.cuda.graph(graph):
            svx.sv_teacher_topk(z, 24, 1.0)
    assert e.value.status == svx.SV_EWORKSPACE
    del graph
    got = svx.sv_teacher_topk(z, 24, 1.0)
    own = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)
    assert same(bits(got), bits(svx.sv_teacher_topk(z, 24, 1.0, workspace=own)))
    assert svx.sv_get_device_error(DEV) == 0


def test_a_verification_captured_before_any_call(fresh):
    """It runs in a buffer of the graph's, which eager calls before the first replay do not meet."""
    tgt = rows(4 * 6, 30011, 2).unflatten(0, (4, 6))
    tok = torch.randint(0, 30011, (4, 5), device=DEV, dtype=torch.int32)
    z = rows(3, 150011, 3)
    own = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)
    want = bits(svx.sv_verify_greedy(tgt, tok, workspace=own))
    want_z = bits(svx.sv_teacher_topk(z, 24, 1.0, workspace=own))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = svx.sv_verify_greedy(tgt, tok)
    for _ in range(3):
        assert same(bits(svx.sv_teacher_topk(z, 24, 1.0)), want_z)
        for v in out.values():
            v.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert same(bits(out), want)
    assert svx.sv_get_device_error(DEV) == 0


def test_replaced_after_a_capture(fresh):
    """A larger eager call replaces the buffer of a capture: replays go on in it, and tensors made since keep their
    values; an error that a replay finds is read."""
    z = rows(3, 150011, 4)
    ids = torch.zeros(2, 4, dtype=torch.int32, device=DEV)  # repeated ids
    vals, few = torch.zeros(2, 4, device=DEV), rows(2, 1000, 5)
    want = bits(svx.sv_teacher_topk(z, 24, 1.0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = svx.sv_teacher_topk(z, 24, 1.0)
        svx.sv_distill_topk(few, ids, vals, 1.0)
    first = svx.Workspace.get(DEV, 0)
    svx.sv_teacher_topk(rows(2048, 30000, 6), 64, 1.0)
    assert svx.Workspace.get(DEV, 0) is not first
    kept = [torch.full((1 << 20,), 3, dtype=torch.uint8, device=DEV) for _ in range(8)]
    for _ in range(3):
        for v in out.values():
            v.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert same(bits(out), want)
        assert same(bits(svx.sv_teacher_topk(z, 24, 1.0)), want)
        assert svx.sv_get_device_error(DEV) == svx.DERR_TOKEN
    assert all(int(t.min()) == 3 and int(t.max()) == 3 for t in kept)


def test_captured_before_any_call_in_a_workspace_of_its_own(fresh):
    z = rows(3, 150011, 7)
    own = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = svx.sv_teacher_topk(z, 24, 1.0, workspace=own)
    want = bits(svx.sv_teacher_topk(z, 24, 1.0))
    for _ in range(3):
        for v in out.values():
            v.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert same(bits(out), want)
