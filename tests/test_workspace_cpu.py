"""The bindings' default workspace without a GPU: which buffer a call gets while a graph is captured, and what becomes of
one that is replaced.  Buffers are meta tensors; the capture is a flag that the tests set."""
import weakref

import pytest
import torch

from lossless_draft_verification_04_amd import specverify as svx

DEV = torch.device("meta", 0)
SMALL, LARGE = 1 << 16, 5 << 20
SHAPE = (svx.SV_DRAFT_TEACHER, svx.SV_BF16, 2048, 1, 151936, 64)  # needs more than the first buffer's 1 MiB


@pytest.fixture
def capture(monkeypatch):
    """Workspaces of their own, and a switch for 'the current stream is being captured'."""
    state = {"on": False}
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["on"])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for name in ("_cache", "_replaced"):
        monkeypatch.setattr(svx.Workspace, name, {}, raising=False)
    return lambda on: state.update(on=on)


def drafter_side(shape=SHAPE):
    return svx._draft_workspace(DEV, *shape)


def test_the_shape_outgrows_the_first_buffer():
    assert svx.draft_workspace_size(*SHAPE) > 1 << 20


def test_drafter_calls_take_the_default_that_is_there(capture):
    first = drafter_side()
    capture(True)
    assert drafter_side() is first and svx.Workspace.get(DEV, SMALL) is first


def test_drafter_calls_refuse_to_make_the_default_in_a_capture(capture):
    capture(True)
    with pytest.raises(svx.SpecVerifyError) as e:
        drafter_side()
    assert e.value.status == svx.SV_EWORKSPACE and "workspace=" in str(e.value)
    assert not svx.Workspace._cache  # nothing is left for later calls
    capture(False)
    assert drafter_side().numel() >= svx.draft_workspace_size(*SHAPE)


def test_drafter_calls_refuse_to_grow_the_default_in_a_capture(capture):
    first = svx.Workspace.get(DEV, SMALL)
    capture(True)
    with pytest.raises(svx.SpecVerifyError):
        drafter_side()
    assert svx.Workspace.get(DEV, SMALL) is first


def test_a_buffer_of_a_graph_is_no_default(capture):
    """What is made in a capture is zero only once the graph has run: calls outside it get another buffer."""
    capture(True)
    born = svx.Workspace.get(DEV, LARGE)
    capture(False)
    eager = drafter_side()
    assert eager is not born and svx.Workspace.get(DEV, SMALL) is eager


def test_a_replaced_buffer_stays_alive(capture):
    first = svx.Workspace.get(DEV, SMALL)
    alive = weakref.ref(first)
    del first
    large = svx.Workspace.get(DEV, LARGE)
    assert alive() is not None and large.numel() >= LARGE
    assert svx.Workspace.get(DEV, SMALL) is large


def test_replaced_buffers_take_less_than_the_default(capture):
    n, total = 1 << 20, []
    for _ in range(200):
        ws = svx.Workspace.get(DEV, n)
        if not total or total[-1] != ws.numel():
            total.append(ws.numel())
        n += 1 << 18
    assert sum(total[:-1]) <= total[-1]


def test_the_error_word_of_every_buffer_is_read(capture, monkeypatch):
    """A graph that keeps a replaced buffer reports its errors as before."""
    small = svx.Workspace.get(DEV, SMALL)
    capture(True)
    born = svx.Workspace.get(DEV, LARGE)
    capture(False)
    large = svx.Workspace.get(DEV, LARGE)
    words = {id(small): svx.DERR_TOKEN, id(born): svx.DERR_ROW, id(large): svx.DERR_RANGE}
    monkeypatch.setattr(svx, "_ptr", lambda t: id(t))
    monkeypatch.setattr(svx, "_stream", lambda d: None)

    class Lib:
        @staticmethod
        def sv_get_device_error(ws, flags, stream):
            flags._obj.value = words.pop(ws)
            return svx.SV_OK

    monkeypatch.setattr(svx, "_lib", Lib)
    assert svx.sv_get_device_error(DEV) == svx.DERR_TOKEN | svx.DERR_ROW | svx.DERR_RANGE and not words
