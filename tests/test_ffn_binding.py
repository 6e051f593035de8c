"""The binding of the feed-forward calls without a GPU: which stream a
workspace is allocated on and tied to, with stand-ins for the library's entry
points and for torch's streams."""
import contextlib
import types

import pytest

from tests.test_ffn_cpu import _handle

svq = pytest.importorskip("bit_spherical_vector_amd.svq")
torch = pytest.importorskip("torch")

CPU = torch.device("cpu")


class Stream:
    def __init__(self, handle, device=CPU):
        self.cuda_stream, self.device, self.waited = handle, device, []

    def wait_stream(self, other):
        self.waited.append(other)


class Memory:
    """What torch.empty returns: where it was allocated and recorded."""

    def __init__(self, nbytes, stream):
        self.nbytes, self.stream, self.recorded, self.device = nbytes, stream, [], CPU

    numel = lambda self: self.nbytes
    element_size = lambda self: 1
    data_ptr = lambda self: 0x4000
    is_contiguous = lambda self: True

    def record_stream(self, stream):
        self.recorded.append(stream)


@pytest.fixture
def gpu(monkeypatch):
    """Stand-ins: ``gpu.current`` is the current stream, ``gpu.calls`` the
    launches as (name, workspace address, stream)."""
    g = types.SimpleNamespace(current=Stream(0), calls=[], capturing=False)

    @contextlib.contextmanager
    def on(stream):
        before, g.current = g.current, stream
        yield
        g.current = before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                *_, ws, size, stream = args
                if ws is None:
                    size._obj.value = 512
                else:
                    g.calls.append((name, ws, stream))
                return svq.SVQ_OK
            return call

    monkeypatch.setattr(svq, "LIB", Library())
    cuda = torch.cuda
    for name, value in dict(device=lambda d: contextlib.nullcontext(), stream=on, current_stream=lambda d=None: g.current,
                            current_device=lambda: None, is_current_stream_capturing=lambda: g.capturing).items():
        monkeypatch.setattr(cuda, name, value)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: g.current.cuda_stream, raising=False)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: Memory(a[0], g.current) if k.get("dtype") == torch.uint8
                        else empty(*a, **k))
    return g


def _call(**over):
    pm = svq.PackedMatrix(None, _handle(96, 520))
    x, y = torch.zeros((3, 520), dtype=torch.bfloat16), torch.zeros((3, 96), dtype=torch.bfloat16)
    return svq.EpilogueCall(pm, x, y, **over)


def test_workspace_of_the_current_stream(gpu):
    call = _call()
    call()
    call()
    assert call.workspace.stream is gpu.current and call.workspace.recorded == []
    assert gpu.calls == [("svq_linear_epilogue", 0x4000, 0)] * 2


def test_workspace_of_the_given_stream(gpu):
    s = Stream(7)
    call = _call(stream=s)
    call()
    assert call.workspace.stream is s and call.workspace.recorded == []
    assert gpu.calls == [("svq_linear_epilogue", 0x4000, 7)]


def test_called_under_another_stream(gpu):
    home, s = gpu.current, Stream(7)
    call = _call()
    with torch.cuda.stream(s):
        call()
        call()
    call()
    assert call.workspace.stream is home
    assert s.waited == [home] and call.workspace.recorded == [s]  # once, before the first call there
    assert [c[2] for c in gpu.calls] == [7, 7, 0]


def test_captured_under_another_stream(gpu):
    """No wait inside a capture; a later eager call there still waits."""
    home, s = gpu.current, Stream(7)
    call = _call()
    with torch.cuda.stream(s):
        gpu.capturing = True
        call()
        assert s.waited == [] and call.workspace.recorded == [s]
        gpu.capturing = False
        call()
    assert s.waited == [home]


def test_given_workspace(gpu):
    """The caller's own: used as it is, on whatever stream; replaced when it
    is too small; refused when the kernels could not use it."""
    given = Memory(512, None)
    call = _call(workspace=given)
    with torch.cuda.stream(Stream(7)):
        call()
    assert call.workspace is given and given.recorded == []
    small = Memory(511, None)
    assert _call(workspace=small).workspace.stream is gpu.current
    with pytest.raises(ValueError, match="workspace must be a contiguous tensor"):
        _call(workspace=torch.zeros(4096, dtype=torch.uint8)[::2])
    elsewhere = Memory(512, None)
    elsewhere.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="workspace must be a contiguous tensor"):
        _call(workspace=elsewhere)
    with pytest.raises(ValueError, match="stream is one of"):
        _call(stream=Stream(7, torch.device("cuda", 1)))
