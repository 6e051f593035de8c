"""The binding of the feed-forward calls without a GPU: which stream a
workspace is allocated on and tied to, with stand-ins for the library's entry
points and for torch's streams; and the operands that it refuses, each by its
own message beside a call that passes."""
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


@pytest.fixture
def prepared(monkeypatch):
    """What a call object hands to the library, in place of the call."""
    seen = []
    monkeypatch.setattr(svq._Call, "_prepare", lambda self, name, args, *rest: seen.append((name, args)))
    return seen


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


PM, SQUARE = svq.PackedMatrix(None, _handle(96, 520)), svq.PackedMatrix(None, _handle(520, 520))
WIDE = z(4, 96)


@pytest.mark.parametrize("over,message", [
    ({}, None), (dict(y=z(3, 96, dtype=torch.float32)), None), (dict(bias=z(96)), None), (dict(x=z(3, 600)), None),
    (dict(residual=z(3, 100)[:, 2:98]), None),
    (dict(x=z(3, 520, dtype=torch.float32)), "x has the wrong type"), (dict(x=z(3, 512)), "x must be 2-D, 3 rows of 520"),
    (dict(x=z(520, 3).t()), "x must be 2-D"), (dict(x=z(3 * 520)[:520]), "x must be 2-D"),
    (dict(y=z(3, 96, dtype=torch.float16)), "y has the wrong type"), (dict(y=z(2, 96)), "y must be 2-D, 3 rows"),
    (dict(y=z(3, 95)), "y must be 2-D, 3 rows of 96"), (dict(bias=z(95)), "bias must be a contiguous vector of 96"),
    (dict(bias=z(192)[::2]), "bias must be a contiguous vector"),
    (dict(bias=z(96, dtype=torch.float64)), "bias must be bf16 or fp32"), (dict(act="swish"), "act must be one of"),
    (dict(residual=z(3, 90)), "residual must be 2-D"), (dict(residual=z(3, 96, dtype=torch.float64)), "residual has the wrong"),
    (dict(residual=z(300).unfold(0, 96, 95)[:3]), "rows of residual overlap"),
    (dict(y=WIDE[:3], residual=WIDE[:3]), None), (dict(y=WIDE[:3], residual=WIDE[1:]), "residual overlaps y"),
    (dict(y=z(3, 96).cpu(), residual=torch.zeros((3, 96), device="meta")), "residual is on meta"),
])
def test_epilogue_operands(prepared, over, message):
    args = dict(x=z(3, 520), y=z(3, 96))
    args.update(over)
    if message is None:
        svq.EpilogueCall(PM, **args)
        assert len(prepared) == 1
        return
    with pytest.raises(ValueError, match=message):
        svq.EpilogueCall(PM, **args)
    assert not prepared


@pytest.mark.parametrize("over,message", [
    ({}, None), (dict(bias_up=z(96, dtype=torch.float32)), None), (dict(up=PM), None),
    (dict(x=z(3, 519)), "x must be 2-D"), (dict(x=z(4, 520)), "y must be 2-D, 4 rows"),
    (dict(y=z(3, 96, dtype=torch.int16)), "y has the wrong type"), (dict(bias_gate=z(97)), "bias_gate must be a contiguous"),
    (dict(bias_gate=z(96), bias_up=z(96, dtype=torch.float32)), "of one type"), (dict(act="silu2"), "act must be one of"),
])
def test_glu_operands(prepared, over, message):
    args = dict(up=PM, x=z(3, 520), y=z(3, 96))
    args.update(over)
    if message is None:
        svq.GluCall(PM, args.pop("up"), **args)
        assert len(prepared) == 1
        return
    with pytest.raises(ValueError, match=message):
        svq.GluCall(PM, args.pop("up"), **args)


@pytest.mark.parametrize("over,message", [
    ({}, None), (dict(w=z(4, 520, dtype=torch.float32)), None), (dict(select_bias=z(4, dtype=torch.float32)), None),
    (dict(ids=z(3, 2, dtype=torch.int64)), "ids must be a contiguous torch.int32"),
    (dict(ids=z(3, 4, dtype=torch.int32)[:, ::2]), "ids must be a contiguous"),
    (dict(weights=z(3, 2)), "weights must be a contiguous torch.float32"),
    (dict(weights=z(2, 3, dtype=torch.float32)), "weights must be a contiguous"),
    (dict(w=z(4, 520, dtype=torch.float16)), "w has the wrong type"), (dict(x=z(3, 512)), "x must be 2-D"),
    (dict(x=z(2, 520)), "x must be 2-D, 3 rows"), (dict(select_bias=z(4)), "select_bias must be torch.float32"),
    (dict(select_bias=z(5, dtype=torch.float32)), "select_bias must be a contiguous"), (dict(score="tanh"), "score must be one of"),
])
def test_route_operands(prepared, over, message):
    args = dict(x=z(3, 520), w=z(4, 520), ids=z(3, 2, dtype=torch.int32), weights=z(3, 2, dtype=torch.float32))
    args.update(over)
    if message is None:
        svq.MoeRouteCall(**args)
        assert len(prepared) == 1
        return
    with pytest.raises(ValueError, match=message):
        svq.MoeRouteCall(**args)


@pytest.mark.parametrize("over,message", [
    ({}, None), (dict(residual=z(3, 520, dtype=torch.float32)), None), (dict(downs=[]), "sequences of one length"),
    (dict(gates=[], ups=[], downs=[]), "sequences of one length"), (dict(ups=[PM] * 2), "sequences of one length"),
    (dict(expert_ids=z(2, 2, dtype=torch.int32)), "x must be 2-D, 2 rows"),
    (dict(expert_ids=z(3, 2, dtype=torch.int64)), "expert_ids must be a contiguous torch.int32"),
    (dict(weights=z(3, 2, dtype=torch.float64)), "weights must be a contiguous torch.float32"),
    (dict(weights=z(3, 1, dtype=torch.float32)), "weights must be a contiguous"), (dict(y=z(3, 519)), "y must be 2-D"),
    (dict(residual=z(3, 519)), "residual must be 2-D"), (dict(act="x"), "act must be one of"),
])
def test_expert_layer_operands(prepared, over, message):
    down = svq.PackedMatrix(None, _handle(520, 96))
    args = dict(gates=[PM], ups=[PM], downs=[down], x=z(3, 520), expert_ids=z(3, 2, dtype=torch.int32),
                weights=z(3, 2, dtype=torch.float32), y=z(3, 520))
    args.update(over)
    if message is None:
        svq.MoeFfnCall(**args)
        assert len(prepared) == 1
        return
    with pytest.raises(ValueError, match=message):
        svq.MoeFfnCall(**args)


def test_outputs_over_the_activations(prepared):
    """An output over x is refused, except an expert layer's that is x itself;
    columns of one wider buffer do not overlap."""
    wide = z(4, 1100)
    x = wide[:3, :520]
    other = z(3, 520)
    call = lambda y, **over: svq.EpilogueCall(SQUARE, x, y, **over)
    call(wide[:3, 520:1040])
    call(wide[:3, 580:])
    call(wide[:3, 520:1040], residual=wide[:3, 520:1040])
    call(other, residual=x)  # the residual may be x
    call(wide[:3, 520:1040], residual=x)
    assert len(prepared) == 5
    for y in (x, wide[1:, :520], wide[:3, 519:1039], wide[1:, 4:524], wide.view(-1)[1000:1000 + 3 * 520].view(3, 520)):
        with pytest.raises(ValueError, match="y overlaps x"):
            call(y)
        with pytest.raises(ValueError, match="y overlaps x"):
            svq.GluCall(SQUARE, SQUARE, x, y)
    with pytest.raises(ValueError, match="residual overlaps y"):
        svq.EpilogueCall(SQUARE, other, wide[:3, 520:1040], residual=wide[:3, 519:1039])
    ids, wt = z(3, 2, dtype=torch.int32), z(3, 2, dtype=torch.float32)
    moe = lambda y, **over: svq.MoeFfnCall([SQUARE], [SQUARE], [SQUARE], x, ids, wt, y, **over)
    before = len(prepared)
    moe(x)
    moe(x, residual=x)
    moe(wide[:3, 520:1040])
    assert len(prepared) == before + 3
    for y in (wide[1:, :520], wide[:3, 1:521]):
        with pytest.raises(ValueError, match="y overlaps x"):
            moe(y)
    # one row: the row strides say nothing
    one = wide[:1, :520]
    svq.MoeFfnCall([SQUARE], [SQUARE], [SQUARE], one, ids[:1], wt[:1], one)
    with pytest.raises(ValueError, match="y overlaps x"):
        svq.EpilogueCall(SQUARE, one, wide[:1, 519:1039])
