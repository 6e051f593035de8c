"""The feed-forward calls (include/svq_ffn.h) on a host without a GPU: the
library exports them, answers workspace queries and refuses bad arguments
before any device work."""
import ctypes
import os
import re

import pytest

from tests.conftest import ROOT

svq = pytest.importorskip("bit_spherical_vector_amd.svq")

BAD, UNSUPPORTED, SMALL = svq.SVQ_ERR_INVALID_ARG, svq.SVQ_ERR_UNSUPPORTED, svq.SVQ_ERR_BUFFER_TOO_SMALL
FAKE = 0x100000  # a non-null device address; no refused call reads it


def _handle(n, k, bd=7):
    """A handle as svq_pack fills it, over an address that is never read."""
    al = lambda v: (v + 255) // 256 * 256
    h = svq.Handle()
    h.dev, h.n, h.k, h.bd, h.br = FAKE, n, k, bd, 10 - bd
    h.n_tiles, h.units = (n + 15) // 16, (k + 511) // 512
    off = 0
    for name, size in (("off_dtab", 4096), ("off_rtab", 2048), ("off_btab", 16384), ("off_xtab", 32768),
                       ("off_perm", h.units * 1024), ("off_codes", h.n_tiles * h.units * 2304)):
        setattr(h, name, off)
        off += al(size)
    h.bytes = off
    return h


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "svq_ffn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"\b(svq_[a-z_]+)\s*\(", text))
    assert declared == set(svq.EXPORTED_FFN)
    for name in declared:
        assert hasattr(svq.LIB, name)


def _call(fn, args, names, ws, nbytes, **over):
    vals = dict(zip(names, args))
    vals.update(over)
    size = ctypes.c_size_t(nbytes)
    return fn(*[vals[n] for n in names], ws, ctypes.byref(size), None), size.value


EPI_NAMES = ("w", "x", "m", "ldx", "ep", "y", "ldy", "ydt")


def _epilogue(ws=None, nbytes=0, handle=None, fields=None, **over):
    h = handle or _handle(96, 520)
    e = svq.Epilogue(**(fields or {}))
    return _call(svq.LIB.svq_linear_epilogue,
                 (ctypes.byref(h), FAKE, 3, 520, ctypes.byref(e), FAKE, 96, svq.SVQ_F32), EPI_NAMES, ws, nbytes,
                 **over)


def test_epilogue_query_matches_linear():
    st, need = _epilogue(m=1, x=None, y=None)
    assert st == 0 and need > 0
    for m in (1, 3):
        st, need = _epilogue(m=m)
        st2, plain = svq.svq_linear(_handle(96, 520), None, m, 520, None, 96, svq.SVQ_F32, None, 0, 0)
        assert (st, st2) == (0, 0) and need == plain
    for m in (9, 16, 17, 40, 300):
        st, need = _epilogue(m=m, x=None, y=None)
        assert st == 0 and _epilogue(ws=FAKE, nbytes=need - 1, m=m)[0] == SMALL


@pytest.mark.parametrize("over,ep,want", [
    (dict(ep=None), {}, BAD), (dict(w=None), {}, BAD), (dict(m=0), {}, BAD), (dict(ldx=519), {}, BAD),
    (dict(ldy=95), {}, BAD), (dict(ydt=2), {}, BAD), ({}, dict(act=5), BAD), ({}, dict(act=-1), BAD),
    ({}, dict(bias=FAKE, bias_dt=3), BAD), ({}, dict(residual=FAKE, ldr=95), BAD),
    ({}, dict(residual=FAKE, ldr=96, residual_dt=7), BAD),
    ({}, dict(residual=FAKE, ldr=97, residual_dt=1), BAD),  # y itself, with another stride
    ({}, dict(residual=FAKE, ldr=96, residual_dt=0), BAD),  # y itself, with another type
    (dict(x=None), {}, BAD), (dict(y=None), {}, BAD),
])
def test_epilogue_refusals(over, ep, want):
    st, _ = _epilogue(ws=FAKE, nbytes=1 << 30, fields=ep, **over)
    assert st == want


def test_epilogue_refuses_small_workspace_and_bad_handle():
    assert _epilogue(ws=FAKE, nbytes=10)[0] == SMALL
    h = _handle(96, 520)
    h.off_codes += 256
    assert _epilogue(handle=h)[0] == BAD


GLU_NAMES = ("gate", "up", "x", "m", "ldx", "act", "bg", "bu", "bdt", "y", "ldy", "ydt")


def _glu(ws=None, nbytes=0, gate=None, up=None, **over):
    g, u = gate or _handle(96, 520), up or _handle(96, 520, 8)
    return _call(svq.LIB.svq_linear_glu,
                 (ctypes.byref(g), ctypes.byref(u), FAKE, 3, 520, 2, None, None, 1, FAKE, 96, 0), GLU_NAMES, ws,
                 nbytes, **over)


@pytest.mark.parametrize("over,want", [
    (dict(gate=_handle(96, 512)), BAD), (dict(up=_handle(95, 520)), BAD), (dict(m=0), BAD), (dict(act=9), BAD),
    (dict(bg=FAKE, bdt=4), BAD), (dict(ldx=512), BAD), (dict(ldy=90), BAD), (dict(ydt=-1), BAD),
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(m=1 << 25), BAD),
])
def test_glu_refusals(over, want):
    assert _glu(ws=FAKE, nbytes=1 << 34, **over)[0] == want


def test_glu_workspace():
    for m in (1, 2, 5, 17, 300):
        st, need = _glu(m=m, x=None, y=None)
        assert st == 0 and need > 0
        assert _glu(ws=FAKE, nbytes=need - 1, m=m)[0] == SMALL


ROUTE_NAMES = ("x", "m", "ldx", "w", "wdt", "e", "k", "ldw", "sb", "score", "renorm", "scale", "topk", "ids", "wt")


def _route(ws=None, nbytes=0, **over):
    return _call(svq.LIB.svq_moe_route,
                 (FAKE, 3, 64, FAKE, 0, 16, 64, 64, None, 0, 1, 1.0, 4, FAKE, FAKE), ROUTE_NAMES, ws, nbytes, **over)


@pytest.mark.parametrize("over,want", [
    (dict(m=0), BAD), (dict(ldx=63), BAD), (dict(ldw=63), BAD), (dict(k=0), BAD), (dict(wdt=2), BAD),
    (dict(e=0), UNSUPPORTED), (dict(e=257), UNSUPPORTED), (dict(topk=0), BAD), (dict(topk=17), BAD),
    (dict(e=64, topk=33), UNSUPPORTED), (dict(score=2), BAD), (dict(renorm=2), BAD),
    (dict(scale=float("nan")), BAD), (dict(x=None), BAD), (dict(w=None), BAD), (dict(ids=None), BAD),
    (dict(wt=None), BAD), (dict(k=70000, ldx=70000, ldw=70000), UNSUPPORTED),
])
def test_route_refusals(over, want):
    assert _route(ws=FAKE, nbytes=1 << 20, **over)[0] == want


def test_route_workspace():
    st, need = _route(x=None, w=None, ids=None, wt=None)
    assert st == 0
    assert _route(ws=FAKE, nbytes=need - 1)[0] == SMALL


FFN_NAMES = ("gate", "up", "down", "e", "x", "ldx", "ids", "wt", "m", "topk", "act", "res", "ldr", "rdt", "y", "ldy",
             "ydt")


def _handles(e, n, k):
    return (svq.Handle * e)(*[_handle(n, k, 6 + i % 3) for i in range(e)])


def _ffn(ws=None, nbytes=0, e=4, n=96, k=520, down=None, up=None, **over):
    return _call(svq.LIB.svq_moe_ffn,
                 (_handles(e, n, k), up or _handles(e, n, k), down or _handles(e, k, n), e, FAKE, k, FAKE, FAKE, 3, 2,
                  2, None, 0, 0, FAKE, k, 0), FFN_NAMES, ws, nbytes, **over)


@pytest.mark.parametrize("over,want", [
    (dict(m=0), BAD), (dict(topk=0), BAD), (dict(topk=5), BAD), (dict(act=8), BAD), (dict(ldx=519), BAD),
    (dict(ldy=519), BAD), (dict(ydt=3), BAD), (dict(up=_handles(4, 96, 512)), BAD),
    (dict(down=_handles(4, 520, 104)), BAD), (dict(res=FAKE, ldr=519), BAD), (dict(res=FAKE, ldr=520, rdt=5), BAD),
    (dict(res=FAKE, ldr=520, rdt=1), BAD), (dict(x=None), BAD), (dict(y=None), BAD), (dict(ids=None), BAD),
    (dict(wt=None), BAD), (dict(m=(1 << 20) + 1), BAD),
])
def test_ffn_refusals(over, want):
    assert _ffn(ws=FAKE, nbytes=1 << 40, **over)[0] == want


def test_ffn_refuses_an_inner_width_beyond_lds():
    n = 40000
    assert _ffn(n=n, m=3, ldx=520)[0] == UNSUPPORTED
    assert _ffn(n=36864, m=3)[0] == 0


def test_misaligned_workspaces_are_refused():
    assert _epilogue(ws=FAKE + 8, nbytes=1 << 30)[0] == BAD
    assert _glu(ws=FAKE + 4, nbytes=1 << 30)[0] == BAD
    assert _route(ws=FAKE + 1, nbytes=1 << 30)[0] == BAD
    assert _ffn(ws=FAKE + 2, nbytes=1 << 30)[0] == BAD


def test_ffn_workspace():
    for m in (1, 8, 32, 33, 600):
        st, need = _ffn(m=m, x=None, y=None, ids=None, wt=None)
        assert st == 0 and need > 0
        assert _ffn(ws=FAKE, nbytes=need - 1, m=m)[0] == SMALL


def test_ffn_refuses_mixed_shapes_and_counts():
    mixed = (svq.Handle * 4)(*[_handle(96, 520) for _ in range(3)], _handle(112, 520))
    assert _ffn(up=mixed)[0] == BAD
    assert _ffn(e=1, topk=1, m=1)[0] == 0
    st, _ = _call(svq.LIB.svq_moe_ffn, (_handles(1, 96, 520), _handles(1, 96, 520), _handles(1, 520, 96), 257, FAKE,
                                        520, FAKE, FAKE, 1, 1, 2, None, 0, 0, FAKE, 520, 0), FFN_NAMES, None, 0)
    assert st == UNSUPPORTED


def test_binding_checks_operands():
    torch = pytest.importorskip("torch")
    pm = svq.PackedMatrix(None, _handle(96, 520))
    x = torch.zeros((3, 520), dtype=torch.bfloat16)
    y = torch.zeros((3, 96), dtype=torch.bfloat16)
    bad = [
        dict(x=x.float()), dict(x=x[:, :512]), dict(x=torch.zeros((520, 3), dtype=torch.bfloat16).t()),
        dict(y=y.half()), dict(y=y[:2]), dict(bias=torch.zeros(95)), dict(bias=torch.zeros(96).double()),
        dict(act="swish"), dict(residual=torch.zeros((3, 90))),
        dict(residual=torch.zeros(300).unfold(0, 96, 95)),  # rows that overlap
    ]
    for over in bad:
        args = dict(x=x, y=y)
        args.update(over)
        with pytest.raises(ValueError):
            svq.EpilogueCall(pm, **args)
    whole = torch.zeros((4, 96), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="overlaps"):
        svq.EpilogueCall(pm, x, whole[:3], residual=whole[1:])
    with pytest.raises(ValueError, match="one type"):
        svq.GluCall(pm, pm, x, y, bias_gate=torch.zeros(96), bias_up=torch.zeros(96, dtype=torch.bfloat16))
    ids, wt = torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2))
    with pytest.raises(ValueError):
        svq.MoeRouteCall(x, torch.zeros((4, 520)), ids.long(), wt)
    with pytest.raises(ValueError):
        svq.MoeRouteCall(x, torch.zeros((4, 520)), ids, wt, score="tanh")
    with pytest.raises(ValueError):
        svq.MoeFfnCall([pm], [pm], [], x, ids, wt, y)
    down = svq.PackedMatrix(None, _handle(96, 96))
    with pytest.raises(ValueError):
        svq.MoeFfnCall([pm], [pm], [down], x, ids[:2], wt, y)
