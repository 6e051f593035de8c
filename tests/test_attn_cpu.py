"""The attention calls (include/svq_attn.h) on a host without a GPU: the
library exports them, answers size queries and refuses bad arguments before
any device work; the binding refuses bad operands, each by its own message."""
import ctypes
import os
import re

import pytest

from tests.conftest import ROOT

svq = pytest.importorskip("bit_spherical_vector_amd.svq")
torch = pytest.importorskip("torch")

BAD, UNSUPPORTED, SMALL = svq.SVQ_ERR_INVALID_ARG, svq.SVQ_ERR_UNSUPPORTED, svq.SVQ_ERR_BUFFER_TOO_SMALL
FAKE = 0x100000  # a non-null device address; no refused call reads it


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "svq_attn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"\b(svq_[a-z_]+)\s*\(", text))
    assert declared == set(svq.EXPORTED_ATTN)
    for name in declared:
        assert hasattr(svq.LIB, name)


def _desc(**over):
    f = dict(dev=FAKE, pages=10, page_size=16, kv_heads=2, head_dim=128, group=64)
    f.update(over)
    return svq.KvCacheDesc(**f)


def _call(fn, names, values, over, ws, nbytes):
    vals = dict(zip(names, values))
    assert not set(over) - set(names)
    vals.update(over)
    size = ctypes.c_size_t(nbytes)
    return fn(*[vals[n] for n in names], ws, ctypes.byref(size), None), size.value


PROMPT = ("q", "ldq", "k", "ldk", "v", "ldv", "q_heads", "kv_heads", "head_dim", "starts", "starts_k", "sequences",
          "tokens", "tokens_k", "causal", "window", "scale", "y", "ldy")


def _prompt(ws=None, nbytes=0, **over):
    return _call(svq.LIB.svq_attn_prompt, PROMPT,
                 (FAKE, 512, FAKE, 256, FAKE, 256, 4, 2, 128, FAKE, None, 3, 50, 50, 1, 0, 0.1, FAKE, 512), over, ws,
                 nbytes)


CACHE = ("cache", "q", "ldq", "q_heads", "table", "ld_table", "lens", "batch", "q_len", "max_len", "window", "scale",
         "y", "ldy")


def _cache(ws=None, nbytes=0, desc=None, **over):
    return _call(svq.LIB.svq_attn_cache, CACHE,
                 (ctypes.byref(desc or _desc()), FAKE, 512, 4, FAKE, 5, FAKE, 3, 1, 80, 0, 0.1, FAKE, 512), over, ws,
                 nbytes)


@pytest.mark.parametrize("over,status", [
    (dict(q_heads=0), BAD), (dict(kv_heads=0), BAD), (dict(q_heads=5), BAD), (dict(head_dim=0), UNSUPPORTED),
    (dict(head_dim=96), UNSUPPORTED), (dict(q_heads=130, ldq=130 * 128, ldy=130 * 128), UNSUPPORTED),
    (dict(q_heads=2050, kv_heads=1025, ldq=1 << 20, ldk=1 << 20, ldv=1 << 20, ldy=1 << 20), UNSUPPORTED),
    (dict(q_heads=16448, kv_heads=257, ldq=1 << 22, ldk=1 << 20, ldv=1 << 20, ldy=1 << 22), UNSUPPORTED),
    (dict(tokens=0), BAD), (dict(tokens=(1 << 24) + 1), BAD), (dict(tokens_k=0), BAD),
    (dict(tokens_k=(1 << 24) + 1), BAD), (dict(sequences=0), BAD), (dict(sequences=65536), BAD),
    (dict(ldq=504), BAD), (dict(ldk=248), BAD), (dict(ldv=248), BAD), (dict(ldy=504), BAD),
    (dict(ldk=(1 << 24) + 8), UNSUPPORTED), (dict(ldv=(1 << 24) + 8), UNSUPPORTED),
    (dict(tokens=1 << 24, q_heads=34, ldq=34 * 128, ldy=34 * 128), UNSUPPORTED),
    (dict(sequences=65535, q_heads=34, kv_heads=34, ldq=34 * 128, ldk=34 * 128, ldv=34 * 128, ldy=34 * 128), UNSUPPORTED),
    (dict(causal=2), BAD), (dict(causal=0, window=4), BAD), (dict(window=-1), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD),
    (dict(q=FAKE + 2), UNSUPPORTED), (dict(k=FAKE + 8), UNSUPPORTED), (dict(v=FAKE + 4), UNSUPPORTED),
    (dict(y=FAKE + 2), UNSUPPORTED), (dict(ldq=516), UNSUPPORTED), (dict(ldk=260), UNSUPPORTED),
    (dict(ldv=257), UNSUPPORTED), (dict(ldy=514), UNSUPPORTED),
])
def test_prompt_refusals(over, status):
    assert _prompt(**over)[0] == status
    assert _prompt(ws=FAKE, nbytes=1 << 40, **over)[0] == status


def test_prompt_workspace():
    st, need = _prompt()
    assert st == svq.SVQ_OK and need > 0
    assert _prompt(ws=FAKE, nbytes=need - 1)[0] == SMALL
    assert _prompt(ws=FAKE + 8, nbytes=need)[0] == BAD
    for name in ("q", "k", "v", "starts", "y"):
        assert _prompt(ws=FAKE, nbytes=need, **{name: None})[0] == BAD
    assert svq.LIB.svq_attn_prompt(FAKE, 512, FAKE, 256, FAKE, 256, 4, 2, 128, FAKE, None, 3, 50, 50, 1, 0, 0.1, FAKE,
                                   512, None, None, None) == BAD


CACHE_FIELDS = [
    (dict(page_size=0), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=512), UNSUPPORTED), (dict(head_dim=32), UNSUPPORTED), (dict(group=16), UNSUPPORTED),
    (dict(group=256, head_dim=256), UNSUPPORTED), (dict(group=128, head_dim=64), UNSUPPORTED),
    (dict(kv_heads=0), BAD), (dict(kv_heads=1025), UNSUPPORTED), (dict(pages=0), BAD),
    (dict(pages=(1 << 31) // 16), UNSUPPORTED),
]


@pytest.mark.parametrize("fields,status", CACHE_FIELDS)
def test_cache_descriptions(fields, status):
    d = _desc(**fields)
    size = ctypes.c_size_t(0)
    ref = ctypes.byref(d)
    assert svq.LIB.svq_kv_bytes(ref, ctypes.byref(size)) == status
    assert svq.LIB.svq_kv_write(ref, FAKE, 256, FAKE, 256, 4, FAKE, None) == status
    assert svq.LIB.svq_kv_read(ref, FAKE, 4, FAKE, 256, FAKE, 256, svq.SVQ_BF16, None) == status
    assert _cache(desc=d)[0] == status


@pytest.mark.parametrize("dev", [None, FAKE + 8])
def test_cache_memory(dev):
    d = _desc(dev=dev)
    ref = ctypes.byref(d)
    size = ctypes.c_size_t(0)
    assert svq.LIB.svq_kv_bytes(ref, ctypes.byref(size)) == svq.SVQ_OK
    assert svq.LIB.svq_kv_write(ref, FAKE, 256, FAKE, 256, 4, FAKE, None) == BAD
    assert svq.LIB.svq_kv_read(ref, FAKE, 4, FAKE, 256, FAKE, 256, svq.SVQ_BF16, None) == BAD
    assert _cache(desc=d)[0] == BAD
    assert svq.LIB.svq_kv_bytes(None, ctypes.byref(size)) == BAD
    assert svq.LIB.svq_kv_bytes(ref, None) == BAD


@pytest.mark.parametrize("dim,group,page,heads,pages", [(64, 32, 16, 1, 1), (128, 64, 64, 8, 100), (256, 128, 256, 3, 7)])
def test_cache_bytes(dim, group, page, heads, pages):
    d = _desc(head_dim=dim, group=group, page_size=page, kv_heads=heads, pages=pages)
    size = ctypes.c_size_t(0)
    assert svq.LIB.svq_kv_bytes(ctypes.byref(d), ctypes.byref(size)) == svq.SVQ_OK
    assert size.value == pages * page * heads * 2 * (dim // 2 + 4 * (dim // group))


WRITE = ("cache", "k", "ldk", "v", "ldv", "tokens", "slots", "stream")
READ = ("cache", "slots", "tokens", "k", "ldk", "v", "ldv", "dt", "stream")


@pytest.mark.parametrize("over,status", [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(slots=None), BAD), (dict(tokens=0), BAD),
    (dict(tokens=(1 << 24) + 1), BAD), (dict(ldk=248), BAD), (dict(ldv=248), BAD),
    (dict(k=FAKE + 2), UNSUPPORTED), (dict(v=FAKE + 8), UNSUPPORTED), (dict(ldk=258), UNSUPPORTED),
    (dict(ldv=259), UNSUPPORTED),
])
def test_write_and_read_refusals(over, status):
    d = ctypes.byref(_desc())
    vals = dict(cache=d, k=FAKE, ldk=256, v=FAKE, ldv=256, tokens=4, slots=FAKE, dt=svq.SVQ_BF16, stream=None, **{})
    vals.update(over)
    assert svq.LIB.svq_kv_write(*[vals[n] for n in WRITE]) == status
    assert svq.LIB.svq_kv_read(*[vals[n] for n in READ]) == status


def test_read_types():
    d = ctypes.byref(_desc())
    assert svq.LIB.svq_kv_read(d, FAKE, 4, FAKE, 256, FAKE, 256, 2, None) == BAD
    # rows of 4-byte values on 16 bytes: every fourth element
    assert svq.LIB.svq_kv_read(d, FAKE, 4, FAKE, 258, FAKE, 256, svq.SVQ_F32, None) == UNSUPPORTED


@pytest.mark.parametrize("over,status", [
    (dict(cache=None), BAD), (dict(q_heads=0), BAD), (dict(q_heads=3), BAD),
    (dict(q_heads=130, ldq=130 * 128, ldy=130 * 128), UNSUPPORTED), (dict(batch=0), BAD), (dict(batch=65536), BAD),
    (dict(q_len=0), BAD), (dict(q_len=1025), BAD), (dict(batch=65535, q_len=1000), BAD), (dict(max_len=0), BAD),
    (dict(max_len=81), BAD), (dict(ld_table=4), BAD), (dict(ld_table=0), BAD),
    (dict(ld_table=1 << 40, max_len=(1 << 30) + 1), BAD), (dict(ldq=504), BAD), (dict(ldy=504), BAD),
    (dict(window=-1), BAD), (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD),
    (dict(q=FAKE + 2), UNSUPPORTED), (dict(y=FAKE + 8), UNSUPPORTED), (dict(ldq=513), UNSUPPORTED),
    (dict(ldy=516), UNSUPPORTED),
])
def test_attention_over_the_cache_refusals(over, status):
    assert _cache(**over)[0] == status
    assert _cache(ws=FAKE, nbytes=1 << 40, **over)[0] == status


@pytest.mark.parametrize("shape", [dict(), dict(batch=1, max_len=1, ld_table=1), dict(q_len=7, window=5),
                                   dict(ld_table=1 << 26, max_len=1 << 30), dict(batch=65535, q_len=256)])
def test_attention_over_the_cache_workspace(shape):
    st, need = _cache(**shape)
    assert st == svq.SVQ_OK and 0 < need < 1 << 36
    assert _cache(ws=FAKE, nbytes=need - 1, **shape)[0] == SMALL
    assert _cache(ws=FAKE + 8, nbytes=need, **shape)[0] == BAD
    for name in ("q", "table", "lens", "y"):
        assert _cache(ws=FAKE, nbytes=need, **{name: None}, **shape)[0] == BAD


# ---- the binding's own checks (CPU tensors: a refused call goes no further) ----

def _cpu_cache(**over):
    f = dict(pages=3, page_size=16, kv_heads=2, head_dim=64, group=32, device="cpu")
    f.update(over)
    return svq.KvCache(**f)


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _i(n):
    return torch.zeros(n, dtype=torch.int32)


def _refused(message, make):
    with pytest.raises((ValueError, svq.SvqError), match=message):
        make()


def test_cache_objects():
    c = _cpu_cache()
    assert c.slots == 48 and c.width == 128 and c.buf.numel() == c.nbytes
    with pytest.raises(svq.SvqError) as e:
        _cpu_cache(head_dim=80)
    assert e.value.status == UNSUPPORTED
    _cpu_cache(buf=torch.zeros(c.nbytes + 16, dtype=torch.uint8))
    _refused("contiguous uint8", lambda: _cpu_cache(buf=torch.zeros(c.nbytes - 1, dtype=torch.uint8)))
    _refused("contiguous uint8", lambda: _cpu_cache(buf=torch.zeros(c.nbytes, dtype=torch.int8)))
    _refused("contiguous uint8", lambda: _cpu_cache(buf=torch.zeros(2 * c.nbytes, dtype=torch.uint8)[::2]))


def test_write_and_read_operands():
    c, wide = _cpu_cache(), _bf(5, 256)
    svq.KvWriteCall(c, wide[:, :128], wide[:, 128:], _i(5))
    _refused("k must be 2-D", lambda: svq.KvWriteCall(c, _bf(4, 128), _bf(5, 128), _i(5)))
    _refused("v must be 2-D", lambda: svq.KvWriteCall(c, _bf(5, 128), _bf(5, 120), _i(5)))
    _refused("k has the wrong type", lambda: svq.KvWriteCall(c, _bf(5, 128).float(), _bf(5, 128), _i(5)))
    _refused("slots must be torch.int32", lambda: svq.KvWriteCall(c, _bf(5, 128), _bf(5, 128), _i(5).long()))
    _refused("slots must be a contiguous", lambda: svq.KvWriteCall(c, _bf(5, 128), _bf(5, 128), _i(10)[::2]))
    svq.KvReadCall(c, _i(5), wide[:, :128], wide[:, 128:])
    _refused("one type", lambda: svq.KvReadCall(c, _i(5), _bf(5, 128), _bf(5, 128).float()))
    _refused("k overlaps v", lambda: svq.KvReadCall(c, _i(5), wide[:, :128], wide[:, 64:192]))
    _refused("rows of k overlap", lambda: svq.KvReadCall(c, _i(5), _bf(1, 128).expand(5, 128), _bf(5, 128)))


def test_prompt_operands():
    wide, y = _bf(6, 512), _bf(6, 256)
    q, k, v = wide[:, :256], wide[:, 256:384], wide[:, 384:]
    # a call that passes every check goes on to the GPU, which is not here
    make = lambda *a, **kw: svq.AttnPromptCall(*a, **kw)
    _refused("whole heads", lambda: make(wide[:, :200], k, v, y, _i(2), 64))
    _refused("whole heads", lambda: make(q, wide[:, :100], v, y, _i(2), 64))
    _refused("whole heads", lambda: make(q, k, v, y, _i(2), 0))
    _refused("one number of heads", lambda: make(q, k, wide[:, 384:448], y, _i(2), 64))
    _refused("v must be 2-D", lambda: make(q, k, v[:5], y, _i(2), 64))
    _refused("y must be 2-D", lambda: make(q, k, v, y[:, :128], _i(2), 64))
    _refused("y has the wrong type", lambda: make(q, k, v, y.float(), _i(2), 64))
    _refused("y overlaps q", lambda: make(q, k, v, q, _i(2), 64))
    _refused("y overlaps k", lambda: make(_bf(6, 256), k, v, wide[:, 192:448], _i(2), 64))
    _refused("y overlaps v", lambda: make(_bf(6, 128), _bf(6, 128), v, wide[:, 384:], _i(2), 64))
    _refused("starts must be torch.int32", lambda: make(q, k, v, y, _i(2).long(), 64))
    _refused("starts_k must be a contiguous", lambda: make(q, k, v, y, _i(2), 64, starts_k=_i(3)))
    _refused("as many keys as queries", lambda: make(q, _bf(7, 128), _bf(7, 128), y, _i(2), 64))


def test_cache_attention_operands():
    c = _cpu_cache()
    q, y, t = _bf(4, 256), _bf(4, 256), torch.zeros(2, 3, dtype=torch.int32)
    make = lambda *a, **kw: svq.AttnCacheCall(*a, **kw)
    _refused("whole heads", lambda: make(c, _bf(4, 200), y, t, _i(2), q_len=2))
    _refused("q_len rows", lambda: make(c, q, y, t, _i(2), q_len=1))
    _refused("q has the wrong type", lambda: make(c, q.float(), y, t, _i(2), q_len=2))
    _refused("y must be 2-D", lambda: make(c, q, _bf(3, 256), t, _i(2), q_len=2))
    _refused("y overlaps q", lambda: make(c, q, q, t, _i(2), q_len=2))
    _refused("lens must be torch.int32", lambda: make(c, q, y, t, _i(2).long(), q_len=2))
    _refused("table must be 2-D", lambda: make(c, q, y, t[:1], _i(2), q_len=2))
    _refused("table has the wrong type", lambda: make(c, q, y, t.long(), _i(2), q_len=2))
    _refused("more than the table", lambda: make(c, q, y, t, _i(2), q_len=2, max_len=49))


def test_windows_are_32_bit_numbers():
    c, t = _cpu_cache(), torch.zeros(2, 3, dtype=torch.int32)
    for window in (-1, 2 ** 31, 2 ** 32 + 5):
        _refused("window must be", lambda: svq.AttnPromptCall(_bf(6, 256), _bf(6, 128), _bf(6, 128), _bf(6, 256), _i(2), 64,
                                                              window=window))
        _refused("window must be", lambda: svq.AttnCacheCall(c, _bf(4, 256), _bf(4, 256), t, _i(2), q_len=2, window=window))
    _refused("table must be 2-D", lambda: svq.AttnCacheCall(c, _bf(2, 256), _bf(2, 256), _i(2), _i(2)))


def test_operands_apart_from_the_cache():
    need = _cpu_cache().nbytes
    memory = torch.zeros(need + 4 * 5 * 256, dtype=torch.uint8)
    c = _cpu_cache(buf=memory[:need])
    rows = lambda at: memory[at:at + 5 * 256].view(torch.bfloat16).view(5, 128)
    inside, last, behind = rows(0), rows(need - 256), rows(need)
    svq.KvWriteCall(c, behind, _bf(5, 128), _i(5))
    svq.KvReadCall(c, _i(5), behind, _bf(5, 128))
    _refused("k overlaps the cache", lambda: svq.KvWriteCall(c, inside, _bf(5, 128), _i(5)))
    _refused("v overlaps the cache", lambda: svq.KvWriteCall(c, _bf(5, 128), last, _i(5)))
    _refused("k overlaps the cache", lambda: svq.KvReadCall(c, _i(5), last, _bf(5, 128)))
    _refused("v overlaps the cache", lambda: svq.KvReadCall(c, _i(5), behind, inside))
    _refused("y overlaps the cache", lambda: svq.AttnCacheCall(c, _bf(5, 128), last, torch.zeros(5, 3, dtype=torch.int32), _i(5)))
