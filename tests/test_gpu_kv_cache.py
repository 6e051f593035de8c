"""The 4-bit cache (svq_kv_write, svq_kv_read, svq_attn_cache) against 64
bits."""
import pytest

from tests.attn_common import P_F16, attend, cache_floor, check, stored, visible
from tests.gpu_common import require_gpu, torch

pytestmark = pytest.mark.gpu

FORMS = [(d, g) for d in (64, 128, 256) for g in (32, 64, 128) if g <= d]


def _rows(n, cols, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(n, cols, generator=g)).to(torch.bfloat16).cuda()


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _written(svq, cache, k, v, slots):
    """Writes, reads back in fp32, compares with the stored form."""
    svq.kv_write(cache, k, v, slots)
    got = svq.kv_read(cache, slots, out_dtype=torch.float32)
    for x, y in zip((k, v), got):
        want = stored(x, cache.desc.group).float()
        assert torch.equal(torch.nan_to_num(y.cpu(), nan=12345.0), torch.nan_to_num(want, nan=12345.0))
    return got


@pytest.mark.parametrize("dim,group", FORMS)
@pytest.mark.parametrize("page,heads,tokens", [(16, 1, 1), (16, 3, 5), (32, 2, 33), (64, 8, 67), (128, 1, 130), (256, 5, 9)])
def test_written_and_read_back(dim, group, page, heads, tokens):
    svq = require_gpu()
    cache = svq.KvCache(4, page, heads, dim, group=group)
    k, v = _rows(tokens, heads * dim, 1, 3.0), _rows(tokens, heads * dim, 2)
    g = torch.Generator().manual_seed(3)
    slots = _ints(torch.randperm(cache.slots, generator=g)[:tokens].tolist())
    got = _written(svq, cache, k, v, slots)
    half = svq.kv_read(cache, slots)
    for a, b in zip(half, got):
        assert torch.equal(a, b.to(torch.bfloat16))


@pytest.mark.parametrize("dim,group", FORMS)
def test_groups_of_every_kind(dim, group):
    """Constant groups, ties of the rounding, ranges from subnormal to the
    largest, infinities and NaN, negative zero."""
    svq = require_gpu()
    rows = []
    half = torch.arange(group) % 31 / 2.0             # s = 1: every second value is a tie
    rows.append(half)
    rows.append(half * 2.0 ** -120 - 2.0 ** -118)
    rows.append(half * 2.0 ** -126)                   # s near the least normal number
    rows.append(half * 2.0 ** -130)                   # subnormal values and scale
    rows.append((half - 7.5) * 2.0 ** 120)
    rows.append(torch.linspace(-1, 1, group) * 3.3e38)
    rows.append(torch.full((group,), 3.25))
    rows.append(torch.zeros(group))
    rows.append(-torch.zeros(group))
    rows.append(torch.where(torch.arange(group) == 5, 1.0, 1e-30))
    rows.append(torch.where(torch.arange(group) == 5, -4.5, 2.0 ** -40))  # borders that a small value decides
    rows.append(torch.where(torch.arange(group) % 3 == 0, -7.5, torch.where(torch.arange(group) % 3 == 1, 7.5, -2.0 ** -60)))
    for bad in (float("inf"), float("-inf"), float("nan")):
        rows.append(torch.where(torch.arange(group) == group - 1, bad, half))
    rows.append(torch.full((group,), float("-inf")))
    x = torch.stack(rows).to(torch.bfloat16)
    per = dim // group
    n = -(-len(rows) // per) * per
    x = torch.cat([x, torch.ones(n - len(rows), group, dtype=torch.bfloat16)]).reshape(-1, dim).cuda()
    cache = svq.KvCache(2, 16, 1, dim, group=group)
    slots = _ints(list(range(len(x))))
    _written(svq, cache, x, x.flip(0).contiguous(), slots)


def test_slots_outside_are_skipped_and_the_rest_stays():
    svq = require_gpu()
    dim, heads = 128, 3
    cache = svq.KvCache(3, 16, heads, dim)
    base_k, base_v = _rows(48, heads * dim, 4), _rows(48, heads * dim, 5)
    every = _ints(list(range(48)))
    svq.kv_write(cache, base_k, base_v, every)
    before = [t.clone() for t in svq.kv_read(cache, every)]
    k, v = _rows(7, heads * dim, 6), _rows(7, heads * dim, 7)
    slots = [-1, 17, 48, -2 ** 31, 2 ** 31 - 1, 3, 18]
    svq.kv_write(cache, k, v, _ints(slots))
    after = svq.kv_read(cache, every)
    for x, a, b in zip((k, v), after, before):
        want = stored(x, 64).to(torch.bfloat16).cuda()
        for i, s in ((1, 17), (5, 3), (6, 18)):
            assert torch.equal(a[s], want[i])
            b[s] = want[i]
        assert torch.equal(a, b)
    for x in svq.kv_read(cache, _ints(slots)):
        for i in (0, 2, 3, 4):
            assert torch.all(x[i] == 0)
        assert torch.all(x[[1, 5, 6]].abs().sum(dim=1) > 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_with_strides(dtype):
    svq = require_gpu()
    dim, heads, n = 64, 2, 21
    cache = svq.KvCache(2, 16, heads, dim, group=32)
    wide = _rows(n, 3 * heads * dim + 8, 8)
    k, v = wide[:, 8:8 + heads * dim], wide[:, 8 + heads * dim:8 + 2 * heads * dim]
    slots = _ints(list(range(n)))
    svq.kv_write(cache, k, v, slots)
    out = torch.full((n, 2 * heads * dim + 24), 7.0, dtype=dtype, device="cuda")
    svq.KvReadCall(cache, slots, out[:, 8:8 + heads * dim], out[:, 16 + heads * dim:16 + 2 * heads * dim])()
    torch.cuda.synchronize()
    want = [stored(x.contiguous(), 32).to(dtype).cuda() for x in (k, v)]
    assert torch.equal(out[:, 8:8 + heads * dim], want[0])
    assert torch.equal(out[:, 16 + heads * dim:16 + 2 * heads * dim], want[1])
    out[:, 8:8 + heads * dim] = 7.0
    out[:, 16 + heads * dim:16 + 2 * heads * dim] = 7.0
    assert torch.all(out == 7.0)


def _filled(svq, lens, page, kv, dim, group, seed=0, spare=2):
    """A cache with sequences of the given lengths on shuffled pages; every
    byte that no token wrote is 0xFF (codes 15, scales and minima NaN), every
    table entry behind a sequence's pages names no page."""
    need = [-(-n // page) for n in lens]
    cache = svq.KvCache(max(sum(need), 1) + spare, page, kv, dim, group=group)
    cache.buf.fill_(255)
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(sum(need) + spare, generator=g).tolist()
    width = max(max(need), 1) + 2
    table = torch.full((len(lens), width), 2 ** 31 - 1, dtype=torch.int32)
    ks, vs = [], []
    for b, n in enumerate(lens):
        mine = [order.pop() for _ in range(need[b])]
        table[b, :need[b]] = torch.tensor(mine, dtype=torch.int32)
        k, v = _rows(max(n, 1), kv * dim, 100 + b)[:n], _rows(max(n, 1), kv * dim, 200 + b)[:n]
        k = k + 2 * _rows(1, kv * dim, 300)
        if n:
            slots = _ints([mine[j // page] * page + j % page for j in range(n)])
            svq.kv_write(cache, k, v, slots)
        ks.append(stored(k, group) if n else k.cpu().double())
        vs.append(stored(v, group) if n else v.cpu().double())
    return cache, table.cuda(), ks, vs


def _check_cache(y, q, ks, vs, lens, q_len, heads, kv, dim, window, scale=None):
    for b, n in enumerate(lens):
        ref = attend(q[b * q_len:(b + 1) * q_len], ks[b], vs[b], heads, kv, dim ** -0.5 if scale is None else scale,
                     visible(q_len, n, True, window))
        check(y[b * q_len:(b + 1) * q_len], *ref, n, P_F16, f"sequence {b} ({n})")


CACHE_CASES = [
    # lens, page, heads, kv, dim, group, q_len, window
    ([1], 16, 1, 1, 64, 32, 1, 0),
    ([1], 16, 8, 2, 128, 64, 1, 0),
    ([17], 16, 4, 1, 256, 128, 1, 0),
    ([0, 5, 0, 33], 16, 4, 2, 128, 32, 1, 0),
    ([15, 16, 17, 31, 32, 33], 16, 4, 1, 128, 64, 1, 0),
    ([63, 64, 65, 127, 128, 129], 64, 2, 2, 64, 64, 1, 0),
    ([255, 257, 600], 256, 8, 1, 128, 128, 1, 0),
    ([300, 2, 129], 32, 16, 1, 128, 64, 1, 0),
    ([200, 40], 32, 17, 1, 64, 32, 1, 0),
    ([77, 300], 128, 64, 1, 128, 64, 1, 0),
    ([130, 3], 16, 6, 3, 256, 32, 1, 0),
    ([130, 3], 16, 6, 3, 256, 64, 2, 0),
    ([1000], 64, 7, 1, 128, 32, 1, 0),
    ([3, 130, 8], 16, 4, 1, 128, 64, 5, 0),       # 3 tokens, 5 queries: two rows without a key
    ([0, 1, 200], 32, 8, 2, 64, 32, 8, 0),
    ([100, 45], 16, 2, 1, 128, 64, 40, 0),
    ([200, 64, 1], 16, 4, 2, 128, 64, 1, 1),
    ([200, 64, 1], 16, 4, 2, 128, 64, 3, 17),
    ([300, 90], 64, 8, 1, 256, 128, 4, 64),
    ([500, 33], 32, 4, 4, 64, 64, 1, 100),
    ([2500, 1100], 64, 4, 1, 128, 64, 1, 0),
    ([2500, 1100], 16, 8, 2, 64, 32, 2, 1500),
]


@pytest.mark.parametrize("case", CACHE_CASES, ids=lambda c: f"{c[0][:3]}-p{c[1]}-h{c[2]}x{c[3]}-d{c[4]}g{c[5]}-q{c[6]}-w{c[7]}")
def test_attention_against_64_bits(case):
    svq = require_gpu()
    lens, page, heads, kv, dim, group, q_len, window = case
    cache, table, ks, vs = _filled(svq, lens, page, kv, dim, group)
    q = _rows(len(lens) * q_len, heads * dim, 9)
    y = svq.attn_cache(cache, q, table, _ints(lens), q_len=q_len, window=window)
    torch.cuda.synchronize()
    _check_cache(y, q, ks, vs, lens, q_len, heads, kv, dim, window)
    # planned for no more than the longest
    if max(lens):
        y = svq.attn_cache(cache, q, table, _ints(lens), q_len=q_len, max_len=max(lens), window=window)
        _check_cache(y, q, ks, vs, lens, q_len, heads, kv, dim, window)


def test_lengths_beyond_the_plan():
    svq = require_gpu()
    heads, kv, dim = 4, 1, 128
    cache, table, ks, vs = _filled(svq, [100, 60], 16, kv, dim, 64)
    q = _rows(2, heads * dim, 10)
    y = svq.attn_cache(cache, q, table, _ints([5000, -3]), max_len=77)
    _check_cache(y, q, [ks[0][:77], ks[1][:0]], [vs[0][:77], vs[1][:0]], [77, 0], 1, heads, kv, dim, 0)


@pytest.mark.parametrize("dim,group", FORMS)
def test_pages_that_do_not_exist(dim, group):
    """Their tokens are not seen; the others are."""
    svq = require_gpu()
    heads, kv, page, n = 4, 2, 16, 150
    cache, table, ks, vs = _filled(svq, [n, n], page, kv, dim, group)
    q = _rows(2 * 2, heads * dim, 11)
    table[0, 2], table[0, 3], table[1, 0], table[1, 9] = -1, int(cache.desc.pages), -2 ** 31, 2 ** 31 - 1
    y = svq.attn_cache(cache, q, table, _ints([n, n]), q_len=2)
    for b, gone in enumerate([(2, 3), (0, 9)]):
        seen = visible(2, n)
        for p in gone:
            seen[:, p * page:(p + 1) * page] = False
        ref = attend(q[2 * b:2 * b + 2], ks[b], vs[b], heads, kv, dim ** -0.5, seen)
        check(y[2 * b:2 * b + 2], *ref, n, P_F16, f"sequence {b}")
    table.fill_(-1)
    y = svq.attn_cache(cache, q, table, _ints([n, n]), q_len=2)
    assert torch.all(y == 0)


@pytest.mark.parametrize("dim,group", FORMS)
def test_values_of_every_size(dim, group):
    """Scales of values from 2^-100 to 2^100 within one sequence, keys too
    where queries are small; a group's minimum far from its range."""
    svq = require_gpu()
    heads, kv, page, n = 4, 1, 16, 90
    cache, table, _, _ = _filled(svq, [n], page, kv, dim, group)
    k, v = _rows(n, kv * dim, 12), _rows(n, kv * dim, 13)
    size = torch.tensor([2.0 ** e for e in (-100, -20, 0, 3, 40, 100)], device="cuda")
    v = (v.float() * size[torch.arange(n, device="cuda") * 6 // n][:, None]).to(torch.bfloat16)
    v[:10] += 5.0
    k = (k.float() + 100.0).to(torch.bfloat16)
    slots = torch.cat([table[0, j // page].view(1) * page + j % page for j in range(n)]).to(torch.int32)
    svq.kv_write(cache, k, v, slots)
    for q_size in (1.0, 2.0 ** -60, 2.0 ** 10):
        q = _rows(3, heads * dim, 14, q_size)
        for last in (10, 15, 40, 70, n):  # later tokens are larger
            y = svq.attn_cache(cache, q, table, _ints([last]), q_len=3)
            values = stored(v, group)[:last]
            ref = attend(q, stored(k, group)[:last], values, heads, kv, dim ** -0.5, visible(3, last))
            check(y, *ref, last, P_F16, f"{last} tokens, queries of {q_size}", floor=cache_floor(values, last))


@pytest.mark.parametrize("dim,group", FORMS)
def test_hidden_tokens_have_no_influence(dim, group):
    """A token that is not finite, seen by some queries of a call only."""
    svq = require_gpu()
    heads, kv, page, n, at = 4, 2, 16, 60, 57
    cache, table, ks, vs = _filled(svq, [n], page, kv, dim, group)
    bad = torch.full((1, kv * dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    svq.kv_write(cache, bad, bad, table[0, at // page].view(1) * page + at % page)
    q = _rows(6, heads * dim, 15)
    y = svq.attn_cache(cache, q, table, _ints([n]), q_len=6)  # queries at 54 .. 59
    ref = attend(q, ks[0], vs[0], heads, kv, dim ** -0.5, visible(6, n))
    check(y[:3], *(r[:3] for r in ref), n, P_F16)
    assert torch.isnan(y[3:].float()).all()
    y = svq.attn_cache(cache, q, table, _ints([n]), q_len=6, window=1)
    ref = attend(q, ks[0], vs[0], heads, kv, dim ** -0.5, visible(6, n, True, 1))
    keep = [0, 1, 2, 4, 5]
    check(y[keep], *(r[keep] for r in ref), n, P_F16)
    # and a query that is not finite
    q[1, :dim] = float("nan")
    y = svq.attn_cache(cache, q, table, _ints([50]), q_len=6)
    ref = attend(q, ks[0][:50], vs[0][:50], heads, kv, dim ** -0.5, visible(6, 50))
    rows = [0, 2, 3, 4, 5]
    check(y[rows], *(r[rows] for r in ref), 50, P_F16)
    check(y[1, dim:], *(r[1, dim:] for r in ref), 50, P_F16)
    assert torch.isnan(y[1, :dim].float()).all()


@pytest.mark.parametrize("scale", [0.0, -1.0, 50.0])
def test_scales(scale):
    svq = require_gpu()
    heads, kv, dim, lens = 4, 1, 128, [150, 33]
    cache, table, ks, vs = _filled(svq, lens, 16, kv, dim, 64)
    q = _rows(2, heads * dim, 16)
    y = svq.attn_cache(cache, q, table, _ints(lens), scale=scale)
    _check_cache(y, q, ks, vs, lens, 1, heads, kv, dim, 0, scale=scale)


def test_rows_of_wider_buffers():
    svq = require_gpu()
    heads, kv, dim, lens = 4, 2, 64, [40, 70]
    cache, table, ks, vs = _filled(svq, lens, 32, kv, dim, 32)
    wide = _rows(4, heads * dim + 16, 17)
    q = wide[:, 8:8 + heads * dim]
    buf = torch.full((4, heads * dim + 32), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[:, 16:16 + heads * dim]
    svq.attn_cache(cache, q, table, _ints(lens), q_len=2, out=y)
    _check_cache(y, q, ks, vs, lens, 2, heads, kv, dim, 0)
    y.fill_(7.0)
    assert torch.all(buf == 7.0)


def test_offsets_past_32_bits():
    """Pages whose bytes lie beyond 2^32 from the cache's start."""
    svq = require_gpu()
    heads, kv, dim, page = 8, 8, 128, 256
    cache = svq.KvCache(15000, page, kv, dim)
    assert cache.nbytes > 1 << 32
    n = 300
    k, v = _rows(n, kv * dim, 18), _rows(n, kv * dim, 19)
    pages = [14999, 14500]
    slots = _ints([pages[j // page] * page + j % page for j in range(n)])
    svq.kv_write(cache, k, v, slots)
    for x, got in zip((k, v), svq.kv_read(cache, slots, out_dtype=torch.float32)):
        assert torch.equal(got.cpu(), stored(x, 64).float())
    q = _rows(1, heads * dim, 20)
    y = svq.attn_cache(cache, q, _ints([pages]), _ints([n]))
    _check_cache(y, q, [stored(k, 64)], [stored(v, 64)], [n], 1, heads, kv, dim, 0)


def test_same_bits_captured_and_on_another_stream():
    """A step (write, attend) captured once and replayed as the sequences
    grow, against eager calls."""
    svq = require_gpu()
    heads, kv, dim, page, lens = 8, 2, 128, 16, [700, 31, 5]
    cache, table, _, _ = _filled(svq, [n + 8 for n in lens], page, kv, dim, 64)
    k, v = _rows(3, kv * dim, 21), _rows(3, kv * dim, 22)
    q = _rows(3, heads * dim, 23)
    y, now = torch.empty_like(q), _ints(lens)
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    write = svq.KvWriteCall(cache, k, v, slots)
    call = svq.AttnCacheCall(cache, q, y, table, now)

    def place(step):
        at = torch.tensor(lens, device="cuda") + step
        slots.copy_(table.gather(1, (at // page)[:, None])[:, 0] * page + at % page)
        now.copy_(at + 1)

    place(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        write()
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        write()
        call()
    for step in range(4):
        place(step)
        k.add_(1.0)
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = y.clone()
        write()
        assert torch.equal(replayed, svq.attn_cache(cache, q, table, now))


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 6, 2, 0])
def test_windows_wider_than_the_sequence(window):
    """Queries before the first token beside some that see tokens, under
    windows up to the largest number."""
    svq = require_gpu()
    lens, q_len, heads, kv, dim = [2, 70, 0, 1], 5, 4, 2, 64
    cache, table, ks, vs = _filled(svq, lens, 16, kv, dim, 32)
    q = _rows(len(lens) * q_len, heads * dim, 11)
    y = svq.attn_cache(cache, q, table, _ints(lens), q_len=q_len, window=window)
    torch.cuda.synchronize()
    _check_cache(y, q, ks, vs, lens, q_len, heads, kv, dim, window)
