"""The attention calls as a decoder layer makes them: products, a prompt's
attention, its keys and values into the 4-bit cache, then token after token
over that cache, the block around it; eager and as a captured graph.  Every
attention output is checked against 64 bits on the operands it was given, the
chain by its final values being the same from call to call."""
import pytest

import synth
from tests.attn_common import P_BF16, P_F16, attend, check, stored, visible
from tests.gpu_common import require_gpu, torch

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM, INNER, PAGE, GROUP = 256, 8, 2, 64, 512, 16, 32
LENS = [37, 5, 64]


class Layer:
    def __init__(self, svq):
        pack = lambda n, k, bd, seed: svq.pack(synth.random_matrix(n, k, bd, seed=(77, seed)))
        self.qkv = [pack(HEADS * DIM, HIDDEN, 7, 1), pack(KV * DIM, HIDDEN, 6, 2), pack(KV * DIM, HIDDEN, 8, 3)]
        self.o = pack(HIDDEN, HEADS * DIM, 7, 4)
        self.gate, self.up = pack(INNER, HIDDEN, 7, 5), pack(INNER, HIDDEN, 8, 6)
        self.down = pack(HIDDEN, INNER, 6, 7)
        self.svq = svq

    def rows(self, n):
        """q, k and v as columns of one buffer."""
        wide = torch.zeros((n, (HEADS + 2 * KV) * DIM), dtype=torch.bfloat16, device="cuda")
        return wide, wide.split([HEADS * DIM, KV * DIM, KV * DIM], dim=1)

    def products(self, x, parts):
        for pm, y in zip(self.qkv, parts):
            self.svq.linear(pm, x, out=y)

    def rest(self, x, y):
        x = self.svq.linear_epilogue(self.o, y, residual=x)
        h = self.svq.linear_glu(self.gate, self.up, x)
        return self.svq.linear_epilogue(self.down, h, residual=x)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tokens(n, seed):
    g = torch.Generator().manual_seed(seed)
    return (0.3 * torch.randn(n, HIDDEN, generator=g)).to(torch.bfloat16).cuda()


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _setup(svq):
    layer = Layer(svq)
    need = [(n + 8 + PAGE - 1) // PAGE for n in LENS]
    cache = svq.KvCache(sum(need), PAGE, KV, DIM, group=GROUP)
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(5)).tolist()
    table = torch.full((len(LENS), max(need)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    slots = _ints([int(table[b, j // PAGE]) * PAGE + j % PAGE for b, n in enumerate(LENS) for j in range(n)])
    return layer, cache, table.cuda(), slots


def test_prompt_then_tokens():
    svq = require_gpu()
    layer, cache, table, slots = _setup(svq)
    at = _starts(LENS)
    x = _tokens(sum(LENS), 1)
    wide, (q, k, v) = layer.rows(len(x))
    layer.products(x, (q, k, v))
    y = svq.attn_prompt(q, k, v, _ints(at), DIM)
    svq.kv_write(cache, k, v, slots)
    out = layer.rest(x, y)
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all()
    ks, vs = [], []
    for b, n in enumerate(LENS):
        rows = slice(at[b], at[b + 1])
        check(y[rows], *attend(q[rows], k[rows], v[rows], HEADS, KV, DIM ** -0.5, visible(n, n)), n, P_BF16, f"prompt {b}")
        ks.append(stored(k[rows].contiguous(), GROUP))
        vs.append(stored(v[rows].contiguous(), GROUP))

    # token after token: the eager step and its captured form, on the same cache
    x = _tokens(len(LENS), 2)
    wide, (q, k, v) = layer.rows(len(LENS))
    y = torch.empty((len(LENS), HEADS * DIM), dtype=torch.bfloat16, device="cuda")
    now, place = _ints(LENS), torch.zeros(len(LENS), dtype=torch.int32, device="cuda")
    write = svq.KvWriteCall(cache, k, v, place)
    attn = svq.AttnCacheCall(cache, q, y, table, now)
    batched = svq.BatchedCall(layer.qkv, [x] * 3, [q, k, v])
    side = torch.cuda.Stream()

    def step():
        batched()
        write()
        attn()

    def advance(t):
        pos = torch.tensor(LENS, device="cuda") + t
        place.copy_(table.gather(1, (pos // PAGE)[:, None])[:, 0] * PAGE + pos % PAGE)
        now.copy_(pos + 1)

    graph = None
    for t in range(6):
        advance(t)
        torch.cuda.synchronize()
        if t == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.stream(side):
                batched = svq.BatchedCall(layer.qkv, [x] * 3, [q, k, v], stream=side)
            with torch.cuda.graph(graph, stream=side):
                step()
        if graph is None:
            step()
        else:
            y.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
        torch.cuda.synchronize()
        for b, n in enumerate(LENS):
            ks[b] = torch.cat([ks[b], stored(k[b:b + 1].contiguous(), GROUP)])
            vs[b] = torch.cat([vs[b], stored(v[b:b + 1].contiguous(), GROUP)])
            ref = attend(q[b:b + 1], ks[b], vs[b], HEADS, KV, DIM ** -0.5, visible(1, len(ks[b])))
            check(y[b:b + 1], *ref, len(ks[b]), P_F16, f"step {t}, sequence {b}")
        out = layer.rest(x, y)
        assert torch.isfinite(out.float()).all()
        x.copy_(out / out.float().abs().amax().clamp(min=1.0).to(torch.bfloat16))


def test_a_prompt_in_two_parts():
    """The second part of a prompt attends over the first, read back from the
    cache, and over itself: with the keys and values that the cache stands
    for, the same as attention over the cache."""
    svq = require_gpu()
    layer, cache, table, slots = _setup(svq)
    at = _starts(LENS)
    x = _tokens(sum(LENS), 3)
    wide, (q, k, v) = layer.rows(len(x))
    layer.products(x, (q, k, v))
    svq.kv_write(cache, k, v, slots)
    ck, cv = svq.kv_read(cache, slots)  # all of it, the new tokens too
    new = [min(4, n) for n in LENS]
    rows = torch.cat([torch.arange(e - m, e) for e, m in zip(at[1:], new)]).cuda()
    y = svq.attn_prompt(q[rows], ck, cv, _ints(_starts(new)), DIM, starts_k=_ints(at))
    z = svq.attn_cache(cache, q[rows], table, _ints(LENS), q_len=4)
    for b, n in enumerate(LENS):
        r = slice(at[b], at[b + 1])
        i = slice(sum(new[:b]), sum(new[:b + 1]))
        seen = visible(new[b], n)
        check(y[i], *attend(q[rows][i], ck[r], cv[r], HEADS, KV, DIM ** -0.5, seen), n, P_BF16, f"part {b}")
        ref = attend(q[rows][i], stored(k[r].contiguous(), GROUP), stored(v[r].contiguous(), GROUP), HEADS, KV, DIM ** -0.5, seen)
        check(z[i], *ref, n, P_F16, f"cache {b}")


def test_two_calls_at_once():
    """Two prepared calls with workspaces of their own on two streams."""
    svq = require_gpu()
    kv, heads, dim, page, n = 2, 8, 128, 16, 1500
    cache = svq.KvCache(2 * 100, page, kv, dim)
    g = torch.Generator().manual_seed(9)
    rows = lambda m, c: torch.randn(m, c, generator=g).to(torch.bfloat16).cuda()
    svq.kv_write(cache, rows(200 * page, kv * dim), rows(200 * page, kv * dim), _ints(list(range(200 * page))))
    tables = [_ints([list(range(100))]), _ints([list(range(100, 200))])]
    q = [rows(1, heads * dim) for _ in range(2)]
    alone = [svq.attn_cache(cache, q[i], tables[i], _ints([n])) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.empty_like(x) for x in q]
    lens = _ints([n])
    calls = [svq.AttnCacheCall(cache, q[i], ys[i], tables[i], lens, stream=streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c in calls:
            c()
    torch.cuda.synchronize()
    for a, y in zip(alone, ys):
        assert torch.equal(a, y)
