"""The expert layer where tests/test_gpu_ffn.py does not reach: several chunks
of tokens, experts with more rows than a work item, and inner widths beyond
what a block keeps in registers or stages in one pass.  Bounds as there."""
import numpy as np
import pytest

import synth
from oracle import svq_oracle as so
from tests.gpu_common import out_to_f64, require_gpu, to_device_bf16, torch
from tests.test_gpu_ffn import U32, act64, check, f64, slope_of, vec

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svq():
    return require_gpu()


def experts(svq, e, n, k, seed):
    mats = [synth.random_matrix(n, k, 6 + (i + seed) % 3, seed=(seed, i, n)) for i in range(e)]
    return mats, [svq.pack(a) for a in mats]


def weights64(mat):
    return so.linear_from_inputs(mat, np.zeros((1, mat.k), dtype=np.uint16))[1]


def layer64(sets, x_bits, ids, wt, act, grouped):
    """(y without the residual, bound), expert by expert."""
    (m, topk), (gates, ups, downs) = ids.shape, sets
    x = so.bf16_bits_to_f64(x_bits)
    y, b = np.zeros((m, downs[0].n)), np.zeros((m, downs[0].n))
    wr = 2.0 ** -11 if grouped else 0.0
    rel = lambda k: (k + 64) * U32 + wr
    for i in range(len(gates)):
        t, j = np.nonzero(ids == i)
        if not len(t):
            continue
        Wg, Wu, Wd = weights64(gates[i]), weights64(ups[i]), weights64(downs[i])
        xi, s = x[t], np.abs(x[t])
        g, u = xi @ Wg.T, xi @ Wu.T
        gb, ub = [rel(Wg.shape[1]) * (s @ np.abs(W).T) + 1e-6 for W in (Wg, Wu)]
        a = act64(g, act)
        h = a * u
        eh = (slope_of(act) * gb + 16 * U32 * np.abs(a)) * np.abs(u) + ub * np.abs(a) + slope_of(act) * gb * ub
        eh = eh + (2.0 ** -11 + U32) * (np.abs(h) + eh)
        # fp16 after a scale: a floor of 2^-39 of the row's largest value
        eh = eh + 2.0 ** -38 * np.abs(h).max(axis=1, keepdims=True)
        d = h @ Wd.T
        ed = eh @ np.abs(Wd).T + rel(Wd.shape[1]) * ((np.abs(h) + eh) @ np.abs(Wd).T) + 1e-6
        w = wt[t, j].astype(np.float64)[:, None]
        np.add.at(y, t, w * d)
        np.add.at(b, t, np.abs(w) * (ed + topk * U32 * (np.abs(d) + ed)))
    return y, b


def _routing(e, m, topk, seed):
    rng = np.random.default_rng(seed)
    ids = rng.random((m, e)).argsort(axis=1)[:, :topk].astype(np.int32)
    return ids, rng.random((m, topk)).astype(np.float32)


def _run(svq, sets, x_bits, ids, wt, **kw):
    (_, gp), (_, up), (_, dp) = sets
    return svq.moe_ffn(gp, up, dp, to_device_bf16(x_bits), torch.from_numpy(ids).cuda(), torch.from_numpy(wt).cuda(), **kw)


@pytest.mark.parametrize("e,topk,m", [(5, 3, 2731), (6, 1, 8193), (200, 3, 2800), (5, 5, 4100)])
def test_more_slots_than_a_chunk(svq, e, topk, m):
    """Chunks of at most 8192 slots of whole tokens (2730 tokens at three slots
    each, so the first chunk does not fill them), one token in the last one or
    many; slots without an expert, one expert twice, strided operands and the
    residual in place, in the last chunk as in the first; ids of more than 128
    experts (gate and up launched apart)."""
    f, k, n = 24, 40, 56
    sets = [experts(svq, e, f, k, 150), experts(svq, e, f, k, 151), experts(svq, e, n, f, 152)]
    x_bits = synth.random_activations(m, k, seed=(150, e, m))
    ids, wt = _routing(e, m, topk, [150, e, m])
    for t in (0, m - 1):
        ids[t, 0] = -1
    if topk > 1:
        ids[m - 1, -1], ids[1, 0], ids[m - 2, 0] = e, ids[1, 1], ids[m - 2, 1]
    wide = vec(m * (n + 5), torch.bfloat16, 26).view(m, n + 5)
    before, y = wide.clone(), wide[:, 2:2 + n]
    r = f64(y)
    _run(svq, sets, x_bits, ids, wt, residual=y, out=y)
    ref, bound = layer64([s[0] for s in sets], x_bits, ids, wt, "silu", True)
    ref = ref + r
    check(y, ref, bound + U32 * (np.abs(ref) + bound), f"e={e} m={m}")
    wide[:, 2:2 + n] = before[:, 2:2 + n]
    assert torch.equal(wide, before)


def test_chunks_captured_and_replayed(svq):
    """A call of two chunks, whose second reuses the first's workspace,
    replayed on a workspace that holds anything."""
    e, f, k, m, topk = 4, 24, 40, 4200, 2
    (_, gp), (_, up), (_, dp) = [experts(svq, e, f, k, 153), experts(svq, e, f, k, 154), experts(svq, e, k, f, 155)]
    ids, wt = _routing(e, m, topk, [153])
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((m, k), dtype=torch.float32, device="cuda")
    call = svq.MoeFfnCall(gp, up, dp, x, torch.from_numpy(ids).cuda(), torch.from_numpy(wt).cuda(), y)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        xi = to_device_bf16(synth.random_activations(m, k, seed=(153, i)))
        want = svq.moe_ffn(gp, up, dp, xi, call.keep[5], call.keep[6], out_dtype=torch.float32)
        x.copy_(xi)
        y.fill_(float("nan"))
        call.workspace.fill_((0xFF, 0x5A)[i % 2])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), f"replay {i}"


@pytest.mark.parametrize("f,k,m", [(2056, 40, 3), (4616, 24, 1), (1032, 40, 40), (4104, 24, 40), (9224, 16, 33),
                                   (40, 2056, 40), (40, 4616, 40), (24, 2568, 3)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_wide_inner_and_outer_widths(svq, f, k, m, act):
    """Inner widths past the values a thread prefetches in the per-slot form
    (2048), past what a lane keeps of act(gate) * up (1024) and past the rows
    that fit in one staging pass (4096) in the grouped one; the same for the
    rows of x (2048, 4096)."""
    e, topk = 3, 2
    sets = [experts(svq, e, f, k, 156), experts(svq, e, f, k, 157), experts(svq, e, 24, f, 158)]
    x_bits = synth.random_activations(m, k, seed=(156, f, m))
    ids, wt = _routing(e, m, topk, [156, f])
    y = _run(svq, sets, x_bits, ids, wt, act=act, out_dtype=torch.float32)
    ref, bound = layer64([s[0] for s in sets], x_bits, ids, wt, act, m * topk > 64)
    check(y, ref, bound, f"f={f} k={k} m={m}")


@pytest.mark.parametrize("e,m", [(1, 97), (1, 1000), (2, 700)])
def test_experts_of_many_items(svq, e, m):
    """More rows an expert than a work item takes (48); all tokens on one
    expert, or on one of two."""
    f, k = 136, 264
    sets = [experts(svq, e, f, k, 159), experts(svq, e, f, k, 160), experts(svq, e, k, f, 161)]
    x_bits = synth.random_activations(m, k, seed=(159, m))
    ids = np.full((m, 1), e - 1, dtype=np.int32)
    wt = np.ones((m, 1), dtype=np.float32)
    for rows in (m, 65):
        y = _run(svq, sets, x_bits[:rows], ids[:rows], wt[:rows], out_dtype=torch.float32)
        ref, bound = layer64([s[0] for s in sets], x_bits[:rows], ids[:rows], wt[:rows], "silu", rows > 64)
        check(y, ref, bound, f"e={e} m={rows}")


def test_inner_width_beyond_the_refused_one(svq):
    """Beyond 64 slots any inner width runs in the documented numerics: inner
    activations and weights in fp16, not through bf16."""
    e, f, k, m = 1, 40008, 8, 70
    sets = [experts(svq, e, f, k, 162), experts(svq, e, f, k, 163), experts(svq, e, 16, f, 164)]
    x_bits = synth.random_activations(m, k, seed=(162, m))
    ids, wt = np.zeros((m, 1), dtype=np.int32), np.ones((m, 1), dtype=np.float32)
    with pytest.raises(RuntimeError, match="unsupported"):
        _run(svq, sets, x_bits[:64], ids[:64], wt[:64])
    y = _run(svq, sets, x_bits, ids, wt, out_dtype=torch.float32)
    ref, bound = layer64([s[0] for s in sets], x_bits, ids, wt, "silu", True)
    check(y, ref, bound, "wide")
    # the bound adds up every rounding's worst case; as a random walk a value
    # rounded to t bits has an error of up to 2^-t, 2^-t / sqrt(3) rms at the
    # most and half of that at the least.  Three roundings of weights and one
    # of the inner value: in fp16 (t = 11 bits after the first) a relative
    # 2-norm of 2 2^-11 / sqrt(3) = 5.6e-4 at the most, in bf16 (t = 8) half
    # of 8 times that, 2.2e-3, at the least
    rel = np.linalg.norm(out_to_f64(y) - ref) / np.linalg.norm(ref)
    assert rel < 8e-4, rel
