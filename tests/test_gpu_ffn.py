"""The feed-forward calls on the GPU against their definitions in 64 bits.

Tolerances, from the documented numerics (half a step of a rounding is
torch.finfo(t).eps / 2 of the value):

* a product of k terms: |p - p64| <= P * S + 1e-6 with S = sum |What||x|;
  accumulation in fp32 costs at most one rounding per term (k + 64 of 2^-24,
  64 for the joins of partial sums), and for more than 16 rows, and from 5
  rows on for a bf16 output, the weights are rounded to fp16 first (2^-11; a weight so small beside its matrix's
  largest that it is subnormal there keeps an error of 2^-39 of that one);
* an activation's slope is at most 1.13 (silu 1.0998, gelu 1.129), so an
  error e of its argument becomes at most 1.13 e, plus a few fp32 roundings
  of the value (expf, one division: 16 of 2^-24);
* sums and products of fp32 values: one rounding each;
* the output: half a step of its type.
"""
import math

import numpy as np
import pytest

import synth
from oracle import svq_oracle as so
from tests.gpu_common import out_to_f64, require_gpu, to_device_bf16, torch

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
SLOPE = 1.13
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module")
def svq():
    return require_gpu()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def act64(v, act):
    if act == "relu":
        return np.maximum(v, 0)
    if act == "silu":
        return v / (1 + np.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + np.vectorize(math.erf)(v / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def slope_of(act):
    return 1.0 if act in ("none", "relu") else SLOPE


def product(mat, x_bits, rounded_weights):
    """(p, bound of |p_gpu - p|) of one matrix."""
    p, W = so.linear_from_inputs(mat, x_bits)
    rel = (mat.k + 64) * U32 + (2.0 ** -11 if rounded_weights else 0.0)
    return p, rel * so.abs_bound(x_bits, W) + 1e-6


def check(y, ref, bound, label):
    got = out_to_f64(y)
    assert got.shape == ref.shape
    tol = bound + half_step(y.dtype) * (np.abs(ref) + bound)
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{label}: {int(bad.sum())} of {bad.size}, worst {float(np.nanmax(err / tol)):.3g} at {np.argwhere(bad)[:4].tolist()}"


def vec(n, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, generator=g).to(dtype).cuda()


def f64(t):
    return t.double().cpu().numpy()


# (n, k, bd, m): every path of the product with ragged edges; the last ones
# reach full 256 x 256 tiles, K splits and neither
SHAPES = [(1, 8, 7, 1), (37, 104, 6, 1), (512, 1024, 8, 1), (100, 1032, 7, 2), (48, 640, 6, 4), (33, 520, 8, 5),
          (130, 2048, 7, 16), (300, 4608, 6, 9), (17, 264, 7, 17), (200, 1032, 8, 40), (515, 648, 6, 63),
          (257, 520, 7, 256), (512, 512, 8, 300), (600, 1544, 6, 515),
          (64, 9728, 7, 16), (90, 264, 8, 129), (20, 65536, 7, 33)]


@pytest.mark.parametrize("n,k,bd,m", SHAPES)
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_epilogue(svq, n, k, bd, m, kind):
    mat = synth.random_matrix(n, k, bd, seed=(70, n, k))
    x_bits = synth.random_activations(m, k, seed=(71, n, m))
    pm, x = svq.pack(mat), to_device_bf16(x_bits)
    out = (torch.float32, torch.bfloat16, torch.bfloat16)[kind]
    p, pb = product(mat, x_bits, m > (4 if kind else 16))
    bias = (None, vec(n, torch.float32, 1), vec(n, torch.bfloat16, 2))[kind]
    res = (vec(m * n, torch.bfloat16, 3).view(m, n), None, vec(m * n, torch.float32, 4).view(m, n))[kind]
    for act in ACTS:
        y = svq.linear_epilogue(pm, x, bias=bias, act=act, residual=res, out_dtype=out)
        v = p + (f64(bias) if bias is not None else 0.0)
        a = act64(v, act)
        r = f64(res) if res is not None else 0.0
        bound = slope_of(act) * (pb + U32 * np.abs(v)) + 16 * U32 * np.abs(a) + U32 * (np.abs(a) + np.abs(r))
        check(y, a + r, bound, f"{act} n={n} k={k} m={m}")


@pytest.mark.parametrize("m", [1, 3, 7, 40, 300])
def test_epilogue_strided_operands_and_neighbours(svq, m):
    """Rows of x, residual and y inside wider buffers at odd offsets, the
    residual in place; nothing beside y's rows is written."""
    n, k, bd = 203, 264, 7
    mat = synth.random_matrix(n, k, bd, seed=(72, n, k))
    x_bits = synth.random_activations(m, k, seed=(72, 1, m))
    xw = torch.zeros((m, k + 13), dtype=torch.bfloat16, device="cuda")
    xw[:, 5:5 + k] = to_device_bf16(x_bits)
    wide = vec((m + 2) * (n + 9), torch.bfloat16, 5).view(m + 2, n + 9)
    before = wide.clone()
    y = wide[1:m + 1, 3:3 + n]
    r = f64(y)
    svq.linear_epilogue(svq.pack(mat), xw[:, 5:5 + k], residual=y, out=y)
    p, pb = product(mat, x_bits, m > 4)
    check(y, p + r, pb + U32 * (np.abs(p) + np.abs(r)), f"in place m={m}")
    wide[1:m + 1, 3:3 + n] = before[1:m + 1, 3:3 + n]
    assert torch.equal(wide, before)


def no_split(svq, n, k, seed):
    """A matrix whose tables admit no split into two fp16 halves."""
    mat = synth.random_matrix(n, k, 7, seed=(73, seed, k))
    mat.radius = mat.radius.copy()
    mat.radius[0], mat.radius[1] = 0x3C01, 0x7B53
    mat.codebook = mat.codebook.copy()
    mat.codebook[0, :] = 0x0001
    pm = svq.pack(mat)
    assert pm.handle.xscale_log2 == svq.SVQ_NO_EXACT_SPLIT
    return mat, pm


def product_bf16(mat, x_bits, m):
    """Without a split: exact up to 16 rows, bf16 weights beyond."""
    p, b = product(mat, x_bits, False)
    W = so.linear_from_inputs(mat, x_bits[:1])[1]
    return p, b + (2.0 ** -8 * so.abs_bound(x_bits, W) if m > 16 else 0.0)


@pytest.mark.parametrize("m", [1, 3, 11, 20, 300])
def test_without_an_exact_split(svq, m):
    """Tables that admit no fp16 split: four rows at a time up to 16 rows (the
    residual follows the rows), the bf16 form beyond; the gated pair as two
    products and a step."""
    n, k = 40, 72
    (mat, pm), (mat2, pm2) = no_split(svq, n, k, 1), no_split(svq, n, k, 2)
    x_bits = synth.random_activations(m, k, seed=(73, 1, m))
    x = to_device_bf16(x_bits)
    res = vec(m * n, torch.float32, 6).view(m, n)
    y = svq.linear_epilogue(pm, x, act="relu", residual=res, out_dtype=torch.float32)
    p, pb = product_bf16(mat, x_bits, m)
    a, r = np.maximum(p, 0), f64(res)
    check(y, a + r, pb + U32 * (np.abs(a) + np.abs(r)), "epilogue")
    u, ub = product_bf16(mat2, x_bits, m)
    y = svq.linear_glu(pm, pm2, x, act="relu", out_dtype=torch.float32)
    check(y, a * u, pb * np.abs(u) + ub * np.abs(a) + pb * ub + U32 * np.abs(a * u), "glu")


def test_moe_without_an_exact_split(svq):
    """The expert layer with one matrix that admits no split: per-slot as ever,
    as separate products beyond."""
    e, f, k, topk = 3, 72, 40, 2
    (gm, gp), (um, up), (dm, dp) = experts(svq, e, f, k, 100), experts(svq, e, f, k, 101), experts(svq, e, k, f, 102)
    gm[1], gp[1] = no_split(svq, f, k, 3)
    for m in (5, 40):
        x_bits = synth.random_activations(m, k, seed=(103, k, m))
        rng = np.random.default_rng([103, m])
        ids = np.stack([rng.permutation(e)[:topk] for _ in range(m)]).astype(np.int32)
        wt = rng.random((m, topk)).astype(np.float32)
        y = svq.moe_ffn(gp, up, dp, to_device_bf16(x_bits), torch.from_numpy(ids).cuda(), torch.from_numpy(wt).cuda(),
                        out_dtype=torch.float32)
        ref, bound = moe64((gm, um, dm), x_bits, ids, wt, "silu", m * topk > 64, bf16=True)
        check(y, ref, bound, f"m={m}")


def test_plain_epilogue_equals_linear(svq):
    """Up to 4 rows the launches and their order of sums are svq_linear's."""
    for n, k, bd, m in SHAPES[:5]:
        mat = synth.random_matrix(n, k, bd, seed=(74, n, k))
        x = to_device_bf16(synth.random_activations(m, k, seed=(74, n, m)))
        pm = svq.pack(mat)
        assert torch.equal(svq.linear_epilogue(pm, x, out_dtype=torch.float32),
                           svq.linear(pm, x, out_dtype=torch.float32))


def test_activations_at_their_limits(svq):
    """Large arguments of either sign, zeros and infinite biases through an
    all-zero product."""
    vals = [0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 20.0, -20.0, 90.0, -90.0, 1e4, -1e4, 3e38, -3e38, math.inf]
    n, k = len(vals), 16
    mat = synth.random_matrix(n, k, 7, seed=(75, n, k))
    pm = svq.pack(mat)
    bias = torch.tensor(vals, dtype=torch.float32, device="cuda")
    for m in (1, 6, 20):
        x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
        for act in ACTS:
            y = f64(svq.linear_epilogue(pm, x, bias=bias, act=act, out_dtype=torch.float32))
            for j, v in enumerate(vals):
                want = v if act == "none" else (max(v, 0.0) if v >= -10 or act == "relu" else None)
                if want is None:  # far negative: silu and gelu vanish
                    assert (np.abs(y[:, j]) <= abs(v) * math.exp(max(v, -700.0)) * 1.01 + 1e-37).all(), (act, v, y[:, j])
                elif abs(v) >= 20 or v == 0 or act in ("none", "relu"):
                    assert np.allclose(y[:, j], want, rtol=1e-6, atol=0), (act, v, y[:, j])


GLU_SHAPES = [(1, 8, 1), (37, 104, 1), (1000, 520, 1), (2000, 2560, 1), (100, 1032, 2), (48, 640, 4), (33, 520, 5),
              (300, 4608, 13), (17, 264, 17), (200, 1032, 40), (257, 520, 256), (512, 1024, 300), (264, 512, 256), (700, 264, 530),
              (40, 9728, 1), (24, 16384, 1), (64, 9728, 16), (90, 264, 129)]


@pytest.mark.parametrize("n,k,m", GLU_SHAPES)
@pytest.mark.parametrize("bds", [(6, 7), (7, 8), (8, 6)])
def test_glu(svq, n, k, m, bds):
    mats = [synth.random_matrix(n, k, bd, seed=(76, n + i, k)) for i, bd in enumerate(bds)]
    x_bits = synth.random_activations(m, k, seed=(76, n, m))
    x = to_device_bf16(x_bits)
    pg, pu = [svq.pack(a) for a in mats]
    for act, bt, out in (("silu", None, torch.bfloat16), ("gelu_tanh", torch.float32, torch.float32),
                         ("none", torch.bfloat16, torch.bfloat16)):
        (g, gb), (u, ub) = [product(a, x_bits, m > (4 if out == torch.bfloat16 else 16)) for a in mats]
        bg = None if bt is None else vec(n, bt, 7)
        bu = None if bt is None or act == "none" else vec(n, bt, 8)
        y = svq.linear_glu(pg, pu, x, act=act, bias_gate=bg, bias_up=bu, out_dtype=out)
        gv = g + (f64(bg) if bg is not None else 0.0)
        uv = u + (f64(bu) if bu is not None else 0.0)
        a = act64(gv, act)
        ea = slope_of(act) * (gb + U32 * np.abs(gv)) + 16 * U32 * np.abs(a)
        eu = ub + U32 * np.abs(uv)
        check(y, a * uv, ea * np.abs(uv) + eu * np.abs(a) + ea * eu + U32 * np.abs(a * uv), f"{act} n={n} k={k} m={m}")


def test_last_round_in_k_ranges(svq):
    """More 256-row tiles than compute units: whole tiles for the full rounds,
    the tiles left over in K ranges that a reduce launch joins; ragged rows
    and columns in both."""
    m, k = 2050, 1032                             # nine tiles of rows, three units
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    n = 256 * (cus // 9 + 1) - 5                  # a few tiles past one round
    mats = [synth.random_matrix(n, k, bd, seed=(98, n, bd)) for bd in (7, 8)]
    x_bits = synth.random_activations(m, k, seed=(98, n, m))
    x = to_device_bf16(x_bits)
    (g, gb), (u, ub) = [product(a, x_bits, True) for a in mats]
    pg, pu = [svq.pack(a) for a in mats]
    bias, res = vec(n, torch.float32, 19), vec(m * n, torch.bfloat16, 20).view(m, n)
    y = svq.linear_epilogue(pg, x, bias=bias, act="relu", residual=res)
    v, r = g + f64(bias), f64(res)
    a = np.maximum(v, 0)
    check(y, a + r, gb + U32 * np.abs(v) + U32 * (a + np.abs(r)), "epilogue")
    y = svq.linear_glu(pg, pu, x, act="relu", bias_up=bias, out_dtype=torch.float32)
    a, b = np.maximum(g, 0), u + f64(bias)
    eb = ub + U32 * np.abs(b)
    check(y, a * b, gb * np.abs(b) + eb * a + gb * eb + U32 * np.abs(a * b), "glu")
    first = y.clone()
    assert torch.equal(svq.linear_glu(pg, pu, x, act="relu", bias_up=bias, out_dtype=torch.float32), first)


@pytest.mark.parametrize("out,res_type", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
                                          (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_whole_tiles_with_aligned_residual(svq, out, res_type, act):
    """256-row tiles in one K range, aligned rows of y and residual, the last
    columns fewer than four; in place where the types agree; nothing beside
    y's columns is written."""
    n, k, m, ld = 515, 264, 290, 520
    mat = synth.random_matrix(n, k, 7, seed=(99, n, k))
    x_bits = synth.random_activations(m, k, seed=(99, n, m))
    wide = vec(m * ld, out, 21).view(m, ld)
    before, y = wide.clone(), wide[:, :n]
    res = y if out == res_type else vec(m * ld, res_type, 22).view(m, ld)[:, :n]
    r, bias = f64(res), vec(n, torch.float32, 23)
    svq.linear_epilogue(svq.pack(mat), to_device_bf16(x_bits), bias=bias, act=act, residual=res, out=y)
    p, pb = product(mat, x_bits, True)
    v = p + f64(bias)
    a = act64(v, act)
    bound = slope_of(act) * (pb + U32 * np.abs(v)) + 16 * U32 * np.abs(a) + U32 * (np.abs(a) + np.abs(r))
    check(y, a + r, bound, act)
    assert torch.equal(wide[:, n:], before[:, n:])


def route64(x, w, topk, score, renorm, scale, sb):
    logits = f64(x) @ f64(w).T
    if score == "softmax":
        z = np.exp(logits - logits.max(axis=1, keepdims=True))
        p = z / z.sum(axis=1, keepdims=True)
    else:
        p = 1 / (1 + np.exp(-logits))
    key = logits if sb is None else p + f64(sb)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :topk]
    wt = np.take_along_axis(p, ids, axis=1)
    if renorm:
        wt = wt / wt.sum(axis=1, keepdims=True)
    return ids, wt * scale


@pytest.mark.parametrize("m,e,k,topk", [(1, 1, 1, 1), (1, 128, 2048, 8), (3, 8, 7, 2), (5, 256, 520, 32),
                                        (257, 60, 264, 6), (300, 17, 1032, 17), (600, 129, 512, 4), (2100, 200, 136, 8)])
@pytest.mark.parametrize("score,renorm,scale,biased", [("softmax", True, 1.0, False), ("sigmoid", True, 2.5, True),
                                                       ("softmax", False, 1.0, True), ("sigmoid", False, 1.0, False)])
def test_route(svq, m, e, k, topk, score, renorm, scale, biased):
    x = to_device_bf16(synth.random_activations(m, k, seed=(77, e, m)))
    w = (vec(e * k, torch.float32, 9).view(e, k) / math.sqrt(k))
    sb = 0.1 * vec(e, torch.float32, 10) if biased else None
    for wt in (w.bfloat16(), w):
        ids, weights = svq.moe_route(x, wt, topk, score=score, renormalize=renorm, scale=scale, select_bias=sb)
        rid, rwt = route64(x, wt, topk, score, renorm, scale, sb)
        assert np.array_equal(ids.cpu().numpy(), rid)
        # the double scores carry far less error than the one rounding to fp32
        assert (np.abs(f64(weights) - rwt) <= U32 * 1.001 * np.abs(rwt) + 1e-40).all()


def test_route_ties_and_strides(svq):
    """Equal router rows: the lower index first.  Rows inside wider buffers at
    odd offsets (no 16-byte alignment)."""
    m, e, k, topk = 9, 40, 136, 12
    x = torch.zeros((m, k + 11), dtype=torch.bfloat16, device="cuda")
    x[:, 3:3 + k] = vec(m * k, torch.bfloat16, 11).view(m, k)
    w = torch.zeros((e, k + 5), dtype=torch.bfloat16, device="cuda")
    w[:, 1:1 + k] = vec(8 * k, torch.bfloat16, 12).view(8, k).repeat(5, 1)
    ids, weights = svq.moe_route(x[:, 3:3 + k], w[:, 1:1 + k], topk)
    rid, rwt = route64(x[:, 3:3 + k], w[:, 1:1 + k], topk, "softmax", True, 1.0, None)
    logits = f64(x[:, 3:3 + k]) @ f64(w[:8, 1:1 + k]).T
    order = np.argsort(-logits, axis=1, kind="stable")
    want = np.stack([np.concatenate([[c + 8 * r for r in range(5)] for c in row])[:topk] for row in order])
    assert np.array_equal(ids.cpu().numpy(), want)
    assert np.allclose(f64(weights), rwt, rtol=1e-6)


def test_route_with_nan_and_infinite_logits(svq):
    """A NaN router row is chosen after every number, ids stay distinct."""
    x = torch.ones((2, 8), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((5, 8), dtype=torch.float32, device="cuda")
    w[0, 0], w[1, 0], w[3, 0], w[4, 0] = math.nan, -math.inf, 2.0, -0.0
    ids, _ = svq.moe_route(x, w, 5)
    assert ids.cpu().tolist() == [[3, 2, 4, 1, 0]] * 2
    ids, weights = svq.moe_route(x, w, 2, score="sigmoid", renormalize=False)
    assert ids.cpu().tolist() == [[3, 2]] * 2
    assert np.allclose(f64(weights), [[1 / (1 + math.exp(-2)), 0.5]] * 2, rtol=1e-6)


def experts(svq, e, n, k, seed):
    mats = [synth.random_matrix(n, k, 6 + (i + seed) % 3, seed=(seed, i, n)) for i in range(e)]
    return mats, [svq.pack(a) for a in mats]


def moe64(sets, x_bits, ids, wt, act, grouped, bf16=False):
    """(y without the residual, bound) from the definition."""
    m, topk = ids.shape
    gates, ups, downs = sets
    e, out = len(gates), downs[0].n
    y, b = np.zeros((m, out)), np.zeros((m, out))
    wr = (2.0 ** -8 if bf16 else 2.0 ** -11) if grouped else 0.0
    hr = 2.0 ** -8 if bf16 and grouped else 2.0 ** -11
    for t in range(m):
        xb = x_bits[t:t + 1]
        for j in range(topk):
            i = int(ids[t, j])
            if i < 0 or i >= e:
                continue
            (g, gb), (u, ub) = [(product_bf16(a[i], xb, 64) if bf16 and grouped else product(a[i], xb, grouped))
                                  for a in (gates, ups)]
            a = act64(g, act)
            h = a * u
            eh = (slope_of(act) * gb + 16 * U32 * np.abs(a)) * np.abs(u) + ub * np.abs(a) + slope_of(act) * gb * ub
            eh = eh + (hr + U32) * (np.abs(h) + eh)
            eh = eh + 2.0 ** -38 * np.abs(h).max()  # fp16 after a scale: a floor of 2^-39 of the largest value
            _, Wd = so.linear_from_inputs(downs[i], np.zeros((1, downs[i].k), dtype=np.uint16))
            d = h @ Wd.T
            ed = eh @ np.abs(Wd).T + (downs[i].k * U32 + 64 * U32 + wr) * ((np.abs(h) + eh) @ np.abs(Wd).T) + 1e-6
            y[t] += wt[t, j] * d[0]
            b[t] += abs(wt[t, j]) * (ed[0] + topk * U32 * (np.abs(d[0]) + ed[0]))
    return y, b


# (experts, inner, k, m, topk): one slot; few slots; the last per-slot sizes
# (64 slots) and the first grouped ones; an odd inner width of one unit and
# more than one
MOE_SHAPES = [(1, 8, 8, 1, 1), (4, 104, 264, 1, 2), (8, 520, 136, 3, 4), (6, 72, 1032, 16, 4), (6, 200, 264, 13, 5),
              (5, 96, 520, 40, 3), (12, 264, 72, 70, 2), (130, 24, 40, 3, 8), (130, 24, 40, 30, 4),
              (130, 24, 40, 45, 4)]


@pytest.mark.parametrize("e,f,k,m,topk", MOE_SHAPES)
@pytest.mark.parametrize("kind", [0, 1])
def test_moe_ffn(svq, e, f, k, m, topk, kind):
    n = k + 8 * kind
    (gm, gp), (um, up), (dm, dp) = experts(svq, e, f, k, 80), experts(svq, e, f, k, 81), experts(svq, e, n, f, 82)
    rng = np.random.default_rng([83, e, m])
    x_bits = synth.random_activations(m, k, seed=(84, k, m))
    ids = np.stack([rng.permutation(e)[:topk] for _ in range(m)]).astype(np.int32)
    if kind and m * topk > 2:
        ids[0, 0], ids[-1, -1] = -1, e            # slots without an expert
        ids[m // 2, 0] = ids[m // 2, topk - 1]    # one expert twice
    wt = rng.random((m, topk)).astype(np.float32)
    wt[0, -1] = -0.5
    d_wt = torch.from_numpy(wt.copy()).cuda()
    if kind and m * topk > 2:
        d_wt[0, 0] = math.nan                     # its weight does not matter
    out = (torch.bfloat16, torch.float32)[kind]
    res = vec(m * n, torch.bfloat16, 13).view(m, n) if kind else None
    act = ("silu", "gelu_tanh")[kind]
    y = svq.moe_ffn(gp, up, dp, to_device_bf16(x_bits), torch.from_numpy(ids).cuda(), d_wt, act=act, residual=res,
                    out_dtype=out)
    ref, bound = moe64((gm, um, dm), x_bits, ids, wt, act, m * topk > max(64, e * 5 // 4))
    if res is not None:
        ref = ref + f64(res)
        bound = bound + U32 * (np.abs(ref) + bound)
    check(y, ref, bound, f"moe e={e} f={f} k={k} m={m}")


def test_moe_ffn_long_rows(svq):
    """Rows too long for a block's LDS: a few slots through the grouped form;
    an inner width beyond it is refused."""
    e, f, k, m = 2, 8, 40000, 3
    (gm, gp), (um, up), (dm, dp) = experts(svq, e, f, k, 105), experts(svq, e, f, k, 106), experts(svq, e, 24, f, 107)
    x_bits = synth.random_activations(m, k, seed=(105, k, m))
    ids = np.array([[0], [1], [1]], dtype=np.int32)
    wt = np.ones((m, 1), dtype=np.float32)
    y = svq.moe_ffn(gp, up, dp, to_device_bf16(x_bits), torch.from_numpy(ids).cuda(), torch.from_numpy(wt).cuda(),
                    out_dtype=torch.float32)
    ref, bound = moe64((gm, um, dm), x_bits, ids, wt, "silu", True)
    check(y, ref, bound, "long rows")


@pytest.mark.parametrize("m", [5, 90])
def test_moe_ffn_in_place_and_all_slots_empty(svq, m):
    e, f, k, topk = 4, 40, 72, 2
    _, gp = experts(svq, e, f, k, 85)
    _, up = experts(svq, e, f, k, 86)
    _, dp = experts(svq, e, k, f, 87)
    x = to_device_bf16(synth.random_activations(m, k, seed=(85, k, m)))
    ids = torch.full((m, topk), -7, dtype=torch.int32, device="cuda")
    wt = torch.ones((m, topk), device="cuda")
    y = vec(m * k, torch.bfloat16, 14).view(m, k)
    before = y.clone()
    svq.moe_ffn(gp, up, dp, x, ids, wt, residual=y, out=y)
    assert torch.equal(y, before)
    assert not svq.moe_ffn(gp, up, dp, x, ids, wt).any()
    ids.zero_()
    a = svq.moe_ffn(gp, up, dp, x, ids, wt, residual=before, out_dtype=torch.bfloat16)
    svq.moe_ffn(gp, up, dp, x, ids, wt, residual=y, out=y)
    assert torch.equal(y, a)


def _block(svq, pms, x, moe):
    """A feed-forward block as a model runs it: dense gated pair, down
    projection added to the stream, then router and experts added to it."""
    gate, up, down, router, gs, us, ds = pms
    h = svq.linear_glu(gate, up, x)
    x1 = svq.linear_epilogue(down, h, residual=x)
    if not moe:
        return x1
    ids, wt = svq.moe_route(x1, router, 2)
    return svq.moe_ffn(gs, us, ds, x1, ids, wt, residual=x1)


def _block_weights(svq, k=264, f=520, e=6, fe=104):
    mats = [synth.random_matrix(*s, seed=(90, *s[:2])) for s in ((f, k, 7), (f, k, 8), (k, f, 6))]
    sets = [experts(svq, e, fe, k, 91), experts(svq, e, fe, k, 92), experts(svq, e, k, fe, 93)]
    router = (vec(e * k, torch.float32, 15).view(e, k) / 8).bfloat16()
    return mats, [s[0] for s in sets], [*map(svq.pack, mats), router, *[s[1] for s in sets]]


def _graded(m, k, seed):
    """Activations of 2^-4 .. 2^2 in bf16, either sign: times 2^-122 .. 2^118
    they are normal numbers still."""
    v = vec(m * k, torch.float32, seed).view(m, k)
    return (torch.sign(v) * v.abs().clamp(2.0 ** -4, 4.0)).bfloat16()


@pytest.mark.parametrize("m", [1, 3, 7, 20, 150, 300])
@pytest.mark.parametrize("shift", [-122, 100])
def test_activations_of_any_power_of_two(svq, m, shift):
    """Every rounding of a product is relative to a power-of-two scale, so x
    times 2^shift gives y times 2^shift, to the last bit while every sum is
    normal; one below 2^-126 is held in steps of 2^-149, half of one for each
    of at most k + 64 roundings.  The gated pair: with the up matrix's sums
    far below its bias of 1 it is the gate's product, with bias 0 and shift
    halved it is homogeneous of degree two."""
    n, k = 72, 1032
    tiny = (k + 64) * 2.0 ** -150
    pg, pu = [svq.pack(synth.random_matrix(n, k, bd, seed=(94, bd, k))) for bd in (7, 8)]
    x = _graded(m, k, 16)
    xs = (x.float() * 2.0 ** shift).bfloat16()
    y = svq.linear_epilogue(pg, x, out_dtype=torch.float32)
    ys = svq.linear_epilogue(pg, xs, out_dtype=torch.float32)
    assert (np.abs(f64(ys) - f64(y) * 2.0 ** shift) <= tiny).all()
    half = (x.float() * 2.0 ** (shift // 2)).bfloat16()
    z = svq.linear_glu(pg, pu, x, act="none", out_dtype=torch.float32)
    zs = svq.linear_glu(pg, pu, half, act="none", out_dtype=torch.float32)
    assert (np.abs(f64(zs) - f64(z) * 2.0 ** shift) <= tiny).all()
    if shift < 0:
        one = torch.ones(n, device="cuda")
        zs = svq.linear_glu(pg, pu, xs, act="none", bias_up=one, out_dtype=torch.float32)
        W = so.linear_from_inputs(synth.random_matrix(n, k, 7, seed=(94, 7, k)), np.zeros((1, k), dtype=np.uint16))[1]
        p, a = f64(xs) @ W.T, np.abs(f64(xs)) @ np.abs(W).T
        # as product(): sums, the weights' rounding, subnormal weights (2^-39
        # of the largest, 0.2, times k values of x, against a weight of 2^-6 at
        # least on average: 2^-25 k of the sum over them)
        assert (np.abs(f64(zs) - p) <= ((k + 64) * U32 + 2.0 ** -11 + k * 2.0 ** -25) * a + tiny).all()


@pytest.mark.parametrize("m", [5, 90])
@pytest.mark.parametrize("shift", [-58, 50])
def test_moe_ffn_activations_of_any_power_of_two(svq, m, shift):
    """Without an activation the expert layer is homogeneous of degree two in
    x: h of about 2^(2 shift) and its scale reach the ends of fp32.  An h
    below 2^-126 is held in steps of 2^-149, which may turn its rounding to
    fp16 (11 bits) the other way: one step of 2^-137 at most, times a weight."""
    e, f, k, topk = 3, 104, 264, 2
    gm, gp = experts(svq, e, f, k, 95)
    um, up = experts(svq, e, f, k, 96)
    dm, dp = experts(svq, e, k, f, 97)
    x = _graded(m, k, 17)
    g = torch.Generator().manual_seed(18)
    ids = torch.stack([torch.randperm(e, generator=g)[:topk] for _ in range(m)]).to(torch.int32).cuda()
    wt = torch.rand((m, topk), generator=g).cuda()
    y = svq.moe_ffn(gp, up, dp, x, ids, wt, act="none", out_dtype=torch.float32)
    ys = svq.moe_ffn(gp, up, dp, (x.float() * 2.0 ** shift).bfloat16(), ids, wt, act="none", out_dtype=torch.float32)
    wmax = max(float(np.abs(so.linear_from_inputs(d, np.zeros((1, f), dtype=np.uint16))[1]).sum(axis=1).max()) for d in dm)
    assert (np.abs(f64(ys) - f64(y) * 2.0 ** (2 * shift)) <= topk * (wmax + 2) * 2.0 ** -137).all()


@pytest.mark.parametrize("m", [1, 4, 16, 48, 300])
def test_run_of_them_together(svq, m):
    """The whole block against 64 bits, stage by stage on the stages' own
    inputs, and repeated calls bit for bit."""
    mats, sets, pms = _block_weights(svq)
    x_bits = synth.random_activations(m, 264, seed=(90, 1, m))
    x = to_device_bf16(x_bits)
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)
    h = svq.linear_glu(pms[0], pms[1], x)
    (g, gb), (u, ub) = [product(a, x_bits, m > 4) for a in mats[:2]]
    a = act64(g, "silu")
    ea = SLOPE * gb + 16 * U32 * np.abs(a)
    check(h, a * u, ea * np.abs(u) + ub * np.abs(a) + ea * ub + U32 * np.abs(a * u), "glu")
    x1 = svq.linear_epilogue(pms[2], h, residual=x)
    p, pb = product(mats[2], bits(h), m > 4)
    check(x1, p + f64(x), pb + U32 * (np.abs(p) + np.abs(f64(x))), "down")
    ids, wt = svq.moe_route(x1, pms[3], 2)
    rid, rwt = route64(x1, pms[3], 2, "softmax", True, 1.0, None)
    assert np.array_equal(ids.cpu().numpy(), rid)
    y = svq.moe_ffn(*pms[4:], x1, ids, wt, residual=x1)
    ref, bound = moe64(sets, bits(x1), rid, f64(wt), "silu", 2 * m > 64)
    ref = ref + f64(x1)
    check(y, ref, bound + U32 * (np.abs(ref) + bound), "moe")
    for _ in range(3):
        assert torch.equal(_block(svq, pms, x, True), y)


@pytest.mark.parametrize("m", [1, 4, 12, 48])
def test_captured_and_replayed(svq, m):
    """Two graphs of the block that share their call objects' workspaces,
    replayed in turn with new inputs and eager work between: every replay
    equals the eager result."""
    _, _, (gate, up, down, router, gs, us, ds) = _block_weights(svq)
    dev = dict(device="cuda")
    x = torch.zeros((m, 264), dtype=torch.bfloat16, **dev)
    h = torch.zeros((m, 520), dtype=torch.bfloat16, **dev)
    x1, y = torch.zeros_like(x), torch.zeros_like(x)
    ids = torch.zeros((m, 2), dtype=torch.int32, **dev)
    wt = torch.zeros((m, 2), **dev)
    ws = torch.empty(32 << 20, dtype=torch.uint8, **dev)
    calls = [svq.GluCall(gate, up, x, h, workspace=ws), svq.EpilogueCall(down, h, x1, residual=x, workspace=ws),
             svq.MoeRouteCall(x1, router, ids, wt, workspace=ws),
             svq.MoeFfnCall(gs, us, ds, x1, ids, wt, y, residual=x1, workspace=ws)]
    for c in calls:
        c()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            for c in calls:
                c()
    for i in range(6):
        xi = to_device_bf16(synth.random_activations(m, 264, seed=(94, i, m)))
        want = _block(svq, (gate, up, down, router, gs, us, ds), xi, True)
        x.copy_(xi)
        y.fill_(float("nan"))
        ws.fill_(0xFF if i % 2 else 0x5A)  # what lies in the workspace does not matter
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), f"replay {i}"


def test_captured_large_calls_in_one_workspace(svq):
    """Pairs of 256-row tiles that meet through memory (one unit, so whole
    tiles) and K ranges with their reduce launch, captured on one workspace
    that holds anything before each replay."""
    m, f, k = 300, 1100, 512
    gate, up = [svq.pack(synth.random_matrix(f, k, bd, seed=(100, bd, k))) for bd in (7, 8)]
    down = svq.pack(synth.random_matrix(k, f - f % 8, 6, seed=(101, k, f)))
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    h = torch.zeros((m, f), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    calls = [svq.GluCall(gate, up, x, h, workspace=ws),
             svq.EpilogueCall(down, h, y, residual=x, workspace=ws)]
    for c in calls:
        c()
        assert c.workspace is ws
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    for i in range(5):
        xi = to_device_bf16(synth.random_activations(m, k, seed=(102, i, m)))
        hi = svq.linear_glu(gate, up, xi)
        want = svq.linear_epilogue(down, hi, residual=xi)
        x.copy_(xi)
        h.fill_(float("nan"))
        y.fill_(float("nan"))
        ws.fill_((0xFF, 0x00, 0x01)[i % 3])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, hi) and torch.equal(y, want), f"replay {i}"


def test_on_another_stream(svq):
    """Calls given a stream run in that stream's order."""
    _, _, (gate, up, down, router, gs, us, ds) = _block_weights(svq)
    s = torch.cuda.Stream()
    for m in (1, 9, 40):
        x = to_device_bf16(synth.random_activations(m, 264, seed=(95, 0, m)))
        want = _block(svq, (gate, up, down, router, gs, us, ds), x, True)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            late = torch.empty_like(x)
            torch.cuda._sleep(2_000_000)
            late.copy_(x)
        h = svq.linear_glu(gate, up, late, stream=s)
        x1 = svq.linear_epilogue(down, h, residual=late, stream=s)
        ids, wt = svq.moe_route(x1, router, 2, stream=s)
        y = svq.moe_ffn(gs, us, ds, x1, ids, wt, residual=x1, stream=s)
        s.synchronize()
        assert torch.equal(y, want)
