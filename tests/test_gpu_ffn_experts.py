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
