"""Infinities and NaN among the activations, at every row count whose products
have a path of their own: an infinite activation makes an infinite output of
the weight's sign (NaN where both signs meet, or in the definition's own
0 * inf), a NaN a NaN, and the other rows keep their values.

The finite rows are checked with the bounds of tests/test_gpu_ffn.py; infinite
and NaN outputs have none: they are what 64 bits give or not.
"""
import math

import numpy as np
import pytest

import synth
from oracle import svq_oracle as so
from tests.gpu_common import out_to_f64, require_gpu, to_device_bf16, torch
from tests.test_gpu_ffn import U32, act64, half_step, slope_of

pytestmark = pytest.mark.gpu

INF, NINF, NAN = 0x7F80, 0xFF80, 0x7FC0
# what a row holds beside finite values: (channel seed, bit pattern) pairs
KINDS = [(), ((3, INF),), ((5, NINF),), ((7, NAN),), ((3, INF), (11, NINF)), ((3, INF), (13, INF))]


@pytest.fixture(scope="module")
def svq():
    return require_gpu()


def rows(m, k, first, seed):
    """uint16 bf16 rows, row t of kind first + t, with finite values of up to
    about 2^9 around the infinities."""
    x = synth.random_activations(m, k, seed=seed)
    x[:, ::9] += 8 << 7  # times 2^8
    for t in range(m):
        for c, bits in KINDS[(first + t) % len(KINDS)]:
            x[t, (c * 37 + 5 * t) % k] = bits
    return x


def product64(mat, x_bits, rounded):
    """(p, bound): every product and sum as 64-bit arithmetic does them."""
    W = so.linear_from_inputs(mat, np.zeros((1, mat.k), dtype=np.uint16))[1]
    assert (W != 0).all()
    x = so.bf16_bits_to_f64(x_bits)
    with np.errstate(invalid="ignore"):
        p = np.stack([(W * r).sum(axis=1) for r in x])
    rel = (mat.k + 64) * U32 + (2.0 ** -11 if rounded else 0.0)
    return p, rel * (np.where(np.isfinite(x), np.abs(x), 0.0) @ np.abs(W).T) + 1e-6


def check(y, ref, bound, label):
    got = out_to_f64(y)
    odd = ~np.isfinite(ref)
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    bad = odd & ~same
    assert not bad.any(), f"{label}: {int(bad.sum())} of {int(odd.sum())} non-finite outputs at {np.argwhere(bad)[:4].tolist()}: " \
                          f"{got[bad][:4].tolist()} for {ref[bad][:4].tolist()}"
    ok = np.abs(got[~odd] - ref[~odd]) <= bound[~odd] + half_step(y.dtype) * (np.abs(ref[~odd]) + bound[~odd])
    assert ok.all(), f"{label}: {int((~ok).sum())} finite outputs outside tolerance"


SIZES = [(40, 72, 1), (40, 4104, 1), (24, 1032, 3), (40, 520, 4), (40, 520, 5), (33, 1032, 16), (24, 9728, 16), (40, 520, 17),
         (40, 1032, 66), (40, 264, 129), (280, 264, 300)]


def cases(sizes):
    """Every kind in turn where a call has fewer rows than there are kinds."""
    return [(n, k, m, first) for n, k, m in sizes for first in range(len(KINDS) if m < len(KINDS) else 2)]


@pytest.mark.parametrize("n,k,m,first", cases(SIZES))
def test_epilogue(svq, n, k, m, first):
    mat = synth.random_matrix(n, k, 7, seed=(120, n, k))
    x_bits = rows(m, k, first, (120, k, m))
    pm, x = svq.pack(mat), to_device_bf16(x_bits)
    for out in (torch.float32, torch.bfloat16):
        p, b = product64(mat, x_bits, m > (16 if out == torch.float32 else 4))
        for act in ("none", "relu", "silu"):
            with np.errstate(invalid="ignore", over="ignore"):
                a = act64(p, act)
            y = svq.linear_epilogue(pm, x, act=act, out_dtype=out)
            check(y, a, slope_of(act) * b + 16 * U32 * np.abs(a), f"{act} {out} m={m}")


@pytest.mark.parametrize("n,k,m,first", cases(SIZES + [(24, 16384, 1), (20, 4608, 9)]))
def test_glu(svq, n, k, m, first):
    mats = [synth.random_matrix(n, k, bd, seed=(121, n + bd, k)) for bd in (6, 8)]
    x_bits = rows(m, k, first, (121, k, m))
    pg, pu = [svq.pack(a) for a in mats]
    x = to_device_bf16(x_bits)
    for out in (torch.float32, torch.bfloat16):
        (g, gb), (u, ub) = [product64(a, x_bits, m > (16 if out == torch.float32 else 4)) for a in mats]
        for act in ("relu", "silu"):
            with np.errstate(invalid="ignore", over="ignore"):
                a = act64(g, act)
                ref = a * u
                ea = slope_of(act) * gb + 16 * U32 * np.abs(a)
                bound = ea * np.abs(u) + ub * np.abs(a) + ea * ub + U32 * np.abs(ref)
            check(svq.linear_glu(pg, pu, x, act=act, out_dtype=out), ref, bound, f"{act} {out} m={m}")


@pytest.mark.parametrize("n,k,m", [(40, 520, 1), (40, 1032, 4), (40, 520, 9), (33, 1032, 16), (40, 520, 40)])
def test_plain_product(svq, n, k, m):
    """svq_linear's paths share the staging of activations."""
    mat = synth.random_matrix(n, k, 8, seed=(122, n, k))
    for first in range(len(KINDS)):
        x_bits = rows(m, k, first, (122, k, m))
        p, b = product64(mat, x_bits, False)
        if m > 16:
            W = so.linear_from_inputs(mat, np.zeros((1, k), dtype=np.uint16))[1]
            x = so.bf16_bits_to_f64(x_bits)
            b = b + 2.0 ** -8 * (np.where(np.isfinite(x), np.abs(x), 0.0) @ np.abs(W).T)
        check(svq.linear(svq.pack(mat), to_device_bf16(x_bits), out_dtype=torch.float32), p, b, f"kind {first} m={m}")


def _one_overflow(f, k):
    """Gate and up matrices and a row x for which exactly one gate * up
    exceeds fp32, by a hundredth at least, and the others stay a factor of two
    below."""
    for seed in range(400):
        gate, up = [synth.random_matrix(f, k, 7, seed=(123, i, seed)) for i in (1, 2)]
        x_bits = synth.random_activations(1, k, seed=(123, 3, seed))
        (g, _), (u, _) = [so.linear_from_inputs(a, x_bits) for a in (gate, up)]
        z = np.sort(np.abs(g * u)[0])
        s = math.ceil(math.log2(2.0 ** 128 / z[-1] * 1.01) / 2)
        if (2.0 ** s) ** 2 * z[-2] < 2.0 ** 127:
            # times 2^s: bf16 exponents (random activations are normal numbers or zero)
            bits = np.where(x_bits & 0x7F80, x_bits + np.uint16(s << 7), x_bits).astype(np.uint16)
            return gate, up, bits
    raise AssertionError("no such row among the seeds")


@pytest.mark.parametrize("m", [1, 3, 90])
def test_one_infinite_inner_value(svq, m):
    """gate * up overflows fp32 in one of the inner channels: the outputs are
    infinite with the sign of that channel's weight, in the per-slot form (up
    to 64 slots) and the grouped one."""
    f, k, n = 8, 40, 56
    gate, up, row = _one_overflow(f, k)
    down = synth.random_matrix(n, f, 8, seed=(124, n, f))
    x = to_device_bf16(np.repeat(row, m, axis=0))
    ids = torch.zeros((m, 1), dtype=torch.int32, device="cuda")
    wt = torch.full((m, 1), 0.5, device="cuda")
    y = svq.moe_ffn([svq.pack(gate)], [svq.pack(up)], [svq.pack(down)], x, ids, wt, act="none", out_dtype=torch.float32)
    (g, _), (u, _), W = so.linear_from_inputs(gate, row), so.linear_from_inputs(up, row), \
        so.linear_from_inputs(down, np.zeros((1, f), dtype=np.uint16))[1]
    h = (g * u)[0]
    j = int(np.argmax(np.abs(h)))
    assert (W[:, j] != 0).all()
    want = np.sign(h[j]) * np.sign(W[:, j]) * math.inf
    assert np.array_equal(out_to_f64(y), np.repeat(want[None], m, axis=0))


@pytest.mark.parametrize("m", [2, 4, 6, 16, 30, 150, 300])
def test_other_rows_are_the_same(svq, m):
    """Rows without an infinity or NaN, bit for bit as beside rows without
    one, in every call and output type."""
    n, k, e, f, topk = 72, 1032, 3, 40, 2
    clean = synth.random_activations(m, k, seed=(125, m))
    dirty = clean.copy()
    for i, t in enumerate(range(0, m, 3)):
        dirty[t, (i * 37) % k] = (INF, NINF, NAN)[i % 3]
    keep = torch.tensor([t for t in range(m) if t % 3], device="cuda")
    pg, pu = [svq.pack(synth.random_matrix(n, k, bd, seed=(125, bd))) for bd in (7, 8)]
    sets = [[svq.pack(synth.random_matrix(a, b, 7, seed=(126, s, i))) for i in range(e)]
            for s, (a, b) in enumerate(((f, k), (f, k), (k, f)))]
    g = torch.Generator().manual_seed(33)
    ids = torch.stack([torch.randperm(e, generator=g)[:topk] for _ in range(m)]).to(torch.int32).cuda()
    wt = torch.rand((m, topk), generator=g).cuda()
    router = torch.randn((e, k), generator=g).cuda()
    for out in (torch.float32, torch.bfloat16):
        for run in (lambda x: svq.linear_epilogue(pg, x, act="silu", out_dtype=out),
                    lambda x: svq.linear_glu(pg, pu, x, out_dtype=out),
                    lambda x: svq.moe_ffn(*sets, x, ids, wt, residual=x, out_dtype=out),
                    lambda x: svq.moe_route(x, router, topk)[1]):
            a, b = run(to_device_bf16(clean)), run(to_device_bf16(dirty))
            assert torch.isfinite(a).all() and torch.equal(a[keep], b[keep])
