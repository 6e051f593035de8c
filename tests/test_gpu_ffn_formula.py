"""One activation formula for the whole of an output: tensors whose columns
are finished by different kernels (256-row tiles in one K range, tiles left
over in K ranges and joined by a launch of their own, ragged last columns)."""
import math

import numpy as np
import pytest

import synth
from oracle import svq_oracle as so
from tests.gpu_common import out_to_f64, require_gpu, to_device_bf16, torch
from tests.test_gpu_ffn import U32, act64, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svq():
    return require_gpu()


def _equal_rows(n, k, bd, seed):
    """A matrix of n equal rows, and the first of them.  1536 channels are 192
    codes, 432 whole bytes a row."""
    assert k // 8 * 18 % 8 == 0
    mat = synth.random_matrix(n, k, bd, seed=seed)
    mat.codes = np.tile(mat.codes[:k // 8 * 18 // 8], n)
    W = so.linear_from_inputs(mat, np.zeros((1, k), dtype=np.uint16))[1]
    assert (W == W[0]).all()
    return mat, W[0]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_equal_columns_are_equal(svq, act, out):
    """Every weight row is the same and x has one value a row, so a product is
    one weight times a power of two: exact up to the weight's rounding to fp16
    (the same in every column), and all columns have to be bit for bit equal.
    The bias brings the argument to -24 .. 24, where an exponential's argument
    rounded to fp32 would show in an fp32 output.

    The values' bound: silu and gelu_tanh are v sigma(s(v)), s = v or
    2 sqrt(2/pi) (v + 0.044715 v^3).  An argument off by d (2^-11 |p| of the
    weight's rounding, 2^-24 |v| of the bias's sum) and an s off by e (4
    roundings of it for the cubic) change that by at most
    sigma (d + |v| (s' d + e)) to first order, since sigma' <= sigma; over
    steps with s' d + e < 0.3, as here, sigma grows by e^0.3 at most: twice
    the first order covers it.  gelu: slope 1.13.  Then 16 roundings of the
    value (expf, one division)."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    m, k = 2050, 1536
    n = 256 * (cus // 9 + 1) - 5
    (mat, w), (mat2, w2) = _equal_rows(n, k, 7, (140, 1)), _equal_rows(n, k, 8, (140, 2))
    cols = (np.arange(m) * 7) % k
    x_bits = np.zeros((m, k), dtype=np.uint16)
    x_bits[np.arange(m), cols] = 0x3F80 + ((np.arange(m) % 4) << 7)  # 1, 2, 4, 8
    x, pg, pu = to_device_bf16(x_bits), svq.pack(mat), svq.pack(mat2)
    x64 = so.bf16_bits_to_f64(x_bits).max(axis=1)
    p, u = (w[cols] * x64)[:, None], (w2[cols] * x64)[:, None]
    for b in (-24.0, -7.0, 0.5, 24.0):
        bias = torch.full((n,), b, dtype=torch.float32, device="cuda")
        res = torch.full((m, n + 1), 0.25, dtype=torch.bfloat16, device="cuda")[:, :n]  # odd stride: unaligned rows
        aligned = torch.full((m, n + 5), 0.25, dtype=torch.bfloat16, device="cuda")[:, :n]
        v = p + b
        d = 2.0 ** -11 * np.abs(p) + U32 * np.abs(v)
        if act == "gelu":
            a, move = act64(v, act), 1.13 * d
        else:
            c = 2 * math.sqrt(2 / math.pi)
            e, ds, sv = (0.0, 1.0, v) if act == "silu" else \
                (4 * U32 * np.abs(c * (v + 0.044715 * v ** 3)), c * (1 + 3 * 0.044715 * v ** 2), c * (v + 0.044715 * v ** 3))
            assert (ds * d + e < 0.3).all()
            with np.errstate(over="ignore"):
                sigma = 1 / (1 + np.exp(-sv))
            # as v sigma: (1 + tanh z) / 2 = sigma(2 z), and the sum with tanh
            # has no digits left in 64 bits from z = -18 on
            a, move = v * sigma, 2 * sigma * (d + np.abs(v) * (ds * d + e))
        rel = 16 * U32
        for r in (None, res, aligned):
            y = svq.linear_epilogue(pg, x, bias=bias, act=act, residual=r, out_dtype=out)
            assert torch.equal(y, y[:, :1].expand_as(y)), (act, b)
            ref = a + (0.0 if r is None else 0.25)
            tol = rel * np.abs(a) + move + U32 * np.abs(ref)
            got = out_to_f64(y[:, :1])
            assert (np.abs(got - ref) <= tol + half_step(out) * (np.abs(ref) + tol)).all(), (act, b)
        h = svq.linear_glu(pg, pu, x, act=act, bias_gate=bias, out_dtype=out)
        assert torch.equal(h, h[:, :1].expand_as(h)), (act, b)
        ref = a * u
        tol = (rel * np.abs(a) + move) * np.abs(u) * (1 + 2.0 ** -11) + np.abs(a * u) * (2.0 ** -11 + U32)
        got = out_to_f64(h[:, :1])
        assert (np.abs(got - ref) <= tol + half_step(out) * (np.abs(ref) + tol)).all(), (act, b)
