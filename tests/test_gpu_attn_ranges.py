"""Prompt attention with few rows for many keys, whose keys are worked on in
ranges that a second launch joins."""
import itertools

import pytest

from tests.attn_common import P_BF16, attend, check, visible
from tests.gpu_common import require_gpu, torch

pytestmark = pytest.mark.gpu


def _starts(lens, first=0):
    return torch.tensor([first] + list(itertools.accumulate(lens, initial=first))[1:], dtype=torch.int32, device="cuda")


def _rows(n, cols, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(n, cols, generator=g)).to(torch.bfloat16).cuda()


def _run(svq, q, k, v, starts, dim, ranges=True, **kw):
    """The call on a workspace of NaN; it has ranges if the workspace holds
    more than nothing."""
    y = torch.full_like(q, 7.0)
    size = svq.AttnPromptCall(q, k, v, y, starts, dim, **kw).ws_size.value
    assert (size > 256) == ranges
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    svq.AttnPromptCall(q, k, v, y, starts, dim, workspace=ws, **kw)()
    torch.cuda.synchronize()
    return y


def _check(y, q, k, v, lens, lens_k, heads, kv, dim, causal, window, scale=None, first=0):
    at, at_k = first, 0
    for i, (n, nk) in enumerate(zip(lens, lens_k)):
        if n:
            ref = attend(q[at:at + n], k[at_k:at_k + nk], v[at_k:at_k + nk], heads, kv,
                         dim ** -0.5 if scale is None else scale, visible(n, nk, causal, window))
            check(y[at:at + n], *ref, nk, P_BF16, f"sequence {i} ({n} of {nk})")
        at += n
        at_k += nk


CASES = [
    # lens, lens_k (None: as lens), heads, kv, dim, causal, window
    ([1024], None, 1, 1, 64, True, 0),                # the fewest keys that have ranges
    ([1500], None, 1, 1, 64, True, 0),
    ([1501], None, 2, 1, 128, True, 0),
    ([2100], None, 4, 1, 256, True, 0),
    ([1], [4000], 1, 1, 128, True, 0),                # sixteen ranges of one row
    ([3], [4097], 7, 1, 64, True, 0),
    ([40], [3000], 16, 2, 128, True, 0),
    ([1300], None, 1, 1, 128, False, 0),
    ([700], [2000], 2, 2, 256, False, 0),
    ([2900], None, 1, 1, 64, True, 1000),
    ([1100, 1200], None, 2, 1, 128, True, 0),
    ([1900, 0, 1, 2900], None, 1, 1, 128, True, 0),   # ranges without a key
    ([900, 5, 30], [600, 4000, 3], 4, 1, 64, True, 0),  # rows that see nothing
    ([1800, 1700], None, 1, 1, 128, True, 1000),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0][:3]}-{'' if c[1] is None else c[1][:3]}-h{c[2]}x{c[3]}-d{c[4]}-{'c' if c[5] else 'f'}{c[6]}")
def test_against_64_bits(case):
    svq = require_gpu()
    lens, lens_k, heads, kv, dim, causal, window = case
    nk = lens if lens_k is None else lens_k
    q, k, v = _rows(sum(lens), heads * dim, 1), _rows(sum(nk), kv * dim, 2), _rows(sum(nk), kv * dim, 3)
    y = _run(svq, q, k, v, _starts(lens), dim, starts_k=None if lens_k is None else _starts(nk), causal=causal,
             window=window)
    _check(y, q, k, v, lens, nk, heads, kv, dim, causal, window)


def test_many_rows_have_no_ranges():
    svq = require_gpu()
    q, k = _rows(2048, 16 * 128, 1), _rows(2048, 16 * 128, 2)
    _run(svq, q, k, k.clone(), _starts([2048]), 128, ranges=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_that_are_not_finite(dim):
    """A hidden key has no influence; single infinite and NaN values reach the
    rows that see them, whatever range they lie in, and no other column."""
    svq = require_gpu()
    heads, kv, n = 2, 1, 1400
    q, k, v = _rows(n, heads * dim, 5), _rows(n, kv * dim, 6), _rows(n, kv * dim, 7)
    v2, k2 = v.clone(), k.clone()
    v2[20, 3], v2[1050, 3], v2[1370, 5], v2[640, 8] = float("inf"), float("-inf"), float("-inf"), float("nan")
    k2[1390], v2[1390] = float("nan"), float("inf")
    y = _run(svq, q, k2, v2, _starts([n]), dim)
    assert not torch.isfinite(y[1390:].float()).any()
    ref = attend(q, k, v, heads, kv, dim ** -0.5, visible(n, n))
    got = y.float().cpu().view(n, heads, dim)[:1390]
    cols = [c for c in range(dim) if c not in (3, 5, 8)]
    ref = [r.view(n, heads, -1)[:1390] for r in ref]
    pick = lambda r, at: r[:, :, at] if r.shape[2] > 1 else r
    check(got[:, :, cols].reshape(1390, -1), *(pick(r, cols).expand(-1, -1, len(cols)).reshape(1390, -1) for r in ref), n, P_BF16)
    for c, first in ((3, 20), (5, 1370), (8, 640)):
        check(got[:first, :, c], *(pick(r, [c])[:first, :, 0] for r in ref), n, P_BF16, f"column {c}")
    assert torch.all(got[20:1050, :, 3] == float("inf")) and torch.isnan(got[1050:, :, 3]).all()
    assert torch.all(got[1370:, :, 5] == float("-inf")) and torch.isnan(got[640:, :, 8]).all()


@pytest.mark.parametrize("scale", [0.0, 3.0, -1.0, 300.0])
def test_scales(scale):
    svq = require_gpu()
    heads, kv, dim, n = 2, 1, 128, 1100
    q, k, v = _rows(n, heads * dim, 11), _rows(n, kv * dim, 12), _rows(n, kv * dim, 13)
    y = _run(svq, q, k, v, _starts([n]), dim, scale=scale)
    _check(y, q, k, v, [n], [n], heads, kv, dim, True, 0, scale=scale)


@pytest.mark.parametrize("offset", [-3e37, -1e4, 1e4, 3e37])
def test_scores_far_from_zero(offset):
    svq = require_gpu()
    heads, kv, dim, n = 2, 1, 64, 1100
    q, k, v = _rows(n, heads * dim, 14), _rows(n, kv * dim, 15), _rows(n, kv * dim, 16)
    q.view(n, heads, dim)[:, :, 0] = 1.0
    k[:, 0] = offset
    if abs(offset) > 1e30:
        q.view(n, heads, dim)[:, :, 1:] = 0  # in fp32 the shift swallows the rest
    y = _run(svq, q, k, v, _starts([n]), dim)
    _check(y, q, k, v, [n], [n], heads, kv, dim, True, 0)


def test_one_range_takes_all():
    """Scores of one range beyond those of every other by more than fp32's
    exponents span."""
    svq = require_gpu()
    dim, n = 64, 1200
    q, k, v = torch.zeros(n, dim).bfloat16().cuda(), torch.zeros(n, dim).bfloat16().cuda(), _rows(n, dim, 17)
    q[:, 0] = 1.0
    k[:, 0] = torch.linspace(-30000, 30000, n).bfloat16().cuda()
    for flip in (1.0, -1.0):
        y = _run(svq, q, (flip * k).contiguous(), v, _starts([n]), dim)
        _check(y, q, (flip * k).contiguous(), v, [n], [n], 1, 1, dim, True, 0)


def test_rows_left_alone():
    svq = require_gpu()
    heads, kv, dim, n = 2, 1, 64, 2300
    q, k, v = _rows(n, heads * dim, 17), _rows(n, kv * dim, 18), _rows(n, kv * dim, 19)
    y = _run(svq, q, k, v, _starts([1200, 1000], 33), dim)
    assert torch.all(y[:33] == 7.0) and torch.all(y[2233:] == 7.0)
    _check(y, q, k[33:], v[33:], [1200, 1000], [1200, 1000], heads, kv, dim, True, 0, first=33)
    y = _run(svq, q, k, v, torch.tensor([-9, 1200, 5000], dtype=torch.int32, device="cuda"), dim)
    _check(y, q, k, v, [1200, 1100], [1200, 1100], heads, kv, dim, True, 0)


def test_same_bits_captured_and_on_another_stream():
    svq = require_gpu()
    heads, kv, dim, n = 4, 1, 128, 2400
    q, k, v = _rows(n, heads * dim, 21), _rows(n, kv * dim, 22), _rows(n, kv * dim, 23)
    y, starts = torch.zeros_like(q), _starts([1000, 1400])
    call = svq.AttnPromptCall(q, k, v, y, starts, dim)
    assert call.ws_size.value > 256
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for step in range(4):
        starts.copy_(_starts([1000 + 400 * step, 1400 - 400 * step]))
        k.mul_(1.5)
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, svq.attn_prompt(q, k, v, starts, dim))
