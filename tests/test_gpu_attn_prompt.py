"""Attention of whole prompts (svq_attn_prompt) against 64 bits."""
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


def _check(y, q, k, v, lens, lens_k, heads, kv, dim, causal, window, scale=None, first=0, first_k=0):
    at, at_k = first, first_k
    scale = dim ** -0.5 if scale is None else scale
    for i, (n, nk) in enumerate(zip(lens, lens_k)):
        if n:
            ref = attend(q[at:at + n], k[at_k:at_k + nk], v[at_k:at_k + nk], heads, kv, scale,
                         visible(n, nk, causal, window))
            check(y[at:at + n], *ref, nk, P_BF16, f"sequence {i} ({n} of {nk})")
        at += n
        at_k += nk


CASES = [
    # lens, lens_k (None: as lens), heads, kv, dim, causal, window
    ([1], None, 1, 1, 64, True, 0),
    ([1], None, 8, 2, 128, True, 0),
    ([2, 1, 3], None, 7, 1, 256, True, 0),
    ([31, 32, 33], None, 4, 1, 128, True, 0),
    ([63, 64, 65], None, 2, 2, 64, True, 0),
    ([127, 130], None, 5, 1, 128, True, 0),
    ([255, 1, 258], None, 2, 1, 256, True, 0),
    ([300], None, 8, 2, 128, True, 0),
    ([5, 0, 70, 0, 0, 1], None, 6, 3, 64, True, 0),
    ([97, 40], None, 4, 2, 128, False, 0),
    ([1, 200], None, 3, 3, 64, False, 0),
    ([66, 19], None, 2, 1, 256, False, 0),
    ([130, 77], None, 4, 1, 128, True, 1),
    ([130, 77], None, 4, 1, 64, True, 2),
    ([300, 9], None, 2, 2, 128, True, 63),
    ([200, 70], None, 4, 1, 128, True, 64),
    ([260], None, 1, 1, 256, True, 65),
    ([150], None, 4, 4, 64, True, 1000),
    ([3, 40, 1], [70, 40, 129], 4, 2, 128, True, 0),       # a prefix in front
    ([3, 40, 1], [70, 40, 129], 4, 2, 64, True, 50),
    ([9, 33], [200, 1], 2, 1, 128, False, 0),
    ([40, 70, 8], [3, 65, 0], 4, 2, 128, True, 0),         # fewer keys than queries: rows without a key
    ([40, 70, 8], [3, 65, 0], 2, 1, 256, True, 7),
    ([5, 6], [0, 9], 2, 2, 64, False, 0),
    ([12, 100], None, 64, 1, 64, True, 0),                 # 64 query heads share one key head
    ([7] * 70 + [1] * 70, None, 2, 1, 64, True, 0),        # more sequences than lanes
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0][:3]}-{'' if c[1] is None else c[1][:3]}-h{c[2]}x{c[3]}-d{c[4]}-{'c' if c[5] else 'f'}{c[6]}")
def test_against_64_bits(case):
    svq = require_gpu()
    lens, lens_k, heads, kv, dim, causal, window = case
    nk = lens if lens_k is None else lens_k
    q = _rows(sum(lens), heads * dim, 1)
    k, v = _rows(max(sum(nk), 1), kv * dim, 2), _rows(max(sum(nk), 1), kv * dim, 3)
    y = svq.attn_prompt(q, k, v, _starts(lens), dim, starts_k=None if lens_k is None else _starts(nk), causal=causal,
                        window=window)
    torch.cuda.synchronize()
    _check(y, q, k, v, lens, nk, heads, kv, dim, causal, window)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_columns_of_wider_rows_and_rows_left_alone(dim):
    """q, k and v as columns of one buffer; y inside a wider buffer; rows
    before the first sequence and behind the last, and the other columns, stay
    as they were; what lies there and between sequences is NaN."""
    svq = require_gpu()
    heads, kv, lens, first = 4, 2, [37, 90], 5
    total = first + sum(lens) + 11
    wide = _rows(total, (heads + 2 * kv) * dim + 16, 4)
    wide[:first] = float("nan")
    wide[first + sum(lens):] = float("nan")
    q = wide[:, 8:8 + heads * dim]
    k = wide[:, 8 + heads * dim:8 + (heads + kv) * dim]
    v = wide[:, 8 + (heads + kv) * dim:8 + (heads + 2 * kv) * dim]
    buf = torch.full((total, heads * dim + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[:, 16:16 + heads * dim]
    svq.attn_prompt(q, k, v, _starts(lens, first), dim, out=y)
    torch.cuda.synchronize()
    _check(y, q, k, v, lens, lens, heads, kv, dim, True, 0, first=first, first_k=first)
    rest = buf.clone()
    rest[first:first + sum(lens), 16:16 + heads * dim] = 7.0
    assert torch.all(rest == 7.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_hidden_keys_have_no_influence(bad, dim):
    """One key's row and value are not finite: the queries that see it have no
    number to give, the others are what they are without it."""
    svq = require_gpu()
    heads, kv, n, window = 4, 2, 150, 40
    q, k, v = _rows(n, heads * dim, 5), _rows(n, kv * dim, 6), _rows(n, kv * dim, 7)
    at = 77
    k2, v2 = k.clone(), v.clone()
    k2[at], v2[at] = bad, bad
    for w in (0, window):
        y = svq.attn_prompt(q, k2, v2, _starts([n]), dim, window=w)
        torch.cuda.synchronize()
        hidden = ~visible(n, n, True, w)[:, at]
        ref = attend(q, k, v, heads, kv, dim ** -0.5, visible(n, n, True, w))
        check(y[hidden.cuda()], *(r[hidden] for r in ref), n, P_BF16, f"window {w}")
        assert not torch.isfinite(y[(~hidden).cuda()].float()).any()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_infinite_values_of_seen_keys(dim):
    """Single infinite and NaN values: their columns become infinite or NaN in
    the rows that see them, everything else keeps its value."""
    svq = require_gpu()
    heads, kv, n = 2, 1, 100
    q, k, v = _rows(n, heads * dim, 8), _rows(n, kv * dim, 9), _rows(n, kv * dim, 10)
    v2 = v.clone()
    v2[20, 3], v2[50, 3], v2[70, 5], v2[40, 8] = float("inf"), float("-inf"), float("-inf"), float("nan")
    y = svq.attn_prompt(q, k, v2, _starts([n]), dim).float().cpu()
    torch.cuda.synchronize()
    ref = attend(q, k, v, heads, kv, dim ** -0.5, visible(n, n))
    got = y.view(n, heads, dim)
    cols = [c for c in range(dim) if c not in (3, 5, 8)]
    check(got[:, :, cols].reshape(n, -1), *(r.view(n, heads, dim)[:, :, cols].reshape(n, -1) for r in ref), n, P_BF16)
    for c, first in ((3, 20), (5, 70), (8, 40)):
        check(got[:first, :, c], *(r.view(n, heads, dim)[:first, :, c] for r in ref), n, P_BF16, f"column {c}")
    assert torch.all(got[20:50, :, 3] == float("inf")) and torch.isnan(got[50:, :, 3]).all()
    assert torch.all(got[70:, :, 5] == float("-inf")) and torch.isnan(got[40:, :, 8]).all()


@pytest.mark.parametrize("scale", [0.0, 3.0, -1.0, 300.0])
def test_scales(scale):
    """Scores of all sizes: equal ones (the mean of the values), and so far
    apart that one key takes all."""
    svq = require_gpu()
    heads, kv, dim, n = 2, 1, 128, 140
    q, k, v = _rows(n, heads * dim, 11), _rows(n, kv * dim, 12), _rows(n, kv * dim, 13)
    y = svq.attn_prompt(q, k, v, _starts([n]), dim, scale=scale)
    _check(y, q, k, v, [n], [n], heads, kv, dim, True, 0, scale=scale)


@pytest.mark.parametrize("offset", [-3e37, -1e4, 1e4, 3e37])
def test_scores_far_from_zero(offset):
    """Every score of a row shifted by the same amount (channel 0 of the keys
    is constant): the softmax is the same."""
    svq = require_gpu()
    heads, kv, dim, n = 2, 1, 64, 90
    q, k, v = _rows(n, heads * dim, 14), _rows(n, kv * dim, 15), _rows(n, kv * dim, 16)
    q.view(n, heads, dim)[:, :, 0] = 1.0
    k[:, 0] = offset
    if abs(offset) > 1e30:
        q.view(n, heads, dim)[:, :, 1:] = 0  # in fp32 the shift swallows the rest
    y = svq.attn_prompt(q, k, v, _starts([n]), dim)
    _check(y, q, k, v, [n], [n], heads, kv, dim, True, 0)


def test_starts_beyond_the_rows():
    svq = require_gpu()
    heads, kv, dim, n = 2, 1, 64, 50
    q, k, v = _rows(n, heads * dim, 17), _rows(n, kv * dim, 18), _rows(n, kv * dim, 19)
    starts = torch.tensor([-9, 20, 2000, 5000], dtype=torch.int32, device="cuda")
    y = torch.full_like(q, 7.0)
    svq.attn_prompt(q, k, v, starts, dim, out=y)
    _check(y, q, k, v, [20, 30], [20, 30], heads, kv, dim, True, 0)


def test_same_bits_every_time_captured_and_on_another_stream():
    svq = require_gpu()
    heads, kv, dim, lens = 8, 2, 128, [130, 1, 400, 77]
    n = sum(lens)
    q, k, v = _rows(n, heads * dim, 20), _rows(n, kv * dim, 21), _rows(n, kv * dim, 22)
    y = torch.empty_like(q)
    starts = _starts(lens)
    call = svq.AttnPromptCall(q, k, v, y, starts, dim)
    call()
    torch.cuda.synchronize()
    first = y.clone()
    assert torch.equal(first, svq.attn_prompt(q, k, v, starts, dim))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(first, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(3):
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, y)
        # other lengths in the same captured launch
        starts.copy_(_starts(lens[::-1]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, svq.attn_prompt(q, k, v, starts, dim))
        starts.copy_(_starts(lens))


def test_rows_past_32_bits():
    """Sequences whose rows lie beyond 2^32 bytes of their buffers."""
    svq = require_gpu()
    heads, kv, dim, lens = 2, 1, 128, [40, 100]
    total, ld = 140000, 16384
    wide = torch.zeros((total, ld), dtype=torch.bfloat16, device="cuda")
    first = total - sum(lens)
    assert first * ld * 2 > 1 << 32
    cols = (heads + 2 * kv) * dim
    wide[first:, 512:512 + cols] = _rows(sum(lens), cols, 23)
    q = wide[:, 512:512 + heads * dim]
    k = wide[:, 512 + heads * dim:512 + (heads + kv) * dim]
    v = wide[:, 512 + (heads + kv) * dim:512 + cols]
    y = wide[:, 8192:8192 + heads * dim]
    svq.attn_prompt(q, k, v, _starts(lens, first), dim, out=y)
    torch.cuda.synchronize()
    _check(y, q, k, v, lens, lens, heads, kv, dim, True, 0, first=first, first_k=first)
    assert torch.all(y[:first] == 0)


def test_more_tiles_than_one_launch_takes():
    """64 query heads a key head leave two tokens a tile: 2^17 tokens are more
    tiles than the grid's second dimension."""
    svq = require_gpu()
    heads, kv, dim, n, each = 64, 1, 64, 1 << 17, 61
    lens = [each] * (n // each) + [n % each]
    q = _rows(n, heads * dim, 24)
    k, v = _rows(n, kv * dim, 25), _rows(n, kv * dim, 26)
    y = svq.attn_prompt(q, k, v, _starts(lens), dim)
    torch.cuda.synchronize()
    for s in (0, 1, 1000, len(lens) - 2, len(lens) - 1):
        at, m = s * each, lens[s]
        rows = slice(at, at + m)
        check(y[rows], *attend(q[rows], k[rows], v[rows], heads, kv, dim ** -0.5, visible(m, m)), m, P_BF16, f"sequence {s}")
    assert torch.isfinite(y.float()).all() and torch.all(y.float().abs().sum(dim=1) > 0)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 45, 3, 0])
def test_windows_wider_than_the_keys(window):
    """Queries whose positions lie before the first key beside some that see
    keys, under windows up to the largest number."""
    svq = require_gpu()
    lens, lens_k, dim = [45, 2], [3, 40], 64
    q, k, v = _rows(47, 4 * dim, 1), _rows(43, 2 * dim, 2), _rows(43, 2 * dim, 3)
    y = svq.attn_prompt(q, k, v, _starts(lens), dim, starts_k=_starts(lens_k), window=window)
    torch.cuda.synchronize()
    _check(y, q, k, v, lens, lens_k, 4, 2, dim, True, window)
    assert torch.all(y[:42] == 0) and torch.all(y[42:].abs().sum(dim=1) > 0)
