"""The attention calls at the ends of their range: scores far from zero,
scales of every size, values and queries of very different sizes, more tiles
than a launch takes, and rows beside others that see more."""
import pytest

from tests.attn_common import P_BF16, P_F16, attend, cache_floor, check, stored, visible
from tests.gpu_common import require_gpu, torch

pytestmark = pytest.mark.gpu

FORMS = [(d, g) for d in (64, 128, 256) for g in (32, 64, 128) if g <= d]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _rows(n, cols, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(n, cols, generator=g)).to(torch.bfloat16).cuda()


def _one_sequence(svq, k, v, kv, dim, group, page=16):
    """A cache that holds one sequence on pages in falling order."""
    n = k.shape[0]
    need = -(-n // page)
    cache = svq.KvCache(need + 1, page, kv, dim, group=group)
    cache.buf.fill_(255)
    pages = list(range(need, 0, -1))
    _write(svq, cache, k, v, pages, 0)
    return cache, pages, _ints([pages])


def _write(svq, cache, k, v, pages, first):
    page = int(cache.desc.page_size)
    slots = [pages[j // page] * page + j % page for j in range(first, first + k.shape[0])]
    svq.kv_write(cache, k.contiguous(), v.contiguous(), _ints(slots))


# ---- turns of tiles ---------------------------------------------------------

def test_more_sequences_than_a_launch_takes():
    """65535 sequences of one token are as many tiles beside 511 that are not
    there, in two launches; a token that sees itself alone gets its value."""
    svq = require_gpu()
    n, dim = 65535, 64
    q, k, v = _rows(n, dim, 1), _rows(n, dim, 2), _rows(n, dim, 3)
    starts = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    y = svq.attn_prompt(q, k, v, starts, dim)
    torch.cuda.synchronize()
    gone = torch.nonzero((y != v).any(dim=1))[:, 0].tolist()
    assert not gone, f"{len(gone)} rows from {gone[0]} on"


# ---- scores far from zero ---------------------------------------------------
#
# Keys whose scores are fp32 numbers: channel 0 brings 255 * 2^26 (q 255 * 2^13,
# k 2^13), another channel j * 1024, the fp32 step there.  So the products and
# their sums are exact, and a score's error is that of its difference to the
# greatest one times the scale: relative 2^-22 for the product and the rounded
# scale, of at most 64 where it matters (weights below e^-64 do not): 2^-16.
FAR_ERR = 2.0 ** -16
FAR_SCALES = [2.0 ** -14, 2.0 ** -10, 2.0 ** -6, 0.125, 8.0]


def _far(n, dim, step, base=255):
    """q row and keys [n, dim]; key j's score is base * 2^26 + step[j] * 1024.  Every
    group of 32 channels is held exactly in 4 bits: a constant one, or whole
    numbers from 0 to 15."""
    q, k = torch.zeros(1, dim), torch.zeros(n, dim)
    q[0, 0], k[:, :32] = base * 2.0 ** 13, 2.0 ** 13
    q[0, 32] = 1024.0
    k[:, 32], k[:, 33] = step, 15.0
    return q.to(torch.bfloat16).cuda(), k.to(torch.bfloat16).cuda()


def _far_reference(step, v, scale):
    p = torch.softmax(torch.as_tensor(step).double() * 1024 * scale, dim=0)
    v = v.detach().cpu().double()
    return (p @ v)[None], (p @ v.abs())[None], torch.full((1, v.shape[1]), FAR_ERR, dtype=torch.float64)


def _steps(n, kind):
    j = torch.arange(n)
    if kind == "late":      # the greatest by one step, in a late tile
        return (j == n - 3).float()
    if kind == "rising":
        return (j * 16 // n).float()
    if kind == "falling":
        return 15.0 - (j * 16 // n).float()
    return (j * 7 % 16).float()


@pytest.mark.parametrize("kind", ["late", "rising", "falling", "mixed"])
@pytest.mark.parametrize("scale", FAR_SCALES)
@pytest.mark.parametrize("n", [200, 1300])
def test_prompt_scores_one_step_apart(n, scale, kind):
    svq = require_gpu()
    step = _steps(n, kind)
    for dim in (64, 128, 256):
        q, k = _far(n, dim, step)
        v = _rows(n, dim, 4)
        y = svq.attn_prompt(q, k, v, _ints([0, 1]), dim, starts_k=_ints([0, n]), scale=scale)
        check(y, *_far_reference(step, v, scale), n, P_BF16, f"{dim} channels")


@pytest.mark.parametrize("n", [1000, 1600])  # without and with ranges of keys
@pytest.mark.parametrize("base,below", [(241, 0.1), (248, 1.1), (250, 0.2), (255, 7.4)])
def test_prompt_scores_that_pass_two_to_the_24th(base, below, n):
    """Most keys' scores lie a little below 2^24 (base 2), one ten beyond it;
    how both are formed changes there."""
    svq = require_gpu()
    scale = (2.0 ** 24 - below) / (base * 2.0 ** 26 * 1.4426950408889634)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    for dim in (64, 128, 256):
        step = torch.zeros(n)
        step[600] = 10
        q, k = _far(n, dim, step, base)
        v = _rows(n, dim, 4)
        y = svq.attn_prompt(q, k, v, _ints([0, 1]), dim, starts_k=_ints([0, n]), scale=scale)
        check(y, *_far_reference(step, v, scale), n, P_BF16, f"{dim} channels")


@pytest.mark.parametrize("kind", ["late", "rising", "falling", "mixed"])
@pytest.mark.parametrize("scale", FAR_SCALES)
@pytest.mark.parametrize("size", [2.0 ** -20, 1.0, 2.0 ** 20])
def test_cache_scores_one_step_apart(size, scale, kind):
    svq = require_gpu()
    n = 700
    step = _steps(n, kind)
    for dim, group in ((64, 32), (128, 32), (256, 32)):
        q, k = _far(n, dim, step)
        v = _rows(n, dim, 5, size)
        cache, _, table = _one_sequence(svq, k, v, 1, dim, group)
        values = stored(v, group)
        for plan in (None, 64 * n):
            if plan:  # many ranges
                table = torch.cat([table, torch.full((1, 64 * n // 16 + 1), -1, dtype=torch.int32, device="cuda")], dim=1)
            y = svq.attn_cache(cache, q, table, _ints([n]), max_len=plan, scale=scale)
            check(y, *_far_reference(step, values, scale), n, P_F16, f"{dim} channels", floor=cache_floor(values, n))


@pytest.mark.parametrize("size", [2.0 ** -14, 2.0 ** -20, 1.0, 1e6, 2.0 ** 20])
@pytest.mark.parametrize("dim,group", FORMS)
def test_cache_of_one_token_with_a_far_score(dim, group, size):
    """A token that is seen alone gives its value, whatever its score."""
    svq = require_gpu()
    for q0, k0 in ((1e5, 3e4), (-1e5, 3e4), (3e10, 3e10), (1e3, 1e3)):
        q, k, v = torch.zeros(1, dim).bfloat16().cuda(), torch.zeros(1, dim).bfloat16().cuda(), _rows(1, dim, 6, size)
        q[0, 0], k[0, 0] = q0, k0
        cache, _, table = _one_sequence(svq, k, v, 1, dim, group)
        values = stored(v, group)
        y = svq.attn_cache(cache, q, table, _ints([1])).double().cpu()
        lim = cache_floor(values, 1) + 2.0 ** -8 * 1.01 * values.abs() + 64 * 2.0 ** -24 * values.abs()
        assert bool(((y - values).abs() <= lim).all()), (q0, k0)


@pytest.mark.parametrize("offset", [-3e37, -1e4, 1e4, 3e37])
def test_cache_scores_far_from_zero(offset):
    """A group of channels shifts every score by about the same amount."""
    svq = require_gpu()
    heads, kv, dim, group, n = 4, 2, 128, 32, 300
    q, k, v = _rows(2, heads * dim, 7), _rows(n, kv * dim, 8), _rows(n, kv * dim, 9)
    q.view(2, heads, dim)[:, :, :32] = 0
    q.view(2, heads, dim)[:, :, 0] = 1.0
    k.view(n, kv, dim)[:, :, :32] = offset
    if abs(offset) > 1e30:
        q.view(2, heads, dim)[:, :, 1:] = 0  # in fp32 the shift swallows the rest
    cache, _, table = _one_sequence(svq, k, v, kv, dim, group)
    y = svq.attn_cache(cache, q, table, _ints([n]), q_len=2)
    ks, vs = stored(k, group), stored(v, group)
    check(y, *attend(q, ks, vs, heads, kv, dim ** -0.5, visible(2, n)), n, P_F16, floor=cache_floor(vs, n))


# ---- scales -----------------------------------------------------------------

@pytest.mark.parametrize("over_cache", [False, True])
@pytest.mark.parametrize("scale", [3.4e38, -3.4e38, 2.5e38])
def test_largest_scales(scale, over_cache):
    """One key takes all, where the greatest score is further from the second
    than fp32 sums are off: (d + 8) 2^-24 of the sum of magnitudes each."""
    svq = require_gpu()
    dim, n = 128, 150
    q, k, v = _rows(n, dim, 10), _rows(n, dim, 11), _rows(n, dim, 12)
    if over_cache:
        cache, _, table = _one_sequence(svq, k, v, 1, dim, 32)
        k, v = stored(k, 32), stored(v, 32)
        y = svq.attn_cache(cache, q, table, _ints([n]), q_len=n, scale=scale)
    else:
        y = svq.attn_prompt(q, k, v, _ints([0, n]), dim, scale=scale)
    q, k, v, y = (t.cpu().double() for t in (q, k, v, y))
    s = q @ k.T * (1 if scale > 0 else -1)
    s = s.masked_fill(~visible(n, n), -float("inf"))
    mag = (q.abs() @ k.abs().T).max(dim=1).values
    top = torch.topk(s, 2, dim=1)
    clear = top.values[:, 0] - top.values[:, 1] > 2 * (dim + 8) * 2.0 ** -24 * mag
    assert int(clear.sum()) > n - 10
    want = v[top.indices[:, 0]]
    lim = 2.0 ** -8 * 1.01 * want.abs() + (cache_floor(v, n) if over_cache else 0) + 64 * 2.0 ** -24 * want.abs()
    assert bool(((y - want).abs() <= lim)[clear].all())


@pytest.mark.parametrize("over_cache", [False, True])
@pytest.mark.parametrize("scale", [0.0, 1e-39, -1e-39, 2e-38])
def test_smallest_scales_of_great_scores(scale, over_cache):
    """Scores from 0 to 2^126 under scales that are subnormal or zero.  The
    scale is an fp32 number of 2^-149 at least, so its product with log2 e is
    off by 2^-150, relative 2^-20 at 1e-39: less than the (d + 8) 2^-24 of a
    score."""
    svq = require_gpu()
    dim, n = 64, 160
    q, k, v = torch.zeros(1, dim), torch.zeros(n, dim), _rows(n, dim, 13)
    q[0, 0] = 2.0 ** 63
    k[:, 0] = (torch.arange(n) % 16) * 2.0 ** 59
    k[:, 1] = 15 * 2.0 ** 59
    q, k = q.to(torch.bfloat16).cuda(), k.to(torch.bfloat16).cuda()
    exact = float(torch.tensor(scale, dtype=torch.float32))
    if over_cache:
        cache, _, table = _one_sequence(svq, k, v, 1, dim, 32)
        assert torch.equal(stored(k, 32), k.double().cpu())
        values = stored(v, 32)
        y = svq.attn_cache(cache, q, table, _ints([n]), scale=scale)
    else:
        values = v
        y = svq.attn_prompt(q, k, v, _ints([0, 1]), dim, starts_k=_ints([0, n]), scale=scale)
    check(y, *attend(q, k, values, 1, 1, exact, visible(1, n)), n, P_F16 if over_cache else P_BF16,
          floor=cache_floor(values, n) if over_cache else 0.0)


# ---- values and queries of different sizes ----------------------------------

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [100, 1100])  # without and with ranges of keys
def test_prompt_values_near_the_largest(n, dim):
    """Later keys whose weights are 2^7 times the first ones', which is no reason
    for a new reference; values of 2^121, so that 30 of them are a number."""
    svq = require_gpu()
    q, k = torch.zeros(1, dim), torch.zeros(n, dim)
    q[0, 0] = 1.0
    k[70:100, 0] = 4.875
    v = torch.sign(_rows(n, dim, 39).float()) * 2.0 ** 121
    v[:70] = 2.0 ** 100
    v[100:] = 2.0 ** 90
    v[70:100, ::2] = 2.0 ** 121
    q, k, v = q.to(torch.bfloat16).cuda(), k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16)
    y = svq.attn_prompt(q, k, v, _ints([0, 1]), dim, starts_k=_ints([0, n]), scale=1.0)
    check(y, *attend(q, k, v, 1, 1, 1.0, visible(1, n, False)), n, P_BF16)


@pytest.mark.parametrize("dim,group", FORMS)
@pytest.mark.parametrize("size", [2.0 ** -112, 2.0 ** -105, 2.0 ** -88, 2.0 ** 90, 2.0 ** 110, 2.0 ** 122])
def test_cache_values_of_one_size(size, dim, group):
    """The smallest and the largest values, under weights from 1 to 2^-20."""
    svq = require_gpu()
    n = 300
    q, k = torch.zeros(1, dim), torch.zeros(n, dim)
    q[0, 0] = 1.0
    k[:, 0], k[:, 1] = (torch.arange(n) * 5 % 16).float(), 15.0
    q, k, v = q.to(torch.bfloat16).cuda(), k.to(torch.bfloat16).cuda(), _rows(n, dim, 14, size)
    cache, _, table = _one_sequence(svq, k, v, 1, dim, group)
    values = stored(v, group)
    y = svq.attn_cache(cache, q, table, _ints([n]), scale=1.0)
    check(y, *attend(q, stored(k, group), values, 1, 1, 1.0, visible(1, n)), n, P_F16, floor=cache_floor(values, n))


@pytest.mark.parametrize("dim,group", FORMS)
@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("small", [0.0, 2.0 ** -100, 1.0])
def test_cache_values_of_different_sizes_side_by_side(small, size, dim, group):
    """32 tokens of large values among as small ones: which tokens' sums a wave
    holds does not change their weights."""
    svq = require_gpu()
    for n, planned in ((128, None), (600, 20000)):
        q, k, v = _rows(1, dim, 15), _rows(n, dim, 16), _rows(n, dim, 17).float() * small
        v[32:64] = _rows(32, dim, 18).float() * size
        v = v.to(torch.bfloat16)
        cache, _, table = _one_sequence(svq, k, v, 1, dim, group)
        if planned:
            table = torch.cat([table, torch.full((1, planned // 16 + 1), -1, dtype=torch.int32, device="cuda")], dim=1)
        values = stored(v, group)
        y = svq.attn_cache(cache, q, table, _ints([n]), max_len=planned)
        check(y, *attend(q, stored(k, group), values, 1, 1, dim ** -0.5, visible(1, n)), n, P_F16,
              floor=cache_floor(values, n))


@pytest.mark.parametrize("dim,group", FORMS)
@pytest.mark.parametrize("size", [1.0, 20.0, 2.0 ** 40, 2.0 ** 120])
def test_cache_constant_values_of_both_signs_behind_zeros(size, dim, group):
    """Groups that are their minimum alone, of another size than a wave has met
    before.  512 sequences (on the same pages) are blocks enough for one range,
    three chunks a wave."""
    svq = require_gpu()
    n, batch = 300, 512
    q, k = _rows(1, dim, 37), _rows(n, dim, 38)
    v = torch.zeros(n, dim)
    v[150:] = (torch.arange(n - 150) % 2 * 2.0 - 1.0)[:, None] * size
    v[160:163] *= 0.5
    v = v.to(torch.bfloat16).cuda()
    cache, _, table = _one_sequence(svq, k, v, 1, dim, group)
    values = stored(v, group)
    assert torch.equal(values, v.cpu().double())
    call = svq.AttnCacheCall(cache, q.repeat(batch, 1), torch.empty_like(q).repeat(batch, 1), table.repeat(batch, 1),
                             _ints([n] * batch))
    assert call.ws_size.value <= 256
    call()
    y = call.keep[2]
    assert torch.equal(y[:1].expand(batch, dim), y)
    check(y[:1], *attend(q, stored(k, group), values, 1, 1, dim ** -0.5, visible(1, n)), n, P_F16, floor=cache_floor(values, n))


@pytest.mark.parametrize("dim,group", FORMS)
def test_cache_values_that_cancel(dim, group):
    """Values that are zero as -7 s + 7 s, s 19/16 (so that a weight times s is no
    fp32 number): what is left of them is the rounding of the weights.  Two fp16
    numbers hold a weight within 2^-23 of it, formed from an fp32 product; the sums
    of the minima take at most 12 roundings of 2^-24 (8 terms a lane, 4 lanes, a
    step), those of the codes 8 (two products of 16 keys, the join).  Weights lie
    within a factor of 2 of each other, so no product is cut beside another."""
    svq = require_gpu()
    heads, n, q_len = 64, 16, 16
    for seed in range(3):
        q, k = _rows(q_len, heads * dim, 100 + seed, 0.02), _rows(n, dim, 200 + seed)
        v = torch.zeros(n, dim)
        v.view(n, -1, group)[:, :, 0], v.view(n, -1, group)[:, :, 1] = -7 * 1.1875, 8 * 1.1875
        v = v.to(torch.bfloat16).cuda()
        assert torch.equal(stored(v, group), v.double().cpu())
        cache, _, table = _one_sequence(svq, k, v, 1, dim, group)
        y = svq.attn_cache(cache, q, table, _ints([n]), q_len=q_len).float().view(q_len, heads, -1, group)[:, :, :, 2:]
        off = y.abs().amax(dim=(2, 3))
        lim = 7 * 1.1875 * (2.0 ** -23 + 21 * 2.0 ** -24)
        assert bool((off <= lim).all()), f"{int((off > lim).sum())} rows, {off.max().item()} over {lim}"


@pytest.mark.parametrize("dim,group", FORMS)
def test_cache_values_that_cancel_under_different_weights(dim, group):
    """As above with weights from 1 to nearly nothing.  Beside the roundings above,
    each of the n products of a code and a weight may be off by 2^-22 of the
    greatest code, 15, times s and the greatest weight, which is at most the sum
    of the weights."""
    svq = require_gpu()
    heads, n, q_len = 64, 16, 16
    for seed in range(3):
        q, k = _rows(q_len, heads * dim, 300 + seed, 4.0), _rows(n, dim, 400 + seed)
        v = torch.zeros(n, dim)
        v.view(n, -1, group)[:, :, 0], v.view(n, -1, group)[:, :, 1] = -7 * 1.1875, 8 * 1.1875
        v = v.to(torch.bfloat16).cuda()
        cache, _, table = _one_sequence(svq, k, v, 1, dim, group)
        y = svq.attn_cache(cache, q, table, _ints([n]), q_len=q_len).float().view(q_len, heads, -1, group)[:, :, :, 2:]
        off = y.abs().amax(dim=(2, 3))
        lim = 7 * 1.1875 * (2.0 ** -23 + 21 * 2.0 ** -24) + n * 15 * 1.1875 * 2.0 ** -22
        assert bool((off <= lim).all()), f"{int((off > lim).sum())} rows, {off.max().item()} over {lim}"


@pytest.mark.parametrize("dim,group", [f for f in FORMS if f[0] > f[1]])
@pytest.mark.parametrize("apart", [2.0 ** 12, 2.0 ** 24, 2.0 ** 32, 2.0 ** 45])
@pytest.mark.parametrize("keys", ["none", "opposite"])
def test_cache_queries_of_different_sizes(keys, apart, dim, group):
    """Queries whose first group of channels is far greater than the others,
    over keys that are zero there, or as much smaller."""
    svq = require_gpu()
    heads, n = 4, 200
    q, k, v = _rows(1, heads * dim, 19), _rows(n, dim, 20), _rows(n, dim, 21)
    q, k = q.float(), k.float()
    q.view(heads, dim)[:, :group] *= apart
    k[:, :group] *= 0.0 if keys == "none" else 1.0 / apart
    q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
    cache, _, table = _one_sequence(svq, k, v, 1, dim, group)
    ks, vs = stored(k, group), stored(v, group)
    y = svq.attn_cache(cache, q, table, _ints([n]), scale=0.25)
    check(y, *attend(q, ks, vs, heads, 1, 0.25, visible(1, n)), n, P_F16, floor=cache_floor(vs, n))


# ---- rows beside others -----------------------------------------------------

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("n", [150, 1300])
def test_prompt_rows_keep_their_bits_beside_hidden_keys(n, window, dim):
    """Keys and values that a row does not see change no bit of it."""
    svq = require_gpu()
    heads, kv = 2, 1
    q, k, v = _rows(n, heads * dim, 22), _rows(n, kv * dim, 23), _rows(n, kv * dim, 24)
    before = svq.attn_prompt(q, k, v, _ints([0, n]), dim, window=window)
    for at in (0, 20, 77, n - 3):
        for factor in (8.0, -2.0 ** 30, float("nan")):
            k2, v2 = k.clone(), v.clone()
            k2[at] *= factor
            v2[at] *= factor
            after = svq.attn_prompt(q, k2, v2, _ints([0, n]), dim, window=window)
            hidden = ~visible(n, n, True, window)[:, at].cuda()
            assert torch.equal(before[hidden], after[hidden]), f"key {at} times {factor}"


@pytest.mark.parametrize("dim,group", FORMS)
@pytest.mark.parametrize("window", [0, 40])
def test_cache_rows_keep_their_bits_beside_hidden_keys(window, dim, group):
    """Later tokens of a call, and those before a window, change no bit of the
    rows that do not see them."""
    svq = require_gpu()
    heads, kv, n, q_len = 2, 1, 90, 7
    q, k, v = _rows(q_len, heads * dim, 25), _rows(n, kv * dim, 26), _rows(n, kv * dim, 27)
    cache, pages, table = _one_sequence(svq, k, v, kv, dim, group)
    before = svq.attn_cache(cache, q, table, _ints([n]), q_len=q_len, window=window)
    for at in (n - 1, n - 3, n - q_len - 39, n - q_len - 36):
        for factor in (8.0, 2.0 ** 20, -2.0 ** 34, float("nan")):
            _write(svq, cache, k[at:at + 1] * factor, v[at:at + 1] * factor, pages, at)
            after = svq.attn_cache(cache, q, table, _ints([n]), q_len=q_len, window=window)
            _write(svq, cache, k[at:at + 1], v[at:at + 1], pages, at)
            hidden = ~visible(q_len, n, True, window)[:, at].cuda()
            assert torch.equal(before[hidden], after[hidden]), f"token {at} times {factor}"


def test_cache_rows_of_tokens_that_later_ones_dwarf():
    """Later tokens of a call whose values are 2^34 times greater: the rows
    before keep the precision of what they see."""
    svq = require_gpu()
    heads, kv, dim, group, n, q_len = 4, 1, 128, 64, 70, 4
    q, k, v = _rows(q_len, heads * dim, 28), _rows(n, kv * dim, 29), _rows(n, kv * dim, 30)
    v[n - 2:] = (v[n - 2:].float() * 2.0 ** 34).to(torch.bfloat16)
    cache, _, table = _one_sequence(svq, k, v, kv, dim, group)
    y = svq.attn_cache(cache, q, table, _ints([n]), q_len=q_len)
    ks, vs = stored(k, group), stored(v, group)
    ref = attend(q, ks, vs, heads, kv, dim ** -0.5, visible(q_len, n))
    check(y[:2], *(r[:2] for r in ref), n, P_F16, floor=cache_floor(vs[:n - 2], n))
    check(y[2:], *(r[2:] for r in ref), n, P_F16, floor=cache_floor(vs, n))


# ---- long ranges, scores of minus infinity ----------------------------------

def test_cache_ranges_of_more_chunks_than_lanes_hold_pages():
    """1024 queries of 8 heads are as many blocks as run at once, so one range
    has all 5000 tokens, 40 chunks a wave."""
    svq = require_gpu()
    heads, kv, dim, group, n, q_len = 8, 8, 64, 32, 5000, 1024
    q, k, v = _rows(q_len, heads * dim, 31), _rows(n, kv * dim, 32), _rows(n, kv * dim, 33)
    cache, _, table = _one_sequence(svq, k, v, kv, dim, group)
    call = svq.AttnCacheCall(cache, q, torch.empty_like(q), table, _ints([n]), q_len=q_len)
    assert call.ws_size.value <= 256
    y = svq.attn_cache(cache, q, table, _ints([n]), q_len=q_len)
    rows = [0, 1, 2, 15, 16, 500, 905, 1022, 1023]
    ks, vs = stored(k, group), stored(v, group)
    check(y[rows], *attend(q[rows], ks, vs, heads, kv, dim ** -0.5, visible(q_len, n)[rows]), n, P_F16)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,first", [(40, 1), (40, 7), (1300, 1), (1300, 900)])
def test_prompt_rows_that_see_scores_of_minus_infinity(n, first, dim):
    """The first keys' scores are minus infinity for every query: rows that see
    no others are zeros, as if they saw nothing, and later ones do not feel them."""
    svq = require_gpu()
    q, k, v = _rows(n, dim, 34), _rows(n, dim, 35), _rows(n, dim, 36)
    q[:, 5] = 1.0
    k2 = k.clone()
    k2[:first, 5] = -float("inf")
    y = svq.attn_prompt(q, k2, v, _ints([0, n]), dim)
    assert torch.all(y[:first] == 0)
    seen = visible(n, n)
    seen[:, :first] = False
    check(y[first:], *(r[first:] for r in attend(q, k, v, 1, 1, dim ** -0.5, seen)), n, P_BF16)
