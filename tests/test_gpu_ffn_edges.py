"""Uses of the feed-forward calls beside one call on one stream's operands:
workspaces across streams, their exact size, outputs over or beside their
inputs, offsets past 32 bits, functions inside a capture, calls at once,
long rows."""
import numpy as np
import pytest

import synth
from tests.gpu_common import require_gpu, to_device_bf16, torch
from tests.test_gpu_ffn import SLOPE, U32, _block, _block_weights, act64, check, half_step, no_split, product, product_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svq():
    return require_gpu()


def _pair(svq, m, n=96, k=1032):
    pair = [svq.pack(synth.random_matrix(n, k, bd, seed=(130, bd, k))) for bd in (7, 8)]
    x = to_device_bf16(synth.random_activations(m, k, seed=(130, 1, m)))
    return pair, x, torch.empty((m, n), dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("m", [3, 9, 40, 300])
def test_workspace_is_not_given_away_early(svq, m, given):
    """A prepared call dropped while its launches are queued on another
    stream: what is allocated next does not get its workspace."""
    pair, x, y = _pair(svq, m)
    want = svq.linear_glu(*pair, x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
    call = svq.GluCall(*pair, x, y, stream=s if given else None)
    if given:
        call()
    else:
        with torch.cuda.stream(s):
            call()
    nbytes = call.workspace.numel()
    del call
    others = [torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(y, want) and all(int(o.min()) == 255 for o in others)


@pytest.mark.parametrize("m", [3, 9, 40, 300])
def test_workspace_waits_for_its_last_user(svq, m):
    """Memory that the allocator hands to a prepared call while a fill of its
    last owner is queued: a call on another stream runs after the fill."""
    pair, x, y = _pair(svq, m)
    want = svq.linear_glu(*pair, x)
    nbytes = svq.GluCall(*pair, x, y).workspace.numel()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(2_000_000)
    block.fill_(255)
    del block
    call = svq.GluCall(*pair, x, y)
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert torch.equal(y, want)
    call()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_captured_on_a_fresh_object(svq):
    """A call whose first stream is a capture's: replayed, and called eagerly
    between the replays."""
    pair, x, y = _pair(svq, 9)
    call, graph = svq.GluCall(*pair, x, y), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        xi = to_device_bf16(synth.random_activations(9, 1032, seed=(131, i)))
        want = svq.linear_glu(*pair, xi)
        x.copy_(xi)
        y.fill_(0)
        (graph.replay if i % 2 else call)()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


@pytest.mark.parametrize("m", [1, 20, 40])
@pytest.mark.parametrize("split", [True, False])
def test_expert_layer_over_its_input(svq, m, split):
    """y is x itself, with and without x as the residual: as into a fresh y,
    in the per-slot form, the grouped one and the one of separate products."""
    e, f, k, topk = 4, 72, 136, 2
    sets = []
    for s, (n, kk) in enumerate(((f, k), (f, k), (k, f))):
        mats = [synth.random_matrix(n, kk, 7, seed=(132, s, i)) for i in range(e)]
        if not split:  # tables that admit no two fp16 halves
            mats[1].radius, mats[1].codebook = mats[1].radius.copy(), mats[1].codebook.copy()
            mats[1].radius[0], mats[1].radius[1], mats[1].codebook[0, :] = 0x3C01, 0x7B53, 0x0001
        sets.append([svq.pack(a) for a in mats])
    x = to_device_bf16(synth.random_activations(m, k, seed=(132, m)))
    g = torch.Generator().manual_seed(24)
    ids = torch.stack([torch.randperm(e, generator=g)[:topk] for _ in range(m)]).to(torch.int32).cuda()
    wt = torch.rand((m, topk), generator=g).cuda()
    for res in (False, True):
        want = svq.moe_ffn(*sets, x, ids, wt, residual=x if res else None)
        y = x.clone()
        svq.moe_ffn(*sets, y, ids, wt, residual=y if res else None, out=y)
        assert torch.equal(y, want)


@pytest.mark.parametrize("m", [1, 7, 40, 150])
def test_operands_as_columns_of_one_buffer(svq, m):
    """x, residual and y side by side in the rows of one buffer."""
    n, k = 96, 264
    pm = svq.pack(synth.random_matrix(n, k, 7, seed=(133, n, k)))
    wide = torch.randn((m, k + 2 * n), generator=torch.Generator().manual_seed(25)).bfloat16().cuda()
    before = wide.clone()
    x, r, y = wide[:, n:n + k], wide[:, n + k:], wide[:, :n]
    want = svq.linear_epilogue(pm, x.contiguous(), residual=r.contiguous(), act="relu")
    svq.linear_epilogue(pm, x, residual=r, act="relu", out=y)
    assert torch.equal(y, want) and torch.equal(wide[:, n:], before[:, n:])


def _calls(svq, m):
    """One call of each kind at m rows, as (make, outputs)."""
    e, f, k, topk = 4, 72, 1032, 2
    pg, pu, pd = [svq.pack(synth.random_matrix(n, kk, bd, seed=(134, n, bd))) for n, kk, bd in
                  ((f, k, 7), (f, k, 8), (k, f, 6))]
    sets = [[svq.pack(synth.random_matrix(n, kk, 7, seed=(135, s, i))) for i in range(e)]
            for s, (n, kk) in enumerate(((f, k), (f, k), (k, f)))]
    x = to_device_bf16(synth.random_activations(m, k, seed=(134, m)))
    g = torch.Generator().manual_seed(27)
    w = torch.randn((e, k), generator=g).cuda()
    ids = torch.stack([torch.randperm(e, generator=g)[:topk] for _ in range(m)]).to(torch.int32).cuda()
    wt = torch.rand((m, topk), generator=g).cuda()
    new = lambda n, t=torch.bfloat16: torch.zeros((m, n), dtype=t, device="cuda")
    h, y, ri, rw, z = new(f), new(f, torch.float32), new(topk, torch.int32), new(topk, torch.float32), new(k)
    return [(lambda ws: svq.GluCall(pg, pu, x, h, workspace=ws), (h,)),
            (lambda ws: svq.EpilogueCall(pg, x, y, act="gelu", workspace=ws), (y,)),
            (lambda ws: svq.MoeRouteCall(x, w, ri, rw, workspace=ws), (ri, rw)),
            (lambda ws: svq.MoeFfnCall(*sets, x, ids, wt, z, workspace=ws), (z,))]


@pytest.mark.parametrize("m", [1, 3, 9, 16, 20, 40, 150, 300, 5000])
def test_nothing_beyond_the_workspace(svq, m):
    """A workspace of exactly the queried size inside a larger buffer: what
    lies around it stays, whatever it held the result is the same, and a byte
    less is replaced."""
    for make, outs in _calls(svq, m):
        call = make(None)
        call()
        want, need = [o.clone() for o in outs], call.workspace.numel()
        buf = torch.empty(need + 8192, dtype=torch.uint8, device="cuda")
        ws = buf[4096:4096 + need]
        for fill in (0xFF, 0x00, 0x5A):
            buf.fill_(fill)
            for o in outs:
                o.zero_()
            call = make(ws)
            assert call.workspace is ws
            call()
            assert all(torch.equal(o, w) for o, w in zip(outs, want)), call.name
            assert bool((buf[:4096] == fill).all()) and bool((buf[4096 + need:] == fill).all()), call.name
        assert make(buf[4096:4095 + need]).workspace.numel() >= need


def _far_rows(m, n, dtype):
    """[m, n] of which the last row starts past element 2^31."""
    ld = -(-2 ** 31 // max(m - 1, 1)) + 24
    return torch.empty((m - 1) * ld + n, dtype=dtype, device="cuda").as_strided((m, n), (ld, 1))


@pytest.mark.parametrize("m", [2, 9, 40, 300])
def test_row_strides_past_32_bits(svq, m):
    """x, residual and y whose last rows lie beyond 2^31 elements, and ids
    that name them."""
    e, n, k, topk = 3, 40, 72, 2
    pg, pu = [svq.pack(synth.random_matrix(n, k, bd, seed=(136, n, bd))) for bd in (7, 8)]
    near = to_device_bf16(synth.random_activations(m, k, seed=(136, m)))
    x = _far_rows(m, k, torch.bfloat16)
    x.copy_(near)
    res = torch.randn((m, k), generator=torch.Generator().manual_seed(28)).bfloat16().cuda()
    y = _far_rows(m, n, torch.float32)
    r = _far_rows(m, n, torch.bfloat16)
    r.copy_(res[:, :n])
    svq.linear_epilogue(pg, x, residual=r, act="silu", out=y)
    assert torch.equal(y, svq.linear_epilogue(pg, near, residual=res[:, :n].contiguous(), act="silu", out_dtype=torch.float32))
    svq.linear_glu(pg, pu, x, out=y)
    assert torch.equal(y, svq.linear_glu(pg, pu, near, out_dtype=torch.float32))
    del y, r
    w = torch.randn((e, k), generator=torch.Generator().manual_seed(29)).cuda()
    ids, wt = svq.moe_route(x, w, topk)
    near_ids, near_wt = svq.moe_route(near, w, topk)
    assert torch.equal(ids, near_ids) and torch.equal(wt, near_wt)
    sets = [[svq.pack(synth.random_matrix(nn, kk, 7, seed=(137, s, i))) for i in range(e)]
            for s, (nn, kk) in enumerate(((n, k), (n, k), (k, n)))]
    want = svq.moe_ffn(*sets, near, ids, wt, residual=res)
    z, r = _far_rows(m, k, torch.bfloat16), _far_rows(m, k, torch.bfloat16)
    r.copy_(res)
    svq.moe_ffn(*sets, x, ids, wt, residual=r, out=z)
    assert torch.equal(z, want)


def test_staged_activations_past_32_bits(svq):
    """More than 2^31 staged activations, 300 rows over and over: every copy
    within the bound of tests/test_gpu_ffn.py (the plan, and with it the order
    of sums, follows the row count)."""
    m, n, k = (1 << 20) + 3, 24, 2104
    mats = [synth.random_matrix(n, k, bd, seed=(138, n, bd)) for bd in (7, 8)]
    pg, pu = [svq.pack(a) for a in mats]
    bits = synth.random_activations(300, k, seed=(138,))
    few = to_device_bf16(bits)
    x = few.repeat(m // 300 + 1, 1)[:m]
    assert m * k > 2 ** 31
    (g, gb), (u, ub) = [product(a, bits, True) for a in mats]
    a = act64(g, "silu")
    ea = SLOPE * gb + 16 * U32 * np.abs(a)
    for run, ref, bound in ((lambda: svq.linear_epilogue(pg, x, act="silu"), a, ea),
                            (lambda: svq.linear_glu(pg, pu, x), a * u,
                             ea * np.abs(u) + ub * np.abs(a) + ea * ub + U32 * np.abs(a * u))):
        y = run()
        ref, tol = [torch.from_numpy(v).cuda() for v in (ref, bound + half_step(y.dtype) * (np.abs(ref) + bound))]
        whole = m // 300 * 300
        assert bool(((y[:whole].view(-1, 300, n).double() - ref).abs() <= tol).all())
        assert bool(((y[whole:].double() - ref[:m - whole]).abs() <= tol[:m - whole]).all())


@pytest.mark.parametrize("m", [1, 12, 48, 300])
def test_functions_captured(svq, m):
    """The plain functions inside a capture: outputs and workspaces come from
    the graph's own memory, one call's workspace perhaps the next one's."""
    _, _, pms = _block_weights(svq)
    x = torch.zeros((m, 264), dtype=torch.bfloat16, device="cuda")
    _block(svq, pms, x, True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = _block(svq, pms, x, True)
    for i in range(4):
        xi = to_device_bf16(synth.random_activations(m, 264, seed=(141, i, m)))
        want = _block(svq, pms, xi, True)
        x.copy_(xi)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), f"replay {i}"


def test_two_calls_at_once(svq):
    """Calls on two streams, each object with a workspace of its own."""
    jobs = []
    for i, m in enumerate((9, 300)):
        pair, x, y = _pair(svq, m)
        s = torch.cuda.Stream()
        jobs.append((svq.GluCall(*pair, x, y, stream=s), y, svq.linear_glu(*pair, x)))
    torch.cuda.synchronize()
    for _ in range(20):
        for call, y, _ in jobs:
            call()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for _, y, want in jobs)


@pytest.mark.parametrize("k,m", [(53248, 1), (65536, 1), (53248, 3), (65536, 4), (65536, 7), (40000, 300)])
def test_long_rows(svq, k, m):
    """Rows too long for the forms that stage them whole, through the epilogue
    and the gated pair, the residual in place."""
    n = 24
    mats = [synth.random_matrix(n, k, bd, seed=(142, bd, k)) for bd in (7, 8)]
    bits = synth.random_activations(m, k, seed=(142, k, m))
    x, (pg, pu) = to_device_bf16(bits), [svq.pack(a) for a in mats]
    (g, gb), (u, ub) = [product(a, bits, m > 16) for a in mats]
    y = torch.randn((m, n), generator=torch.Generator().manual_seed(30)).cuda()
    r = y.double().cpu().numpy()
    svq.linear_epilogue(pg, x, act="relu", residual=y, out=y)
    a = np.maximum(g, 0)
    check(y, a + r, gb + U32 * (a + np.abs(r)), "epilogue")
    y = svq.linear_glu(pg, pu, x, act="relu", out_dtype=torch.float32)
    check(y, a * u, gb * np.abs(u) + ub * a + gb * ub + U32 * np.abs(a * u), "glu")


@pytest.mark.parametrize("m", [2, 13, 20, 200, 300])
@pytest.mark.parametrize("n", [40, 500])
def test_no_split_in_k_ranges(svq, n, m):
    """Tables without two fp16 halves and a K of nine units: beyond 16 rows
    the bf16 form's K ranges, joined by the launch that applies the epilogue."""
    k = 4608
    (mat, pm), (mat2, pm2) = no_split(svq, n, k, 11), no_split(svq, n, k, 12)
    bits = synth.random_activations(m, k, seed=(143, n, m))
    x = to_device_bf16(bits)
    (g, gb), (u, ub) = product_bf16(mat, bits, m), product_bf16(mat2, bits, m)
    bias = torch.randn(n, generator=torch.Generator().manual_seed(31)).cuda()
    y = torch.randn((m, n + 3), generator=torch.Generator().manual_seed(32)).cuda()[:, 1:1 + n]
    r, v = y.double().cpu().numpy(), g + bias.double().cpu().numpy()
    svq.linear_epilogue(pm, x, bias=bias, act="relu", residual=y, out=y)
    a = np.maximum(v, 0)
    check(y, a + r, gb + U32 * np.abs(v) + U32 * (a + np.abs(r)), "epilogue")
    a = np.maximum(g, 0)
    y = svq.linear_glu(pm, pm2, x, act="relu", out_dtype=torch.float32)
    check(y, a * u, gb * np.abs(u) + ub * a + gb * ub + U32 * np.abs(a * u), "glu")
