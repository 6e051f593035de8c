"""Uses of the feed-forward calls beside one call on one stream's operands:
workspaces across streams, outputs over or beside their inputs."""
import pytest

import synth
from tests.gpu_common import require_gpu, to_device_bf16, torch

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
