"""Uses of the feed-forward calls beside one call on one stream's operands:
workspaces across streams."""
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
