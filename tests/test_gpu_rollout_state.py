"""Steps of a rollout that are captured and replayed: the rollout sees on the device
that they ran, and weighs the queries that they asked."""
import pytest
import torch

from test_gpu_drafts import BF, _randn

pytestmark = pytest.mark.gpu

TREES = [[-1, 0, 0, 1], [-1, -1, 1]]


@pytest.fixture(scope="module")
def path():
    from merged_attention_autoregressive_gb300 import path
    return path


def _captured(r, *args):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.step(*args)
    return graph.replay


@pytest.mark.parametrize("own_stream", [False, True])
def test_replayed_steps_count(path, own_stream):
    gen = torch.Generator().manual_seed(5)
    plain, drafts = ([_randn(gen, 2, 20, 64) for _ in range(3)] for _ in range(2))
    eager, r = (path.BranchRollout(2, 2, 64, 20, 64, page=16, block=1, budget=16, recent=8, decay=0.9)
                for _ in range(2))
    stream = torch.cuda.Stream() if own_stream else torch.cuda.current_stream()
    stream.wait_stream(torch.cuda.current_stream())
    kw = dict(stream=stream) if own_stream else {}
    replays = []
    for turn in range(3):
        eager.extend([10, 7])
        eager.step(*plain)
        r.extend([10, 7], **kw)
        with pytest.raises(ValueError, match="weighed"):
            r.evict(**kw)
        if turn == 0:
            torch.cuda.synchronize()
            replays.append(_captured(r, *plain))
            torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            replays[0]()
        eager.evict()
        r.evict(**kw)
        eager.extend([4, 3], parents=TREES)
        eager.step(*drafts)
        r.extend([4, 3], parents=TREES, **kw)
        with pytest.raises(ValueError, match="attended"):
            r.accept([3, 2], **kw)
        if turn == 0:
            torch.cuda.synchronize()
            replays.append(_captured(r, *drafts))
            torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            replays[1]()
        assert eager.accept([3, 2]) == r.accept([3, 2], **kw)
        torch.cuda.synchronize()
        assert r.lengths == eager.lengths == r.pages.len.tolist() and int(r.status) == int(eager.status) == 0
        assert r.held == eager.held
        for b in range(2):
            ids = torch.tensor(r.held[b], device="cuda")
            for x, y in ((r.pages.K, eager.pages.K), (r.pages.V, eager.pages.V), (r.mass.mass, eager.mass.mass),
                         (r.mass.born, eager.mass.born)):
                x, y = (t[ids].transpose(1, 2).reshape(len(r.held[b]) * 16, -1)[:r.lengths[b]] for t in (x, y))
                assert torch.equal(x, y)
