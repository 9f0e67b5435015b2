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


@pytest.mark.parametrize("dtype,D", [(BF, 128), (torch.float32, 64)])
def test_attending_again_leaves_the_masses(path, dtype, D):
    """Steps that do not weigh before the one that does leave what it alone leaves."""
    gen = torch.Generator().manual_seed(7)
    q, k, v = (_randn(gen, 2, 20, D, dtype=dtype) for _ in range(3))
    got = []
    for again in (0, 2):
        r = path.BranchRollout(2, 2, D, 20, 64, page=16, block=1, budget=16, recent=8, decay=0.9, dtype=dtype)
        for _ in range(2):
            r.extend([10, 7])
            for _ in range(again):
                r.step(q, k, v, weigh=False)
            out, lse = r.step(q, k, v)
        assert int(r.status) == 0
        got.append([x.clone() for x in (out, lse, r.mass.mass, r.mass.born, r.pages.K, r.pages.V)])
    assert all(torch.equal(x, y) for x, y in zip(*got)) and bool(got[0][2].any())


@pytest.mark.parametrize("forked", [False, True])
def test_steps_captured_on_a_stream_that_is_named(path, forked):
    """The step's stream is looked at, whether or not it is the current one."""
    gen = torch.Generator().manual_seed(6)
    q, k, v = (_randn(gen, 2, 20, 64) for _ in range(3))
    r = path.BranchRollout(2, 2, 64, 20, 64, page=16, block=1, budget=16, recent=8)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    r.extend([10, 7], stream=main)
    r.step(q, k, v, stream=main, weigh=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        if forked:
            side.wait_stream(main)
        r.step(q, k, v, stream=side if forked else main)
        if forked:
            main.wait_stream(side)
    torch.cuda.synchronize()
    assert not bool(r.mass.mass.any())
    with pytest.raises(ValueError, match="weighed"):
        r.evict(stream=main)
    with torch.cuda.stream(main):
        graph.replay()
    r.evict(stream=main)
    torch.cuda.synchronize()
    assert bool(r.mass.mass.any()) and int(r.status) == 0
    r.extend([10, 7], stream=main)
    r.step(q, k, v, stream=side.cuda_stream if forked else main)  # eager again; a raw handle
    torch.cuda.synchronize()
    r.evict(stream=main)
    assert r.lengths == [16, 14]
