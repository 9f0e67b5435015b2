"""Host threads that make calls of different sizes at the same time: none takes the
shared memory that another one's launch asks for."""
import itertools
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def _together(works, times):
    import merged_attention_autoregressive_gb300 as m
    failed, start = [], threading.Barrier(len(works))

    def run(work):
        start.wait()
        try:
            for _ in range(times):
                work()
        except m.FastarError as e:
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return failed


def test_bucket_lists():
    import merged_attention_autoregressive_gb300 as m
    works, kept = [], []
    for B in (12, 9):
        codes = torch.randint(0, 1 << B, (1, 300), dtype=torch.int32, device="cuda")
        perm, offsets = torch.empty_like(codes), torch.empty(1, (1 << B) + 1, dtype=torch.int32, device="cuda")
        stream = torch.cuda.Stream()
        kept.append((codes, perm, stream))
        works.append(lambda a=(codes, B, perm, offsets), s=stream: m.fastar_bucket_csr(*a, stream=s))
    assert not _together(works, 3000)
    for codes, perm, _ in kept:
        assert torch.equal(perm[0].long(), torch.sort(codes[0], stable=True).indices)


def test_merges_of_frames_of_different_sizes():
    from merged_attention_autoregressive_gb300.path import ChunkPath
    works, paths = [], []
    for n_f in (3000, 1600):
        p = ChunkPath(1, 64, n_f, 1, 16, 1, 6, 8192, 0.9, torch.float32)
        k, v = (torch.randn(1, n_f, 64, device="cuda") for _ in range(2))
        p.planes.normal_()
        stream = torch.cuda.Stream()
        works.append(lambda p=p, k=k, v=v, s=stream, f=itertools.count(): p.merge(k, v, next(f), stream=s))
        paths.append((p, k, v, n_f))
    assert not _together(works, 2000)
    for p, _, _, n_f in paths:  # every later frame is merged into the first one
        assert int(p.status) == 0 and int(p.cache.size[0]) == n_f
