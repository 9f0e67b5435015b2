"""What the header promises of the calls for bounded pages, where calls meet their
limits."""
import threading

import pytest
import torch

from test_gpu_drafts import BF, F32, _ints, _status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import merged_attention_autoregressive_gb300 as m
    return m


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
def test_evictions_of_two_host_threads(m, dtype, D):
    """Tables of different room by one instantiation of the kernel: what one thread
    asks for shared memory takes nothing from the other."""
    calls = []
    for room in (1 << 19, 140000):
        page, length = 256, 50
        K = torch.zeros(1, 1, page, D, dtype=dtype, device="cuda")
        pages = m.PagedKV.view(K, torch.zeros_like(K), torch.zeros(1, -(-room // page), dtype=torch.int32, device="cuda"),
                               _ints([length]))
        calls.append((pages, m.PageMass(pages), room // 2, _status(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(calls))

    def work(pages, held, budget, status, stream):
        start.wait()
        try:
            for _ in range(3000):
                m.fastar_page_evict(pages, held, budget, status=status, stream=stream)
        except m.FastarError as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and all(int(c[3]) == 0 for c in calls)
