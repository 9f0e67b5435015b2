"""What the header promises of the calls for bounded pages, where calls meet their
limits."""
import math
import threading

import numpy as np
import pytest
import torch

from oracle import draft_oracle as O
from test_gpu_drafts import BF, F32, _f64, _ints, _layout, _pages, _randn, _status

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


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("H,room", [(1, 64), (1, 16384), (3, 512)])
def test_page_ids_of_branches_under_the_budget(m, H, room, apart):
    """They are looked at where something is read or written: with masses apart."""
    page = 32
    pool = 8
    K = torch.randn(pool, H, page, 64, device="cuda")
    table = torch.zeros(2, room // page, dtype=torch.int32, device="cuda")
    table[0, :2] = _ints([3, pool])  # the second id is none
    table[1, :2] = _ints([1, 2])
    pages = m.PagedKV.view(K, K.clone(), table, _ints([40, 50]))
    held, out, st = m.PageMass(pages), m.PageMass(pages), _status()
    held.mass.uniform_()
    out.mass.fill_(7.0)
    before = [x.clone() for x in (pages.K, pages.V, held.mass)]
    m.fastar_page_evict(pages, held, 60, out=out if apart else None, status=st)
    assert int(st) == (18 if apart else 0)
    assert all(torch.equal(x, y) for x, y in zip((pages.K, pages.V, held.mass), before))
    if not apart:
        assert (out.mass == 7).all()


SCALES = [1e-44, 3e-39, 1e-37, 1e-31, 1e-29, 1.0, 1e29, 1e31]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype,D,n", [(BF, 128, 150), (BF, 64, 150), (BF, 128, 3), (F32, 64, 150)])
def test_masses_at_any_scale(m, scale, dtype, D, n):
    """Whatever the scale, lse / scale need not be a number of 32 bits: queries are
    such that scale q . k stays within +-4, and lse is near what attention gives."""
    rng, gen = np.random.default_rng(1), torch.Generator().manual_seed(1)
    cu, length, table, pool = _layout(rng, [n, 2], [100, 40], 32)
    K, V, pages = _pages(m, gen, pool, 2, 32, D, dtype, table, length)
    q = _randn(gen, 2, n + 2, D, dtype=F32)
    q = (q * min(1.0, 0.1 / scale)).to(dtype) if scale >= 1e-30 else q.to(dtype)
    lse = (5.0 + torch.rand(2, n + 2, generator=gen)).cuda()
    held = m.PageMass.view((3 * torch.rand(pool, 2, 32, generator=gen)).cuda())
    ref = _f64(held.mass)
    exact = float(np.float32(scale))
    tol = O.page_mass(_f64(K), _f64(q), _f64(lse), None, cu, table, length, exact, 1, 0.5, ref, None, None)
    st = _status()
    m.fastar_page_mass(pages, q, lse, _ints(cu), scale, held, block=1, decay=0.5, status=st)
    assert int(st) == 0
    assert (np.abs(_f64(held.mass) - ref) <= 1.05 * tol).all()
    assert math.isfinite(float(held.mass.sum())) and (ref.max() > 0.05)
