"""Ends of the ranges of the calls for drafts and bounded pages: infinities and
NaN, errors found on the device, streams and graphs, far offsets, empty branches.
Bounds as in test_gpu_drafts.py."""
import math

import numpy as np
import pytest
import torch

import test_gpu_drafts as T
from oracle import draft_oracle as O
from test_gpu_drafts import BF, F32, _f64, _ints, _layout, _pages, _randn, _status, _tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import merged_attention_autoregressive_gb300 as m
    return m


class Call:
    """A call of each kind on inputs of its own, and what it leaves."""

    def __init__(self, m, kind, dtype=BF, D=128, seed=0, new=(40, 1, 3), past=(200, 100, 64), g=2, block=1):
        rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.m, self.kind, self.D, self.block = m, kind, D, block
        self.cu, self.length, self.table, self.pool = _layout(rng, list(new), list(past), 32)
        H, N = 2, int(self.cu[-1])
        self.K, self.V, self.pages = _pages(m, gen, self.pool, H, 32, D, dtype, self.table, self.length)
        self.q = _randn(gen, H * g, N, D, dtype=dtype, scale=1.5)
        self.out = torch.zeros_like(self.q)
        self.lse = _randn(gen, H * g, N, dtype=F32) + 7 if kind == "mass" else torch.zeros(H * g, N, device="cuda")
        self.offsets = _ints(self.cu)
        self.parent = _ints(np.concatenate([_tree(rng, "random", n) for n in new]))
        kept = [list(range(0, n, 2)) for n in new]
        self.rows = _ints([int(self.cu[b]) + i for b, k in enumerate(kept) for i in k])
        self.cu_keep = _ints(np.concatenate(([0], np.cumsum([len(k) for k in kept]))))
        self.mass = m.PageMass.view(torch.rand(self.pool, H, 32, generator=gen).cuda(),
                                    torch.randint(0, 500, (self.pool, H, 32), generator=gen, dtype=torch.int32).cuda(),
                                    _ints(self.length + 300))
        self.ws = torch.empty(max(m.mass_workspace_size(H * g, H, N, D), m.branch_workspace_size(H * g, H, N, D)),
                              dtype=torch.uint8, device="cuda")
        self.status = _status()

    def run(self, **kw):
        m, kw = self.m, dict(kw, status=self.status)
        if self.kind == "tree":
            m.fastar_tree_attention(self.q, self.offsets, self.parent, None, self.pages, self.D ** -0.5, self.out,
                                    lse=self.lse, ws=self.ws, **kw)
        elif self.kind == "keep":
            m.fastar_page_keep(self.pages, self.offsets, self.rows, self.cu_keep, **kw)
        elif self.kind == "mass":
            m.fastar_page_mass(self.pages, self.q, self.lse, self.offsets, self.D ** -0.5, self.mass, block=self.block,
                               ws=self.ws, **kw)
        else:
            m.fastar_page_evict(self.pages, self.mass, 90, first=3, recent=20, **kw)

    def left(self):
        return [self.K, self.V, self.out, self.mass.mass, self.mass.born] + ([self.lse] if self.kind == "tree" else [])


KINDS = ["tree", "keep", "mass", "evict"]
TYPES = [(BF, 128), (F32, 64)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,D", TYPES)
def test_streams_and_graphs(m, kind, dtype, D):
    plain, other, graphed = (Call(m, kind, dtype, D) for _ in range(3))
    plain.run()
    torch.cuda.synchronize()
    assert any(not torch.equal(a, b) for a, b in zip(plain.left(), other.left()))  # it does something
    side = torch.cuda.Stream()
    other.run(stream=side)
    side.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    before = [x.clone() for x in graphed.left()]
    with torch.cuda.stream(side):
        graphed.run()
        for x, y in zip(graphed.left(), before):
            x.copy_(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.run()
    for _ in range(2):
        for x, y in zip(graphed.left(), before):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(plain.left(), other.left(), graphed.left()):
            assert torch.equal(a, b) and torch.equal(a, c)
    assert int(plain.status) == int(other.status) == int(graphed.status) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,D", TYPES)
def test_an_earlier_error_stops_the_call(m, kind, dtype, D):
    c = Call(m, kind, dtype, D)
    before = [x.clone() for x in c.left()]
    c.status.fill_(17)
    c.run()
    assert int(c.status) == 17
    for a, b in zip(c.left(), before):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,D", TYPES)
@pytest.mark.parametrize("spoil", ["page", "page below", "length", "length below", "cu", "cu behind", "rows"])
def test_device_errors(m, kind, dtype, D, spoil):
    c = Call(m, kind, dtype, D)
    if spoil in ("cu", "cu behind") and kind == "evict" or spoil == "rows" and kind != "keep":
        pytest.skip("not an argument of this call")
    if spoil.startswith("page"):
        c.pages.table[0] = c.pool if spoil == "page" else -1
    elif spoil.startswith("length"):
        c.pages.len[0] = 10 ** 6 if spoil == "length" else -5
    elif spoil == "cu":
        c.offsets[1] = 60
    elif spoil == "cu behind":
        c.offsets[3] = 2 ** 30
        c.cu_keep[3] = 2 ** 30
    else:
        c.rows[3] = c.rows[2]
    c.run()
    assert int(c.status) == 18
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,D", TYPES + [(BF, 64)])
@pytest.mark.parametrize("new", [(1, 1, 1), (40, 1, 3), (300, 40, 130)])
def test_masses_of_other_branches_keep_clear_of_spoiled_ones(m, dtype, D, new):
    """A query that is no number spoils its own branch, a key its own mass."""
    calls = [Call(m, "mass", dtype, D, new=new, past=(200, 100, 64)) for _ in range(2)]
    clean, c = calls
    lo, hi = int(c.cu[1]), int(c.cu[2])
    c.q[:, lo:hi] = math.nan
    c.q[1, lo] = math.inf
    page, slot = int(c.table[0, 1]), 5  # position 37 of branch 0
    c.K[page, 0, slot, 3] = math.inf
    c.K[page, 1, slot] = math.nan
    for b in range(3):  # what lies behind the lengths
        p = int(c.length[b])
        if p % 32:
            c.K[int(c.table[b, p // 32]), :, p % 32:] = math.nan
    for x in calls:
        x.run()
        assert int(x.status) == 0
    a, b = clean.mass.mass.clone(), c.mass.mass.clone()
    for x in (a, b):
        x[page, :, slot] = 0
        x[c.table[1]] = 0
    assert torch.equal(a, b)
    assert not torch.isfinite(c.mass.mass[page, 1, slot])
    own = c.mass.mass[int(c.table[1, 0]), 0, :32]
    assert own.isnan().all()


@pytest.mark.parametrize("dtype,D", TYPES)
def test_rows_that_saw_nothing_add_nothing(m, dtype, D):
    c = Call(m, "mass", dtype, D, new=(130, 2, 9))
    c.lse[:] = -math.inf
    c.q[:, 5] = math.nan
    before = c.mass.mass.clone()
    c.run()
    fresh = torch.zeros_like(before, dtype=torch.bool)
    for b in range(3):
        for p in range(int(c.length[b]) - int(c.cu[b + 1] - c.cu[b]), int(c.length[b])):
            fresh[int(c.table[b, p // 32]), :, p % 32] = True
    assert torch.equal(c.mass.mass, torch.where(fresh, 0.0, before)) and int(c.status) == 0


@pytest.mark.parametrize("dtype,D", TYPES)
def test_tree_isolates_branches(m, dtype, D):
    clean, c = (Call(m, "tree", dtype, D, new=(20, 7, 33)) for _ in range(2))
    for b in (1,):
        c.K[c.table[b]] = math.nan
        c.V[c.table[b]] = math.inf
    for x in (clean, c):
        x.run()
    lo, hi = int(c.cu[1]), int(c.cu[2])
    for a, b in ((clean.out, c.out), (clean.lse, c.lse)):
        a, b = a.clone(), b.clone()
        a[:, lo:hi] = b[:, lo:hi] = 0
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,D", TYPES)
@pytest.mark.parametrize("kind", KINDS)
def test_empty_branches(m, kind, dtype, D):
    c = Call(m, kind, dtype, D, new=(0, 0, 0), past=(30, 0, 5)) if kind == "evict" else \
        Call(m, kind, dtype, D, new=(0, 1, 0), past=(30, 0, 0))
    before = [x.clone() for x in c.left()]
    c.run()
    assert int(c.status) == 0
    if kind in ("keep", "evict"):
        for a, b in zip(c.left(), before):
            assert torch.equal(a, b)
    if kind == "tree":  # the one token sees itself
        assert torch.equal(c.out[0, 0], c.V[int(c.table[1, 0]), 0, 0])


def test_far_pages(m):
    """Rows behind 2^32 bytes of a pool, and behind 2^31 elements."""
    H, page, D, n_pages = 2, 256, 128, 40000  # 5.2 GB of keys
    K = torch.zeros(n_pages, H, page, D, dtype=BF, device="cuda")
    V = torch.zeros_like(K)
    gen = torch.Generator().manual_seed(4)
    ids = torch.tensor([39999, 3, 38000, 17], device="cuda")
    K[ids] = _randn(gen, 4, H, page, D)
    V[ids] = _randn(gen, 4, H, page, D)
    near = m.PagedKV.view(K[ids].clone(), V[ids].clone(), _ints([[0, 1, 2, 3]]), _ints([900]))
    far = m.PagedKV.view(K, V, ids.to(torch.int32)[None], _ints([900]))
    masses = [m.PageMass(p) for p in (near, far)]
    q, cu = _randn(gen, 2, 40, D), _ints([0, 40])
    parent, rows = _ints(np.maximum(np.arange(40) - 3, -1)), _ints(np.arange(1, 40, 2))
    got = []
    for p, x in zip((near, far), masses):
        x.total.fill_(900)
        st, out, lse = _status(), torch.empty_like(q), torch.empty(2, 40, device="cuda")
        m.fastar_tree_attention(q, cu, parent, None, p, 0.1, out, lse=lse, status=st)
        m.fastar_page_keep(p, cu, rows, _ints([0, 20]), status=st)
        p.len.fill_(880)
        for tokens in (20, 1):
            m.fastar_page_mass(p, q, lse, _ints([0, tokens]), 0.1, x, block=1, rows=rows, status=st)
        m.fastar_page_evict(p, x, 500, first=4, recent=100, status=st)
        assert int(st) == 0
        pick = (lambda t: t) if p is near else (lambda t: t[ids])
        live = [pick(t).transpose(1, 2).reshape(1024, H, -1)[:500].clone() for t in (p.K, p.V, x.mass, x.born)]
        got.append([out, lse] + live)
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_masses_of_prompts_that_are_cut(m):
    """One branch of many rows on few heads: its items are cut and joined."""
    rng, gen = np.random.default_rng(8), torch.Generator().manual_seed(8)
    for dtype, D, n, past, block in ((BF, 128, 1500, 300, 1), (BF, 64, 900, 0, 0), (F32, 64, 700, 100, 1)):
        cu, length, table, pool = _layout(rng, [n], [past], 64)
        K, V, pages = _pages(m, gen, pool, 1, 64, D, dtype, table, length)
        q = _randn(gen, 1, n, D, dtype=dtype, scale=1.5)
        lse = _randn(gen, 1, n, dtype=F32) + 8
        held = m.PageMass.view(torch.rand(pool, 1, 64, generator=gen).cuda())
        ref = _f64(held.mass)
        tol = O.page_mass(_f64(K), _f64(q), _f64(lse), None, cu, table, length, D ** -0.5, block, 1.0, ref)
        st = _status()
        m.fastar_page_mass(pages, q, lse, _ints(cu), D ** -0.5, held, block=block, status=st)
        assert int(st) == 0 and (np.abs(_f64(held.mass) - ref) <= 1.05 * tol).all()


def test_two_calls_at_once(m):
    """Calls on two streams, each with its own inputs and workspace."""
    for kind in KINDS:
        alone = [Call(m, kind, seed=s, new=(200, 40, 5)) for s in (1, 2)]
        both = [Call(m, kind, seed=s, new=(200, 40, 5)) for s in (1, 2)]
        for c in alone:
            c.run()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in both]
        for c, s in zip(both, streams):
            c.run(stream=s)
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            for x, y in zip(a.left(), b.left()):
                assert torch.equal(x, y)


def test_graph_of_a_budgeted_step(m):
    """A step of a rollout under a budget, captured between two extends."""
    from merged_attention_autoregressive_gb300.path import BranchRollout
    gen = torch.Generator().manual_seed(6)
    rolls = [BranchRollout(2, 2, 64, 20, 64, page=16, block=1, budget=32, recent=8) for _ in range(2)]
    q, k, v = (_randn(gen, 2, 20, 64) for _ in range(3))
    for r in rolls:
        r.extend([10, 7])
    rolls[0].step(q, k, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rolls[1].step(q, k, v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rolls[1].step(q, k, v)
    rolls[1].mass.mass.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(rolls[0].mass.mass, rolls[1].mass.mass) and torch.equal(rolls[0].out, rolls[1].out)
    assert torch.equal(rolls[0].mass.born, rolls[1].mass.born)


def test_a_rollout_may_keep_no_draft(m):
    from merged_attention_autoregressive_gb300.path import BranchRollout
    gen = torch.Generator().manual_seed(9)
    r = BranchRollout(2, 2, 64, 20, 64, page=16, block=1, budget=32, recent=8)
    q, k, v = (_randn(gen, 2, 20, 64) for _ in range(3))
    r.extend([10, 7])
    r.step(q, k, v)
    before = r.mass.mass.clone()
    r.extend([4, 3], parents=[[-1, 0, 0, 1], [-1, -1, 1]])
    out = r.step(q, k, v)[0].clone()
    assert r.accept([-1, -1]) == [[], []] and r.lengths == [10, 7] == r.pages.len.tolist()
    assert torch.equal(r.mass.mass, before)
    r.extend([4, 3], parents=[[-1, 0, 0, 1], [-1, -1, 1]])  # again, as if nothing had been
    assert torch.equal(r.step(q, k, v)[0][:, :7], out[:, :7])
    assert r.accept([3, 2]) == [[0, 1, 3], [5, 6]] and int(r.status) == 0
    r.evict()
    assert r.lengths == [13, 9]


# tables longer than the branches, so that each way of sharing a head's rows is taken:
# heads, room of a table, lengths, budget
LONG = [
    (2, 3008, [3000, 20], 1500),
    (80, 8192, [4500, 10], 1999),
    (350, 8192, [300, 4], 97),
    (1, 16384, [9000], 4096),
    (38, 32768, [9000, 5], 8999),
    (38, 65536, [3000, 5], 1),
    (80, 16384, [2500, 31], 1250),
    (80, 65536, [2500, 31], 640),
]


@pytest.mark.parametrize("H,room,lengths,budget", LONG)
@pytest.mark.parametrize("kind", ["random", "ties"])
def test_eviction_of_long_tables(m, H, room, lengths, budget, kind):
    rng, gen, page, D = np.random.default_rng(H + budget), torch.Generator().manual_seed(H), 64, 64
    _, length, table, pool = _layout(rng, lengths, [0] * len(lengths), page)
    table = np.concatenate((table, np.full((len(lengths), room // page - table.shape[1]), -1, np.int32)), 1)
    K, V, pages = _pages(m, gen, pool, H, page, D, BF, table, length)
    x = rng.random((pool, H, page)).astype(np.float32)
    if kind == "ties":
        x = np.floor(x * 3).astype(np.float32)
    born = rng.integers(0, max(lengths) + 50, (pool, H, page)).astype(np.int32)
    total = length + 50
    mass, stamp = torch.from_numpy(x).cuda(), torch.from_numpy(born).cuda()
    want = [K.float().cpu().numpy(), V.float().cpu().numpy(), x.copy(), born.copy()]
    O.page_evict(want, x, born, total, table, length, budget, 0, min(40, budget // 2))
    held, st = m.PageMass.view(mass, stamp, _ints(total)), _status()
    # an earlier error, and a length that the table has no room for: nothing is written
    for spoil in ("status", "long", "negative"):
        st.fill_(5 if spoil == "status" else 0)
        if spoil != "status":
            pages.len[0] = room + 1 if spoil == "long" else -1
        before = [y.clone() for y in (K, V, mass, stamp)] if spoil == "status" else before
        m.fastar_page_evict(pages, held, budget, first=0, recent=min(40, budget // 2), status=st)
        assert int(st) == (5 if spoil == "status" else 18)
        pages.len.copy_(_ints(length))
        if spoil == "status" or len(lengths) == 1 or max(lengths[1:]) <= budget:
            assert all(torch.equal(a, b) for a, b in zip(before, (K, V, mass, stamp)))
    for y, y0 in zip((K, V, mass, stamp), before):
        y.copy_(y0)
    st.zero_()
    m.fastar_page_evict(pages, held, budget, first=0, recent=min(40, budget // 2), status=st)
    assert int(st) == 0
    kept = np.zeros((pool, page), bool)
    for b, n in enumerate(lengths):
        for p in range(min(n, budget)):
            kept[table[b, p // page], p % page] = True
    for y, w, y0 in zip((K, V, mass, stamp), want, before):
        y, y0 = (t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy() for t in (y, y0))
        assert np.array_equal(y.swapaxes(1, 2)[kept], w.swapaxes(1, 2)[kept])
        assert np.array_equal(y.swapaxes(1, 2)[~kept], y0.swapaxes(1, 2)[~kept])


FEW32 = [
    # D, H, g, page, new, past, block, rows, decay, born, pad
    (128, 2, 1, 64, [1, 1, 1, 1], [300, 0, 63, 1000], 0, False, 1.0, True, 0),
    (128, 3, 5, 16, [1, 0, 1], [500, 7, 255], 1, False, 0.9, True, 4),
    (64, 2, 8, 256, [2, 1, 1], [2000, 255, 0], 0, True, 0.0, False, 1),
    (128, 8, 1, 64, [1] * 40, list(range(300, 700, 10)), 0, False, 1.0, True, 0),
    (64, 12, 1, 16, [1] * 40, list(range(300, 700, 10)), 1, False, 1.0, True, 5),
    (128, 1, 1, 128, [15], [200], 7, False, 1.0, True, 0),
    # many rows where few are to be expected
    (64, 1, 1, 32, [100] + [0] * 39, [50] + [0] * 39, 1, False, 1.0, True, 0),
    (128, 2, 2, 32, [0, 43] + [0] * 38, [0, 129] + [0] * 38, 0, True, 0.5, True, 7),
    # branches of a few rows beside some of many
    (64, 2, 1, 16, [16, 17, 1, 0, 33, 3], [100, 64, 5, 9, 300, 127], 1, False, 0.7, True, 3),
    (128, 2, 4, 32, [3, 4, 1, 1, 6, 2], [77, 500, 64, 300, 129, 1], 3, True, 1.0, True, 3),
]


@pytest.mark.parametrize("D,H,g,page,new,past,block,taken,decay,stamps,pad", FEW32)
def test_masses_of_a_few_rows_in_32_bits(m, D, H, g, page, new, past, block, taken, decay, stamps, pad):
    T.test_page_mass(m, F32, D, H, g, page, new, past, block, taken, decay, stamps, pad)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_few_rows_keep_clear_of_spoiled_ones(m, dtype):
    """As for longer drafts: a query spoils its own branch, a key its own mass."""
    calls = [Call(m, "mass", dtype, 128, new=(2, 1, 3), past=(200, 100, 64)) for _ in range(2)]
    clean, c = calls
    c.q[:, int(c.cu[1])] = math.nan
    page = int(c.table[0, 1])
    c.K[page, 0, 5, 3] = math.inf
    c.K[page, 1, 5] = math.nan
    for b in range(3):  # what lies behind the lengths
        p = int(c.length[b])
        c.K[int(c.table[b, p // 32]), :, p % 32:] = math.nan
    for x in calls:
        x.run()
        assert int(x.status) == 0
    a, b = clean.mass.mass.clone(), c.mass.mass.clone()
    for x in (a, b):
        x[page, :, 5] = 0
        x[c.table[1]] = 0
    assert torch.equal(a, b)
    assert not torch.isfinite(c.mass.mass[page, 1, 5])
    assert c.mass.mass[int(c.table[1, 0]), 0, :32].isnan().all()


def test_shared_evictions_captured_and_on_a_stream(m):
    """Clusters that share a head's rows: one call behind the other on a stream, and
    captured and replayed, leave what single calls leave."""
    rng, gen, page, D, H = np.random.default_rng(5), torch.Generator().manual_seed(5), 64, 64, 3
    lengths = [3000, 2900, 40]
    _, length, table, pool = _layout(rng, lengths, [0] * 3, page)
    K, V, pages = _pages(m, gen, pool, H, page, D, BF, table, length)
    mass = torch.rand(pool, H, page, generator=gen).cuda()
    born = torch.randint(0, 3000, (pool, H, page), generator=gen, dtype=torch.int32).cuda()
    held, st = m.PageMass.view(mass, born, _ints(length)), _status()
    state = [K, V, mass, born, pages.len]
    first = [x.clone() for x in state]

    def steps():
        m.fastar_page_evict(pages, held, 2048, first=4, recent=200, status=st)
        pages.len.clamp_(max=2048)
        m.fastar_page_evict(pages, held, 1000, first=4, recent=200, status=st)

    steps()
    torch.cuda.synchronize()
    want = [x.clone() for x in state]

    def restore():
        for x, y in zip(state, first):
            x.copy_(y)
        torch.cuda.synchronize()

    restore()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        steps()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(state, want)) and int(st) == 0
    restore()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for _ in range(2):
        restore()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(state, want)) and int(st) == 0
