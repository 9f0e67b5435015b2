"""Drafts and bounded pages on the GPU against the 64-bit oracle.

Bounds.  u is half a step of the output's type (finfo.eps / 2).
Tree attention: as for the attention of branches: with X the row's largest scale
sum |q k|, A = sum p |v| and n keys, score error d <= (D + 4) 2^-23 X + 2^-20, so
  |err| <= u |out| + ((2^-8 for bf16) + 3 d + n 2^-22) A,  lse: d + n 2^-23 + 2^-22 |lse|.
Masses: a weight exp(x - lse) has the relative error of its exponent in
absolute terms: (D + 4) 2^-23 X of the product, 2^-23 (2 |lse| + 2 X) of the scaling
and the difference, 2^-21 of the exponential; a sum of r weights adds r 2^-23, the
old mass's product and sum 2^-22.  page_mass of the oracle returns their sum; the
test allows it times 1.05.
Moves are exact.
"""
import numpy as np
import pytest
import torch

from oracle import branch_oracle as B0
from oracle import draft_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    import merged_attention_autoregressive_gb300 as m
    return m


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _f64(t):
    return t.detach().double().cpu().numpy()


def _randn(g, *shape, dtype=BF, scale=1.0):
    return (scale * torch.randn(*shape, generator=g)).to(dtype).cuda()


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _layout(rng, new, past, page, spare=3):
    length = np.array([a + b for a, b in zip(new, past)], np.int32)
    most = max(1, -(-int(length.max()) // page))
    pool = len(new) * most + spare
    table = rng.permutation(pool)[:len(new) * most].reshape(len(new), most).astype(np.int32)
    return np.concatenate(([0], np.cumsum(new))).astype(np.int32), length, table, pool


def _tree(rng, kind, n):
    if kind == "chain":
        return np.arange(n) - 1
    if kind == "star":
        return np.full(n, -1)
    if kind == "binary":
        return (np.arange(n) + 1) // 2 - 1
    return np.array([rng.integers(-1, i) if i else -1 for i in range(n)])


def _pages(m, g, pool, H, page, D, dtype, table, length):
    K, V = _randn(g, pool, H, page, D, dtype=dtype), _randn(g, pool, H, page, D, dtype=dtype)
    return K, V, m.PagedKV.view(K, V, _ints(table), _ints(length))


TREES = [
    # dtype, D, H, g, page, new, past, C, counts, kind, pad
    (BF, 128, 2, 1, 64, [15, 15, 15], [300, 20, 0], 200, True, "binary", 0),
    (BF, 128, 3, 5, 16, [64, 1, 0, 33], [127, 128, 50, 0], 130, False, "random", 9),
    (BF, 64, 2, 3, 32, [200, 7], [100, 1000], 0, False, "random", 3),
    (BF, 128, 1, 1, 128, [1], [0], 0, False, "star", 0),
    (BF, 64, 1, 8, 256, [129, 64, 65], [63, 64, 191], 64, True, "star", 0),
    (BF, 128, 2, 1, 16, [300], [5], 257, True, "random", 1),
    (BF, 128, 2, 2, 64, [600], [70], 0, False, "random", 0),
    (F32, 64, 2, 1, 32, [63, 63], [256, 1], 100, True, "binary", 0),
    (F32, 128, 1, 3, 16, [40, 0, 9], [0, 5, 77], 65, False, "random", 5),
    (F32, 64, 1, 2, 64, [130], [63], 0, False, "chain", 0),
]


@pytest.mark.parametrize("dtype,D,H,g,page,new,past,C,counts,kind,pad", TREES)
def test_tree_attention(m, dtype, D, H, g, page, new, past, C, counts, kind, pad):
    rng = np.random.default_rng(sum(new) * 31 + H)
    gen = torch.Generator().manual_seed(sum(new) + C)
    cu, length, table, pool = _layout(rng, new, past, page)
    N = int(cu[-1]) + pad
    K, V, pages = _pages(m, gen, pool, H, page, D, dtype, table, length)
    q = _randn(gen, H * g, N, D, dtype=dtype, scale=1.5)
    parent = np.concatenate([_tree(rng, kind, n) for n in new] + [np.full(pad, 7)])
    prefix = px = None
    if C:
        pK, pV = _randn(gen, H, C, D, dtype=dtype), _randn(gen, H, C, D, dtype=dtype)
        mm = torch.randint(0, 30, (H, C), generator=gen, dtype=torch.int32).cuda() if counts else None
        size = _ints([C - 3 * h for h in range(H)])
        prefix = m.Prefix(pK, pV, m=mm, size=size)
        px = (_f64(pK), _f64(pV), None if mm is None else mm.cpu().numpy(), size.cpu().numpy())
    out = torch.full((H * g, N, D), 7.0, dtype=dtype, device="cuda")
    lse, st = torch.full((H * g, N), 7.0, device="cuda"), _status()
    m.fastar_tree_attention(q, _ints(cu), _ints(parent), prefix, pages, D ** -0.5, out, lse=lse, status=st)
    assert int(st) == 0
    ref, rl, mag, big, keys = O.tree_attention(_f64(q), cu, parent, px, _f64(K), _f64(V), table, length, D ** -0.5)
    T = int(cu[-1])
    d = (D + 4) * 2.0 ** -23 * big + 2.0 ** -20
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + ((2.0 ** -8 if dtype == BF else 0) + 3 * d + keys * 2.0 ** -22)[..., None] * mag
    o, l = _f64(out), _f64(lse)
    assert (np.abs(o - ref)[:, :T] <= 1.01 * tol[:, :T]).all()
    none = rl[:, :T] == -np.inf
    assert (l[:, :T][none] == -np.inf).all()
    ok = np.abs(l - rl) <= d + keys * 2.0 ** -23 + 2.0 ** -22 * np.abs(rl)
    assert ok[:, :T][~none].all()
    assert (o[:, T:] == 7).all() and (l[:, T:] == 7).all()
    if kind == "chain":  # a chain is a row of tokens
        plain, pl = torch.empty_like(out), torch.empty_like(lse)
        m.fastar_branch_attention(q, _ints(cu), prefix, pages, D ** -0.5, plain, lse=pl, block=1)
        assert torch.equal(plain[:, :T], out[:, :T]) and torch.equal(pl[:, :T], lse[:, :T])


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
def test_tree_refuses_parents_on_the_device(m, dtype, D):
    gen, rng = torch.Generator().manual_seed(1), np.random.default_rng(1)
    cu, length, table, pool = _layout(rng, [20, 20], [30, 100], 16)
    K, V, pages = _pages(m, gen, pool, 1, 16, D, dtype, table, length)
    q = _randn(gen, 1, 40, D, dtype=dtype)
    for at, p in ((25, 5), (25, 19), (3, -2), (39, 2 ** 31 - 1), (0, 0)):
        parent, st = np.concatenate([np.arange(20) - 1] * 2), _status()
        parent[at] = p
        m.fastar_tree_attention(q, _ints(cu), _ints(parent), None, pages, 0.1, torch.empty_like(q), status=st)
        assert int(st) == 18


KEEPS = [
    # dtype, D, H, page, new, past, kept tokens of each branch
    (BF, 128, 3, 64, [31, 31, 0, 5], [100, 63, 8, 0], [[0, 2, 6, 14, 30], [], [], [4]]),
    (BF, 64, 2, 16, [300, 77], [0, 1000], [list(range(0, 300, 3)), list(range(77))]),
    (F32, 128, 1, 32, [500], [17], [list(range(250, 500))]),
    (F32, 64, 5, 256, [1, 2000], [255, 1], [[0], list(range(1, 2000))]),
    (BF, 128, 2, 128, [4680], [4680], [list(range(1, 4680, 2))]),
    (F32, 128, 2, 64, [3000], [1], [list(range(100, 3000))]),
    (F32, 128, 20, 64, [500, 600], [1, 9], [list(range(100, 500)), list(range(0, 600, 2))]),
]


@pytest.mark.parametrize("dtype,D,H,page,new,past,kept", KEEPS)
def test_page_keep(m, dtype, D, H, page, new, past, kept):
    gen, rng = torch.Generator().manual_seed(2), np.random.default_rng(2)
    cu, length, table, pool = _layout(rng, new, past, page)
    K, V, pages = _pages(m, gen, pool, H, page, D, dtype, table, length)
    rows = np.array([int(cu[b]) + i for b, k in enumerate(kept) for i in k], np.int32)
    ck = np.concatenate(([0], np.cumsum([len(k) for k in kept]))).astype(np.int32)
    k0, v0 = K.clone(), V.clone()
    ref = [x.float().cpu().numpy() for x in (K, V)]
    O.page_keep(*ref, cu, rows, ck, table, length)
    st = _status()
    m.fastar_page_keep(pages, _ints(cu), _ints(rows), _ints(ck), status=st)
    assert int(st) == 0
    live = np.zeros((pool, page), bool)  # what lies behind the last kept token is unspecified
    for b, k in enumerate(kept):
        for p in range(int(length[b]) - new[b] + len(k)):
            live[table[b, p // page], p % page] = True
    owned = np.zeros((pool, page), bool)
    for b in range(len(new)):
        for p in range(int(length[b])):
            owned[table[b, p // page], p % page] = True
    for x, x0, y in ((K, k0, ref[0]), (V, v0, ref[1])):
        got = x.float().cpu().numpy().swapaxes(1, 2)
        assert np.array_equal(got[live], y.swapaxes(1, 2)[live])
        assert np.array_equal(got[~owned], x0.float().cpu().numpy().swapaxes(1, 2)[~owned])


MASSES = [
    # dtype, D, H, g, page, new, past, block, rows, decay, born, pad
    (BF, 128, 2, 1, 64, [1, 1, 1, 1], [300, 0, 63, 1000], 0, False, 1.0, True, 0),
    (BF, 128, 3, 5, 16, [1, 0, 1], [500, 7, 255], 1, False, 0.9, True, 4),
    (BF, 64, 2, 3, 32, [70, 200], [0, 129], 1, False, 1.0, False, 2),
    (BF, 128, 1, 2, 128, [300], [200], 100, False, 0.5, True, 0),
    (BF, 128, 1, 1, 64, [700], [64], 7, False, 1.0, True, 0),
    (BF, 128, 2, 8, 64, [24, 3, 17], [700, 0, 31], 1, True, 1.0, True, 40),
    (BF, 64, 1, 1, 256, [1, 2], [2000, 255], 0, True, 0.0, False, 1),
    (BF, 128, 1, 1, 64, [1300], [100], 0, False, 1.0, True, 0),
    # several items, and tiles of rows, one after the other on every SM
    (BF, 128, 8, 1, 64, [1] * 40, list(range(300, 700, 10)), 0, False, 1.0, True, 0),
    (BF, 64, 16, 1, 128, [400, 100, 399, 1, 300, 128], [700, 0, 37, 600, 1000, 128], 1, False, 0.9, True, 0),
    (BF, 128, 12, 3, 32, [40, 21, 64, 33], [1500, 2000, 900, 1111], 5, True, 1.0, True, 10),
    # branches of a few rows beside some of many
    (BF, 128, 3, 1, 64, [40, 1, 0, 1, 33, 2, 32], [100, 500, 3, 64, 300, 0, 129], 1, False, 0.7, True, 3),
    (BF, 64, 2, 4, 16, [8, 1, 30, 9, 3, 2, 1, 1], [77, 500, 3, 64, 300, 1, 128, 129], 3, True, 1.0, True, 3),
    (F32, 64, 2, 1, 32, [1, 1], [256, 1], 0, False, 1.0, True, 0),
    (F32, 64, 12, 1, 32, [90] * 5, [700] * 5, 1, False, 1.0, True, 0),
    (F32, 128, 1, 3, 16, [40, 0, 9], [0, 5, 77], 1, True, 0.9, True, 11),
    (F32, 64, 1, 2, 64, [400], [63], 13, False, 1.0, True, 0),
]


@pytest.mark.parametrize("dtype,D,H,g,page,new,past,block,taken,decay,stamps,pad", MASSES)
def test_page_mass(m, dtype, D, H, g, page, new, past, block, taken, decay, stamps, pad):
    rng = np.random.default_rng(sum(new) * 17 + D)
    gen = torch.Generator().manual_seed(sum(new) + g)
    cu, length, table, pool = _layout(rng, new, past, page)
    T = int(cu[-1])
    N = T + pad
    K, V, pages = _pages(m, gen, pool, H, page, D, dtype, table, length)
    q = _randn(gen, H * g, N, D, dtype=dtype, scale=1.5)
    lse = (_randn(gen, H * g, N, dtype=F32) + 7.0)
    lse[:, N // 3] = -torch.inf  # a row that saw nothing
    rows = np.sort(rng.permutation(N)[:T]).astype(np.int32) if taken else None
    mass = (3 * torch.rand(pool, H, page, generator=gen)).cuda()
    born = torch.full((pool, H, page), -5, dtype=torch.int32, device="cuda") if stamps else None
    total = _ints(length + 100) if stamps else None
    held = m.PageMass.view(mass, born, total)
    ref, rb = _f64(mass), None if born is None else born.cpu().numpy().copy()
    tol = O.page_mass(_f64(K), _f64(q), _f64(lse), rows, cu, table, length, D ** -0.5, block, decay, ref, rb,
                      length + 100)
    st = _status()
    offsets = _ints(cu)
    # rows of padding behind the last branch's (M counts them too)
    ids = None if rows is None else _ints(np.concatenate((rows, np.full(2, 2 ** 30))))
    m.fastar_page_mass(pages, q, lse, offsets, D ** -0.5, held, block=block, rows=ids, decay=decay, status=st)
    assert int(st) == 0
    assert (np.abs(_f64(mass) - ref) <= 1.05 * tol).all()
    if born is not None:
        assert np.array_equal(born.cpu().numpy(), rb)
    before = mass.clone()
    if decay == 1.0 and not stamps:
        return
    # the same call gives the same bits
    mass.copy_(before)
    m.fastar_page_mass(pages, q, lse, offsets, D ** -0.5, held, block=block, rows=ids, decay=decay, status=st)
    once = mass.clone()
    mass.copy_(before)
    m.fastar_page_mass(pages, q, lse, offsets, D ** -0.5, held, block=block, rows=ids, decay=decay, status=st)
    assert torch.equal(once, mass) and int(st) == 0


EVICTS = [
    # dtype, D, H, page, lengths, budget, first, recent, stamps, masses
    (BF, 128, 3, 64, [300, 100, 101, 0], 100, 4, 20, True, "random"),
    (BF, 64, 2, 16, [1000, 33], 32, 0, 32, False, "random"),
    (F32, 128, 1, 32, [700], 333, 7, 0, True, "ties"),
    (F32, 64, 4, 256, [5000, 257], 1, 0, 0, True, "random"),
    (BF, 128, 2, 128, [2049, 2048], 2048, 16, 100, True, "random"),
    (BF, 128, 1, 16, [500], 0, 0, 0, True, "random"),
    (BF, 64, 2, 64, [9000, 8193], 4097, 3, 64, False, "odd"),
    (F32, 64, 1, 64, [40000], 20001, 3, 64, True, "ties"),
    (BF, 128, 2, 32, [96, 97], 96, 0, 96, True, "random"),
    (BF, 64, 90, 32, [64] * 4, 30, 1, 5, True, "ties"),
]


@pytest.mark.parametrize("dtype,D,H,page,lengths,budget,first,recent,stamps,kind", EVICTS)
@pytest.mark.parametrize("apart", [False, True])
def test_page_evict(m, dtype, D, H, page, lengths, budget, first, recent, stamps, kind, apart):
    rng = np.random.default_rng(sum(lengths) + budget)
    gen = torch.Generator().manual_seed(sum(lengths))
    cu, length, table, pool = _layout(rng, lengths, [0] * len(lengths), page)
    K, V, pages = _pages(m, gen, pool, H, page, D, dtype, table, length)
    x = rng.random((pool, H, page)).astype(np.float32)
    if kind == "ties":
        x = np.floor(x * 4).astype(np.float32)
    if kind == "odd":
        x[x < 0.1] = np.nan
        x[(x > 0.1) & (x < 0.2)] = -0.0
        x[x > 0.97] = np.inf
        x[(x > 0.9) & (x < 0.95)] = -np.inf
        x[(x > 0.2) & (x < 0.25)] = 0.0
        x[(x > 0.25) & (x < 0.3)] = 1e-41  # below the normal numbers
    born = np.zeros((pool, H, page), np.int32)
    for b, n in enumerate(lengths):  # an order of their own in every head
        for h in range(H):
            for p, t in enumerate(rng.permutation(n + 10)[:n]):
                born[table[b, p // page], h, p % page] = t
    total = length + 10
    mass, stamp = torch.from_numpy(x).cuda(), torch.from_numpy(born).cuda()
    held = m.PageMass.view(mass, stamp if stamps else None, _ints(total) if stamps else None)
    mass0, born0, k0, v0 = mass.clone(), stamp.clone(), K.clone(), V.clone()
    out = None
    if apart:
        out = m.PageMass.view(torch.full_like(mass, 7.0), torch.full_like(stamp, 7) if stamps else None, held.total)
    want = [K.float().cpu().numpy(), V.float().cpu().numpy(), x.copy(), born.copy()]
    O.page_evict(want, x, born if stamps else None, total, table, length, budget, first, recent)
    st = _status()
    m.fastar_page_evict(pages, held, budget, first=first, recent=recent, out=out, status=st)
    assert int(st) == 0
    kept = np.zeros((pool, page), bool)
    for b, n in enumerate(lengths):
        for p in range(min(n, budget)):
            kept[table[b, p // page], p % page] = True
    to = held if out is None else out
    got = [K, V, to.mass] + ([to.born] if stamps else [])
    for y, w in zip(got, want):
        y = y.float().cpu().numpy() if y.is_floating_point() else y.cpu().numpy()
        assert np.array_equal(y.swapaxes(1, 2)[kept], w.swapaxes(1, 2)[kept], equal_nan=y.dtype.kind == "f")
    if apart:
        assert torch.equal(mass.view(torch.int32), mass0.view(torch.int32)) and torch.equal(stamp, born0)
        rest = torch.from_numpy(~kept).cuda()
        assert (out.mass.transpose(1, 2)[rest] == 7).all()
    # nothing but positions below the budget is written
    outside = torch.from_numpy(~kept).cuda()
    for y, y0 in ((K, k0), (V, v0)):
        assert torch.equal(y.transpose(1, 2)[outside], y0.transpose(1, 2)[outside])


def _attend_rows(x, rows):
    return x[:, torch.as_tensor(rows, device="cuda", dtype=torch.long)]


@pytest.mark.parametrize("dtype,D,g", [(BF, 128, 2), (F32, 64, 1)])
def test_rollout_of_drafts_under_a_budget(m, dtype, D, g):
    """Steps of drafts, accepted paths, a step of plain tokens and evictions, as a
    rollout strings them together, against the oracle's own pages."""
    from merged_attention_autoregressive_gb300.path import BranchRollout
    rng, gen = np.random.default_rng(3), torch.Generator().manual_seed(3)
    B, H, page, tokens, budget = 3, 2, 16, 90, 60
    Hq, C = H * g, 70
    pK, pV = _randn(gen, H, C, D, dtype=dtype), _randn(gen, H, C, D, dtype=dtype)
    plan = m.RopePlan(D, (D,))
    r = BranchRollout(B, H, D, tokens, 200, prefix=m.Prefix(pK, pV), Hq=Hq, page=page, plan=plan, block=1, dtype=dtype,
                      budget=budget, first=2, recent=10, decay=0.97)
    free = len(r.free)
    # the oracle's state: rows of each branch and head, their masses and token numbers
    rows = [[[] for _ in range(H)] for _ in range(B)]
    count = [0] * B
    for step in range(6):
        drafted = step % 3 != 2
        new = [int(rng.integers(0, 30)) for _ in range(B)]
        trees = [list(map(int, _tree(rng, "random", n))) for n in new]
        T = sum(new)
        r.extend(new, parents=trees if drafted else None)
        q, k, v = (_randn(gen, h, tokens, D, dtype=dtype) for h in (Hq, H, H))
        pos = np.zeros((tokens, 1), np.int32)
        at = 0
        for b, n in enumerate(new):
            for i in range(n):
                depth = len(O.above(trees[b], i)) if drafted else i + 1
                pos[at + i] = count[b] + depth - 1
            at += n
        out, lse = r.step(q, k, v, _ints(pos))
        turned = [torch.empty_like(x) for x in (q, k)]
        for x, y in zip((q, k), turned):
            m.fastar_rope(x, _ints(pos), plan, y)
        qf, kf, vf = _f64(turned[0]), _f64(turned[1]), _f64(v)
        o, l = _f64(out), _f64(lse)
        leaves, at = [], 0
        for b, n in enumerate(new):
            past = [[e for e in rows[b][h]] for h in range(H)]
            paths = [O.above(trees[b], i) if drafted else list(range(i + 1)) for i in range(n)]
            leaf = int(rng.integers(-1, n)) if n else -1
            leaves.append(leaf)
            stay = (paths[leaf] if leaf >= 0 else []) if drafted else list(range(n))
            for h in range(H):
                for i in range(n):
                    ks = np.array([_f64(pK)[h, c] for c in range(C)] + [e[0] for e in past[h]] + [kf[h, at + j] for j in paths[i]])
                    vs = np.array([_f64(pV)[h, c] for c in range(C)] + [e[1] for e in past[h]] + [vf[h, at + j] for j in paths[i]])
                    for e in range(h * g, (h + 1) * g):
                        x = D ** -0.5 * (ks @ qf[e, at + i])
                        w = np.exp(x - x.max())
                        ref, rl = (w / w.sum()) @ vs, x.max() + np.log(w.sum())
                        X = D ** -0.5 * (np.abs(ks) @ np.abs(qf[e, at + i])).max()
                        d = (D + 4) * 2.0 ** -23 * X + 2.0 ** -20
                        mag = (w / w.sum()) @ np.abs(vs)
                        tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + ((2.0 ** -8 if dtype == BF else 0) + 3 * d + len(ks) * 2.0 ** -22) * mag
                        assert (np.abs(o[e, at + i] - ref) <= 1.01 * tol).all()
                        assert abs(l[e, at + i] - rl) <= d + len(ks) * 2.0 ** -23 + 2.0 ** -22 * abs(rl)
                # weights of the tokens that stay, over all rows they see
                kept = [[kf[h, at + i], vf[h, at + i], 0.0, count[b] + j] for j, i in enumerate(stay)]
                for e in rows[b][h]:
                    e[2] *= 0.97 if stay else 1.0
                for j, i in enumerate(stay):
                    for e in rows[b][h] + kept[:j + 1]:
                        for head in range(h * g, (h + 1) * g):
                            e[2] += np.exp(D ** -0.5 * (e[0] @ qf[head, at + i]) - l[head, at + i])
                rows[b][h] += kept
            count[b] += len(stay)
            at += n
        if drafted:
            ids = r.accept(leaves)
            assert [len(x) for x in ids] == [len(O.above(t, x)) for t, x in zip(trees, leaves)]
        assert r.lengths == [len(rows[b][0]) for b in range(B)]
        if step in (2, 4, 5):
            r.evict()
            for b in range(B):
                for h in range(H):
                    x = rows[b][h]
                    if len(x) <= budget:
                        continue
                    order = sorted(range(len(x)), key=lambda p: (not (x[p][3] < 2 or x[p][3] >= count[b] - 10), -x[p][2], p))
                    safe = sum(x[p][3] < 2 or x[p][3] >= count[b] - 10 for p in order)
                    last, next_ = x[order[budget - 1]][2], x[order[budget]][2]
                    assert safe >= budget or last - next_ > 1e-4 * last  # (no decision within the masses' errors)
                    kept = set(order[:budget])
                    holes = [p for p in range(budget) if p not in kept]
                    for dst, src in zip(holes, sorted(p for p in kept if p >= budget)):
                        x[dst] = x[src]
                    del x[budget:]
        # the rows in the pages, their masses and numbers
        assert sorted([p for x in r.held for p in x] + r.free) == list(range(free))
        for b in range(B):
            assert r.pages.len[b].item() == len(rows[b][0]) == r.lengths[b] and len(r.held[b]) == -(-r.lengths[b] // page)
            for h in range(H):
                for p, e in enumerate(rows[b][h]):
                    i, s = r.held[b][p // page], p % page
                    assert np.array_equal(_f64(r.pages.K[i, h, s]), e[0]) and np.array_equal(_f64(r.pages.V[i, h, s]), e[1])
                    assert r.mass.born[i, h, s].item() == e[3]
                    assert abs(r.mass.mass[i, h, s].item() - e[2]) <= 1e-4 * e[2]
    assert int(r.status) == 0
