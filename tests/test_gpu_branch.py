"""Branched rollouts on the GPU against the 64-bit oracle: rotary positions
with several axes, the append to pages, the attention over a shared prefix.

Bounds.  u is half a step of the output's type (finfo.eps / 2).
Rotation: each product and the sum round once in 32 bits, the half turns and
their sine and cosine are within 2^-22, the result rounds once:
  |err| <= u |y| + 2^-20 (|x0| + |x1|) + the angle's own error, which is that of
  64-bit products on both sides: 2^-51 |pos freq| (|x0| + |x1|).
Attention: with X the row's largest scale sum |q k|, A = sum p |v| and n keys,
  score error d <= (D + 4) 2^-23 X + 2^-20 (32-bit sums in any order, the bias
  and the exponential), so p changes by at most 2 d + n 2^-23 in relation to
  its sum, and bf16 rounds each p by at most 2^-8:
  |err| <= u |out| + ((2^-8 for bf16) + 3 d + n 2^-22) A,  lse: d + n 2^-23 + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest
import torch

from oracle import branch_oracle as O

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


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _rope_bound(x, y, pos, dims, freqs, halves, dtype):
    axis = np.repeat(np.arange(len(dims)), [d // 2 for d in dims])
    n = len(axis)
    angle = np.abs(np.asarray(pos, np.float64)[:, axis] * freqs)
    i = np.arange(n)
    a, b = (i, i + n) if halves else (2 * i, 2 * i + 1)
    t = np.zeros_like(y)
    pair = (np.abs(x[..., a]) + np.abs(x[..., b])) * (2.0 ** -20 + angle * 2.0 ** -51)
    t[..., a] = t[..., b] = pair
    return t * 1.01 + _half(dtype) * np.abs(y) * 1.001 * (t > 0)


ROPE = [
    # dtype, D, dims, halves, H, N, inverse
    (BF, 128, (44, 42, 42), False, 12, 1, False),
    (BF, 128, (44, 42, 42), False, 3, 333, True),
    (BF, 128, (128,), True, 5, 65, False),
    (BF, 128, (64, 32, 32), True, 40, 31, True),
    (BF, 128, (32, 16), True, 2, 40, False),
    (BF, 128, (30, 8), False, 7, 33, False),
    (BF, 64, (24, 20, 20), False, 4, 129, False),
    (BF, 64, (16,), True, 1, 7, False),
    (BF, 64, (2,), False, 9, 64, True),
    (F32, 128, (44, 42, 42), False, 4, 50, False),
    (F32, 128, (0, 64, 48), True, 6, 17, True),
    (F32, 64, (16, 24, 24), True, 5, 257, True),
    (F32, 64, (10, 6, 4, 2), False, 3, 100, False),
]


@pytest.mark.parametrize("dtype,D,dims,halves,H,N,inverse", ROPE)
@pytest.mark.parametrize("layout", ["token", "head", "pitch"])
def test_rope(m, dtype, D, dims, halves, H, N, inverse, layout):
    g = torch.Generator().manual_seed(N * 7 + H)
    if layout == "head":
        x = _randn(g, H, N, D, dtype=dtype)
    else:
        pad = 8 if layout == "pitch" else 0
        x = _randn(g, N, H * D + pad, dtype=dtype)[:, :H * D].view(N, H, D).transpose(0, 1)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (N, len(dims)), generator=g, dtype=torch.int64)
    pos[::2] %= 100000
    pos = pos.to(torch.int32).cuda()
    freqs = O.ladder(dims, 10000.0)
    plan = m.RopePlan(D, dims, pairing="halves" if halves else "adjacent")
    out = torch.full((N, H, D) if layout == "pitch" else (H, N, D), 7.0, dtype=dtype, device="cuda")
    view = out.transpose(0, 1) if layout == "pitch" else out
    st = _status()
    m.fastar_rope(x, pos, plan, view, inverse=inverse, status=st)
    ref = O.rope(_f64(x), pos.cpu().numpy(), dims, freqs, halves, inverse)
    tol = _rope_bound(_f64(x), ref, pos.cpu().numpy(), dims, freqs, halves, dtype)
    assert (np.abs(_f64(view) - ref) <= tol).all()
    assert int(st) == 0
    # in place, and back again
    y = x.clone().contiguous()
    m.fastar_rope(y, pos, plan, y, inverse=inverse, status=st)
    assert torch.equal(y, view.contiguous())


def test_rope_copies_the_channels_behind_and_takes_any_value(m):
    x = torch.zeros(1, 2, 64, device="cuda")
    x[0, 0, 8:] = torch.tensor([math.inf, -math.inf, math.nan, -0.0] * 14, device="cuda")
    x[0, 1, :8] = math.inf
    pos = torch.tensor([[3], [0]], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    m.fastar_rope(x, pos, m.RopePlan(64, (8,)), out)
    assert torch.equal(out[0, 0, 8:].view(torch.int32), x[0, 0, 8:].view(torch.int32))
    assert out[0, 1, :8].isnan().any()  # inf cos - inf sin, as the formula has it


def test_rope_reads_expanded_rows(m):
    g = torch.Generator().manual_seed(5)
    one = _randn(g, 1, 20, 64)
    pos = torch.arange(20, dtype=torch.int32, device="cuda")[:, None]
    plan, out = m.RopePlan(64, (64,)), torch.empty(6, 20, 64, dtype=BF, device="cuda")
    m.fastar_rope(one.expand(6, 20, 64), pos, plan, out)
    ref = torch.empty(1, 20, 64, dtype=BF, device="cuda")
    m.fastar_rope(one, pos, plan, ref)
    assert torch.equal(out, ref.expand(6, 20, 64))


def _layout(rng, new, past, page, spare=3):
    """cu, len and a scattered page table for branches of `past` positions
    that add `new` tokens."""
    length = np.array([a + b for a, b in zip(new, past)], np.int32)
    most = max(1, -(-int(length.max()) // page))
    pool = len(new) * most + spare
    table = rng.permutation(pool)[:len(new) * most].reshape(len(new), most).astype(np.int32)
    cu = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    return cu, length, table, pool


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


APPEND = [
    # dtype, D, H, Hq, page, new, past, pad, dims, halves
    (BF, 128, 12, 12, 64, [1] * 16, [63, 64, 65, 0] * 4, 0, (44, 42, 42), False),
    (BF, 128, 3, 6, 16, [5, 0, 17, 1, 33], [0, 9, 15, 16, 31], 4, (44, 42, 42), True),
    (BF, 64, 5, 0, 256, [300, 1], [1, 255], 0, (24, 20, 20), False),
    (F32, 64, 2, 2, 32, [40, 0, 0, 24], [100, 0, 3, 8], 9, (16, 16), True),
    (F32, 128, 1, 4, 128, [129], [0], 1, (128,), False),
    (BF, 64, 1, 1, 16, [0, 0], [4, 5], 3, (64,), False),
    (BF, 128, 2, 0, 64, [1] * 300, [0] * 300, 0, (44, 42, 42), False),
]


@pytest.mark.parametrize("dtype,D,H,Hq,page,new,past,pad,dims,halves", APPEND)
@pytest.mark.parametrize("turned", [True, False])
def test_page_append(m, dtype, D, H, Hq, page, new, past, pad, dims, halves, turned):
    if dims == (44, 42, 42) and halves:
        dims = (48, 40, 40)
    rng = np.random.default_rng(len(new) + page)
    g = torch.Generator().manual_seed(page)
    cu, length, table, pool = _layout(rng, new, past, page)
    N = int(cu[-1]) + pad
    rows = _randn(g, N, Hq + 2 * H, D, dtype=dtype).transpose(0, 1)
    q, k, v = rows[:Hq], rows[Hq:Hq + H], rows[Hq + H:]
    pos = torch.randint(-50, 100000, (N, len(dims)), generator=g, dtype=torch.int32).cuda()
    pages = m.PagedKV(H, D, page, pool, len(new), table.shape[1], dtype)
    pages.K.copy_(_randn(g, *pages.K.shape, dtype=dtype))
    pages.V.copy_(_randn(g, *pages.V.shape, dtype=dtype))
    pages.table.copy_(_cuda(table))
    pages.len.copy_(_cuda(length))
    K0, V0 = _f64(pages.K), _f64(pages.V)
    q_out = torch.full((Hq, N, D), 3.0, dtype=dtype, device="cuda") if Hq else None
    plan = m.RopePlan(D, dims, pairing="halves" if halves else "adjacent")
    st = _status()
    m.fastar_page_append(pages, k, v, _cuda(cu), pos=pos if turned else None, plan=plan if turned else None,
                         q=q if Hq else None, q_out=q_out, status=st)
    assert int(st) == 0
    freqs, p = O.ladder(dims), pos.cpu().numpy()
    turn = (lambda x: O.rope(x, p, dims, freqs, halves)) if turned else (lambda x: x)
    tol = (lambda x: _rope_bound(x, turn(x), p, dims, freqs, halves, dtype)) if turned else (lambda x: np.zeros_like(x))
    KT, VT = np.zeros_like(K0), np.zeros_like(V0)
    O.page_append(K0, V0, turn(_f64(k)), _f64(v), cu, table, length)
    O.page_append(KT, VT, tol(_f64(k)), 0 * _f64(v), cu, table, length)
    assert (np.abs(_f64(pages.K) - K0) <= KT).all()  # rows of no token: unchanged to the bit
    np.testing.assert_array_equal(_f64(pages.V), V0)
    if Hq:
        n = int(cu[-1])
        assert (np.abs(_f64(q_out) - turn(_f64(q)))[:, :n] <= tol(_f64(q))[:, :n]).all()
        assert bool((q_out[:, n:] == 3.0).all())


def _attention_case(m, dtype, D, H, g, page, new, past, C, counts, block, pad=0, seed=0, qscale=1.5, spoil=True):
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    cu, length, table, pool = _layout(rng, new, past, page)
    N = int(cu[-1]) + pad
    q = _randn(gen, H * g, N, D, dtype=dtype, scale=qscale)
    pages = m.PagedKV(H, D, page, pool, len(new), table.shape[1], dtype)
    pages.K.copy_(_randn(gen, *pages.K.shape, dtype=dtype))
    pages.V.copy_(_randn(gen, *pages.V.shape, dtype=dtype))
    pages.table.copy_(_cuda(table))
    pages.len.copy_(_cuda(length))
    size = rng.integers(0, C + 1, H).astype(np.int32)
    if C:
        size[0] = C
    cnt = rng.integers(0 if C > 1 else 1, 50, (H, C)).astype(np.int32)
    pK, pV = _randn(gen, H, C, D, dtype=dtype), _randn(gen, H, C, D, dtype=dtype)
    prefix = None
    if C:
        prefix = (pK, pV, cnt if counts else None, size if counts else None)
    if spoil:
        # nobody's rows hold anything at all: rows behind a branch's length,
        # spare pages, prefix rows behind a head's size, padding queries
        used = np.zeros((pool, page), bool)
        for b in range(len(new)):
            p = np.arange(length[b])
            used[table[b][p // page], p % page] = True
        free = _cuda(~used)[:, None, :, None]
        pages.K.masked_fill_(free, math.nan)
        pages.V.masked_fill_(free, math.inf)
        if C and counts:
            dead = _cuda(np.arange(C)[None] >= size[:, None])[..., None]
            pK.masked_fill_(dead, -math.inf)
            pV.masked_fill_(dead, math.nan)
        q[:, int(cu[-1]):] = math.nan
    return q, _cuda(cu), prefix, pages, cu, length, table


def _check_attention(m, dtype, q, cu, prefix, pages, scale, block, cu_h, length, table, ws=None):
    Hq, N, D = q.shape
    out = torch.full_like(q, 9.0)
    lse = torch.full((Hq, N), 9.0, device="cuda")
    st = _status()
    px = None
    if prefix is not None:
        pK, pV, cnt, size = prefix
        px = m.Prefix(pK, pV, m=None if cnt is None else _cuda(cnt), size=None if size is None else _cuda(size))
    m.fastar_branch_attention(q, cu, px, pages, scale, out, lse=lse, block=block, ws=ws, status=st)
    assert int(st) == 0
    n = int(cu_h[-1])
    host = None if prefix is None else (_f64(prefix[0]), _f64(prefix[1]), prefix[2], prefix[3])
    ref, rl, A, X, keys = O.branch_attention(_f64(q), cu_h, host, _f64(pages.K), _f64(pages.V), table, length, scale,
                                             block, bounds=True)
    d = (D + 4) * 2.0 ** -23 * X + 2.0 ** -20
    p = (2.0 ** -8 if dtype == BF else 0.0) + 3 * d + keys * 2.0 ** -22
    err = np.abs(_f64(out) - ref)[:, :n]
    tol = (_half(dtype) * np.abs(ref) + p[..., None] * A)[:, :n]
    assert np.isfinite(_f64(out)[:, :n]).all()
    assert (err <= tol).all(), f"worst {np.max(err / np.maximum(tol, 1e-30)):.3g} of the bound"
    got = _f64(lse)[:, :n]
    none = np.isneginf(rl[:, :n])
    assert (np.isneginf(got) == none).all()
    assert (_f64(out)[:, :n][none] == 0).all()
    with np.errstate(invalid="ignore"):
        le = np.where(none, 0, np.abs(got - rl[:, :n]))
        lt = np.where(none, 0, d[:, :n] + keys[:, :n] * 2.0 ** -23 + 2.0 ** -22 * np.abs(rl[:, :n]))
    assert (le <= lt).all()
    # padding rows stay as they were
    assert bool((out[:, n:] == 9.0).all()) and bool((lse[:, n:] == 9.0).all())
    return out, lse


ATTEND = [
    # D, H, g, page, new, past, C, counts, block, pad
    (128, 2, 1, 64, [1], [0], 0, False, 0, 0),                       # one token, its own key only
    (128, 12, 1, 64, [1] * 4, [300, 0, 63, 64], 500, True, 0, 0),    # single tokens over a history
    (128, 3, 5, 16, [1] * 9, [0, 1, 15, 16, 17, 127, 128, 129, 400], 1000, True, 0, 2),
    (128, 1, 8, 32, [1] * 40, list(range(0, 800, 20)), 257, False, 0, 0),  # more than 256 rows, many branches
    (64, 4, 3, 16, [7, 0, 130, 1, 64], [9, 3, 0, 255, 31], 0, False, 1, 5),  # causal, no prefix
    (128, 2, 1, 128, [200, 60], [56, 196], 640, True, 256, 0),       # causal by block, past 256 rows
    (128, 2, 2, 256, [300], [0], 100, False, 1, 0),
    (64, 1, 1, 64, [128], [0], 128, True, 0, 0),                     # exact tiles
    (64, 2, 7, 64, [37, 19], [5, 0], 129, True, 7, 1),               # odd groups, odd blocks
    (128, 5, 1, 16, [0, 0, 3], [0, 7, 0], 1, True, 1, 0),
    (128, 1, 1, 64, [700], [0], 2000, False, 0, 3),
    (128, 3, 1, 32, [3, 3], [-2, 500], 0, False, 1, 0),              # tokens in front of the branch see nothing
    (64, 2, 1, 16, [2] * 70, [0] * 70, 40, True, 2, 0),              # many small branches in a tile
]


@pytest.mark.parametrize("case", range(len(ATTEND)))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_branch_attention(m, case, dtype):
    D, H, g, page, new, past, C, counts, block, pad = ATTEND[case]
    q, cu, prefix, pages, cu_h, length, table = _attention_case(m, dtype, D, H, g, page, new, past, C, counts, block,
                                                                pad, seed=case)
    _check_attention(m, dtype, q, cu, prefix, pages, D ** -0.5, block, cu_h, length, table)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_of_far_apart_scores(m, dtype):
    """Scores over hundreds: the running maximum is raised again and again."""
    q, cu, prefix, pages, cu_h, length, table = _attention_case(
        m, dtype, 128, 2, 2, 64, [70, 1], [500, 900], 700, True, 0, seed=3, qscale=40.0)
    _check_attention(m, dtype, q, cu, prefix, pages, 128 ** -0.5, 0, cu_h, length, table)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_over_nothing_at_all(m, dtype):
    """No prefix row lives and a branch is empty: 0 and -inf, written."""
    q, cu, prefix, pages, cu_h, length, table = _attention_case(
        m, dtype, 64, 2, 1, 16, [3, 2], [-3, 4], 50, True, 0, seed=4, spoil=False)
    prefix = (prefix[0], prefix[1], np.zeros_like(prefix[2]), prefix[3])  # every group hidden
    out, lse = _check_attention(m, dtype, q, cu, prefix, pages, 0.1, 0, cu_h, length, table)
    assert bool((out[:, :3] == 0).all()) and bool(torch.isneginf(lse[:, :3]).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,H,g,new,past,C,block", [
    (128, 2, 3, [1, 1, 1], [5, 0, 200], 1000, 0),    # single tokens
    (64, 2, 1, [40, 9], [0, 3], 300, 1),             # rows of several branches in a tile
    (128, 8, 1, [600, 640], [0, 100], 9700, 640),    # 256 rows at a time
])
def test_hidden_groups_may_hold_anything(m, dtype, D, H, g, new, past, C, block):
    q, cu, prefix, pages, cu_h, length, table = _attention_case(m, dtype, D, H, g, 64, new, past, C, True, block, seed=6)
    pK, pV, cnt, size = prefix
    cnt[:, C // 3:C // 3 + 150] = 0
    out, lse = _check_attention(m, dtype, q, cu, prefix, pages, D ** -0.5, block, cu_h, length, table)
    hidden = _cuda(cnt <= 0)[..., None]
    pK.masked_fill_(hidden, math.nan)
    pV.masked_fill_(hidden, math.inf)
    again, lse2 = torch.full_like(out, 9.0), torch.full_like(lse, 9.0)
    m.fastar_branch_attention(q, cu, m.Prefix(pK, pV, m=_cuda(cnt), size=_cuda(size)), pages, D ** -0.5, again,
                              lse=lse2, block=block)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tables_far_longer_than_the_branches(m, dtype):
    """Room for 2^31 positions a branch: the units are counted in 64 bits."""
    q, cu, prefix, pages, cu_h, length, table = _attention_case(
        m, dtype, 64, 2, 2, 256, [1] * 5, [0, 255, 256, 600, 31], 300, True, 0, seed=8)
    big = torch.zeros(5, 2 ** 23 - 1, dtype=torch.int32, device="cuda")
    big[:, :table.shape[1]] = pages.table
    far = m.PagedKV.view(K=pages.K, V=pages.V, table=big, length=pages.len)
    _check_attention(m, dtype, q, cu, prefix, far, 0.125, 0, cu_h, length, table)


def test_a_visible_nan_is_not_swallowed(m):
    q, cu, prefix, pages, cu_h, length, table = _attention_case(
        m, BF, 128, 2, 1, 64, [2, 2], [100, 100], 300, False, 0, seed=5, spoil=False)
    prefix[0][0, 17] = math.nan  # a key of head 0 that every token sees
    out, lse = torch.zeros_like(q), torch.zeros(2, 4, device="cuda")
    m.fastar_branch_attention(q, cu, m.Prefix(prefix[0], prefix[1]), pages, 0.1, out, lse=lse)
    assert bool(out[0].isnan().all()) and bool(lse[0].isnan().all())
    assert bool(out[1].isfinite().all()) and bool(lse[1].isfinite().all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_over_a_prefix_past_4_gib(m, dtype):
    """The prefix of the last head lies past 32-bit byte and element offsets."""
    H, D = 40, 128
    C = 500000 if dtype == BF else 450000
    K = torch.zeros(H, C, D, dtype=dtype, device="cuda")
    V = torch.zeros(H, C, D, dtype=dtype, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    K[-1].normal_(generator=gen)
    V[-1].normal_(generator=gen)
    size = torch.full((H,), 3, dtype=torch.int32, device="cuda")
    size[-1] = C
    pages = m.PagedKV(H, D, 64, 4, 1, 2, dtype)
    pages.len.fill_(1)
    q = torch.randn(H, 1, D, generator=gen, device="cuda").to(dtype)
    out, cu = torch.zeros_like(q), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    st = _status()
    m.fastar_branch_attention(q, cu, m.Prefix(K, V, size=size), pages, 0.1, out, status=st)
    x = torch.cat((K[-1].double() @ q[-1, 0].double() * 0.1, torch.zeros(1, device="cuda", dtype=torch.float64)))
    p = torch.softmax(x, 0)
    ref = p[:-1] @ V[-1].double()
    A = p[:-1] @ V[-1].double().abs()
    tol = _half(dtype) * ref.abs() + ((2.0 ** -8 if dtype == BF else 0) + C * 2.0 ** -22) * A
    assert bool(((out[-1, 0].double() - ref).abs() <= tol).all()) and int(st) == 0
    # ... a bound that a wrong row cannot meet: the mean of the values is far smaller than a value
    assert float(tol.max()) < 0.2 * float(V[-1].abs().mean())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_results_do_not_change_from_run_to_run(m, dtype):
    q, cu, prefix, pages, cu_h, length, table = _attention_case(m, dtype, 128, 4, 2, 64, [90, 1, 40], [700, 30, 5],
                                                                900, True, 1, seed=6)
    px = m.Prefix(prefix[0], prefix[1], m=_cuda(prefix[2]), size=_cuda(prefix[3]))
    outs = []
    for _ in range(3):
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        m.fastar_branch_attention(q, cu, px, pages, 0.09, out, lse=lse, block=1)
        outs.append((out, lse))
    assert all(torch.equal(a, outs[0][0]) and torch.equal(b, outs[0][1]) for a, b in outs)


@pytest.mark.parametrize("D,H,new,C,block", [
    (128, 40, [1300, 748], 700, 0),    # 256 rows at a time, items that are finished one after the other in a run
    (64, 40, [1300, 748], 700, 1),
    (128, 12, [40] * 50, 300, 8),      # 128 rows at a time
])
def test_many_items_of_a_run_do_not_disturb_each_other(m, D, H, new, C, block):
    q, cu, prefix, pages, *_ = _attention_case(m, BF, D, H, 1, 64, new, [300] * len(new), C, True, block, seed=9,
                                               spoil=False)
    px = m.Prefix(prefix[0], prefix[1], m=_cuda(prefix[2]))
    want = None
    for _ in range(60):
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        m.fastar_branch_attention(q, cu, px, pages, 0.09, out, lse=lse, block=block)
        if want is None:
            want = out, lse
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_sticky_status_and_device_refusals(m):
    """Bad lengths, offsets and page ids set the status word; a set word
    stops every call; nothing faults."""
    q, cu, prefix, pages, cu_h, length, table = _attention_case(m, BF, 128, 2, 1, 64, [3, 2], [100, 90], 200, True, 0,
                                                                seed=7)
    px = m.Prefix(prefix[0], prefix[1], m=_cuda(prefix[2]), size=_cuda(prefix[3]))
    k = torch.zeros(2, 5, 128, dtype=BF, device="cuda")

    def attend(cu=cu, pages=pages, px=px, st=None):
        out = torch.full_like(q, 5.0)
        st = _status() if st is None else st
        m.fastar_branch_attention(q, cu, px, pages, 0.1, out, status=st)
        return int(st), out

    def append(cu=cu, pages=pages, st=None):
        st = _status() if st is None else st
        m.fastar_page_append(pages, k, k, cu, status=st)
        return int(st)

    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    other = lambda table=None, length=None: m.PagedKV.view(  # noqa: E731
        pages.K, pages.V, pages.table if table is None else table, pages.len if length is None else length)
    assert attend()[0] == 0
    for bad in (i32(0, 4, 3), i32(0, 3, 6), i32(1, 3, 5), i32(0, -1, 5)):
        rc, out = attend(cu=bad)
        assert rc == 18 and bool((out == 5.0).all())
        assert append(cu=bad) == 18
    for bad in (i32(103, -1), i32(103, 100000)):
        rc, out = attend(pages=other(length=bad))
        assert rc == 18 and bool((out == 5.0).all())
        assert append(pages=other(length=bad)) == 18
    for bad in (-1, pages.n_pages, 2 ** 31 - 1):
        t = pages.table.clone()
        t[1, 1] = bad
        assert attend(pages=other(table=t))[0] == 18
        assert append(pages=other(table=t)) == 18
    for bad in (-1, 201):
        assert attend(px=m.Prefix(prefix[0], prefix[1], size=i32(5, bad)))[0] == 18
    before = pages.K.clone()
    st = _status() + 16
    rc, out = attend(st=st)
    assert rc == 16 and bool((out == 5.0).all())
    assert append(st=st) == 16 and torch.equal(before.view(torch.int16), pages.K.view(torch.int16))
    out = torch.full_like(q, 5.0)
    m.fastar_rope(q, torch.zeros(5, 1, dtype=torch.int32, device="cuda"), m.RopePlan(128, (128,)), out, status=st)
    assert bool((out == 5.0).all())


def test_a_rollout_of_branches_step_by_step(m):
    """Append, rotate and attend as a rollout does: a chunk of frames, then
    single tokens, on branches that grow at different rates, captured once
    and replayed with other lengths, positions and page tables."""
    rng, gen = np.random.default_rng(8), torch.Generator().manual_seed(8)
    H, g, D, page, B, C, dims = 2, 2, 128, 32, 3, 300, (44, 42, 42)
    N = 24
    pages = m.PagedKV(H, D, page, 40, B, 8)
    plan, freqs = m.RopePlan(D, dims), O.ladder(dims)
    pK, pV = _randn(gen, H, C, D), _randn(gen, H, C, D)
    cnt, size = rng.integers(1, 9, (H, C)).astype(np.int32), np.array([C, C - 45], np.int32)
    px = m.Prefix(pK, pV, m=_cuda(cnt), size=_cuda(size))
    rows = torch.zeros(N, 4 * H, D, dtype=BF, device="cuda")
    pos = torch.zeros(N, 3, dtype=torch.int32, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    q_out = torch.zeros(H * g, N, D, dtype=BF, device="cuda")
    out, lse = torch.zeros_like(q_out), torch.zeros(H * g, N, device="cuda")
    ws = torch.empty(m.branch_workspace_size(H * g, H, N, D), dtype=torch.uint8, device="cuda")
    st = _status()

    def step():
        x = rows.transpose(0, 1)
        m.fastar_page_append(pages, x[2 * H:3 * H], x[3 * H:], cu, pos=pos, plan=plan, q=x[:2 * H], q_out=q_out,
                             status=st)
        m.fastar_branch_attention(q_out, cu, px, pages, D ** -0.5, out, lse=lse, block=8, ws=ws, status=st)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    K, V = _f64(pages.K), _f64(pages.V)
    table = np.zeros((B, 8), np.int32)
    free, length = list(rng.permutation(40)), np.zeros(B, np.int32)
    for i, new in enumerate(([8, 16, 0], [8, 0, 8], [1, 1, 1], [1, 1, 1], [0, 17, 7], [1, 0, 1])):
        length += np.array(new, np.int32)
        for b in range(B):
            for p in range(-(-int(length[b]) // page)):
                if table[b, p] == 0:
                    table[b, p] = free.pop()
        off = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        rows.copy_(torch.randn(*rows.shape, generator=gen))
        pos.copy_(torch.randint(0, 5000, pos.shape, generator=gen))
        cu.copy_(_cuda(off))
        pages.len.copy_(_cuda(length))
        pages.table.copy_(_cuda(table))
        torch.cuda.synchronize()
        if i % 2:
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert int(st) == 0
        x, p, n = _f64(rows).transpose(1, 0, 2), pos.cpu().numpy(), int(off[-1])
        tq, tk = (O.rope(y, p, dims, freqs, False) for y in (x[:2 * H], x[2 * H:3 * H]))
        O.page_append(K, V, tk, x[3 * H:], off, table, length)
        assert (np.abs(_f64(pages.K) - K) <= 2.0 ** -8 * np.abs(K) + 2.0 ** -17).all()
        # from here on the stored (rounded) keys and queries are the inputs
        K = _f64(pages.K)
        got_q = _f64(q_out)
        assert (np.abs(got_q - tq)[:, :n] <= 2.0 ** -8 * np.abs(tq[:, :n]) + 2.0 ** -17).all()
        ref, rl, A, X, keys = O.branch_attention(got_q, off, (_f64(pK), _f64(pV), cnt, size), K, V, table, length,
                                                 D ** -0.5, 8, bounds=True)
        d = (D + 4) * 2.0 ** -23 * X + 2.0 ** -20
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 3 * d + keys * 2.0 ** -22)[..., None] * A
        assert (np.abs(_f64(out) - ref)[:, :n] <= tol[:, :n]).all()


def test_two_calls_at_once_with_a_workspace_each(m):
    cases = [_attention_case(m, BF, 128, 3, 1, 64, [50, 1], [400, 90], 3000, True, 0, seed=s) for s in (11, 12)]
    streams = [torch.cuda.Stream() for _ in cases]
    want, got = [], []
    for q, cu, prefix, pages, *_ in cases:
        px = m.Prefix(prefix[0], prefix[1], m=_cuda(prefix[2]), size=_cuda(prefix[3]))
        out = torch.zeros_like(q)
        m.fastar_branch_attention(q, cu, px, pages, 0.1, out)
        want.append((q, cu, px, pages, out))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (q, cu, px, pages, _) in zip(streams, want):
            got.append(torch.zeros_like(q))
            s.wait_stream(torch.cuda.current_stream())
            m.fastar_branch_attention(q, cu, px, pages, 0.1, got[-1], stream=s)
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert torch.equal(out, want[i % 2][4])


def test_groups_wider_than_a_row_tile(m):
    """150 query heads share a key/value head: a token's heads lie in two tiles."""
    q, cu, prefix, pages, cu_h, length, table = _attention_case(m, BF, 64, 1, 150, 16, [3, 2], [20, 33], 70, True, 1,
                                                                seed=13)
    _check_attention(m, BF, q, cu, prefix, pages, 0.125, 1, cu_h, length, table)


@pytest.mark.parametrize("shape", [
    # D, H, g, page, new, past, C, counts, block, pad: the ways a call is laid out
    (128, 8, 1, 64, [520, 300], [100, 900], 20000, True, 260, 7),      # wide items, long runs
    (64, 4, 2, 128, [700], [64], 16000, False, 0, 0),                  # wide items, D 64
    (64, 1, 2, 64, [4500], [0], 0, False, 16, 0),                      # more than 64 row tiles: planned
    (128, 2, 1, 16, [1100] + [0] * 40 + [700], [0] * 42, 0, False, 1, 3),  # many row tiles, short items
    (64, 1, 1, 16, [9] * 700, [5] * 700, 33, True, 3, 0),              # many tiles and branches: planned
    (128, 40, 5, 32, [1] * 30, list(range(0, 300, 10)), 260, True, 0, 0),  # two row tiles, more items than CTAs / 2
    (64, 16, 5, 32, [1] * 128, list(range(0, 64)) * 2, 8000, True, 0, 3),  # many single tokens over a long prefix: wide
])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_branch_attention_layouts(m, shape, dtype):
    D, H, g, page, new, past, C, counts, block, pad = shape
    q, cu, prefix, pages, cu_h, length, table = _attention_case(m, dtype, D, H, g, page, new, past, C, counts, block,
                                                                pad, seed=21)
    _check_attention(m, dtype, q, cu, prefix, pages, D ** -0.5, block, cu_h, length, table)


def test_workspace_and_streams_may_be_left_to_the_call(m):
    q, cu, prefix, pages, cu_h, length, table = _attention_case(m, BF, 128, 2, 1, 64, [3, 1], [40, 9], 200, False, 0,
                                                                seed=14)
    px = m.Prefix(prefix[0], prefix[1])
    want = torch.zeros_like(q)
    m.fastar_branch_attention(q, cu, px, pages, 0.1, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = torch.zeros_like(q)
    m.fastar_branch_attention(q, cu, px, pages, 0.1, got, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    got.zero_()
    torch.cuda.synchronize()
    m.fastar_branch_attention(q, cu, px, pages, 0.1, got, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_branches_of_a_merged_cache(m):
    """A chunk is merged into the cache; two branches continue it and attend
    its live groups; a branch that is released starts again on freed pages."""
    from merged_attention_autoregressive_gb300.path import ChunkPath
    gen, rng = torch.Generator().manual_seed(30), np.random.default_rng(30)
    H, D, n_f = 3, 128, 96
    p = ChunkPath(H, D, n_f, 2, 16, 2, 6, 512, 0.95)
    p.planes.copy_(_randn(gen, *p.planes.shape))
    base = torch.randn(H, 1, n_f, D, generator=gen)
    k = (base + 0.05 * torch.randn(H, 2, n_f, D, generator=gen)).reshape(H, 2 * n_f, D).to(BF).cuda()
    p.merge(k, _randn(gen, H, 2 * n_f, D), 0)
    snap = p.cache.snapshot()
    assert int(p.cache.m.max()) > 1
    dims = (44, 42, 42)
    plan, freqs = m.RopePlan(D, dims), O.ladder(dims)
    roll = p.branches(2, 64, 100, page=16, n_pages=12, plan=plan, block=32, Hq=6)
    host = [np.zeros((2, H, 100, D)), np.zeros((2, H, 100, D))]
    lengths = [0, 0]
    for new in ([32, 32], [1, 0], [32, 20], [1, 1]):
        if new == [32, 20]:
            roll.release(1)
            lengths[1] = 0
        roll.extend(new)
        x = _randn(gen, 64, 4 * H, D).transpose(0, 1)
        pos = torch.randint(0, 9000, (64, 3), generator=gen, dtype=torch.int32).cuda()
        out, lse = roll.step(x[:2 * H], x[2 * H:3 * H], x[3 * H:], pos)
        assert int(roll.status) == 0
        off, ph = np.concatenate(([0], np.cumsum(new))), pos.cpu().numpy()
        K = np.zeros((2, H, 100, D))
        for b in range(2):
            lengths[b] += new[b]
            for i in range(lengths[b]):
                at = int(roll.pages.table[b, i // 16])
                K[b, :, i] = _f64(roll.pages.K[at, :, i % 16])
                host[1][b, :, i] = _f64(roll.pages.V[at, :, i % 16])
        turned = O.rope(_f64(x[2 * H:3 * H]), ph, dims, freqs, False)
        for b in range(2):
            own = turned[:, off[b]:off[b + 1]]
            stored = K[b, :, lengths[b] - new[b]:lengths[b]]
            assert (np.abs(stored - own) <= 2.0 ** -8 * np.abs(own) + 2.0 ** -17).all()
            # what was there before is still there
            assert (K[b, :, :lengths[b] - new[b]] == host[0][b, :, :lengths[b] - new[b]]).all()
        host[0] = K
        table, pages = np.arange(2)[:, None], (K, host[1])
        ref, rl, A, X, keys = O.branch_attention(
            _f64(roll.q), off, (_f64(p.cache.K), _f64(p.cache.V), p.cache.m.cpu().numpy(), p.cache.size.cpu().numpy()),
            pages[0], pages[1], table, np.array(lengths), roll.scale, 32, bounds=True)
        n = off[-1]
        d = (D + 4) * 2.0 ** -23 * X + 2.0 ** -20
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 3 * d + keys * 2.0 ** -22)[..., None] * A
        assert (np.abs(_f64(out) - ref)[:, :n] <= tol[:, :n]).all()
        assert (np.abs(_f64(lse) - rl)[:, :n] <= (d + keys * 2.0 ** -23 + 2.0 ** -22 * np.abs(rl))[:, :n]).all()
    for name, t in snap.items():  # the history is read only
        assert torch.equal(t.view(torch.uint8), getattr(p.cache, name).view(torch.uint8))
    with pytest.raises(ValueError):
        roll.extend([64, 0])      # longer than max_len
    with pytest.raises(ValueError):
        roll.extend([33, 32])     # more than `tokens`
