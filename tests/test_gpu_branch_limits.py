"""The branched-rollout calls at the ends of what they accept: lengths near
2^31, a status word that is set already, bad page ids beside good ones."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def m():
    import merged_attention_autoregressive_gb300 as m
    return m


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("branches,new", [(1, 1), (5, 1), (1, 130)])  # without a plan, with one, several row tiles
def test_a_branch_of_almost_2_31_positions(m, dtype, branches, new):
    """max_pages * page = 2^31 - 64 positions: one page stands in all places of
    the table but the first, so softmax and log-sum-exp have a closed form.

    Bounds.  A run has n units of TN keys.  Its sums take n terms, each
    rounded by at most 2^-24 of the sum, and its products with the values 8
    steps a unit on the tensor cores (each off by at most 2^-23 of the sum) or
    64 multiply-adds a unit (2^-24 each); scores and weights as in the tests
    of ordinary lengths.  All values are positive, so that the sum of p |v| is
    the result itself."""
    D, page, last = 64, 64, 2 ** 25 - 1
    gen = torch.Generator().manual_seed(branches + new)
    K = torch.randn(2, 1, page, D, generator=gen).to(dtype).cuda()
    V = (1 + torch.rand(2, 1, page, D, generator=gen)).to(dtype).cuda()
    V[0] *= 50
    table = torch.zeros(branches, last, dtype=I32, device="cuda")
    table[0, 1:] = 1
    length = torch.full((branches,), 64, dtype=I32, device="cuda")
    length[0] = last * page
    N = new + branches - 1
    cu = torch.tensor([0] + list(range(new, N + 1)), dtype=I32, device="cuda")
    q = torch.randn(1, N, D, generator=gen).to(dtype).cuda()
    out, lse = torch.zeros_like(q), torch.zeros(1, N, device="cuda")
    st = torch.zeros(1, dtype=I32, device="cuda")
    m.fastar_branch_attention(q, cu, None, m.PagedKV.view(K, V, table, length), D ** -0.5, out, lse=lse, status=st)
    assert int(st) == 0
    scale = D ** -0.5
    x = scale * (q[0].double() @ K[:, 0].double().flatten(0, 1).T)        # [N][128]: first page, repeated page
    copies = torch.ones(N, 2 * page, dtype=torch.float64, device="cuda")
    copies[:new, page:] = last - 1
    copies[new:, page:] = 0                                               # the other branches: the first page alone
    top = x.amax(1, keepdim=True)
    w = copies * (x - top).exp()
    total = w.sum(1, keepdim=True)
    ref, rl = (w @ V[:, 0].double().flatten(0, 1)) / total, (top + total.log())[:, 0]
    X = float((scale * (q[0].double().abs() @ K[:, 0].double().abs().flatten(0, 1).T)).max())
    d = (D + 4) * 2.0 ** -23 * X + 2.0 ** -20
    tiles = -(-N // (128 if dtype == BF else 64))
    runs, TN = (152, 128) if dtype == BF else (304, 64)
    n = tiles * (last * page // TN + branches) / runs + 1
    sums = (n + runs) * 2.0 ** -24
    products = n * 8 * 2.0 ** -23 if dtype == BF else n * 64 * 2.0 ** -24
    rounding = 2.0 ** -8 + 2.0 ** -8 if dtype == BF else 0.0              # the weights, the result
    assert bool(((lse[0].double() - rl).abs() <= d + sums * 1.01 + 2.0 ** -22 * rl.abs()).all())
    assert bool(((out[0].double() - ref).abs() <= (rounding + 3 * d + (sums + products) * 1.2) * ref).all())
    assert float(rl[:new].min()) > math.log(last) - X                     # a bound that a lost branch cannot meet


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_set_status_stops_a_planned_call_on_a_workspace_of_any_content(m, dtype):
    """The status word is set before the call, which has more row tiles than go
    without a plan: no list of the workspace is read that was not written."""
    H, N, D, page = 2, 9000, 64, 64
    pages = m.PagedKV(H, D, page, 150, 1, 150, dtype)
    pages.table.copy_(torch.arange(150, dtype=I32)[None])
    pages.len.fill_(N)
    q = torch.randn(H, N, D, device="cuda").to(dtype)
    cu = torch.tensor([0, N], dtype=I32, device="cuda")
    ws = torch.full((m.branch_workspace_size(H, H, N, D),), 0x7f, dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(q, 5.0), torch.full((H, N), 5.0, device="cuda")
    st = torch.full((1,), 18, dtype=I32, device="cuda")
    m.fastar_branch_attention(q, cu, None, pages, 0.1, out, lse=lse, block=1, ws=ws, status=st)
    torch.cuda.synchronize()
    assert int(st) == 18 and bool((out == 5.0).all()) and bool((lse == 5.0).all())
    st.zero_()  # the same call on the same workspace with a clear word
    m.fastar_branch_attention(q, cu, None, pages, 0.1, out, lse=lse, block=1, ws=ws, status=st)
    assert int(st) == 0 and bool((out[:, :, 0] != 5.0).any()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("bad", [-1, 2 ** 31 - 1])
def test_append_skips_the_tokens_of_a_bad_page_and_no_others(m, dtype, D, where, bad):
    """Several waves of CTAs: the ones that start after the status word was set
    by a token of the same call go on."""
    H, Hq, page, per, B = 12, 3, 64, 5000, 8
    most = -(-per // page)
    gen = torch.Generator(device="cuda").manual_seed(D)
    rows = torch.randn(B * per, Hq + 2 * H, D, generator=gen, device="cuda").to(dtype).transpose(0, 1)
    q, k, v = rows[:Hq], rows[Hq:Hq + H], rows[Hq + H:]
    cu = torch.arange(0, B * per + 1, per, dtype=I32, device="cuda")
    table = torch.arange(B * most, dtype=I32, device="cuda").view(B, most)
    at = {"first": (0, 0), "middle": (3, most // 2), "last": (B - 1, most - 1)}[where]
    pos = torch.arange(B * per, dtype=I32, device="cuda")[:, None]
    plan = m.RopePlan(D, (D,))

    def append(t):
        pages = m.PagedKV(H, D, page, B * most, B, most, dtype)
        pages.K.fill_(7.0), pages.V.fill_(7.0)
        pages.table.copy_(t)
        pages.len.fill_(per)
        q_out, st = torch.full((Hq, B * per, D), 7.0, dtype=dtype, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
        m.fastar_page_append(pages, k, v, cu, pos=pos, plan=plan, q=q, q_out=q_out, status=st)
        return pages.K, pages.V, q_out, int(st)

    K, V, q_out, st = append(table)
    assert st == 0
    mine = int(table[at])                            # nobody else has that page
    first = at[0] * per + at[1] * page
    K[mine] = V[mine] = 7.0
    q_out[:, first:min(first + page, (at[0] + 1) * per)] = 7.0
    spoiled = table.clone()
    spoiled[at] = bad
    for _ in range(5):
        got = append(spoiled)
        assert got[3] == 18
        assert torch.equal(got[0], K) and torch.equal(got[1], V) and torch.equal(got[2], q_out)


def test_append_writes_nothing_where_the_status_was_set_before(m):
    pages = m.PagedKV(2, 64, 16, 8, 2, 4)
    pages.table.copy_(torch.arange(8, dtype=I32).view(2, 4))
    pages.len.fill_(20)
    k, cu = torch.ones(2, 40, 64, dtype=BF, device="cuda"), torch.tensor([0, 20, 40], dtype=I32, device="cuda")
    for word in (16, 17, 18):
        st = torch.full((1,), word, dtype=I32, device="cuda")
        m.fastar_page_append(pages, k, k, cu, status=st)
        assert int(st) == word and not bool(pages.K.any()) and not bool(pages.V.any())
    for word in (16, 17):  # with a bad page of its own, too
        pages.table[1, 0] = -1
        st = torch.full((1,), word, dtype=I32, device="cuda")
        m.fastar_page_append(pages, k, k, cu, status=st)
        assert int(st) == word and not bool(pages.K.any())
    pages.table[1, 0] = 4
    m.fastar_page_append(pages, k, k, cu)
    assert bool((pages.K[:, :, 0] == 1).any())


def test_append_refuses_every_position_of_a_negative_length(m):
    """A table of 2^31 - 64 positions: len - n must not come round to its end."""
    page, most, n = 64, 2 ** 25 - 1, 100
    pages = m.PagedKV(1, 64, page, 2, 2, 1)
    pages.table = torch.zeros(2, most, dtype=I32, device="cuda")
    pages.table[1, 0] = 1
    k, cu = torch.ones(1, n + 1, 64, dtype=BF, device="cuda"), torch.tensor([0, n, n + 1], dtype=I32, device="cuda")
    for length in (-2 ** 31, -2 ** 31 + 60, -1):
        pages.len.copy_(torch.tensor([length, 1], dtype=I32))
        pages.K.zero_()
        st = torch.zeros(1, dtype=I32, device="cuda")
        m.fastar_page_append(pages, k, k, cu, status=st)
        assert int(st) == 18 and not bool(pages.K[0].any())
        assert bool((pages.K[1, 0, 0] == 1).all())   # the other branch's token


@pytest.mark.parametrize("kind", ["none", "stream", "handle"])
def test_a_workspace_of_the_call_belongs_to_its_stream(m, monkeypatch, kind):
    """A block of the current stream's pool may still be in use there by a
    tensor that has been freed, so the allocation is made on the call's stream."""
    side = torch.cuda.Stream()
    pages = m.PagedKV(1, 64, 16, 2, 1, 2)
    pages.len.fill_(20)
    q, cu = torch.ones(1, 20, 64, dtype=BF, device="cuda"), torch.tensor([0, 20], dtype=I32, device="cuda")
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    made, empty = [], torch.empty

    def spy(*a, **kw):
        made.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", spy)
    stream = {"none": None, "stream": side, "handle": side.cuda_stream}[kind]
    before = torch.cuda.current_stream()
    m.fastar_branch_attention(q, cu, None, pages, 0.1, out, stream=stream)
    assert made == [before.cuda_stream if stream is None else side.cuda_stream]
    assert torch.cuda.current_stream() == before


def test_a_rollout_may_be_used_on_another_stream_at_once(m):
    """The buffers of a rollout are filled on the stream that is current when it
    is made; a step on another stream does not run ahead of that."""
    from merged_attention_autoregressive_gb300.path import BranchRollout
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(2, 20, 64, generator=gen).to(BF).cuda() for _ in range(3))
    side = torch.cuda.Stream()
    got = []
    for stream in (None, side):
        torch.cuda.synchronize()
        torch.cuda._sleep(400_000_000)  # the current stream is busy for a fraction of a second
        r = BranchRollout(2, 2, 64, 20, 32, page=16, block=1)
        r.extend([13, 7], stream=stream)
        out, lse = r.step(q, k, v, stream=stream)
        torch.cuda.synchronize()
        assert r.cu.tolist() == [0, 13, 20] and r.pages.len.tolist() == [13, 7] and int(r.status) == 0
        got.append((out.clone(), lse.clone(), r.pages.K.clone()))
    assert bool(got[0][0].any()) and all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("inverse", [False, True])
def test_rotation_in_32_bits_keeps_the_bits_of_the_angle(m, inverse):
    """Rows (1, 0) turn into cosines and sines.  From the nearest quarter turn the
    rest of the angle is at most 1/4 half turn, 2^-27 of a half turn off as a
    32-bit number (pi 2^-27 in the angle) and 2^-31 by the fixed-point product's
    lower half, which is dropped; sine and cosine of it are within one unit in the
    last place."""
    import numpy as np
    D, N = 64, 30000
    plan = m.RopePlan(D, (D,), base=500.0)
    gen = torch.Generator().manual_seed(3)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (N, 1), generator=gen, dtype=torch.int64)
    pos[:200, 0] = torch.arange(-100, 100)
    x = torch.zeros(1, N, D, device="cuda")
    x[..., 0::2] = 1.0
    y = torch.empty_like(x)
    m.fastar_rope(x, pos.to(torch.int32).cuda(), plan, y, inverse=inverse)
    turn = np.array(list(plan.struct.turn)[:D // 2], dtype=np.uint64)
    with np.errstate(over="ignore"):
        frac = pos.numpy().astype(np.int64).view(np.uint64) * turn[None]             # of a turn, modulo 1
    quarter = (frac + np.uint64(1 << 61)) >> np.uint64(62)
    rest = (frac - (quarter << np.uint64(62))).view(np.int64) * (2.0 * np.pi / 2.0 ** 64)
    s, c = np.sin(rest), np.cos(rest)
    k = quarter.astype(np.int64)
    sin = np.choose(k, (s, c, -s, -c)) * (-1.0 if inverse else 1.0)
    cos = np.choose(k, (c, -s, -c, s))
    got = y[0].double().cpu().numpy()
    for ref, g in ((cos, got[:, 0::2]), (sin, got[:, 1::2])):
        tol = np.spacing(np.abs(ref).astype(np.float32)).astype(np.float64) + np.pi * 2.0 ** -27 + np.pi * 2.0 ** -31
        err = np.abs(g - ref)
        assert (err <= tol).all(), f"worst {(err / tol).max():.3g} of the bound"


@pytest.mark.parametrize("dtype,D,dims,pairing", [(BF, 128, (44, 42, 42), "adjacent"), (F32, 64, (32, 16), "halves")])
def test_rotation_there_and_back(m, dtype, D, dims, pairing):
    """The inverse undoes the rotation: each way products and sum round in 32
    bits (2^-20 of |x0| + |x1| with the angle's error) and once to the type."""
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(5, 300, D, generator=gen).to(dtype).cuda()
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (300, len(dims)), generator=gen, dtype=torch.int64).to(torch.int32).cuda()
    plan, y = m.RopePlan(D, dims, pairing=pairing), x.clone()
    m.fastar_rope(y, pos, plan, y)
    assert not torch.equal(y, x)
    m.fastar_rope(y, pos, plan, y, inverse=True)
    turned = sum(dims)
    z, back = x[..., :turned].double(), y[..., :turned].double()
    if pairing == "halves":
        size = z.abs().unflatten(-1, (2, -1)).sum(-2).repeat(1, 1, 2)
    else:
        size = z.abs().unflatten(-1, (-1, 2)).sum(-1, keepdim=True).expand(-1, -1, -1, 2).flatten(-2)
    half = torch.finfo(dtype).eps / 2
    # a pair's turned values are at most |x0| + |x1| each, and come back through a sine and a cosine
    tol = 2 * 1.01 * (2.0 ** -20 + half) * size + half * z.abs() * 1.01
    assert bool(((back - z).abs() <= tol).all())
    assert torch.equal(y[..., turned:], x[..., turned:])


def test_branches_of_a_layer_attend_with_its_scale(m):
    from merged_attention_autoregressive_gb300.path import ChunkPath
    p = ChunkPath(2, 64, 32, 1, 8, 2, 4, 64, 0.9)
    assert p.branches(1, 8, 32).scale == 0.125
    p.scale = 0.3
    assert p.branches(1, 8, 32).scale == 0.3 and p.branches(1, 8, 32, scale=0.2).scale == 0.2


@pytest.mark.parametrize("at", [0, 31, 32, 299, 777])
def test_append_of_many_branches_skips_the_one_of_a_bad_page(m, at):
    """A token each, and one branch with a prompt of several pages in front of them."""
    B, H, D, page, prompt = 778, 24, 128, 16, 2000
    new = [prompt] + [1] * (B - 1)
    gen = torch.Generator(device="cuda").manual_seed(at)
    N = sum(new)
    rows = torch.randn(N, 2 * H, D, generator=gen, device="cuda").to(BF).transpose(0, 1)
    cu = torch.tensor([0] + [prompt + i for i in range(B)], dtype=I32, device="cuda")
    table = torch.zeros(B, prompt // page, dtype=I32, device="cuda")
    table[0] = torch.arange(prompt // page)
    table[1:, 0] = prompt // page + torch.arange(B - 1)
    spoiled = table.clone()
    spoiled[at, 70 if at == 0 else 0] = -5
    got = []
    for t in (table, spoiled, spoiled):
        pages = m.PagedKV(H, D, page, prompt // page + B, B, prompt // page)
        pages.table.copy_(t)
        pages.len.copy_(torch.tensor(new, dtype=I32))
        st = torch.zeros(1, dtype=I32, device="cuda")
        m.fastar_page_append(pages, rows[:H], rows[H:], cu, status=st)
        got.append((pages.K, pages.V, int(st)))
    assert [g[2] for g in got] == [0, 18, 18]
    mine = int(table[at, 70 if at == 0 else 0])
    for i in (0, 1):
        assert bool(got[0][i][mine].any())
        got[0][i][mine] = 0.0
        assert torch.equal(got[1][i], got[0][i]) and torch.equal(got[2][i], got[0][i])
