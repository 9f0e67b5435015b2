"""Refusals of the branched-rollout calls: host checks only, nothing is
launched, so these run without a GPU."""
import ctypes
import math
import types

import pytest
import torch

VP = ctypes.c_void_p
FAKE, ODD = VP(0x1000), VP(0x1008)  # never dereferenced: the checks come first
OK, ARG, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4


@pytest.fixture(scope="module")
def m():
    import merged_attention_autoregressive_gb300 as m
    from merged_attention_autoregressive_gb300 import build
    build.build()
    m.lib()
    return m


def _plan(m, D=128, dims=(44, 42, 42), pairing=0, freq=None):
    s = m.RopePlanStruct()
    f = None if freq is None else (ctypes.c_double * len(freq))(*freq)
    rc = m.lib().fastar_rope_plan_init(ctypes.addressof(s), D, len(dims), (ctypes.c_int * len(dims))(*dims), pairing, f)
    return rc, s


def test_plan_holds_the_fractions_of_a_turn(m):
    rc, s = _plan(m)
    assert rc == OK and (s.D, s.axes, s.pairs, s.pairing) == (128, 3, 64, 0)
    assert list(s.axis[:64]) == [0] * 22 + [1] * 21 + [2] * 21
    for p, (i, d) in enumerate([(i, d) for d in (44, 42, 42) for i in range(d // 2)]):
        turns = 10000.0 ** (-2.0 * i / d) / (2 * math.pi)
        assert abs(s.turn[p] / 2.0 ** 64 - turns) < 1e-15
    # negative and whole turns wrap
    rc, s = _plan(m, 64, (4,), 0, [-1e-30, 4 * math.pi])
    assert rc == OK and s.turn[0] in (0, 2 ** 64 - 1) and min(s.turn[1], 2 ** 64 - s.turn[1]) < 2 ** 14
    assert m.RopePlan(64, (64,), base=500.0, pairing="halves").struct.pairs == 32


@pytest.mark.parametrize("kw,rc", [
    (dict(D=96, dims=(96,)), UNSUPPORTED), (dict(dims=(44, 42, 44)), ARG), (dict(dims=(43, 42)), ARG),
    (dict(dims=(0, 0)), ARG), (dict(dims=(-2, 4)), ARG), (dict(dims=(2,) * 5), ARG), (dict(pairing=2), ARG),
    (dict(dims=(24,), pairing=1), ARG), (dict(dims=(4,), freq=[1.0, math.inf]), ARG),
    (dict(dims=(4,), freq=[1.0, math.nan]), ARG), (dict(dims=(2 ** 31 - 2, 2 ** 31 - 2)), ARG)])
def test_plan_refusals(m, kw, rc):
    assert _plan(m, **kw)[0] == rc


def test_plan_binding_refusals(m):
    with pytest.raises(ValueError):
        m.RopePlan(128, (64,), pairing="pairs")
    with pytest.raises(ValueError):
        m.RopePlan(128, (64,), freqs=[1.0])
    with pytest.raises(m.FastarError):
        m.RopePlan(128, (256,))


def _rope(m, dt=0, x=FAKE, xh=1280, xt=128, H=2, N=10, D=128, pos=FAKE, plan=0, out=FAKE, oh=1280, ot=128):
    keep = _plan(m)[1]
    p = ctypes.addressof(keep) if plan == 0 else plan
    return m.lib().fastar_rope(dt, x, xh, xt, H, N, D, pos, p, 0, out, oh, ot, None, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=2), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(D=64), ARG), (dict(plan=None), ARG), (dict(H=-1), ARG),
    (dict(N=-1), ARG), (dict(x=None), ARG), (dict(out=None), ARG), (dict(pos=None), ARG), (dict(x=ODD), ARG),
    (dict(out=ODD), ARG), (dict(xt=132), ARG), (dict(dt=1, xt=130), ARG), (dict(oh=0), ARG), (dict(ot=64), ARG),
    (dict(H=0, x=None), OK), (dict(N=0, out=None), OK)])
def test_rope_refusals(m, kw, rc):
    assert _rope(m, **kw) == rc


def test_rope_refuses_a_spoiled_plan(m):
    for field, value in (("axes", 0), ("axes", 5), ("pairs", 0), ("pairs", 65), ("pairing", 3), ("D", 64)):
        s = _plan(m)[1]
        setattr(s, field, value)
        assert _rope(m, plan=ctypes.addressof(s)) == ARG
    s = _plan(m)[1]
    s.axis[5] = 3
    assert _rope(m, plan=ctypes.addressof(s)) == ARG


def _pages(m, H=2, D=128, page=64, n_pages=8, B=3, max_pages=4, dt=0, K=FAKE, V=FAKE, table=FAKE, length=FAKE):
    return m.PagesStruct(H, D, page, n_pages, B, max_pages, dt, K, V, table, length)


BAD_PAGES = [(dict(D=96), UNSUPPORTED), (dict(dt=3), UNSUPPORTED), (dict(page=8), UNSUPPORTED),
             (dict(page=48), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(H=0), ARG), (dict(B=-1), ARG),
             (dict(n_pages=-1), ARG), (dict(max_pages=-1), ARG), (dict(K=None), ARG), (dict(V=ODD), ARG),
             (dict(table=None), ARG), (dict(length=None), ARG), (dict(n_pages=0), ARG),
             (dict(n_pages=2 ** 24, page=256), UNSUPPORTED), (dict(max_pages=2 ** 25), UNSUPPORTED)]


def _append(m, pages, k=FAKE, v=FAKE, N=10, cu=FAKE, pos=FAKE, plan=0, q=None, Hq=0, q_out=None, tok=256):
    keep = _plan(m)[1]
    p = ctypes.addressof(keep) if plan == 0 else plan
    return m.lib().fastar_page_append(ctypes.addressof(pages) if pages is not None else None, k, 128, tok, v, 128,
                                      tok, N, cu, pos, p, q, 128, tok, Hq, q_out, None, None)


@pytest.mark.parametrize("kw,rc", BAD_PAGES)
def test_append_refuses_bad_pages(m, kw, rc):
    assert _append(m, _pages(m, **kw)) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(k=None), ARG), (dict(v=ODD), ARG), (dict(cu=None), ARG), (dict(N=-1), ARG), (dict(pos=None), ARG),
    (dict(plan=None), ARG), (dict(tok=130), ARG), (dict(q=FAKE), ARG), (dict(q=FAKE, Hq=2), ARG),
    (dict(Hq=2), ARG), (dict(q=ODD, Hq=2, q_out=FAKE), ARG), (dict(q=FAKE, Hq=2, q_out=ODD), ARG),
    (dict(Hq=-1), ARG), (dict(N=0, k=None), OK)])
def test_append_refusals(m, kw, rc):
    assert _append(m, _pages(m), **kw) == rc
    assert _append(m, None) == ARG
    assert _append(m, _pages(m, B=0, table=None, length=None)) == OK


def _attend(m, pages, prefix=None, dt=0, q=FAKE, Hq=4, N=10, cu=FAKE, scale=0.1, block=0, out=FAKE, ws=VP(0x10000),
            nbytes=1 << 40):
    return m.lib().fastar_branch_attention(dt, q, Hq, N, cu, None if prefix is None else ctypes.addressof(prefix),
                                           ctypes.addressof(pages) if pages is not None else None, scale, block, out,
                                           None, ws, nbytes, None, None)


def _prefix(m, H=2, C=100, D=128, dt=0, K=FAKE, V=FAKE):
    return m.PrefixStruct(H, C, D, dt, K, V, None, None)


@pytest.mark.parametrize("kw,rc", BAD_PAGES)
def test_attention_refuses_bad_pages(m, kw, rc):
    dt = kw.get("dt", 0)
    assert _attend(m, _pages(m, **kw), dt=dt) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), ARG), (dict(out=ODD), ARG), (dict(cu=None), ARG), (dict(N=-1), ARG), (dict(Hq=3), ARG),
    (dict(Hq=-2), ARG), (dict(dt=1), ARG), (dict(block=-1), ARG), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG),
    (dict(scale=math.inf), ARG), (dict(scale=math.nan), ARG), (dict(ws=None), WORKSPACE), (dict(nbytes=16), WORKSPACE),
    (dict(ws=VP(0x10010)), WORKSPACE), (dict(N=2 ** 30, Hq=4), UNSUPPORTED), (dict(N=0, q=None), OK),
    (dict(Hq=0, q=None), OK)])
def test_attention_refusals(m, kw, rc):
    assert _attend(m, _pages(m), **kw) == rc
    assert _attend(m, None) == ARG


@pytest.mark.parametrize("kw,rc", [
    (dict(H=4), ARG), (dict(D=64), ARG), (dict(dt=1), ARG), (dict(C=-1), ARG), (dict(K=None), ARG), (dict(V=ODD), ARG),
    (dict(C=2 ** 30), UNSUPPORTED)])
def test_attention_refuses_bad_prefixes(m, kw, rc):
    assert _attend(m, _pages(m), prefix=_prefix(m, **kw)) == rc


def test_workspace_size(m):
    size = m.branch_workspace_size
    assert size(4, 3, 10, 128) == 0 and size(0, 1, 10, 128) == 0 and size(4, 2, 0, 128) == 0
    need = size(4, 2, 10, 128)
    assert need % 256 == 0 and _attend(m, _pages(m), nbytes=need - 1) == WORKSPACE
    # bounded: the split of a long cache does not grow with the tokens
    assert size(40, 40, 100000, 128) < (64 << 20) and size(12, 12, 1, 128) < (1 << 20)


def test_binding_refuses_host_tensors_and_other_shapes(m):
    import torch
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    plan = m.RopePlan(64, (64,))
    with pytest.raises(ValueError):
        m.fastar_rope(z(2, 3, 64), z(3, 1, dt=torch.int32), plan, z(2, 3, 64))     # not on the GPU
    with pytest.raises(ValueError):
        m.fastar_rope(z(2, 3, 64), z(3, 1, dt=torch.int32), plan, z(2, 4, 64))
    with pytest.raises(ValueError):
        m.PagedKV.view(z(4, 2, 16, 64), z(4, 2, 16, 64), z(2, 2, dt=torch.int32), z(2, dt=torch.int64))
    with pytest.raises(ValueError):
        m.Prefix(z(2, 3, 64), z(2, 4, 64))


def test_rollout_hands_out_pages():
    from merged_attention_autoregressive_gb300.path import BranchRollout
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.int32)
    r = BranchRollout.__new__(BranchRollout)  # the host's part of one
    r.B, r.tokens, r.max_len, r.lengths, r.held, r.free = 3, 100, 96, [0] * 3, [[], [], []], [4, 3, 2, 1, 0]
    r.pages = types.SimpleNamespace(page=32, max_pages=3, n_pages=5, table=zeros(3, 3), len=zeros(3))
    r.cu = zeros(4)

    def check():
        used = [p for h in r.held for p in h]
        assert sorted(used + r.free) == list(range(5))  # no page twice, none lost
        assert r.pages.len.tolist() == r.lengths
        for b, h in enumerate(r.held):
            assert len(h) == -(-r.lengths[b] // 32)
            assert r.pages.table[b, :len(h)].tolist() == h

    r.extend([1, 0, 40])
    assert r.cu.tolist() == [0, 1, 1, 41]
    check()
    r.extend([31, 1, 0])  # the first branch's page is full now
    assert r.cu.tolist() == [0, 31, 32, 32]
    check()
    held = [list(h) for h in r.held]
    for new, why in [([64, 0, 25], "no pages"), ([65, 0, 0], "longer"), ([0, 0, 101], "at most"), ([0, -1, 0], "count"),
                     ([1, 1], "per branch")]:
        with pytest.raises(ValueError, match=why):
            r.extend(new)
        assert r.held == held and r.lengths == [32, 1, 40]  # as it was
    r.release(2)
    assert len(r.free) == 3 and r.lengths == [32, 1, 0]
    r.extend([64, 0, 1])
    check()
