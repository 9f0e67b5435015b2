"""Refusals of the calls for drafts and bounded pages, and the host's part of a
rollout that drafts: nothing is launched, so these run without a GPU."""
import ctypes
import math
import types

import numpy as np
import pytest
import torch

from oracle import draft_oracle as O

VP = ctypes.c_void_p
FAKE, ODD = VP(0x1000), VP(0x1008)  # never dereferenced: the checks come first
OTHER = VP(0x2000)
OK, ARG, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4


@pytest.fixture(scope="module")
def m():
    import merged_attention_autoregressive_gb300 as m
    from merged_attention_autoregressive_gb300 import build
    build.build()
    m.lib()
    return m


def _pages(m, H=2, D=128, page=64, n_pages=8, B=3, max_pages=4, dt=0, K=FAKE, V=FAKE, table=FAKE, length=FAKE):
    return m.PagesStruct(H, D, page, n_pages, B, max_pages, dt, K, V, table, length)


def _at(x):
    return None if x is None else ctypes.addressof(x)


BAD_PAGES = [(dict(D=96), UNSUPPORTED), (dict(dt=3), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(H=0), ARG),
             (dict(B=-1), ARG), (dict(K=None), ARG), (dict(V=ODD), ARG), (dict(table=None), ARG),
             (dict(length=None), ARG), (dict(max_pages=2 ** 25), UNSUPPORTED)]


def _tree(m, pages, dt=0, q=FAKE, Hq=4, N=10, cu=FAKE, parent=FAKE, prefix=None, scale=0.1, out=FAKE, ws=FAKE, size=1 << 40):
    return m.lib().fastar_tree_attention(dt, q, Hq, N, cu, parent, _at(prefix), _at(pages), scale, out, None, ws, size,
                                         None, None)


def _keep(m, pages, cu=FAKE, rows=FAKE, M=5, ck=FAKE):
    return m.lib().fastar_page_keep(_at(pages), cu, rows, M, ck, None, None)


def _mass(m, pages, q=FAKE, lse=FAKE, Hq=4, N=10, rows=None, M=10, cu=FAKE, scale=0.1, block=0, decay=1.0,
          mass=(FAKE, FAKE, FAKE), ws=FAKE, size=1 << 40):
    x = None if mass is None else m.MassStruct(*mass)
    return m.lib().fastar_page_mass(_at(pages), q, lse, Hq, N, rows, M, cu, scale, block, decay, _at(x), ws, size, None,
                                    None)


def _evict(m, pages, mass=(FAKE, FAKE, FAKE), budget=10, first=1, recent=2, out=None):
    x = None if mass is None else m.MassStruct(*mass)
    y = None if out is None else m.MassStruct(*out)
    return m.lib().fastar_page_evict(_at(pages), _at(x), budget, first, recent, _at(y), None, None)


@pytest.mark.parametrize("kw,rc", BAD_PAGES)
def test_bad_pages(m, kw, rc):
    for call in (_tree, _keep, _mass, _evict):
        assert call(m, _pages(m, **kw)) == rc
        assert call(m, None) == ARG


def test_nothing_to_do(m):
    none = _pages(m, B=0, table=None, length=None)
    for call in (_tree, _keep, _mass, _evict):
        assert call(m, none) == OK
    assert _tree(m, _pages(m), N=0, q=None, parent=None) == OK
    assert _keep(m, _pages(m), M=0, rows=None) == OK
    assert _mass(m, _pages(m), M=0, N=0, q=None) == OK
    assert _mass(m, _pages(m), M=0, N=10, rows=None) == OK  # (an empty tensor of rows is NULL)
    assert _evict(m, _pages(m, max_pages=0, table=None)) == OK


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=1), ARG), (dict(q=None), ARG), (dict(q=ODD), ARG), (dict(out=None), ARG), (dict(out=ODD), ARG),
    (dict(cu=None), ARG), (dict(parent=None), ARG), (dict(Hq=3), ARG), (dict(N=-1), ARG), (dict(scale=0.0), ARG),
    (dict(scale=math.inf), ARG), (dict(scale=math.nan), ARG), (dict(ws=None), WORKSPACE), (dict(size=100), WORKSPACE),
    (dict(ws=VP(0x1010)), WORKSPACE), (dict(N=2 ** 30), UNSUPPORTED)])
def test_tree_refusals(m, kw, rc):
    assert _tree(m, _pages(m), **kw) == rc


def test_tree_refuses_a_prefix_of_another_shape(m):
    for kw in (dict(H=3), dict(D=64), dict(dt=1), dict(K=None)):
        p = dict(H=2, C=5, D=128, dt=0, K=FAKE, V=FAKE, m=None, size=None)
        p.update(kw)
        assert _tree(m, _pages(m), prefix=m.PrefixStruct(*p.values())) == ARG


@pytest.mark.parametrize("kw,rc", [(dict(cu=None), ARG), (dict(rows=None), ARG), (dict(ck=None), ARG), (dict(M=-1), ARG)])
def test_keep_refusals(m, kw, rc):
    assert _keep(m, _pages(m), **kw) == rc
    assert _keep(m, _pages(m, B=65536)) == UNSUPPORTED


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), ARG), (dict(q=ODD), ARG), (dict(lse=None), ARG), (dict(cu=None), ARG), (dict(Hq=3), ARG),
    (dict(N=9), ARG), (dict(N=-1, M=-1), ARG), (dict(M=-1, rows=FAKE), ARG), (dict(scale=-1.0), ARG),
    (dict(scale=math.nan), ARG), (dict(block=-1), ARG), (dict(decay=-0.5), ARG), (dict(decay=math.nan), ARG),
    (dict(decay=math.inf), ARG), (dict(mass=None), ARG), (dict(mass=(None, None, None)), ARG),
    (dict(mass=(ODD, None, None)), ARG), (dict(mass=(FAKE, FAKE, None)), ARG), (dict(mass=(FAKE, None, FAKE)), ARG),
    (dict(ws=None), WORKSPACE), (dict(size=64), WORKSPACE), (dict(M=2 ** 30, rows=FAKE), UNSUPPORTED)])
def test_mass_refusals(m, kw, rc):
    assert _mass(m, _pages(m), **kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(mass=None), ARG), (dict(mass=(None, None, None)), ARG), (dict(mass=(FAKE, FAKE, None)), ARG),
    (dict(budget=-1, first=0, recent=0), ARG), (dict(first=-1), ARG), (dict(recent=-1), ARG), (dict(budget=2), ARG),
    (dict(budget=2 ** 31 - 1, first=2 ** 31 - 1, recent=1), ARG), (dict(out=(None, OTHER, FAKE)), ARG),
    (dict(out=(OTHER, None, None)), ARG), (dict(out=(FAKE, OTHER, FAKE)), ARG), (dict(out=(OTHER, FAKE, FAKE)), ARG),
    (dict(out=(ODD, OTHER, FAKE)), ARG), (dict(mass=(FAKE, None, None), out=(OTHER, OTHER, FAKE)), ARG)])
def test_evict_refusals(m, kw, rc):
    assert _evict(m, _pages(m), **kw) == rc


def test_evict_refuses_tables_with_more_room_than_its_words(m):
    assert _evict(m, _pages(m, page=256, max_pages=2049)) == UNSUPPORTED


def test_workspace_of_the_masses(m):
    assert m.mass_workspace_size(4, 2, 10, 128) > 0
    assert m.mass_workspace_size(4, 3, 10, 128) == 0 and m.mass_workspace_size(4, 2, 0, 128) == 0


def test_masses_need_their_pages_shapes(m, monkeypatch):
    monkeypatch.setattr(m, "_gpu", lambda t: t.get_device())
    z = torch.zeros
    K = z(4, 2, 16, 64, dtype=torch.bfloat16)
    pages = m.PagedKV.view(K, K.clone(), z(2, 3, dtype=torch.int32), z(2, dtype=torch.int32))
    mass, born, total = z(4, 2, 16), z(4, 2, 16, dtype=torch.int32), z(2, dtype=torch.int32)
    assert m.PageMass.view(mass, born, total)._fits(pages)
    for bad in ((mass.double(), born, total), (mass, born, None), (mass, None, total), (mass, born.long(), total),
                (mass, born[:3], total), (mass.view(8, 16), born, total)):
        with pytest.raises(ValueError):
            m.PageMass.view(*bad)
    for other in (m.PageMass.view(z(4, 2, 32)), m.PageMass.view(mass, born, z(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            other._fits(pages)
    x = m.PageMass.view(mass)
    old = x.addr
    x.mass = z(4, 2, 16)  # another tensor: the struct follows it
    assert x.struct.mass == x.mass.data_ptr() and x.addr != old


def _rollout(m, monkeypatch, **kw):
    """The host's part of a rollout on host tensors; the calls are recorded."""
    from merged_attention_autoregressive_gb300 import path
    seen = []
    for name in ("fastar_page_keep", "fastar_page_mass", "fastar_page_evict"):
        monkeypatch.setattr(path, name, lambda *a, _n=name, **k: seen.append((_n, a, k)))
    import contextlib
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    r = path.BranchRollout.__new__(path.BranchRollout)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    r.B, r.tokens, r.max_len, r.lengths, r.totals = 3, 100, 96, [0] * 3, [0] * 3
    r.held, r.free = [[], [], []], [8, 7, 6, 5, 4, 3, 2, 1, 0]
    r.pages = types.SimpleNamespace(page=32, max_pages=3, n_pages=9, table=z(3, 3), len=z(3))
    r.cu, r.parent, r.status = z(4), z(100), z(1)
    r.scale, r.lse, r.ws_mass, r._asked = 0.1, None, None, "q"
    r.budget, r.first, r.recent, r.decay = kw.get("budget"), 0, 0, 1.0
    r.mass = types.SimpleNamespace(total=z(3)) if r.budget is not None else None
    return r, seen


def test_rollout_counts_drafts_and_accepted_paths(m, monkeypatch):
    r, seen = _rollout(m, monkeypatch, budget=40)
    r.extend([30, 0, 5])
    trees = [[-1, 0, 0, 1, 3], [-1, -1], [0 - 1]]
    r.extend([5, 2, 1], parents=trees)
    r._asked = None
    with pytest.raises(ValueError, match="attended"):
        r.accept([0, 0, 0])
    r._asked = "q"
    assert r.parent[:8].tolist() == [-1, 0, 0, 1, 3, -1, -1, -1] and r.lengths == [35, 2, 6] and len(r.held[0]) == 2
    for call in (lambda: r.extend([1, 1, 1]), lambda: r.release(0), r.evict):
        with pytest.raises(ValueError, match="accepted"):
            call()
    for leaves in ([5, 0, 0], [-2, 0, 0], [0, 0]):
        with pytest.raises(ValueError):
            r.accept(leaves)
    assert r.accept([4, -1, 0]) == [[0, 1, 3, 4], [], [7]]
    assert r.lengths == [34, 0, 6] == r.pages.len.tolist() and r.totals == [34, 0, 6] == r.mass.total.tolist()
    assert [n for n, _, _ in seen] == ["fastar_page_keep", "fastar_page_mass"]
    assert seen[0][1][2].tolist() == [0, 1, 3, 4, 7] and seen[0][1][3].tolist() == [0, 4, 4, 5] == r.cu.tolist()
    assert seen[1][2]["rows"].tolist() == [0, 1, 3, 4, 7] and seen[1][1][1] == "q" and seen[1][2]["block"] == 1
    assert sorted([p for h in r.held for p in h] + r.free) == list(range(9))
    with pytest.raises(ValueError, match="no drafts"):
        r.accept([-1, -1, -1])
    r.extend([40, 0, 0])
    assert len(r.held[0]) == 3
    r.evict()
    assert r.lengths == [40, 0, 6] == r.pages.len.tolist() and r.totals == [74, 0, 6] and len(r.held[0]) == 2
    assert sorted([p for h in r.held for p in h] + r.free) == list(range(9))


@pytest.mark.parametrize("parents", [[[-1], [], []], [[-1, 1], [], []], [[-1, -2], [], []], [[-1, 0], []]])
def test_rollout_refuses_parents(m, monkeypatch, parents):
    r, _ = _rollout(m, monkeypatch)
    with pytest.raises(ValueError):
        r.extend([2, 0, 0], parents=parents)
    assert r.lengths == [0, 0, 0] and r.drafts is None


def test_rollout_refuses_budgets(m):
    from merged_attention_autoregressive_gb300.path import BranchRollout
    for kw in (dict(budget=10, first=6, recent=5), dict(budget=10, first=-1), dict(budget=10, block=4), dict(budget=-1)):
        with pytest.raises(ValueError):
            BranchRollout(2, 2, 64, 20, 32, **kw)


# ---- pins of the oracle

def test_oracle_tree_of_a_chain_is_causal_attention():
    from oracle import branch_oracle as B
    rng = np.random.default_rng(0)
    K, V = rng.normal(size=(2, 4, 1, 16, 8)), None
    K, V = K
    q = rng.normal(size=(2, 9, 8))
    table, cu, length = np.array([[2, 0]]), [0, 9], [25]
    a = O.tree_attention(q, cu, np.arange(9) - 1, None, K, V, table, length, 0.3)
    b = B.branch_attention(q, cu, None, K, V, table, length, 0.3, block=1)
    assert np.allclose(a[0], b[0], atol=1e-13) and np.allclose(a[1], b[1], atol=1e-13)
    # siblings do not see one another: the second child of a root is the first one in a call of its own
    t = O.tree_attention(q, cu, np.array([-1, 0, 0, 1, 2, 3, 4, 5, 6]), None, K, V, table, length, 0.3)
    assert np.abs(t[0] - b[0])[:, 2:].max() > 1e-3 and np.allclose(t[0][:, :2], b[0][:, :2], atol=1e-13)
    assert O.above([-1, 0, 0, 2], 3) == [0, 2, 3]


def test_oracle_masses_sum_to_the_rows():
    rng = np.random.default_rng(1)
    K, q = rng.normal(size=(3, 2, 16, 8)), rng.normal(size=(4, 5, 8))
    table, cu, length = np.array([[1, 2]]), [0, 5], [20]
    from oracle import branch_oracle as B
    lse = B.branch_attention(q, cu, None, K, K, table, length, 0.4, block=1)[1]
    mass, born = np.full((3, 2, 16), 9.0), np.zeros((3, 2, 16), int)
    O.page_mass(K, q, lse, None, cu, table, length, 0.4, 1, 0.0, mass, born, [30])
    live = np.concatenate((mass[1], mass[2][:, :4]), 1)
    assert np.allclose(live.sum(1), 10) and (mass[0] == 9).all()  # 5 tokens of 2 heads each
    assert (born[1, 0, 15], born[2, 1, 3], born[1, 1, 14]) == (25, 29, 0)


def test_oracle_evicts_by_hand():
    mass = np.array([5.0, 1.0, 3.0, 3.0, 3.0, 0.5, 9.0, 0.1]).reshape(1, 1, 8)
    x = np.arange(8.0).reshape(1, 1, 8)
    # the last two positions are recent; of the rest the 5, and of three equal 3s the lowest
    O.page_evict([x], mass, None, None, np.array([[0]]), [8], 4, 0, 2)
    assert x[0, 0].tolist() == [0, 6, 2, 7, 4, 5, 6, 7]
