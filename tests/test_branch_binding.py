"""What the binding of the branched-rollout calls hands to the library,
looked at on host tensors: the library's calls are replaced by recorders,
so nothing is launched."""
import types

import pytest
import torch

BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture
def m(monkeypatch):
    import merged_attention_autoregressive_gb300 as m
    from merged_attention_autoregressive_gb300 import build
    build.build()
    m.lib()
    monkeypatch.setattr(m, "_gpu", lambda t: t.get_device())  # host tensors are taken as they are
    monkeypatch.setattr(m, "_current_gpu", lambda: -1)
    monkeypatch.setattr(m, "_raw_stream", lambda dev: 0)
    return m


@pytest.fixture
def calls(m, monkeypatch):
    """The structs of each call, as the library would read them at that time."""
    seen = []

    def record(pages, prefix=None):
        copy = lambda kind, at: None if at is None else kind.from_buffer_copy(kind.from_address(at))  # noqa: E731
        seen.append(types.SimpleNamespace(pages=copy(m.PagesStruct, pages), prefix=copy(m.PrefixStruct, prefix)))
        return 0

    monkeypatch.setattr(m, "_lib", types.SimpleNamespace(
        fastar_page_append=lambda *a: record(a[0]),
        fastar_branch_attention=lambda *a: record(a[6], a[5])))
    return seen


def _pages(m, B=2, n_pages=4, most=3):
    z = torch.zeros
    return m.PagedKV.view(z(n_pages, 2, 16, 64, dtype=BF), z(n_pages, 2, 16, 64, dtype=BF), z(B, most, dtype=I32),
                          z(B, dtype=I32))


def _attend(m, pages, prefix=None):
    q = torch.zeros(2, 3, 64, dtype=BF)
    m.fastar_branch_attention(q, torch.zeros(pages.B + 1, dtype=I32), prefix, pages, 0.1, torch.zeros_like(q),
                              ws=torch.zeros(8, dtype=torch.uint8))


def _append(m, pages):
    k = torch.zeros(2, 3, 64, dtype=BF)
    m.fastar_page_append(pages, k, k, torch.zeros(pages.B + 1, dtype=I32))


def _fits(p, pages):
    shape = (p.n_pages, p.H, p.page, p.D)
    return (shape == tuple(pages.K.shape) and (p.B, p.max_pages) == tuple(pages.table.shape) and
            (p.K, p.V, p.table, p.len) == tuple(t.data_ptr() for t in (pages.K, pages.V, pages.table, pages.len)))


@pytest.mark.parametrize("call", [_append, _attend])
def test_calls_read_the_tensors_that_the_pages_hold_now(m, calls, call):
    pages = _pages(m)
    call(m, pages)
    assert _fits(calls[-1].pages, pages)
    pages.len = pages.len + 1                                        # another tensor: the old one is freed
    call(m, pages)
    assert _fits(calls[-1].pages, pages)
    pages.table = torch.zeros(2, 7, dtype=I32)                       # a longer table
    assert pages.max_pages == 7
    call(m, pages)
    assert _fits(calls[-1].pages, pages)
    pages.K, pages.V = torch.zeros(9, 2, 16, 64, dtype=BF), torch.zeros(9, 2, 16, 64, dtype=BF)  # a larger pool
    assert pages.n_pages == 9
    call(m, pages)
    assert _fits(calls[-1].pages, pages)
    pages.table, pages.len = torch.zeros(5, 2, dtype=I32), torch.zeros(5, dtype=I32)             # more branches
    call(m, pages)
    assert pages.B == 5 and _fits(calls[-1].pages, pages)


@pytest.mark.parametrize("name,value", [
    ("len", torch.zeros(2, dtype=torch.int64)), ("len", torch.zeros(3, dtype=I32)), ("table", torch.zeros(2, dtype=I32)),
    ("table", torch.zeros(3, 4, dtype=I32).t()), ("V", torch.zeros(4, 2, 16, 64)), ("K", torch.zeros(5, 2, 16, 64, dtype=BF))])
def test_calls_refuse_assigned_tensors_that_do_not_fit(m, calls, name, value):
    for call in (_append, _attend):
        pages = _pages(m)
        setattr(pages, name, value)
        with pytest.raises(ValueError):
            call(m, pages)
    assert not calls


def test_calls_read_the_tensors_that_the_prefix_holds_now(m, calls):
    z = torch.zeros
    pages, px = _pages(m), m.Prefix(z(2, 5, 64, dtype=BF), z(2, 5, 64, dtype=BF))

    def check():
        _attend(m, pages, px)
        p, at = calls[-1].prefix, lambda t: None if t is None else t.data_ptr()
        assert (p.H, p.C, p.D) == tuple(px.K.shape)
        assert (p.K, p.V, p.m, p.size) == tuple(at(t) for t in (px.K, px.V, px.m, px.size))

    check()
    px.size = torch.ones(2, dtype=I32)
    check()
    px.size = px.size + 1
    px.m = torch.ones(2, 5, dtype=I32)
    check()
    px.K, px.V, px.m = z(2, 9, 64, dtype=BF), z(2, 9, 64, dtype=BF), None
    check()
    px.m = torch.ones(2, 5, dtype=I32)  # of another length
    with pytest.raises(ValueError):
        _attend(m, pages, px)


def test_unknown_attributes_are_refused(m):
    with pytest.raises(AttributeError):
        _pages(m).lengths
    with pytest.raises(AttributeError):
        m.PagedKV.__new__(m.PagedKV).K
