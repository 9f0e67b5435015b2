"""The order of a rollout's calls, on the host: what may follow what, and what is
refused.  The calls to the device are recorded, so these run without a GPU."""
import contextlib
import types

import pytest
import torch

from merged_attention_autoregressive_gb300 import path


def _rollout(monkeypatch, block=1, budget=None, tokens=100, max_len=96, page=16):
    """A rollout of three branches on host tensors, and the calls that it makes."""
    seen = []
    for name in ("fastar_page_keep", "fastar_page_mass", "fastar_page_evict", "fastar_page_append",
                 "fastar_branch_attention", "fastar_tree_attention"):
        monkeypatch.setattr(path, name, lambda *a, _n=name[7:], **k: seen.append((_n, a, k)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    r = path.BranchRollout.__new__(path.BranchRollout)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    most = -(-max_len // page)
    r.B, r.tokens, r.max_len, r.lengths, r.totals = 3, tokens, max_len, [0] * 3, [0] * 3
    r.held, r.free = [[], [], []], list(range(3 * most))[::-1]
    r.pages = types.SimpleNamespace(page=page, max_pages=most, n_pages=3 * most, table=z(3, most), len=z(3))
    r.cu, r.parent, r.status = z(4), z(tokens), z(1)
    r.plan = r.prefix = None
    r.q, r.out, r.lse, r.ws, r.ws_mass = "rotated", "out", "lse", None, None
    r.scale, r.block = 0.1, block
    r.budget, r.first, r.recent, r.decay = budget, 0, 0, 1.0
    r._graphs, r._replayed = [], z(1)
    if budget is not None:
        r.mass = types.SimpleNamespace(total=z(3))
    return r, seen


def _state(r):
    return [list(r.lengths), list(r.totals), [list(h) for h in r.held], list(r.free), r.pages.len.tolist()]


def test_evictions_by_frames_take_whole_frames(monkeypatch):
    """A branch of 20 positions in frames of 8 that is cut to 16 would put the rest of
    its third frame into the place of a whole one, and every later frame across a
    border."""
    r, seen = _rollout(monkeypatch, block=8, budget=16)
    r.extend([24, 16, 5])
    r.step("q", "k", "v")
    r.evict()  # a whole frame goes; a frame that is not full yet stays with a short branch
    assert r.lengths == [16, 16, 5]
    r.extend([4, 0, 3])
    r.step("q", "k", "v")
    before, calls = _state(r), len(seen)
    with pytest.raises(ValueError, match="whole blocks"):
        r.evict()
    assert _state(r) == before and len(seen) == calls
    r.extend([4, 0, 0])  # the rest of the frame
    r.step("q", "k", "v")
    r.evict()
    assert r.lengths == [16, 16, 8]


@pytest.mark.parametrize("block", [0, 1])
def test_evictions_by_tokens_take_any_length(monkeypatch, block):
    r, _ = _rollout(monkeypatch, block=block, budget=16)
    r.extend([20, 3, 16])
    r.step("q", "k", "v")
    r.evict()
    assert r.lengths == [16, 3, 16]


def test_drafts_by_frames_are_refused(monkeypatch):
    """A path of any length would leave the later frames across a border."""
    r, _ = _rollout(monkeypatch, block=8)
    r.extend([8, 8, 8])
    before = _state(r)
    with pytest.raises(ValueError, match="block"):
        r.extend([3, 0, 0], parents=[[-1, 0, 0], [], []])
    assert _state(r) == before and r.drafts is None
    r.extend([8, 0, 0])  # the next frame
    for block in (0, 1):
        r, _ = _rollout(monkeypatch, block=block)
        r.extend([3, 0, 0], parents=[[-1, 0, 0], [], []])
        assert r.drafts == [[-1, 0, 0], [], []]


TREES = [[-1, 0, 0], [-1], []]


@pytest.mark.parametrize("budget", [None, 16])
def test_drafts_are_attended_before_they_are_accepted(monkeypatch, budget):
    """Every time, not only the first: nothing of an earlier step counts."""
    r, seen = _rollout(monkeypatch, budget=budget)
    for n in range(3):
        r.extend([3, 1, 0], parents=TREES)
        before, calls = _state(r), len(seen)
        with pytest.raises(ValueError, match="attended"):
            r.accept([2, -1, -1])
        assert _state(r) == before and len(seen) == calls and r.drafts is not None
        r.step(f"q{n}", "k", "v")
        assert r.accept([2, -1, -1]) == [[0, 2], [], []]
        if budget is not None:
            assert seen[-1][0] == "page_mass" and seen[-1][1][1] == f"q{n}"
        r.extend([1, 1, 1])  # plain tokens in between are no attention of drafts
        r.step("other", "k", "v")


def test_rows_are_weighed_before_an_eviction(monkeypatch):
    r, seen = _rollout(monkeypatch, budget=16)
    for _ in range(2):
        r.extend([20, 3, 0])
        before, calls = _state(r), len(seen)
        for call in (r.evict, lambda: r.extend([1, 0, 0])):
            with pytest.raises(ValueError, match="weighed"):
                call()
            assert _state(r) == before and len(seen) == calls
        r.step("q", "k", "v")
        r.evict()
        assert r.lengths[0] == 16
    r.extend([3, 1, 0], parents=TREES)
    r.step("q", "k", "v")
    with pytest.raises(ValueError, match="accepted"):
        r.evict()
    r.accept([1, 0, -1])  # which weighs
    r.evict()
    r.extend([0, 0, 0])  # no tokens: nothing to weigh
    r.evict()
    r.extend([0, 0, 5])
    r.release(2)  # nor of a branch that starts again
    r.evict()
    r.extend([1, 0, 0])


def test_a_rollout_without_a_budget_extends_as_often_as_it_likes(monkeypatch):
    r, _ = _rollout(monkeypatch)
    for _ in range(3):
        r.extend([2, 0, 1])
    assert r.lengths == [6, 0, 3]


@pytest.mark.parametrize("budget", [None, 16])
def test_a_step_is_over_when_its_drafts_are_accepted(monkeypatch, budget):
    """The rows of the drafts that went are others' now: the same tokens again would
    be written over them."""
    r, seen = _rollout(monkeypatch, budget=budget)
    r.extend([3, 1, 0], parents=TREES)
    r.step("q", "k", "v")
    r.step("q", "k", "v")  # as often as one likes before that
    r.accept([2, 0, -1])
    calls = len(seen)
    with pytest.raises(ValueError, match="extend"):
        r.step("q", "k", "v")
    assert len(seen) == calls
    r.extend([1, 0, 0])
    r.step("q", "k", "v")


def test_a_step_is_over_when_its_rows_are_evicted(monkeypatch):
    r, seen = _rollout(monkeypatch, budget=16)
    r.extend([10, 0, 0])
    r.step("q", "k", "v")
    r.evict()  # nothing is over the budget
    r.step("q", "k", "v")
    r.extend([10, 0, 0])
    r.step("q", "k", "v")
    r.evict()
    calls = len(seen)
    with pytest.raises(ValueError, match="extend"):
        r.step("q", "k", "v")
    assert len(seen) == calls


def _captured(monkeypatch, r, *args):
    """A captured step: nothing runs, the graph holds the word's number."""
    word = int(r._replayed)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    r.step(*args)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    number = int(r._replayed)
    r._replayed.fill_(word)
    return lambda: r._replayed.fill_(number)


def test_replayed_steps_count(monkeypatch):
    r, seen = _rollout(monkeypatch, budget=16)
    plain = _captured(monkeypatch, r, "q", "k", "v")  # before any extend
    r.extend([20, 1, 0])
    with pytest.raises(ValueError, match="weighed"):
        r.evict()
    plain()
    r.evict()
    second = _captured(monkeypatch, r, "q", "k", "v")  # also behind an eviction, for the tokens to come
    r.extend([1, 1, 1])
    with pytest.raises(ValueError, match="weighed"):
        r.extend([1, 1, 1])
    second()
    r.extend([3, 1, 0], parents=TREES)
    first = _captured(monkeypatch, r, "q1", "k", "v")
    other = _captured(monkeypatch, r, "q2", "k", "v")
    with pytest.raises(ValueError, match="attended"):
        r.accept([0, 0, -1])
    plain()  # a step of plain tokens is no attention of drafts
    with pytest.raises(ValueError, match="attended"):
        r.accept([0, 0, -1])
    for replay, q in ((first, "q1"), (other, "q2"), (first, "q1")):  # each graph's own queries are weighed
        replay()
        r.accept([0, 0, -1])
        assert seen[-1][0] == "page_mass" and seen[-1][1][1] == q
        r.extend([3, 1, 0], parents=TREES)
    first()
    r.step("q3", "k", "v")  # the last one of an extend counts
    r.accept([0, 0, -1])
    assert seen[-1][1][1] == "q3"
    r.extend([1, 0, 0])
    first()  # (a graph of drafts weighs nothing)
    with pytest.raises(ValueError, match="weighed"):
        r.evict()


def test_steps_of_the_parts_calls(monkeypatch):
    r, seen = _rollout(monkeypatch, budget=16)
    r.extend([20, 0, 0])
    r.stepped()
    r.evict()
    for plan, q, want in (("plan", None, "rotated"), ("plan", "mine", "mine"), (None, "mine", "mine")):
        r.plan = plan
        r.extend([3, 1, 0], parents=TREES)
        if plan is None:
            with pytest.raises(ValueError, match="queries"):  # nothing was rotated into the object's buffer
                r.stepped()
        r.stepped(q)
        r.accept([0, -1, -1])
        assert seen[-1][1][1] == want


def test_a_step_may_attend_without_weighing(monkeypatch):
    """A frame that is attended once per denoising step is weighed once."""
    r, seen = _rollout(monkeypatch, block=8, budget=16)
    r.extend([8, 0, 8])
    for _ in range(3):
        r.step("q", "k", "v", weigh=False)
    assert [n for n, _, _ in seen] == ["page_append", "branch_attention"] * 3
    for call in (r.evict, lambda: r.extend([8, 0, 0])):  # nothing is weighed yet
        with pytest.raises(ValueError, match="weighed"):
            call()
    r.step("q", "k", "v")
    assert [n for n, _, _ in seen].count("page_mass") == 1
    r.evict()
    r.extend([8, 0, 0])
    calls = len(seen)
    replay = _captured(monkeypatch, r, "q", "k", "v", None, None, False)  # (weigh=False)
    assert len(seen) == calls + 2
    replay()
    with pytest.raises(ValueError, match="weighed"):
        r.evict()


def test_drafts_are_weighed_when_they_are_accepted(monkeypatch):
    r, seen = _rollout(monkeypatch, budget=16)
    for weigh in (True, False):
        r.extend([3, 1, 0], parents=TREES)
        r.step("q", "k", "v", weigh=weigh)
        assert seen[-1][0] == "tree_attention"
        r.accept([2, 0, -1])
        assert seen[-1][0] == "page_mass"
        r.evict()
