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
