"""Branches are independent: infinities and NaN among the keys and values of one
change no bit of another's results, whichever rows share a tile."""
import math

import pytest
import torch

import test_gpu_branch as T

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

CASES = [
    # D, H, g, page, new, past, C, counts, block, pad
    (128, 2, 1, 64, [1] * 9, [300, 0, 63, 64, 5, 1, 130, 700, 20], 500, True, 0, 0),   # single tokens, a prefix
    (64, 3, 1, 16, [1] * 40, list(range(40)), 0, False, 0, 2),                          # no prefix: pages come first
    (128, 1, 3, 32, [1] * 30, list(range(0, 600, 20)), 0, False, 0, 0),                 # groups across rows of four
    (64, 2, 5, 16, [1] * 70, [7, 90, 200] * 23 + [3], 100, False, 0, 1),                # several tiles, tokens across them
    (128, 2, 2, 64, [5, 0, 17, 1, 33, 64, 2], [9, 3, 0, 255, 31, 0, 140], 300, True, 1, 3),
    (64, 12, 1, 64, [20] * 60, [0, 100] * 30, 0, False, 7, 0),                          # items that are not cut
    (128, 8, 1, 64, [300, 200, 1, 1, 300, 17], [500, 0, 9, 900, 64, 5], 9000, True, 0, 0),  # more than 128 rows, long prefix
    (128, 12, 1, 128, [520, 300, 40, 200], [100, 900, 7, 0], 20000, False, 260, 5),     # 256 rows to an item
    (64, 16, 5, 32, [1] * 128, list(range(0, 64)) * 2, 8000, True, 0, 3),               # many single tokens, long prefix
]


@pytest.fixture(scope="module")
def m():
    import merged_attention_autoregressive_gb300 as m
    return m


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_spoiled_branch_leaves_the_others_as_they_are(m, case, dtype):
    D, H, g, page, new, past, C, counts, block, pad = CASES[case]
    q, cu, prefix, pages, cu_h, length, table = T._attention_case(m, dtype, D, H, g, page, new, past, C, counts, block,
                                                                  pad, seed=40 + case, spoil=False)
    px = None
    if prefix is not None:
        px = m.Prefix(prefix[0], prefix[1], m=None if prefix[2] is None else T._cuda(prefix[2]),
                      size=None if prefix[3] is None else T._cuda(prefix[3]))

    def attend():
        out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
        st = T._status()
        m.fastar_branch_attention(q, cu, px, pages, D ** -0.5, out, lse=lse, block=block, status=st)
        assert int(st) == 0
        return out, lse

    clean, clean_lse = attend()
    assert bool(clean.isfinite().all())
    K, V = pages.K.clone(), pages.V.clone()
    with_tokens = [b for b in range(len(new)) if new[b]]
    for b in {with_tokens[0], with_tokens[len(with_tokens) // 2], with_tokens[-1]}:
        own = torch.as_tensor(table[b][:-(-int(length[b]) // page)], dtype=torch.long, device="cuda")
        for value in (math.nan, math.inf, -math.inf):
            pages.K.copy_(K), pages.V.copy_(V)
            pages.V[own] = value
            if math.isnan(value):
                pages.K[own] = value
            out, lse = attend()
            mine = torch.zeros(q.shape[1], dtype=torch.bool, device="cuda")
            mine[int(cu_h[b]):int(cu_h[b + 1])] = True
            assert torch.equal(out[:, ~mine], clean[:, ~mine]) and torch.equal(lse[:, ~mine], clean_lse[:, ~mine])
            assert not bool(out[:, mine].isfinite().any())   # its own tokens see them
