"""Calls whose items differ in length, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import test_gpu_branch as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import merged_attention_autoregressive_gb300 as m
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,H,g,new,past,C,rest", [
    (128, 40, 1, [1] * 4, [30, 0, 63, 64], 9000, 300),    # one head full, the others near empty
    (64, 12, 1, [1, 1], [10, 200], 20000, 700),
    (128, 2, 5, [1] * 3, [0, 5, 300], 8000, 1),
    (64, 3, 2, [2, 1], [0, 400], 5000, 0),                # nothing in the others
    (64, 24, 1, [1] * 9, [0] * 9, 3000, 2999),
])
def test_heads_of_different_lengths(m, dtype, D, H, g, new, past, C, rest):
    q, cu, prefix, pages, cu_h, length, table = T._attention_case(m, dtype, D, H, g, 64, new, past, C, True, 0, 1, seed=31)
    pK, pV, cnt, _ = prefix
    for full in (0, H - 1):
        size = np.full(H, rest, np.int32)
        size[full] = C
        k, v = pK.nan_to_num(0.5, 0.5, 0.5), pV.nan_to_num(0.5, 0.5, 0.5)
        dead = T._cuda(np.arange(C)[None] >= size[:, None])[..., None]
        k.masked_fill_(dead, float("nan"))
        v.masked_fill_(dead, float("inf"))
        T._check_attention(m, dtype, q, cu, (k, v, cnt, size), pages, D ** -0.5, 0, cu_h, length, table)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,H,g,new,past,C,block", [
    (64, 8, 1, [1] * 2560, [90, 0, 31, 400] * 640, 0, 0),        # 128 branches to a tile, more items than CTAs
    (128, 5, 2, [1] * 1300, list(range(130)) * 10, 130, 1),
    (64, 40, 1, [1] * 7 + [600], [500] * 7 + [20], 0, 1),        # single tokens beside a prompt
    (64, 12, 1, [20] * 120, list(range(0, 240, 2)), 0, 1),       # several short prompts to a tile
])
def test_many_branches_to_a_tile(m, dtype, D, H, g, new, past, C, block):
    q, cu, prefix, pages, cu_h, length, table = T._attention_case(m, dtype, D, H, g, 64, new, past, C, True, block, 3, seed=32)
    T._check_attention(m, dtype, q, cu, prefix, pages, D ** -0.5, block, cu_h, length, table)
