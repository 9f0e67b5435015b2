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
