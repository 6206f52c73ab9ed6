"""GPU tests of the window attention with infinities and NaN among its rows,
against the fp64 oracle; bounds as in test_gpu_cache_ops.py."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as ora
from tests.test_gpu_cache_ops import BF, check_attention, f64, status

pytestmark = pytest.mark.gpu


def inputs(B, Lq, Lk, G, d, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, Lq, G, d, generator=g).to(BF).cuda()
    k, v = (torch.randn(B, Lk, 1, d, generator=g).to(BF).cuda() for _ in "kv")
    return q, k, v


def test_a_newest_key_without_weight_beside_masked_nan(cuda_lib):
    """Keys whose logits are -inf weigh nothing, also when they are a row's
    newest and the row shares its tile with values of NaN that it does not see."""
    hs2, L, G, d = cuda_lib, 200, 4, 64
    q, k, v = inputs(1, L, L, G, d, 1)
    q[..., 5] = q[..., 5].abs() + 0.5
    none = [100, 101, 102]
    k[0, none, 0, 5] = -math.inf
    v[0, 110] = math.nan
    o, lse = hs2.hs2_window_attn(q, k, v, 64, 0)
    assert status(hs2) == 0
    at = list(range(90, 110)) + list(range(174, 200))
    for t in at:
        seen = [s for s in range(max(0, t - 63), t + 1) if s not in none]
        r = ora.attend(f64(q[0, t]), f64(k[0, seen, 0]), f64(v[0, seen, 0]), 1 / math.sqrt(d))
        r = {n: np.broadcast_to(x, (G, d) if n in ("o", "av", "vmax") else (G,))[None, None] for n, x in r.items()}
        check_attention(o[:, t:t + 1], lse[:, t:t + 1], r, None, d, 64, 2.0**-8, False)
