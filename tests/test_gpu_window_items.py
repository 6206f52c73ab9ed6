"""GPU tests of the window attention's items of one and two key tiles, many to a
CTA (narrow windows of long prompts, batches of short ones), against the fp64
oracle; bounds as in test_gpu_cache_ops.py."""
import math

import pytest
import torch

from oracle import cache_ops as ora
from tests.test_gpu_cache_ops import BF, check_attention, f64, status

pytestmark = pytest.mark.gpu


def inputs(B, L, G, Hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(B, L, G * Hkv, d, generator=g) * 1.5).to(BF)
    k, v = (torch.randn(B, L, Hkv, d, generator=g).to(BF) for _ in "kv")
    return q, k, v


def check_rows(o, lse, q, k, v, b, at, window, n_sink):
    d = q.shape[-1]
    one = [f64(x[b:b + 1]) for x in (q, k, v)]
    r = ora.window_attn(*one, window, n_sink, 1 / math.sqrt(d), rows=at)
    check_attention(o[b:b + 1, at], lse[b:b + 1, at], r, None, d, min(q.shape[1], window + n_sink), 2.0**-8, False)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 4), (17, 0), (17, 4), (33, 0), (33, 16), (49, 0), (50, 4)])
@pytest.mark.parametrize("G,d", [(16, 128), (16, 64), (8, 128)])
def test_narrow_windows_of_a_long_prompt(cuda_lib, G, d, window, n_sink):
    hs2, L = cuda_lib, 23001
    q, k, v = inputs(1, L, G, 1, d, seed=window)
    dev = [x.cuda() for x in (q, k, v)]
    o, lse = hs2.hs2_window_attn(*dev, window, n_sink)
    o2, lse2 = hs2.hs2_window_attn(*dev, window, n_sink)
    assert status(hs2) == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    at = sorted({0, 1, 15, 16, 17, 63, 64, 65, L - 2, L - 1} | set(range(31, L, 211)))
    check_rows(o, lse, q, k, v, 0, at, window, n_sink)


@pytest.mark.parametrize("B,L,G,Hkv,d", [(64, 64, 4, 8, 128), (300, 100, 16, 1, 128), (700, 33, 1, 2, 64),
                                         (2000, 1, 16, 1, 64)])
def test_batches_of_short_prompts(cuda_lib, B, L, G, Hkv, d):
    """Items of one tile, and (100 tokens) of one and two in turn."""
    hs2 = cuda_lib
    q, k, v = inputs(B, L, G, Hkv, d, seed=L)
    dev = [x.cuda() for x in (q, k, v)]
    o, lse = hs2.hs2_window_attn(*dev, 1000)
    o2, lse2 = hs2.hs2_window_attn(*dev, 1000)
    assert status(hs2) == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for b in range(0, B, max(1, B // 24)):
        check_rows(o, lse, q, k, v, b, sorted({0, L // 2, (b * 7) % L, L - 1}), 1000, 0)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (33, 0), (17, 4)])
def test_narrow_windows_of_a_batch_padded_with_nan(cuda_lib, window, n_sink):
    hs2, L, G, d, n = cuda_lib, 20000, 16, 128, 9875
    q, k, v = inputs(2, L, G, 1, d, seed=3)
    dev = [x.cuda() for x in (q, k, v)]
    want, want_lse = hs2.hs2_window_attn(*dev, window, n_sink)
    for x in dev:
        x[1, n:] = math.nan
    o, lse = hs2.hs2_window_attn(*dev, window, n_sink)
    assert status(hs2) == 0
    assert torch.equal(o[0], want[0]) and torch.equal(lse[0], want_lse[0])
    assert o[1, n:].isnan().all() and lse[1, n:].isnan().all()
    at = sorted({0, 1, n - 1, n - 2, n - 8, n - 17} | set(range(5, n, 397)))
    check_rows(o, lse, q, k, v, 1, at, window, n_sink)
