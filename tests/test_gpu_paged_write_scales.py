"""GPU test of rows written into pages whose scales this writer did not choose."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as ora
from tests.test_gpu_cache_ops import BF, U8, ints, status, values

pytestmark = pytest.mark.gpu


def test_rows_under_an_earlier_scale_that_is_no_power_of_two(cuda_lib):
    """Codes are those of the fp32 quotients: quotients at e4m3's ties, where the
    product with a rounded reciprocal falls on the other side."""
    hs2, P, page, d = cuda_lib, 400, 16, 64
    g = np.random.default_rng(0)
    ties = 1 + (2 * np.arange(8) + 1) / 16
    x = np.zeros((P, d), np.float32)
    s = np.zeros(P, np.float32)
    n = 0
    while n < P:
        top = np.float32(g.integers(128, 256))
        s[n] = top / g.choice(ties)
        xs = g.integers(128, 256, 5000).astype(np.float32)
        off = xs[ora.e4m3_round(xs / s[n]) != ora.e4m3_round(xs * (np.float32(1) / s[n]))]
        if len(off):
            x[n] = g.choice(off, d)
            n += 1
    k, v = (torch.zeros(P, 1, page, d, dtype=U8, device="cuda") for _ in "kv")
    ks, vs = (torch.from_numpy(s).cuda().view(P, 1).clone() for _ in "kv")
    table = torch.arange(P, dtype=torch.int32, device="cuda").view(P, 1)
    rows = torch.from_numpy(x).to(BF).cuda().view(P, 1, 1, d)
    hs2.hs2_paged_kv_write(rows, -rows, table, ints([1] * P), k, v, ks, vs)
    assert status(hs2) == 0
    np.testing.assert_array_equal(ks.cpu().numpy()[:, 0], s)
    want = ora.e4m3_round(x / s[:, None])
    np.testing.assert_array_equal(values(k)[:, 0, 1], want)
    np.testing.assert_array_equal(values(v)[:, 0, 1], -want)
