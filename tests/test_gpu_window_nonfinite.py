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


def seen_by(L, window, n_sink):
    t, s = torch.arange(L).view(-1, 1), torch.arange(L)
    return (s <= t) & ((s > t - window) | (s < n_sink))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("L,G,d,window,n_sink", [
    (700, 16, 128, 100, 3), (700, 1, 64, 100, 0), (600, 4, 128, 2**31 - 1, 0), (500, 8, 64, 7, 20), (3000, 7, 64, 40, 1),
])
def test_values_that_are_not_finite_reach_the_rows_and_dims_that_see_them(cuda_lib, L, G, d, window, n_sink, bad):
    """Single value elements of NaN or infinity, keys and queries finite: a dim of
    an output is finite exactly where no value in its row's sight is bad in it,
    and right there."""
    hs2 = cuda_lib
    q, k, v = inputs(1, L, L, G, d, L + d)
    want = ora.window_attn(f64(q), f64(k), f64(v), window, n_sink, 1 / math.sqrt(d))
    g = torch.Generator().manual_seed(3)
    at = [0, 2, n_sink, 130, 131, L // 2, L - 2] + torch.randint(0, L, (4,), generator=g).tolist()
    spoil = torch.zeros(L, d, dtype=torch.bool)
    for i, s in enumerate(at):
        spoil[s, [(5 * i) % d, d - 1 - i]] = True
    spoil[L - 9] = True
    v[0, spoil.view(L, 1, d).cuda()] = bad
    o, lse = hs2.hs2_window_attn(q, k, v, window, n_sink)
    o2, _ = hs2.hs2_window_attn(q, k, v, window, n_sink)
    assert status(hs2) == 0
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16))
    meant = (seen_by(L, window, n_sink).float() @ spoil.float() > 0).view(1, L, 1, d).expand(1, L, G, d)
    assert torch.equal(o.isfinite().cpu(), ~meant)
    # (the rows' bounds are those of the values without the bad ones)
    o = torch.where(meant, torch.from_numpy(want["o"]), o.double().cpu())
    check_attention(o, lse, want, None, d, min(L, window + n_sink), 2.0**-8, False)


def ms_of(call, times=3):
    call()
    a, b = torch.cuda.Event(True), torch.cuda.Event(True)
    torch.cuda.synchronize()
    a.record()
    for _ in range(times):
        call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / times


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("what", ["value", "value row", "key row", "both rows"])
def test_a_bad_row_that_a_whole_prompt_sees_costs_little(cuda_lib, what, bad):
    """The first row of one sequence, in sight of all of its queries: the other
    sequence keeps its bits, nothing times out, and the call is not slowed down
    by redoing what is meant to be."""
    hs2, L, G, d = cuda_lib, 12000, 8, 128
    q, k, v = inputs(2, L, L, G, d, 5)
    call = lambda: hs2.hs2_window_attn(q, k, v, L)  # noqa: E731
    o, lse = call()
    fine = ms_of(call)
    if what == "value":
        v[0, 0, 0, 7] = bad
    if what in ("value row", "both rows"):
        v[0, 0] = bad
    if what in ("key row", "both rows"):
        k[0, 0] = bad
    o2, lse2 = call()
    assert status(hs2) == 0
    assert torch.equal(o2[1], o[1]) and torch.equal(lse2[1], lse[1])
    if what == "value":
        assert not o2[0, :, :, 7].isfinite().any()
        rest = [e for e in range(d) if e != 7]
        assert torch.equal(o2[0][..., rest], o[0][..., rest]) and torch.equal(lse2[0], lse[0])
    elif what == "value row" or math.isnan(bad):
        assert not o2[0].isfinite().any()
    else:  # the key's logits are NaN (both infinities in a sum)
        assert o2[0].isnan().all()
    assert ms_of(call) < 3 * fine, (ms_of(call), fine)


def test_padding_of_bad_values_alone_in_wide_windows(cuda_lib):
    """Keys of the padding finite, values not: the rows in front of it are right,
    its own rows not finite.  One CTA does the rows of one item again, 156 rows of
    11,000 keys (about 18 times a clean call; all rows behind it would be 1000)."""
    hs2, L, G, d, n = cuda_lib, 20000, 4, 128, 11111
    q, k, v = inputs(2, L, L, G, d, 6)
    call = lambda: hs2.hs2_window_attn(q, k, v, L)  # noqa: E731
    o, lse = call()
    fine = ms_of(call)
    for bad in (math.nan, math.inf):
        v[1, n:] = bad
        o2, lse2 = call()
        assert status(hs2) == 0
        assert torch.equal(o2[0], o[0]) and torch.equal(lse2, lse)
        assert not o2[1, n:].isfinite().any()
        np.testing.assert_allclose(f64(o2[1, :n]), f64(o[1, :n]), rtol=2.0**-7, atol=2.0**-8)
        assert ms_of(call) < 60 * fine, (ms_of(call), fine)


def test_logits_far_below_zero(cuda_lib):
    """All of a row's logits near -1e31: equal keys, so that the output is the
    values' mean."""
    hs2, L, G, d = cuda_lib, 100, 16, 64
    q, k, v = inputs(1, L, L, G, d, 7)
    q[:], k[:] = 2.0**50, -(2.0**50)
    o, lse = hs2.hs2_window_attn(q, k, v, 20)
    assert status(hs2) == 0
    for t in (0, 5, 19, 20, 99):
        vis = f64(v[0, max(0, t - 19):t + 1, 0])
        np.testing.assert_allclose(f64(o[0, t]), np.broadcast_to(vis.mean(0), (G, d)),
                                   rtol=2.0**-8, atol=2.0**-7 * np.abs(vis).mean(0).max())
    np.testing.assert_allclose(f64(lse), -(2.0**100) * d / math.sqrt(d), rtol=2.0**-20)
