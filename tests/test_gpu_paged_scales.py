"""GPU tests of the paged decode with value scales that differ widely, against
the fp64 oracle.

Bounds as in test_gpu_cache_ops.py, but what the kernel drops of a weight is
counted against what the head's tokens contribute, not against the largest
scale: at most 2^-28 of the largest (softmax weight) x (V scale) per token, for
at most 448 of that."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as ora
from tests.test_gpu_cache_ops import BF, U8, Pool, f64, ints, q_top, status, values

pytestmark = pytest.mark.gpu


def check(hs2, pool, q, lengths, window=None, n_sink=0):
    B, Hq, d = q.shape
    G = Hq // pool.Hkv
    scale = 1 / math.sqrt(d)
    o, lse = hs2.hs2_paged_decode(q, *pool.args(), ints(lengths), window=window, n_sink=n_sink)
    assert status(hs2) == 0
    o, lse = f64(o), f64(lse)
    kv, vv, ks, vs, qa = values(pool.k), values(pool.v), f64(pool.ks), f64(pool.vs), q_top(q, pool.Hkv)
    q = f64(q)
    w = 2**31 - 1 if window is None else window
    for b, T in enumerate(lengths):
        pos = np.arange(T)
        pos = pos[(pos >= T - w) | (pos < n_sink)]
        k, v = (ora.paged_rows(z, s, pool.table_np[b], pool.page, pos) for z, s in ((kv, ks), (vv, vs)))
        sv = vs[pool.table_np[b][pos // pool.page]]  # [n, Hkv]
        for h in range(pool.Hkv):
            at = slice(h * G, (h + 1) * G)
            r = ora.attend(q[b, at], k[:, h], v[:, h], scale)
            L = (d + 8) * 2.0**-23 * r["x"] + 2.0**-21 * qa[b, at] * r["k1"]
            p = np.exp(q[b, at] @ k[:, h].T * scale - r["lse"][:, None])
            floor = len(pos) * 2.0**-28 * 448 * (p * sv[:, h]).max(1)
            tol = (2.0**-8 * np.abs(r["o"]) + (2.0**-9 + 2.0**-20 + 4 * L)[:, None] * r["av"] * 1.01
                   + floor[:, None] + 2.0**-133)
            err = np.abs(o[b, at] - r["o"])
            assert np.isfinite(o[b, at]).all() and (err <= tol).all(), float((err / tol).max())
            tl = L + 2.0**-20 + len(pos) * 2.0**-24 + 2.0**-22 * np.abs(r["lse"])
            assert (np.abs(lse[b, at] - r["lse"]) <= tl).all()


def query(B, Hq, d, seed):
    return torch.randn(B, Hq, d, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


def aside(pool, pid, octaves):
    """Pages whose V scale is 2^octaves above the others', which hardly any
    weight falls on: their keys point away from the queries."""
    pool.k[pid] = (torch.ones_like(pool.k[pid].float()) * -96).to(torch.float8_e4m3fn).view(U8)
    pool.ks[pid] = 2.0**-4
    pool.vs[pid] = 2.0**(octaves - 6)


@pytest.mark.parametrize("octaves", [8, 16, 24, 30, 60, 100])
@pytest.mark.parametrize("G,Hkv,d,page", [(16, 1, 128, 64), (8, 1, 64, 16), (4, 2, 64, 32), (1, 1, 128, 128)])
def test_large_scales_without_weight_cost_the_others_nothing(cuda_lib, G, Hkv, d, page, octaves):
    hs2, lengths = cuda_lib, [1500, 9, 700]
    pool = Pool(3, Hkv, d, page, -(-1500 // page), seed=G).fill(lengths, seed=octaves)
    pool.vs[pool.table[0].long()] = pool.vs[pool.table[0].long()].clamp(max=2.0**-6)
    last = (1500 - 1) // page
    aside(pool, pool.table[0, [0, last // 2, last]].long(), octaves)
    aside(pool, pool.table[2, :1].long(), octaves)
    q = query(3, G * Hkv, d, octaves).abs()  # (logits near -6 d / sqrt(d) on the pages set aside)
    check(hs2, pool, q, lengths)
    check(hs2, pool, q, lengths, window=300, n_sink=5)


@pytest.mark.parametrize("G", [16, 8, 4])
def test_heads_that_attend_to_pages_of_different_scales(cuda_lib, G):
    """Half of the heads look at the pages of large values, the others away from
    them: each head keeps its own pages' bits."""
    hs2, d, T = cuda_lib, 128, 2000
    pool = Pool(1, 1, d, 64, 32, seed=2).fill([T], seed=3)
    pid = pool.table[0].long()
    big = pid[torch.arange(32, device="cuda") % 3 == 1]
    pool.vs[pid] = 2.0**-6
    pool.vs[big] = 2.0**22
    pool.k[big] = (torch.rand(len(big), 1, 64, d, generator=torch.Generator().manual_seed(1)) * 32 + 64).to(
        torch.float8_e4m3fn).view(U8).cuda()
    pool.ks[big] = 2.0**-4
    q = query(1, G, d, 4).abs()
    q[:, G // 2:] *= -1
    check(hs2, pool, q, [T])


@pytest.mark.parametrize("low,high", [(-126, -126), (-132, -130), (100, 110), (-126, -40), (-40, 40), (0, 90)])
def test_scales_of_any_size(cuda_lib, low, high):
    """All scales tiny (products of codes and scales down to subnormals), all
    huge, and spread over up to 2^90, rising and falling along the sequence."""
    hs2, d, T = cuda_lib, 64, 1900
    for rising in (True, False):
        pool = Pool(2, 1, d, 32, 60, seed=7).fill([T, 33], seed=8)
        e = torch.linspace(low, high, 60, device="cuda").round()
        pid = pool.table.long()
        pool.vs[pid[0]] = torch.exp2((e if rising else e.flip(0)).double()).float()[:, None]
        pool.vs[pid[1]] = 2.0**low
        for g in (3, 16):
            check(hs2, pool, query(2, g, d, g), [T, 33])


def test_parts_of_a_long_sequence_with_uneven_scales(cuda_lib):
    """Parts on many CTAs, joined: some see large scales without weight only."""
    hs2, d, T = cuda_lib, 128, 60000
    pool = Pool(1, 1, d, 128, -(-T // 128), seed=9).fill([T], seed=10)
    pid = pool.table[0].long()
    pool.vs[pid] = pool.vs[pid].clamp(max=2.0**-6)
    aside(pool, pid[100:200], 40)
    aside(pool, pid[300:310], 90)
    check(hs2, pool, query(1, 16, d, 5).abs(), [T])


def test_the_largest_weight_stays_whole_and_the_others_unbiased(cuda_lib):
    """Rounding weights to nine bits neither touches the token that dominates a
    sharp softmax nor shifts the sum of many: over 2^15 outputs the least-squares
    factor between output and value is 1 within four of its deviations (weights
    off by 2^-9 at most, of 700 to 3000 tokens, and 2^-8 of a bf16 output, both
    at random: under 2^-16 together; a bias of half a step would be 2^-11.5)."""
    hs2, G, d = cuda_lib, 16, 128
    lengths = [700, 1500, 3000, 2222] * 4
    pool = Pool(16, 1, d, 64, 47, seed=12).fill(lengths, seed=13)
    pool.ks[:] = 2.0**-9                # logits of deviation 1: every weight counts a little
    pool.v[:] = pool.v.bitwise_and(0x7F)  # values of one sign, whose sum shows a bias
    q = query(16, G, d, 14)
    o, _ = hs2.hs2_paged_decode(q, *pool.args(), ints(lengths))
    assert status(hs2) == 0
    r = pool.oracle(q, lengths, 2**31 - 1, 0, 1 / math.sqrt(d))["o"]
    o = f64(o)
    assert abs((o * r).sum() / (r * r).sum() - 1) < 2.0**-14
    # one token with all but 2^-20 of the weight: its value, to bf16's rounding
    T = 1000
    pool = Pool(1, 1, d, 64, 16, seed=15).fill([T], seed=16)
    q = query(1, G, d, 17).abs()
    pid, s = int(pool.table[0, 11]), 11 * 64 + 5
    pool.ks[pool.table[0].long()] = 2.0**-5
    pool.k[pool.table[0].long()] = 0x80 | 0x38      # -1
    pool.k[pid, 0, 5] = 0x7E                         # 448
    o, _ = hs2.hs2_paged_decode(q, *pool.args(), ints([T]))
    want = torch.from_numpy(values(pool.v)[pid, 0, 5] * float(pool.vs[pid, 0])).to(BF)
    assert s < T and status(hs2) == 0
    assert torch.equal(o.cpu(), want.expand(1, G, d))


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("G,d,page", [(16, 128, 64), (8, 128, 32), (4, 128, 16)])
def test_heads_that_look_at_a_page_of_zeros_alone(cuda_lib, G, d, page, first):
    """Half of the heads at a page of zeros (scale 2^-126), 100 nats above all
    else, the others at values of thousands: these are right, and those are what
    is left, next to nothing."""
    hs2, T = cuda_lib, 1500
    mp = -(-T // page)
    pool = Pool(1, 1, d, page, mp, seed=18).fill([T], seed=19)
    pid = pool.table[0].long()
    pool.vs[pid] = 2.0**6
    pool.ks[pid] = 2.0**-4
    pool.k[pid] = 0x80 | 0x6C                 # -96
    zero = pid[0 if first else mp - 1]
    pool.k[zero] = 0x6C
    pool.v[zero], pool.vs[zero] = 0, 2.0**-126
    q = query(1, G, d, 20).abs()
    q[:, 1::2] *= -1
    o, lse = hs2.hs2_paged_decode(q, *pool.args(), ints([T]))
    assert status(hs2) == 0
    r = pool.oracle(q, [T], 2**31 - 1, 0, 1 / math.sqrt(d))
    tol = (2.0**-8 * np.abs(r["o"]) + (2.0**-9 + 2.0**-10) * r["av"])[:, 1::2]
    assert (np.abs(f64(o) - r["o"])[:, 1::2] <= tol).all()
    assert (np.abs(f64(o) - r["o"])[:, ::2] <= 2.0**-60 * 2.0**6 * 448).all()
    np.testing.assert_allclose(f64(lse), r["lse"], rtol=2.0**-20, atol=2.0**-10)


@pytest.mark.parametrize("G", [16, 8, 3])
@pytest.mark.parametrize("rising", [True, False])
def test_logits_far_apart_on_pages_of_zeros(cuda_lib, G, rising):
    """Logits that rise or fall by 160 nats along pages of zeros, whose weights
    are too small to show it, in front of ordinary pages at the height of the top."""
    hs2, d, page, T = cuda_lib, 128, 64, 31 * 64
    mp = T // page
    pool = Pool(1, 1, d, page, mp, seed=21).fill([T], seed=22)
    pid, zeros = pool.table[0].long(), mp - 4
    x = torch.linspace(-80, 80, zeros * page).view(zeros, 1, page, 1).expand(zeros, 1, page, d)
    x = (x if rising else x.flip(0, 2)) / math.sqrt(d) * 2**4
    pool.k[pid[:zeros]] = x.to(torch.float8_e4m3fn).view(U8).cuda()
    pool.ks[pid] = 2.0**-4
    pool.v[pid[:zeros]], pool.vs[pid[:zeros]] = 0, 2.0**-126
    pool.k[pid[zeros:]] = torch.tensor(80 / math.sqrt(d) * 2**4).to(torch.float8_e4m3fn).view(U8).cuda()
    for order in (pid, pid.flip(0)):
        pool.table[0] = order.int()
        pool.table_np = pool.table.cpu().numpy()
        check(hs2, pool, torch.ones(1, G, d, dtype=BF, device="cuda"), [T])


def test_nan_codes_in_sight(cuda_lib):
    """A key of NaN makes the outputs of its KV head NaN, a value element of NaN
    its dim; the other heads and sequences keep their bits."""
    hs2, d, page = cuda_lib, 64, 32
    lengths = [900, 500]
    pool = Pool(2, 3, d, page, 29, seed=23).fill(lengths, seed=24)
    q = query(2, 12, d, 25)
    o, lse = hs2.hs2_paged_decode(q, *pool.args(), ints(lengths))
    pool.k[int(pool.table[0, 7]), 1, 3, 5] = 0x7F
    pool.v[int(pool.table[1, 0]), 2, 9, 30] = 0xFF
    o2, lse2 = hs2.hs2_paged_decode(q, *pool.args(), ints(lengths))
    assert status(hs2) == 0
    assert o2[0, 4:8].isnan().all() and lse2[0, 4:8].isnan().all()
    assert o2[1, 8:, 30].isnan().all()
    for x in (o, lse, o2, lse2):
        x[0, 4:8] = 0
    o[1, 8:, 30] = o2[1, 8:, 30] = 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
