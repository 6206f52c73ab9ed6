"""GPU tests of the cache and window operators against the fp64 oracle.

Quantised values and scales are compared exactly.  Attention outputs are held
to bounds made of their roundings, with x = max_s sum_i |q_i k_si| scale, n
visible keys, av = sum_s p_s |v_s|:
  logits   L = (d + 8) 2^-23 x (fp32 products and sums of d terms, on tensor
           cores rounded toward zero); the paged decode also splits q into two
           e4m3 pieces that leave at most 2^-21 max|q| (over the heads that
           share a KV head) of an element
  weights  2^-8 relative (bf16, window) or 2^-9 (nine significant bits, paged),
           and 2^-20 + 4 L for exp2 and the logits; the paged decode drops what
           is below 2^-28 of (largest weight) x (largest V scale), which counts
           for at most 448 times that scale
  o        one rounding to bf16, 2^-8 relative
  lse      L + 2^-20 + n 2^-24 (the fp32 sum) + 2^-22 |lse|
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as ora

pytestmark = pytest.mark.gpu

BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


def ints(v):
    return torch.tensor(list(v), dtype=I32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


def values(codes):
    return ora.e4m3_decode(codes.view(U8).cpu().numpy())


def status(hs2):
    torch.cuda.synchronize()
    return hs2.hs2_get_last_device_error()


def q_top(q, Hkv):
    """[B,Hq]: max|q| over the heads that share a KV head."""
    B, Hq, d = q.shape
    t = q.abs().view(B, Hkv, -1).amax(-1, keepdim=True)
    return f64(t.expand(B, Hkv, Hq // Hkv).reshape(B, Hq))


def check_attention(o, lse, r, q_abs, d, n, weight, split):
    o, lse = f64(o), f64(lse)
    L = (d + 8) * 2.0**-23 * r["x"] + (2.0**-21 * q_abs * r["k1"] if split else 0.0)
    some = np.isfinite(r["lse"])
    tol = (2.0**-8 * np.abs(r["o"]) + (weight + 2.0**-20 + 4 * L)[..., None] * r["av"] * 1.01
           + (n * 2.0**-28 * r["vmax"] if split else 0) + 1e-30)
    np.testing.assert_array_equal(o[~some], 0)
    np.testing.assert_array_equal(lse[~some], r["lse"][~some])
    err = np.abs(o - r["o"])
    assert np.isfinite(o).all() and (err <= tol)[some].all(), float((err / tol)[some].max())
    tl = L + 2.0**-20 + n * 2.0**-24 + 2.0**-22 * np.abs(np.where(some, r["lse"], 0))
    with np.errstate(invalid="ignore"):
        e = np.abs(lse - r["lse"])
    assert (e <= tl)[some].all(), float((e / tl)[some].max())


# ------------------------------------------------------------ the token cache
def token_cache(B, Tmax, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = lambda: torch.randint(0, 256, (B, Tmax, d), generator=g, device="cuda").to(U8)  # noqa: E731
    scale = lambda: torch.rand(B, Tmax, generator=g, device="cuda") + 0.25  # noqa: E731
    return g, codes(), codes(), scale(), scale()


def rows(g, *shape):
    size = torch.exp2(torch.rand(*shape[:-1], 1, generator=g, device="cuda") * 40 - 20)
    return (torch.randn(*shape, generator=g, device="cuda") * size).to(BF)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,N,start,count", [
    (1, 1, [0], None), (3, 1, [0, 7, 99], [1, 0, 1]), (2, 37, [0, 63], [37, 20]), (1, 100, [0], None),
    (2, 63, [5, 37], [0, 1]),
])
def test_token_write_and_read(cuda_lib, d, B, N, start, count):
    hs2, Tmax = cuda_lib, 100
    g, kc, vc, ks, vs = token_cache(B, Tmax, d, 10 * N + d)
    k, v = rows(g, B, N, d), rows(g, B, N, d)
    k[0, 0] = 0
    v[-1, -1] = 2.0**-133  # the smallest subnormal: scale and codes below fp32's normal range
    want = [x.clone() for x in (kc, vc, ks, vs)]
    st = ints(start)
    cn = None if count is None else ints(count)
    n = [N] * B if count is None else count
    hs2.hs2_kv_write(k, v, st, kc, vc, ks, vs, count=cn)
    assert status(hs2) == 0
    for x, cache, scale, c0, s0 in ((k, kc, ks, want[0], want[2]), (v, vc, vs, want[1], want[3])):
        val, sc = values(c0), s0.cpu().numpy()
        for b in range(B):
            at = slice(start[b], start[b] + n[b])
            val[b, at], sc[b, at] = ora.token_quantise(x[b, :n[b]].float().cpu().numpy())
        np.testing.assert_array_equal(scale.cpu().numpy(), sc)
        np.testing.assert_array_equal(values(cache), val)
    # and back; rows past the count stay as they were
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    hs2.hs2_kv_read(kc, vc, ks, vs, st, N, count=cn, k=ko, v=vo)
    assert status(hs2) == 0
    for out, cache, scale in ((ko, kc, ks), (vo, vc, vs)):
        val = values(cache).astype(np.float32) * scale.cpu().numpy()[..., None]
        exp = np.full(out.shape, 7.0, dtype=np.float32)
        for b in range(B):
            exp[b, :n[b]] = ora.bf16_round(val[b, start[b]:start[b] + n[b]])
        np.testing.assert_array_equal(out.float().cpu().numpy(), exp)


def test_token_write_leaves_sequences_out_of_range_alone(cuda_lib):
    hs2 = cuda_lib
    g, kc, vc, ks, vs = token_cache(5, 32, 64, 1)
    k, v = rows(g, 5, 4, 64), rows(g, 5, 4, 64)
    before = [x.clone() for x in (kc, vc, ks, vs)]
    st, cn = ints([-1, 29, 2**31 - 1, 0, 0]), ints([4, 4, 4, 5, -1])
    hs2.hs2_kv_write(k, v, st, kc, vc, ks, vs, count=cn)
    assert status(hs2) == hs2.HS2_ERR_DEVICE_DATA
    for a, b in zip(before, (kc, vc, ks, vs)):
        assert torch.equal(a, b)
    ko = torch.full_like(k, 3.0)
    hs2.hs2_kv_read(kc, vc, ks, vs, st, 4, count=cn, k=ko, v=ko.clone())
    assert status(hs2) == hs2.HS2_ERR_DEVICE_DATA and (ko == 3).all()
    assert status(hs2) == 0


def test_token_write_of_infinities_and_nan(cuda_lib):
    """The finite values of the row keep their precision; the others are flagged."""
    hs2 = cuda_lib
    g, kc, vc, ks, vs = token_cache(1, 8, 128, 2)
    k = torch.randn(1, 2, 128, generator=g, device="cuda").to(BF)
    k[0, 0, 3], k[0, 0, 9], k[0, 0, 40] = math.inf, -math.inf, math.nan
    hs2.hs2_kv_write(k, k, ints([4]), kc, vc, ks, vs)
    assert status(hs2) == hs2.HS2_ERR_DEVICE_DATA
    val, sc = ora.token_quantise(k[0].float().cpu().numpy())
    np.testing.assert_array_equal(values(kc)[0, 4:6], val)
    np.testing.assert_array_equal(ks[0, 4:6].cpu().numpy(), sc)
    assert val[0, 3] == 448 and val[0, 9] == -448 and np.isnan(val[0, 40])


def test_the_decode_layer_reads_what_the_writer_writes(cuda_lib):
    """A cache filled by hs2_kv_write in a prompt and single tokens serves
    hs2_decode_select as the host's recipe does."""
    from token_level_top_hs2_b200 import inputs
    hs2 = cuda_lib
    x = inputs.make_decode(2, 900, 16, 128, 32, 64, kv="bf16", seed=5, n_sparse=1)
    kr, vr = x.k_cache.cuda(), x.v_cache.cuda()
    want = [t for z in (x.k_cache, x.v_cache) for t in inputs.quantize_e4m3_per_token(z)]
    kc, vc = torch.zeros(2, 904, 128, dtype=U8, device="cuda"), torch.zeros(2, 904, 128, dtype=U8, device="cuda")
    ks, vs = torch.zeros(2, 904, device="cuda"), torch.zeros(2, 904, device="cuda")
    hs2.hs2_kv_write(kr[:, :897].contiguous(), vr[:, :897].contiguous(), ints([0, 0]), kc, vc, ks, vs)
    for t in range(897, 900):
        hs2.hs2_kv_write(kr[:, t:t + 1].contiguous(), vr[:, t:t + 1].contiguous(), ints([t, t]), kc, vc, ks, vs)
    o, _, idx = hs2.hs2_decode_select(x.q.cuda(), kc, vc, ints([900, 900]), 32, 64, k_scale=ks, v_scale=vs)
    assert status(hs2) == 0
    for got, w in ((kc, want[0]), (ks, want[1]), (vc, want[2]), (vs, want[3])):
        assert torch.equal(got[:, :900].cpu(), w)
    pad = lambda t: torch.nn.functional.pad(t, (0, 0, 0, 4) if t.dim() == 3 else (0, 4)).cuda()  # noqa: E731
    o2, _, idx2 = hs2.hs2_decode_select(x.q.cuda(), pad(want[0]), pad(want[2]), ints([900, 900]), 32, 64,
                                        k_scale=pad(want[1]), v_scale=pad(want[3]))
    assert torch.equal(o, o2) and torch.equal(idx.sort(-1)[0], idx2.sort(-1)[0])


# ------------------------------------------------------------ the paged cache
class Pool:
    """A pool of pages whose unused rows and scales hold NaN."""

    def __init__(self, B, Hkv, d, page, mp, seed, spare=2):
        g = np.random.default_rng(seed)
        self.B, self.Hkv, self.d, self.page, self.mp, self.P = B, Hkv, d, page, mp, B * mp + spare
        self.table_np = g.permutation(self.P)[:B * mp].reshape(B, mp)
        self.table = torch.from_numpy(self.table_np.astype(np.int32)).cuda()
        full = lambda: torch.full((self.P, Hkv, page, d), 0x7F, dtype=U8, device="cuda")  # noqa: E731
        self.k, self.v = full(), full()
        self.ks, self.vs = (torch.full((self.P, Hkv), math.nan, device="cuda") for _ in "kv")

    def fill(self, lengths, seed, pow2=True):
        """Random codes and scales in every row that a sequence holds."""
        g = torch.Generator().manual_seed(seed)
        for pages, scale in ((self.k, self.ks), (self.v, self.vs)):
            x = (torch.randn(self.P, self.Hkv, self.page, self.d, generator=g) * 60).clamp(-448, 448)
            c = x.to(torch.float8_e4m3fn).view(U8).cuda()
            s = torch.exp2(torch.randint(-8, -3, (self.P, self.Hkv), generator=g).float())
            if not pow2:
                s = s * (torch.rand(self.P, self.Hkv, generator=g) + 0.5)
            for b in range(self.B):
                for j in range(self.mp):
                    n = min(self.page, lengths[b] - j * self.page)
                    if n > 0:
                        p = int(self.table_np[b, j])
                        pages[p, :, :n] = c[p, :, :n]
                        scale[p] = s[p].cuda()
        return self

    def args(self):
        return self.k, self.v, self.ks, self.vs, self.table

    def oracle(self, q, lengths, window, n_sink, scale, table=None):
        return ora.paged_decode(f64(q), values(self.k), values(self.v), f64(self.ks), f64(self.vs),
                                self.table_np if table is None else table, lengths, window, n_sink, scale)


def check_write(hs2, pool, x, start, count, calls=1):
    """One write of K rows x and V rows -x against the oracle."""
    kv, vv = values(pool.k), values(pool.v)
    ks, vs = f64(pool.ks), f64(pool.vs)
    n = [x.shape[1]] * x.shape[0] if count is None else count
    cn = None if count is None else ints(count)
    hs2.hs2_paged_kv_write(x, -x, pool.table, ints(start), pool.k, pool.v, pool.ks, pool.vs, count=cn)
    ora.paged_write(f64(x), pool.table_np, start, n, kv, ks)
    ora.paged_write(-f64(x), pool.table_np, start, n, vv, vs)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(f64(pool.ks), ks)
    np.testing.assert_array_equal(f64(pool.vs), vs)
    np.testing.assert_array_equal(values(pool.k), kv)
    np.testing.assert_array_equal(values(pool.v), vv)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_paged_write_and_read(cuda_lib, d, page, Hkv):
    hs2 = cuda_lib
    pool = Pool(3, Hkv, d, page, 5, seed=page + d)
    g = torch.Generator(device="cuda").manual_seed(page)
    n1 = [2 * page + 3, 0, page]
    check_write(hs2, pool, rows(g, 3, 3 * page, Hkv, d), [0, 0, 0], n1)
    # onto partly filled pages, some of whose scales rise, and over earlier rows
    check_write(hs2, pool, rows(g, 3, page + 5, Hkv, d), [2 * page + 3, 0, page // 2], [page + 5, 1, page])
    for i in range(3):
        check_write(hs2, pool, rows(g, 3, 1, Hkv, d), [3 * page + 8 + i, 1 + i, 3 * page // 2 + i], None)
    assert status(hs2) == 0
    start, n, N = [page // 2, 0, 3], [2 * page, 3, 0], 2 * page
    out = [torch.full((3, N, Hkv, d), 5.0, dtype=BF, device="cuda") for _ in "kv"]
    hs2.hs2_paged_kv_read(*pool.args(), ints(start), N, count=ints(n), k=out[0], v=out[1])
    assert status(hs2) == 0
    for o, pages, scale in ((out[0], pool.k, pool.ks), (out[1], pool.v, pool.vs)):
        exp = np.full(o.shape, 5.0, dtype=np.float32)
        val, sc = values(pages).astype(np.float32), scale.cpu().numpy()
        for b in range(3):
            pos = start[b] + np.arange(n[b])
            pid = pool.table_np[b, pos // page]
            exp[b, :n[b]] = ora.bf16_round(val[pid, :, pos % page] * sc[pid][..., None])
        np.testing.assert_array_equal(o.float().cpu().numpy(), exp)


def test_paged_write_edges(cuda_lib):
    """Zeros, the smallest and largest values, a first row after zeros."""
    hs2 = cuda_lib
    pool = Pool(1, 1, 64, 16, 2, seed=1)
    x = torch.zeros(1, 4, 1, 64, dtype=BF, device="cuda")
    check_write(hs2, pool, x, [0], None)
    x[0, 0, 0, 5], x[0, 2, 0, 9] = 2.0**-133, -2.0**-126
    check_write(hs2, pool, x, [4], None)
    x[0, 1, 0, 7] = 3.0
    check_write(hs2, pool, x, [8], None)
    x[0, 3, 0, 0] = torch.finfo(BF).max
    check_write(hs2, pool, x, [12], None)
    x[:] = torch.finfo(BF).max
    check_write(hs2, pool, -x, [16], None)
    assert status(hs2) == 0


def test_paged_write_flags_and_skips(cuda_lib):
    hs2 = cuda_lib
    pool = Pool(4, 2, 64, 16, 3, seed=2)
    g = torch.Generator(device="cuda").manual_seed(4)
    pool.table[1, 1] = pool.P       # one page behind the pool's end
    pool.table[2, 0] = -1
    pool.table_np = pool.table.cpu().numpy()
    check_write(hs2, pool, rows(g, 4, 20, 2, 64), [0, 8, 0, 29], [20, 20, 20, 20])
    assert status(hs2) == hs2.HS2_ERR_DEVICE_DATA
    out = torch.full((4, 20, 2, 64), 2.0, dtype=BF, device="cuda")
    hs2.hs2_paged_kv_read(*pool.args(), ints([0, 8, 0, 29]), 20, k=out, v=out.clone())
    assert status(hs2) == hs2.HS2_ERR_DEVICE_DATA
    assert (out[1, 8:] == 2).all() and (out[2, :16] == 2).all() and (out[3] == 2).all()
    assert (out[1, :8] != 2).any() and (out[2, 16:] != 2).any()
    # an earlier scale that is not one: replaced, and flagged
    pool.ks[int(pool.table_np[0, 1])] = math.nan
    check_write(hs2, pool, rows(g, 4, 1, 2, 64), [20, 0, 47, 0], [1, 0, 0, 0])
    assert status(hs2) == hs2.HS2_ERR_DEVICE_DATA
    # infinities and NaN
    x = rows(g, 4, 1, 2, 64)
    x[0, 0, 0, 3], x[0, 0, 1, 4] = math.inf, math.nan
    check_write(hs2, pool, x, [21, 0, 0, 0], [1, 0, 0, 0])
    assert status(hs2) == hs2.HS2_ERR_DEVICE_DATA


DECODE = [
    # G, Hkv, d, page, lengths, window, n_sink
    (16, 1, 128, 64, [1, 0, 63, 64, 65, 200], None, 0),
    (16, 1, 64, 16, [1, 15, 16, 17, 127, 128, 129], None, 0),
    (4, 2, 128, 32, [1000, 1, 511], None, 0),
    (8, 3, 64, 128, [700, 129], None, 0),
    (1, 2, 128, 16, [333, 32], None, 0),
    (5, 1, 64, 32, [257, 31, 5000], None, 0),
    (16, 2, 128, 128, [2500, 1300], 128, 4),
    (7, 1, 128, 64, [900, 3, 130], 1, 0),
    (16, 1, 128, 16, [4000, 100], 17, 130),
    (3, 4, 64, 64, [1111, 200], 300, 1),
    (16, 1, 64, 128, [640, 129], 256, 2**31 - 1),
    (2, 1, 128, 64, [20000], None, 0),
    (16, 1, 128, 64, [70000, 40], None, 0),
]


@pytest.mark.parametrize("G,Hkv,d,page,lengths,window,n_sink", DECODE)
def test_paged_decode(cuda_lib, G, Hkv, d, page, lengths, window, n_sink):
    hs2, B = cuda_lib, len(lengths)
    pool = Pool(B, Hkv, d, page, max(1, -(-max(lengths) // page)), seed=G).fill(lengths, seed=d + G, pow2=G != 5)
    # pages that no visible position lies on may name anything
    table = pool.table_np.copy()
    for b, T in enumerate(lengths):
        table[b, -(-T // page):] = -7
    pool.table = torch.from_numpy(table.astype(np.int32)).cuda()
    q = (torch.randn(B, G * Hkv, d, generator=torch.Generator().manual_seed(G)) * 1.5).to(BF).cuda()
    o, lse = hs2.hs2_paged_decode(q, *pool.args(), ints(lengths), window=window, n_sink=n_sink)
    assert status(hs2) == 0
    w = 2**31 - 1 if window is None else window
    r = pool.oracle(q, lengths, w, n_sink, 1 / math.sqrt(d), table)
    n = max(min(T, w + n_sink) for T in lengths)
    check_attention(o, lse, r, q_top(q, Hkv), d, n, 2.0**-9, True)
    o2, none = hs2.hs2_paged_decode(q, *pool.args(), ints(lengths), window=window, n_sink=n_sink,
                                    want_lse=False)
    assert none is None and torch.equal(o, o2)  # the same bits every time


@pytest.mark.parametrize("spread", [0.0, 40.0])
def test_paged_decode_of_needles_and_flat_rows(cuda_lib, spread):
    """Logits from all equal to 2^57 apart, rising along the sequence."""
    hs2, T, d, G = cuda_lib, 3000, 128, 16
    pool = Pool(1, 1, d, 64, 47, seed=3).fill([T], seed=8)
    q = torch.ones(1, G, d, dtype=BF, device="cuda")
    if spread:
        x = torch.linspace(-spread / 2, spread / 2, 47 * 64).view(47, 1, 64, 1).expand(47, 1, 64, d)
        x = x + torch.rand(47, 1, 64, d, generator=torch.Generator().manual_seed(1))
        pool.k[pool.table[0].long()] = (x / math.sqrt(d) * 2**6).to(torch.float8_e4m3fn).view(U8).cuda()
        pool.ks[:] = 2.0**-6
    else:
        pool.k[:] = 0x30  # 0.5
    o, lse = hs2.hs2_paged_decode(q, *pool.args(), ints([T]))
    assert status(hs2) == 0
    r = pool.oracle(q, [T], 2**31 - 1, 0, 1 / math.sqrt(d))
    check_attention(o, lse, r, np.ones((1, G)), d, T, 2.0**-9, True)


def test_paged_decode_of_uneven_value_scales(cuda_lib):
    """V scales that differ by 2^30 between pages, and one of 2^-126 (a page of zeros)."""
    hs2, d, G, T = cuda_lib, 64, 4, 1000
    pool = Pool(1, 1, d, 32, 32, seed=5).fill([T], seed=9)
    pid = pool.table[0].long()
    pool.vs[pid] = torch.exp2(torch.arange(32, device="cuda").float() - 20)[:, None]
    pool.vs[pid[3]], pool.v[pid[3]] = 2.0**-126, 0
    q = torch.randn(1, G, d, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    o, lse = hs2.hs2_paged_decode(q, *pool.args(), ints([T]))
    assert status(hs2) == 0
    r = pool.oracle(q, [T], 2**31 - 1, 0, 1 / math.sqrt(d))
    check_attention(o, lse, r, q_top(q, 1), d, T, 2.0**-9, True)


def test_paged_decode_flags_bad_lengths_and_pages(cuda_lib):
    hs2, d, page = cuda_lib, 128, 64
    lengths = [100, 257, -1, 200]
    pool = Pool(4, 1, d, page, 4, seed=4).fill([100, 256, 0, 200], seed=1)
    table = pool.table_np.copy()
    table[3, 1] = pool.P
    pool.table = torch.from_numpy(table.astype(np.int32)).cuda()
    q = torch.randn(4, 16, d, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    o, lse = hs2.hs2_paged_decode(q, *pool.args(), ints(lengths))
    assert status(hs2) == hs2.HS2_ERR_DEVICE_DATA
    r = pool.oracle(q, lengths, 2**31 - 1, 0, 1 / math.sqrt(d), table)
    check_attention(o, lse, r, q_top(q, 1), d, 256, 2.0**-9, True)
    assert status(hs2) == 0


def test_paged_decode_of_a_pool_past_4_gib(cuda_lib):
    hs2, d, page, Hkv = cuda_lib, 128, 128, 1
    P = 2**32 // (page * d) + 40
    if torch.cuda.mem_get_info()[0] < 3 * 2**32:
        pytest.skip("needs 12 GiB of device memory")
    k, v = (torch.empty(P, Hkv, page, d, dtype=U8, device="cuda") for _ in "kv")
    small = Pool(1, Hkv, d, page, 12, seed=6).fill([1500], seed=4)
    ks, vs = (torch.empty(P, Hkv, device="cuda") for _ in "kv")
    far = torch.tensor([0] + [P - 1 - 3 * i for i in range(11)], device="cuda")
    pid = small.table[0].long()
    k[far], v[far], ks[far], vs[far] = small.k[pid], small.v[pid], small.ks[pid], small.vs[pid]
    q = torch.randn(1, 16, d, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    table = far.to(I32).view(1, -1)
    o, lse = hs2.hs2_paged_decode(q, k, v, ks, vs, table, ints([1500]))
    o1, lse1 = hs2.hs2_paged_decode(q, *small.args(), ints([1500]))
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    x = torch.randn(1, 40, 1, d, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
    hs2.hs2_paged_kv_write(x, x, table, ints([1480]), k, v, ks, vs)
    hs2.hs2_paged_kv_write(x, x, small.table, ints([1480]), small.k, small.v, small.ks, small.vs)
    got = hs2.hs2_paged_kv_read(k, v, ks, vs, table, ints([0]), 1520)
    want = hs2.hs2_paged_kv_read(*small.args(), ints([0]), 1520)
    assert status(hs2) == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_paged_decode_captured_and_on_two_streams(cuda_lib):
    """Replays follow the lengths and the cache; calls on two streams with
    workspaces of their own do not disturb one another."""
    hs2, d, G = cuda_lib, 128, 16
    pool = Pool(2, 1, d, 64, 40, seed=7).fill([2560, 2560], seed=2)
    q = torch.randn(2, G, d, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    lengths = ints([2000, 5])
    shape = hs2.paged_shape(2, 1, d, 64, pool.P, 40)
    ws = [torch.empty(hs2.hs2_paged_decode_workspace(shape, G), dtype=U8, device="cuda") for _ in range(2)]
    o, lse = torch.empty_like(q), torch.empty(2, G, device="cuda")
    call = lambda i, o, l, s=None: hs2.hs2_paged_decode(  # noqa: E731
        q, *pool.args(), lengths, o=o, lse=l, workspace=ws[i], stream=s)
    call(0, o, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0, o, lse)
    for lens in ([2000, 5], [1, 2560], [0, 700]):
        lengths.copy_(ints(lens))
        o.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        r = pool.oracle(q, lens, 2**31 - 1, 0, 1 / math.sqrt(d))
        check_attention(o, lse, r, q_top(q, 1), d, 2560, 2.0**-9, True)
    lengths.copy_(ints([2560, 2200]))
    call(0, o, lse)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(q), torch.empty_like(lse)) for _ in range(2)]
    for _ in range(20):
        for i, s in enumerate(streams):
            call(i, *outs[i], s)
    torch.cuda.synchronize()
    assert status(hs2) == 0
    for a, b in outs:
        assert torch.equal(a, o) and torch.equal(b, lse)


# ------------------------------------------------------------------ the window
WINDOW = [
    # B, Lq, Lk, G, Hkv, d, window, n_sink
    (1, 1, 1, 16, 1, 128, 1, 0),
    (1, 1, 300, 4, 2, 128, 128, 4),
    (2, 5, 5, 16, 1, 64, 3, 1),
    (1, 128, 128, 16, 1, 128, 128, 0),
    (1, 257, 257, 16, 1, 128, 128, 4),
    (1, 200, 777, 8, 2, 64, 100, 16),
    (2, 100, 333, 3, 1, 128, 40, 5),
    (1, 300, 300, 1, 3, 64, 1, 0),
    (1, 400, 400, 1, 2, 128, 130, 129),
    (1, 300, 300, 7, 1, 64, 64, 0),
    (1, 333, 333, 4, 1, 64, 2**31 - 1, 0),
    (1, 260, 400, 2, 1, 128, 17, 2**31 - 1),
    (1, 64, 1500, 5, 2, 128, 1000, 300),
    (1, 700, 700, 16, 1, 128, 513, 4),
]


@pytest.mark.parametrize("B,Lq,Lk,G,Hkv,d,window,n_sink", WINDOW)
def test_window_attn(cuda_lib, B, Lq, Lk, G, Hkv, d, window, n_sink):
    hs2 = cuda_lib
    g = torch.Generator().manual_seed(Lq + G)
    q = (torch.randn(B, Lq, G * Hkv, d, generator=g) * 1.5).to(BF).cuda()
    k, v = (torch.randn(B, Lk, Hkv, d, generator=g).to(BF).cuda() for _ in "kv")
    o, lse = hs2.hs2_window_attn(q, k, v, window, n_sink)
    assert status(hs2) == 0
    r = ora.window_attn(f64(q), f64(k), f64(v), window, n_sink, 1 / math.sqrt(d))
    check_attention(o, lse, r, None, d, min(Lk, window + n_sink), 2.0**-8, False)
    o2, none = hs2.hs2_window_attn(q, k, v, window, n_sink, want_lse=False)
    assert none is None and torch.equal(o, o2)


def test_window_attn_of_a_long_prompt(cuda_lib):
    hs2, L, G, d, window, n_sink = cuda_lib, 20000, 16, 128, 700, 4
    g = torch.Generator().manual_seed(1)
    q = (torch.randn(1, L, G, d, generator=g) * 1.5).to(BF)
    k, v = (torch.randn(1, L, 1, d, generator=g).to(BF) for _ in "kv")
    o, lse = hs2.hs2_window_attn(q.cuda(), k.cuda(), v.cuda(), window, n_sink)
    assert status(hs2) == 0
    at = sorted({0, 1, 699, 700, 701, 703, 704, 705, L - 1, L - 2} | set(range(37, L, 997)))
    r = ora.window_attn(f64(q), f64(k), f64(v), window, n_sink, 1 / math.sqrt(d), rows=at)
    check_attention(o[:, at], lse[:, at], r, None, d, 704, 2.0**-8, False)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, torch.finfo(BF).max])
def test_window_attn_never_uses_rows_a_query_does_not_see(cuda_lib, bad):
    """Rows of padding, rows behind the window and rows between the sinks and
    the window hold anything; the rows that see them are not compared."""
    hs2, L, G, d, window, n_sink = cuda_lib, 500, 4, 128, 60, 3
    g = torch.Generator().manual_seed(2)
    q = torch.randn(2, L, G, d, generator=g).to(BF).cuda()
    k, v = (torch.randn(2, L, 1, d, generator=g).to(BF).cuda() for _ in "kv")
    want = ora.window_attn(f64(q), f64(k), f64(v), window, n_sink, 1 / math.sqrt(d))
    k2, v2 = k.clone(), v.clone()
    for b, at in ((0, [140, 141, 300]), (1, [400 + i for i in range(100)])):
        k2[b, at], v2[b, at] = bad, bad
    o, lse = hs2.hs2_window_attn(q, k2, v2, window, n_sink)
    assert status(hs2) == 0
    seen = np.zeros((2, L), dtype=bool)
    for s in (140, 141, 300):
        seen[0, s:s + window] = True
    seen[1, 400:] = True
    keep = {n: x[~seen] for n, x in want.items()}
    check_attention(o[torch.from_numpy(~seen)], lse[torch.from_numpy(~seen)], keep, None, d, window + n_sink,
                    2.0**-8, False)
    if math.isnan(bad):
        assert o[torch.from_numpy(seen)].isnan().all()


def test_window_attn_of_sharp_rows_and_large_logits(cuda_lib):
    hs2, L, d = cuda_lib, 400, 64
    g = torch.Generator().manual_seed(4)
    q = (torch.randn(1, L, 8, d, generator=g) * 30).to(BF).cuda()
    k, v = (torch.randn(1, L, 2, d, generator=g).to(BF).cuda() for _ in "kv")
    k[:, ::7] *= 4
    o, lse = hs2.hs2_window_attn(q, k, v, 150, 8)
    assert status(hs2) == 0
    r = ora.window_attn(f64(q), f64(k), f64(v), 150, 8, 1 / math.sqrt(d))
    check_attention(o, lse, r, None, d, 158, 2.0**-8, False)


def test_window_attn_of_keys_past_4_gib(cuda_lib):
    hs2, d, Lk = cuda_lib, 128, 2**24 + 1000
    if torch.cuda.mem_get_info()[0] < 3 * 2**32:
        pytest.skip("needs 12 GiB of device memory")
    g = torch.Generator().manual_seed(5)
    k, v = (torch.empty(1, Lk, 1, d, dtype=BF, device="cuda") for _ in "kv")
    ks, vs = (torch.randn(1, 304, 1, d, generator=g).to(BF).cuda() for _ in "kv")
    for big, small in ((k, ks), (v, vs)):
        big[:, :4], big[:, -300:] = small[:, :4], small[:, 4:]
    q = torch.randn(1, 100, 4, d, generator=g).to(BF).cuda()
    o, lse = hs2.hs2_window_attn(q, k, v, 128, 4)
    o1, lse1 = hs2.hs2_window_attn(q, ks, vs, 128, 4)
    assert status(hs2) == 0
    np.testing.assert_allclose(f64(o), f64(o1), rtol=2.0**-7, atol=2.0**-8)
    np.testing.assert_allclose(f64(lse), f64(lse1), atol=1e-4)


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("d,Hkv,G,page", [(128, 1, 16, 64), (64, 2, 3, 16)])
def test_a_prompt_in_chunks_then_decode_steps(cuda_lib, d, Hkv, G, page):
    """A window layer as a server runs it: each chunk of the prompt attends to
    the cached rows read back and its own, its rows are written to the pages,
    then tokens are decoded one by one; on a side stream, as captured steps."""
    hs2, window, n_sink = cuda_lib, 90, 4
    L, steps, chunks = 300, 5, [0, 128, 211, 300]
    g = torch.Generator().manual_seed(7)
    n = L + steps
    q = (torch.randn(1, n, G * Hkv, d, generator=g) * 1.5).to(BF).cuda()
    k, v = (torch.randn(1, n, Hkv, d, generator=g).to(BF).cuda() for _ in "kv")
    pool = Pool(1, Hkv, d, page, -(-n // page), seed=8)
    cache = (pool.k, pool.v, pool.ks, pool.vs)
    scale = 1 / math.sqrt(d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for a, b in zip(chunks, chunks[1:]):
            if a:
                kr, vr = hs2.hs2_paged_kv_read(*cache, pool.table, ints([0]), a)
            else:
                kr, vr = k[:, :0], v[:, :0]
            kk, vv = torch.cat([kr, k[:, a:b]], 1), torch.cat([vr, v[:, a:b]], 1)
            o, lse = hs2.hs2_window_attn(q[:, a:b].contiguous(), kk, vv, window, n_sink)
            r = ora.window_attn(f64(q[:, a:b]), f64(kk), f64(vv), window, n_sink, scale)
            check_attention(o, lse, r, None, d, window + n_sink, 2.0**-8, False)
            hs2.hs2_paged_kv_write(k[:, a:b].contiguous(), v[:, a:b].contiguous(), pool.table, ints([a]), *cache)
        at, length = ints([L]), ints([L + 1])
        kn, vn, qn = k[:, L:L + 1].clone(), v[:, L:L + 1].clone(), q[:, L].clone()
        on, ln = torch.empty_like(qn), torch.empty(1, G * Hkv, device="cuda")
        ws = torch.empty(hs2.hs2_paged_decode_workspace(
            hs2.paged_shape(1, Hkv, d, page, pool.P, pool.mp), G * Hkv), dtype=U8, device="cuda")

        def step():
            hs2.hs2_paged_kv_write(kn, vn, pool.table, at, *cache)
            hs2.hs2_paged_decode(qn, *cache, pool.table, length, window=window, n_sink=n_sink, o=on, lse=ln,
                                 workspace=ws)

        kv0 = [x.clone() for x in cache]
        step()
        torch.cuda.synchronize()
        for x, y in zip(cache, kv0):
            x.copy_(y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        for t in range(L, n):
            kn.copy_(k[:, t:t + 1]), vn.copy_(v[:, t:t + 1]), qn.copy_(q[:, t])
            at.fill_(t), length.fill_(t + 1)
            graph.replay()
            torch.cuda.synchronize()
            r = pool.oracle(qn, [t + 1], window, n_sink, scale)
            check_attention(on, ln, r, q_top(qn, Hkv), d, window + n_sink, 2.0**-9, True)
    assert status(hs2) == 0


def test_window_attn_of_a_batch_padded_with_nan(cuda_lib):
    """Whole padding, keys, values and queries, of NaN: the padding's own rows
    come out NaN and quickly, the others as if it were not there."""
    hs2, L, G, d, window = cuda_lib, 6000, 4, 64, 5000
    g = torch.Generator().manual_seed(6)
    q = torch.randn(2, L, G, d, generator=g).to(BF).cuda()
    k, v = (torch.randn(2, L, 1, d, generator=g).to(BF).cuda() for _ in "kv")
    o, lse = hs2.hs2_window_attn(q, k, v, window, 2)
    n = 2345
    for x in (q, k, v):
        x[1, n:] = math.nan
    o2, lse2 = hs2.hs2_window_attn(q, k, v, window, 2)
    assert status(hs2) == 0
    assert torch.equal(o2[0], o[0]) and torch.equal(lse2[0], lse[0])
    assert o2[1, n:].isnan().all() and lse2[1, n:].isnan().all()
    np.testing.assert_allclose(f64(o2[1, :n]), f64(o[1, :n]), rtol=2.0**-7, atol=2.0**-8)
    np.testing.assert_allclose(f64(lse2[1, :n]), f64(lse[1, :n]), atol=1e-4)


def test_two_window_calls_at_once_and_one_replayed(cuda_lib):
    """Calls on two streams, and a captured call replayed with other inputs."""
    hs2, L, G, d = cuda_lib, 3000, 8, 128
    g = torch.Generator().manual_seed(8)
    q = torch.randn(1, L, G, d, generator=g).to(BF).cuda()
    k, v = (torch.randn(1, L, 1, d, generator=g).to(BF).cuda() for _ in "kv")
    want = hs2.hs2_window_attn(q, k, v, 300, 4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(q), torch.empty(1, L, G, device="cuda")) for _ in range(2)]
    for _ in range(10):
        for (o, lse), s in zip(outs, streams):
            hs2.hs2_window_attn(q, k, v, 300, 4, o=o, lse=lse, stream=s)
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    o, lse = outs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs2.hs2_window_attn(q, k, v, 300, 4, o=o, lse=lse)
    q.mul_(0.5)
    graph.replay()
    want = hs2.hs2_window_attn(q, k, v, 300, 4)
    torch.cuda.synchronize()
    assert status(hs2) == 0 and torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("B,lengths", [(1, [0]), (3, [0, 0, 0]), (200, None)])
def test_paged_decode_of_empty_and_many_sequences(cuda_lib, B, lengths):
    """No tokens at all, and more sequences than a warp scans at once, most
    items smaller than a CTA's share."""
    hs2, d, Hkv, G, page = cuda_lib, 64, 2, 3, 16
    if lengths is None:
        lengths = [(37 * i) % 300 if i % 3 else 0 for i in range(B)]
    pool = Pool(B, Hkv, d, page, max(1, -(-max(lengths) // page)), seed=B).fill(lengths, seed=B)
    q = torch.randn(B, G * Hkv, d, generator=torch.Generator().manual_seed(B)).to(BF).cuda()
    o, lse = torch.full_like(q, 7.0), torch.full((B, G * Hkv), 7.0, device="cuda")
    hs2.hs2_paged_decode(q, *pool.args(), ints(lengths), o=o, lse=lse)
    assert status(hs2) == 0
    r = pool.oracle(q, lengths, 2**31 - 1, 0, 1 / math.sqrt(d))
    check_attention(o, lse, r, q_top(q, Hkv), d, 300, 2.0**-9, True)


def test_calls_on_a_side_stream_keep_their_memory(cuda_lib):
    """What a call allocates for another stream is not reused under it."""
    hs2, L, G, d = cuda_lib, 2000, 16, 128
    g = torch.Generator().manual_seed(9)
    q = torch.randn(1, L, G, d, generator=g).to(BF).cuda()
    k, v = (torch.randn(1, L, 1, d, generator=g).to(BF).cuda() for _ in "kv")
    pool = Pool(4, 1, d, 64, 40, seed=9).fill([2500] * 4, seed=9)
    qd = torch.randn(4, G, d, generator=g).to(BF).cuda()
    want, dec = hs2.hs2_window_attn(q, k, v, 400, 0)[0], hs2.hs2_paged_decode(qd, *pool.args(), ints([2500] * 4))[0]
    lengths = ints([2500] * 4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        o = hs2.hs2_window_attn(q, k, v, 400, 0, stream=s)[0]
        od = hs2.hs2_paged_decode(qd, *pool.args(), lengths, stream=s)[0]
        junk = [torch.full((1 << 20,), 9.0, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        del junk
        assert torch.equal(o, want) and torch.equal(od, dec)
