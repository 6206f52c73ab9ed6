"""CPU tests of the cache and window operators: their fp64 oracle against
independent computations, and the C ABI's and the binding's refusals."""
import ctypes

import numpy as np
import pytest
import torch

import token_level_top_hs2_b200 as hs2
from oracle import cache_ops as ora
from token_level_top_hs2_b200 import build as hs2_build
from token_level_top_hs2_b200 import inputs

FAKE = 1 << 20  # 16-byte aligned non-null stand-in: never dereferenced on failure


@pytest.fixture(scope="module")
def lib():
    hs2_build.build()
    return hs2.load()


# ----------------------------------------------------------------- the oracle
def test_e4m3_rounding_and_decoding_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(ora.e4m3_decode(codes), want)
    g = np.random.default_rng(0)
    x = np.concatenate([g.normal(size=20000) * np.exp2(g.uniform(-12, 9, 20000)),
                        np.arange(-448, 449) / 64.0, np.arange(0, 64) * 2.0**-11]).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(ora.e4m3_round(x), want)


def test_token_quantisation_matches_the_input_recipe():
    x = torch.randn(300, 128, generator=torch.Generator().manual_seed(1)) * 3
    x[7] = 0
    codes, s = inputs.quantize_e4m3_per_token(x)
    v, so = ora.token_quantise(x.numpy())
    np.testing.assert_array_equal(so, s.numpy())
    np.testing.assert_array_equal(v, codes.view(torch.float8_e4m3fn).float().numpy())


def test_page_power_is_the_least_that_fits():
    for top in [1e-40, 2.0**-130, 1.0, 448.0, 449.0, 447.0, 896.0, 1e5, 3e38]:
        p = ora.page_power(top)
        assert top <= 448 * p and (p == 2.0**-126 or top > 448 * p / 2)
    assert ora.page_power(0.0) == 2.0**-126


def test_paged_write_in_pieces_equals_at_once_without_subnormals():
    """Powers of two rescale exactly, so appending row by row ends where one call
    does as long as nothing is rounded below e4m3's normal range."""
    g = np.random.default_rng(3)
    B, N, H, page, d = 1, 40, 2, 16, 8
    x = (g.integers(8, 16, (B, N, H, d)) * np.exp2(g.integers(-2, 4, (B, N, H, d)))
         * g.choice([-1, 1], (B, N, H, d))).astype(np.float64)
    table = np.array([[2, 0, 1]])
    a, sa = np.zeros((3, H, page, d)), np.full((3, H), np.nan)
    ora.paged_write(x, table, [0], [N], a, sa)
    b, sb = np.zeros((3, H, page, d)), np.full((3, H), np.nan)
    for i in range(N):
        ora.paged_write(x[:, i:i + 1], table, [i], [1], b, sb)
    np.testing.assert_array_equal(sa, sb)
    np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (5, 0), (5, 3), (100, 0), (3, 100), (100, 100)])
def test_window_oracle_matches_a_masked_softmax(window, n_sink):
    g = torch.Generator().manual_seed(5)
    B, Lq, Lk, Hq, Hkv, d = 2, 9, 23, 6, 2, 8
    q, k, v = (torch.randn(B, L, H, d, generator=g, dtype=torch.float64)
               for L, H in ((Lq, Hq), (Lk, Hkv), (Lk, Hkv)))
    r = ora.window_attn(q.numpy(), k.numpy(), v.numpy(), window, n_sink, 0.3)
    t = torch.arange(Lk - Lq, Lk).view(-1, 1)
    s = torch.arange(Lk)
    seen = (s <= t) & ((s > t - window) | (s < n_sink))
    kk, vv = (z.repeat_interleave(Hq // Hkv, 2) for z in (k, v))
    x = torch.einsum("bihd,bshd->bhis", q, kk) * 0.3
    x = x.masked_fill(~seen, float("-inf"))
    o = torch.einsum("bhis,bshd->bihd", torch.softmax(x, -1), vv)
    np.testing.assert_allclose(r["o"], o.numpy(), atol=1e-13)
    np.testing.assert_allclose(r["lse"], torch.logsumexp(x, -1).transpose(1, 2).numpy(), atol=1e-13)


def test_paged_oracle_is_the_window_oracle_through_pages():
    g = np.random.default_rng(6)
    B, Hq, Hkv, page, d, mp = 2, 4, 2, 4, 8, 3
    table = np.array([[5, 1, 3], [0, 4, 2]])
    kp, vp = (ora.e4m3_round(g.normal(size=(6, Hkv, page, d)) * 9) for _ in "kv")
    ks, vs = (np.exp2(g.integers(-3, 3, (6, Hkv))) for _ in "kv")
    q = g.normal(size=(B, Hq, d))
    lengths = [11, 6]
    r = ora.paged_decode(q, kp, vp, ks, vs, table, lengths, 4, 2, 0.4)
    for b, T in enumerate(lengths):
        k, v = (np.concatenate([z[p].transpose(1, 0, 2) * s[p][None, :, None] for p in table[b]])[:T]
                for z, s in ((kp, ks), (vp, vs)))
        w = ora.window_attn(q[b][None, None], k[None], v[None], 4, 2, 0.4)
        np.testing.assert_allclose(r["o"][b], w["o"][0, 0], atol=1e-13)
        np.testing.assert_allclose(r["lse"][b], w["lse"][0, 0], atol=1e-13)
    bad = table.copy()
    bad[0, 1] = 6
    r = ora.paged_decode(q, kp, vp, ks, vs, bad, [4, 0], 100, 0, 0.4)
    assert np.isneginf(r["lse"][1]).all() and not r["o"][1].any()
    whole = ora.paged_decode(q, kp, vp, ks, vs, table, [4, 0], 100, 0, 0.4)
    np.testing.assert_array_equal(
        ora.paged_decode(q, kp, vp, ks, vs, bad, [8, 0], 100, 0, 0.4)["o"][0], whole["o"][0])


# ------------------------------------------------------------------- refusals
PTR = [FAKE] * 16


def token(B=2, Tmax=64, d=128):
    return hs2.CacheShape(B, Tmax, d)


def paged(B=2, Hkv=2, d=128, page=64, n_pages=8, max_pages=4):
    return hs2.PagedShape(B, Hkv, d, page, n_pages, max_pages)


@pytest.mark.parametrize("fields,N,code", [
    (dict(B=0), 1, hs2.HS2_ERR_INVALID_ARG),
    (dict(B=65536), 1, hs2.HS2_ERR_INVALID_ARG),
    (dict(Tmax=0), 1, hs2.HS2_ERR_INVALID_ARG),
    (dict(d=96), 1, hs2.HS2_ERR_UNSUPPORTED),
    (dict(Tmax=2**31 - 1), 1, hs2.HS2_ERR_UNSUPPORTED),
    (dict(), 0, hs2.HS2_ERR_INVALID_ARG),
    (dict(), 65, hs2.HS2_ERR_INVALID_ARG),
])
def test_token_calls_reject_bad_shapes(lib, fields, N, code):
    for f in (lib.hs2_kv_write, lib.hs2_kv_read):
        assert f(token(**fields), N, *PTR[:8], None) == code


def test_token_calls_reject_bad_pointers(lib):
    for f, optional in ((lib.hs2_kv_write, 3), (lib.hs2_kv_read, 5)):
        assert f(None, 1, *PTR[:8], None) == hs2.HS2_ERR_INVALID_ARG
        for i in range(8):
            a = list(PTR[:8])
            a[i] = FAKE + 4
            assert f(token(), 1, *a, None) == hs2.HS2_ERR_INVALID_ARG, i
            if i != optional:
                a[i] = None
                assert f(token(), 1, *a, None) == hs2.HS2_ERR_INVALID_ARG, i


BAD_PAGED = [
    (dict(B=0), hs2.HS2_ERR_INVALID_ARG),
    (dict(Hkv=0), hs2.HS2_ERR_INVALID_ARG),
    (dict(n_pages=0), hs2.HS2_ERR_INVALID_ARG),
    (dict(max_pages=0), hs2.HS2_ERR_INVALID_ARG),
    (dict(page=0), hs2.HS2_ERR_INVALID_ARG),
    (dict(page=48), hs2.HS2_ERR_UNSUPPORTED),
    (dict(page=256), hs2.HS2_ERR_UNSUPPORTED),
    (dict(d=32), hs2.HS2_ERR_UNSUPPORTED),
    (dict(max_pages=2**25), hs2.HS2_ERR_UNSUPPORTED),
    (dict(max_pages=2**25 - 1), hs2.HS2_ERR_UNSUPPORTED),     # positions up to 2^31 - 64
    (dict(n_pages=2**30, Hkv=2), hs2.HS2_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("fields,code", BAD_PAGED)
def test_paged_calls_reject_bad_shapes(lib, fields, code):
    s = paged(**fields)
    assert lib.hs2_paged_kv_write(s, 1, *PTR[:9], None) == code
    assert lib.hs2_paged_kv_read(s, 1, *PTR[:9], None) == code
    assert lib.hs2_paged_decode_workspace(s, 4) == 0
    assert lib.hs2_paged_decode(s, 4 * max(1, fields.get("Hkv", 1)), 8, 0, 0.1, *PTR[:10], 1 << 40,
                                None) == code


def test_paged_calls_reject_bad_arguments(lib):
    s = paged()
    for f, optional in ((lib.hs2_paged_kv_write, 4), (lib.hs2_paged_kv_read, 6)):
        assert f(None, 1, *PTR[:9], None) == hs2.HS2_ERR_INVALID_ARG
        assert f(s, 0, *PTR[:9], None) == hs2.HS2_ERR_INVALID_ARG
        assert f(s, 4 * 64 + 1, *PTR[:9], None) == hs2.HS2_ERR_INVALID_ARG
        for i in range(9):
            a = list(PTR[:9])
            a[i] = FAKE + 8
            assert f(s, 1, *a, None) == hs2.HS2_ERR_INVALID_ARG, i
            if i != optional:
                a[i] = None
                assert f(s, 1, *a, None) == hs2.HS2_ERR_INVALID_ARG, i
    need = lib.hs2_paged_decode_workspace(s, 4)
    assert need > 0

    def decode(Hq=4, window=8, n_sink=0, scale=0.1, args=PTR[:10], ws=need):
        return lib.hs2_paged_decode(s, Hq, window, n_sink, scale, *args, ws, None)

    assert decode(Hq=3) == hs2.HS2_ERR_INVALID_ARG          # not a multiple of Hkv
    assert decode(Hq=0) == hs2.HS2_ERR_INVALID_ARG
    assert decode(Hq=34) == hs2.HS2_ERR_UNSUPPORTED         # 17 per KV head
    assert decode(window=0) == hs2.HS2_ERR_INVALID_ARG
    assert decode(n_sink=-1) == hs2.HS2_ERR_INVALID_ARG
    for scale in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert decode(scale=scale) == hs2.HS2_ERR_INVALID_ARG
    assert decode(ws=need - 1) == hs2.HS2_ERR_WORKSPACE
    crowd = hs2.PagedShape(65535, 64, 64, 128, 1, 8192)  # 2^35 tiles of 128 tokens and more
    assert lib.hs2_paged_decode(crowd, 64, 2**31 - 1, 0, 0.1, *PTR[:10], 1 << 30, None) \
        == hs2.HS2_ERR_UNSUPPORTED
    for i in range(10):
        a = list(PTR[:10])
        a[i] = FAKE + 4
        assert decode(args=a) == hs2.HS2_ERR_INVALID_ARG, i
        if i != 8:  # lse
            a[i] = None
            assert decode(args=a) == hs2.HS2_ERR_INVALID_ARG, i


@pytest.mark.parametrize("fields,code", [
    (dict(B=0), hs2.HS2_ERR_INVALID_ARG),
    (dict(B=65536), hs2.HS2_ERR_INVALID_ARG),
    (dict(Lq=0), hs2.HS2_ERR_INVALID_ARG),
    (dict(Lq=65), hs2.HS2_ERR_INVALID_ARG),                 # more queries than positions
    (dict(window=0), hs2.HS2_ERR_INVALID_ARG),
    (dict(n_sink=-1), hs2.HS2_ERR_INVALID_ARG),
    (dict(scale=0.0), hs2.HS2_ERR_INVALID_ARG),
    (dict(scale=float("inf")), hs2.HS2_ERR_INVALID_ARG),
    (dict(scale=3e38), hs2.HS2_ERR_INVALID_ARG),
    (dict(Hq=5), hs2.HS2_ERR_INVALID_ARG),
    (dict(Hkv=0), hs2.HS2_ERR_INVALID_ARG),
    (dict(Hq=34), hs2.HS2_ERR_UNSUPPORTED),
    (dict(d=256), hs2.HS2_ERR_UNSUPPORTED),
    (dict(Lk=2**31 - 1), hs2.HS2_ERR_UNSUPPORTED),
    (dict(Lq=2**28, Lk=2**28, Hq=16, Hkv=1), hs2.HS2_ERR_UNSUPPORTED),  # 2^32 rows
])
def test_window_rejects_bad_shapes(lib, fields, code):
    base = dict(B=1, Lq=16, Lk=64, Hq=4, Hkv=2, d=128, window=8, n_sink=0, scale=0.1)
    base.update(fields)
    assert lib.hs2_window_attn(hs2.WindowShape(**base), *PTR[:5], None) == code


def test_window_rejects_bad_pointers(lib):
    s = hs2.WindowShape(1, 16, 64, 4, 2, 128, 8, 0, 0.1)
    assert lib.hs2_window_attn(None, *PTR[:5], None) == hs2.HS2_ERR_INVALID_ARG
    for i in range(5):
        a = list(PTR[:5])
        a[i] = FAKE + 2
        assert lib.hs2_window_attn(s, *a, None) == hs2.HS2_ERR_INVALID_ARG, i
        if i != 4:
            a[i] = None
            assert lib.hs2_window_attn(s, *a, None) == hs2.HS2_ERR_INVALID_ARG, i


def test_binding_refuses_host_strided_mistyped_and_misshaped_tensors(monkeypatch, lib):
    monkeypatch.setattr(hs2, "_current_device", lambda: 0)
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    rows, cache = torch.zeros(2, 4, 128, dtype=bf), torch.zeros(2, 64, 128, dtype=u8)
    sc, st = torch.zeros(2, 64), torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="k_new: must be a CUDA tensor"):
        hs2.hs2_kv_write(rows, rows, st, cache, cache, sc, sc)
    with pytest.raises(ValueError, match="k_cache: must be a CUDA tensor"):
        hs2.hs2_kv_read(cache, cache, sc, sc, st, 4)
    with pytest.raises(ValueError, match="k_cache: 2 dimensions, expected 3"):
        hs2.hs2_kv_read(cache[0], cache, sc, sc, st, 4)
    with pytest.raises(TypeError, match="q: expected a torch.Tensor"):
        hs2.hs2_window_attn([0], rows, rows, 4)
    with pytest.raises(ValueError, match="v_new: must be contiguous"):
        hs2._dense(rows.transpose(0, 1), "v_new", (bf,), (4, 2, 128), 0)
    with pytest.raises(TypeError, match="v_new: dtype torch.float32"):
        hs2._dense(rows.float(), "v_new", (bf,), rows.shape, 0)
    with pytest.raises(ValueError, match=r"v_new: shape \(2, 4, 128\), expected \(2, 5, 128\)"):
        hs2._dense(rows, "v_new", (bf,), (2, 5, 128), 0)
    with pytest.raises(ValueError, match="v_new: must be a CUDA tensor"):
        hs2._dense(rows, "v_new", (bf,), rows.shape, 0)
    assert hs2._dense_or_none(None, "count", (i32,), (2,), 0) is None
    with pytest.raises(TypeError, match="count: expected a torch.Tensor"):
        hs2._dense(None, "count", (i32,), (2,), 0)
    del f32
