// Writers and readers of the 8-bit K/V caches.
//
//   token cache   codes [B, Tmax, d], one fp32 scale per token:
//                 s = max|x| / 448 (1 for a row of zeros), code = e4m3(x / s)
//   paged cache   pages [P, Hkv, page, d], one scale per page and KV head, a
//                 power of two: the least s >= 2^-126 with max|x| <= 448 s
//
// e4m3 rounding is to nearest even, saturated to +-448.  A page's scale is a
// power of two so that a page that is appended to can raise it and re-round
// its older codes without a second rounding: code * 2^-n is exact unless it
// falls below 2^-6, where e4m3 has a fixed step.  It costs less than one of
// e4m3's 17 octaves of range and no precision inside it.
//
// All of these move bytes once: a write reads 2 bytes and stores 1 per
// element, a read the reverse.
#pragma once

#include "common.cuh"

namespace hs2 {
namespace kvc {

constexpr float kE4m3Max = 448.f;

// Two floats -> two e4m3 codes (lo in bits 0..7), nearest even, saturated.
HS2_DEV uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Largest |x| of the eight bf16 values of w, as bf16 bits (they order like the
// magnitudes), non-finite values left out; *bad is set if there are any.
HS2_DEV uint32_t amax_bits(uint4 w, bool* bad) {
    const uint32_t a0 = w.x & 0x7FFF7FFFu, a1 = w.y & 0x7FFF7FFFu;
    const uint32_t a2 = w.z & 0x7FFF7FFFu, a3 = w.w & 0x7FFF7FFFu;
    const uint32_t m = __vmaxu2(__vmaxu2(a0, a1), __vmaxu2(a2, a3));
    uint32_t r = max(m & 0xFFFFu, m >> 16);
    if (r >= 0x7F80u) {
        *bad = true;
        r = 0;
        const uint32_t a[4] = {a0, a1, a2, a3};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t lo = a[i] & 0xFFFFu, hi = a[i] >> 16;
            if (lo < 0x7F80u) r = max(r, lo);
            if (hi < 0x7F80u) r = max(r, hi);
        }
    }
    return r;
}

// The least power of two s >= 2^-126 with top <= 448 s (top >= 0, finite; 448
// is 1.75 * 2^8, so the answer is read off top's exponent and whether its
// significand exceeds 1.75).
HS2_DEV float page_scale(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)max(e, 1) << 23);  // a subnormal or zero top gives 2^-126
}

// ------------------------------------------------------------- token cache
constexpr int kThreads = 256;
constexpr int kRows = 2;  // rows of K and of V that a reading thread has in flight

// Eight elements of a row over its scale, as e4m3 codes of the fp32 quotients.
// A division's ten instructions each took two thirds of this kernel's time
// (128k rows in 28.7 us), so the quotient is formed by Markstein's method
// (IBM J. Res. Dev. 34, 1990): with r = 1 / s rounded to nearest and q = x r,
// the fused q + r (x - q s) is x / s rounded to nearest.  It needs the exact
// remainder to be representable; below s = 2^-60, and with infinities among
// the elements, they are divided.
HS2_DEV uint2 quantise8(uint4 w, float s, float r, bool finite) {
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        y[2 * i] = bf16_lo(in[i]);
        y[2 * i + 1] = bf16_hi(in[i]);
    }
    if (s >= 8.67361738e-19f && finite) {  // 2^-60
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float q = y[i] * r;
            y[i] = fmaf(fmaf(-q, s, y[i]), r, q);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = y[i] / s;
    }
    return make_uint2(e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16,
                      e4m3x2(y[4], y[5]) | e4m3x2(y[6], y[7]) << 16);
}

// One group of D/16 lanes per row, sixteen elements of K and of V a lane (the
// row's maximum, its scale and the reciprocal are the lanes' common cost: with
// eight elements 128k rows of 128 took 24.6 us, now 22.2: 4.6 TB/s, with 67% of
// the issue slots in use; short blocks whose loads only other blocks cover).
// grid (rows, B).
template <int D>
__global__ void __launch_bounds__(kThreads)
token_write_kernel(const __nv_bfloat16* __restrict__ k_new, const __nv_bfloat16* __restrict__ v_new,
                   const int32_t* __restrict__ start, const int32_t* __restrict__ count,
                   uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache,
                   float* __restrict__ k_scale, float* __restrict__ v_scale, int N, int Tmax,
                   unsigned* __restrict__ flags) {
    constexpr int LPR = D / 16;
    const int b = blockIdx.y;
    const int lane = threadIdx.x % LPR;
    const int s0 = start[b], n = count ? count[b] : N;
    const int i = blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
    uint4 w[2][2];
    const size_t src = ((size_t)b * N + i) * D + lane * 16;
#pragma unroll
    for (int j = 0; j < 2; j++) {
        w[0][j] = i < N ? ldg_stream(k_new + src + 8 * j) : make_uint4(0, 0, 0, 0);
        w[1][j] = i < N ? ldg_stream(v_new + src + 8 * j) : make_uint4(0, 0, 0, 0);
    }
    if (n < 0 || n > N || s0 < 0 || s0 > Tmax - n) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(flags, FLAG_BAD_LENGTH);
        return;
    }
    bool bad = false;
#pragma unroll
    for (int x = 0; x < 2; x++) {
        bool odd = false;
        uint32_t top = max(amax_bits(w[x][0], &odd), amax_bits(w[x][1], &odd));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
        if (i < n) {
            const float s = top ? __uint_as_float(top << 16) / kE4m3Max : 1.f, r = 1.f / s;
            const uint2 lo = quantise8(w[x][0], s, r, !odd), hi = quantise8(w[x][1], s, r, !odd);
            const size_t row = (size_t)b * Tmax + s0 + i;
            *reinterpret_cast<uint4*>((x ? v_cache : k_cache) + row * D + lane * 16) =
                make_uint4(lo.x, lo.y, hi.x, hi.y);
            if (lane == 0) (x ? v_scale : k_scale)[row] = s;
            bad |= odd;
        }
    }
    if (bad) atomicOr(flags, FLAG_NONFINITE);
}

// Eight codes and their scale -> eight bf16 (rounded to nearest even: fp32's
// rounding of the product is 2^-24 relative, far below bf16's).
HS2_DEV uint4 dequant8(uint2 c, float s) {
    const uint32_t w[4] = {c.x, c.x >> 16, c.y, c.y >> 16};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 a = f16x2_to_float2(e4m3x2_lo_to_f16x2(w[i]));
        r[i] = pack_bf16(a.x * s, a.y * s);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
HS2_DEV uint2 ldg_stream8(const void* p) {
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// Eight codes a lane, so that a warp's stores are whole 512-byte runs.  38.5 MB
// (4 sequences of 16-32k rows of 64) in 10.3 us, of which the bytes need 6 and
// the launch most of the rest; 407 MB (512k rows of 128) in 65.7 us, 6.2 TB/s.
// grid (rows, B).
template <int D>
__global__ void __launch_bounds__(kThreads)
token_read_kernel(const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
                  const float* __restrict__ k_scale, const float* __restrict__ v_scale,
                  const int32_t* __restrict__ start, const int32_t* __restrict__ count,
                  __nv_bfloat16* __restrict__ k, __nv_bfloat16* __restrict__ v, int N, int Tmax,
                  unsigned* __restrict__ flags) {
    constexpr int LPR = D / 8;
    constexpr int RPB = kThreads / LPR;
    const int b = blockIdx.y;
    const int lane = threadIdx.x % LPR;
    const int s0 = start[b], n = count ? count[b] : N;
    if (n < 0 || n > N || s0 < 0 || s0 > Tmax - n) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(flags, FLAG_BAD_LENGTH);
        return;
    }
    const int i0 = blockIdx.x * (RPB * kRows) + threadIdx.x / LPR;
    uint2 c[2 * kRows];
    float s[2 * kRows];
#pragma unroll
    for (int r = 0; r < kRows; r++) {
        const int i = min(i0 + r * RPB, n - 1);  // (n = 0: nothing is stored, row s0 - 1 or 0 is read)
        const size_t row = (size_t)b * Tmax + max(s0 + i, 0);
        c[2 * r] = ldg_stream8(k_cache + row * D + lane * 8);
        c[2 * r + 1] = ldg_stream8(v_cache + row * D + lane * 8);
        s[2 * r] = __ldg(k_scale + row);
        s[2 * r + 1] = __ldg(v_scale + row);
    }
#pragma unroll
    for (int r = 0; r < kRows; r++) {
        const int i = i0 + r * RPB;
        if (i >= n) break;
        const size_t dst = ((size_t)b * N + i) * D + lane * 8;
        *reinterpret_cast<uint4*>(k + dst) = dequant8(c[2 * r], s[2 * r]);
        *reinterpret_cast<uint4*>(v + dst) = dequant8(c[2 * r + 1], s[2 * r + 1]);
    }
}

// ------------------------------------------------------------- paged cache
// One block per (touched page, KV head, K or V) and sequence; the page's new
// rows stay in registers between the search for their largest magnitude and
// the rounding, so they are read once.  604 MB (4 sequences of 16-32k rows, 8
// heads of 128) in 98 to 108 us, 5.6 to 6.2 TB/s: bound by the memory.  grid
// (pages * Hkv * 2, B).
constexpr int kPageThreads = 128;

template <int D, int PAGE>
__global__ void __launch_bounds__(kPageThreads)
paged_write_kernel(const __nv_bfloat16* __restrict__ k_new, const __nv_bfloat16* __restrict__ v_new,
                   const int32_t* __restrict__ table, const int32_t* __restrict__ start,
                   const int32_t* __restrict__ count, uint8_t* __restrict__ k_pages,
                   uint8_t* __restrict__ v_pages, float* __restrict__ k_scale,
                   float* __restrict__ v_scale, int N, int Hkv, int n_pages, int max_pages,
                   unsigned* __restrict__ flags) {
    constexpr int LPR = D / 8;                                      // lanes per row
    constexpr int UNITS = PAGE * LPR;                               // 16-byte pieces of new rows
    constexpr int U = (UNITS + kPageThreads - 1) / kPageThreads;    // a thread's pieces
    __shared__ uint32_t s_top[kPageThreads / 32];
    const int b = blockIdx.y, tid = threadIdx.x;
    const int which = blockIdx.x & 1;
    const int h = (blockIdx.x >> 1) % Hkv;
    const int s0 = start[b], n = count ? count[b] : N;
    if (n < 0 || n > N || s0 < 0 || s0 > max_pages * PAGE - n) {
        if (blockIdx.x == 0 && tid == 0) atomicOr(flags, FLAG_BAD_LENGTH);
        return;
    }
    // rows [first, first + PAGE) of the call, counted from its first page's start
    const int nth = (int)(blockIdx.x >> 1) / Hkv, lead = s0 % PAGE, first = nth * PAGE - lead;
    const int p0 = nth == 0 ? lead : 0, p1 = min(PAGE, n - first);
    if (p0 >= p1) return;  // the rows do not reach this page
    const int pid = table[(size_t)b * max_pages + (s0 / PAGE + nth)];
    if (pid < 0 || pid >= n_pages) {
        if (tid == 0) atomicOr(flags, FLAG_BAD_INDEX);
        return;
    }
    const __nv_bfloat16* src = which ? v_new : k_new;
    const size_t ph = (size_t)pid * Hkv + h;
    uint8_t* dst = (which ? v_pages : k_pages) + ph * (PAGE * D);
    float* scale = (which ? v_scale : k_scale) + ph;
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int unit = u * kPageThreads + tid, r = unit / LPR;
        const bool in = r >= p0 && r < p1;
        const size_t i = (size_t)b * N + (first + r);
        w[u] = in ? ldg_stream(src + (i * Hkv + h) * D + (unit % LPR) * 8) : make_uint4(0, 0, 0, 0);
    }
    const float had = p0 > 0 ? *scale : 0.f;
    bool bad = false;
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < U; u++) top = max(top, amax_bits(w[u], &bad));
    top = __reduce_max_sync(~0u, top);
    if ((tid & 31) == 0) s_top[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPageThreads / 32; i++) top = max(top, s_top[i]);
    float s = page_scale(__uint_as_float(top << 16));
    if (p0 > 0) {
        if (had > 0.f && had < INFINITY) {
            if (s > had) {
                // the older rows' codes under the raised scale
                const float f = had / s;
                for (int unit = tid; unit < p0 * (D / 4); unit += kPageThreads) {
                    uint32_t* c = reinterpret_cast<uint32_t*>(dst) + unit;
                    const uint32_t old = *c;
                    const float2 a = f16x2_to_float2(e4m3x2_lo_to_f16x2(old));
                    const float2 e = f16x2_to_float2(e4m3x2_lo_to_f16x2(old >> 16));
                    *c = e4m3x2(a.x * f, a.y * f) | e4m3x2(e.x * f, e.y * f) << 16;
                }
            } else {
                s = had;
            }
        } else if (tid == 0) {
            atomicOr(flags, FLAG_SCALE_RANGE);
        }
    }
    const float inv = 1.f / s;
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int unit = u * kPageThreads + tid, r = unit / LPR;
        if (r >= p0 && r < p1) {
            const uint32_t c0 = e4m3x2(bf16_lo(w[u].x) * inv, bf16_hi(w[u].x) * inv);
            const uint32_t c1 = e4m3x2(bf16_lo(w[u].y) * inv, bf16_hi(w[u].y) * inv);
            const uint32_t c2 = e4m3x2(bf16_lo(w[u].z) * inv, bf16_hi(w[u].z) * inv);
            const uint32_t c3 = e4m3x2(bf16_lo(w[u].w) * inv, bf16_hi(w[u].w) * inv);
            *reinterpret_cast<uint2*>(dst + (size_t)unit * 8) = make_uint2(c0 | c1 << 16, c2 | c3 << 16);
        }
    }
    if (__float_as_uint(s) & 0x7FFFFFu) {
        // no power of two, so the reciprocal is not exact: a page that another
        // writer began.  Its rows are read again and divided (a division in the
        // loop above costs every call: 604 MB in 146 us, not 102)
#pragma unroll 1
        for (int unit = tid; unit < p1 * LPR; unit += kPageThreads) {  // (the same thread's as above)
            if (unit / LPR < p0) continue;
            const size_t i = (size_t)b * N + (first + unit / LPR);
            const uint4 x = ldg_stream(src + (i * Hkv + h) * D + (unit % LPR) * 8);
            *reinterpret_cast<uint2*>(dst + (size_t)unit * 8) = quantise8(x, s, 1.f, false);
        }
    }
    if (tid == 0) *scale = s;
    if (bad) atomicOr(flags, FLAG_NONFINITE);
}

constexpr int kPagedRows = 4;  // (a page number comes before each: 2 took 61 us where 4 take 57)

// Rows [start, start + count) of each sequence and one KV head, as
// token_read_kernel.  302 MB in 56.9 us, 5.3 TB/s.  grid (rows, B, Hkv).
template <int D>
__global__ void __launch_bounds__(kThreads)
paged_read_kernel(const uint8_t* __restrict__ k_pages, const uint8_t* __restrict__ v_pages,
                  const float* __restrict__ k_scale, const float* __restrict__ v_scale,
                  const int32_t* __restrict__ table, const int32_t* __restrict__ start,
                  const int32_t* __restrict__ count, __nv_bfloat16* __restrict__ k,
                  __nv_bfloat16* __restrict__ v, int N, int log_page, int n_pages, int max_pages,
                  unsigned* __restrict__ flags) {
    constexpr int LPR = D / 8;
    constexpr int RPB = kThreads / LPR;
    const int b = blockIdx.y, h = blockIdx.z, Hkv = gridDim.z;
    const int lane = threadIdx.x % LPR;
    const int s0 = start[b], n = count ? count[b] : N;
    if (n < 0 || n > N || s0 < 0 || s0 > (max_pages << log_page) - n) {
        if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) atomicOr(flags, FLAG_BAD_LENGTH);
        return;
    }
    const int i0 = blockIdx.x * (RPB * kPagedRows) + threadIdx.x / LPR;
    int pid[kPagedRows];
    uint2 c[2 * kPagedRows];
    float s[2 * kPagedRows];
#pragma unroll
    for (int r = 0; r < kPagedRows; r++) {
        const int i = i0 + r * RPB;
        pid[r] = i < n ? __ldg(table + (size_t)b * max_pages + ((s0 + i) >> log_page)) : 0;
    }
#pragma unroll
    for (int r = 0; r < kPagedRows; r++) {
        const int i = i0 + r * RPB;
        const bool ok = i < n && pid[r] >= 0 && pid[r] < n_pages;
        if (i < n && !ok) atomicOr(flags, FLAG_BAD_INDEX);
        if (!ok) pid[r] = -1;
        const size_t ph = (size_t)(ok ? pid[r] : 0) * Hkv + h;
        const size_t at = ((ph << log_page) + (ok ? (s0 + i) & ((1 << log_page) - 1) : 0)) * D + lane * 8;
        c[2 * r] = ldg_stream8(k_pages + at);
        c[2 * r + 1] = ldg_stream8(v_pages + at);
        s[2 * r] = __ldg(k_scale + ph);
        s[2 * r + 1] = __ldg(v_scale + ph);
    }
#pragma unroll
    for (int r = 0; r < kPagedRows; r++) {
        const int i = i0 + r * RPB;
        if (pid[r] < 0 || i >= n) continue;
        const size_t dst = (((size_t)b * N + i) * Hkv + h) * D + lane * 8;
        *reinterpret_cast<uint4*>(k + dst) = dequant8(c[2 * r], s[2 * r]);
        *reinterpret_cast<uint4*>(v + dst) = dequant8(c[2 * r + 1], s[2 * r + 1]);
    }
}

}  // namespace kvc
}  // namespace hs2
