// One query token per sequence over a paged e4m3 cache with a scale per page
// and KV head: all of the sequence's tokens, or its last `window` and its first
// `n_sink`.
//   o = sum_s softmax_s(scale <q, k_s>) v_s,   lse = ln sum_s exp(scale <q, k_s>)
#pragma once

#include "common.cuh"

namespace hs2 {
namespace pgd {

template <int D>
__global__ void __launch_bounds__(32)
paged_rows_kernel(const __nv_bfloat16* __restrict__ q, const uint8_t* __restrict__ k_pages,
                  const uint8_t* __restrict__ v_pages, const float* __restrict__ k_scale,
                  const float* __restrict__ v_scale, const int32_t* __restrict__ table,
                  const int32_t* __restrict__ lengths, __nv_bfloat16* __restrict__ o,
                  float* __restrict__ lse, int Hq, int Hkv, int page, int n_pages, int max_pages,
                  int window, int n_sink, float scale2, unsigned* __restrict__ flags) {
    constexpr int E = D / 32;
    const int lane = lane_id(), h = blockIdx.x, b = blockIdx.y;
    const int hk = h / (Hq / Hkv);
    int T = lengths[b];
    if (T < 0 || T > max_pages * page) {
        if (lane == 0 && h == 0) atomicOr(flags, FLAG_BAD_LENGTH);
        T = 0;
    }
    float qf[E], acc[E], m = -INFINITY, l = 0.f;
    const size_t row = (size_t)b * Hq + h;
#pragma unroll
    for (int e = 0; e < E; e++) {
        qf[e] = __bfloat162float(q[row * D + lane * E + e]) * scale2;
        acc[e] = 0.f;
    }
    const int w0 = max(0, T - window);
    const int ns = min(n_sink, w0);
    for (int i = 0; i < ns + T - w0; i++) {
        const int s = i < ns ? i : w0 + i - ns;
        const int pid = table[(size_t)b * max_pages + s / page];
        if (pid < 0 || pid >= n_pages) {
            if (lane == 0) atomicOr(flags, FLAG_BAD_INDEX);
            continue;
        }
        const size_t ph = (size_t)pid * Hkv + hk;
        const size_t at = (ph * page + s % page) * D + lane * E;
        float kf[E], vf[E];
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 a = f16x2_to_float2(
                e4m3x2_lo_to_f16x2(*reinterpret_cast<const uint16_t*>(k_pages + at + e)));
            const float2 c = f16x2_to_float2(
                e4m3x2_lo_to_f16x2(*reinterpret_cast<const uint16_t*>(v_pages + at + e)));
            kf[e] = a.x, kf[e + 1] = a.y, vf[e] = c.x, vf[e + 1] = c.y;
        }
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; e++) x = fmaf(qf[e], kf[e], x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(~0u, x, off);
        x *= k_scale[ph];
        const float mn = fmaxf(m, x);
        const float a = ex2(m - mn), p = ex2(x - mn);
        m = mn;
        l = fmaf(l, a, p);
        const float pv = p * v_scale[ph];
#pragma unroll
        for (int e = 0; e < E; e++) acc[e] = fmaf(acc[e], a, pv * vf[e]);
    }
    const bool any = m > -INFINITY || l != 0.f;  // (l is NaN where a visible logit is)
    const float inv = any ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < E; e++) o[row * D + lane * E + e] = __float2bfloat16(any ? acc[e] * inv : 0.f);
    if (lse && lane == 0) lse[row] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace pgd
}  // namespace hs2
