// Causal attention to a window of recent tokens and the first tokens (sinks).
//
// Query i of a chunk of Lq sits at position t = Lk - Lq + i and sees the keys
// s <= t with s > t - window or s < n_sink:
//   o = sum_s softmax_s(scale <q, k_s>) v_s,   lse = ln sum_s exp(scale <q, k_s>)
#pragma once

#include "common.cuh"

namespace hs2 {
namespace win {

// One query row and head by one warp, in fp32: the running maximum and sum of
// the softmax over the visible keys alone, one key at a time, so that nothing
// a masked row holds (NaN or infinities of a padded batch) is ever read.
// Lane i owns the D/32 dims from i * D/32.
template <int D>
HS2_DEV void attend_row(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                        const __nv_bfloat16* __restrict__ v, int64_t ld, int t, int window,
                        int n_sink, float scale2, __nv_bfloat16* __restrict__ o,
                        float* __restrict__ lse) {
    constexpr int E = D / 32;
    const int lane = lane_id();
    float qf[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; e++) {
        qf[e] = __bfloat162float(q[lane * E + e]) * scale2;
        acc[e] = 0.f;
    }
    const int w0 = max(0, t - window + 1);  // (t - window does not wrap: both are >= 0)
    const int ns = min(n_sink, w0);
    for (int i = 0; i < ns + t + 1 - w0; i++) {
        const int s = i < ns ? i : w0 + i - ns;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; e++)
            x = fmaf(qf[e], __bfloat162float(k[s * ld + lane * E + e]), x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(~0u, x, off);
        const float mn = fmaxf(m, x);
        const float a = ex2(m - mn), p = ex2(x - mn);
        m = mn;
        l = fmaf(l, a, p);
#pragma unroll
        for (int e = 0; e < E; e++)
            acc[e] = fmaf(acc[e], a, p * __bfloat162float(v[s * ld + lane * E + e]));
    }
    const float inv = 1.f / l;
#pragma unroll
    for (int e = 0; e < E; e++) o[lane * E + e] = __float2bfloat16(acc[e] * inv);
    if (lse && lane == 0) *lse = (m + log2f(l)) * kLn2;
}

// grid: a warp per (sequence, query, head)
template <int D>
__global__ void __launch_bounds__(128)
window_rows_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                   const __nv_bfloat16* __restrict__ v, __nv_bfloat16* __restrict__ o,
                   float* __restrict__ lse, int B, int Lq, int Lk, int Hq, int Hkv, int window,
                   int n_sink, float scale2) {
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)B * Lq * Hq) return;
    const int h = (int)(row % Hq), i = (int)(row / Hq % Lq), b = (int)(row / Hq / Lq);
    const size_t kv = ((size_t)b * Lk * Hkv + h / (Hq / Hkv)) * D;
    attend_row<D>(q + row * D, k + kv, v + kv, (int64_t)Hkv * D, Lk - Lq + i, window, n_sink, scale2,
                  o + row * D, lse ? lse + row : nullptr);
}

}  // namespace win
}  // namespace hs2
