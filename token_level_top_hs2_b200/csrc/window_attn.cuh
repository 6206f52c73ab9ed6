// Causal attention to a window of recent tokens and the first tokens (sinks).
//
// Query i of a chunk of Lq sits at position t = Lk - Lq + i and sees the keys
// s <= t with s > t - window or s < n_sink:
//   o = sum_s softmax_s(scale <q, k_s>) v_s,   lse = ln sum_s exp(scale <q, k_s>)
//
// The G query heads of a KV head share their keys, so the 128 rows of a
// tensor-core tile are nt = floor(128 / G) tokens x G heads (row = token * G +
// head): with 16 heads a tile of 8 tokens and a window of 128 needs 135 keys,
// where 128 tokens of one head would need 255.  One persistent CTA per SM
// takes items of two such tiles (2 nt tokens of one KV head), which use the
// same keys: the sinks, rounded up to 16 rows, then the rows from the first
// token's window to the last token, in tiles of 64.
//
// Both tiles' logits are double-buffered in tensor memory (2 x 2 x 64 columns,
// beside two accumulators of D), so that QK^T of the tile after next is issued
// behind PV of this one and a softmax warp finds its next logits there when it
// is done: the chain softmax -> PV -> QK^T -> softmax of a single buffer is cut.
//   warps 0, 2  TMA producers: queries (two items) and the K ring; the V ring
//   warps 1, 3  MMA issuers of tiles 0 and 1: S_x = Q_x K^T, O_x += P_x V
//   warps 4-7   outputs of both tiles: accumulator, maximum and sum to o and lse;
//               at the end, rows that masked NaN or infinities have spoilt
//   warps 8-11  softmax of tile 0, thread = row = TMEM lane
//   warps 12-15 softmax of tile 1
// P overwrites its logits, rounded to bf16 since both operands of the product
// have V's type (the sum is of the unrounded weights: outputs are off by 0.0021
// to 0.0023 of their size where a bf16 output alone is by 0.0017); the running
// maximum is raised only when a tile exceeds it by 2^8, so the accumulator is
// rarely rescaled.
//
// Measured: 128k queries of 16 heads of 128, window 128 (1.15 GB), 243 to 253
// us in a burst of calls (4.5 to 4.7 TB/s), 300 over seconds at the power cap
// (3.8 TB/s), bound by the chain of an item's softmax steps (most of its tiles
// of keys are partly masked); 2 x 16k queries of 32 heads in 8 groups, window
// 4096 (2.16 TF), 1.86 to 2.07 ms in a burst, 2.14 over seconds (1.0 PF/s), 55% of
// the tensor pipe's cycles, bound by exponentials and power.  An item's keys are
// not split: with fewer items than SMs the longest one is the call's time, 69 us
// for one query of 16 heads over 4,096 keys, 1.48 ms over 100,000.
#pragma once

#include <float.h>
#include <limits.h>

#include "tc.cuh"

namespace hs2 {
namespace win {

using namespace hs2::tc;

constexpr int BM = 128;           // rows of a tile
constexpr int BN = 64;            // keys of a tile
constexpr int kThreads = 512;
constexpr float kRaiseLog2 = 8.f;

struct Shape {
    int B, Lq, Lk, Hq, Hkv, G, nt, window, n_sink, blocks, items;
    float scale2;
};
struct Rows {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16* o;
    float* lse;
};

// The keys of an item as a list of entries: [0, pre) are positions 0 .. pre-1
// (the sinks, rounded up to 16), entry e >= pre is position base + e - pre.
struct Item {
    int b, hk, i0, t0;         // sequence, KV head, first query, its position
    int pre, base, entries, tiles;
};
HS2_DEV Item item_of(const Shape& s, int n) {
    Item it;
    const int rest = n / s.blocks;
    it.i0 = (n - rest * s.blocks) * 2 * s.nt;
    it.b = rest / s.Hkv;
    it.hk = rest - it.b * s.Hkv;
    it.t0 = s.Lk - s.Lq + it.i0;
    const int last = min(s.Lk - 1, it.t0 + 2 * s.nt - 1);
    const int w0 = max(0, it.t0 - s.window + 1);
    // sinks that reach into the window's rows, or nearly: one run of rows
    const bool joined = s.n_sink > w0 - 16;
    it.base = joined && s.n_sink > 0 ? 0 : w0;
    it.pre = joined || s.n_sink == 0 ? 0 : (s.n_sink + 15) & ~15;
    it.entries = it.pre - it.base + last + 1;
    it.tiles = (it.entries + BN - 1) / BN;
    return it;
}
// rows of tile j that are loaded: a multiple of 16
HS2_DEV int rows_of(const Item& it, int j) { return min(BN, (it.entries - j * BN + 15) & ~15); }

// A walk over a CTA's tiles, item by item.
struct Walk {
    Item it;
    int n, j, count;  // item, tile in it, items before it
    HS2_DEV void start(const Shape& s, int first) {
        n = first;
        j = count = 0;
        if (n < s.items) it = item_of(s, n);
    }
    HS2_DEV bool done(const Shape& s) const { return n >= s.items; }
    HS2_DEV void next(const Shape& s, int step) {
        if (++j < it.tiles) return;
        j = 0;
        count++;
        n += step;
        if (n < s.items) it = item_of(s, n);
    }
};

template <int D>
struct Cfg {
    static constexpr int DB = D / 64;                // 64-column blocks
    static constexpr int QT = BM * D * 2;            // one tile's queries
    static constexpr int KT = BN * D * 2;            // a K or V tile
    static constexpr int OFF_K = 4 * QT;             // (two items of two tiles before it)
    static constexpr int OFF_V = OFF_K + 2 * KT;
    static constexpr int OFF_O = OFF_V + 2 * KT;     // 32 rows x 64 columns per output warp
    static constexpr int SMEM = OFF_O + 4 * 4096 + 1024;
    static constexpr uint32_t COL_O = 256;           // S: [tile][buffer] of 64 columns
};

struct Bars {
    uint64_t q_full[2], q_empty[2];  // [item & 1]
    // [tile & 1]: K and V have two places; that of tile c is free for tile c + 2
    // once both rows' tiles have taken theirs (s_full, pv_done)
    uint64_t k_full[2], v_full[2];
    // [rows' tile][tile & 1]: a softmax warp can be one tile ahead of the thread
    // that waits for it, so each barrier is used every other time
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2], drain[2];
    // [rows' tile][item & 1]; [rows' tile].  o_free: the outputs have read an
    // item's accumulator, and its maxima and sums before that
    uint64_t ml_full[2][2], o_free[2];
    float2 ml[2][2][BM];                // [rows' tile][item & 1]: a row's maximum and sum
    uint32_t tmem;
    int abort_;
    int redo_first, redo_last;          // the CTA's items with rows to do again
};

struct Maps {
    CUtensorMap q;                   // [B, Lq, Hq, D]: 64 columns x G heads x nt tokens
    CUtensorMap k64, k16, v64, v16;  // [B, Lk, Hkv, D]: 64 columns x 64 or 16 positions
};

// The low n bits (n <= 0: none, n >= 32: all).
HS2_DEV uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; }

// Values of two bf16 in w that are not finite, as bits 0 and 1.
HS2_DEV uint32_t not_finite(uint32_t w) {
    return ((w & 0x7F80u) == 0x7F80u ? 1u : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 2u : 0u);
}

// Barrier of the four warps of the outputs; true if any of their threads passes true.
HS2_DEV bool outputs_any(bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred)
        : "memory");
    return r != 0;
}

// An output row whose softmax itself is not finite (NaN, and so meant to be)
// opens with this pair of NaN, whose sign no conversion to bf16 gives.
constexpr uint32_t kMeantNan = 0xFFFFFFFFu;

// Output dims that a key row out of the query's sight has spoilt, done again in
// fp32 from the keys in sight.  0 * NaN is NaN on the tensor cores, so a masked
// value row of NaN or infinities (the padding of a padded batch) spoils the
// rows that share its tile; maxima and sums are never spoilt, since masked
// logits are replaced.  The warps of the outputs come here once all of the CTA's
// items are stored and no role waits for another, so it may take its time: a
// row costs its window.  What keeps that rare: dims in which a key that the whole
// item sees holds something not finite are right as they are (one pass over the
// item's values finds them), a row is done from its newest key on and ends when
// all of its dims have met such a value, and masked rows in a tile lie within
// 2 nt + 15 positions of its queries or of their windows' starts.  Four rows and
// 32 keys take about 5 us (a warp's own instructions: deeper batches of loads
// change nothing): two sequences of 20,000 tokens, 4 heads of 128, plain causal,
// 0.96 ms, with NaN from 11,111 on in the second 17.5 ms (398 ms with a row at a
// time, a key per step, inside the pipeline).
template <int D>
static __device__ __noinline__ void redo_items(const Rows& io, const Shape& sh, int first, int last) {
    extern __shared__ uint8_t smem_raw[];
    float* shared = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(smem_raw) + 15) & ~(uintptr_t)15);
    constexpr int E = D / 32, W = E / 2;  // dims of a lane, in words
    constexpr int R = 4;
    const int lane = lane_id(), warp = threadIdx.x >> 5 & 3;
    uint32_t* legit = reinterpret_cast<uint32_t*>(shared);  // [lane]: its dims not finite in common keys
    float* qf = shared + 32 + warp * (R * D + 128);
    float4* pw = reinterpret_cast<float4*>(qf + R * D);  // the rows' weights of 32 keys
    // the lane's dims of a row, and which of them are not finite
    auto dims = [&](const __nv_bfloat16* row, uint32_t (&w)[W]) {
        if constexpr (W == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(row + lane * E);
            w[0] = x.x, w[1] = x.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t*>(row + lane * E);
        }
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < W; i++) bits |= not_finite(w[i]) << (2 * i);
        return bits;
    };
    const int64_t ld = (int64_t)sh.Hkv * D;
    for (int n = first; n <= last; n += gridDim.x) {
        const Item it = item_of(sh, n);
        const int tokens = min(2 * sh.nt, sh.Lq - it.i0), rows = tokens * sh.G;
        const __nv_bfloat16* kb = io.k + ((size_t)it.b * sh.Lk * sh.Hkv + it.hk) * D;
        const __nv_bfloat16* vb = io.v + ((size_t)it.b * sh.Lk * sh.Hkv + it.hk) * D;
        auto at = [&](int r) {
            return (((size_t)it.b * sh.Lq + it.i0 + r / sh.G) * sh.Hq + it.hk * sh.G + r % sh.G) * D;
        };
        auto spoilt = [&](int r, uint32_t (&w)[W]) {
            const uint32_t bits = dims(io.o + at(r), w);
            return __shfl_sync(~0u, w[0], 0) == kMeantNan ? 0u : bits;
        };
        bool any = false;
        uint32_t w[W];
        for (int r = warp; r < rows; r += 4) any |= spoilt(r, w) != 0;
        if (warp == 0) legit[lane] = 0;
        if (!outputs_any(any)) continue;
        // the keys that all of the item's queries see
        uint32_t bits = 0;
        const int lo = max(0, it.t0 + tokens - sh.window), sinks = min(sh.n_sink, min(lo, it.t0 + 1));
        const int common = sinks + max(0, it.t0 + 1 - lo);
#pragma unroll 4
        for (int i = warp; i < common; i += 4)
            bits |= dims(vb + (i < sinks ? i : lo + i - sinks) * ld, w);
        if (bits) atomicOr(&legit[lane], bits);
        outputs_any(false);
        const uint32_t meant = legit[lane];
        // four rows at a time: they share what they read
        for (int r0 = warp * R; r0 < rows; r0 += 4 * R) {
            uint32_t todo[R], left = 0;
            int t[R];
#pragma unroll
            for (int r = 0; r < R; r++) {
                todo[r] = r0 + r < rows ? spoilt(r0 + r, w) & ~meant : 0u;
                t[r] = it.t0 + min(r0 + r, rows - 1) / sh.G;
                left |= todo[r];
            }
            if (!__any_sync(~0u, left)) continue;
            __syncwarp();
#pragma unroll
            for (int r = 0; r < R; r++)
                for (int e = lane; e < D; e += 32)
                    qf[r * D + e] = __bfloat162float(io.q[at(min(r0 + r, rows - 1)) + e]) * sh.scale2;
            __syncwarp();
            const int w0 = max(0, t[0] - sh.window + 1);  // (t - window does not wrap: both are >= 0)
            const int ns = min(sh.n_sink, w0);
            float acc[R][E], m[R], l[R];
#pragma unroll
            for (int r = 0; r < R; r++) {
                m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
                for (int e = 0; e < E; e++) acc[r][e] = 0.f;
            }
            // 32 keys at a time, the newest first: a lane per key for the logits, the
            // lane's dims of each key's values for the sums
            for (int i0 = ns + t[R - 1] - w0; i0 >= 0; i0 -= 32) {
                const int i = i0 - lane, s = i < 0 ? 0 : i < ns ? i : w0 + i - ns;
                const uint4* kr = reinterpret_cast<const uint4*>(kb + s * ld);
                float x[R] = {};
#pragma unroll 4
                for (int c = 0; c < D / 8; c++) {
                    const uint4 z = kr[c];
                    const uint32_t zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                    for (int r = 0; r < R; r++) {
                        const float* f = qf + r * D + 8 * c;
#pragma unroll
                        for (int u = 0; u < 4; u++)
                            x[r] = fmaf(f[2 * u + 1], bf16_hi(zw[u]), fmaf(f[2 * u], bf16_lo(zw[u]), x[r]));
                    }
                }
                float p[R];  // a weight, or -1 for a key out of the row's sight
#pragma unroll
                for (int r = 0; r < R; r++) {
                    const bool see = i >= 0 && s <= t[r] && (s > t[r] - sh.window || s < sh.n_sink);
                    float mn = see ? x[r] : -INFINITY;
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) mn = fmaxf(mn, __shfl_xor_sync(~0u, mn, off));
                    mn = fmaxf(m[r], mn);
                    const bool some = mn > -INFINITY;  // (else no weight yet)
                    const float a = some ? ex2(m[r] - mn) : 1.f;
                    p[r] = see ? some ? ex2(x[r] - mn) : 0.f : -1.f;
                    m[r] = mn;
                    float sum = fmaxf(p[r], 0.f);
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(~0u, sum, off);
                    l[r] = fmaf(l[r], a, sum);
#pragma unroll
                    for (int e = 0; e < E; e++) acc[r][e] *= a;
                }
                __syncwarp();
                pw[lane] = make_float4(p[0], p[1], p[2], p[3]);
                __syncwarp();
                const int keys = min(32, i0 + 1);
                auto add = [&](int j, bool all) {
                    dims(vb + __shfl_sync(~0u, s, j) * ld, w);
                    const float4 pj = pw[j];
                    const float pr[R] = {pj.x, pj.y, pj.z, pj.w};
#pragma unroll
                    for (int r = 0; r < R; r++)
                        if (all || pr[r] >= 0.f)
#pragma unroll
                            for (int e = 0; e < E; e++)
                                acc[r][e] =
                                    fmaf(pr[r], e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]), acc[r][e]);
                };
                if (__all_sync(~0u, fminf(fminf(p[0], p[1]), fminf(p[2], p[3])) >= 0.f)) {
#pragma unroll 8
                    for (int j = 0; j < 32; j++) add(j, true);
                } else {
#pragma unroll 1
                    for (int j = 0; j < keys; j++) add(j, false);
                }
                bool open = false;
#pragma unroll
                for (int r = 0; r < R; r++)
#pragma unroll
                    for (int e = 0; e < E; e++) open |= (todo[r] >> e & 1) && acc[r][e] * 0.f == 0.f;
                if (!__any_sync(~0u, open)) break;
            }
#pragma unroll
            for (int r = 0; r < R; r++) {
                const float inv = 1.f / l[r];
#pragma unroll
                for (int e = 0; e < E; e++)
                    if (todo[r] >> e & 1) io.o[at(r0 + r) + lane * E + e] = __float2bfloat16(acc[r][e] * inv);
            }
        }
        outputs_any(false);  // (all have read `legit`)
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_attn_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Rows io,
                   const __grid_constant__ Shape sh, unsigned* __restrict__ flags) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ Bars bars;
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = lane_id(), step = gridDim.x;
    volatile int* abort_ = &bars.abort_;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; i++) {
            mbar_init(&bars.q_full[i], 1);
            mbar_init(&bars.q_empty[i], 2);  // both tiles' MMAs
            mbar_init(&bars.k_full[i], 1);
            mbar_init(&bars.v_full[i], 1);
            mbar_init(&bars.drain[i], 1);
            mbar_init(&bars.o_free[i], 4);
            for (int j = 0; j < 2; j++) {
                mbar_init(&bars.s_full[i][j], 1);
                mbar_init(&bars.p_full[i][j], 4);
                mbar_init(&bars.pv_done[i][j], 1);
                mbar_init(&bars.ml_full[i][j], 4);
            }
        }
        bars.abort_ = 0;
        bars.redo_first = INT_MAX, bars.redo_last = -1;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars.tmem, 512);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k64);
        tma_prefetch_map(&maps.v64);
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = __shfl_sync(~0u, bars.tmem, 0);
    const uint32_t base = __shfl_sync(~0u, smem_u32(smem), 0);
    Walk w;
    w.start(sh, blockIdx.x);

    // Registers go where they are needed: the 65,536 that 512 threads launch
    // with are 128 x (40 + 136 + 168 + 168).
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0 || warp == 2) {
            // ------------------------------------------------- producers
            // Warp 0 loads queries and K, warp 2 V.  The queries of the next item
            // go out ahead of this item's last tile.
            const bool is_v = warp == 2;
            const CUtensorMap* m64 = is_v ? &maps.v64 : &maps.k64;
            const CUtensorMap* m16 = is_v ? &maps.v16 : &maps.k16;
            uint64_t* full = is_v ? bars.v_full : bars.k_full;
            uint64_t(*taken)[2] = is_v ? bars.pv_done : bars.s_full;
            const uint32_t ring = base + (is_v ? C::OFF_V : C::OFF_K);
            int c = 0, q_armed = 0;  // tiles and items loaded
            bool ok = true;
            auto load_q = [&](const Item& it, int count) {
                const int set = count & 1;
                ok = wait_warp(&bars.q_empty[set], ((count >> 1) & 1) ^ 1, abort_, flags);
                if (!ok) return;
                mbar_arrive_expect_tx_w(&bars.q_full[set], 2 * C::DB * 128 * sh.G * sh.nt);
                for (int x = 0; x < 2; x++)
                    for (int db = 0; db < C::DB; db++)
                        tma_load_4d_w(base + (2 * set + x) * C::QT + db * (BM * 128), &maps.q, 64 * db,
                                      it.hk * sh.G, it.i0 + x * sh.nt, it.b, &bars.q_full[set]);
                q_armed++;
            };
            if (!is_v && !w.done(sh)) load_q(w.it, 0);
            while (ok && !w.done(sh)) {
                const int rows = rows_of(w.it, w.j), e0 = w.j * BN;
                const int st = c & 1;
                // (the first two pass)
                if (!wait_warp(&taken[0][st], ((c >> 1) & 1) ^ 1, abort_, flags) ||
                    !wait_warp(&taken[1][st], ((c >> 1) & 1) ^ 1, abort_, flags))
                    break;
                mbar_arrive_expect_tx_w(&full[st], rows * D * 2);
                const uint32_t dst = ring + st * C::KT;
                if (rows == BN && e0 >= w.it.pre) {
                    for (int db = 0; db < C::DB; db++)
                        tma_load_4d_w(dst + db * (BN * 128), m64, 64 * db, w.it.hk,
                                      w.it.base + e0 - w.it.pre, w.it.b, &full[st]);
                } else {
                    for (int r = 0; r < rows; r += 16) {
                        const int e = e0 + r, pos = e < w.it.pre ? e : w.it.base + e - w.it.pre;
                        for (int db = 0; db < C::DB; db++)
                            tma_load_4d_w(dst + db * (BN * 128) + r * 128, m16, 64 * db, w.it.hk, pos,
                                          w.it.b, &full[st]);
                    }
                }
                c++;
                if (!is_v && w.j == w.it.tiles - 1 && w.n + step < sh.items)
                    load_q(item_of(sh, w.n + step), w.count + 1);
                w.next(sh, step);
            }
            if (*abort_) {  // let the copies in flight land before the CTA leaves
                volatile int no_abort = 0;
                for (int i = max(0, q_armed - 2); i < q_armed; i++)
                    mbar_wait(&bars.q_full[i & 1], (i >> 1) & 1, &no_abort, flags);
                for (int i = max(0, c - 2); i < c; i++)
                    mbar_wait(&full[i & 1], (i >> 1) & 1, &no_abort, flags);
            }
        } else if (warp == 1 || warp == 3) {
            // ----------------------------------------------- MMA issuers
            const int x = warp >> 1;
            const uint64_t q0 = sdesc_sw128(base + x * C::QT, 16, 1024);
            const uint64_t k0 = sdesc_sw128(base + C::OFF_K, 16, 1024);
            const uint64_t v0 = sdesc_sw128(base + C::OFF_V, BN * 128, 1024);
            constexpr uint32_t id_pv = idesc_bf16_f32(BM, D, false, true);
            const uint32_t s_col = tmem + x * 128, o_col = tmem + C::COL_O + x * D;
            int ca = 0, cw = 0, items = 0;  // tiles whose logits and whose outputs are issued; items of those
            int freed = 0;                  // items whose accumulator the outputs have read
            auto o_free = [&](int n) {      // the first n items'
                while (freed < n)
                    if (!wait_warp(&bars.o_free[x], freed++ & 1, abort_, flags)) return false;
                return true;
            };
            // of a tile, until its PV: rows / 16, and 256 if it opens its item
            uint32_t next[2] = {0, 0};
            auto qk = [&]() {
                const uint32_t rows = rows_of(w.it, w.j);
                const uint32_t id = idesc_bf16_f32(BM, 0, false, false) | (rows >> 3 << 17);
                const uint64_t dq = q0 + ((2 * (w.count & 1) * C::QT) >> 4);
                const uint64_t dk = k0 + (((ca & 1) * C::KT) >> 4);
                const uint32_t d = s_col + (ca & 1) * 64;
#pragma unroll
                for (int ks = 0; ks < D / 16; ks++)
                    mma_ss_w(d, dq + (((ks >> 2) * (BM * 128) + (ks & 3) * 32) >> 4),
                             dk + (((ks >> 2) * (BN * 128) + (ks & 3) * 32) >> 4), id, ks > 0);
                mma_commit_w(&bars.s_full[x][ca & 1]);
                if (w.j == w.it.tiles - 1) mma_commit_w(&bars.q_empty[w.count & 1]);
                const uint32_t info = rows >> 4 | (w.j == 0 ? 256u : 0u);
                ca++;
                w.next(sh, step);
                return info;
            };
            auto ready = [&]() {  // the next tile's operands
                return (w.j > 0 || wait_warp(&bars.q_full[w.count & 1], (w.count >> 1) & 1, abort_, flags)) &&
                       wait_warp(&bars.k_full[ca & 1], (ca >> 1) & 1, abort_, flags);
            };
            bool ok = true;
            for (int i = 0; i < 2; i++) {
                if (w.done(sh)) break;
                ok = ok && ready();
                if (!ok) break;
                fence_after_sync();
                next[i] = qk();
            }
            while (ok && cw < ca) {
                const bool more = !w.done(sh);
                // an item's first product overwrites the accumulator of the one before
                const bool opens = next[0] >= 256;
                if (opens && !o_free(items++)) break;
                if (!wait_warp(&bars.v_full[cw & 1], (cw >> 1) & 1, abort_, flags) || (more && !ready()) ||
                    !wait_warp(&bars.p_full[x][cw & 1], (cw >> 1) & 1, abort_, flags))
                    break;
                fence_after_sync();
                const uint64_t dv = v0 + (((cw & 1) * C::KT) >> 4);
                const uint32_t p = s_col + (cw & 1) * 64, n = next[0] & 255;
                mma_ts_w(o_col, p, dv, id_pv, !opens);
#pragma unroll
                for (int ks = 1; ks < BN / 16; ks++)
                    if (ks < n) mma_ts_w(o_col, p + ks * 8, dv + ((ks * 2048) >> 4), id_pv, 1u);
                mma_commit_w(&bars.pv_done[x][cw & 1]);
                next[0] = next[1];
                if (more) {
                    // (an item's maxima and sums go where those of two items before
                    // were, which the outputs must have read: items of one tile in a
                    // row are ordered by nothing else)
                    if (w.j == w.it.tiles - 1 && !o_free(w.count - 1)) break;
                    next[1] = qk();
                }
                cw++;
            }
            // every MMA issued must finish before TMEM is released
            mma_commit_w(&bars.drain[x]);
            volatile int no_abort = 0;
            mbar_wait(&bars.drain[x], 0, &no_abort, flags);
        }
    } else if (warp < 8) {
        // ------------------------------------------------------ outputs
        asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int tok = row / sh.G, head = row - tok * sh.G;
        uint4* stage = reinterpret_cast<uint4*>(smem + C::OFF_O + (warp - 4) * 4096);
        bool ok = true;
        for (int c = 0; ok && !w.done(sh); w.n += step, w.count++) {
            const Item it = item_of(sh, w.n);
            c += it.tiles;
            for (int x = 0; ok && x < 2; x++) {
                ok = __all_sync(~0u, mbar_wait(&bars.ml_full[x][w.count & 1], (w.count >> 1) & 1, abort_,
                                               flags) &&
                                         mbar_wait(&bars.pv_done[x][(c - 1) & 1], ((c - 1) >> 1) & 1,
                                                   abort_, flags));
                if (!ok) break;
                fence_after_sync();
                const float2 ml = bars.ml[x][w.count & 1][row];
                const int i = it.i0 + x * sh.nt + tok;
                const bool real = tok < sh.nt && i < sh.Lq;
                const float inv = 1.f / ml.y;
                const bool sane = ml.y > 0.f && ml.y < INFINITY;
                // NaN once anything is not finite
                __nv_bfloat162 zero = __float2bfloat162_rn(ml.y * 0.f);
                const __nv_bfloat162 nought = __float2bfloat162_rn(0.f);
                uint32_t p[D / 2];
#pragma unroll
                for (int u = 0; u < D; u += 32) {
                    uint32_t r[32];
                    tmem_ld32(lanes + C::COL_O + x * D + u, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int z = 0; z < 32; z += 2) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[z]) * inv,
                                                                       __uint_as_float(r[z + 1]) * inv);
                        zero = __hfma2(v, nought, zero);
                        p[(u + z) / 2] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                }
                if (!sane) p[0] = kMeantNan;
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.o_free[x]);
                const int at = real ? (it.b * sh.Lq + i) * sh.Hq + it.hk * sh.G + head : -1;
                // through the warp's shared memory, 64 columns at a time, so that
                // each store instruction writes whole 128-byte lines of four rows
#pragma unroll
                for (int u = 0; u < D; u += 64) {
#pragma unroll
                    for (int z = 0; z < 8; z++) {
                        const uint32_t* e = p + u / 2 + z * 4;
                        stage[lane * 8 + (z ^ (lane & 7))] = make_uint4(e[0], e[1], e[2], e[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int z = 0; z < 8; z++) {
                        const int r4 = z * 4 + (lane >> 3), to = __shfl_sync(~0u, at, r4);
                        const uint4 v = stage[r4 * 8 + ((lane & 7) ^ (r4 & 7))];
                        if (to >= 0)
                            *reinterpret_cast<uint4*>(io.o + (size_t)to * D + u + (lane & 7) * 8) = v;
                    }
                    __syncwarp();
                }
                if (io.lse && real) io.lse[at] = (ml.x + __log2f(ml.y)) * kLn2;
                const bool fine = __low2float(zero) + __high2float(zero) == 0.f;
                if (__any_sync(~0u, real && !fine && sane) && lane == 0) {
                    atomicMin(&bars.redo_first, w.n);
                    atomicMax(&bars.redo_last, w.n);
                }
            }
        }
        // every product of the CTA has been read by now: its shared memory is free
        if (!outputs_any(!ok) && bars.redo_last >= 0)
            redo_items<D>(io, sh, bars.redo_first, bars.redo_last);
    } else {
        // ------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        // (waits in line: a call would keep the compiler from the extra registers)
        const int x = (warp >> 2) - 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t o_col = lanes + C::COL_O + x * D;
        const int tok = row / sh.G;
        bool ok = true;
        int c = 0;
        while (ok && !w.done(sh)) {
            const Item it = w.it;
            const int t = it.t0 + x * sh.nt + tok;
            // the row's keys as entries: [0, e_sink) and [e_lo, e_hi)
            const int e_sink = min(sh.n_sink, t + 1);
            const int e_lo = it.pre - it.base + max(t - sh.window + 1, 0);
            const int e_hi = it.pre - it.base + t + 1;
            // entries that every row of the tile sees: from the last row's window
            // start up to the first row
            const int t_min = it.t0 + x * sh.nt;
            const int all_lo = it.pre - it.base + max(t_min + sh.nt - sh.window, 0);
            const int all_hi = it.pre - it.base + t_min + 1;
            float m = -FLT_MAX, l = 0.f;  // (below any finite logit: the first one raises it)
            for (int j = 0; j < it.tiles; j++, c++) {
                const int e0 = j * BN;
                const bool second = e0 + 32 < it.entries;  // (else PV reads the first 32 keys at most)
                const uint32_t s_col = lanes + x * 128 + (c & 1) * 64;
                ok = __all_sync(~0u, mbar_wait(&bars.s_full[x][c & 1], (c >> 1) & 1, abort_, flags));
                if (!ok) break;
                fence_after_sync();
                float s[BN], mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    if (h == 1 && !second) break;
                    uint32_t r[32];
                    tmem_ld32(s_col + h * 32, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int u = 0; u < 32; u++) s[h * 32 + u] = __uint_as_float(r[u]);
                    const int e = e0 + h * 32;
                    if (!(e >= all_lo && e + 32 <= all_hi)) {
                        const uint32_t see =
                            low_bits(e_sink - e) | (low_bits(e_hi - e) & ~low_bits(e_lo - e));
#pragma unroll
                        for (int u = 0; u < 32; u++)
                            s[h * 32 + u] = see >> u & 1 ? s[h * 32 + u] : -INFINITY;
                    }
#pragma unroll
                    for (int u = 0; u < 32; u += 8)
#pragma unroll
                        for (int z = 0; z < 4; z++)
                            mx[z] = fmax3(mx[z], s[h * 32 + u + z], s[h * 32 + u + 4 + z]);
                }
                const float top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * sh.scale2;
                const bool raise = top > m + kRaiseLog2;
                if (__any_sync(~0u, raise)) {
                    const float mn = raise ? top : m;
                    const float alpha = ex2(m - mn);
                    m = mn;
                    l *= alpha;
                    if (j > 0) {
                        // O holds the sum up to tile j - 1: once that is there, rescale it
                        ok = __all_sync(~0u, mbar_wait(&bars.pv_done[x][(c - 1) & 1], ((c - 1) >> 1) & 1,
                                                  abort_, flags));
                        if (!ok) break;
                        fence_after_sync();
#pragma unroll 1
                        for (int u = 0; u < D; u += 16) {
                            uint32_t r[16];
                            tmem_ld16(o_col + u, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int z = 0; z < 16; z++)
                                r[z] = __float_as_uint(__uint_as_float(r[z]) * alpha);
                            tmem_st16(o_col + u, r);
                        }
                    }
                }
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    if (h == 1 && !second) break;
                    uint32_t r[16];
#pragma unroll
                    for (int u = 0; u < 16; u++) {
                        const float p0 = ex2(fmaf(s[h * 32 + 2 * u], sh.scale2, -m));
                        const float p1 = ex2(fmaf(s[h * 32 + 2 * u + 1], sh.scale2, -m));
                        sum[u & 3] += p0 + p1;
                        r[u] = pack_bf16(p0, p1);
                    }
                    tmem_st16(s_col + h * 16, r);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_st_wait();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[x][c & 1]);
            }
            if (!ok) break;
            bars.ml[x][w.count & 1][row] = make_float2(m, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.ml_full[x][w.count & 1]);
            w.j = it.tiles - 1;
            w.next(sh, step);
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace win
}  // namespace hs2
