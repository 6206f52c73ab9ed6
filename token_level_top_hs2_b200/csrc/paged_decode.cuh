// One query token per sequence over a paged e4m3 cache with a scale per page
// and KV head: all of the sequence's tokens, or its last `window` and its first
// `n_sink`.
//   o = sum_s softmax_s(scale <q, k_s>) v_s,   lse = ln sum_s exp(scale <q, k_s>)
//
// The K and V codes go to the tensor cores as they are: 8-bit operands of
// tcgen05.mma kind::f8f6f4, straight from the TMA's shared-memory tiles, with
// tokens (QK^T) and dims (PV) as the 128 rows.  The other operand is split so
// that nothing is lost to its 8 bits:
//   * q (bf16, 8 significant bits) = hi + lo / 16, two e4m3 pieces of 4 bits
//     each after a common power of two per KV head that puts max|q| in
//     [128, 256).  Exact for every element above 2^-14 of the largest; below,
//     the error is at most 2^-21 of the largest.
//   * a weight w (nine significant bits, rounded to nearest) = three e5m2
//     pieces of 3 bits each, the top bytes of an f16 and of its exact
//     remainders; what falls below 2^-16 is dropped, with the largest weight
//     kept between 2^12 and 2^15.
// The pieces are columns of one MMA (N = 2 or 3 times the heads) and are summed
// in fp32.  The page's K scale multiplies the logit, its V scale the weight.
#pragma once

#include "tc.cuh"

namespace hs2 {
namespace pgd {

using namespace hs2::tc;

constexpr int kTile = 128;       // tokens per tile
constexpr int kThreads = 384;    // producer, QK, PV, Q warps and two softmax groups of four
constexpr int kMaxCtas = 148;    // one per SM
constexpr float kTopLog2 = 12.f;    // a raised reference maps the largest weight to 2^12
constexpr float kRaiseLog2 = 14.f;  // weights above 2^14 (before the V scale) raise it again

// A sequence's visible tokens as tiles: those of the first ns tokens, then
// those of the window [w0, T).
struct Span {
    int T, w0, ns, sink_tiles, first, tiles;
};
HS2_DEV Span span_of(int T, int window, int n_sink) {
    Span s;
    s.T = T;
    s.w0 = max(0, T - window);
    s.ns = min(n_sink, s.w0);
    s.sink_tiles = (s.ns + kTile - 1) / kTile;
    s.first = max(s.w0 / kTile, s.sink_tiles);
    s.tiles = s.sink_tiles + (T + kTile - 1) / kTile - s.first;
    if (T == 0) s.tiles = 0;
    return s;
}
HS2_DEV int length_of(const int32_t* lengths, int b, int cap, bool* bad) {
    const int T = __ldg(lengths + b);
    if (T >= 0 && T <= cap) return T;
    *bad = true;
    return 0;
}

// The tiles of all (sequence, KV head) items in one line, cut evenly over the
// CTAs: CTA c of n takes [c * total / n, (c + 1) * total / n).
HS2_DEV int64_t cut(int64_t total, int c, int n) { return (int64_t)c * total / n; }

struct Work {
    const int32_t* lengths;
    int B, cap, window, n_sink, Hkv;
};

// A walk along that line.
struct Walk {
    Span s;
    int b, h, t;
    HS2_DEV void load(const Work& w) {
        bool bad = false;
        s = span_of(length_of(w.lengths, b, w.cap, &bad), w.window, w.n_sink);
    }
    HS2_DEV void next(const Work& w, bool more) {
        if (++t < s.tiles) return;
        t = 0;
        if (++h < w.Hkv) return;
        h = 0;
        if (!more) return;
        do {
            b++;
            load(w);
        } while (s.tiles == 0 && b + 1 < w.B);
    }
    HS2_DEV int tile() const { return t < s.sink_tiles ? t : s.first + t - s.sink_tiles; }
    HS2_DEV bool last() const { return t + 1 == s.tiles; }
};

template <int D, int NG>
struct Cfg {
    static constexpr int KV = kTile * D;             // bytes of a K or V tile
    static constexpr int STAGES = D == 128 ? 6 : 12;
    static constexpr int NQ = 2 * NG;                // columns of a logit tile
    static constexpr int PLANES = NG == 16 ? 3 : 2;  // 16-byte planes of weight pieces per token
    static constexpr int NP = 16 * PLANES;           // columns of an output accumulator
    static constexpr int PB = PLANES * kTile * 16;   // bytes of a weight tile
    static constexpr int QB = NQ * D;                // bytes of an item's q pieces
    static constexpr int OFF_V = STAGES * KV;
    static constexpr int OFF_P = 2 * STAGES * KV;
    static constexpr int OFF_Q = OFF_P + 2 * PB;
    static constexpr int OFF_X = OFF_Q + 2 * QB;     // one group's result for the other
    static constexpr int SMEM = OFF_X + NG * D * 4 + 1024;
    static constexpr uint32_t COL_O = 4 * 32;        // S: 4 x 32 columns, O: 2 x 64
    static constexpr int PART = 16 * D + 32;         // floats of a partial result
    static_assert(SMEM <= 227 * 1024 - 4096, "shared memory");
};

struct Bars {
    uint64_t full[12], empty[12];
    uint64_t s_full[4], s_empty[4];  // [2 * group + buffer]
    uint64_t p_full[2], p_empty[2];  // [group]
    uint64_t q_full[2], q_empty[2], x_full, x_empty, drain[2];
    float2 sc[12][8];       // K and V scale of each page of a stage's tile
    uint32_t pages[12];     // which of them were there to load
    float qf[8];            // per item: scale log2(e) over q's power of two
    float red[2][4][20];    // per group and warp: per-head maxima or sums, largest V scale
    float xr[16], xl[16];
    unsigned long long total;
    int b0, h0, t0;
    uint32_t tmem;
    int abort_;
};

// Shared-memory matrix descriptor with another swizzle than sdesc_sw128's.
// layout: 0 none, 2 128-byte, 4 64-byte.
HS2_DEV uint64_t sdesc(uint32_t layout, uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)layout << 61;
}
// Instruction descriptor, kind::f8f6f4: fp32 accumulation, M = 128, A e4m3,
// B e4m3 (bfmt 0) or e5m2 (1).
constexpr uint32_t idesc_f8(int N, uint32_t bfmt, bool a_mn, bool b_mn) {
    return (1u << 4) | (bfmt << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
HS2_DEV void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
HS2_DEV void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Barrier of the 128 threads of a softmax group; true if any of them passes true.
HS2_DEV bool group_any(int group, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred), "r"(group + 1)
        : "memory");
    return r != 0;
}

template <int N>
HS2_DEV void tmem_ldn(uint32_t taddr, uint32_t (&r)[N]) {
    if constexpr (N == 32)
        tmem_ld32(taddr, r);
    else
        tmem_ld16(taddr, r);
}

template <int D, int NG, int PAGE>
__global__ void __launch_bounds__(kThreads, 1)
paged_decode_kernel(const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const __nv_bfloat16* __restrict__ q,
                    const float* __restrict__ k_scale, const float* __restrict__ v_scale,
                    const int32_t* __restrict__ table, const Work work, int G, int n_pages,
                    int max_pages, float scale2, __nv_bfloat16* __restrict__ o,
                    float* __restrict__ lse, float* __restrict__ part,
                    unsigned* __restrict__ flags) {
    using C = Cfg<D, NG>;
    constexpr int NST = C::STAGES;
    constexpr uint32_t SWZ = D == 128 ? 2 : 4;         // 128- or 64-byte rows
    constexpr uint32_t ATOM = 8 * D;                   // bytes of eight rows
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ Bars bars;
    const int tid = threadIdx.x, warp = tid >> 5, lane = lane_id();
    volatile int* abort_ = &bars.abort_;
    const int Hkv = work.Hkv;

    if (tid == 0) {
        for (int i = 0; i < NST; i++) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 4; i++) {
            mbar_init(&bars.s_full[i], 2);   // the MMAs, and the issuing thread itself
            mbar_init(&bars.s_empty[i], 4);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&bars.p_full[i], 4);
            mbar_init(&bars.p_empty[i], 1);
            mbar_init(&bars.q_full[i], 1);
            mbar_init(&bars.q_empty[i], 1);
            mbar_init(&bars.drain[i], 1);
        }
        mbar_init(&bars.x_full, 4);
        mbar_init(&bars.x_empty, 4);
        bars.abort_ = 0;
        bars.total = 0;
        bars.b0 = bars.h0 = bars.t0 = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars.tmem, 256);
        tmem_relinquish();
    }
    griddep_launch();
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&map_k);
        tma_prefetch_map(&map_v);
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    // the length of the whole line of tiles
    {
        unsigned long long n = 0;
        bool bad = false;
        for (int b = tid; b < work.B; b += kThreads)
            n += span_of(length_of(work.lengths, b, work.cap, &bad), work.window, work.n_sink).tiles;
        if (n) atomicAdd(&bars.total, n);
        if (bad && blockIdx.x == 0) atomicOr(flags, FLAG_BAD_LENGTH);
    }
    __syncthreads();
    const int64_t total = (int64_t)bars.total * Hkv;
    const int n_cta = (int)min((int64_t)gridDim.x, total), cta = blockIdx.x;
    const int64_t g0 = cta < n_cta ? cut(total, cta, n_cta) : 0;
    const int n_tiles = cta < n_cta ? (int)(cut(total, cta + 1, n_cta) - g0) : 0;
    if (n_tiles > 0 && warp == 0) {
        // the item that the CTA starts in
        int64_t before = 0;
        for (int b = 0; b < work.B; b += 32) {
            bool bad = false;
            const int nt = b + lane < work.B ? span_of(length_of(work.lengths, b + lane, work.cap, &bad),
                                                  work.window, work.n_sink).tiles
                                        : 0;
            int64_t sum = nt;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t u = __shfl_up_sync(~0u, sum, off);
                if (lane >= off) sum += u;
            }
            const int64_t at = g0 - (before + sum - nt) * Hkv;
            if (at >= 0 && at < (int64_t)nt * Hkv) {
                bars.b0 = b + lane;
                bars.h0 = (int)(at / nt);
                bars.t0 = (int)(at % nt);
            }
            before += __shfl_sync(~0u, sum, 31);
            if (before * Hkv > g0) break;
        }
    }
    __syncthreads();
    const uint32_t tmem = bars.tmem;
    Walk w = {};
    if (n_tiles > 0) {
        w.b = bars.b0, w.h = bars.h0, w.t = bars.t0;
        w.load(work);
    }

    if (warp == 0) {
        // ------------------------------------------------------ producer
        // A lane per page: 32 pages (TPB tiles) at a time, whose numbers and
        // scales are fetched while the tiles before them are issued.
        constexpr int PP = kTile / PAGE, TPB = 32 / PP;
        constexpr uint32_t BYTES = PAGE * D;
        int pid = -1, pos = 0;
        bool want = false;
        float ks = 0.f, vs = 0.f;
        int64_t ph = 0;
        int hk = 0;
        auto locate = [&](int i0) {  // this lane's page of tiles i0 .. i0 + TPB - 1
            want = false;
            for (int s = 0; s < TPB && i0 + s < n_tiles; s++) {
                if (lane / PP == s) {
                    const int p = w.tile() * PP + lane % PP;
                    pos = p * PAGE;
                    want = pos < w.s.T && (pos + PAGE > w.s.w0 || pos < w.s.ns);
                    pid = want ? __ldg(table + (size_t)w.b * max_pages + p) : -1;
                    hk = w.h;
                }
                w.next(work, i0 + s + 1 < n_tiles);
            }
        };
        auto scales = [&]() {
            if (want && (pid < 0 || pid >= n_pages)) {
                atomicOr(flags, FLAG_BAD_INDEX);
                want = false;
            }
            ph = (int64_t)pid * Hkv + hk;
            ks = want ? __ldg(k_scale + ph) : 0.f;
            vs = want ? __ldg(v_scale + ph) : 0.f;
        };
        int armed = 0;
        bool ok = true;
        locate(0);
        scales();
        for (int i0 = 0; ok && i0 < n_tiles; i0 += TPB) {
            const bool want_c = want;
            const float ks_c = ks, vs_c = vs;
            const int ph_c = (int)ph;
            for (int s = 0; s < TPB && i0 + s < n_tiles; s++) {
                const int i = i0 + s, st = i % NST;
                if (i >= NST)
                    ok = __all_sync(~0u, mbar_wait(&bars.empty[st], (i / NST - 1) & 1, abort_, flags));
                if (!ok) break;
                const bool mine = lane / PP == s, load = mine && want_c;
                if (mine) bars.sc[st][lane % PP] = make_float2(ks_c, vs_c);
                const uint32_t mask = __ballot_sync(~0u, load) >> (s * PP);
                if (lane == 0) bars.pages[st] = mask;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_expect_tx(&bars.full[st],
                                          2 * BYTES * __popc(mask & ((1u << PP) - 1)));
                __syncwarp();
                if (load) {
                    const int row = (lane % PP) * PAGE;
                    tma_load_3d(smem + st * C::KV + row * D, &map_k, 0, 0, ph_c, &bars.full[st]);
                    tma_load_3d(smem + C::OFF_V + st * C::KV + row * D, &map_v, 0, 0, ph_c,
                                &bars.full[st]);
                }
                armed++;
                if (s == 0) locate(i0 + TPB);
                if (s == TPB / 2) scales();
            }
        }
        if (*abort_) {  // let the copies still in flight land before the CTA leaves
            volatile int no_abort = 0;
            for (int i = max(0, armed - NST); i < armed; i++)
                mbar_wait(&bars.full[i % NST], (i / NST) & 1, &no_abort, flags);
        }
    } else if (warp == 1) {
        // ------------------------------------------------- S^T = K q^T
        constexpr uint32_t id = idesc_f8(C::NQ, 0, false, false);
        if (lane == 0 && n_tiles > 0) {
            bool fresh = true;
            int seg = 0;
            for (int i = 0; i < n_tiles; i++) {
                const int st = i % NST, sb = (i & 1) * 2 + ((i >> 1) & 1);
                if (fresh && !mbar_wait(&bars.q_full[seg & 1], (seg >> 1) & 1, abort_, flags)) break;
                if (!mbar_wait(&bars.full[st], (i / NST) & 1, abort_, flags)) break;
                if (i >= 4 && !mbar_wait(&bars.s_empty[sb], ((i >> 2) - 1) & 1, abort_, flags)) break;
                fence_after_sync();
                const uint32_t a = smem_u32(smem + st * C::KV);
                const uint32_t bq = smem_u32(smem + C::OFF_Q + (seg & 1) * C::QB);
#pragma unroll
                for (int ks = 0; ks < D / 32; ks++)
                    mma_f8(tmem + sb * 32, sdesc(SWZ, a + ks * 32, 16, ATOM),
                           sdesc(SWZ, bq + ks * 32, 16, ATOM), id, ks > 0);
                mma_commit(&bars.s_full[sb]);
                fresh = w.last();
                if (fresh) mma_commit(&bars.q_empty[seg++ & 1]);
                mbar_arrive(&bars.s_full[sb]);
                w.next(work, i + 1 < n_tiles);
            }
            mma_commit(&bars.drain[0]);
            volatile int no_abort = 0;
            mbar_wait(&bars.drain[0], 0, &no_abort, flags);
        }
    } else if (warp == 2) {
        // ----------------------------------------------- O^T += V^T w^T
        constexpr uint32_t id = idesc_f8(C::NP, 1, true, true);
        if (lane == 0 && n_tiles > 0) {
            bool acc[2] = {false, false};
            for (int i = 0; i < n_tiles; i++) {
                const int st = i % NST, g = i & 1;
                if (!mbar_wait(&bars.p_full[g], (i >> 1) & 1, abort_, flags)) break;
                fence_after_sync();
                const uint32_t a = smem_u32(smem + C::OFF_V + st * C::KV);
                const uint32_t bp = smem_u32(smem + C::OFF_P + g * C::PB);
#pragma unroll
                for (int ks = 0; ks < kTile / 32; ks++)
                    // V: dims contiguous, eight tokens per atom; 64 dims are read twice
                    // (a zero step between 64-dim blocks) for the 128 rows
                    mma_f8(tmem + C::COL_O + g * 64, sdesc(SWZ, a + ks * 32 * D, 0, ATOM),
                           sdesc(0, bp + ks * 512, 128, kTile * 16), id,
                           (acc[g] || ks > 0) ? 1u : 0u);
                mma_commit(&bars.empty[st]);
                mma_commit(&bars.p_empty[g]);
                acc[g] = true;
                if (w.last()) acc[0] = acc[1] = false;
                w.next(work, i + 1 < n_tiles);
            }
            mma_commit(&bars.drain[1]);
            volatile int no_abort = 0;
            mbar_wait(&bars.drain[1], 0, &no_abort, flags);
        }
    } else if (warp == 3) {
        // --------------------------------------------------- q's pieces
        int seg = 0;
        for (int i = 0; i < n_tiles; seg++) {
            if (seg >= 2 &&
                !__all_sync(~0u, mbar_wait(&bars.q_empty[seg & 1], ((seg >> 1) - 1) & 1, abort_, flags)))
                break;
            uint8_t* dst = smem + C::OFF_Q + (seg & 1) * C::QB;
            const __nv_bfloat16* src = q + ((size_t)w.b * Hkv + w.h) * G * D;
            constexpr int PER = NG * D / 8 / 32;  // 16-byte pieces per lane
            uint4 x[PER];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < PER; j++) {
                const int unit = j * 32 + lane;
                x[j] = unit / (D / 8) < G ? ldg_nc(src + unit * 8) : make_uint4(0, 0, 0, 0);
                const uint32_t m = __vmaxu2(__vmaxu2(x[j].x & 0x7FFF7FFFu, x[j].y & 0x7FFF7FFFu),
                                            __vmaxu2(x[j].z & 0x7FFF7FFFu, x[j].w & 0x7FFF7FFFu));
                top = max(top, max(m & 0xFFFFu, m >> 16));
            }
            top = __reduce_max_sync(~0u, top);
            if (top >= 0x7F80u && lane == 0) atomicOr(flags, FLAG_Q_RANGE);
            // 2^e max|q| in [128, 256)
            const int e = min(120, 7 - ((int)(top >> 7) - 127));
            const float f = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
            for (int j = 0; j < PER; j++) {
                const int unit = j * 32 + lane, h = unit / (D / 8), c = unit % (D / 8);
                const uint32_t in[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const float a = bf16_lo(in[u]) * f, b = bf16_hi(in[u]) * f;
                    uint16_t ph_, pl_;
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(ph_) : "f"(b), "f"(a));
                    const float2 r = f16x2_to_float2(e4m3x2_lo_to_f16x2(ph_));
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                        : "=h"(pl_)
                        : "f"((b - r.y) * 16.f), "f"((a - r.x) * 16.f));
                    hi[u >> 1] |= (uint32_t)ph_ << (16 * (u & 1));
                    lo[u >> 1] |= (uint32_t)pl_ << (16 * (u & 1));
                }
                // rows of D bytes, the 16-byte pieces of a row permuted as the
                // 128-byte (64-byte) swizzle has them
                auto at = [&](int row) {
                    const uint32_t a = (uint32_t)row * D + c * 8;
                    return a ^ (D == 128 ? (a >> 3) & 0x70u : (a >> 3) & 0x30u);
                };
                *reinterpret_cast<uint2*>(dst + at(h)) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2*>(dst + at(NG + h)) = make_uint2(lo[0], lo[1]);
            }
            if (lane == 0) bars.qf[seg & 7] = scale2 / f;
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.q_full[seg & 1]);
            // on to the next item
            const int left = w.s.tiles - w.t;
            i += left;
            w.t = w.s.tiles - 1;
            w.next(work, i < n_tiles);
        }
    } else {
        // ------------------------------------------------------ softmax
        // Two groups of four warps take the tiles in turn, each with its own
        // reference, sums and accumulator.  thread = token = TMEM lane of S^T,
        // and = dim = TMEM lane of O^T.  A wait that gives up clears ok; the
        // group leaves together at its next meeting (group_any).
        const int g = (warp >> 2) - 1, wq = warp & 3, row = wq * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        const uint32_t o_col = lanes + C::COL_O + g * 64;
        float R[NG], l[NG], vref = 0.f, vinv = 0.f;
        int own = 0, other = 0;    // tiles of the segment that each group takes
        int seg = 0, n_x = 0;      // segments and hand-overs so far
        bool at_start = true;        // the segment begins where the CTA does
        bool from_top = w.t == 0;    // the segment begins where its item does
        bool has = false, ok = true;  // R and vref are set
#pragma unroll
        for (int h = 0; h < NG; h++) R[h] = 0.f, l[h] = 0.f;

        for (int i = 0; i < n_tiles; i++) {
            if ((i & 1) == g) {
                const int k = i >> 1, st = i % NST, sb = g * 2 + (k & 1);
                ok = ok && mbar_wait(&bars.s_full[sb], (k >> 1) & 1, abort_, flags);
                fence_after_sync();
                const int s = w.tile() * kTile + row;
                const float2 sc = bars.sc[st][row / PAGE];
                const bool vis = s < w.s.T && (s >= w.s.w0 || s < w.s.ns) &&
                                 ((bars.pages[st] >> (row / PAGE)) & 1);
                const float f = vis ? sc.x * bars.qf[seg & 7] : 0.f;
                const float sv = vis ? sc.y : 0.f;
                uint32_t r[C::NQ];
                tmem_ldn<C::NQ>(lanes + sb * 32, r);
                tmem_ld_wait();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.s_empty[sb]);
                float y[NG], top = -INFINITY;
#pragma unroll
                for (int h = 0; h < NG; h++) {
                    const float x = fmaf(__uint_as_float(r[NG + h]), 0.0625f, __uint_as_float(r[h]));
                    y[h] = fmaf(x, f, -R[h]);
                    top = fmaxf(top, y[h]);
                }
                const bool raise = vis && (!has || top > kRaiseLog2 || sv > 2.f * vref);
                if (group_any(g, raise || !ok)) {
                    // a new reference (the segment's first tile, or a larger weight)
                    if (ok && own > 0)
                        ok = mbar_wait(&bars.p_empty[g], (k - 1) & 1, abort_, flags);
                    fence_after_sync();
#pragma unroll
                    for (int h = 0; h < NG; h++) {
                        float x = vis ? y[h] + R[h] : -INFINITY;
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 2));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
                        if (lane == 0) bars.red[g][wq][h] = x;
                    }
                    const float sm = __uint_as_float(
                        __reduce_max_sync(~0u, __float_as_uint(fmaxf(sv, 0.f))));
                    if (lane == 0) bars.red[g][wq][16] = sm;
                    if (group_any(g, !ok)) {
                        ok = false;
                        break;
                    }
                    float vnew = vref;
#pragma unroll
                    for (int u = 0; u < 4; u++) vnew = fmaxf(vnew, bars.red[g][u][16]);
                    const float beta = vnew > 0.f ? vref / vnew : 0.f;
                    vref = vnew;
                    vinv = vnew > 0.f ? 1.f / vnew : 0.f;
                    float a[NG];
#pragma unroll
                    for (int h = 0; h < NG; h++) {
                        float m = bars.red[g][0][h];
#pragma unroll
                        for (int u = 1; u < 4; u++) m = fmaxf(m, bars.red[g][u][h]);
                        const float Rn = has ? fmaxf(R[h], m - kTopLog2) : m - kTopLog2;
                        a[h] = has ? ex2(R[h] - Rn) : 0.f;
                        y[h] += R[h] - Rn;
                        R[h] = Rn;
                        l[h] *= a[h];
                    }
                    has = true;
                    if (own > 0) {
#pragma unroll
                        for (int c = 0; c < C::NP; c += 16) {
                            uint32_t v[16];
                            tmem_ld16(o_col + c, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int u = 0; u < 16; u++)
                                v[u] = __float_as_uint(__uint_as_float(v[u]) *
                                                       (a[(c + u) % NG] * beta));
                            tmem_st16(o_col + c, v);
                        }
                        tmem_st_wait();
                    }
                    fence_before_sync();
                }
                // weights, their sums and their pieces
                const float rv = sv * vinv;
                uint32_t pc[NG / 2];
#pragma unroll
                for (int h = 0; h < NG; h += 2) {
                    const float p0 = vis ? ex2(y[h]) : 0.f, p1 = vis ? ex2(y[h + 1]) : 0.f;
                    l[h] += p0;
                    l[h + 1] += p1;
                    // nine significant bits: half a step added, the last two bits cut
                    pc[h / 2] = (pack_f16(p0 * rv, p1 * rv) + 0x00020002u) & 0xFFFCFFFCu;
                }
                uint32_t b1[NG / 4], b2[NG / 4], b3[NG / 4];
#pragma unroll
                for (int j = 0; j < NG / 4; j++) {
                    uint32_t x0 = pc[2 * j], x1 = pc[2 * j + 1];
                    auto rest = [](uint32_t x) {
                        const uint32_t t = x & 0xFF00FF00u;
                        const __half2 d = __hsub2(*reinterpret_cast<__half2*>(&x),
                                                  *reinterpret_cast<const __half2*>(&t));
                        return *reinterpret_cast<const uint32_t*>(&d);
                    };
                    b1[j] = prmt(x0, x1, 0x7531u);
                    x0 = rest(x0), x1 = rest(x1);
                    b2[j] = prmt(x0, x1, 0x7531u);
                    x0 = rest(x0), x1 = rest(x1);
                    b3[j] = prmt(x0, x1, 0x7531u);
                }
                if (k > 0) ok = ok && mbar_wait(&bars.p_empty[g], (k - 1) & 1, abort_, flags);
                uint8_t* p = smem + C::OFF_P + g * C::PB + row * 16;
                if constexpr (NG == 16) {
                    *reinterpret_cast<uint4*>(p) = make_uint4(b1[0], b1[1], b1[2], b1[3]);
                    *reinterpret_cast<uint4*>(p + kTile * 16) = make_uint4(b2[0], b2[1], b2[2], b2[3]);
                    *reinterpret_cast<uint4*>(p + kTile * 32) = make_uint4(b3[0], b3[1], b3[2], b3[3]);
                } else {
                    *reinterpret_cast<uint4*>(p) = make_uint4(b1[0], b1[1], b2[0], b2[1]);
                    *reinterpret_cast<uint4*>(p + kTile * 16) = make_uint4(b3[0], b3[1], 0u, 0u);
                }
                if (!vis) {
                    // 0 * NaN is NaN: a row that is not visible must not hold one
                    ok = ok && mbar_wait(&bars.full[st], (i / NST) & 1, abort_, flags);
                    uint4* v = reinterpret_cast<uint4*>(smem + C::OFF_V + st * C::KV + row * D);
                    if (ok)
#pragma unroll
                        for (int u = 0; u < D / 16; u++) v[u] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[g]);
            }
            own += (i & 1) == g;
            other += (i & 1) != g;
            const bool item_end = w.last();
            if (item_end || i + 1 == n_tiles) {
                // ------------------------------------ the segment's result
                if (own > 0) {
                    const int k = (i - ((i & 1) != g)) >> 1;  // the group's last tile
                    ok = ok && mbar_wait(&bars.p_empty[g], k & 1, abort_, flags);
                    fence_after_sync();
#pragma unroll
                    for (int h = 0; h < NG; h++) {
                        float x = l[h];
#pragma unroll
                        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(~0u, x, off);
                        if (lane == 0) bars.red[g][wq][h] = x;
                    }
                    if (group_any(g, !ok)) {
                        ok = false;
                        break;
                    }
                    float O[NG];
                    {
                        uint32_t v[16];
                        tmem_ld16(o_col, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int h = 0; h < NG; h++) O[h] = __uint_as_float(v[h]);
                        if constexpr (NG == 8) {
#pragma unroll
                            for (int h = 0; h < NG; h++) O[h] += __uint_as_float(v[8 + h]);
                        }
#pragma unroll
                        for (int c = 16; c < C::NP; c += 16) {
                            tmem_ld16(o_col + c, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int h = 0; h < NG; h++) O[h] += __uint_as_float(v[h]);
                        }
                    }
                    fence_before_sync();
#pragma unroll
                    for (int h = 0; h < NG; h++) {
                        O[h] *= vref;
                        l[h] = 0.f;
#pragma unroll
                        for (int u = 0; u < 4; u++) l[h] += bars.red[g][u][h];
                        if (!has) R[h] = -1e30f;  // nothing visible: no weight when merged
                    }
                    float* xo = reinterpret_cast<float*>(smem + C::OFF_X);
                    const bool both = other > 0;
                    if (both && g == 1) {
                        // hand the result to group 0
                        if (n_x > 0)
                            ok = ok && mbar_wait(&bars.x_empty, (n_x - 1) & 1, abort_, flags);
                        if (row < D)
#pragma unroll
                            for (int h = 0; h < NG; h++) xo[h * D + row] = O[h];
                        if (row == 0)
#pragma unroll
                            for (int h = 0; h < NG; h++) bars.xr[h] = R[h], bars.xl[h] = l[h];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars.x_full);
                    } else {
                        if (both) {
                            ok = ok && mbar_wait(&bars.x_full, n_x & 1, abort_, flags);
#pragma unroll
                            for (int h = 0; h < NG; h++) {
                                const float xr = bars.xr[h], M = fmaxf(R[h], xr);
                                const float a = ex2(R[h] - M), b = ex2(xr - M);
                                O[h] = O[h] * a + (row < D ? xo[h * D + row] : 0.f) * b;
                                l[h] = l[h] * a + bars.xl[h] * b;
                                R[h] = M;
                            }
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bars.x_empty);
                        }
                        const size_t q0 = ((size_t)w.b * Hkv + w.h) * G;
                        if (ok && from_top && item_end) {
#pragma unroll
                            for (int h = 0; h < NG; h++) {
                                if (h >= G) break;
                                const bool any = l[h] != 0.f;
                                if (row < D)
                                    o[(q0 + h) * D + row] = __float2bfloat16(any ? O[h] / l[h] : 0.f);
                                if (lse && row == h)
                                    lse[q0 + h] = any ? (R[h] + log2f(l[h])) * kLn2 : -INFINITY;
                            }
                        } else if (ok) {
                            float* ps = part + (size_t)(2 * cta + (at_start ? 0 : 1)) * C::PART;
#pragma unroll
                            for (int h = 0; h < NG; h++) {
                                if (row < D) ps[h * D + row] = O[h];
                                if (row == h) ps[16 * D + h] = R[h], ps[16 * D + 16 + h] = l[h];
                            }
                        }
                    }
                    if (both) n_x++;
#pragma unroll
                    for (int h = 0; h < NG; h++) R[h] = 0.f, l[h] = 0.f;
                    vref = vinv = 0.f;
                    has = false;
                }
                own = other = 0;
                seg++;
                at_start = false;
                from_top = true;
            }
            w.next(work, i + 1 < n_tiles);
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_dealloc(tmem, 256);
    }
}

// Items cut between CTAs: their parts in the order of the line.  Sequences
// without visible tokens get zeros.  grid (Hkv, B), a thread per dim.
template <int D>
__global__ void __launch_bounds__(D)
paged_merge_kernel(const Work work, int G, int n_grid, __nv_bfloat16* __restrict__ o,
                   float* __restrict__ lse, const float* __restrict__ part) {
    constexpr int PART = 16 * D + 32;
    __shared__ unsigned long long s_before, s_total;
    const int tid = threadIdx.x, hk = blockIdx.x, b = blockIdx.y;
    if (tid == 0) s_before = s_total = 0;
    __syncthreads();
    unsigned long long before = 0, total = 0;
    bool bad = false;
    for (int i = tid; i < work.B; i += D) {
        const int nt = span_of(length_of(work.lengths, i, work.cap, &bad), work.window, work.n_sink).tiles;
        total += nt;
        if (i < b) before += nt;
    }
    if (total) atomicAdd(&s_total, total);
    if (before) atomicAdd(&s_before, before);
    __syncthreads();
    const int64_t all = (int64_t)s_total * work.Hkv;
    const int nt = span_of(length_of(work.lengths, b, work.cap, &bad), work.window, work.n_sink).tiles;
    const size_t q0 = ((size_t)b * work.Hkv + hk) * G;
    griddep_wait();
    if (nt == 0) {
        for (int h = 0; h < G; h++) {
            o[(q0 + h) * D + tid] = __float2bfloat16(0.f);
            if (lse && tid == h) lse[q0 + h] = -INFINITY;
        }
        return;
    }
    const int n = (int)min((int64_t)n_grid, all);
    const int64_t t0 = (int64_t)s_before * work.Hkv + (int64_t)hk * nt, t1 = t0 + nt;
    auto owner = [&](int64_t t) { return (int)(((t + 1) * n + all - 1) / all) - 1; };
    const int c0 = owner(t0), c1 = owner(t1 - 1);
    if (c0 == c1) return;
    const int first = 2 * c0 + (cut(all, c0, n) == t0 ? 0 : 1);
    for (int h = 0; h < G; h++) {
        float M = -INFINITY;
        for (int c = c0; c <= c1; c++)
            M = fmaxf(M, part[(size_t)(c == c0 ? first : 2 * c) * PART + 16 * D + h]);
        float O = 0.f, l = 0.f;
        for (int c = c0; c <= c1; c++) {
            const float* p = part + (size_t)(c == c0 ? first : 2 * c) * PART;
            const float a = ex2(p[16 * D + h] - M);
            O = fmaf(a, p[h * D + tid], O);
            l = fmaf(a, p[16 * D + 16 + h], l);
        }
        const bool any = l != 0.f;
        o[(q0 + h) * D + tid] = __float2bfloat16(any ? O / l : 0.f);
        if (lse && tid == h) lse[q0 + h] = any ? (M + log2f(l)) * kLn2 : -INFINITY;
    }
}

}  // namespace pgd
}  // namespace hs2
