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
//   * a weight w (nine significant bits, one more than a bf16 output has) =
//     a + b + c / 32,
//     three e5m2 pieces of 3 bits each: the top bytes of an f16, of its exact
//     remainder and of 32 times the next.  c's smallest step stands for 2^-21:
//     smaller weights round to a multiple of it, with the largest weight
//     kept between 2^8 and 2^14.  (Those six octaves are room for a maximum
//     that grows: with c unscaled and three octaves, a batch with uneven pages
//     raised its references 13 times per CTA and took 65.0 us, not 62.7.)
// The pieces are columns of one MMA (N = 2 or 3 times the heads, rounded up to
// 16) and are summed in fp32.  The page's K scale multiplies the logit, its V
// scale the weight: w = exp * V scale / C with a C per head that follows the
// largest product of the two, so that a page of large values that a head does
// not look at takes no bits from the pages that it does.  The token that sets C
// has the weight 2^8 exactly: a sharp softmax keeps its largest weight whole.
// The sum of the softmax is of the exponentials alone, in fp32.
//
// Measured: 16 sequences of 256k tokens, 16 heads of 128 (1.07 GB), 179 to 185
// us in a burst of calls (5.8 to 6.0 TB/s, 90 to 93% of a copy's rate), 207 over
// seconds at the power cap (5.2 TB/s, 80%); 48 ragged sequences with a window of
// 4096, 8 KV heads of 64 and groups of four (202 MB), 53.1 us either way or 3.8
// TB/s, bound by the softmax warps' latency per tile; one sequence of 1k tokens
// 12.4 us, of which 7 are one tile's way through the kernel (13k cycles: 3,500
// to the first copy, 3,500 to its logits, 2,200 for a first reference, 1,400 for
// weights and outputs, 2,500 for the part's end) and the merge most of the rest.
#pragma once

#include <float.h>

#include "kv_cache.cuh"
#include "tc.cuh"

namespace hs2 {
namespace pgd {

using namespace hs2::tc;
using kvc::e4m3x2;

constexpr int kTile = 128;       // tokens per tile
constexpr int kThreads = 512;    // QK, PV, q, -; four producers; two softmax groups of four
constexpr int kMaxCtas = 148;    // one per SM
constexpr float kTopLog2 = 8.f;     // a raised reference maps the largest weight to 2^8
constexpr float kHalfStep = 2.384185791015625e-7f;  // 2^-22, half of the pieces' smallest step
constexpr uint32_t kRaise = 0x7400; // weights above 2^14 (as f16) raise it again,
constexpr float kRaiseLogit = 60.f; // and so do exponentials above 2^60 (of pages with small scales)

// Scales of pages by their number in the CTA's line of tiles, modulo this: at
// most 12 stages x 8 pages in flight and two batches of 32 behind them.
constexpr int kScRing = 256;
constexpr float kAbsent = -INFINITY;

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

// The tiles of all (sequence, KV head) items in one line (at most 2^31 - 1, as
// the host checks), cut evenly over the CTAs: each takes `each`, the first
// `more` of them one more.
struct Cut {
    int each, more;
    HS2_DEV int start(int cta) const { return cta * each + min(cta, more); }
    // the CTA that owns tile t
    HS2_DEV int owner(int t) const {
        const int big = more * (each + 1);
        return t < big ? t / (each + 1) : more + (t - big) / each;
    }
};

// What a CTA leaves for the merge: where the parts of the item that it began
// and did not end are.  parts 0: it began none.
struct Split {
    int row, first, parts, unused;  // (sequence, KV head), the item's first part, their number
};

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
    // n tiles on, at most to the item's end; `more`: the line goes on behind them
    HS2_DEV void skip(const Work& w, int n, bool more) {
        t += n;
        if (t < s.tiles) return;
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
};

template <int D, int NG>
struct Cfg {
    static constexpr int KV = kTile * D;             // bytes of a K or V tile
    static constexpr int STAGES = D == 128 ? 6 : 12;
    static constexpr int NQ = NG == 4 ? 16 : 2 * NG;  // columns of a logit tile (4 heads leave half unread)
    static constexpr int PLANES = (3 * NG + 15) / 16;  // 16-byte planes of weight pieces per token
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
};

// A softmax group's references per head, and what a change multiplies its sums
// and its accumulator by (a copy per warp).
struct Refs {
    float R[16], ci[16], down[16], a[16];
};

struct Bars {
    uint64_t full[12], empty[12];
    uint64_t s_full[4], s_empty[4];  // [2 * group + buffer]
    uint64_t p_full[2];              // [group]
    uint64_t q_full[2], q_empty[2], x_full, x_empty, drain[2];
    float2 sc[kScRing];     // K and V scale of the line's pages, kAbsent for one not loaded
    float qf[2];            // per item & 1: scale log2(e) over the power of two in q's pieces
    float sqf[4];           // the same per logit buffer
    float red[2][4][32];    // per group and warp and head: maxima of logit and of weight, or sums
    float xr[16], xl[16];
    alignas(16) Refs refs[2][4];
    float C[2][16];         // per group and head: 1 / ci
    Cut cut;
    int n_cta, b0, h0, t0;  // CTAs with tiles; where this one starts
    uint32_t tmem;
    int abort_;
};
static_assert(Cfg<128, 16>::SMEM + sizeof(Bars) <= 227 * 1024 && Cfg<64, 16>::SMEM + sizeof(Bars) <= 227 * 1024,
              "shared memory");

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
HS2_DEV void mma_f8_w(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 1 / x of an x in [2^-126, 2^126], up to an eighth more
HS2_DEV float inverse(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

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

// Largest value of a warp's lanes (NaN left out).
HS2_DEV float warp_max(float x) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

template <int N>
HS2_DEV void tmem_ldn(uint32_t taddr, uint32_t (&r)[N]) {
    if constexpr (N == 32)
        tmem_ld32(taddr, r);
    else if constexpr (N == 16)
        tmem_ld16(taddr, r);
    else
        tmem_ld8(taddr, r);
}

// One warp splits the G <= NG queries of an item (rows of D bf16) into the
// rows of their e4m3 pieces, hi in rows 0 .. NG-1 and lo in the next NG, in the
// K-major layout of the TMA's swizzle.  Returns their power of two.
template <int D, int NG>
HS2_DEV float split_q(const __nv_bfloat16* __restrict__ src, int G, uint8_t* dst,
                      unsigned* flags) {
    constexpr int PER = NG * D / 8 / 32;  // 16-byte pieces per lane
    const int lane = lane_id();
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
            const uint32_t p = e4m3x2(a, b);
            const float2 r = f16x2_to_float2(e4m3x2_lo_to_f16x2(p));
            hi[u >> 1] |= p << (16 * (u & 1));
            lo[u >> 1] |= e4m3x2((a - r.x) * 16.f, (b - r.y) * 16.f) << (16 * (u & 1));
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
    return f;
}

template <int D, int NG, int PAGE>
__global__ void __launch_bounds__(kThreads, 1)
paged_decode_kernel(const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const __nv_bfloat16* __restrict__ q,
                    const float* __restrict__ k_scale, const float* __restrict__ v_scale,
                    const int32_t* __restrict__ table, const Work work, int G, int n_pages,
                    int max_pages, float scale2, __nv_bfloat16* __restrict__ o,
                    float* __restrict__ lse, float* __restrict__ part,
                    Split* __restrict__ splits, unsigned* __restrict__ flags) {
    using C = Cfg<D, NG>;
    constexpr int NST = C::STAGES;
    constexpr uint32_t SWZ = D == 128 ? 2 : 4;         // 128- or 64-byte rows
    constexpr uint32_t ATOM = 8 * D;                   // bytes of eight rows
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ Bars bars;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = lane_id();
    volatile int* abort_ = &bars.abort_;
    const int Hkv = work.Hkv;

    if (tid == 0) {
        for (int i = 0; i < NST; i++) {
            mbar_init(&bars.full[i], 2);   // the K and the V producer
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 4; i++) {
            mbar_init(&bars.s_full[i], 2);   // the MMAs, and the warp that issues them
            mbar_init(&bars.s_empty[i], 4);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&bars.p_full[i], 4);
            mbar_init(&bars.q_full[i], 1);
            mbar_init(&bars.q_empty[i], 1);
            mbar_init(&bars.drain[i], 1);
        }
        mbar_init(&bars.x_full, 4);
        mbar_init(&bars.x_empty, 4);
        bars.abort_ = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars.tmem, 256);
        tmem_relinquish();
    }
    griddep_launch();
    if (warp == 4) {
        tma_prefetch_map(&map_k);
        tma_prefetch_map(&map_v);
    }
    if (warp == 3 && lane == 0) splits[blockIdx.x] = Split{0, 0, 0, 0};
    if (warp == 2) {
        // the length of the whole line of tiles, and the item that the CTA starts in
        const int cta = blockIdx.x;
        bool bad = false;
        int total = 0;
#pragma unroll 4
        for (int b = lane; b < work.B; b += 32)
            total += span_of(length_of(work.lengths, b, work.cap, &bad), work.window, work.n_sink).tiles;
        if (bad && cta == 0) atomicOr(flags, FLAG_BAD_LENGTH);
        total = __reduce_add_sync(~0u, total) * Hkv;
        const int n = min((int)gridDim.x, total);
        const Cut cut = {n > 0 ? total / n : 0, n > 0 ? total % n : 0};
        if (lane == 0) bars.cut = cut, bars.n_cta = n, bars.b0 = bars.h0 = bars.t0 = 0;
        __syncwarp();
        if (cta < n) {
            const int first = cut.start(cta);
            int before = 0;
            for (int b = 0; b < work.B && before * Hkv <= first; b += 32) {
                const int nt = b + lane < work.B ? span_of(length_of(work.lengths, b + lane, work.cap, &bad),
                                                           work.window, work.n_sink).tiles
                                                 : 0;
                int upto = nt;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int u = __shfl_up_sync(~0u, upto, off);
                    if (lane >= off) upto += u;
                }
                const int at = first - (before + upto - nt) * Hkv;
                if (at >= 0 && at < nt * Hkv) {
                    bars.b0 = b + lane;
                    bars.h0 = at / nt;
                    bars.t0 = at % nt;
                }
                before += __shfl_sync(~0u, upto, 31);
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const int cta = blockIdx.x;
    const int n_tiles = cta < bars.n_cta ? bars.cut.each + (cta < bars.cut.more ? 1 : 0) : 0;
    const uint32_t tmem = __shfl_sync(~0u, bars.tmem, 0);
    const uint32_t base = __shfl_sync(~0u, smem_u32(smem), 0);
    Walk w = {};
    if (n_tiles > 0) {
        w.b = bars.b0, w.h = bars.h0, w.t = bars.t0;
        w.load(work);
    }

    // (16 heads' softmax needs more registers than 512 threads get at launch;
    // the 65,536 are 512 x 128 = 256 x 80 + 256 x 176)
    if (warp < 8) {
        if constexpr (NG == 16) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp >= 4) {
            // ------------------------------------------------------ producers
            // Warps 4 and 6 load K, 5 and 7 V, of every other tile (D = 64; D =
            // 128: 4 and 5 of all tiles): a warp's copies move at most 14 bytes
            // per cycle whatever their size (its scheduler's share of the copy
            // engine), two warps' 24 to 28, four warps' what the memory gives, 30
            // to 33.  At D = 128 four warps took 183 us against two warps' 179,
            // since SMs then get unequal shares of the memory; at D = 64, with
            // half the bytes per tile, 67.7 against 74.
            // A lane per page: 32 pages (a batch of TPB of the warp's tiles) at a
            // time, whose numbers and scales are fetched while the tiles before
            // them are issued.
            constexpr int PP = kTile / PAGE, TPB = 32 / PP;
            constexpr int EVERY = D == 128 ? 1 : 2;
            const int is_v = warp & 1, odd = (warp >> 1) & 1;
            // the warp's tiles: odd, odd + EVERY, ...
            const int n_own = odd < EVERY ? (n_tiles + EVERY - 1 - odd) / EVERY : 0;
            if (odd && n_own > 0) w.skip(work, 1, true);
            const float* scale = is_v ? v_scale : k_scale;
            const CUtensorMap* map = is_v ? &map_v : &map_k;
            const uint32_t ring = base + (is_v ? C::OFF_V : 0);
            Walk mine = w;      // where this lane's page is
            int pid = -1;
            bool want = false;
            float sc = 0.f;
            int ph = -1;
            // this lane's page of the warp's tiles i0 .. i0 + TPB - 1, and its number
            auto locate = [&](int i0) {
                mine = w;
                int left = EVERY * min(lane / PP, n_own - 1 - i0);  // tiles on from i0's
                while (left > 0 && mine.t + left >= mine.s.tiles) {
                    const int n = mine.s.tiles - mine.t;
                    left -= n;
                    mine.skip(work, n, true);
                }
                mine.t += max(left, 0);
                const int p = mine.tile() * PP + lane % PP, pos = p * PAGE;
                want = i0 + lane / PP < n_own && pos < mine.s.T &&
                       (pos + PAGE > mine.s.w0 || pos < mine.s.ns);
                pid = want ? __ldg(table + (size_t)mine.b * max_pages + p) : -1;
            };
            // the first tile of the batch behind lane 31's
            auto move_on = [&](int i0) {
                if (i0 + TPB >= n_own) return;
                w.b = __shfl_sync(~0u, mine.b, 31);
                w.h = __shfl_sync(~0u, mine.h, 31);
                w.t = __shfl_sync(~0u, mine.t, 31);
                w.load(work);
                for (int u = 0; u < EVERY; u++) w.skip(work, 1, true);
            };
            auto scales = [&]() {
                if (want && (pid < 0 || pid >= n_pages)) {
                    atomicOr(flags, FLAG_BAD_INDEX);
                    want = false;
                }
                ph = want ? pid * Hkv + mine.h : -1;
                sc = want ? __ldg(scale + ph) : kAbsent;
            };
            int armed = 0, st = odd;
            uint32_t ring_phase = 1;  // of the empty barriers: the first round passes
            bool ok = true;
            locate(0);
            scales();
            for (int i0 = 0; ok && i0 < n_own; i0 += TPB) {
                const int cnt = min(TPB, n_own - i0), ph_c = ph;
                float2* to = &bars.sc[((EVERY * (i0 + lane / PP) + odd) * PP + lane % PP) & (kScRing - 1)];
                if (is_v)
                    to->y = sc;
                else
                    to->x = sc;
                __syncwarp();
                move_on(i0);
                locate(i0 + TPB);  // (their numbers arrive during the first half)
                for (int j = 0; j < cnt; j++) {
                    int phs[PP], n = 0;
#pragma unroll
                    for (int u = 0; u < PP; u++) phs[u] = __shfl_sync(~0u, ph_c, j * PP + u);
#pragma unroll
                    for (int u = 0; u < PP; u++) n += phs[u] >= 0;
                    ok = wait_warp(&bars.empty[st], ring_phase, abort_, flags);
                    if (!ok) break;
                    mbar_arrive_expect_tx_w(&bars.full[st], PAGE * D * n);
#pragma unroll
                    for (int u = 0; u < PP; u++)
                        if (phs[u] >= 0)
                            tma_load_3d_w(ring + st * C::KV + u * PAGE * D, map, 0, 0, phs[u], &bars.full[st]);
                    armed++;
                    st += EVERY;
                    if (st >= NST) st -= NST, ring_phase ^= 1;
                    if (j == (cnt - 1) / 2) scales();
                }
            }
            if (*abort_) {  // let the copies in flight land before the CTA leaves
                // (the other producer's share of a barrier may never come: the wait
                // is bounded, and by its end the copies have landed)
                volatile int no_abort = 0;
                for (int j = max(0, armed - NST / EVERY); j < armed; j++)
                    mbar_wait(&bars.full[(EVERY * j + odd) % NST], ((EVERY * j + odd) / NST) & 1, &no_abort,
                              flags);
            }
        } else if (warp == 0) {
            // ------------------------------------------------- S^T = K q^T
            constexpr uint32_t id = idesc_f8(C::NQ, 0, false, false);
            if (n_tiles > 0) {
                const uint64_t a0 = sdesc(SWZ, base, 16, ATOM), q0 = sdesc(SWZ, base + C::OFF_Q, 16, ATOM);
                int st = 0, seg = 0;
                uint32_t ring_phase = 0;
                bool ok = true;
                for (int i = 0; ok && i < n_tiles; seg++) {
                    const int n = min(w.s.tiles - w.t, n_tiles - i);
                    ok = wait_warp(&bars.q_full[seg & 1], (seg >> 1) & 1, abort_, flags);
                    const float qf = bars.qf[seg & 1];
                    for (const int end = i + n; ok && i < end; i++) {
                        const int sb = (i & 1) * 2 + ((i >> 1) & 1);
                        if (!wait_warp(&bars.full[st], ring_phase, abort_, flags) ||
                            !wait_warp(&bars.s_empty[sb], ((i >> 2) & 1) ^ 1, abort_, flags)) {
                            ok = false;
                            break;
                        }
                        fence_after_sync();
                        const uint64_t a = a0 + ((st * C::KV) >> 4), bq = q0 + (((seg & 1) * C::QB) >> 4);
#pragma unroll
                        for (int ks = 0; ks < D / 32; ks++)
                            mma_f8_w(tmem + sb * 32, a + ks * 2, bq + ks * 2, id, ks > 0);
                        mma_commit_w(&bars.s_full[sb]);
                        if (i + 1 == end) mma_commit_w(&bars.q_empty[seg & 1]);
                        if (lane == 0) {
                            bars.sqf[sb] = qf;
                            mbar_arrive(&bars.s_full[sb]);
                        }
                        __syncwarp();
                        if (++st == NST) st = 0, ring_phase ^= 1;
                    }
                    w.skip(work, n, i < n_tiles);
                }
                mma_commit_w(&bars.drain[0]);
                volatile int no_abort = 0;
                mbar_wait(&bars.drain[0], 0, &no_abort, flags);
            }
        } else if (warp == 1) {
            // ----------------------------------------------- O^T += V^T w^T
            constexpr uint32_t id = idesc_f8(C::NP, 1, true, true);
            if (n_tiles > 0) {
                // V: dims contiguous, eight tokens per atom; 64 dims are read twice
                // (a zero step between 64-dim blocks) for the 128 rows
                const uint64_t a0 = sdesc(SWZ, base + C::OFF_V, 0, ATOM);
                const uint64_t p0 = sdesc(0, base + C::OFF_P, 128, kTile * 16);
                int st = 0;
                bool ok = true;
                for (int i = 0; ok && i < n_tiles;) {
                    const int n = min(w.s.tiles - w.t, n_tiles - i);
                    for (int j = 0; j < n; j++, i++) {
                        const int g = i & 1;
                        if (!wait_warp(&bars.p_full[g], (i >> 1) & 1, abort_, flags)) {
                            ok = false;
                            break;
                        }
                        fence_after_sync();
                        const uint64_t a = a0 + ((st * C::KV) >> 4), bp = p0 + ((g * C::PB) >> 4);
#pragma unroll
                        for (int ks = 0; ks < kTile / 32; ks++)
                            mma_f8_w(tmem + C::COL_O + g * 64, a + ((ks * 32 * D) >> 4),
                                     bp + ((ks * 512) >> 4), id, (j > 1 || ks > 0) ? 1u : 0u);
                        mma_commit_w(&bars.empty[st]);
                        if (++st == NST) st = 0;
                    }
                    w.skip(work, n, i < n_tiles);
                }
                mma_commit_w(&bars.drain[1]);
                volatile int no_abort = 0;
                mbar_wait(&bars.drain[1], 0, &no_abort, flags);
            }
        } else if (warp == 3) {
            // ------------------------- sequences without visible tokens
            const int row = Hkv * G * D;
            for (int b = cta; b < work.B; b += gridDim.x) {
                bool bad = false;
                if (length_of(work.lengths, b, work.cap, &bad) > 0) continue;
                for (int e = lane * 8; e < row; e += 256)
                    *reinterpret_cast<uint4*>(o + (size_t)b * row + e) = make_uint4(0, 0, 0, 0);
                if (lse)
                    for (int h = lane; h < Hkv * G; h += 32) lse[(size_t)b * Hkv * G + h] = -INFINITY;
            }
        } else if (warp == 2) {
            // --------------------------------------------------- q's pieces
            bool ok = true;
            int seg = 0;
            for (int i = 0; ok && i < n_tiles; seg++) {
                ok = wait_warp(&bars.q_empty[seg & 1], ((seg >> 1) & 1) ^ 1, abort_, flags);
                if (!ok) break;
                const float f = split_q<D, NG>(q + ((size_t)w.b * Hkv + w.h) * G * D, G,
                                               smem + C::OFF_Q + (seg & 1) * C::QB, flags);
                if (lane == 0) bars.qf[seg & 1] = scale2 / f;
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.q_full[seg & 1]);
                const int n = min(w.s.tiles - w.t, n_tiles - i);
                i += n;
                w.skip(work, n, i < n_tiles);
            }
        }
    } else {
        // (waits in line: a call would keep the compiler from the extra registers)
        if constexpr (NG == 16) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        // ------------------------------------------------------ softmax
        // Two groups of four warps take the tiles in turn, each with its own
        // reference, sums and accumulator.  thread = token = TMEM lane of S^T,
        // and = dim = TMEM lane of O^T.  A wait that gives up clears ok; the
        // group leaves together at its next meeting (group_any).
        const int g = (warp >> 2) - 2, wq = warp & 3, row = wq * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        const uint32_t o_col = lanes + C::COL_O + g * 64;
        // rounds two f16 to nine significant bits: halves go up at even tokens and
        // down at odd ones (all up, outputs came out 2^-11.5 too large)
        const uint32_t nine = lane & 1 ? 0x00010001u : 0x00020002u;
        // exponentials are 2^(logit - R), weights exponential * V scale * ci; svlim
        // keeps V scale * ci finite, below svlow it may be under 2^-40
        float R[NG], ci[NG], l[NG], svlim = FLT_MAX, svlow = 0.f;
        int n_x = 0;                  // hand-overs so far
        int st = g, st_was = 0;       // stages of the group's tile and of its last one
        uint32_t ph = 0, ph_was = 0;  // and their barriers' phases
        bool at_start = true;         // the segment begins where the CTA does
        bool from_top = w.t == 0;     // the segment begins where its item does
        bool has = false, ok = true;  // R and ci are set; no wait has given up
#pragma unroll
        for (int h = 0; h < NG; h++) R[h] = 0.f, ci[h] = 1.f, l[h] = 0.f;

        for (int i0 = 0; i0 < n_tiles;) {
            const int n = min(w.s.tiles - w.t, n_tiles - i0);  // tiles of the segment
            const int mine = (n + 1 - ((i0 ^ g) & 1)) / 2, others = n - mine;
            int j = (i0 ^ g) & 1;
            for (; j < n; j += 2) {
                const int k = (i0 + j) >> 1, sb = g * 2 + (k & 1);
                const int t = w.t + j;
                const int s = (t < w.s.sink_tiles ? t : w.s.first + t - w.s.sink_tiles) * kTile + row;
                // the tile's copies have landed: its scales are there
                ok = ok && mbar_wait(&bars.full[st], ph, abort_, flags);
                const float2 sc = bars.sc[((i0 + j) * (kTile / PAGE) + row / PAGE) & (kScRing - 1)];
                const bool vis = s < w.s.T && (s >= w.s.w0 || s < w.s.ns) && sc.x != kAbsent;
                const float sv = vis ? sc.y : 0.f;
                ok = ok && mbar_wait(&bars.s_full[sb], (k >> 1) & 1, abort_, flags);
                fence_after_sync();
                const float f = vis ? sc.x * bars.sqf[sb] : 0.f;
                uint32_t r[2 * NG];
                tmem_ldn<2 * NG>(lanes + sb * 32, r);
                tmem_ld_wait();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.s_empty[sb]);
                // exponentials, and weights: nine significant bits, and no step below
                // 2^-21: half a step of each added, what is below it cut
                float y[NG], p[NG];
                uint32_t pc[NG / 2], top = 0;
                auto weigh = [&]() {
                    const float svc = fminf(sv, svlim);
#pragma unroll
                    for (int h = 0; h < NG; h += 2) {
                        p[h] = vis ? ex2(y[h]) : 0.f;
                        p[h + 1] = vis ? ex2(y[h + 1]) : 0.f;
                        pc[h / 2] = pack_f16(fmaf(p[h], svc * ci[h], kHalfStep),
                                             fmaf(p[h + 1], svc * ci[h + 1], kHalfStep));
                    }
                };
#pragma unroll
                for (int h = 0; h < NG; h++) {
                    const float x = fmaf(__uint_as_float(r[NG + h]), 0.0625f, __uint_as_float(r[h]));
                    y[h] = fmaf(x, f, -R[h]);
                }
                weigh();
                // (non-negative: their bits order as they do)
#pragma unroll
                for (int h = 0; h < NG / 2; h++) top = __vmaxu2(top, pc[h]);
                bool raise = !has || max(top & 0xFFFFu, top >> 16) > kRaise;
                if (vis && sv < svlow) {  // (weights too small to tell how large the exponentials are)
#pragma unroll
                    for (int h = 0; h < NG; h++) raise |= y[h] > kRaiseLogit;
                }
                if (group_any(g, (raise && vis) || !ok)) {
                    // new references (the segment's first tile, or a larger weight)
                    if (j > 1) ok = ok && mbar_wait(&bars.empty[st_was], ph_was, abort_, flags);
                    fence_after_sync();
                    // the tile's largest logit and largest log2 of exponential * V scale
                    const float lsv = vis ? __log2f(sv) : -INFINITY;
#pragma unroll
                    for (int h = 0; h < NG; h++) {
                        const float x = vis ? y[h] + R[h] : -INFINITY;
                        const float xm = warp_max(x), zm = warp_max(x + lsv);
                        if (lane == 0) bars.red[g][wq][h] = xm, bars.red[g][wq][NG + h] = zm;
                    }
                    if (group_any(g, !ok)) {
                        ok = false;
                        break;
                    }
                    // each warp for itself, a lane per head
                    Refs& refs = bars.refs[g][wq];
                    {
                        const int h = lane % NG;
                        float xm = bars.red[g][0][h], zm = bars.red[g][0][NG + h];
#pragma unroll
                        for (int u = 1; u < 4; u++) {
                            xm = fmaxf(xm, bars.red[g][u][h]);
                            zm = fmaxf(zm, bars.red[g][u][NG + h]);
                        }
                        xm -= kTopLog2;
                        const float Ro = has ? refs.R[h] : xm, co = has ? refs.ci[h] : 0x1p125f;
                        float Rn = fmaxf(Ro, xm);
                        if (Rn == -INFINITY) Rn = 0.f;  // (logits of NaN alone)
                        const float e = fminf(fmaxf(Rn + kTopLog2 - zm, -125.f), 125.f);
                        float cn = fminf(ex2(e), co * ex2(fminf(Rn - Ro, 125.f)));
                        // at most 2^60 apart, so that svlim touches only tokens that
                        // contribute less than 2^-67 of their V scale to any head (a
                        // head may look at a page of zeros alone, whose scale is 2^-126)
                        const float least = -warp_max(-cn);
                        cn = fminf(cn, least * 0x1p60f);
                        const float down = has ? ex2(Ro - Rn) : 0.f;
                        svlim = inverse(warp_max(cn)) * 0x1p126f * 2.f;  // (at most infinity)
                        svlow = inverse(least) * 0x1p-40f;
                        __syncwarp();
                        refs.R[h] = Rn, refs.ci[h] = cn, refs.down[h] = down;
                        refs.a[h] = __fdividef(cn * down, co);
                        bars.C[g][h] = __fdividef(1.f, cn);  // (the same from every warp)
                        __syncwarp();
                    }
                    has = true;
#pragma unroll
                    for (int h = 0; h < NG; h++) {
                        y[h] += R[h] - refs.R[h];
                        R[h] = refs.R[h];
                        ci[h] = refs.ci[h];
                        l[h] *= refs.down[h];
                    }
                    if (j > 1) {
#pragma unroll 1
                        for (int c = 0; c < C::NP; c += 16) {
                            uint32_t v[16];
                            tmem_ld16(o_col + c, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int u = 0; u < 16; u++)
                                v[u] = __float_as_uint(__uint_as_float(v[u]) * refs.a[u % NG]);
                            tmem_st16(o_col + c, v);
                        }
                        tmem_st_wait();
                    }
                    fence_before_sync();
                    weigh();
                }
                // the exponentials' sums, and the weights' pieces
#pragma unroll
                for (int h = 0; h < NG; h += 2) {
                    l[h] += p[h];
                    l[h + 1] += p[h + 1];
                    pc[h / 2] = (pc[h / 2] + nine) & 0xFFFCFFFCu;
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
                    auto times32 = [](uint32_t x) {
                        const __half2 d = __hmul2(*reinterpret_cast<__half2*>(&x), __float2half2_rn(32.f));
                        return *reinterpret_cast<const uint32_t*>(&d);
                    };
                    b1[j] = prmt(x0, x1, 0x7531u);
                    x0 = rest(x0), x1 = rest(x1);
                    b2[j] = prmt(x0, x1, 0x7531u);
                    x0 = times32(rest(x0)), x1 = times32(rest(x1));
                    b3[j] = prmt(x0, x1, 0x7531u);
                }
                if (k > 0) ok = ok && mbar_wait(&bars.empty[st_was], ph_was, abort_, flags);
                uint8_t* pp = smem + C::OFF_P + g * C::PB + row * 16;
                if constexpr (NG == 16) {
                    *reinterpret_cast<uint4*>(pp) = make_uint4(b1[0], b1[1], b1[2], b1[3]);
                    *reinterpret_cast<uint4*>(pp + kTile * 16) = make_uint4(b2[0], b2[1], b2[2], b2[3]);
                    *reinterpret_cast<uint4*>(pp + kTile * 32) = make_uint4(b3[0], b3[1], b3[2], b3[3]);
                } else if constexpr (NG == 8) {
                    *reinterpret_cast<uint4*>(pp) = make_uint4(b1[0], b1[1], b2[0], b2[1]);
                    *reinterpret_cast<uint4*>(pp + kTile * 16) = make_uint4(b3[0], b3[1], 0u, 0u);
                } else {
                    *reinterpret_cast<uint4*>(pp) = make_uint4(b1[0], b2[0], b3[0], 0u);
                }
                if (!vis) {
                    // 0 * NaN is NaN: a row that is not visible must not hold one
                    uint4* v = reinterpret_cast<uint4*>(smem + C::OFF_V + st * C::KV + row * D);
                    if (ok)
#pragma unroll
                        for (int u = 0; u < D / 16; u++) v[u] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[g]);
                st_was = st, ph_was = ph;
                st += 2;
                if (st >= NST) st -= NST, ph ^= 1;
            }
            if (j < n) break;  // the group has given up
            const bool item_end = w.t + n == w.s.tiles;
            if (mine > 0) {
                // ------------------------------------ the segment's result
                ok = ok && mbar_wait(&bars.empty[st_was], ph_was, abort_, flags);
                fence_after_sync();
                // sums over the warp's lanes: each step halves the heads a lane holds
#pragma unroll
                for (int c = NG / 2, off = 16; off > 0; c /= 2, off /= 2) {
                    const bool up = lane & off;
                    if (c == 0) {
                        l[0] += __shfl_xor_sync(~0u, l[0], off);
                    } else {
#pragma unroll
                        for (int h = 0; h < c; h++) {
                            const float give = up ? l[h] : l[h + c];
                            l[h] = (up ? l[h + c] : l[h]) + __shfl_xor_sync(~0u, give, off);
                        }
                    }
                }
                if (lane % (32 / NG) == 0) bars.red[g][wq][lane / (32 / NG)] = l[0];
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
                    if constexpr (NG == 4) {
#pragma unroll
                        for (int h = 0; h < NG; h++)
                            O[h] = fmaf(__uint_as_float(v[8 + h]), 0.03125f, O[h] + __uint_as_float(v[4 + h]));
                    }
#pragma unroll
                    for (int c = 16; c < C::NP; c += 16) {
                        tmem_ld16(o_col + c, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int h = 0; h < NG; h++) O[h] = fmaf(__uint_as_float(v[h]), c == C::NP - 16 ? 0.03125f : 1.f, O[h]);
                    }
                }
                fence_before_sync();
#pragma unroll
                for (int h = 0; h < NG; h++) {
                    l[h] = 0.f;
#pragma unroll
                    for (int u = 0; u < 4; u++) l[h] += bars.red[g][u][h];
                    // over the power of two in l, so that O is at most twice the
                    // segment's largest value (division by l itself: 2 us more)
                    const uint32_t two = __float_as_uint(l[h]) & 0x7F800000u;
                    const float ln = __uint_as_float((254u << 23) - two);
                    O[h] = has ? O[h] * ln * bars.C[g][h] : 0.f;
                    l[h] *= ln;
                    R[h] += (float)((int)(two >> 23) - 127);
                    if (!has) R[h] = -1e30f;  // nothing visible: no weight when merged
                }
                float* xo = reinterpret_cast<float*>(smem + C::OFF_X);
                const bool both = others > 0;
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
                                o[(q0 + h) * D + row] = __float2bfloat16(any ? O[h] * __frcp_rn(l[h]) : 0.f);
                            if (lse && row == h)
                                lse[q0 + h] = any ? (R[h] + log2f(l[h])) * kLn2 : -INFINITY;
                        }
                    } else if (ok) {
                        if (from_top && row == 0) {
                            const int last = bars.cut.start(cta) + i0 + w.s.tiles - 1;
                            splits[cta] = Split{w.b * Hkv + w.h, 2 * cta + (at_start ? 0 : 1),
                                                bars.cut.owner(last) - cta + 1, 0};
                        }
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
                for (int h = 0; h < NG; h++) R[h] = 0.f, ci[h] = 1.f, l[h] = 0.f;
                svlim = FLT_MAX, svlow = 0.f;
                has = false;
                }
            at_start = false;
            from_top = true;
            i0 += n;
            w.skip(work, n, i0 < n_tiles);
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_dealloc(tmem, 256);
    }
}

// Items cut between CTAs: their parts in the order of the line.  grid (CTAs of
// the kernel before, G): the item that CTA began, a thread per dim; the parts'
// references and sums are read by a lane each, their outputs eight at a time.
template <int D>
__global__ void __launch_bounds__(D)
paged_merge_kernel(int G, __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
                   const float* __restrict__ part, const Split* __restrict__ splits) {
    constexpr int PART = 16 * D + 32;
    __shared__ float s_a[kMaxCtas];
    const int tid = threadIdx.x, c0 = blockIdx.x, h = blockIdx.y;
    griddep_wait();
    const Split sp = splits[c0];
    const int np = sp.parts;
    if (np == 0) return;
    const size_t row = (size_t)sp.row * G + h;
    auto at = [&](int i) { return part + (size_t)(i == 0 ? sp.first : 2 * (c0 + i)) * PART; };
    // every warp finds the common reference and the sum
    float M = -INFINITY, l = 0.f;
    for (int i = tid & 31; i < np; i += 32) M = fmaxf(M, at(i)[16 * D + h]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, off));
    for (int i = tid & 31; i < np; i += 32) {
        const float* p = at(i) + 16 * D;
        const float a = ex2(p[h] - M);
        if (tid < 32) s_a[i] = a;
        l = fmaf(a, p[16 + h], l);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(~0u, l, off);
    __syncthreads();
    float O = 0.f;
    for (int i0 = 0; i0 < np; i0 += 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = i0 + j < np ? at(i0 + j)[h * D + tid] : 0.f;
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (i0 + j < np) O = fmaf(s_a[i0 + j], v[j], O);
    }
    const bool any = l != 0.f;
    o[row * D + tid] = __float2bfloat16(any ? O / l : 0.f);
    if (lse && tid == 0) lse[row] = any ? (M + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace pgd
}  // namespace hs2
