// C ABI of the cache and window operators (declared in include/hs2.h): the
// e4m3 caches' writers and readers, the paged decode attention and the window
// attention.  Argument validation and launches; the kernels live in the headers.
#include <limits.h>

#include <algorithm>
#include <atomic>

#include "host.cuh"
#include "kv_cache.cuh"
#include "paged_decode.cuh"
#include "window_attn.cuh"

using namespace hs2;

namespace {

constexpr int kMaxGroup = 16;  // query heads per KV head
// Positions are 32-bit, and so are the ends of the tiles that hold them.
constexpr int kMaxPositions = INT_MAX - 1024;
constexpr int kMaxHeads = 4096;

// (the kernels work with scale * log2 e)
bool scale_ok(float s) { return s > 0.f && isfinite(s) && isfinite(s * kLog2e); }

// SMs of the current device, at most one CTA of the persistent kernels each.
int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return std::min(n, pgd::kMaxCtas);
}

template <class... P>
bool pointers_ok(const P*... p) {
    return ((p != nullptr && aligned16(p)) && ...);
}

hs2_status check_cache(const hs2_cache_shape* s) {
    if (!s) return HS2_ERR_INVALID_ARG;
    if (s->B < 1 || s->B > 65535 || s->Tmax < 1) return HS2_ERR_INVALID_ARG;
    if ((s->d != 64 && s->d != 128) || s->Tmax > kMaxPositions) return HS2_ERR_UNSUPPORTED;
    return HS2_OK;
}

hs2_status check_paged(const hs2_paged_shape* s) {
    if (!s) return HS2_ERR_INVALID_ARG;
    if (s->B < 1 || s->B > 65535 || s->Hkv < 1 || s->page < 1 || s->n_pages < 1 || s->max_pages < 1)
        return HS2_ERR_INVALID_ARG;
    if (s->d != 64 && s->d != 128) return HS2_ERR_UNSUPPORTED;
    if (s->page != 16 && s->page != 32 && s->page != 64 && s->page != 128)
        return HS2_ERR_UNSUPPORTED;
    if (s->Hkv > kMaxHeads) return HS2_ERR_UNSUPPORTED;
    // (page, head) numbers are 32-bit too
    if ((int64_t)s->max_pages * s->page > kMaxPositions) return HS2_ERR_UNSUPPORTED;
    if ((int64_t)s->n_pages * s->Hkv > INT_MAX) return HS2_ERR_UNSUPPORTED;
    return HS2_OK;
}

hs2_status check_groups(int Hq, int Hkv) {
    if (Hq < 1 || Hkv < 1 || Hq % Hkv) return HS2_ERR_INVALID_ARG;
    if (Hq / Hkv > kMaxGroup || Hkv > kMaxHeads) return HS2_ERR_UNSUPPORTED;
    return HS2_OK;
}

template <int D>
hs2_status launch_page_write(const hs2_paged_shape* s, int N, const void* k_new, const void* v_new,
                             const int32_t* table, const int32_t* start, const int32_t* count,
                             void* k_pages, void* v_pages, float* k_scale, float* v_scale,
                             cudaStream_t st, unsigned* flags) {
    // pages that N rows can touch, wherever they start
    const int64_t slots = ((int64_t)N + s->page - 2) / s->page + 1;
    const int64_t blocks = slots * s->Hkv * 2;
    if (blocks > INT_MAX) return HS2_ERR_UNSUPPORTED;
    auto run = [&](auto kern) {
        kern<<<dim3((unsigned)blocks, s->B), kvc::kPageThreads, 0, st>>>(
            static_cast<const __nv_bfloat16*>(k_new), static_cast<const __nv_bfloat16*>(v_new),
            table, start, count, static_cast<uint8_t*>(k_pages), static_cast<uint8_t*>(v_pages),
            k_scale, v_scale, N, s->Hkv, s->n_pages, s->max_pages, flags);
        return launch_status();
    };
    switch (s->page) {
        case 16: return run(kvc::paged_write_kernel<D, 16>);
        case 32: return run(kvc::paged_write_kernel<D, 32>);
        case 64: return run(kvc::paged_write_kernel<D, 64>);
        default: return run(kvc::paged_write_kernel<D, 128>);
    }
}

// Pages [n_pages * Hkv, page, D] of e4m3 codes: a box is one page of one head.
bool map_pages(CUtensorMap* m, const void* x, int64_t n, int page, int D) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)page, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)D * page};
    const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)page, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(x), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct PagedCall {
    const hs2_paged_shape* s;
    const void *q, *k, *v;
    const float *ks, *vs;
    const int32_t *table, *lengths;
    void* o;
    float *lse, *part;
    int G, window, n_sink;
    float scale;
    cudaStream_t st;
    unsigned* flags;
};

template <class K>
int launch_registers(K kernel) {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kernel) == cudaSuccess ? a.numRegs : 0;
}

// The registers that the kernel's setmaxnreg splits are 512 x 128: it must have
// been built to launch with exactly those (its warps would wait for them in vain).
template <int D, int NG, int PAGE>
bool registers_ok() {
    if (NG != 16) return true;
    static const bool ok = launch_registers(pgd::paged_decode_kernel<D, NG, PAGE>) == 128;
    return ok;
}

// The most tiles that a call's sequences and heads can have together.
int64_t paged_tiles(const hs2_paged_shape* s, int window, int n_sink) {
    const int64_t seen = std::min<int64_t>(s->max_pages * s->page, (int64_t)window + n_sink);
    return (seen / pgd::kTile + 3) * s->Hkv * s->B;
}

template <int D, int NG>
hs2_status run_paged(const PagedCall& c) {
    const hs2_paged_shape* s = c.s;
    CUtensorMap mk, mv;
    const int64_t n = (int64_t)s->n_pages * s->Hkv;
    if (!map_pages(&mk, c.k, n, s->page, D) || !map_pages(&mv, c.v, n, s->page, D))
        return HS2_ERR_CUDA;
    const int cap = s->max_pages * s->page;
    const pgd::Work work = {c.lengths, s->B, cap, c.window, c.n_sink, s->Hkv};
    // no more CTAs than tiles there can be
    const int grid = (int)std::min<int64_t>(paged_tiles(s, c.window, c.n_sink), sm_count());
    if (grid < 1) return HS2_ERR_CUDA;
    auto* splits = reinterpret_cast<pgd::Split*>(c.part + (size_t)2 * pgd::kMaxCtas * (16 * D + 32));
    auto run = [&](auto kern, bool ok) {
        const size_t smem = pgd::Cfg<D, NG>::SMEM;
        if (!ok || !set_smem(kern, smem)) return HS2_ERR_CUDA;
        kern<<<grid, pgd::kThreads, smem, c.st>>>(
            mk, mv, static_cast<const __nv_bfloat16*>(c.q), c.ks, c.vs, c.table, work, c.G,
            s->n_pages, s->max_pages, c.scale * kLog2e, static_cast<__nv_bfloat16*>(c.o), c.lse,
            c.part, splits, c.flags);
        return launch_status();
    };
    hs2_status e;
    switch (s->page) {
        case 16: e = run(pgd::paged_decode_kernel<D, NG, 16>, registers_ok<D, NG, 16>()); break;
        case 32: e = run(pgd::paged_decode_kernel<D, NG, 32>, registers_ok<D, NG, 32>()); break;
        case 64: e = run(pgd::paged_decode_kernel<D, NG, 64>, registers_ok<D, NG, 64>()); break;
        default: e = run(pgd::paged_decode_kernel<D, NG, 128>, registers_ok<D, NG, 128>());
    }
    if (e != HS2_OK) return e;
    return launch_pdl(pgd::paged_merge_kernel<D>, dim3(grid, c.G), dim3(D), 0, c.st, c.G,
                      static_cast<__nv_bfloat16*>(c.o), c.lse, static_cast<const float*>(c.part),
                      static_cast<const pgd::Split*>(splits)) == cudaSuccess
               ? HS2_OK
               : HS2_ERR_CUDA;
}

// [B, L, H, D] bf16: a box of 64 columns, `heads` heads and `rows` positions.
bool map_rows(CUtensorMap* m, const void* x, int B, int L, int H, int D, int heads, int rows) {
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)L, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2,
                                   (cuuint64_t)L * H * D * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)heads, (cuuint32_t)rows, 1};
    return map_bf16(m, x, 4, dims, strides, box);
}

template <int D>
hs2_status run_window(const win::Shape& s, const void* q, const void* k, const void* v, void* o,
                      float* lse, cudaStream_t st, unsigned* flags) {
    win::Maps m;
    if (!map_rows(&m.q, q, s.B, s.Lq, s.Hq, D, s.G, s.nt) ||
        !map_rows(&m.k64, k, s.B, s.Lk, s.Hkv, D, 1, win::BN) ||
        !map_rows(&m.k16, k, s.B, s.Lk, s.Hkv, D, 1, 16) ||
        !map_rows(&m.v64, v, s.B, s.Lk, s.Hkv, D, 1, win::BN) ||
        !map_rows(&m.v16, v, s.B, s.Lk, s.Hkv, D, 1, 16))
        return HS2_ERR_CUDA;
    const int grid = std::min(s.items, sm_count());
    const size_t smem = win::Cfg<D>::SMEM;
    // (setmaxnreg in the kernel, as in registers_ok)
    static const bool built = launch_registers(win::window_attn_kernel<D>) == 128;
    if (!built || grid < 1 || !set_smem(win::window_attn_kernel<D>, smem)) return HS2_ERR_CUDA;
    win::window_attn_kernel<D><<<grid, win::kThreads, smem, st>>>(
        m, {static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
            static_cast<const __nv_bfloat16*>(v), static_cast<__nv_bfloat16*>(o), lse},
        s, flags);
    return launch_status();
}

}  // namespace

extern "C" {

hs2_status hs2_kv_write(const hs2_cache_shape* shape, int N, const void* k_new, const void* v_new,
                        const int32_t* start, const int32_t* count, void* k_cache, void* v_cache,
                        float* k_scale, float* v_scale, hs2_stream_t stream) {
    hs2_status e = check_cache(shape);
    if (e != HS2_OK) return e;
    if (N < 1 || N > shape->Tmax) return HS2_ERR_INVALID_ARG;
    if (!pointers_ok(k_new, v_new, start, k_cache, v_cache, k_scale, v_scale) || !aligned16(count))
        return HS2_ERR_INVALID_ARG;
    unsigned* flags = device_flags();
    if (!flags) return HS2_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int rows = kvc::kThreads / (shape->d / 16);
    const dim3 grid((N + rows - 1) / rows, shape->B);
    auto run = [&](auto kern) {
        kern<<<grid, kvc::kThreads, 0, st>>>(static_cast<const __nv_bfloat16*>(k_new),
                                   static_cast<const __nv_bfloat16*>(v_new), start, count,
                                   static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache),
                                   k_scale, v_scale, N, shape->Tmax, flags);
        return launch_status();
    };
    return shape->d == 128 ? run(kvc::token_write_kernel<128>) : run(kvc::token_write_kernel<64>);
}

hs2_status hs2_kv_read(const hs2_cache_shape* shape, int N, const void* k_cache, const void* v_cache,
                       const float* k_scale, const float* v_scale, const int32_t* start,
                       const int32_t* count, void* k, void* v, hs2_stream_t stream) {
    hs2_status e = check_cache(shape);
    if (e != HS2_OK) return e;
    if (N < 1 || N > shape->Tmax) return HS2_ERR_INVALID_ARG;
    if (!pointers_ok(k_cache, v_cache, k_scale, v_scale, start, k, v) || !aligned16(count))
        return HS2_ERR_INVALID_ARG;
    unsigned* flags = device_flags();
    if (!flags) return HS2_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int rows = kvc::kThreads / (shape->d / 8) * kvc::kRows;
    const dim3 grid((N + rows - 1) / rows, shape->B);
    auto run = [&](auto kern) {
        kern<<<grid, kvc::kThreads, 0, st>>>(static_cast<const uint8_t*>(k_cache),
                                   static_cast<const uint8_t*>(v_cache), k_scale, v_scale, start,
                                   count, static_cast<__nv_bfloat16*>(k),
                                   static_cast<__nv_bfloat16*>(v), N, shape->Tmax, flags);
        return launch_status();
    };
    return shape->d == 128 ? run(kvc::token_read_kernel<128>) : run(kvc::token_read_kernel<64>);
}

hs2_status hs2_paged_kv_write(const hs2_paged_shape* shape, int N, const void* k_new,
                              const void* v_new, const int32_t* table, const int32_t* start,
                              const int32_t* count, void* k_pages, void* v_pages, float* k_scale,
                              float* v_scale, hs2_stream_t stream) {
    hs2_status e = check_paged(shape);
    if (e != HS2_OK) return e;
    if (N < 1 || N > shape->max_pages * shape->page) return HS2_ERR_INVALID_ARG;
    if (!pointers_ok(k_new, v_new, table, start, k_pages, v_pages, k_scale, v_scale) ||
        !aligned16(count))
        return HS2_ERR_INVALID_ARG;
    unsigned* flags = device_flags();
    if (!flags) return HS2_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (shape->d == 128)
        return launch_page_write<128>(shape, N, k_new, v_new, table, start, count, k_pages, v_pages,
                                      k_scale, v_scale, st, flags);
    return launch_page_write<64>(shape, N, k_new, v_new, table, start, count, k_pages, v_pages,
                                 k_scale, v_scale, st, flags);
}

hs2_status hs2_paged_kv_read(const hs2_paged_shape* shape, int N, const void* k_pages,
                             const void* v_pages, const float* k_scale, const float* v_scale,
                             const int32_t* table, const int32_t* start, const int32_t* count,
                             void* k, void* v, hs2_stream_t stream) {
    hs2_status e = check_paged(shape);
    if (e != HS2_OK) return e;
    if (N < 1 || N > shape->max_pages * shape->page) return HS2_ERR_INVALID_ARG;
    if (!pointers_ok(k_pages, v_pages, k_scale, v_scale, table, start, k, v) || !aligned16(count))
        return HS2_ERR_INVALID_ARG;
    unsigned* flags = device_flags();
    if (!flags) return HS2_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int rows = kvc::kThreads / (shape->d / 8) * kvc::kPagedRows;
    int log_page = 0;
    while (1 << log_page < shape->page) log_page++;
    auto run = [&](auto kern) {
        kern<<<dim3((N + rows - 1) / rows, shape->B, shape->Hkv), kvc::kThreads, 0, st>>>(
            static_cast<const uint8_t*>(k_pages), static_cast<const uint8_t*>(v_pages), k_scale,
            v_scale, table, start, count, static_cast<__nv_bfloat16*>(k),
            static_cast<__nv_bfloat16*>(v), N, log_page, shape->n_pages, shape->max_pages, flags);
        return launch_status();
    };
    return shape->d == 128 ? run(kvc::paged_read_kernel<128>) : run(kvc::paged_read_kernel<64>);
}

size_t hs2_paged_decode_workspace(const hs2_paged_shape* shape, int Hq) {
    if (check_paged(shape) != HS2_OK || check_groups(Hq, shape->Hkv) != HS2_OK) return 0;
    // two parts of an item per CTA, and what the merge is to do
    return (size_t)pgd::kMaxCtas * (2 * (16 * shape->d + 32) * sizeof(float) + sizeof(pgd::Split));
}

hs2_status hs2_paged_decode(const hs2_paged_shape* shape, int Hq, int window, int n_sink,
                            float scale, const void* q, const void* k_pages, const void* v_pages,
                            const float* k_scale, const float* v_scale, const int32_t* table,
                            const int32_t* lengths, void* o, float* lse, void* workspace,
                            size_t workspace_bytes, hs2_stream_t stream) {
    hs2_status e = check_paged(shape);
    if (e != HS2_OK) return e;
    e = check_groups(Hq, shape->Hkv);
    if (e != HS2_OK) return e;
    if (window < 1 || n_sink < 0 || !scale_ok(scale)) return HS2_ERR_INVALID_ARG;
    // a CTA counts its tiles in 32 bits
    if (paged_tiles(shape, window, n_sink) > INT_MAX) return HS2_ERR_UNSUPPORTED;
    if (!pointers_ok(q, k_pages, v_pages, k_scale, v_scale, table, lengths, o) || !aligned16(lse) ||
        !pointers_ok(workspace))
        return HS2_ERR_INVALID_ARG;
    if (workspace_bytes < hs2_paged_decode_workspace(shape, Hq)) return HS2_ERR_WORKSPACE;
    unsigned* flags = device_flags();
    if (!flags) return HS2_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const PagedCall c = {shape, q, k_pages, v_pages, k_scale, v_scale, table, lengths,
                         o,     lse, static_cast<float*>(workspace), Hq / shape->Hkv, window, n_sink,
                         scale, st, flags};
    // a thread's exponentials and registers go by the heads it is built for.  48
    // ragged sequences of 8 KV heads: groups of four, heads of 64, 53.1 us built
    // for four against 59.9 for eight; heads of 128, 77.4 against 79.0; groups of
    // eight, 62.5 built for eight against 86.7 for sixteen; 81.2 against 92.5.
    // 8 sequences of 60k tokens, 4 KV heads of 128: groups of four 55.2 against
    // 56.5, of eight 56.4 against 62.9
    if (shape->d == 128)
        return c.G > 8 ? run_paged<128, 16>(c) : c.G > 4 ? run_paged<128, 8>(c) : run_paged<128, 4>(c);
    return c.G > 8 ? run_paged<64, 16>(c) : c.G > 4 ? run_paged<64, 8>(c) : run_paged<64, 4>(c);
}

hs2_status hs2_window_attn(const hs2_window_shape* shape, const void* q, const void* k,
                           const void* v, void* o, float* lse, hs2_stream_t stream) {
    const hs2_window_shape* s = shape;
    if (!s) return HS2_ERR_INVALID_ARG;
    if (s->B < 1 || s->B > 65535 || s->Lq < 1 || s->Lk < s->Lq || s->window < 1 || s->n_sink < 0 ||
        !scale_ok(s->scale))
        return HS2_ERR_INVALID_ARG;
    hs2_status e = check_groups(s->Hq, s->Hkv);
    if (e != HS2_OK) return e;
    if ((s->d != 64 && s->d != 128) || s->Lk > kMaxPositions) return HS2_ERR_UNSUPPORTED;
    if (!pointers_ok(q, k, v, o) || !aligned16(lse)) return HS2_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int G = s->Hq / s->Hkv, nt = win::BM / G;
    const int64_t blocks = ((int64_t)s->Lq + 2 * nt - 1) / (2 * nt);
    // items and rows are counted in 32 bits
    if (blocks * s->B * s->Hkv > INT_MAX || (int64_t)s->B * s->Lq * s->Hq > INT_MAX)
        return HS2_ERR_UNSUPPORTED;
    unsigned* flags = device_flags();
    if (!flags) return HS2_ERR_CUDA;
    const win::Shape sh = {s->B, s->Lq, s->Lk, s->Hq, s->Hkv, G, nt, s->window, s->n_sink, (int)blocks,
                           (int)(blocks * s->B * s->Hkv), s->scale * kLog2e};
    return s->d == 128 ? run_window<128>(sh, q, k, v, o, lse, st, flags)
                       : run_window<64>(sh, q, k, v, o, lse, st, flags);
}

}  // extern "C"
