// Host helpers of the C ABI's translation units: argument and launch checks,
// shared-memory limits, programmatic launches and tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <utility>

#include "../../include/hs2.h"

namespace hs2 {
// The current device's word of device-side data flags (FLAG_* in common.cuh,
// read and cleared by hs2_get_last_device_error); nullptr on a CUDA error.
__attribute__((visibility("hidden"))) unsigned* device_flags();
}  // namespace hs2

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

hs2_status launch_status() {
    return cudaGetLastError() == cudaSuccess ? HS2_OK : HS2_ERR_CUDA;
}

// Raise a kernel's dynamic shared-memory limit once per (kernel, device) and
// size increase, so repeated calls -- including calls under stream capture --
// make no further attribute calls.
struct SmemLimit {
    const void* fn;
    int dev;
    size_t bytes;
};
SmemLimit g_smem_limits[512];
int g_n_smem_limits = 0;
std::mutex g_smem_mutex;

template <class K>
bool set_smem(K kernel, size_t bytes) {
    // (static + dynamic shared memory above 48 KiB needs the opt-in, so any
    // nonzero request is registered; the table makes it once per kernel/device)
    if (bytes == 0) return true;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const void* fn = reinterpret_cast<const void*>(kernel);
    std::lock_guard<std::mutex> lock(g_smem_mutex);
    SmemLimit* e = nullptr;
    for (int i = 0; i < g_n_smem_limits; i++)
        if (g_smem_limits[i].fn == fn && g_smem_limits[i].dev == dev) e = &g_smem_limits[i];
    if (e && e->bytes >= bytes) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) !=
        cudaSuccess)
        return false;
    if (!e) {
        if (g_n_smem_limits == 512) return true;  // table full: set again next time
        e = &g_smem_limits[g_n_smem_limits++];
        e->fn = fn;
        e->dev = dev;
    }
    e->bytes = bytes;
    return true;
}

// Launch with programmatic stream serialisation: the kernel may start while
// the previous kernel of the stream drains (its prologue overlaps that
// kernel's tail); it calls griddep_wait() before reading that kernel's
// results.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t st, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// ------------------------------------------------------------ tensor maps
// cuTensorMapEncodeTiled through the runtime's driver entry point (no direct
// libcuda link).  bf16 tensors, 128-byte swizzle, 64-element inner box.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void* p = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

bool map_bf16(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
              const cuuint64_t* strides, const cuuint32_t* box) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides,
               box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
