// tmap.cuh -- host side of the kernels over dense and 4-bit weights and of the norm pair: the driver's
// tensor-map encoder, the SM count and the shared-memory attribute of a kernel (each looked up once per
// process or device), and a launch that may begin while the kernel before it in the stream ends.
#pragma once

#include <atomic>
#include <cuda.h>   // CUtensorMap and its enums (the encoder is fetched from the driver at run time)

#include "internal.cuh"

namespace moe {
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
    static std::atomic<EncodeTiledFn> fn{nullptr};
    EncodeTiledFn got = fn.load(std::memory_order_acquire);
    if (!got) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            got = reinterpret_cast<EncodeTiledFn>(f);
            fn.store(got, std::memory_order_release);
        }
    }
    return got;
}

// A map with boxes of box0 x box1 (x 1) elements, 128-byte swizzle, zeros outside.  dims and strides
// (bytes) from the inner dimension.
inline bool encode_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t (&dims)[3],
                       const cuuint64_t (&strides)[2], int box0, int box1) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint32_t box[3] = {(cuuint32_t)box0, (cuuint32_t)box1, 1u}, one[3] = {1u, 1u, 1u};
    return fn(m, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Programmatic dependent launch: a kernel launched by launch_early may be set up while the one before
// it ends; it calls wait_for_previous before its first access to memory, which returns when that kernel is done and
// its writes are visible, and allow_next so that its own successor may do the same.  Between two calls in a
// stream that saves 1 to 2 us.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
inline cudaError_t launch_early(const void* fn, dim3 grid, unsigned threads, size_t smem, cudaStream_t s, void** args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// SMs of the current device; a kernel's dynamic shared memory is raised to `smem` there, once per
// device (ready: the kernel's own bits).
inline cudaError_t prepare_kernel(const void* fn, int smem, std::atomic<uint64_t>& ready, int* sms) {
    static std::atomic<int> counts[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const bool known = dev >= 0 && dev < 64;
    int n = known ? counts[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if ((err = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return err;
        if (known) counts[dev].store(n, std::memory_order_relaxed);
    }
    *sms = n;
    const uint64_t bit = known ? 1ull << dev : 0;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        if ((err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return err;
        ready.fetch_or(bit, std::memory_order_release);
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace moe
