// rows.cuh -- what the row operators (layer norm, embedding, router balance) and
// the cross entropy's small kernels share: element conversions, 16-byte pieces
// of rows, reductions, and launches that overlap the tail of the kernel before
// them on the stream.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <set>
#include <type_traits>
#include <utility>

#include "epilogue.cuh"
#include "internal.h"
#include "ptx_sm100.cuh"

namespace libgemm {

// Sets the device's second error word: a kernel met numbers (targets, tokens,
// experts) that its arguments rule out, and left them out.
__device__ __forceinline__ void report_bad_value(ErrWord* err) { atomicOr(err + 1, 1ull); }

// Launches `kern` so that its blocks may start while the kernel before it on the
// stream ends; every kernel launched this way calls pdl_wait() before it touches
// global memory that an earlier kernel may write or read.
template <typename... P, typename... A>
int launch_dependent(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                     A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return kCuda;
    }
    note_launch();
    return kOk;
}

// Lets a kernel take `bytes` of dynamic shared memory on this device.
template <typename K>
int allow_smem(K kern, int bytes, const DeviceInfo& dev) {
    if (bytes <= 40 * 1024) return kOk;
    static std::mutex mu;
    static std::set<std::pair<const void*, int>> allowed;
    std::lock_guard<std::mutex> lock(mu);
    const std::pair<const void*, int> key(reinterpret_cast<const void*>(kern), dev.device);
    if (allowed.count(key)) return kOk;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
        cudaSuccess) {
        cudaGetLastError();
        return kCuda;
    }
    allowed.insert(key);
    return kOk;
}

}  // namespace libgemm
