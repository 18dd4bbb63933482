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

// 16 (or fewer) aligned bytes of a row.
template <int BYTES>
struct alignas(BYTES) Piece {
    uint32_t w[BYTES / 4];
};
// r = the words from byte `off` (below 4 WORDS_OFF) of w on. `off` is the same in
// every lane, so that the cases are branches and not selections.
template <int WORDS, int WORDS_OFF, int HAVE>
__device__ __forceinline__ void shift_words(const uint32_t (&w)[HAVE], uint32_t off,
                                            uint32_t (&r)[WORDS]) {
    const uint32_t bits = off % 4 * 8;
#pragma unroll
    for (int k = 0; k < WORDS_OFF; ++k)
        if (off / 4 == (uint32_t)k) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i)
                r[i] = __funnelshift_r(w[i + k], i + k + 1 < HAVE ? w[i + k + 1] : 0u, bits);
        }
}

// G elements of a row from column c on, held by each lane of a warp one group after
// the other (the whole warp calls it, lanes past the row's end too). Where the row
// starts on no 16-byte boundary, lanes hand the beginning of their groups to the
// lane before, so that all but the warp's first and last elements still leave in
// 16-byte stores (2-byte stores instead touch eight times as many sectors).
template <typename O, int G>
__device__ __forceinline__ void store_row(O* row, int64_t K, int64_t c, const float (&v)[G]) {
    constexpr int ES = (int)sizeof(O), WORDS = G * ES / 4, PER = 16 / ES;
    static_assert(WORDS % 4 == 0, "whole 16-byte pieces");
    alignas(16) O o[G];
#pragma unroll
    for (int e = 0; e < G; ++e) o[e] = from_f32<O>(v[e]);
    uint32_t w[WORDS + 4];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = reinterpret_cast<uint32_t*>(o)[i];
    const int lane = threadIdx.x & 31;
    // bytes up to the next 16-byte boundary: the same for every lane
    const uint32_t skip = (uint32_t)(-(intptr_t)reinterpret_cast<uintptr_t>(row + c)) & 15u;
    if (skip == 0) {
        if (c + G <= K) {
#pragma unroll
            for (int g = 0; g < WORDS / 4; ++g)
                reinterpret_cast<uint4*>(row + c)[g] =
                    make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < G; ++e)
                if (c + e < K) row[c + e] = o[e];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[WORDS + i] = __shfl_down_sync(0xffffffffu, w[i], 1);
    uint32_t s[WORDS];
    shift_words<WORDS, 4>(w, skip, s);
    const int ahead = (int)skip / ES;  // elements that the lane before takes
#pragma unroll
    for (int g = 0; g < WORDS / 4; ++g) {
        const int64_t c0 = c + ahead + g * PER;  // the piece's first element
        // of the last lane's last piece the next warp has the rest
        const int have = lane == 31 && g == WORDS / 4 - 1 ? PER - ahead : PER;
        if (c0 + PER <= K && have == PER) {
            *reinterpret_cast<uint4*>(row + c0) =
                make_uint4(s[4 * g], s[4 * g + 1], s[4 * g + 2], s[4 * g + 3]);
        } else {
            const O* piece = reinterpret_cast<const O*>(s + 4 * g);
#pragma unroll
            for (int e = 0; e < PER; ++e)
                if (e < have && c0 + e < K) row[c0 + e] = piece[e];
        }
    }
    if (lane == 0) {  // no lane before
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (e < ahead && c + e < K) row[c + e] = o[e];
    }
}

// v + beta times what the row holds from column c on, in 16-byte reads where
// it lies so; the whole warp calls it, before it stores there.
template <typename O, int G>
__device__ __forceinline__ void add_row(const O* row, int64_t K, int64_t c, float beta,
                                        float (&v)[G]) {
    constexpr int PER = 16 / (int)sizeof(O);
    if (reinterpret_cast<uintptr_t>(row + c) % 16 == 0 && c + G <= K) {
#pragma unroll
        for (int j = 0; j < G; j += PER) {
            const Piece<16> old = *reinterpret_cast<const Piece<16>*>(row + c + j);
#pragma unroll
            for (int e = 0; e < PER; ++e)
                v[j + e] = fmaf(beta, to_f32(reinterpret_cast<const O*>(&old)[e]), v[j + e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < G; ++e)
            if (c + e < K) v[e] = fmaf(beta, to_f32(row[c + e]), v[e]);
    }
    __syncwarp();  // every lane has read what it adds to: lanes store for their neighbours
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
