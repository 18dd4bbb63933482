// ptx_ragged.cuh -- inline-PTX wrappers that only the ragged products use (3-D
// TMA copies, tensor maps edited on the device, stores to cluster peers, global
// additions); the rest is in ptx_sm100.cuh. From the public PTX ISA, as there.
#pragma once

#include "ptx_sm100.cuh"

namespace gemm_ptx {

// mbar_arrive_cluster without ordering this thread's memory accesses.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];"
                 :: "r"(cluster_bar) : "memory");
}

// A tensor map in shared memory (128-byte aligned): sets the size of its
// dimension 1 (rows of a 2-D map).
__device__ __forceinline__ void tma_desc_set_rows(uint32_t smem_map, uint32_t rows) {
    asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;"
                 :: "r"(smem_map), "r"(rows) : "memory");
}

// Copies a tensor map from shared to global memory (both 128-byte aligned) and
// releases it for use by TMA; the whole warp calls it.
__device__ __forceinline__ void tma_desc_publish(void* map, uint32_t smem_map) {
    asm volatile(
        "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned"
        " [%0], [%1], 128;" :: "l"(map), "r"(smem_map) : "memory");
}

// Before this thread's first TMA copy through a map that tma_desc_publish wrote.
__device__ __forceinline__ void tma_desc_acquire(const void* map) {
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" :: "l"(map) : "memory");
}

// 3-D tiled TMA load; as tma_load_2d with a third coordinate.
template <int CG>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z) {
    if constexpr (CG == 2) {
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];"
            :: "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
    } else {
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];"
            :: "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
    }
}

// Stores a float at a shared::cluster address (own or peer CTA).
__device__ __forceinline__ void st_cluster_f32(uint32_t cluster_addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(cluster_addr), "f"(v) : "memory");
}

// *p += v in global memory, rounded to nearest; nothing comes back.
__device__ __forceinline__ void red_add_f32(float* p, float v) {
    asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" :: "l"(p), "f"(v) : "memory");
}

// Four words at a 16-byte aligned shared::cluster address.
__device__ __forceinline__ void st_cluster_v4(uint32_t cluster_addr, uint32_t x, uint32_t y,
                                              uint32_t z, uint32_t w) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};"
                 :: "r"(cluster_addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 3-D tiled TMA store.
__device__ __forceinline__ void tma_store_3d(const void* map, uint32_t src, int32_t x, int32_t y,
                                             int32_t z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];"
                 :: "l"(map), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
}

// Wait until all but the last committed bulk store have finished reading.
__device__ __forceinline__ void bulk_wait_read_1() {
    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}

// fence_proxy_async_smem for every state space (shared memory of cluster peers
// included).
__device__ __forceinline__ void fence_proxy_async_all() {
    asm volatile("fence.proxy.async;" ::: "memory");
}

}  // namespace gemm_ptx
