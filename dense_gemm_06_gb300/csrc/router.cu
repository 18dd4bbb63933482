// router.cu -- router_balance() and router_balance_grad(): the experts' counts
// and group limits, the balance loss of a router, and its gradient.
//
//   p_t   = softmax(logits_t)          over the E experts, of every row that counts
//   f_e   = counts_e / (top n),        P_e = sum_t p_te / n,   n rows that count
//   loss  = E sum_e f_e P_e
//   dlogits_te = alpha dloss E / n p_te (f_e - sum_j f_j p_tj) + beta dlogits_te
//
// Both are bound by memory for many rows and by latency for few. A warp takes a
// row, a lane every 32nd expert, so the softmax and the inner product are warp
// reductions; four rows are in flight in a warp. The forward pass keeps each
// lane's sum of p over its rows in registers; a block's sums and counts are added
// by a second kernel in the order of the blocks (counts are whole numbers, sums
// do not depend on timing).
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gemm.h"
#include "internal.h"
#include "policy.h"
#include "rows.cuh"

namespace libgemm {
namespace {

bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

constexpr int kWarps = 8;         // of a block
constexpr int kMaxExperts = 1024;

__device__ __forceinline__ float sum32(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float max32(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// *p of the block `rank` of the cluster.
template <typename T>
__device__ __forceinline__ T ld_cluster(const T* p, int rank) {
    static_assert(sizeof(T) == 4, "words");
    uint32_t v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];"
                 : "=r"(v)
                 : "r"(gemm_ptx::mapa_shared(gemm_ptx::smem_u32(p), (uint32_t)rank))
                 : "memory");
    return *reinterpret_cast<T*>(&v);
}

// A row's probabilities: NE of them in each lane, expert lane + 32 i.
template <int NE>
__device__ __forceinline__ void softmax_row(float (&v)[NE]) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) m = fmaxf(m, v[i]);
    m = max32(m);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        v[i] = expf(v[i] - m);
        s += v[i];
    }
    s = 1.f / sum32(s);
#pragma unroll
    for (int i = 0; i < NE; ++i) v[i] *= s;
}

struct BalanceArgs {
    int64_t T;
    int E, top;
    const void* logits;
    int64_t ldl;
    const int32_t* expert;
    float* part_p;      // blocks x E sums of p
    int32_t* part_n;    // blocks x (E + 1) counts, the last the rows that count
    ErrWord* err;
};

template <typename T, int NE, int ROWS>
__global__ void __launch_bounds__(32 * kWarps) balance_kernel(const BalanceArgs a) {
    gemm_ptx::pdl_launch_dependents();
    extern __shared__ int32_t counts[];  // E + 1, then kWarps x E sums
    float* sums = reinterpret_cast<float*>(counts + a.E + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e <= a.E; e += 32 * kWarps) counts[e] = 0;
    __syncthreads();
    gemm_ptx::pdl_wait();
    float total[NE] = {};
    int rows = 0;
    auto count = [&](int e) {
        if (e >= a.E) report_bad_value(a.err);
        else if (e >= 0) atomicAdd(&counts[e], 1);
    };
    const int64_t step = (int64_t)gridDim.x * kWarps;
    for (int64_t t0 = (int64_t)blockIdx.x * kWarps + warp; t0 < a.T; t0 += ROWS * step) {
        float v[ROWS][NE];
        int first[ROWS];
        bool in[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int64_t t = t0 + r * step;
            const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
            // read whether the row counts or not, so that one latency covers both
#pragma unroll
            for (int i = 0; i < NE; ++i)
                v[r][i] = t < a.T && lane + 32 * i < a.E ? to_f32(row[lane + 32 * i]) : -INFINITY;
            first[r] = -1;
            if (t < a.T && lane < a.top) first[r] = a.expert[t * a.top + lane];
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            in[r] = __shfl_sync(0xffffffffu, first[r], 0) >= 0;
            if (!in[r]) continue;
            count(first[r]);
            for (int k = lane + 32; k < a.top; k += 32)
                count(a.expert[(t0 + r * step) * a.top + k]);
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (!in[r]) continue;
            ++rows;
            softmax_row<NE>(v[r]);
#pragma unroll
            for (int i = 0; i < NE; ++i) total[i] += v[r][i];
        }
    }
    if (lane == 0) atomicAdd(&counts[a.E], rows);
#pragma unroll
    for (int i = 0; i < NE; ++i)
        if (lane + 32 * i < a.E) sums[warp * a.E + lane + 32 * i] = total[i];
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += 32 * kWarps) {
        a.part_n[(int64_t)blockIdx.x * (a.E + 1) + e] = counts[e];
        if (e == a.E) continue;
        float s = 0.f;
        for (int w = 0; w < kWarps; ++w) s += sums[w * a.E + e];
        a.part_p[(int64_t)blockIdx.x * a.E + e] = s;
    }
}

// A cluster of kJoin blocks: each adds up its share of the blocks' sums and
// counts, the first one the shares, and writes the limits and the loss. `shares`
// threads an expert (a power of two), each a share of the block's.
constexpr int kJoin = 8;
__global__ void __cluster_dims__(kJoin, 1, 1) __launch_bounds__(1024)
    balance_join_kernel(const float* __restrict__ part_p, const int32_t* __restrict__ part_n,
                        int blocks, int E, int top, int shares, int32_t* __restrict__ counts,
                        int32_t* __restrict__ offsets, float* __restrict__ prob,
                        float* __restrict__ loss) {
    gemm_ptx::pdl_launch_dependents();
    __shared__ float p[1024];
    __shared__ int32_t c[1024], warp_n[32];
    __shared__ float warp_f[32];
    __shared__ int32_t all_rows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)gemm_ptx::cluster_ctarank();
    gemm_ptx::pdl_wait();
    const int b0 = (int)((int64_t)blocks * rank / kJoin);
    const int b1 = (int)((int64_t)blocks * (rank + 1) / kJoin);
    int n = 0;  // rows that count
    for (int b = b0 + threadIdx.x; b < b1; b += 1024) n += part_n[(int64_t)b * (E + 1) + E];
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) warp_n[warp] = n;
    // an expert's shares lie a whole number of experts apart
    const int wide = 1024 / shares;
    const int e = threadIdx.x % wide, share = threadIdx.x / wide;
    float s = 0.f;
    int32_t k = 0;
    if (e < E) {
#pragma unroll 8
        for (int b = b0 + share; b < b1; b += shares) {
            s += part_p[(int64_t)b * E + e];
            k += part_n[(int64_t)b * (E + 1) + e];
        }
    }
    p[threadIdx.x] = s;
    c[threadIdx.x] = k;
    __syncthreads();
    for (int o = shares / 2; o; o /= 2) {
        if (share < o) {
            p[threadIdx.x] += p[threadIdx.x + o * wide];
            c[threadIdx.x] += c[threadIdx.x + o * wide];
        }
        __syncthreads();
    }
    if (warp == 0) {
        n = __reduce_add_sync(0xffffffffu, warp_n[lane]);
        if (lane == 0) all_rows = n;
    }
    gemm_ptx::cluster_sync_all();
    const bool mine = rank == 0 && threadIdx.x < E;
    int32_t own = 0;
    s = 0.f;
    n = 0;
    if (rank == 0) {
        for (int r = 0; r < kJoin; ++r) {
            n += ld_cluster(&all_rows, r);
            if (mine) {
                s += ld_cluster(&p[threadIdx.x], r);
                own += ld_cluster(&c[threadIdx.x], r);
            }
        }
    }
    gemm_ptx::cluster_sync_all();  // no block leaves, or writes, while its sums are read
    if (rank != 0) return;
    const int m = n > 0 ? n : 1;
    float term = 0.f;
    if (mine) {
        const float mean = s / (float)m;
        counts[threadIdx.x] = own;
        prob[threadIdx.x] = mean;
        term = (float)((double)own / ((double)top * m)) * mean;
    }
    // the limits: a sum up to each expert; the loss: a sum in a fixed order
    int32_t upto = own;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int32_t add = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += add;
    }
    term = sum32(term);
    if (lane == 31) warp_n[warp] = upto;
    if (lane == 0) warp_f[warp] = term;
    __syncthreads();
    if (offsets) {
        int32_t before = lane < warp ? warp_n[lane] : 0;
        before = __reduce_add_sync(0xffffffffu, before);
        if (mine) offsets[threadIdx.x + 1] = before + upto;
        if (threadIdx.x == 0) offsets[0] = 0;
    }
    if (warp == 0) {
        term = sum32(warp_f[lane]);
        if (lane == 0) {
            *loss = (float)E * term;
            counts[E] = n;
        }
    }
}

struct BalanceGradArgs {
    int64_t T;
    int E, top;
    const void* logits;
    int64_t ldl;
    const int32_t* expert;
    const int32_t* counts;
    const float* dloss;  // null: 1
    float alpha, beta;
    void* dlogits;
    int64_t ldd;
};

template <typename T, typename O, int NE, int ROWS>
__global__ void __launch_bounds__(32 * kWarps) balance_grad_kernel(const BalanceGradArgs a) {
    gemm_ptx::pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    gemm_ptx::pdl_wait();
    const int n = a.counts[a.E];
    const float by = n > 0 ? 1.f / (float)n : 0.f;
    float f[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i)
        f[i] = lane + 32 * i < a.E ? (float)a.counts[lane + 32 * i] / (float)a.top * by : 0.f;
    const float d = a.alpha * (a.dloss ? *a.dloss : 1.f) * (float)a.E * by;
    const int64_t step = (int64_t)gridDim.x * kWarps;
    for (int64_t t0 = (int64_t)blockIdx.x * kWarps + warp; t0 < a.T; t0 += ROWS * step) {
        float v[ROWS][NE];
        bool in[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int64_t t = t0 + r * step;
            in[r] = t < a.T && a.expert[t * a.top] >= 0;
            const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                v[r][i] = t < a.T && lane + 32 * i < a.E ? to_f32(row[lane + 32 * i]) : -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int64_t t = t0 + r * step;
            if (t >= a.T) continue;
            float inner = 0.f;
            if (in[r]) {
                softmax_row<NE>(v[r]);
#pragma unroll
                for (int i = 0; i < NE; ++i) inner = fmaf(v[r][i], f[i], inner);
                inner = sum32(inner);
            }
            O* row = static_cast<O*>(a.dlogits) + t * a.ldd;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 32 * i;
                if (e >= a.E) continue;
                const float g = in[r] ? d * v[r][i] * (f[i] - inner) : 0.f;
                row[e] = from_f32<O>(a.beta != 0.f ? fmaf(a.beta, to_f32(row[e]), g) : g);
            }
        }
    }
}

bool rows_ok(const void* p, int64_t rows, int64_t cols, int64_t ld, int es) {
    return p && aligned_to(p, es) && ld >= cols &&
           (__int128)(rows - 1) * ld + cols <= (__int128)(INT64_MAX / es);
}

// Calls f with an integral constant NE (numbers of a lane) and ROWS (rows in
// flight: 32 numbers a lane at most, and four rows).
template <typename F>
int with_lanes(int E, F&& f) {
    using std::integral_constant;
    if (E <= 32) return f(integral_constant<int, 1>{}, integral_constant<int, 4>{});
    if (E <= 64) return f(integral_constant<int, 2>{}, integral_constant<int, 4>{});
    if (E <= 128) return f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
    if (E <= 192) return f(integral_constant<int, 6>{}, integral_constant<int, 4>{});
    if (E <= 256) return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
    if (E <= 512) return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
}

int check_router(int64_t T, int64_t E, int64_t top, const void* logits, int64_t ldl,
                 const int32_t* expert, int dtype) {
    if (dtype < GEMM_F32 || dtype > GEMM_BF16_BF16) return kInvalidArg;
    if (T < 0 || E < 1 || top < 1 || T > INT32_MAX || E > INT32_MAX || top > INT32_MAX)
        return kInvalidArg;
    if ((__int128)T * top > INT32_MAX) return kInvalidArg;  // counts and limits are 32-bit
    if (E > kMaxExperts) return kUnsupported;
    if (T == 0) return kOk;
    if (!rows_ok(logits, T, E, ldl, dtype == GEMM_F32 ? 4 : 2) || !expert ||
        !aligned_to(expert, 4))
        return kInvalidArg;
    return kOk;
}

int balance(int64_t T, int64_t E, int64_t top, const void* logits, int64_t ldl,
            const int32_t* expert, int32_t* counts, int32_t* offsets, float* prob, float* loss,
            int dtype, cudaStream_t s) {
    int rc = check_router(T, E, top, logits, ldl, expert, dtype);
    if (rc != kOk) return rc;
    if (!counts || !prob || !loss || !aligned_to(counts, 4) || !aligned_to(offsets, 4) ||
        !aligned_to(prob, 4) || !aligned_to(loss, 4))
        return kInvalidArg;
    DeviceInfo* dev = nullptr;
    cudaMemPool_t pool = nullptr;
    rc = current_device_info(&dev, &pool);
    if (rc != kOk) return rc;
    const void* ptrs[6] = {T > 0 ? logits : nullptr, T > 0 ? expert : nullptr, counts, offsets,
                           prob, loss};
    rc = check_device_pointers(ptrs, 6, dev->device);
    if (rc != kOk) return rc;
    int64_t blocks = (T + kWarps - 1) / kWarps;
    const int64_t most = (int64_t)dev->sm_count * 4;
    if (blocks > most) blocks = most;
    Scratch scratch{pool, s, dev->device};
    BalanceArgs a{T, (int)E, (int)top, logits, ldl, expert, nullptr, nullptr, dev->err_word};
    if (blocks > 0) {
        char* mem = static_cast<char*>(scratch.get((size_t)(blocks * (2 * E + 1) * 4)));
        if (!mem) return kCuda;
        a.part_p = reinterpret_cast<float*>(mem);
        a.part_n = reinterpret_cast<int32_t*>(mem + blocks * E * 4);
        const size_t smem = (size_t)(E + 1 + kWarps * E) * 4;
        rc = with_lanes((int)E, [&](auto ne, auto rows) {
            constexpr int NE = decltype(ne)::value, ROWS = decltype(rows)::value;
            const dim3 grid((unsigned)blocks), block(32 * kWarps);
            if (dtype == GEMM_F32)
                return launch_dependent(balance_kernel<float, NE, ROWS>, grid, block, smem, s, a);
            if (dtype == GEMM_BF16_F32 || dtype == GEMM_BF16_BF16)
                return launch_dependent(balance_kernel<__nv_bfloat16, NE, ROWS>, grid, block, smem,
                                        s, a);
            return launch_dependent(balance_kernel<__half, NE, ROWS>, grid, block, smem, s, a);
        });
    }
    if (rc == kOk) {
        int shares = 1;
        while (shares * 2 * E <= 1024) shares *= 2;
        rc = launch_dependent(balance_join_kernel, dim3(kJoin), dim3(1024), 0, s,
                              (const float*)a.part_p, (const int32_t*)a.part_n, (int)blocks,
                              (int)E, (int)top, shares, counts, offsets, prob, loss);
    }
    scratch.release();
    return rc;
}

int balance_grad(int64_t T, int64_t E, int64_t top, const void* logits, int64_t ldl,
                 const int32_t* expert, const int32_t* counts, const float* dloss, void* dlogits,
                 int64_t ldd, float alpha, float beta, int dtype, cudaStream_t s) {
    int rc = check_router(T, E, top, logits, ldl, expert, dtype);
    if (rc != kOk || T == 0) return rc;
    const int os = dtype <= GEMM_BF16_F32 ? 4 : 2;
    if (!counts || !aligned_to(counts, 4) || !aligned_to(dloss, 4) ||
        !rows_ok(dlogits, T, E, ldd, os))
        return kInvalidArg;
    DeviceInfo* dev = nullptr;
    rc = current_device_info(&dev, nullptr);
    if (rc != kOk) return rc;
    const void* ptrs[5] = {logits, expert, counts, dloss, dlogits};
    rc = check_device_pointers(ptrs, 5, dev->device);
    if (rc != kOk) return rc;
    const BalanceGradArgs a{T, (int)E, (int)top, logits, ldl, expert, counts, dloss, alpha, beta,
                            dlogits, ldd};
    int64_t blocks = (T + kWarps - 1) / kWarps;
    const int64_t most = (int64_t)dev->sm_count * 8;
    if (blocks > most) blocks = most;
    return with_lanes((int)E, [&](auto ne, auto rows) {
        constexpr int NE = decltype(ne)::value, ROWS = decltype(rows)::value;
        const dim3 grid((unsigned)blocks), block(32 * kWarps);
        switch (dtype) {
            case GEMM_F32:
                return launch_dependent(balance_grad_kernel<float, float, NE, ROWS>, grid, block,
                                        0, s, a);
            case GEMM_F16_F32:
                return launch_dependent(balance_grad_kernel<__half, float, NE, ROWS>, grid, block,
                                        0, s, a);
            case GEMM_BF16_F32:
                return launch_dependent(balance_grad_kernel<__nv_bfloat16, float, NE, ROWS>, grid,
                                        block, 0, s, a);
            case GEMM_F16_F16:
                return launch_dependent(balance_grad_kernel<__half, __half, NE, ROWS>, grid, block,
                                        0, s, a);
            default:
                return launch_dependent(
                    balance_grad_kernel<__nv_bfloat16, __nv_bfloat16, NE, ROWS>, grid, block, 0, s,
                    a);
        }
    });
}

}  // namespace
}  // namespace libgemm

using namespace libgemm;

extern "C" {

int router_balance(int64_t T, int64_t E, int64_t top, const void* logits, int64_t ldl,
                   const int32_t* expert, int32_t* counts, int32_t* offsets, float* prob,
                   float* loss, int dtype, void* stream) {
    try {
        return balance(T, E, top, logits, ldl, expert, counts, offsets, prob, loss, dtype,
                       static_cast<cudaStream_t>(stream));
    } catch (...) {
        return kCuda;
    }
}

int router_balance_grad(int64_t T, int64_t E, int64_t top, const void* logits, int64_t ldl,
                        const int32_t* expert, const int32_t* counts, const float* dloss,
                        void* dlogits, int64_t ldd, float alpha, float beta, int dtype,
                        void* stream) {
    try {
        return balance_grad(T, E, top, logits, ldl, expert, counts, dloss, dlogits, ldd, alpha,
                            beta, dtype, static_cast<cudaStream_t>(stream));
    } catch (...) {
        return kCuda;
    }
}

}  // extern "C"
