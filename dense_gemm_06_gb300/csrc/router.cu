// router.cu -- router_balance() and router_balance_grad(): the experts' counts
// and group limits, the balance loss of a router, and its gradient.
//
//   p_t   = softmax(logits_t)          over the E experts, of every row that counts
//   f_e   = counts_e / (top n),        P_e = sum_t p_te / n,   n rows that count
//   loss  = E sum_e f_e P_e
//   dlogits_te = alpha dloss E / n p_te (f_e - sum_j f_j p_tj) + beta dlogits_te
//
// Both are bound by memory for many rows and by latency for few. A row sits on 8
// or 32 lanes of a warp, so the softmax and the inner product are reductions over
// those, and several rows are in flight in a warp. The forward pass keeps each
// lane's sum of p over its rows in registers; the blocks of a cluster add theirs in
// the order of their ranks, and where there are several clusters a second kernel adds
// the clusters' (counts are whole numbers, sums do not depend on timing). 32768 rows
// of 160, fp32, us: forward 9 and 6.5 for the join, gradient 10.7; 48 rows of 64: 4.3.
// Both kernels are chains of latencies: a load, two reductions, expf, a barrier.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gemm.h"
#include "internal.h"
#include "policy.h"
#include "rows.cuh"

namespace libgemm {
namespace {

bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

constexpr int kMaxExperts = 1024;

// Sums and maxima over the LANES lanes that share a row.
template <int LANES>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int LANES>
__device__ __forceinline__ float max_lanes(float v) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
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

// A row's probabilities: NE of them in each of its lanes.
template <int LANES, int NE>
__device__ __forceinline__ void softmax_row(float (&v)[NE]) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) m = fmaxf(m, v[i]);
    m = max_lanes<LANES>(m);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        v[i] = expf(v[i] - m);
        s += v[i];
    }
    s = 1.f / sum_lanes<LANES>(s);
#pragma unroll
    for (int i = 0; i < NE; ++i) v[i] *= s;
}

// Expert i of the NE that a lane holds: groups of four side by side.
template <int LANES>
__device__ __forceinline__ int expert_of(int sub, int i) {
    return (sub + LANES * (i / 4)) * 4 + i % 4;
}

// A lane's logits of a row, -inf past the last expert (and for no row); four at a
// time where E and every row's address allow it.
template <typename T, int LANES, int NE>
__device__ __forceinline__ void load_row(const T* row, bool in, int E, int sub, bool fours,
                                         float (&v)[NE]) {
    if (fours) {
#pragma unroll
        for (int i = 0; i < NE; i += 4) {
            const int e = expert_of<LANES>(sub, i);
            Piece<4 * sizeof(T)> p;
            if (in && e < E) p = *reinterpret_cast<const Piece<4 * sizeof(T)>*>(row + e);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4) {
                    v[i + j] = __uint_as_float(p.w[j]);
                } else {
                    const uint16_t h = (uint16_t)(p.w[j / 2] >> (j % 2 * 16));
                    v[i + j] = to_f32(*reinterpret_cast<const T*>(&h));
                }
                if (!in || e >= E) v[i + j] = -INFINITY;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = expert_of<LANES>(sub, i);
            v[i] = in && e < E ? to_f32(row[e]) : -INFINITY;
        }
    }
}

struct BalanceArgs {
    int64_t T;
    int E, top;
    const void* logits;
    int64_t ldl;
    bool fours;
    const int32_t* expert;
    int32_t* counts;
    int32_t* offsets;   // or null
    float* prob;
    float* loss;
    float* part_p;      // clusters x E sums of p
    int32_t* part_n;    // clusters x (E + 1) counts, the last the rows that count
    ErrWord* err;
};

// Writes the results from the experts' counts and sums of p (in shared memory) of n
// rows that count: a thread takes 1024 / THREADS experts in a row. The whole block
// calls it; the sums are added in one order whatever the timing.
template <int THREADS>
__device__ __forceinline__ void write_balance(const BalanceArgs& a, int n, const float* p,
                                              const int32_t* c) {
    constexpr int PER = kMaxExperts / THREADS, WARPS = THREADS / 32;
    __shared__ int32_t warp_c[WARPS];
    __shared__ float warp_f[WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = threadIdx.x * PER, m = n > 0 ? n : 1;
    int32_t upto[PER], all = 0;
    float term = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        upto[j] = all;
        if (e0 + j >= a.E) continue;
        const int32_t own = c[e0 + j];
        const float mean = p[e0 + j] / (float)m;
        a.counts[e0 + j] = own;
        a.prob[e0 + j] = mean;
        term += (float)((double)own / ((double)a.top * m)) * mean;
        all += own;
        upto[j] = all;
    }
    int32_t before = all;  // of the warp's threads up to this one
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int32_t add = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += add;
    }
    term = sum_lanes<32>(term);
    if (lane == 31) warp_c[warp] = before;
    if (lane == 0) warp_f[warp] = term;
    __syncthreads();
    if (a.offsets) {
        before += __reduce_add_sync(0xffffffffu, lane < warp ? warp_c[lane] : 0) - all;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (e0 + j < a.E) a.offsets[e0 + j + 1] = before + upto[j];
        if (threadIdx.x == 0) a.offsets[0] = 0;
    }
    if (warp == 0) {
        term = sum_lanes<32>(lane < WARPS ? warp_f[lane] : 0.f);
        if (lane == 0) {
            *a.loss = (float)a.E * term;
            a.counts[a.E] = n;
        }
    }
}

// A row on LANES lanes, four experts in a row on each; a warp takes 32 / LANES rows at
// a time, ROWS times over with their reads in flight together. The blocks of a cluster
// (CL) add up their sums in the order of their ranks; a cluster that is alone writes the
// results, else each leaves one part.
constexpr int kWarps = 8, kCluster = 8;
// Blocks on an SM, by the probabilities that a lane holds.
constexpr int resident(int held) { return held <= 20 ? 4 : held <= 24 ? 3 : 2; }
template <typename T, int LANES, int NE, int ROWS, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(32 * kWarps, resident(NE * ROWS))
    balance_kernel(const BalanceArgs a) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int SIDE = 32 / LANES;  // rows of a warp side by side
    extern __shared__ int32_t counts[];  // E + 1, then kWarps x E sums
    float* sums = reinterpret_cast<float*>(counts + a.E + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane % LANES, side = lane / LANES;
    for (int e = threadIdx.x; e <= a.E; e += 32 * kWarps) counts[e] = 0;
    __syncthreads();
    gemm_ptx::pdl_wait();
    float total[NE] = {};
    int rows = 0;
    auto count = [&](int e) {
        if (e >= a.E) report_bad_value(a.err);
        else if (e >= 0) atomicAdd(&counts[e], 1);
    };
    const int64_t step = (int64_t)gridDim.x * kWarps * SIDE;
    for (int64_t w0 = ((int64_t)blockIdx.x * kWarps + warp) * SIDE; w0 < a.T; w0 += ROWS * step) {
        float v[ROWS][NE];
        int first[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int64_t t = w0 + side + r * step;
            const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
            // read whether the row counts or not, so that one latency covers both
            load_row<T, LANES>(row, t < a.T, a.E, sub, a.fours, v[r]);
            first[r] = t < a.T && sub < a.top ? a.expert[t * a.top + sub] : -1;
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const bool in = __shfl_sync(0xffffffffu, first[r], lane - sub) >= 0;
            softmax_row<LANES, NE>(v[r]);
            if (!in) continue;
            rows += sub == 0;
            count(first[r]);
            for (int k = sub + LANES; k < a.top; k += LANES)
                count(a.expert[(w0 + side + r * step) * a.top + k]);
#pragma unroll
            for (int i = 0; i < NE; ++i) total[i] += v[r][i];
        }
        __syncwarp();
    }
    rows = __reduce_add_sync(0xffffffffu, rows);
    if (lane == 0) atomicAdd(&counts[a.E], rows);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
#pragma unroll
        for (int o = LANES; o < 32; o *= 2)
            total[i] += __shfl_xor_sync(0xffffffffu, total[i], o);
        const int e = expert_of<LANES>(sub, i);
        if (side == 0 && e < a.E) sums[warp * a.E + e] = total[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 32 * kWarps) {
        float s = 0.f;
        for (int w = 0; w < kWarps; ++w) s += sums[w * a.E + e];
        sums[e] = s;
    }
    if constexpr (CL == 1) {
        __syncthreads();
        write_balance<32 * kWarps>(a, counts[a.E], sums, counts);
    } else {
        gemm_ptx::cluster_sync_all();
        const int rank = (int)gemm_ptx::cluster_ctarank();
        const bool alone = gridDim.x == CL;
        // alone: all of them into the second and third warp's place; else a share each
        const int e0 = alone ? (rank == 0 ? 0 : a.E + 1) : (a.E + 1) * rank / CL;
        const int e1 = alone ? a.E + 1 : (a.E + 1) * (rank + 1) / CL;
        float* all_p = alone ? sums + a.E : a.part_p + (int64_t)(blockIdx.x / CL) * a.E;
        int32_t* all_n = alone ? reinterpret_cast<int32_t*>(sums + 2 * a.E)
                               : a.part_n + (int64_t)(blockIdx.x / CL) * (a.E + 1);
        for (int e = e0 + threadIdx.x; e < e1; e += 32 * kWarps) {
            float p[CL];
            int32_t n[CL];
#pragma unroll
            for (int r = 0; r < CL; ++r) {
                p[r] = e < a.E ? ld_cluster(&sums[e], r) : 0.f;
                n[r] = ld_cluster(&counts[e], r);
            }
#pragma unroll
            for (int r = 1; r < CL; ++r) {
                p[0] += p[r];
                n[0] += n[r];
            }
            if (e < a.E) all_p[e] = p[0];
            all_n[e] = n[0];
        }
        gemm_ptx::cluster_sync_all();  // no block leaves while its sums are read
        if (alone && rank == 0) write_balance<32 * kWarps>(a, all_n[a.E], all_p, all_n);
    }
}

// Adds up the parts that several clusters left: `shares` threads an expert (a power of
// two), each with its share of the parts, whose reads are in flight together.
__global__ void __launch_bounds__(1024)
    balance_join_kernel(const BalanceArgs a, int parts, int shares) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int AHEAD = 8;
    __shared__ float p[1024];
    __shared__ int32_t c[1024], warp_n[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.E;
    gemm_ptx::pdl_wait();
    int n = 0;  // rows that count
    for (int b = threadIdx.x; b < parts; b += 1024) n += a.part_n[(int64_t)b * (E + 1) + E];
    // an expert's shares lie a whole number of experts apart
    const int wide = 1024 / shares;
    const int e = threadIdx.x % wide, share = threadIdx.x / wide;
    float s = 0.f;
    int32_t k = 0;
    if (e < E)
        for (int b = share; b < parts; b += AHEAD * shares) {
            float ps[AHEAD];
            int32_t ns[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int64_t at = b + j * shares;
                ps[j] = at < parts ? a.part_p[at * E + e] : 0.f;
                ns[j] = at < parts ? a.part_n[at * (E + 1) + e] : 0;
            }
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                s += ps[j];
                k += ns[j];
            }
        }
    p[threadIdx.x] = s;
    c[threadIdx.x] = k;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) warp_n[warp] = n;
    __syncthreads();
    for (int o = shares / 2; o; o /= 2) {
        if (share < o) {
            p[threadIdx.x] += p[threadIdx.x + o * wide];
            c[threadIdx.x] += c[threadIdx.x + o * wide];
        }
        __syncthreads();
    }
    n = __reduce_add_sync(0xffffffffu, warp_n[lane]);
    write_balance<1024>(a, n, p, c);
}

struct BalanceGradArgs {
    int64_t T;
    int E, top;
    const void* logits;
    int64_t ldl;
    bool fours;
    const int32_t* expert;
    const int32_t* counts;
    const float* dloss;  // null: 1
    float alpha, beta;
    void* dlogits;
    int64_t ldd;
};

constexpr int kGradWarps = 8;
template <typename T, typename O, int LANES, int NE, int ROWS>
__global__ void __launch_bounds__(32 * kGradWarps, NE * (ROWS + 1) <= 48 ? 3 : 2)
    balance_grad_kernel(const BalanceGradArgs a) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int SIDE = 32 / LANES;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane % LANES, side = lane / LANES;
    gemm_ptx::pdl_wait();
    const int64_t step = (int64_t)gridDim.x * kGradWarps * SIDE;
    int64_t w0 = ((int64_t)blockIdx.x * kGradWarps + warp) * SIDE;
    float v[ROWS][NE];
    bool in[ROWS];
    auto load = [&] {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int64_t t = w0 + side + r * step;
            const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
            in[r] = t < a.T && a.expert[t * a.top] >= 0;
            load_row<T, LANES>(row, t < a.T, a.E, sub, a.fours, v[r]);
        }
    };
    load();  // beside the counts
    const int n = a.counts[a.E];
    const float by = n > 0 ? 1.f / (float)n : 0.f;
    const float each = by / (float)a.top;
    float f[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = expert_of<LANES>(sub, i);
        f[i] = e < a.E ? (float)a.counts[e] * each : 0.f;
    }
    const float d = a.alpha * (a.dloss ? *a.dloss : 1.f) * (float)a.E * by;
    for (; w0 < a.T; w0 += ROWS * step, load()) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int64_t t = w0 + side + r * step;
            softmax_row<LANES, NE>(v[r]);
            float inner = 0.f;
#pragma unroll
            for (int i = 0; i < NE; ++i) inner = fmaf(v[r][i], f[i], inner);
            inner = sum_lanes<LANES>(inner);
            if (t >= a.T) continue;
            O* row = static_cast<O*>(a.dlogits) + t * a.ldd;
#pragma unroll
            for (int i = 0; i < NE; ++i) v[r][i] = in[r] ? d * v[r][i] * (f[i] - inner) : 0.f;
            if (a.fours && a.beta == 0.f) {
#pragma unroll
                for (int i = 0; i < NE; i += 4) {
                    const int e = expert_of<LANES>(sub, i);
                    if (e >= a.E) continue;
                    alignas(16) O o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = from_f32<O>(v[r][i + j]);
                    *reinterpret_cast<Piece<4 * sizeof(O)>*>(row + e) =
                        *reinterpret_cast<Piece<4 * sizeof(O)>*>(o);
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = expert_of<LANES>(sub, i);
                if (e >= a.E) continue;
                row[e] = from_f32<O>(a.beta != 0.f ? fmaf(a.beta, to_f32(row[e]), v[r][i])
                                                   : v[r][i]);
            }
        }
        __syncwarp();
    }
}

bool rows_ok(const void* p, int64_t rows, int64_t cols, int64_t ld, int es) {
    return p && aligned_to(p, es) && ld >= cols &&
           (__int128)(rows - 1) * ld + cols <= (__int128)(INT64_MAX / es);
}

// Every row begins on, and is a whole number of, four elements.
bool in_fours(const void* p, int64_t E, int64_t ld, int es) {
    return aligned_to(p, 4 * es) && E % 4 == 0 && ld % 4 == 0;
}

// Calls f with integral constants LANES, NE (numbers of a lane) and ROWS. Eight
// lanes a row where that leaves a lane at most 32 numbers: three steps of each
// reduction instead of five, and four rows to an instruction (32768 rows of 160
// experts, forward and gradient: 11.0 and 17.0 us on 32 lanes).
template <typename F>
int with_lanes(int E, F&& f) {
#define BALANCE_RUN(LANES, NE, ROWS)                                                        \
    return f(std::integral_constant<int, LANES>{}, std::integral_constant<int, NE>{},       \
             std::integral_constant<int, ROWS>{})
    if (E <= 32) BALANCE_RUN(8, 4, 4);
    if (E <= 64) BALANCE_RUN(8, 8, 2);
    if (E <= 128) BALANCE_RUN(8, 16, 2);
    if (E <= 160) BALANCE_RUN(8, 20, 1);
    if (E <= 192) BALANCE_RUN(8, 24, 1);
    if (E <= 256) BALANCE_RUN(8, 32, 1);
    if (E <= 512) BALANCE_RUN(32, 16, 2);
    BALANCE_RUN(32, 32, 1);
#undef BALANCE_RUN
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
    // Rows of a block at a time. Two rounds are a block's, up to two for each of its
    // blocks a cluster's, which saves the second kernel (us: 48 rows of E = 64 5.4 by a
    // block, 5.7 by a cluster; 200 rows of E = 160 5.3 by a cluster, 6.1 by blocks and a
    // join, 1024 rows, four rounds, 7.8 and 6.6). Many rows are those of as many blocks
    // as run at once (an eighth less: clusters do not fill the SMs evenly), as many
    // rounds each.
    const int64_t each = kWarps * (E <= 256 ? 4 : 1), rounds = (T + each - 1) / each;
    const size_t smem = (size_t)(E + 1 + kWarps * E) * 4;
    Scratch scratch{pool, s, dev->device};
    const bool fours = in_fours(logits, E, ldl, dtype == GEMM_F32 ? 4 : 2);
    BalanceArgs a{T,      (int)E,  (int)top, logits, ldl,     fours,   expert,
                  counts, offsets, prob,     loss,   nullptr, nullptr, dev->err_word};
    rc = with_lanes((int)E, [&](auto lanes, auto ne, auto rows) {
        constexpr int LANES = decltype(lanes)::value;
        constexpr int NE = decltype(ne)::value, ROWS = decltype(rows)::value;
        const bool single = rounds <= 2;
        const int64_t most =
            (int64_t)dev->sm_count * resident(NE * ROWS) * 7 / 8 / kCluster * kCluster;
        int64_t blocks = single ? 1 : kCluster;
        if (rounds > kCluster * 2) {
            const int64_t turns = (rounds + most - 1) / most;
            blocks = ((rounds + turns - 1) / turns + kCluster - 1) / kCluster * kCluster;
        }
        const int clusters = (int)(blocks / kCluster);
        if (clusters > 1) {
            char* mem = static_cast<char*>(scratch.get((size_t)(clusters * (2 * E + 1) * 4)));
            if (!mem) return (int)kCuda;
            a.part_p = reinterpret_cast<float*>(mem);
            a.part_n = reinterpret_cast<int32_t*>(mem + clusters * E * 4);
        }
        auto run = [&](auto t) {
            using L = decltype(t);
            return launch_dependent(single ? balance_kernel<L, LANES, NE, ROWS, 1>
                                           : balance_kernel<L, LANES, NE, ROWS, kCluster>,
                                    dim3((unsigned)blocks), dim3(32 * kWarps), smem, s, a);
        };
        const int r = dtype == GEMM_F32 ? run(float{})
                      : dtype == GEMM_BF16_F32 || dtype == GEMM_BF16_BF16 ? run(__nv_bfloat16{})
                                                                          : run(__half{});
        if (r != kOk || clusters < 2) return r;
        int shares = 1;
        while (shares * 2 * E <= 1024) shares *= 2;
        return launch_dependent(balance_join_kernel, dim3(1), dim3(1024), 0, s, a, clusters,
                                shares);
    });
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
    const bool fours = in_fours(logits, E, ldl, dtype == GEMM_F32 ? 4 : 2) &&
                       in_fours(dlogits, E, ldd, os);
    const BalanceGradArgs a{T,      (int)E, (int)top, logits, ldl,  fours,   expert,
                            counts, dloss,  alpha,    beta,   dlogits, ldd};
    const int each = kGradWarps * (E <= 256 ? 4 : 1);  // rows of a block at a time
    int64_t blocks = (T + each - 1) / each;
    const int64_t most = (int64_t)dev->sm_count * 8;
    if (blocks > most) blocks = most;
    return with_lanes((int)E, [&](auto lanes, auto ne, auto rows) {
        constexpr int LANES = decltype(lanes)::value;
        constexpr int NE = decltype(ne)::value, ROWS = decltype(rows)::value;
        auto run = [&](auto t, auto o) {
            return launch_dependent(balance_grad_kernel<decltype(t), decltype(o), LANES, NE, ROWS>,
                                    dim3((unsigned)blocks), dim3(32 * kGradWarps), 0, s, a);
        };
        switch (dtype) {
            case GEMM_F32: return run(float{}, float{});
            case GEMM_F16_F32: return run(__half{}, float{});
            case GEMM_BF16_F32: return run(__nv_bfloat16{}, float{});
            case GEMM_F16_F16: return run(__half{}, __half{});
            default: return run(__nv_bfloat16{}, __nv_bfloat16{});
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
