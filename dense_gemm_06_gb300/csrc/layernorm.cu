// layernorm.cu -- layernorm_rows() and layernorm_rows_grad().
//
//   mean = sum x / N,  rstd = 1 / sqrt(sum (x - mean)^2 / N + eps)
//   xhat = (x - mean) rstd,  y = xhat weight + bias
//   g = dy weight,  dx = rstd (g - sum g / N - xhat sum (g xhat) / N)
//   dweight = sum over rows of dy xhat,  dbias = sum over rows of dy
//
// Both are bound by memory. Forward: a row sits in the registers of one warp (or
// 4 or 16 warps), so x is read once, and the squares are summed around the mean,
// not as a difference of large sums. Backward: a thread owns 16 columns and walks
// down the rows of its block with 32 running sums in registers, so x and dy are
// read once for dx, dweight and dbias together; the blocks' sums, N numbers each,
// are added by a second kernel in the order of the blocks, so results do not
// depend on timing. 8192 rows of 2048, bf16 with fp32 weights: forward 13.8 us (4.9
// TB/s), gradient 19.5 us (5.2 TB/s) and 4.9 us for the sums; 10007 rows of 8191,
// fp32: 311 us together, 5.3 TB/s.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gemm.h"
#include "internal.h"
#include "policy.h"
#include "rows.cuh"

namespace libgemm {
namespace {

// VEC elements at once (16 bytes of them, or one).
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

// VEC numbers from `p` (VEC > 1: 16-byte aligned), or `other` where p is null.
template <typename W, int VEC>
__device__ __forceinline__ void load_weights(const W* p, int64_t at, float other,
                                             float (&out)[VEC]) {
    constexpr int PER = VEC == 1 ? 1 : 16 / (int)sizeof(W);
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[e] = other;
    if (!p) return;
#pragma unroll
    for (int j = 0; j < VEC; j += PER) {
        const Pack<W, PER> k = *reinterpret_cast<const Pack<W, PER>*>(p + at + j);
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (j + e < VEC) out[j + e] = to_f32(k.v[e]);
    }
}

// Two fp32 numbers that one instruction works on (each rounded as by itself): the
// kernels that walk down the rows are bound by instructions as much as by memory.
struct Two {
    unsigned long long v;
};
__device__ __forceinline__ Two two(float a, float b) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 apart(Two a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float sum2(Two a) {
    const float2 f = apart(a);
    return f.x + f.y;
}

// A vector's elements in pairs, and back.
template <typename T, int VEC>
__device__ __forceinline__ void to_pairs(const Pack<T, VEC>& p, Two (&out)[VEC / 2]) {
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(&p)[j];
            out[j] = two(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        } else {
            out[j] = two(to_f32(p.v[2 * j]), to_f32(p.v[2 * j + 1]));
        }
    }
}
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> from_pairs(const Two (&in)[VEC / 2]) {
    Pack<T, VEC> p;
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
        const float2 f = apart(in[j]);
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
            reinterpret_cast<__nv_bfloat162*>(&p)[j] = __floats2bfloat162_rn(f.x, f.y);
        else if constexpr (std::is_same<T, __half>::value)
            reinterpret_cast<__half2*>(&p)[j] = __floats2half2_rn(f.x, f.y);
        else
            p.v[2 * j] = f.x, p.v[2 * j + 1] = f.y;
    }
    return p;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums over the WARPS warps that share a row (a whole block when WARPS > 1);
// `slots` holds WARPS x K numbers, and every use of it is one barrier apart from
// the next use of the same half.
template <int WARPS, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* slots) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
    if constexpr (WARPS > 1) {
        const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) slots[w * K + k] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float t = lane < WARPS ? slots[lane * K + k] : 0.f;
#pragma unroll
            for (int o = (WARPS > 16 ? 32 : WARPS) / 2; o; o >>= 1)
                t += __shfl_xor_sync(0xffffffffu, t, o);
            v[k] = __shfl_sync(0xffffffffu, t, 0);
        }
    }
}

struct NormArgs {
    int64_t M;
    int N;
    const void* x;
    int64_t ldx;
    const void* weight;  // null: ones
    const void* bias;    // null: zeros
    float eps;
    void* y;
    int64_t ldy;
    float* mean;  // null: not kept
    float* rstd;
};

// A row for each WARPS warps; NV vectors of VEC elements in each thread. Blocks
// of BLOCK threads hold BLOCK / (32 WARPS) rows.
template <typename T, typename W, int WARPS, int NV, int VEC, int BLOCK>
__global__ void __launch_bounds__(BLOCK) norm_kernel(const NormArgs a) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int TR = 32 * WARPS;  // threads of a row
    __shared__ float slots[2][WARPS > 1 ? WARPS : 1];
    const int tid = threadIdx.x % TR;
    const int64_t row = (int64_t)blockIdx.x * (BLOCK / TR) + threadIdx.x / TR;
    gemm_ptx::pdl_wait();
    if (row >= a.M) return;  // a whole warp, or (WARPS > 1) a whole block
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    Pack<T, VEC> v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TR + tid) * VEC;
        if (c < a.N) v[i] = *reinterpret_cast<const Pack<T, VEC>*>(x + c);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((i * TR + tid) * VEC < a.N) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[0] += to_f32(v[i].v[e]);
        }
    row_sum<WARPS, 1>(s, slots[0]);
    const float mean = s[0] / (float)a.N;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((i * TR + tid) * VEC < a.N) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = to_f32(v[i].v[e]) - mean;
                s[0] = fmaf(d, d, s[0]);
            }
        }
    row_sum<WARPS, 1>(s, slots[1]);
    const float rstd = rsqrtf(s[0] / (float)a.N + a.eps);
    if (tid == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(a.y) + row * a.ldy;
    const W* weight = static_cast<const W*>(a.weight);
    const W* bias = static_cast<const W*>(a.bias);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TR + tid) * VEC;
        if (c >= a.N) continue;
        float w[VEC], b[VEC];
        load_weights<W, VEC>(weight, c, 1.f, w);
        load_weights<W, VEC>(bias, c, 0.f, b);
        Pack<T, VEC> o;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            o.v[e] = from_f32<T>(fmaf((to_f32(v[i].v[e]) - mean) * rstd, w[e], b[e]));
        *reinterpret_cast<Pack<T, VEC>*>(y + c) = o;
    }
}

// A copy of 16 bytes into shared memory that this thread waits for itself.
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"(gemm_ptx::smem_u32(to)), "l"(from) : "memory");
}

constexpr int kOwn = 16;  // columns of a thread in the kernels that walk down the rows

// Many rows: a block of WARPS x LANES warps walks down the rows, LANES of them side
// by side, each on WARPS warps (LANES > 1 only with one warp a row). Thread tid of a
// row owns the columns (i TR + tid) VEC + e, i < kOwn / VEC: their weights stay in
// its registers, and it copies its own parts of the next rows into its own shared
// memory, so that the copies need no barrier. (A row a warp, the weights read from
// L1 for each: 8192 rows of 2048, bf16 with fp32 weights, 19 us.)
constexpr int kWalkStages = 4;
template <typename T, typename W, int WARPS, int LANES, int VEC>
__global__ void __launch_bounds__(32 * WARPS * LANES) norm_walk_kernel(const NormArgs a) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int TR = 32 * WARPS, NV = kOwn / VEC, P = kOwn / 2;
    constexpr int THREADS = TR * LANES, STAGES = kWalkStages;
    constexpr bool RING = VEC > 1;  // single elements: the next row in registers
    using V = Pack<T, VEC>;
    extern __shared__ __align__(16) uint8_t ring[];  // STAGES x NV x THREADS vectors
    __shared__ float slots[2][WARPS];
    const int tid = threadIdx.x % TR;
    // the column of a thread's number k
    auto column = [&](int k) { return (k / VEC * TR + tid) * VEC + k % VEC; };
    gemm_ptx::pdl_wait();
    Two w[P], b[P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = column(i * VEC);
        const bool in = c < a.N;
        float f[VEC], g[VEC];
        load_weights<W, VEC>(in ? static_cast<const W*>(a.weight) : nullptr, c, 1.f, f);
        load_weights<W, VEC>(in ? static_cast<const W*>(a.bias) : nullptr, c, 0.f, g);
        if constexpr (VEC > 1) {
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                w[i * VEC / 2 + j] = two(f[2 * j], f[2 * j + 1]);
                b[i * VEC / 2 + j] = two(g[2 * j], g[2 * j + 1]);
            }
        } else if (i % 2 == 0) {
            w[i / 2] = two(f[0], 0.f);
            b[i / 2] = two(g[0], 0.f);
        } else {
            w[i / 2] = two(apart(w[i / 2]).x, f[0]);
            b[i / 2] = two(apart(b[i / 2]).x, g[0]);
        }
    }
    const int64_t step = (int64_t)gridDim.x * LANES;
    const int64_t row0 = (int64_t)blockIdx.x * LANES + threadIdx.x / TR;
    auto slot = [&](int stage, int i) {
        return reinterpret_cast<V*>(ring) + (stage * NV + i) * THREADS + threadIdx.x;
    };
    V x[NV];
    auto fetch = [&](int64_t row, int stage) {
        if (row < a.M) {
            const T* from = static_cast<const T*>(a.x) + row * a.ldx;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = column(i * VEC);
                if (c >= a.N) continue;
                if constexpr (RING) copy_async(slot(stage, i), from + c);
                else x[i] = *reinterpret_cast<const V*>(from + c);
            }
        }
        if constexpr (RING) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (RING) {
        for (int k = 0; k < STAGES - 1; ++k) fetch(row0 + k * step, k);
    } else {
        fetch(row0, 0);
    }
    const float inv = 1.f / (float)a.N;
    int stage = 0;
    for (int64_t row = row0; row < a.M; row += step) {
        Two v[P], t = two(0.f, 0.f);
        if constexpr (RING) {
            asm volatile("cp.async.wait_group %0;" :: "n"(STAGES - 2) : "memory");
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (column(i * VEC) >= a.N) continue;
                Two part[VEC / 2 > 0 ? VEC / 2 : 1];
                to_pairs<T, VEC>(*slot(stage, i), part);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    v[i * VEC / 2 + j] = part[j];
                    t = add2(t, part[j]);
                }
            }
            fetch(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
            if (++stage == STAGES) stage = 0;
        } else {
#pragma unroll
            for (int k = 0; k < P; ++k) {
                v[k] = two(column(2 * k) < a.N ? to_f32(x[2 * k].v[0]) : 0.f,
                           column(2 * k + 1) < a.N ? to_f32(x[2 * k + 1].v[0]) : 0.f);
                t = add2(t, v[k]);
            }
            fetch(row + step, 0);
        }
        float s[1] = {sum2(t)};
        row_sum<WARPS, 1>(s, slots[0]);
        const float mean = s[0] / (float)a.N;
        const Two off = two(-mean, -mean);
        t = two(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            if (column(2 * k) >= a.N) continue;
            v[k] = add2(v[k], off);
            if (VEC == 1 && column(2 * k + 1) >= a.N) v[k] = two(apart(v[k]).x, 0.f);
            t = fma2(v[k], v[k], t);
        }
        s[0] = sum2(t);
        row_sum<WARPS, 1>(s, slots[1]);
        const float rstd = rsqrtf(s[0] * inv + a.eps);
        if (tid == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        const Two by = two(rstd, rstd);
        T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
        for (int k = 0; k < P; ++k) v[k] = fma2(mul2(v[k], by), w[k], b[k]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column(i * VEC);
            if (c >= a.N) continue;
            if constexpr (VEC > 1) {
                Two part[VEC / 2];
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) part[j] = v[i * VEC / 2 + j];
                *reinterpret_cast<V*>(y + c) = from_pairs<T, VEC>(part);
            } else {
                const float2 f = apart(v[i / 2]);
                y[c] = from_f32<T>(i % 2 ? f.y : f.x);
            }
        }
    }
    if constexpr (RING) asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Rows too long for the registers of a block: x is read three times (from L2
// after the first).
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
    gemm_ptx::pdl_launch_dependents();
    __shared__ float slots[2][32];
    gemm_ptx::pdl_wait();
    const W* weight = static_cast<const W*>(a.weight);
    const W* bias = static_cast<const W*>(a.bias);
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        T* y = static_cast<T*>(a.y) + row * a.ldy;
        float s[1] = {0.f};
        for (int64_t c = threadIdx.x; c < a.N; c += 1024) s[0] += to_f32(x[c]);
        row_sum<32, 1>(s, slots[0]);
        const float mean = s[0] / (float)a.N;
        s[0] = 0.f;
        for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
            const float d = to_f32(x[c]) - mean;
            s[0] = fmaf(d, d, s[0]);
        }
        row_sum<32, 1>(s, slots[1]);
        const float rstd = rsqrtf(s[0] / (float)a.N + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
            const float h = (to_f32(x[c]) - mean) * rstd;
            const float w = weight ? to_f32(weight[c]) : 1.f;
            y[c] = from_f32<T>(fmaf(h, w, bias ? to_f32(bias[c]) : 0.f));
        }
    }
}

struct NormGradArgs {
    int64_t M;
    int N;
    const void* x;
    int64_t ldx;
    const void* weight;
    const float* mean;
    const float* rstd;
    const void* dy;
    int64_t lddy;
    void* dx;  // null: not wanted
    int64_t lddx;
    float* part;  // blocks x 2 x N sums, or null: not wanted
};

constexpr int kGradWarps = 16;  // on an SM

// Rows on their way to a thread, the one that it works on included. With 16-bit
// rows of 2048, 128 threads and four blocks on an SM that is 96 KB in flight.
template <typename T, int WARPS>
constexpr int kNormStages = sizeof(T) == 2 && WARPS < 32 ? 4 : 3;

// A block of WARPS x LANES warps: LANES rows side by side, each on WARPS warps
// (LANES > 1 only with one warp a row). Thread tid of a row owns the columns
// (i TR + tid) VEC + e, i < kOwn / VEC. It copies its own parts of the next rows
// into its own shared memory, so that the copies need no barrier. (Single elements
// go to registers, one row ahead: 4-byte copies of 10007 rows of 8191 took 222 us,
// loads 166.)
template <typename T, typename W, int WARPS, int LANES, int VEC>
__global__ void __launch_bounds__(32 * WARPS * LANES)
    norm_grad_kernel(const NormGradArgs a) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int TR = 32 * WARPS, NV = kOwn / VEC, THREADS = TR * LANES;
    constexpr int STAGES = kNormStages<T, WARPS>;
    constexpr bool RING = VEC > 1;
    using V = Pack<T, VEC>;
    extern __shared__ __align__(16) uint8_t ring[];  // STAGES x (x, dy) x NV x THREADS vectors
    __shared__ float slots[2][2 * WARPS];
    __shared__ float merge[LANES > 1 ? (LANES - 1) * TR * 2 : 1];
    const int tid = threadIdx.x % TR, sub = threadIdx.x / TR;
    gemm_ptx::pdl_wait();
    float w[kOwn];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TR + tid) * VEC;
        float f[VEC];
        load_weights<W, VEC>(c < a.N ? static_cast<const W*>(a.weight) : nullptr, c, 1.f, f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[i * VEC + e] = f[e];
    }
    float dw[kOwn] = {}, db[kOwn] = {};
    const float inv = 1.f / (float)a.N;
    const int64_t step = (int64_t)gridDim.x * LANES;
    const int64_t row0 = (int64_t)blockIdx.x * LANES + sub;
    auto slot = [&](int stage, int which, int i) {
        return reinterpret_cast<V*>(ring) + ((stage * 2 + which) * NV + i) * THREADS + threadIdx.x;
    };
    V xv[NV], gv[NV];
    auto fetch = [&](int64_t row, int stage) {
        if (row < a.M) {
            const T* x = static_cast<const T*>(a.x) + row * a.ldx;
            const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TR + tid) * VEC;
                if (c >= a.N) continue;
                if constexpr (RING) {
                    copy_async(slot(stage, 0, i), x + c);
                    copy_async(slot(stage, 1, i), dy + c);
                } else {
                    xv[i] = *reinterpret_cast<const V*>(x + c);
                    gv[i] = *reinterpret_cast<const V*>(dy + c);
                }
            }
        }
        if constexpr (RING) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (RING) {
        for (int k = 0; k < STAGES - 1; ++k) fetch(row0 + k * step, k);
    } else {
        fetch(row0, 0);
    }
    // the rows' statistics: of one of the block's next 32 rows in each lane, or (not
    // RING) of the next row
    float means = 0.f, rstds = 0.f;
    if (!RING && row0 < a.M) means = a.mean[row0], rstds = a.rstd[row0];
    int turn = 0, stage = 0, at = 0;
    for (int64_t row = row0; row < a.M; row += step, turn ^= 1, at = (at + 1) & 31) {
        if (RING && at == 0) {
            const int64_t t = row + (threadIdx.x & 31) * step;
            if (t < a.M) means = a.mean[t], rstds = a.rstd[t];
        }
        float h[kOwn], g[kOwn], s[2] = {0.f, 0.f};
        const float m = RING ? __shfl_sync(0xffffffffu, means, at) : means;
        const float r = RING ? __shfl_sync(0xffffffffu, rstds, at) : rstds;
        if constexpr (RING) {
            asm volatile("cp.async.wait_group %0;" :: "n"(STAGES - 2) : "memory");
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                xv[i] = *slot(stage, 0, i);
                gv[i] = *slot(stage, 1, i);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = (i * TR + tid) * VEC < a.N;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int k = i * VEC + e;
                h[k] = in ? (to_f32(xv[i].v[e]) - m) * r : 0.f;
                const float d = in ? to_f32(gv[i].v[e]) : 0.f;
                dw[k] = fmaf(d, h[k], dw[k]);
                db[k] += d;
                g[k] = d * w[k];
                s[0] += g[k];
                s[1] = fmaf(g[k], h[k], s[1]);
            }
        }
        // the next rows' reads beside this one's sums (the stage that was read the
        // round before)
        if constexpr (RING) fetch(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
        else fetch(row + step, 0);
        if (!RING && row + step < a.M) means = a.mean[row + step], rstds = a.rstd[row + step];
        if (++stage == STAGES) stage = 0;
        if (a.dx) {
            row_sum<WARPS, 2>(s, slots[turn]);
            const float c0 = s[0] * inv, c1 = s[1] * inv;
            T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TR + tid) * VEC;
                if (c >= a.N) continue;
                V o;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int k = i * VEC + e;
                    o.v[e] = from_f32<T>(r * (g[k] - c0 - h[k] * c1));
                }
                *reinterpret_cast<V*>(dx + c) = o;
            }
        }
    }
    if constexpr (RING) asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!a.part) return;
    if constexpr (LANES > 1) {  // the block's rows, in the order of its warps
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            __syncthreads();
            if (sub > 0) {
                merge[((sub - 1) * TR + tid) * 2] = dw[k];
                merge[((sub - 1) * TR + tid) * 2 + 1] = db[k];
            }
            __syncthreads();
            if (sub > 0) continue;
#pragma unroll 1
            for (int o = 0; o < LANES - 1; ++o) {
                dw[k] += merge[(o * TR + tid) * 2];
                db[k] += merge[(o * TR + tid) * 2 + 1];
            }
        }
        if (sub > 0) return;
    }
    // whole vectors at once: single stores of 608 blocks' sums of 2048 columns took a
    // third of the kernel
    constexpr int PER = VEC == 1 ? 1 : 4;
    struct alignas(4 * PER) Out { float v[PER]; };
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.N;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TR + tid) * VEC;
        if (c >= a.N) continue;
#pragma unroll
        for (int e = 0; e < VEC; e += PER) {
            Out u, v;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                u.v[k] = dw[i * VEC + e + k];
                v.v[k] = db[i * VEC + e + k];
            }
            *reinterpret_cast<Out*>(part + c + e) = u;
            *reinterpret_cast<Out*>(part + a.N + c + e) = v;
        }
    }
}

// Long rows, first pass: dx of a row per block; x and dy are read twice.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_grad_long_kernel(const NormGradArgs a) {
    gemm_ptx::pdl_launch_dependents();
    __shared__ float slots[2][64];
    gemm_ptx::pdl_wait();
    const W* weight = static_cast<const W*>(a.weight);
    const float inv = 1.f / (float)a.N;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        T* dx = static_cast<T*>(a.dx) + row * a.lddx;
        const float mean = a.mean[row], r = a.rstd[row];
        float s[2] = {0.f, 0.f};
        for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
            const float g = to_f32(dy[c]) * (weight ? to_f32(weight[c]) : 1.f);
            s[0] += g;
            s[1] = fmaf(g, (to_f32(x[c]) - mean) * r, s[1]);
        }
        row_sum<32, 2>(s, slots[turn]);
        for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
            const float g = to_f32(dy[c]) * (weight ? to_f32(weight[c]) : 1.f);
            const float h = (to_f32(x[c]) - mean) * r;
            dx[c] = from_f32<T>(r * (g - s[0] * inv - h * (s[1] * inv)));
        }
    }
}

// Long rows, second pass: a block's 256 columns over its share of the rows.
template <typename T>
__global__ void __launch_bounds__(256) norm_grad_long_sums_kernel(const NormGradArgs a) {
    gemm_ptx::pdl_launch_dependents();
    gemm_ptx::pdl_wait();
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= a.N) return;
    float u = 0.f, v = 0.f;
    for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y) {
        const float d = to_f32(static_cast<const T*>(a.dy)[row * a.lddy + c]);
        const float x = to_f32(static_cast<const T*>(a.x)[row * a.ldx + c]);
        u = fmaf(d, (x - a.mean[row]) * a.rstd[row], u);
        v += d;
    }
    float* part = a.part + (int64_t)blockIdx.y * 2 * a.N;
    part[c] = u;
    part[a.N + c] = v;
}

// dweight and dbias: the blocks' sums, added in their order within 32 shares.
constexpr int kShares = 32;
template <typename W>
__global__ void __launch_bounds__(32 * kShares)
    norm_join_kernel(const float* __restrict__ part, int blocks, int N, W* __restrict__ dweight,
                     W* __restrict__ dbias, float beta) {
    gemm_ptx::pdl_launch_dependents();
    __shared__ float got[kShares][32];
    gemm_ptx::pdl_wait();
    const int share = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;  // of 2 N: dweight, then dbias
    float s = 0.f;
    constexpr int AHEAD = 10;  // reads in flight
    if (c < 2 * (int64_t)N)
        for (int b = share; b < blocks; b += AHEAD * kShares) {
            float v[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int64_t at = b + j * kShares;
                v[j] = at < blocks ? part[at * 2 * N + c] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) s += v[j];
        }
    got[share][lane] = s;
    __syncthreads();
    for (int o = kShares / 2; o; o /= 2) {
        if (share < o) got[share][lane] += got[share + o][lane];
        __syncthreads();
    }
    if (share > 0 || c >= 2 * (int64_t)N) return;
    s = got[0][lane];
    W* out = c < N ? dweight : dbias;
    if (!out) return;
    W* at = out + (c < N ? c : c - N);
    *at = from_f32<W>(beta != 0.f ? fmaf(beta, to_f32(*at), s) : s);
}

int row_bytes(int dtype) { return dtype == GEMM_F32 ? 4 : 2; }
int weight_bytes(int dtype) { return dtype <= GEMM_BF16_F32 ? 4 : 2; }
bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool rows_ok(const void* p, int64_t M, int64_t N, int64_t ld, int es) {
    return p && aligned_to(p, es) && ld >= N &&
           (__int128)(M - 1) * ld + N <= (__int128)(INT64_MAX / es);
}
bool vec_ready(const void* p, int64_t ld, int es) {
    return aligned_to(p, 16) && ld * es % 16 == 0;
}

template <typename T, typename W, int VEC>
int norm_dispatch(const NormArgs& a, const DeviceInfo& dev, cudaStream_t s) {
    auto run = [&](auto warps, auto nv, auto block) {
        constexpr int WARPS = decltype(warps)::value, NV = decltype(nv)::value;
        constexpr int BLOCK = decltype(block)::value, ROWS = BLOCK / (32 * WARPS);
        return launch_dependent(norm_kernel<T, W, WARPS, NV, VEC, BLOCK>,
                                dim3((unsigned)((a.M + ROWS - 1) / ROWS)), dim3(BLOCK), 0, s, a);
    };
    auto walk = [&](auto warps, auto lanes) {
        constexpr int WARPS = decltype(warps)::value, LANES = decltype(lanes)::value;
        constexpr int THREADS = 32 * WARPS * LANES;
        constexpr int SMEM = VEC > 1 ? kWalkStages * kOwn * (int)sizeof(T) * THREADS : 0;
        auto kern = norm_walk_kernel<T, W, WARPS, LANES, VEC>;
        const int rc = allow_smem(kern, SMEM, dev);
        if (rc != kOk) return rc;
        constexpr int WALK_WARPS = 24;  // on an SM
        const int64_t rows = (a.M + LANES - 1) / LANES;
        const int64_t most = dev.sm_count * (WALK_WARPS / (WARPS * LANES));
        return launch_dependent(kern, dim3((unsigned)(rows < most ? rows : most)), dim3(THREADS),
                                SMEM, s, a);
    };
    using std::integral_constant;
#define NORM_RUN(WARPS, NV, BLOCK)                                                     \
    return run(integral_constant<int, WARPS>{}, integral_constant<int, NV>{},          \
               integral_constant<int, BLOCK>{})
#define NORM_WALK(WARPS, LANES) \
    return walk(integral_constant<int, WARPS>{}, integral_constant<int, LANES>{})
    // vectors of a thread: 8 at most by 16 bytes, 32 single elements
    constexpr int MOST = VEC == 1 ? 32 : 8;
    const int64_t vecs = (a.N + VEC - 1) / VEC;
    // Some rows for each block, which then reads the weights once for them (us, bf16:
    // 8192 rows of 2048 13.8, a row a warp 19; of 2047, single elements, 22.4 and 38.4;
    // fp16, 16384 rows of 1001 25.8 and 22.9).
    if (a.M * a.N >= (int64_t)dev.sm_count * 16384) {
        if (a.N <= 32 * kOwn) NORM_WALK(1, 4);
        if (a.N <= 64 * kOwn) NORM_WALK(2, 1);
        if (a.N <= 128 * kOwn) NORM_WALK(4, 1);
        if (a.N <= 256 * kOwn) NORM_WALK(8, 1);
    }
    if (vecs <= 32) NORM_RUN(1, 1, 128);
    if (vecs <= 128 * (MOST / 4)) NORM_RUN(4, MOST / 4, 128);
    if (vecs <= 128 * MOST) NORM_RUN(4, MOST, 128);
    if (vecs <= 512 * (MOST / 2)) NORM_RUN(16, MOST / 2, 512);
    if (vecs <= 512 * MOST) NORM_RUN(16, MOST, 512);
#undef NORM_RUN
#undef NORM_WALK
    return launch_dependent(norm_long_kernel<T, W>,
                            dim3((unsigned)(a.M < dev.sm_count * 2 ? a.M : dev.sm_count * 2)),
                            dim3(1024), 0, s, a);
}

template <typename T, typename W>
int norm_forward(const NormArgs& a, const DeviceInfo& dev, cudaStream_t s) {
    const bool vec = vec_ready(a.x, a.ldx, sizeof(T)) && vec_ready(a.y, a.ldy, sizeof(T)) &&
                     a.N % (16 / sizeof(T)) == 0 && aligned_to(a.weight, 16) &&
                     aligned_to(a.bias, 16);
    return vec ? norm_dispatch<T, W, 16 / sizeof(T)>(a, dev, s) : norm_dispatch<T, W, 1>(a, dev, s);
}

// The backward kernel's blocks (its sums' parts) for rows of N columns: 0 where
// the rows are too long for it. 32 warps a row leave a thread 64 registers, which
// pays only for 16-bit rows read in vectors (2048 rows, us, by them and by the kernels
// of long rows: 12000 bf16 87 and 141; 12001 bf16, single elements, 167 and 141, fp16 244
// and 137, though 16383 bf16 187 and 198; 12000 fp32 297 and 161). 16 warps on an SM:
// 19.5 us for 8192 rows of 2048, 5.2 TB/s.
struct GradPlan {
    int warps, lanes, blocks;
};
GradPlan grad_plan(int64_t M, int64_t N, bool vec16, int sm_count) {
    GradPlan g{32, 1, 0};
    if (N > (vec16 ? 32 : 16) * 32 * kOwn) return g;
    for (int w : {1, 2, 4, 8, 16, 32})
        if (N <= 32 * w * kOwn) {
            g.warps = w;
            break;
        }
    g.lanes = g.warps == 1 ? 4 : 1;
    const int64_t rows = (M + g.lanes - 1) / g.lanes;
    const int64_t most = (int64_t)sm_count * (g.warps == 32 ? 1 : kGradWarps / (g.warps * g.lanes));
    g.blocks = (int)(rows < most ? rows : most);
    return g;
}
constexpr int kLongShares = 32;

template <typename T, typename W, int WARPS, int LANES, int VEC>
int run_norm_grad(const NormGradArgs& a, int blocks, const DeviceInfo& dev, cudaStream_t s) {
    constexpr int THREADS = 32 * WARPS * LANES;
    constexpr int STAGES = kNormStages<T, WARPS>;
    constexpr int SMEM = VEC > 1 ? STAGES * 2 * kOwn * (int)sizeof(T) * THREADS : 0;
    auto kern = norm_grad_kernel<T, W, WARPS, LANES, VEC>;
    const int rc = allow_smem(kern, SMEM, dev);
    if (rc != kOk) return rc;
    return launch_dependent(kern, dim3(blocks), dim3(THREADS), SMEM, s, a);
}

template <typename T, typename W>
int norm_backward(NormGradArgs a, W* dweight, W* dbias, float beta, const DeviceInfo& dev,
                  cudaMemPool_t pool, cudaStream_t s) {
    const bool sums = dweight || dbias;
    int rc = kOk;
    const bool vec = vec_ready(a.x, a.ldx, sizeof(T)) && vec_ready(a.dy, a.lddy, sizeof(T)) &&
                     (!a.dx || vec_ready(a.dx, a.lddx, sizeof(T))) &&
                     a.N % (16 / sizeof(T)) == 0 && aligned_to(a.weight, 16);
    const GradPlan g = grad_plan(a.M, a.N, vec && sizeof(T) == 2, dev.sm_count);
    const int parts = g.blocks > 0 ? g.blocks : (int)(a.M < kLongShares ? a.M : kLongShares);
    Scratch scratch{pool, s, dev.device};
    if (sums && a.M > 0) {
        a.part = static_cast<float*>(scratch.get((size_t)parts * 2 * a.N * 4));
        if (!a.part) return kCuda;
    }
    if (a.M > 0 && g.blocks > 0) {
#define NORM_GRAD_RUN(WARPS, LANES)                                                        \
    rc = vec ? run_norm_grad<T, W, WARPS, LANES, 16 / (int)sizeof(T)>(a, g.blocks, dev, s) \
             : run_norm_grad<T, W, WARPS, LANES, 1>(a, g.blocks, dev, s)
        switch (g.warps) {
            case 1: NORM_GRAD_RUN(1, 4); break;
            case 2: NORM_GRAD_RUN(2, 1); break;
            case 4: NORM_GRAD_RUN(4, 1); break;
            case 8: NORM_GRAD_RUN(8, 1); break;
            case 16: NORM_GRAD_RUN(16, 1); break;
            default:
                if constexpr (sizeof(T) == 2)
                    rc = run_norm_grad<T, W, 32, 1, 8>(a, g.blocks, dev, s);
                break;
        }
#undef NORM_GRAD_RUN
    } else if (a.M > 0) {
        // the sums first: dx may be written over x or dy
        if (sums)
            rc = launch_dependent(norm_grad_long_sums_kernel<T>,
                                  dim3((unsigned)((a.N + 255) / 256), (unsigned)parts), dim3(256),
                                  0, s, a);
        if (rc == kOk && a.dx)
            rc = launch_dependent(norm_grad_long_kernel<T, W>,
                                  dim3((unsigned)(a.M < dev.sm_count * 2 ? a.M
                                                                         : dev.sm_count * 2)),
                                  dim3(1024), 0, s, a);
    }
    if (rc == kOk && sums)
        rc = launch_dependent(norm_join_kernel<W>, dim3((unsigned)((2 * (int64_t)a.N + 31) / 32)),
                              dim3(32 * kShares), 0, s, (const float*)a.part,
                              a.M > 0 ? parts : 0, a.N, dweight, dbias, beta);
    scratch.release();
    return rc;
}

int layernorm(int64_t M, int64_t N, const void* x, int64_t ldx, const void* weight,
              const void* bias, float eps, void* y, int64_t ldy, float* mean, float* rstd,
              int dtype, cudaStream_t s) {
    if (dtype < GEMM_F32 || dtype > GEMM_BF16_BF16) return kInvalidArg;
    if (M < 0 || N < 0 || M > INT32_MAX || N > INT32_MAX || !(eps >= 0.f)) return kInvalidArg;
    if (M == 0 || N == 0) return kOk;
    const int es = row_bytes(dtype), ws = weight_bytes(dtype);
    if (!rows_ok(x, M, N, ldx, es) || !rows_ok(y, M, N, ldy, es)) return kInvalidArg;
    if (!aligned_to(weight, ws) || !aligned_to(bias, ws) || !aligned_to(mean, 4) ||
        !aligned_to(rstd, 4))
        return kInvalidArg;
    DeviceInfo* dev = nullptr;
    int rc = current_device_info(&dev, nullptr);
    if (rc != kOk) return rc;
    const void* ptrs[6] = {x, y, weight, bias, mean, rstd};
    rc = check_device_pointers(ptrs, 6, dev->device);
    if (rc != kOk) return rc;
    const NormArgs a{M, (int)N, x, ldx, weight, bias, eps, y, ldy, mean, rstd};
    switch (dtype) {
        case GEMM_F32: return norm_forward<float, float>(a, *dev, s);
        case GEMM_F16_F32: return norm_forward<__half, float>(a, *dev, s);
        case GEMM_BF16_F32: return norm_forward<__nv_bfloat16, float>(a, *dev, s);
        case GEMM_F16_F16: return norm_forward<__half, __half>(a, *dev, s);
        default: return norm_forward<__nv_bfloat16, __nv_bfloat16>(a, *dev, s);
    }
}

int layernorm_grad(int64_t M, int64_t N, const void* x, int64_t ldx, const void* weight,
                   const float* mean, const float* rstd, const void* dy, int64_t lddy, void* dx,
                   int64_t lddx, void* dweight, void* dbias, float beta, int dtype,
                   cudaStream_t s) {
    if (dtype < GEMM_F32 || dtype > GEMM_BF16_BF16) return kInvalidArg;
    if (M < 0 || N < 0 || M > INT32_MAX || N > INT32_MAX) return kInvalidArg;
    const int es = row_bytes(dtype), ws = weight_bytes(dtype);
    if (!aligned_to(weight, ws) || !aligned_to(dweight, ws) || !aligned_to(dbias, ws))
        return kInvalidArg;
    if (N == 0 || (!dx && !dweight && !dbias) || (M == 0 && !dweight && !dbias)) return kOk;
    if (M > 0) {
        if (!rows_ok(x, M, N, ldx, es) || !rows_ok(dy, M, N, lddy, es) || !mean || !rstd ||
            !aligned_to(mean, 4) || !aligned_to(rstd, 4))
            return kInvalidArg;
        if (dx && !rows_ok(dx, M, N, lddx, es)) return kInvalidArg;
    }
    DeviceInfo* dev = nullptr;
    cudaMemPool_t pool = nullptr;
    int rc = current_device_info(&dev, &pool);
    if (rc != kOk) return rc;
    const void* ptrs[8] = {M ? x : nullptr,  M ? weight : nullptr, M ? mean : nullptr,
                           M ? rstd : nullptr, M ? dy : nullptr,   M ? dx : nullptr,
                           dweight, dbias};
    rc = check_device_pointers(ptrs, 8, dev->device);
    if (rc != kOk) return rc;
    const NormGradArgs a{M, (int)N, x, ldx, weight, mean, rstd, dy, lddy, dx, lddx, nullptr};
    auto run = [&](auto t, auto w) {
        using T = decltype(t);
        using W = decltype(w);
        return norm_backward<T, W>(a, static_cast<W*>(dweight), static_cast<W*>(dbias), beta, *dev,
                                   pool, s);
    };
    switch (dtype) {
        case GEMM_F32: return run(float{}, float{});
        case GEMM_F16_F32: return run(__half{}, float{});
        case GEMM_BF16_F32: return run(__nv_bfloat16{}, float{});
        case GEMM_F16_F16: return run(__half{}, __half{});
        default: return run(__nv_bfloat16{}, __nv_bfloat16{});
    }
}

}  // namespace
}  // namespace libgemm

using namespace libgemm;

extern "C" {

int layernorm_rows(int64_t M, int64_t N, const void* x, int64_t ldx, const void* weight,
                   const void* bias, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                   int dtype, void* stream) {
    try {
        return layernorm(M, N, x, ldx, weight, bias, eps, y, ldy, mean, rstd, dtype,
                         static_cast<cudaStream_t>(stream));
    } catch (...) {
        return kCuda;
    }
}

int layernorm_rows_grad(int64_t M, int64_t N, const void* x, int64_t ldx, const void* weight,
                        const float* mean, const float* rstd, const void* dy, int64_t lddy,
                        void* dx, int64_t lddx, void* dweight, void* dbias, float beta, int dtype,
                        void* stream) {
    try {
        return layernorm_grad(M, N, x, ldx, weight, mean, rstd, dy, lddy, dx, lddx, dweight, dbias,
                              beta, dtype, static_cast<cudaStream_t>(stream));
    } catch (...) {
        return kCuda;
    }
}

}  // extern "C"
