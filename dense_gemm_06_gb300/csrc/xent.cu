// xent.cu -- gemm_xent() and gemm_xent_grad(): the softmax cross entropy of a
// projection onto a large vocabulary, and its gradients, without keeping the
// logits.
//
//   z_tv   = sum_k X[t][k] W[v][k]
//   lse_t  = log sum_v exp(z_tv),     loss_t = lse_t - z_t,target
//   G_tv   = alpha dloss_t (exp(z_tv - lse_t) - [v = target_t])
//   dX     = G W,                     dW = beta dW + G^T X
//
// Forward: the kernel of xent.cuh leaves a (maximum, sum of exponentials) pair
// for every row and half tile (128 columns by CTA pairs, 16 to 64 by single CTAs),
// which a second kernel joins: exp(m_i - m) s_i summed over the pairs, the online
// softmax identity. The logits are never stored, only 8 bytes for each pair: 1/64 of
// fp32 logits by CTA pairs.
//
// Backward: piece by piece of the vocabulary the same kernel computes the logits
// again and writes G as 16-bit numbers, which are multiplied with the piece's rows of
// W (dX, summed over the pieces in fp32, in shares of the depth where its tiles are
// few) and with X (the piece's rows of dW, complete). G takes at most 512 MB for each
// of its numbers, or 4096 columns. dX's product adds up its sums every 704 of depth: on
// one accumulator for all of it, gemm()'s way, dX came out 8e-4 too small from 131072
// columns, 2e-4 from 32000 (the means of rows whose terms have one sign; fp16's own
// rounding, of either sign, is 2e-4). The time differs by -6 to 8 % with the fill of the
// last round (bf16 from 32000, dX alone, us: 4096 x 2048 657 and 650 by gemm()'s kernel,
// 4096 x 1280 539 and 497, 1024 x 1280 189 and 202).
//
// Rounding. G is 16-bit because the tensor cores take 16-bit operands: its
// relative 2^-8 (bf16) is that of a 16-bit result itself. An fp32 dW would
// show it, so for that G is two numbers, hi + lo (2^-17 of g), and X is multiplied
// with both in one product of twice the depth, on gemm_grouped_k's kernel.
// G is divided by the largest |alpha dloss|, which the products are multiplied with
// again in fp32 before they are rounded: a mean's 1 / n, rounded to 16 bits, would
// put the same error into every term (0.2 % of dX in bf16), and fp16 has exponents
// only near 1 (there the largest is 2^12, and probabilities reach down to 2^-36).
// That costs the scale's launch and dX an fp32 pass (4096 x 32000 x 2048: 14 of
// 1310 us).
//
// Rows whose target does not count (prompts, padding) take no part: a first kernel
// lists the others, which are copied side by side, and G's kernel and both products
// work on as many tiles as these fill, a number that stays on the device (8192 rows of
// 2048 from 32000, bf16, dX alone: 1286 us, 1015 with 30 % left out, 352 with 80 %). The
// last tile's rows past them are zero in G and in the copy of X (0 times an infinity
// would be NaN).
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "../../include/gemm.h"
#include "internal.h"
#include "policy.h"
#include "repack16.cuh"
#include "rows.cuh"
#include "xent.cuh"

namespace libgemm {
namespace {

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool is_bf16(int dtype) { return dtype == GEMM_BF16_F32 || dtype == GEMM_BF16_BF16; }
bool tma_ready(const void* p, int64_t ld) { return aligned_to(p, 16) && ld % 8 == 0; }

// `rows` rows of `cols` elements, ld apart, stay addressable.
bool span_fits(int64_t rows, int64_t cols, int64_t ld, int esize) {
    if (rows <= 0 || cols <= 0) return true;
    return (__int128)(rows - 1) * ld + cols <= (__int128)(INT64_MAX / esize);
}

// Joins the pairs of a row: a block takes ROWS rows, its threads a row and every
// (kJoinThreads / ROWS)th half tile of it each.
constexpr int kJoinThreads = 512;
template <int ROWS>
__global__ void __launch_bounds__(kJoinThreads)
    xent_join_kernel(const float2* __restrict__ part, int64_t ld, int parts, int M,
                     const float* __restrict__ picked, const int32_t* __restrict__ target,
                     int vocab, float* __restrict__ loss, float* __restrict__ lse) {
    gemm_ptx::pdl_launch_dependents();
    gemm_ptx::pdl_wait();
    constexpr int SHARES = kJoinThreads / ROWS, AHEAD = 8;
    __shared__ float2 got[SHARES][ROWS];
    const int share = threadIdx.x / ROWS, r = threadIdx.x % ROWS;
    const int row = blockIdx.x * ROWS + r;
    float m = -INFINITY, s = 0.f;
    auto join = [&](float2 o) {
        const float nm = fmaxf(m, o.x);
        const float from = nm == -INFINITY ? 0.f : nm;
        s = s * ex2((m - from) * kLog2e) + o.y * ex2((o.x - from) * kLog2e);
        m = nm;
    };
    if (row < M) {
        const float2* at = part + row;
        for (int i = share; i < parts; i += AHEAD * SHARES) {
            float2 v[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                v[j] = i + j * SHARES < parts ? at[(int64_t)(i + j * SHARES) * ld]
                                              : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) join(v[j]);
        }
    }
    got[share][r] = make_float2(m, s);
    for (int o = SHARES / 2; o; o /= 2) {
        __syncthreads();
        if (share < o) {
            join(got[share + o][r]);
            got[share][r] = make_float2(m, s);
        }
    }
    if (share != 0 || row >= M) return;
    const float l = m + logf(s);
    if (lse) lse[row] = l;
    const int t = target[row];
    loss[row] = t >= 0 && t < vocab ? l - picked[row] : 0.f;
}

// K == 0: every logit is zero.
__global__ void xent_uniform_kernel(int M, int vocab, const int32_t* target, float* loss,
                                    float* lse, ErrWord* err) {
    const float l = (float)log((double)vocab);
    for (int r = blockIdx.x * blockDim.x + threadIdx.x; r < M; r += gridDim.x * blockDim.x) {
        const int t = target[r];
        if (t >= vocab) report_bad_value(err);
        if (lse) lse[r] = l;
        loss[r] = t >= 0 && t < vocab ? l : 0.f;
    }
}

// One block: the rows of a gradient that count, in their order (order[j], and place[t]
// the j of row t or -1); scale[0]: what brings the largest finite |alpha dloss_t| of
// them to `to`; scale[1]: its inverse.
__global__ void __launch_bounds__(1024)
    xent_order_kernel(int M, const int32_t* __restrict__ target, int vocab,
                      const float* __restrict__ dloss, float alpha, float to, int tile, int copies,
                      int32_t* __restrict__ order, int32_t* __restrict__ place,
                      XentInfo* __restrict__ info, float* __restrict__ scale, ErrWord* err) {
    gemm_ptx::pdl_launch_dependents();
    gemm_ptx::pdl_wait();
    constexpr int PER = 8;  // rows of a thread
    __shared__ float most[32];
    __shared__ int found[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float top = 0.f;
    int count = 0;
    for (int base = 0; base < M; base += 1024 * PER) {
        const int t0 = base + threadIdx.x * PER;
        int v[PER];
        uint32_t kept = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = t0 + i < M ? target[t0 + i] : -1;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (v[i] >= vocab) report_bad_value(err);
            if (v[i] < 0 || v[i] >= vocab) continue;
            kept |= 1u << i;
            const float d = fabsf(dloss ? alpha * dloss[t0 + i] : alpha);
            if (d < INFINITY) top = fmaxf(top, d);
        }
        int upto = __popc(kept);
        for (int o = 1; o < 32; o *= 2) {
            const int n = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += n;
        }
        if (lane == 31) found[warp] = upto;
        __syncthreads();
        const int n = found[lane];
        int j = count + upto - __popc(kept) +
                __reduce_add_sync(0xffffffffu, lane < warp ? n : 0);
        count += __reduce_add_sync(0xffffffffu, n);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (t0 + i >= M) continue;
            const bool in = kept >> i & 1;
            place[t0 + i] = in ? j : -1;
            if (in) order[j++] = t0 + i;
        }
        __syncthreads();
    }
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) most[warp] = top;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int i = 1; i < 32; ++i) top = fmaxf(top, most[i]);
    if (top == 0.f) top = to;
    top = fminf(fmaxf(top, 0x1p-100f), 0x1p100f);
    scale[0] = to / top;
    scale[1] = top / to;
    const int used = count > 0 ? (count + tile - 1) / tile * tile : tile;
    *info = XentInfo{{0, used * copies}, count, used};
}

// The rows of X that count, one after the other in rows of TMA's alignment, then zeros
// up to whole tiles; with copies == 2 the same again below. A warp per row.
__global__ void __launch_bounds__(256)
    xent_rows_kernel(const uint16_t* __restrict__ X, int64_t ldx, int64_t K,
                     const int32_t* __restrict__ order, const XentInfo* __restrict__ info,
                     uint16_t* __restrict__ out, int64_t ldo, int copies) {
    gemm_ptx::pdl_launch_dependents();
    gemm_ptx::pdl_wait();
    const int count = info->count, used = info->used;
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x / 32);
    for (int64_t r = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
         r < (int64_t)used * copies; r += warps) {
        const int j = (int)(r < used ? r : r - used);
        uint16_t* dst = out + r * ldo;
        if (j < count) {
            repack16_row(X + order[j] * ldx, dst, K, lane);
            for (int64_t c = K + lane; c < ldo; c += 32) dst[c] = 0;
        } else {
            for (int64_t c = lane * 8; c < ldo; c += 256)
                *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
        }
    }
}

// Row t of dX = *scale * (the sum of row place[t] of `parts` matrices, part_rows rows
// apart), rounded once, or zero; rows x cols. A warp takes 32 groups of 8 columns of
// two rows at a time, and stores them in 16-byte pieces whatever dX's alignment.
template <typename T>
__global__ void __launch_bounds__(256)
    xent_finish_kernel(const float* __restrict__ sum, int64_t lds, int parts, int64_t part_rows,
                       T* __restrict__ out, int64_t ldo, int64_t rows, int cols,
                       const int32_t* __restrict__ place, const float* __restrict__ scale) {
    gemm_ptx::pdl_launch_dependents();
    gemm_ptx::pdl_wait();
    constexpr int ROWS = 2, G = 8;
    const float by = *scale;
    const int c = (blockIdx.y * 32 + (threadIdx.x & 31)) * G;
    const int64_t warps = (int64_t)gridDim.x * 8;
    for (int64_t r0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * ROWS; r0 < rows;
         r0 += warps * ROWS) {
        float v[ROWS][G] = {};
        int at[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) at[j] = r0 + j < rows ? place[r0 + j] : -1;
        const float* from = sum + c;
        for (int p = 0; p < parts; ++p, from += part_rows * lds)
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
#pragma unroll
                for (int q = 0; q < G; q += 4) {
                    if (at[j] < 0 || c + q >= lds) continue;  // lds % 4 == 0
                    const float4 f =
                        *reinterpret_cast<const float4*>(from + (int64_t)at[j] * lds + q);
                    v[j][q] += f.x, v[j][q + 1] += f.y, v[j][q + 2] += f.z, v[j][q + 3] += f.w;
                }
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (r0 + j >= rows) continue;
#pragma unroll
            for (int e = 0; e < G; ++e) v[j][e] *= by;
            store_row<T, G>(out + (r0 + j) * ldo, cols, c, v[j]);
        }
    }
}

int finish(const float* sum, int64_t lds, int parts, int64_t part_rows, void* out, int64_t ldo,
           int64_t rows, int64_t cols, const int32_t* place, const float* scale, bool bf16,
           const DeviceInfo& dev, cudaStream_t s) {
    const int64_t across = (cols + 255) / 256;  // warps for a row
    const int64_t turns = (rows + 15) / 16, most = (dev.sm_count * 8 + across - 1) / across;
    const dim3 grid((unsigned)(turns < most ? turns : most), (unsigned)across);
    auto run = [&](auto t) {
        using T = decltype(t);
        return launch_dependent(xent_finish_kernel<T>, grid, dim3(256), 0, s, sum, lds, parts,
                                part_rows, static_cast<T*>(out), ldo, rows, (int)cols, place,
                                scale);
    };
    return bf16 ? run(__nv_bfloat16{}) : run(__half{});
}

// Checks of X, W and target that both calls make; no CUDA calls.
int check_inputs(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const void* W,
                 int64_t ldw, const int32_t* target, int dtype) {
    if (dtype < GEMM_F32 || dtype > GEMM_BF16_BF16) return kInvalidArg;
    if (M < 0 || N < 1 || K < 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX)
        return kInvalidArg;
    if (dtype == GEMM_F32 || N > kXentMaxVocab) return kUnsupported;
    if (M == 0) return kOk;
    if (!target || !aligned_to(target, 4)) return kInvalidArg;
    if (K == 0) return kOk;
    if (!X || !W || !aligned_to(X, 2) || !aligned_to(W, 2) || ldx < K || ldw < K)
        return kInvalidArg;
    if (!span_fits(M, K, ldx, 2) || !span_fits(N, K, ldw, 2)) return kInvalidArg;
    return kOk;
}

// The parts of one scratch buffer, 256-byte aligned.
struct Parts {
    int64_t bytes = 0;
    int64_t add(int64_t n) {
        const int64_t at = bytes;
        bytes += up(n, 256);
        return at;
    }
};

// Copies an operand whose rows TMA cannot read (offset `at` of the scratch).
int repack_one(const void*& p, int64_t& ld, int64_t rows, int64_t cols, char* to,
               const DeviceInfo& dev, cudaStream_t s) {
    Repack16 job{static_cast<const uint16_t*>(p), reinterpret_cast<uint16_t*>(to), ld, up(cols, 8),
                 rows, cols};
    repack16_kernel<<<repack16_blocks(rows, dev.sm_count), 256, 0, s>>>(job, Repack16{});
    if (cudaGetLastError() != cudaSuccess) return kCuda;
    note_launch();
    dispatch_log("repack of a misaligned 16-bit operand, %lld x %lld", (long long)rows,
                 (long long)cols);
    p = job.dst;
    ld = job.ldd;
    return kOk;
}

int launch(XentParams& xp, int mode, bool bf16, const XentShape& shape, const DeviceInfo& dev,
           cudaStream_t s);

// The depth that one accumulator takes: equal parts of at most kXentFold blocks.
void fold_depth(XentParams& xp) {
    const int parts = (xp.num_kb + kXentFold - 1) / kXentFold;
    xp.part_kb = parts > 0 ? (xp.num_kb + parts - 1) / parts : 1;
}

void xent_params(XentParams& xp, int64_t M, int64_t N, int64_t K, const XentShape& shape,
                 int64_t vocab, const int32_t* target, const DeviceInfo& dev) {
    std::memset(&xp, 0, sizeof(xp));
    xp.M = (int)M;
    xp.N = (int)N;
    xp.num_kb = (int)((K + XBK - 1) / XBK);
    fold_depth(xp);
    xp.tile_n = shape.tile_n;
    xp.tiles_m = (int)((M + XROWS * shape.cta_group - 1) / (XROWS * shape.cta_group));
    xp.tiles_n = (int)((N + shape.tile_n - 1) / shape.tile_n);
    xp.x_rows = M < XROWS ? (int)up(M, 8) : XROWS;
    xp.stage_bytes = (xp.x_rows + shape.tile_n) * XBK * 2;
    xp.band = 8;
    xp.vocab = (int)vocab;
    xp.target = target;
    xp.alpha = 1.f;
    xp.err = dev.err_word;
    xp.gen = next_generation();
    xp.wait_limit_ns = option_wait_limit_ns();
    xp.fault_inject = option_tc_fault_inject();
}

// The stages that fit the ring of a mode.
int stages_of(const XentParams& xp, int mode) {
    const int ring = mode == kXentGrad2 ? XentCfg<kXentGrad2>::RING : XentCfg<kXentGrad>::RING;
    const int n = ring / xp.stage_bytes;
    return n < XentCfg<kXentStats>::MOST ? n : XentCfg<kXentStats>::MOST;
}

bool xent_maps(XentParams& xp, bool bf16, const void* X, int64_t ldx, const void* W, int64_t ldw,
               int64_t K, const XentShape& shape) {
    return encode_tma_16(&xp.map_x, bf16, X, (uint64_t)K, (uint64_t)xp.M, (uint64_t)ldx, 0, 0, XBK,
                         shape.cta_group == 2 ? XROWS : (uint32_t)xp.x_rows) &&
           encode_tma_16(&xp.map_w, bf16, W, (uint64_t)K, (uint64_t)xp.N, (uint64_t)ldw, 0, 0, XBK,
                         (uint32_t)(shape.tile_n / shape.cta_group));
}

// dX's part of a piece (n columns, in a vocabulary cut into pieces of `piece`) in
// shares of the depth that are the same for every piece: sums (+)= G W.
int launch_sum(const XentSumPlan& plan, int64_t M, int64_t K, int64_t piece, int64_t n,
               const void* g, int64_t ldg, const void* W, int64_t ldw, float* sums,
               int64_t sum_rows, bool add, const XentInfo* info, bool bf16,
               const DeviceInfo& dev, cudaStream_t s) {
    XentParams xp;
    xent_params(xp, M, K, 0, plan.shape, 0, nullptr, dev);
    xp.all_kb = (int)((n + XBK - 1) / XBK);
    xp.num_kb = (int)plan.each(piece);
    xp.splits = (xp.all_kb + xp.num_kb - 1) / xp.num_kb;
    fold_depth(xp);
    xp.sums = sums;
    xp.sum_ld = up(K, 4);
    xp.sum_rows = sum_rows;
    xp.add = add ? 1 : 0;
    xp.info = info;
    if (!encode_tma_16(&xp.map_x, bf16, g, (uint64_t)n, (uint64_t)M, (uint64_t)ldg, 0, 0, XBK,
                       plan.shape.cta_group == 2 ? XROWS : (uint32_t)xp.x_rows) ||
        !encode_tma_16(&xp.map_w, bf16, W, (uint64_t)K, (uint64_t)n, (uint64_t)ldw, 0, 0, 64, XBK))
        return kCuda;
    return launch(xp, kXentSum, bf16, plan.shape, dev, s);
}

// A piece's rows of a 16-bit dW (n x K) = factor G^T X, `rows` deep; dW's rows lie as
// TMA wants them, and end on 16 bytes: a box that crosses the end of a row in the middle
// of 16 bytes may be stored up to their end.
int launch_table(int64_t n, int64_t K, int64_t rows, const void* g, int64_t ldg, const void* X,
                 int64_t ldx, void* dW, int64_t lddw, const float* factor, const XentInfo* info,
                 bool bf16, const DeviceInfo& dev, cudaStream_t s) {
    const XentShape shape{2, 256};
    XentParams xp;
    xent_params(xp, n, K, rows, shape, 0, nullptr, dev);
    xp.scale = factor;
    xp.info = info;
    if (!encode_tma_16(&xp.map_x, bf16, g, (uint64_t)ldg, (uint64_t)rows, (uint64_t)ldg, 0, 0, 64,
                       XBK) ||
        !encode_tma_16(&xp.map_w, bf16, X, (uint64_t)K, (uint64_t)rows, (uint64_t)ldx, 0, 0, 64,
                       XBK) ||
        !encode_tma_16(&xp.map_g, bf16, dW, (uint64_t)K, (uint64_t)n, (uint64_t)lddw, 0, 0, 64,
                       32))
        return kCuda;
    return launch(xp, kXentTable, bf16, shape, dev, s);
}

int launch(XentParams& xp, int mode, bool bf16, const XentShape& shape, const DeviceInfo& dev,
           cudaStream_t s) {
    const int64_t units = (int64_t)xp.tiles_m * xp.tiles_n * (mode == kXentSum ? xp.splits : 1);
    if (units * 2 > INT32_MAX) return kUnsupported;
    xp.stages = stages_of(xp, mode);
    const int rc = bf16 ? launch_xent_bf16(xp, mode, shape.cta_group, dev, s)
                        : launch_xent_f16(xp, mode, shape.cta_group, dev, s);
    dispatch_log("cross entropy %s %dx%d, %d k-blocks: %s, %d x %d tiles of %d columns",
                 mode == kXentStats   ? "logits"
                 : mode == kXentSum   ? "dX"
                 : mode == kXentTable ? "dW"
                                      : "gradient's logits",
                 xp.M, xp.N, xp.num_kb,
                 shape.cta_group == 2 ? "CTA pairs" : "one CTA per tile", xp.tiles_m, xp.tiles_n,
                 xp.tile_n);
    return rc;
}

int forward(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const void* W,
            int64_t ldw, const int32_t* target, float* loss, float* lse, int dtype,
            cudaStream_t s) {
    int rc = check_inputs(M, N, K, X, ldx, W, ldw, target, dtype);
    if (rc != kOk || M == 0) return rc;
    if (!loss || !aligned_to(loss, 4) || !aligned_to(lse, 4)) return kInvalidArg;
    if (M > kXentMaxRows) return kUnsupported;
    DeviceInfo* dev = nullptr;
    cudaMemPool_t pool = nullptr;
    rc = current_device_info(&dev, &pool);
    if (rc != kOk) return rc;
    const void* ptrs[5] = {K > 0 ? X : nullptr, K > 0 ? W : nullptr, target, loss, lse};
    rc = check_device_pointers(ptrs, 5, dev->device);
    if (rc != kOk) return rc;
    if (K == 0) {
        const int64_t blocks = (M + 255) / 256;
        xent_uniform_kernel<<<(unsigned)(blocks < dev->sm_count ? blocks : dev->sm_count), 256, 0,
                              s>>>((int)M, (int)N, target, loss, lse, dev->err_word);
        if (cudaGetLastError() != cudaSuccess) return kCuda;
        note_launch();
        return kOk;
    }
    const bool bf16 = is_bf16(dtype);
    const XentShape shape = plan_xent(M, N, dev->sm_count, true);
    const int64_t panel = xent_panel_rows(M, N, shape.tile_n);
    const int64_t parts = (N + shape.tile_n - 1) / shape.tile_n * 2;
    Parts at;
    const int64_t part_at = at.add(parts * up(panel, 32) * 8);
    const int64_t picked_at = at.add(panel * 4);
    const int64_t x_at = tma_ready(X, ldx) ? -1 : at.add(M * up(K, 8) * 2);
    const int64_t w_at = tma_ready(W, ldw) ? -1 : at.add(N * up(K, 8) * 2);
    Scratch scratch{pool, s, dev->device};
    char* mem = static_cast<char*>(scratch.get((size_t)at.bytes));
    if (!mem) return kCuda;
    if (x_at >= 0) rc = repack_one(X, ldx, M, K, mem + x_at, *dev, s);
    if (rc == kOk && w_at >= 0) rc = repack_one(W, ldw, N, K, mem + w_at, *dev, s);
    for (int64_t r0 = 0; r0 < M && rc == kOk; r0 += panel) {
        const int64_t m = M - r0 < panel ? M - r0 : panel;
        XentParams xp;
        xent_params(xp, m, N, K, shape, N, target + r0, *dev);
        if (!xent_maps(xp, bf16, static_cast<const uint16_t*>(X) + r0 * ldx, ldx, W, ldw, K,
                       shape)) {
            rc = kCuda;
            break;
        }
        xp.part = reinterpret_cast<float2*>(mem + part_at);
        xp.part_ld = up(panel, 32);
        xp.picked = reinterpret_cast<float*>(mem + picked_at);
        rc = launch(xp, kXentStats, bf16, shape, *dev, s);
        if (rc != kOk) break;
        // few rows: more threads for each
        const int rows = m <= 4 * dev->sm_count ? 2 : m <= 24 * dev->sm_count ? 8 : 32;
        auto join = [&](auto kern) {
            return launch_dependent(kern, dim3((unsigned)((m + rows - 1) / rows)),
                                    dim3(kJoinThreads), 0, s, (const float2*)xp.part, xp.part_ld,
                                    (int)parts, (int)m, (const float*)xp.picked, target + r0,
                                    (int)N, loss + r0, lse ? lse + r0 : nullptr);
        };
        rc = rows == 2 ? join(xent_join_kernel<2>)
                       : rows == 8 ? join(xent_join_kernel<8>) : join(xent_join_kernel<32>);
    }
    scratch.release();
    return rc;
}

// dW = beta dW + *scale G^T X on the product over the rows of one group, {0, depth}
// in `limits`: it adds up fp32 sums in parts of the depth (the tensor core's cut-off
// additions would show in an fp32 dW), and takes the factor from device memory.
int product_rows(int64_t M, int64_t N, int64_t depth, const void* A, int64_t lda, const void* B,
                 int64_t ldb, void* C, int64_t ldc, int dtype, float beta, const float* scale,
                 const int32_t* limits, cudaStream_t s) {
    return launch_grouped_k(1, M, N, depth, limits, A, lda, B, ldb, C, ldc, M * ldc, dtype, beta,
                            scale, s);
}

int backward(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const void* W,
             int64_t ldw, const int32_t* target, const float* lse, const float* dloss, void* dX,
             int64_t lddx, void* dW, int64_t lddw, float alpha, float beta, int dtype,
             cudaStream_t s) {
    int rc = check_inputs(M, N, K, X, ldx, W, ldw, target, dtype);
    if (rc != kOk) return rc;
    if (K > kXentMaxDepth) return kUnsupported;
    const int we = dtype <= GEMM_BF16_F32 ? 4 : 2;
    if (!aligned_to(dX, 2) || !aligned_to(dW, we)) return kInvalidArg;
    if (K > 0 && ((dX && M > 0 && lddx < K) || (dW && lddw < K))) return kInvalidArg;
    if ((dX && !span_fits(M, K, lddx, 2)) || (dW && !span_fits(N, K, lddw, we)))
        return kInvalidArg;
    if (M > 0 && K > 0 && (dX || dW) &&
        (!lse || !aligned_to(lse, 4) || !aligned_to(dloss, 4)))
        return kInvalidArg;
    if (M > kXentMaxRows) return kUnsupported;
    if (K == 0 || (!dX && !dW) || (M == 0 && !dW)) return kOk;
    DeviceInfo* dev = nullptr;
    cudaMemPool_t pool = nullptr;
    rc = current_device_info(&dev, &pool);
    if (rc != kOk) return rc;
    const bool bf16 = is_bf16(dtype);
    if (M == 0) {  // no rows: dW = beta dW
        rc = check_device_pointers(&dW, 1, dev->device);
        if (rc != kOk) return rc;
        Problem p{N, K, 0, nullptr, 0, true, nullptr, 0, true, dW, lddw, dtype,
                  EpiParams{1, 1.f, beta, nullptr, 0, GEMM_ACT_NONE}};
        return launch_epilogue_only(p, *dev, s);
    }
    const void* ptrs[7] = {X, W, target, lse, dloss, dX, dW};
    rc = check_device_pointers(ptrs, 7, dev->device);
    if (rc != kOk) return rc;

    const int parts = dW && we == 4 ? 2 : 1;  // numbers that hold an entry of G
    const int64_t piece = xent_piece_cols(up(M, 256), N);
    const XentShape shape = plan_xent(M, piece, dev->sm_count, false);  // of every piece
    const int rows = (int)up(M, XROWS * shape.cta_group);        // that the tiles cover
    const int64_t pieces = (N + piece - 1) / piece;
    // dX: in shares of the depth where its tiles are few
    const XentSumPlan plan = plan_xent_sum(M, K, piece, dev->sm_count);
    const int64_t ldg = up(piece, 256), ldk = up(K, 8);
    Parts at;
    const int64_t g_at = at.add(ldg * rows * parts * 2);
    const int64_t x_at = at.add(ldk * rows * parts * 2);
    const int64_t w_at = tma_ready(W, ldw) ? -1 : at.add(N * ldk * 2);
    const int64_t dx_at = dX ? at.add(plan.splits * M * up(K, 4) * 4) : -1;
    const int64_t order_at = at.add(M * 4), place_at = at.add(M * 4);
    const int64_t scale_at = at.add(8), info_at = at.add(sizeof(XentInfo));
    Scratch scratch{pool, s, dev->device};
    char* mem = static_cast<char*>(scratch.get((size_t)at.bytes));
    if (!mem) return kCuda;
    float* dx_sum = dX ? reinterpret_cast<float*>(mem + dx_at) : nullptr;
    int32_t* order = reinterpret_cast<int32_t*>(mem + order_at);
    int32_t* place = reinterpret_cast<int32_t*>(mem + place_at);
    float* scale = reinterpret_cast<float*>(mem + scale_at);
    XentInfo* info = reinterpret_cast<XentInfo*>(mem + info_at);
    char *g = mem + g_at, *xc = mem + x_at;

    rc = launch_dependent(xent_order_kernel, dim3(1), dim3(1024), 0, s, (int)M, target, (int)N,
                          dloss, alpha, bf16 ? 1.f : 4096.f, XROWS * shape.cta_group, parts, order,
                          place, info, scale, dev->err_word);
    if (rc == kOk) {
        const int64_t blocks = ((int64_t)rows * parts + 7) / 8, most = dev->sm_count * 8;
        rc = launch_dependent(xent_rows_kernel, dim3((unsigned)(blocks < most ? blocks : most)),
                              dim3(256), 0, s, static_cast<const uint16_t*>(X), ldx, K,
                              (const int32_t*)order, (const XentInfo*)info,
                              reinterpret_cast<uint16_t*>(xc), ldk, parts);
    }
    if (rc == kOk && w_at >= 0) rc = repack_one(W, ldw, N, K, mem + w_at, *dev, s);
    for (int64_t v0 = 0; v0 < N && rc == kOk; v0 += piece) {
        const int64_t n = N - v0 < piece ? N - v0 : piece;
        const void* wp = static_cast<const uint16_t*>(W) + v0 * ldw;
        XentParams xp;
        xent_params(xp, M, n, K, shape, N, target, *dev);
        xp.col0 = (int)v0;
        xp.order = order;
        xp.info = info;
        xp.lse = lse;
        xp.dloss = dloss;
        xp.alpha = alpha;
        xp.scale = scale;
        if (!xent_maps(xp, bf16, xc, ldk, wp, ldw, K, shape) ||
            !encode_tma_16(&xp.map_g, bf16, g, (uint64_t)ldg, (uint64_t)rows * parts,
                           (uint64_t)ldg, 0, 0, 64, 32)) {
            rc = kCuda;
            break;
        }
        rc = launch(xp, parts == 2 ? kXentGrad2 : kXentGrad, bf16, shape, *dev, s);
        if (rc == kOk && dX)
            rc = launch_sum(plan, M, K, piece, n, g, ldg, wp, ldw, dx_sum, M, v0 > 0, info, bf16,
                            *dev, s);
        if (rc != kOk || !dW) continue;
        void* dst = static_cast<char*>(dW) + v0 * lddw * we;
        rc = we == 2 && beta == 0.f && tma_ready(dW, lddw) && K % 8 == 0 && rows <= kXentTableRows
                 ? launch_table(n, K, rows, g, ldg, xc, ldk, dst, lddw, scale + 1, info, bf16,
                                *dev, s)
                 : product_rows(n, K, (int64_t)rows * parts, g, ldg, xc, ldk, dst, lddw, dtype,
                                beta, scale + 1, info->limits, s);
    }
    if (rc == kOk && dX)
        rc = finish(dx_sum, up(K, 4), plan.used(piece), M, dX, lddx, M, K, place, scale + 1, bf16,
                    *dev, s);
    scratch.release();
    return rc;
}

}  // namespace
}  // namespace libgemm

using namespace libgemm;

extern "C" {

int gemm_xent(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const void* W,
              int64_t ldw, const int32_t* target, float* loss, float* lse, int dtype,
              void* stream) {
    try {
        return forward(M, N, K, X, ldx, W, ldw, target, loss, lse, dtype,
                       static_cast<cudaStream_t>(stream));
    } catch (...) {
        return kCuda;
    }
}

int gemm_xent_grad(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const void* W,
                   int64_t ldw, const int32_t* target, const float* lse, const float* dloss,
                   void* dX, int64_t lddx, void* dW, int64_t lddw, float alpha, float beta,
                   int dtype, void* stream) {
    try {
        return backward(M, N, K, X, ldx, W, ldw, target, lse, dloss, dX, lddx, dW, lddw, alpha,
                        beta, dtype, static_cast<cudaStream_t>(stream));
    } catch (...) {
        return kCuda;
    }
}

}  // extern "C"
