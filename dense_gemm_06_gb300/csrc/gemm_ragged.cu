// gemm_ragged.cu -- gemm_grouped(), gemm_grouped_k() and gemm_lora(): products
// whose row groups are known on the device only, on the tcgen05 kernel of
// gemm_ragged.cuh.
//
// Mathematics. With t a row (a token), n a feature, and everything accumulated
// in fp32:
//
//   rows   C[t][n]   = sum_k A[t][k] B_g[n][k]           offsets[g] <= t < offsets[g+1]
//   depth  C_g[m][n] = sum_{t in group g} A[t][m] B[t][n]
//   lora   C[t][n]   = sum_k A[t][k] B[n][k] + sum_r T[t][r] LB_a[r][n],
//          T[t][r]   = scale_a sum_k A[t][k] LA_a[r][k],   a = adapter[t]
//
// Design, with the reasons:
//
//   * Units of work are found on the device: a warp per CTA (or pair) walks the
//     group limits (RowWalk: 128 groups per warp step) and passes the units to
//     the other roles through shared memory, so a call needs no host copy of the
//     limits and can be captured in a graph. (Each role walking by itself put
//     the walk, up to 1.4 us, before every unit's first MMA: 363 us against
//     339 us for 64 groups, 49152 rows, 2816 x 2048.)
//   * The weights are the MMA's M side and the rows its N side. A unit is as
//     wide as its group has rows (in steps of 16, 32 for a CTA pair), so a
//     ragged group wastes at most one step instead of most of a 128-row tile,
//     and a decode step's few rows cost few tensor cycles and little shared
//     memory traffic beside the weights it streams.
//   * depth: a small launch first writes each group's tensor maps, cut off at its
//     last row (TMA then fills the last block with zeros), and the order of the
//     groups, longest first; pairs take the units by counting. 64 gradients of
//     2816 x 2048 over 49152 uneven rows: 573 us with a fixed walk in the given
//     order, 478 us so. They are bound by the SMs' memory port: operands (32 KB
//     per CTA and k-block) and 128 KB of fp32 results per unit share it; without
//     the stores the same call takes 349 us, with them to a small region that
//     stays in L2 460 us.
//   * lora: the adapters ride in the same accumulator. A row tile's distinct
//     adapters are listed; the first launch (shrink) computes T of every row
//     against every listed adapter on the tensor cores and keeps the row's own
//     (zeros elsewhere), so that to the second launch (expand) T is just more
//     depth: k-blocks of T against the stacked LB of the list, after the
//     k-blocks of X against W. C is written once, W is read once, and rows of
//     any adapter order share the tile.
//   * T is carried as two 16-bit numbers, hi = rn(t) and lo = rn(t - hi), both
//     multiplied: one 16-bit T would add a rounding of the adapter's part as
//     large as C's own, two leave 2^-17 (bf16) or 2^-22 (fp16) of it; small T in
//     fp16, where the second runs out of exponents, takes two more (see T_SMALL
//     in gemm_ragged.cuh).
//   * For few rows the shrink is plain dot products (kRagShrinkRows).
//   * A zero of T against an infinite or NaN LB of another row's adapter would
//     be NaN. The shrink scans the listed LBs (bringing them into L2 for the
//     expand); a tile with such an adapter adds the adapters' part per row in
//     the epilogue instead.
//   * Few units (decoding): a cluster of 2, 4 or 8 CTAs shares each unit's
//     depth; partial sums go through distributed shared memory to the CTA that
//     owns the row and are added in rank order, so results do not depend on
//     timing.
//   * The expand is a programmatic dependent of the shrink: where it runs it
//     starts on X and W at once and waits for the shrink only before its first
//     block of T. It runs on an SM once the shrink's blocks there are done: its
//     CTA takes 226 KB of shared memory, and not even a block of dot products
//     (4 KB, 16384 registers) fits beside it. One token's shrink is 20 blocks, so
//     most of the expand overlaps it; 48 rows of rank 16 are 256 blocks, on every
//     SM, and the overlap is the shrink's last round.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "../../include/gemm.h"
#include "gemm_ragged.cuh"
#include "internal.h"
#include "policy.h"
#include "repack16.cuh"

namespace libgemm {
namespace {

int c_bytes(int dtype) { return dtype <= GEMM_BF16_F32 ? 4 : 2; }
bool is_bf16(int dtype) { return dtype == GEMM_BF16_F32 || dtype == GEMM_BF16_BF16; }
int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// (outer - 1) * ld + inner elements, `mats` times mat_stride apart, stay
// addressable.
bool span_fits(int64_t mats, int64_t mat_stride, int64_t outer, int64_t inner, int64_t ld,
               int esize) {
    if (mats <= 0 || outer <= 0 || inner <= 0) return true;
    const __int128 last = (__int128)(mats - 1) * mat_stride + (__int128)(outer - 1) * ld + inner;
    return last <= (__int128)(INT64_MAX / esize);
}

bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// One 16-bit operand: `mats` matrices (mat_stride apart) of `outer` rows of
// `inner` contiguous elements, ld apart.
struct Operand {
    const void* ptr;
    int64_t mats, mat_stride, outer, inner, ld;

    bool tma_ready() const {
        return aligned_to(ptr, 16) && ld % 8 == 0 && (mats <= 1 || mat_stride % 8 == 0);
    }
    int64_t packed_ld() const { return up(inner, 8); }
    int64_t packed_bytes() const { return up(mats * outer * packed_ld() * 2, 256); }
};

struct RepackMats {
    const uint16_t* src;
    uint16_t* dst;
    int64_t rows;  // of all matrices
    int64_t mat_stride, outer, ld, inner, ldd;
};
constexpr int kMaxRepacks = 4;
struct RepackJobs {
    RepackMats job[kMaxRepacks];
    int n;
};

// Copies operands whose rows TMA cannot read into 16-byte aligned rows, matrix
// after matrix, their padding zero; a warp per row, all operands in one launch.
__global__ void __launch_bounds__(256)
    repack16_mats_kernel(const __grid_constant__ RepackJobs jobs) {
    gemm_ptx::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x / 32);
    int64_t r = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
    for (int k = 0; k < jobs.n; ++k) {
        const RepackMats& j = jobs.job[k];
        for (; r < j.rows; r += warps) {
            const int64_t m = r / j.outer, o = r - m * j.outer;
            uint16_t* dst = j.dst + r * j.ldd;
            repack16_row(j.src + m * j.mat_stride + o * j.ld, dst, j.inner, lane);
            for (int64_t c = j.inner + lane; c < j.ldd; c += 32) dst[c] = 0;
        }
        r -= j.rows;
    }
}

// gemm_grouped_k: the two operands' tensor maps once per group, cut off at the
// group's last row, so that TMA fills its last block with zeros; the order of
// the groups, the longest first (for up to kMaxSorted groups: each warp ranks
// its group among all), so that the units handed out last are short ones; and
// the count of units taken. A warp per group. (Zeroing the block in shared
// memory instead put a hand-over of 1-2 us between the copy and the MMA of every
// unit: 64 groups of 769 rows took 536 us that way, 389 this way, 64 of 768,
// which need no zeros, 351.)
constexpr int kMapWarps = 4, kMaxSorted = 4096;
__global__ void __launch_bounds__(32 * kMapWarps)
    depth_maps_kernel(const __grid_constant__ CUtensorMap pm,
                      const __grid_constant__ CUtensorMap qm, const int32_t* offsets, int G,
                      int depth, CUtensorMap* out, int32_t* order, unsigned int* ticket) {
    gemm_ptx::pdl_launch_dependents();
    __shared__ __align__(128) uint32_t maps[kMapWarps][2][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = blockIdx.x * kMapWarps + w;
    if (g >= G) return;
    maps[w][0][lane] = reinterpret_cast<const uint32_t*>(&pm)[lane];
    maps[w][1][lane] = reinterpret_cast<const uint32_t*>(&qm)[lane];
    const int lo = clampi(offsets[g], 0, depth);
    const int hi = clampi(offsets[g + 1], lo, depth);
    if (g == 0 && lane == 0) *ticket = 0;
    int rank = 0;
    if (G <= kMaxSorted)
        for (int h = lane; h < G; h += 32) {
            const int a = clampi(offsets[h], 0, depth);
            const int n = clampi(offsets[h + 1], a, depth) - a;
            rank += n > hi - lo || (n == hi - lo && h < g);
        }
    rank = __reduce_add_sync(0xffffffffu, rank);
    if (lane == 0) order[G <= kMaxSorted ? rank : g] = g;
    if (depth == 0) return;  // no maps, and no use of them
    __syncwarp();
    for (int i = 0; i < 2; ++i) {
        const uint32_t at = gemm_ptx::smem_u32(&maps[w][i][0]);
        if (lane == 0) gemm_ptx::tma_desc_set_rows(at, (uint32_t)(hi > 0 ? hi : 1));
        __syncwarp();
        gemm_ptx::tma_desc_publish(out + 2 * (int64_t)g + i, at);
    }
}

// Scratch of the copies of those operands that are not TMA-ready.
int64_t repack_bytes(Operand* const* ops, int n) {
    int64_t bytes = 0;
    for (int i = 0; i < n; ++i)
        if (!ops[i]->tma_ready()) bytes += ops[i]->packed_bytes();
    return bytes;
}

// Replaces the operands that are not TMA-ready by their copies at `at`.
int repack(Operand* const* ops, int n, char* at, const DeviceInfo& dev, cudaStream_t s) {
    RepackJobs jobs{};
    int64_t rows = 0;
    for (int i = 0; i < n; ++i) {
        Operand& o = *ops[i];
        if (o.tma_ready()) continue;
        RepackMats& j = jobs.job[jobs.n++];
        j = {static_cast<const uint16_t*>(o.ptr), reinterpret_cast<uint16_t*>(at),
             o.mats * o.outer, o.mat_stride, o.outer, o.ld, o.inner, o.packed_ld()};
        at += o.packed_bytes();
        rows += j.rows;
        o.ptr = j.dst;
        o.ld = j.ldd;
        o.mat_stride = o.outer * j.ldd;
    }
    if (jobs.n == 0) return kOk;
    repack16_mats_kernel<<<repack16_blocks(rows, dev.sm_count), 256, 0, s>>>(jobs);
    if (cudaGetLastError() != cudaSuccess) return kCuda;
    note_launch();
    dispatch_log("repack of %d misaligned 16-bit operands, %lld rows", jobs.n, (long long)rows);
    return kOk;
}

bool map_2d(RaggedParams& rp, int i, bool bf16, const Operand& o, uint32_t box_outer) {
    return encode_tma_16(&rp.map[i], bf16, o.ptr, (uint64_t)o.inner, (uint64_t)o.outer,
                         (uint64_t)o.ld, 0, 0, 64, box_outer);
}
bool map_3d(RaggedParams& rp, int i, bool bf16, const Operand& o, uint32_t box_outer) {
    // one matrix: its stride is never used, but has to be a valid one
    const int64_t stride = o.mats > 1 ? o.mat_stride : up(o.outer * o.ld, 8);
    return encode_tma_16(&rp.map[i], bf16, o.ptr, (uint64_t)o.inner, (uint64_t)o.outer,
                         (uint64_t)o.ld, (uint64_t)o.mats, (uint64_t)stride, 64, box_outer);
}

// A 16-bit C by TMA where its rows (and matrices) are 16-byte aligned: a box is
// one staging tile, 32 features by 32 rows.
void map_c(RaggedParams& rp, int dtype, void* C, int64_t mats, int64_t stride, int64_t rows,
           int64_t cols, int64_t ld) {
    if (c_bytes(dtype) != 2 || !aligned_to(C, 16) || ld % 8 ||
        (mats > 1 && stride % 8))
        return;
    rp.c_tma = encode_tma_c16(&rp.map[kMapC], is_bf16(dtype), C, (uint64_t)cols, (uint64_t)rows,
                              (uint64_t)ld, (uint64_t)mats,
                              (uint64_t)(mats == 1 ? rows * ld : stride), 32, 32)
                   ? 1 : 0;
}

void common_params(RaggedParams& rp, const DeviceInfo& dev) {
    rp.pdl = 1;
    rp.err = dev.err_word;
    rp.check = dev.check_word;
    rp.gen = next_generation();
    rp.wait_limit_ns = option_wait_limit_ns();
    rp.fault_inject = option_tc_fault_inject();
    rp.split = 0;
    rp.chains = 1;
    rp.lanes = 128;
    rp.slot = 16;
    rp.list_w = 128;
#ifdef LIBGEMM_TC_TRACE
    rp.trace = trace_buffer();
    rp.trace_ctas = kTraceCtas;
#endif
}

int launch(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units, int dtype,
           const DeviceInfo& dev, cudaStream_t s) {
    switch (dtype) {
        case GEMM_F16_F32: return launch_ragged_f16_f32(rp, mode, cg, p_mn, units, dev, s);
        case GEMM_BF16_F32: return launch_ragged_bf16_f32(rp, mode, cg, p_mn, units, dev, s);
        case GEMM_F16_F16: return launch_ragged_f16_f16(rp, mode, cg, p_mn, units, dev, s);
        case GEMM_BF16_BF16: return launch_ragged_bf16_bf16(rp, mode, cg, p_mn, units, dev, s);
        default: return kInvalidArg;
    }
}

int log2_of(int x) {
    int n = 0;
    while (x > 1) x /= 2, ++n;
    return n;
}

int check_epilogue(const gemm_epilogue* e, int dtype) {
    if (!e) return kOk;
    if (e->activation < GEMM_ACT_NONE || e->activation > GEMM_ACT_GELU) return kInvalidArg;
    if (e->bias && !aligned_to(e->bias, c_bytes(dtype))) return kInvalidArg;
    return kOk;
}

EpiParams epi_params(const gemm_epilogue* e) {
    if (!e || (e->alpha == 1.f && e->beta == 0.f && !e->bias && e->activation == GEMM_ACT_NONE))
        return EpiParams{0, 1.f, 0.f, nullptr, 0, 0};
    return EpiParams{1, e->alpha, e->beta, e->bias, 0, e->activation};
}

RaggedOut ragged_out(const EpiParams& e, int dtype) {
    const bool reads = e.active && e.beta != 0.f;
    if (c_bytes(dtype) == 2) return reads ? kOut16Reads : kOut16;
    if (!e.active) return kOut32;
    return reads && !adds(e) ? kOut32Reads : kOut32Epilogue;
}

bool sizes_ok(int64_t a, int64_t b, int64_t c, int64_t d) {
    for (int64_t x : {a, b, c, d})
        if (x < 0 || x > INT32_MAX) return false;
    return true;
}

// The units (and with a pair or a cluster, the CTAs) fit the kernels' ints.
bool units_fit(int64_t units, int ctas) { return units <= INT32_MAX / (ctas < 2 ? 2 : ctas); }

int grouped(int64_t G, int64_t M, int64_t N, int64_t K, const int32_t* offsets, const void* A,
            int64_t lda, const void* B, int64_t ldb, int64_t strideb, int b_major, void* C,
            int64_t ldc, int dtype, const gemm_epilogue* epi, cudaStream_t s) {
    if (dtype == GEMM_F32) return kUnsupported;
    if (dtype < GEMM_F32 || dtype > GEMM_BF16_BF16 || (b_major != 0 && b_major != 1))
        return kInvalidArg;
    if (!sizes_ok(G, M, N, K)) return kInvalidArg;
    int rc = check_epilogue(epi, dtype);
    if (rc != kOk) return rc;
    if (G == 0 || M == 0 || N == 0) return kOk;
    const int oe = c_bytes(dtype);
    if (!offsets || !aligned_to(offsets, 4)) return kInvalidArg;
    if (!C || ldc < N || !aligned_to(C, oe) || !span_fits(1, 0, M, N, ldc, oe)) return kInvalidArg;
    const bool kmaj = b_major == GEMM_MAJOR_K;
    Operand a{A, 1, 0, M, K, lda};
    Operand b{B, G, strideb, kmaj ? N : K, kmaj ? K : N, ldb};
    if (K > 0) {
        if (!A || !B || !aligned_to(A, 2) || !aligned_to(B, 2)) return kInvalidArg;
        if (lda < a.inner || ldb < b.inner) return kInvalidArg;
        if (!span_fits(1, 0, a.outer, a.inner, lda, 2)) return kInvalidArg;
        if (!span_fits(1, 0, b.outer, b.inner, ldb, 2)) return kInvalidArg;  // so the next sum fits
        if (G > 1 && strideb < (b.outer - 1) * ldb + b.inner) return kInvalidArg;
        if (!span_fits(G, strideb, b.outer, b.inner, ldb, 2)) return kInvalidArg;
    }
    DeviceInfo* dev = nullptr;
    cudaMemPool_t pool = nullptr;
    rc = current_device_info(&dev, &pool);
    if (rc != kOk) return rc;
    const void* ptrs[5] = {K > 0 ? A : nullptr, K > 0 ? B : nullptr, C, offsets,
                           epi ? epi->bias : nullptr};
    rc = check_device_pointers(ptrs, 5, dev->device);
    if (rc != kOk) return rc;

    const int64_t num_kb = (K + BK - 1) / BK;
    const EpiParams ep = epi_params(epi);
    const RaggedShape shape =
        plan_grouped(G, M, N, num_kb, dev->sm_count, ragged_out(ep, dtype));
    const bool bf16 = is_bf16(dtype);
    RaggedParams rp;
    std::memset(&rp, 0, sizeof(rp));
    common_params(rp, *dev);
    rp.offsets = offsets;
    rp.G = (int)G;
    rp.rows = (int)M;
    rp.feats = (int)N;
    rp.num_kb = (int)num_kb;
    rp.tile_w = shape.tile_w;
    rp.tiles_f = (int)((N + 128 * shape.cta_group - 1) / (128 * shape.cta_group));
    rp.split = log2_of(shape.split);
    rp.C = C;
    rp.ldc = ldc;
    rp.epi = ep;
    map_c(rp, dtype, C, 0, 0, M, N, ldc);
    const int64_t units = ((G < M ? G : M) + M / shape.tile_w) * rp.tiles_f;
    if (!units_fit(units, shape.cta_group * shape.split)) return kUnsupported;

    Scratch scratch{pool, s, dev->device};
    Operand* const ops[2] = {&a, &b};
    const int64_t ticket_bytes =
        plan_grouped_ticket(shape, M, N, num_kb, dev->sm_count) ? 256 : 0;
    const int64_t bytes = ticket_bytes + (K > 0 ? repack_bytes(ops, 2) : 0);
    char* at = nullptr;
    if (bytes > 0 && !(at = static_cast<char*>(scratch.get((size_t)bytes)))) return kCuda;
    if (ticket_bytes > 0) {
        rp.ticket = reinterpret_cast<unsigned int*>(at);
        if (cudaMemsetAsync(rp.ticket, 0, sizeof(unsigned int), s) != cudaSuccess) {
            cudaGetLastError();
            rc = kCuda;
        }
    }
    if (K > 0 && rc == kOk) {
        rc = repack(ops, 2, at + ticket_bytes, *dev, s);
        if (rc == kOk &&
            !(map_3d(rp, kMapP, bf16, b, kmaj ? 128 : BK) &&
              map_2d(rp, kMapQ, bf16, a, (uint32_t)(shape.tile_w / shape.cta_group)) &&
              map_2d(rp, kMapQ16, bf16, a, 16)))
            rc = kCuda;
    }
    if (rc == kOk) rc = launch(rp, kRagRows, shape.cta_group, !kmaj, units, dtype, *dev, s);
    scratch.release();
    if (rc == kOk)
        dispatch_log("grouped %lld groups, %lldx%lldx%lld: %s, units up to %d rows, split %d",
                     (long long)G, (long long)M, (long long)N, (long long)K,
                     shape.cta_group == 2 ? "CTA pairs" : "one CTA per unit", shape.tile_w,
                     shape.split);
    return rc;
}

int grouped_k(int64_t G, int64_t M, int64_t N, int64_t K, const int32_t* offsets, const void* A,
              int64_t lda, const void* B, int64_t ldb, void* C, int64_t ldc, int64_t stridec,
              int dtype, const gemm_epilogue* epi, cudaStream_t s) {
    if (dtype == GEMM_F32) return kUnsupported;
    if (dtype < GEMM_F32 || dtype > GEMM_BF16_BF16) return kInvalidArg;
    if (!sizes_ok(G, M, N, K)) return kInvalidArg;
    int rc = check_epilogue(epi, dtype);
    if (rc != kOk) return rc;
    if (G == 0 || M == 0 || N == 0) return kOk;
    const int oe = c_bytes(dtype);
    if (!offsets || !aligned_to(offsets, 4)) return kInvalidArg;
    if (!C || ldc < N || !aligned_to(C, oe)) return kInvalidArg;
    if (!span_fits(1, 0, M, N, ldc, oe)) return kInvalidArg;
    if (G > 1 && stridec < (M - 1) * ldc + N) return kInvalidArg;
    if (!span_fits(G, stridec, M, N, ldc, oe)) return kInvalidArg;
    Operand a{A, 1, 0, K, M, lda}, b{B, 1, 0, K, N, ldb};
    if (K > 0) {
        if (!A || !B || !aligned_to(A, 2) || !aligned_to(B, 2)) return kInvalidArg;
        if (lda < M || ldb < N) return kInvalidArg;
        if (!span_fits(1, 0, K, M, lda, 2) || !span_fits(1, 0, K, N, ldb, 2)) return kInvalidArg;
    }
    DeviceInfo* dev = nullptr;
    cudaMemPool_t pool = nullptr;
    rc = current_device_info(&dev, &pool);
    if (rc != kOk) return rc;
    const void* ptrs[5] = {K > 0 ? A : nullptr, K > 0 ? B : nullptr, C, offsets,
                           epi ? epi->bias : nullptr};
    rc = check_device_pointers(ptrs, 5, dev->device);
    if (rc != kOk) return rc;

    const EpiParams ep = epi_params(epi);
    const RaggedShape shape =
        plan_grouped_k(G, M, N, dev->sm_count, ragged_out(ep, dtype), K / G);
    const bool bf16 = is_bf16(dtype);
    RaggedParams rp;
    std::memset(&rp, 0, sizeof(rp));
    common_params(rp, *dev);
    rp.offsets = offsets;
    rp.G = (int)G;
    rp.rows = (int)M;
    rp.feats = (int)N;
    rp.depth = (int)K;
    rp.tile_w = shape.tile_w;
    rp.tiles_f = (int)((N + 128 * shape.cta_group - 1) / (128 * shape.cta_group));
    rp.tiles_r = (int)((M + shape.tile_w - 1) / shape.tile_w);
    rp.split = log2_of(shape.split);
    rp.C = C;
    rp.ldc = ldc;
    rp.stridec = stridec;
    rp.epi = ep;
    map_c(rp, dtype, C, G, stridec, M, N, ldc);
    const int64_t units = G * rp.tiles_f * rp.tiles_r;
    if ((int64_t)rp.tiles_f * rp.tiles_r > INT32_MAX / G ||
        !units_fit(units, shape.cta_group * shape.split))
        return kUnsupported;

    Scratch scratch{pool, s, dev->device};
    Operand* const ops[2] = {&a, &b};
    const int64_t map_bytes = G * 2 * (int64_t)sizeof(CUtensorMap);
    const int64_t plan_bytes = up(map_bytes + (G + 1) * 4, 256);
    char* at = static_cast<char*>(
        scratch.get((size_t)(plan_bytes + (K > 0 ? repack_bytes(ops, 2) : 0))));
    if (!at) return kCuda;
    CUtensorMap* gmaps = reinterpret_cast<CUtensorMap*>(at);
    int32_t* order = reinterpret_cast<int32_t*>(at + map_bytes);
    unsigned int* ticket = reinterpret_cast<unsigned int*>(order + G);
    rp.gmaps = gmaps;
    rp.order = order;
    rp.ticket = ticket;
    if (K > 0) {
        rc = repack(ops, 2, at + plan_bytes, *dev, s);
        if (rc == kOk && !(map_2d(rp, kMapP, bf16, b, BK) && map_2d(rp, kMapQ, bf16, a, BK)))
            rc = kCuda;
    }
    if (rc == kOk) {
        depth_maps_kernel<<<(int)((G + kMapWarps - 1) / kMapWarps), 32 * kMapWarps, 0, s>>>(
            rp.map[kMapP], rp.map[kMapQ], offsets, (int)G, (int)K, gmaps, order, ticket);
        if (cudaGetLastError() != cudaSuccess) rc = kCuda;
        else note_launch();
    }
    if (rc == kOk) rc = launch(rp, kRagDepth, shape.cta_group, true, units, dtype, *dev, s);
    scratch.release();
    if (rc == kOk)
        dispatch_log("grouped depth, %lld groups, %lldx%lldx%lld: %s, units of %d rows",
                     (long long)G, (long long)M, (long long)N, (long long)K,
                     shape.cta_group == 2 ? "CTA pairs" : "one CTA per unit", shape.tile_w);
    return rc;
}

// Rows of gemm_lora computed at a time: as many as keep T within this.
constexpr int64_t kMaxTBytes = 512ll << 20;

int lora(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R, const void* A, int64_t lda,
         const void* B, int64_t ldb, int b_major, const int32_t* adapter, const void* lora_a,
         const void* lora_b, const float* scale, void* C, int64_t ldc, int dtype,
         const gemm_epilogue* epi, cudaStream_t s) {
    if (dtype == GEMM_F32 || dtype == GEMM_F16_F32 || dtype == GEMM_BF16_F32) return kUnsupported;
    if (dtype < GEMM_F32 || dtype > GEMM_BF16_BF16 || (b_major != 0 && b_major != 1))
        return kInvalidArg;
    if (!sizes_ok(M, N, K, L) || R < 0 || R > 128) return kInvalidArg;
    int rc = check_epilogue(epi, dtype);
    if (rc != kOk) return rc;
    if (M == 0 || N == 0) return kOk;
    const bool adapters = K > 0 && L > 0 && R > 0;
    const bool kmaj = b_major == GEMM_MAJOR_K;
    Operand x{A, 1, 0, M, K, lda};
    Operand w{B, 1, 0, kmaj ? N : K, kmaj ? K : N, ldb};
    Operand la{lora_a, L, R * K, R, K, K}, lb{lora_b, L, R * N, R, N, N};
    if (!C || ldc < N || !aligned_to(C, 2) || !span_fits(1, 0, M, N, ldc, 2)) return kInvalidArg;
    if (K > 0) {
        if (!A || !B || !aligned_to(A, 2) || !aligned_to(B, 2)) return kInvalidArg;
        if (lda < x.inner || ldb < w.inner) return kInvalidArg;
        if (!span_fits(1, 0, x.outer, x.inner, lda, 2) ||
            !span_fits(1, 0, w.outer, w.inner, ldb, 2))
            return kInvalidArg;
    }
    if (adapters) {
        if (!adapter || !lora_a || !lora_b || !aligned_to(adapter, 4) || !aligned_to(lora_a, 2) ||
            !aligned_to(lora_b, 2) || !aligned_to(scale, 4))
            return kInvalidArg;
        if (!span_fits(L, R * K, R, K, K, 2) || !span_fits(L, R * N, R, N, N, 2))
            return kInvalidArg;
    }
    DeviceInfo* dev = nullptr;
    cudaMemPool_t pool = nullptr;
    rc = current_device_info(&dev, &pool);
    if (rc != kOk) return rc;
    const void* ptrs[8] = {K > 0 ? A : nullptr, K > 0 ? B : nullptr, C, epi ? epi->bias : nullptr,
                           adapters ? adapter : nullptr, adapters ? lora_a : nullptr,
                           adapters ? lora_b : nullptr, adapters ? scale : nullptr};
    rc = check_device_pointers(ptrs, 8, dev->device);
    if (rc != kOk) return rc;
    if (!adapters)  // nothing to add to the shared product
        return gemm_ex(M, N, K, A, lda, GEMM_MAJOR_K, B, ldb, b_major, C, ldc, GEMM_MAJOR_MN,
                       dtype, epi, s);

    const bool bf16 = is_bf16(dtype);
    const int64_t num_kb = (K + BK - 1) / BK;
    const int slot = R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128;
    // The list of a row tile holds at most as many adapters as the tile has
    // rows; the tile is 256 rows wide at most.
    const int64_t most = M < 256 ? M : 256;
    const LoraShape shape =
        plan_lora(M, N, num_kb, L < most ? L : most, slot, dev->sm_count);
    const RaggedShape& ex = shape.expand;
    const int W = ex.tile_w;
    const int64_t list_n = L < (M < W ? M : W) ? L : (M < W ? M : W);
    const int64_t ldt =
        up(list_n * slot, EXT_K) / EXT_K * (bf16 ? T_BLOCK<__nv_bfloat16> : T_BLOCK<__half>);
    const int subs = W / shape.shrink_w;
    const int flags = shape.rows_blocks > 0
                          ? shape.scan_blocks + (bf16 ? 0 : shape.rows_blocks)
                          : subs * shape.chains * shape.shrink_split * EPI_WARPS;
    const int list_pitch = 1 + 2 * W + flags;

    // the kernels count the 16-byte groups of a list's LBs in 32 bits
    if (list_n * R * (lb.packed_ld() / 8) > INT32_MAX) return kUnsupported;

    // Row panels bound T; each is a whole number of tiles.
    int64_t panel = kMaxTBytes / (ldt * 2) / W * W;
    if (panel < W) panel = W;
    if (panel > M) panel = M;
    const int64_t t_bytes = up(panel * ldt * 2, 256);
    const int64_t list_bytes = up((panel + W - 1) / W * list_pitch * 4, 256);
    Operand* const ops[4] = {&x, &w, &la, &lb};
    const int64_t bytes = t_bytes + list_bytes + repack_bytes(ops, 4);
    Scratch scratch{pool, s, dev->device};
    char* at = static_cast<char*>(scratch.get((size_t)bytes));
    if (!at) return kCuda;
    void* T = at;
    at += t_bytes;
    int32_t* lists = reinterpret_cast<int32_t*>(at);
    at += list_bytes;
    rc = repack(ops, 4, at, *dev, s);

    for (int64_t m0 = 0; m0 < M && rc == kOk; m0 += panel) {
        const int64_t m = M - m0 < panel ? M - m0 : panel;
        Operand xp{static_cast<const uint16_t*>(x.ptr) + m0 * x.ld, 1, 0, m, K, x.ld};
        const Operand tp{T, 1, 0, m, ldt, ldt};
        RaggedParams rp;
        std::memset(&rp, 0, sizeof(rp));
        common_params(rp, *dev);
        rp.rows = (int)m;
        rp.feats = (int)N;
        rp.num_kb = (int)num_kb;
        rp.adapter = adapter + m0;
        rp.scale = scale;
        rp.x = xp.ptr;
        rp.ldx = xp.ld;
        rp.lora_a = la.ptr;
        rp.ldla = la.ld;
        rp.depth = (int)K;
        rp.lora_b = lb.ptr;
        rp.ldlb = lb.ld;
        rp.L = (int)L;
        rp.R = (int)R;
        rp.slot = slot;
        rp.list_w = W;
        rp.chains = shape.chains;
        rp.lists = lists;
        rp.list_pitch = list_pitch;
        rp.flags = flags;
        rp.T = T;
        rp.ldt = ldt;
        RaggedParams sh = rp;  // the shrink
        sh.lanes = shape.lanes;
        sh.tile_w = shape.shrink_w;
        sh.split = log2_of(shape.shrink_split);
#ifdef LIBGEMM_TC_TRACE
        rp.trace_ctas = sh.trace_ctas = kTraceCtas / 2;  // the buffer's lower and upper half
        if (sh.trace) sh.trace += 64 * (kTraceCtas / 2);
#endif
        const int64_t tiles = (m + W - 1) / W;
        const int64_t clusters = tiles * subs * shape.chains;
        rp.C = static_cast<uint16_t*>(C) + m0 * ldc;
        rp.ldc = ldc;
        rp.epi = epi_params(epi);
        map_c(rp, dtype, rp.C, 0, 0, m, N, ldc);
        rp.tile_w = W;
        rp.tiles_r = (int)tiles;
        rp.tiles_f = (int)((N + 128 * ex.cta_group - 1) / (128 * ex.cta_group));
        rp.split = log2_of(ex.split);
        const int64_t units = tiles * rp.tiles_f;
        if (!units_fit(units, ex.cta_group * ex.split) ||
            !units_fit(clusters, shape.shrink_split)) {
            rc = kUnsupported;
            break;
        }
        const uint32_t share = (uint32_t)(W / ex.cta_group);
        if (!(map_3d(sh, kMapP, bf16, la, (uint32_t)slot) &&
              map_2d(sh, kMapQ, bf16, xp, (uint32_t)sh.tile_w) &&
              map_2d(sh, kMapQ16, bf16, xp, 16) &&
              map_3d(rp, kMapP, bf16, w, kmaj ? 128 : BK) &&
              map_2d(rp, kMapQ, bf16, xp, share) && map_2d(rp, kMapQ16, bf16, xp, 16) &&
              map_3d(rp, kMapLB, bf16, lb, (uint32_t)(slot < EXT_K ? slot : EXT_K)) &&
              map_2d(rp, kMapT, bf16, tp, share) && map_2d(rp, kMapT16, bf16, tp, 16))) {
            rc = kCuda;
            break;
        }
        auto run = bf16 ? launch_lora_bf16 : launch_lora_f16;
        if (shape.rows_blocks > 0) {
            sh.chains = shape.rows_blocks;
            rc = run(sh, kRagShrinkRows, 1, false, shape.rows_blocks + shape.scan_blocks, *dev, s);
        } else {
            rc = run(sh, kRagShrink, 1, false, clusters, *dev, s);
        }
        if (rc == kOk) rc = run(rp, kRagLora, ex.cta_group, !kmaj, units, *dev, s);
    }
    scratch.release();
    if (rc == kOk)
        dispatch_log("lora %lldx%lldx%lld, %lld adapters of rank %lld: shrink %d blocks of dot "
                     "products or %d lanes x %d rows, %d chains, split %d; expand %s, units of "
                     "%d rows, split %d",
                     (long long)M, (long long)N, (long long)K, (long long)L, (long long)R,
                     shape.rows_blocks, shape.lanes, shape.shrink_w, shape.chains,
                     shape.shrink_split, ex.cta_group == 2 ? "CTA pairs" : "one CTA per unit", W,
                     ex.split);
    return rc;
}

}  // namespace
}  // namespace libgemm

using namespace libgemm;

extern "C" {

int gemm_grouped(int64_t G, int64_t M, int64_t N, int64_t K, const int32_t* offsets,
                 const void* A, int64_t lda, const void* B, int64_t ldb, int64_t strideb,
                 int b_major, void* C, int64_t ldc, int dtype, const gemm_epilogue* epi,
                 void* stream) {
    try {
        return grouped(G, M, N, K, offsets, A, lda, B, ldb, strideb, b_major, C, ldc, dtype, epi,
                       static_cast<cudaStream_t>(stream));
    } catch (...) {
        return kCuda;
    }
}

int gemm_grouped_k(int64_t G, int64_t M, int64_t N, int64_t K, const int32_t* offsets,
                   const void* A, int64_t lda, const void* B, int64_t ldb, void* C, int64_t ldc,
                   int64_t stridec, int dtype, const gemm_epilogue* epi, void* stream) {
    try {
        return grouped_k(G, M, N, K, offsets, A, lda, B, ldb, C, ldc, stridec, dtype, epi,
                         static_cast<cudaStream_t>(stream));
    } catch (...) {
        return kCuda;
    }
}

int gemm_lora(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R, const void* A, int64_t lda,
              const void* B, int64_t ldb, int b_major, const int32_t* adapter, const void* lora_a,
              const void* lora_b, const float* scale, void* C, int64_t ldc, int dtype,
              const gemm_epilogue* epi, void* stream) {
    try {
        return lora(M, N, K, L, R, A, lda, B, ldb, b_major, adapter, lora_a, lora_b, scale, C,
                    ldc, dtype, epi, static_cast<cudaStream_t>(stream));
    } catch (...) {
        return kCuda;
    }
}

}  // extern "C"
