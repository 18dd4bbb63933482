// xent.cuh -- the tcgen05 kernel of gemm_xent() and gemm_xent_grad(): tiles of
// the logits Z = X W^T that never leave the chip.
//
//   kStats  each tile's row maxima and sums of exp(z - maximum), and the
//           target's logit, taken from the accumulators as they are read;
//   kGrad   G = d (exp(z - lse) - [v = target]) rounded to 16 bits, for the
//           products dX = G W and dW = G^T X (16-bit results);
//   kGrad2  the same as two 16-bit numbers, hi = rn(g) and lo = rn(g - hi), for
//           an fp32 dW;
//   kSum    dX = G W in fp32; where its tiles are few, the depth (the piece's columns
//           of the vocabulary) is shared by several CTAs or pairs a tile, each of
//           which leaves a part (1531 rows of 1037 from 50001 columns: 220 us
//           with a CTA for each of 108 whole tiles, 100 us so);
//   kTable  a 16-bit dW = factor G^T X of few rows, the factor read from device
//           memory, stored by TMA from the boxes that G leaves through (32000 x 2048
//           of 300 rows: 111 us with the logits, 138 on gemm_grouped_k's kernel, whose
//           lanes store their own 2 bytes).
//
// The pipeline is the dense kernel's: warp 0 copies 64-deep blocks of X and W by
// TMA into a ring, warp 1 issues the MMAs (a CTA pair on 256 x 256 tiles, or one
// CTA on 128 rows by up to 128 columns) into one of two TMEM accumulators, and
// eight warps read the other one. A tile row is one TMEM lane, so one thread sees
// 64 columns of a row at a time: the softmax needs no exchange between threads,
// and per element one maximum, one fma, one ex2 and one addition.
//
// The tensor core cuts off what an addition shifts below its last bits, so a long
// sum of products drifts towards zero by half a step to a step for every 16 of depth:
// losses of K = 2048 were off by 6e-6 of themselves, dX from 131072 columns by 8e-4.
// So an accumulator takes at most kXentFold blocks of depth, and the epilogue warps
// add up those parts in registers, rounded to nearest (128 numbers a thread; the warps
// that only issue copies and MMAs hand over registers for them). With K = 2048 these
// take about 1,100 of the 8,192 cycles that a tile's MMAs take, and they run beside the
// next tile's MMAs: the tensor pipe bounds the kernel.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "internal.h"
#include "ptx_sm100.cuh"
#include "rows.cuh"

namespace libgemm {

enum XentMode { kXentStats = 0, kXentGrad = 1, kXentGrad2 = 2, kXentSum = 3, kXentTable = 4 };

// The rows of a gradient that count, found on the device.
struct XentInfo {
    int32_t limits[2];  // of dW's depth: 0, and the rows in use of all copies of X
    int32_t count;      // rows that count
    int32_t used;       // the same in whole tiles, one at least: the second copies of X
                        // and G begin there
};

struct XentParams {
    // kSum: X is G (rows of the piece's columns), W its rows of W read N-major, M x N
    // the rows and columns of dX, num_kb the blocks of one share of the depth.
    // kTable: X is G read M-major, W the rows of X read N-major, M x N the rows and
    // columns of the piece's dW, num_kb the blocks of rows.
    CUtensorMap map_x;   // M x K: boxes of 64 x 128 (one CTA a tile: x_rows) rows
    CUtensorMap map_w;   // the piece's N x K: boxes of 64 x (tile_n / CG) rows
    CUtensorMap map_g;   // kGrad, kGrad2: G, kTable: dW, boxes of 64 columns x 32 rows
    int M, N;            // rows, and columns of this piece of the vocabulary
    int num_kb;          // 64-deep blocks of K
    int part_kb;         // blocks whose sums one accumulator takes (see kXentFold)
    int tiles_m, tiles_n, tile_n;
    int x_rows;          // one CTA a tile: rows of X in a stage; the MMA reads on into what
                         // follows, which only rows past M see
    int stage_bytes, stages;  // one CTA a tile: the ring, as deep as its stages are small
    int band;            // tile rows of a raster band
    int col0;            // the piece's first vocabulary number
    int vocab;           // the whole vocabulary: targets at or past it do not count
    const int32_t* target;
    // All but kStats: only the rows that count take part, side by side. The kernel's row
    // j is row order[j] of the caller's; `info` says how many.
    const int32_t* order;
    const XentInfo* info;
    float2* part;        // kStats: (maximum, sum) of each row, half tile by half tile
    int64_t part_ld;     // rows of a half tile in `part`
    float* picked;       // kStats: each row's target logit
    float* sums;         // kSum: splits x sum_rows x sum_ld
    int64_t sum_ld, sum_rows;
    int splits, all_kb;  // shares of the depth, and the blocks of all of them
    int add;             // kSum: add to what `sums` holds
    const float* lse;
    const float* dloss;  // null: ones
    const float* scale;  // a factor on alpha, or null
    float alpha;
    ErrWord* err;
    ErrWord gen;
    unsigned long long wait_limit_ns;
    int fault_inject;    // test hook: 1 = the epilogue waits on a barrier that nothing completes
};

int launch_xent_f16(XentParams& xp, int mode, int cg, const DeviceInfo& dev, cudaStream_t s);
int launch_xent_bf16(XentParams& xp, int mode, int cg, const DeviceInfo& dev, cudaStream_t s);

namespace {

using namespace gemm_ptx;

constexpr int XBK = 64;            // depth of a stage: one 128-byte swizzled row
constexpr int XROWS = 128;         // rows of X in a CTA (TMEM lanes)
constexpr int XSTAGE = 2 * XROWS * XBK * 2;  // X and at most 128 rows of W: 32 KB
constexpr int kXentFold = 11;      // 704 of depth, as in the ragged products
constexpr int XEPI_WARP0 = 4, XEPI_WARPS = 8;
constexpr int XREGS = 168;         // of a thread at launch: 65536 / 384, in steps of 8
constexpr int XREGS_ISSUE = 56, XREGS_EPI = 224;
constexpr int XTHREADS = 32 * (XEPI_WARP0 + XEPI_WARPS);
static_assert(XEPI_WARP0 * XREGS_ISSUE + XEPI_WARPS * XREGS_EPI <=
                  (XEPI_WARP0 + XEPI_WARPS) * XREGS,
              "setmaxnreg hands out what the block was launched with");

template <int MODE> struct XentCfg {
    static constexpr int BOXES = MODE == kXentGrad2 ? 2 : 1;  // 64 x 32 boxes of G per warp
    static constexpr int STAGES = MODE == kXentGrad2 ? 5 : 6;
    static constexpr int RING = STAGES * XSTAGE;
    static constexpr int STAGING = XEPI_WARPS * BOXES * 32 * 128;
    static constexpr int MOST = 16;  // stages of one CTA's ring
    static constexpr int BARS = 2 * MOST + 6;
    static constexpr int SMEM = RING + STAGING + BARS * 8 + 16 + 1024;  // + alignment
    static_assert(SMEM <= 232448, "over the 227 KB of shared memory a CTA may use");
};

__device__ __noinline__ bool xent_wait_slow(uint32_t bar, uint32_t parity, ErrWord* err,
                                            ErrWord gen, unsigned long long limit) {
    const uint64_t t0 = globaltimer_ns();
    uint32_t n = 0;
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((++n & 31u) == 0) {
            if (gen_failed(err, gen)) return false;
            if (globaltimer_ns() - t0 > limit) {
                gen_record_timeout(err, gen);
                return false;
            }
        }
    }
}

// Bounded wait of a whole warp; the outcome is the same in every lane.
__device__ __forceinline__ bool xent_wait(uint32_t bar, uint32_t parity, const XentParams& p) {
    const bool ok = mbar_try_wait(bar, parity) ||
                    xent_wait_slow(bar, parity, p.err, p.gen, p.wait_limit_ns);
    return __all_sync(0xffffffffu, ok);
}

// The same without a call: the epilogue waits with 128 sums in its registers.
__device__ __forceinline__ bool xent_wait_inline(uint32_t bar, uint32_t parity,
                                                 const XentParams& p) {
    bool ok = mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        const uint64_t t0 = globaltimer_ns();
        uint32_t n = 0;
        while (!ok) {
            ok = mbar_try_wait(bar, parity);
            if (ok || (++n & 31u)) continue;
            if (gen_failed(p.err, p.gen)) break;
            if (globaltimer_ns() - t0 > p.wait_limit_ns) {
                gen_record_timeout(p.err, p.gen);
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool xent_elect() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void xent_sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z,
                                            uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(a), "r"(x), "r"(y), "r"(z),
                 "r"(w) : "memory");
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

template <bool BF16>
__device__ __forceinline__ float2 unpack16(uint32_t u) {
    if constexpr (BF16) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    } else {
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
    }
}

// All four warps of the issuing warp group call it.
__device__ __forceinline__ void give_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(XREGS_ISSUE));
}

constexpr float kLog2e = 1.4426950408889634f;

// Tiles in raster order: bands of `band` tile rows, column after column, every
// other band backwards, so that the tiles running at one time share X and W in L2.
__device__ __forceinline__ int2 xent_tile(int t, int tiles_m, const XentParams& p) {
    const int band_tiles = p.band * p.tiles_n;
    const int band = t / band_tiles;
    const int within = t - band * band_tiles;
    const int rows = min(p.band, tiles_m - band * p.band);
    int tn = within / rows;
    const int tm = band * p.band + (within - tn * rows);
    if (band & 1) tn = p.tiles_n - 1 - tn;
    return make_int2(tm, tn);
}

// What there is to do. All but kStats read it from the device: after pdl_wait().
struct XentWork {
    int tiles_m, tiles, total, num_kb;
};
template <int MODE, int CG>
__device__ __forceinline__ XentWork xent_work(const XentParams& p) {
    XentWork w{p.tiles_m, 0, 0, p.num_kb};
    if constexpr (MODE != kXentStats) {
        const int used = p.info->used;
        if constexpr (MODE == kXentTable) w.num_kb = used / XBK;
        else w.tiles_m = min(p.tiles_m, (used + XROWS * CG - 1) / (XROWS * CG));
    }
    w.tiles = w.tiles_m * p.tiles_n;
    w.total = MODE == kXentSum ? w.tiles * p.splits : w.tiles;
    return w;
}

template <int MODE, int CG, bool BF16>
__global__ void __launch_bounds__(XTHREADS, 1) xent_kernel(const __grid_constant__ XentParams p) {
    using C_ = XentCfg<MODE>;
    constexpr int MOST = C_::MOST;
    const int stages = CG == 2 ? C_::STAGES : p.stages;
    const int stage_bytes = CG == 2 ? XSTAGE : p.stage_bytes;
    const int x_bytes = CG == 2 ? XROWS * XBK * 2 : p.x_rows * XBK * 2;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // 128-byte swizzle atoms: 1024 bytes
    uint8_t* smem = smem_raw + (base - raw);
    const uint32_t staging0 = base + C_::RING;
    const uint32_t bar0 = staging0 + C_::STAGING;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (MOST + s); };
    auto accf_bar = [&](int a) { return bar0 + 8u * (2 * MOST + a); };
    auto acce_bar = [&](int a) { return bar0 + 8u * (2 * MOST + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * MOST + 4);
    const uint32_t never_bar = bar0 + 8u * (2 * MOST + 5);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C_::RING + C_::STAGING + 8 * C_::BARS);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const int cluster = CG == 2 ? (int)cluster_id_x() : (int)blockIdx.x;
    const int nclusters = CG == 2 ? (int)num_clusters_x() : (int)gridDim.x;
    constexpr int ACC_COLS = CG == 2 ? 256 : 128;  // TMEM columns of an accumulator
    // depth blocks of a unit (kSum: the last share may be shorter)
    auto blocks_of = [&](int split, const XentWork& w) {
        return MODE == kXentSum ? min(p.num_kb, p.all_kb - split * p.num_kb) : w.num_kb;
    };

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&p.map_x);
        tma_prefetch_desc(&p.map_w);
        for (int s = 0; s < stages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(accf_bar(a), 1);
            mbar_init(acce_bar(a), CG * XEPI_WARPS);
        }
        mbar_init(drain_bar, 1);
        mbar_init(never_bar, 1);
        fence_mbarrier_init_cluster();
    }
    if (warp == 1) {
        tmem_alloc<CG>(smem_u32(tmem_slot), 2 * ACC_COLS);
        tmem_relinquish<CG>();
    }
    tc_fence_before_sync();
    if constexpr (CG == 2) cluster_sync_all(); else __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
    bool aborted = false;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer --
        give_registers();
        pdl_wait();
        const XentWork work = xent_work<MODE, CG>(p);
        int stage = 0;
        uint32_t phase = 0;
        const int b_rows = p.tile_n / CG;
        const uint32_t bytes = (uint32_t)(CG * (x_bytes + b_rows * XBK * 2));
        for (int t = cluster; t < work.total && !aborted; t += nclusters) {
            const int split = MODE == kXentSum ? t / work.tiles : 0;
            const int2 tile = xent_tile(t - split * work.tiles, work.tiles_m, p);
            const int x_row = (tile.x * CG + (int)rank) * XROWS;
            const int w_row = tile.y * p.tile_n + (int)rank * b_rows;
            const int kb0 = split * p.num_kb, kbs = blocks_of(split, work);
            for (int kb = 0; kb < kbs; ++kb) {
                if (!xent_wait(empty_bar(stage), phase ^ 1u, p)) { aborted = true; break; }
                const uint32_t fb = CG == 2 ? mapa_shared(full_bar(stage), 0) : full_bar(stage);
                const uint32_t at = base + stage * stage_bytes;
                if (xent_elect()) {
                    if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), bytes);
                    if constexpr (MODE == kXentTable) {
                        for (int j = 0; j < XROWS / 64; ++j)  // boxes of 64 rows of dW
                            tma_load_2d<CG>(at + j * 64 * XBK * 2, &p.map_x, fb, x_row + 64 * j,
                                            kb * XBK);
                    } else {
                        tma_load_2d<CG>(at, &p.map_x, fb, (kb0 + kb) * XBK, x_row);
                    }
                    if constexpr (MODE == kXentSum || MODE == kXentTable) {
                        for (int j = 0; j < b_rows / 64; ++j)  // boxes of 64 columns
                            tma_load_2d<CG>(at + x_bytes + j * 64 * XBK * 2, &p.map_w, fb,
                                            w_row + 64 * j, (kb0 + kb) * XBK);
                    } else {
                        tma_load_2d<CG>(at + x_bytes, &p.map_w, fb, kb * XBK, w_row);
                    }
                }
                __syncwarp();
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
        }
        if (aborted) {  // let issued copies land
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 200000) {
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer --
        give_registers();
        if (rank == 0) {
            // the limit of the waits below begins when the kernel before this one on the
            // stream has ended, however long that takes beside this one's start
            pdl_wait();
            const XentWork work = xent_work<MODE, CG>(p);
            // X and W are K-major, 32 bytes a step of 16 deep, or (W of kSum, both of
            // kTable) M- or N-major, 16 rows of 128
            constexpr bool X_MN = MODE == kXentTable, W_MN = MODE == kXentSum || X_MN;
            constexpr uint64_t X_STEP = X_MN ? 16 * 128 >> 4 : 32 >> 4;
            constexpr uint64_t W_STEP = W_MN ? 16 * 128 >> 4 : 32 >> 4;
            const uint32_t idesc = make_idesc_f16(BF16, X_MN, W_MN, (uint32_t)(XROWS * CG),
                                                  (uint32_t)p.tile_n);
            const uint64_t x_desc0 = make_sdesc_sw128(base, X_MN ? 64 * XBK * 2 : 16, 1024);
            const uint64_t w_desc0 =
                make_sdesc_sw128(base + x_bytes, W_MN ? 64 * XBK * 2 : 16, 1024);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            for (int t = cluster; t < work.total && !aborted; t += nclusters) {
                const int kbs = blocks_of(MODE == kXentSum ? t / work.tiles : 0, work);
                for (int kb = 0; kb < kbs && !aborted;) {
                    if (!xent_wait(acce_bar(acc), acc_phase ^ 1u, p)) { aborted = true; break; }
                    tc_fence_after_sync();
                    const uint32_t d = tmem_base + (uint32_t)(acc * ACC_COLS);
                    const int end = min(kb + p.part_kb, kbs);
                    uint32_t add = 0;
                    for (; kb < end; ++kb) {
                        if (!xent_wait(full_bar(stage), phase, p)) { aborted = true; break; }
                        tc_fence_after_sync();
                        const uint64_t xd = x_desc0 + (uint64_t)(stage * (stage_bytes >> 4));
                        const uint64_t wd = w_desc0 + (uint64_t)(stage * (stage_bytes >> 4));
                        if (xent_elect()) {
#pragma unroll
                            for (int j = 0; j < XBK / 16; ++j)
                                mma_f16<CG>(d, xd + X_STEP * (uint64_t)j,
                                            wd + W_STEP * (uint64_t)j, idesc, j > 0 ? 1u : add);
                            mma_commit<CG>(empty_bar(stage));
                        }
                        __syncwarp();
                        add = 1;
                        if (++stage == stages) { stage = 0; phase ^= 1u; }
                    }
                    if (aborted) break;
                    if (xent_elect()) mma_commit<CG>(accf_bar(acc));
                    __syncwarp();
                    if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
                }
            }
            // every MMA issued above has completed before the CTA lets go of its memory
            if (xent_elect()) {
                if constexpr (CG == 2) mma_commit_pair(drain_bar, (uint16_t)1);
                else mma_commit_local(drain_bar);
            }
            __syncwarp();
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() - t0 < 1000000000ull) {
            }
        }
        __syncwarp();
    } else if (warp >= XEPI_WARP0) {
        // ------------------------------------------------------ epilogue --
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(XREGS_EPI));
        const int q = (warp - XEPI_WARP0) & 3;      // TMEM lane quarter
        const int half = (warp - XEPI_WARP0) >> 2;  // even or odd 64-column blocks
        constexpr int BLOCKS = CG;                  // of a tile, at most, in a warp
        const uint32_t staging =
            staging0 + (uint32_t)((warp - XEPI_WARP0) * C_::BOXES * 32 * 128);
        const uint32_t my_row = staging + (uint32_t)lane * 128u;
        int acc = 0;
        uint32_t acc_phase = 0;
        // the accumulator has been read: the MMAs may write it again
        auto release = [&](int a) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) mbar_arrive_cluster(mapa_shared(acce_bar(a), 0));
                else mbar_arrive_local(acce_bar(a));
            }
        };
        pdl_wait();
        const XentWork work = xent_work<MODE, CG>(p);
        float alpha = p.alpha;
        if (MODE != kXentStats && p.scale) alpha *= *p.scale;
        if (p.fault_inject == 1 && !xent_wait_inline(never_bar, 0u, p)) aborted = true;
        for (int t = cluster; t < work.total && !aborted; t += nclusters) {
            const int split = MODE == kXentSum ? t / work.tiles : 0;
            const int2 tile = xent_tile(t - split * work.tiles, work.tiles_m, p);
            const int kbs = blocks_of(split, work);
            const int row0 = (tile.x * CG + (int)rank) * XROWS + q * 32;
            const int row = row0 + lane;
            int target = -1;
            float lse2 = 0.f, d = 0.f;
            if constexpr (MODE == kXentStats) {
                if (row < p.M) {
                    const int v = p.target[row];
                    if (v >= 0 && v < p.vocab) target = v;
                    if (v >= p.vocab) report_bad_value(p.err);
                }
            } else if constexpr (MODE != kXentSum && MODE != kXentTable) {
                if (row < p.info->count) {
                    const int from = p.order[row];
                    target = p.target[from];
                    lse2 = p.lse[from] * kLog2e;
                    d = p.dloss ? alpha * p.dloss[from] : alpha;
                }
            }
            const bool counts = target >= 0 || MODE == kXentTable;
            const int rel = target - p.col0;  // the target's column in this piece
            // the parts of the depth before the last, added up
            const uint32_t lanes = tmem_base + ((uint32_t)(q * 32) << 16);
            float parts[BLOCKS * 64];
#pragma unroll
            for (int i = 0; i < BLOCKS * 64; ++i) parts[i] = 0.f;
            for (int kb = p.part_kb; kb < kbs; kb += p.part_kb) {
                if (!xent_wait_inline(accf_bar(acc), acc_phase, p)) { aborted = true; break; }
                tc_fence_after_sync();
#pragma unroll
                for (int j = 0; j < BLOCKS; ++j) {
                    const int b = half + 2 * j;
                    if (CG == 1 && b * 64 >= p.tile_n) continue;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(lanes + (uint32_t)(acc * ACC_COLS + b * 64 + h * 32), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            parts[j * 64 + h * 32 + i] += __uint_as_float(v[i]);
                    }
                }
                release(acc);
                if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
            }
            if (aborted) break;
            if (!xent_wait_inline(accf_bar(acc), acc_phase, p)) { aborted = true; break; }
            tc_fence_after_sync();
            const uint32_t taddr = lanes + (uint32_t)(acc * ACC_COLS);
            const int c0 = tile.y * p.tile_n, end = min(c0 + p.tile_n, p.N);
            float m = -INFINITY, sum = 0.f;
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j) {
                const int b = half + 2 * j;
                if (CG == 1 && b * 64 >= p.tile_n) continue;
                const int col = c0 + b * 64;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(taddr + (uint32_t)(b * 64 + h * 32), v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] = __float_as_uint(parts[j * 64 + h * 32 + i] + __uint_as_float(v[i]));
                    const int first = col + h * 32;
                    // the target's place in v
                    const int at = target >= 0 && rel < end ? rel - first : -1;
                    if constexpr (MODE == kXentSum) {
                        if (row < p.M) {
                            float* to = p.sums + (split * p.sum_rows + row) * p.sum_ld + first;
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                if (first + i >= p.sum_ld) continue;  // sum_ld % 4 == 0
                                float4 o = make_float4(
                                    __uint_as_float(v[i]), __uint_as_float(v[i + 1]),
                                    __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                                if (p.add) {
                                    const float4 old = *reinterpret_cast<const float4*>(to + i);
                                    o.x += old.x, o.y += old.y, o.z += old.z, o.w += old.w;
                                }
                                *reinterpret_cast<float4*>(to + i) = o;
                            }
                        }
                    } else if constexpr (MODE == kXentStats) {
                        if (end - first < 32) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (first + i >= end) v[i] = 0xff800000u;  // -infinity
                        }
                        float top = __uint_as_float(v[0]);
#pragma unroll
                        for (int i = 1; i < 32; ++i) top = fmaxf(top, __uint_as_float(v[i]));
                        const float nm = fmaxf(m, top);
                        const float from = nm == -INFINITY ? 0.f : nm;
                        const float off = -from * kLog2e;
                        sum *= ex2((m - from) * kLog2e);
                        float s0 = 0.f, s1 = 0.f;
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            s0 += ex2(fmaf(__uint_as_float(v[i]), kLog2e, off));
                            s1 += ex2(fmaf(__uint_as_float(v[i + 1]), kLog2e, off));
                        }
                        sum += s0 + s1;
                        m = nm;
                        if ((unsigned)at < 32u) {
                            float z = 0.f;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i == at) z = __uint_as_float(v[i]);
                            p.picked[row] = z;
                        }
                    } else {
                        float g[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            g[i] = MODE == kXentTable
                                       ? alpha * __uint_as_float(v[i])
                                       : d * ex2(fmaf(__uint_as_float(v[i]), kLog2e, -lse2));
                        if (MODE != kXentTable && (unsigned)at < 32u) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i == at)
                                    g[i] = d * (ex2(fmaf(__uint_as_float(v[i]), kLog2e, -lse2)) -
                                                1.f);
                        }
                        // The staging box: 16-byte unit u of row r sits at u ^ (r & 7), the
                        // map's 128-byte swizzle. Rows that do not count are zero whatever
                        // their logits are.
                        if (h == 0) {
                            if (lane == 0) bulk_wait_read_all();
                            __syncwarp();
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint32_t hi[4], lo[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float a = g[8 * u + 2 * e], c = g[8 * u + 2 * e + 1];
                                hi[e] = counts ? pack16<BF16>(a, c) : 0u;
                                if constexpr (MODE == kXentGrad2) {
                                    // what hi left; an infinity or NaN is hi's alone
                                    const float2 back = unpack16<BF16>(hi[e]);
                                    const float ra = a - back.x, rc = c - back.y;
                                    lo[e] = counts ? pack16<BF16>(fabsf(ra) < INFINITY ? ra : 0.f,
                                                                  fabsf(rc) < INFINITY ? rc : 0.f)
                                                   : 0u;
                                }
                            }
                            const uint32_t dst =
                                my_row + (uint32_t)(((h * 4 + u) ^ (lane & 7)) * 16);
                            xent_sts128(dst, hi[0], hi[1], hi[2], hi[3]);
                            if constexpr (MODE == kXentGrad2)
                                xent_sts128(dst + 32 * 128, lo[0], lo[1], lo[2], lo[3]);
                        }
                        if (h == 1) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            // (G has room for whole tiles, dW has not)
                            if (lane == 0 && (MODE != kXentTable || (row0 < p.M && col < p.N))) {
                                tma_store_2d(&p.map_g, staging, col, row0);
                                if constexpr (MODE == kXentGrad2)
                                    tma_store_2d(&p.map_g, staging + 32 * 128, col,
                                                 p.info->used + row0);
                                bulk_commit_group();
                            }
                        }
                    }
                }
            }
            if constexpr (MODE == kXentStats)
                if (row < p.M)
                    p.part[(int64_t)(tile.y * 2 + half) * p.part_ld + row] = make_float2(m, sum);
            release(acc);
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
        if (MODE != kXentStats && MODE != kXentSum && lane == 0) bulk_wait_all();
        __syncwarp();
    } else {
        give_registers();
    }

    // ------------------------------------------------------------ teardown --
    tc_fence_before_sync();
    if constexpr (CG == 2) cluster_sync_all(); else __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<CG>(tmem_base, 2 * ACC_COLS);
    }
}

template <int MODE, int CG, bool BF16>
int launch_xent_variant(XentParams& xp, const DeviceInfo& dev, cudaStream_t stream) {
    constexpr int SMEM = XentCfg<MODE>::SMEM;
    auto kern = xent_kernel<MODE, CG, BF16>;
    static std::mutex mu;
    static uint64_t configured = 0;  // bit per device
    static int resident[64];
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.blockDim = dim3(XTHREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    {
        std::lock_guard<std::mutex> lock(mu);
        const uint64_t bit = 1ull << (dev.device & 63);
        if (!(configured & bit)) {
            // the epilogue's registers come out of what the block is launched with
            cudaFuncAttributes fa;
            if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return refused();
            if (fa.numRegs != XREGS) return kCuda;
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) !=
                cudaSuccess)
                return refused();
            int n = dev.sm_count / CG;
            if (CG > 1) {
                int fit = 0;
                cfg.gridDim = dim3(CG * n);
                if (cudaOccupancyMaxActiveClusters(&fit, kern, &cfg) == cudaSuccess && fit > 0)
                    n = fit;
                else
                    cudaGetLastError();
            }
            resident[dev.device & 63] = n;
            configured |= bit;
        }
    }
    const int64_t tiles = (int64_t)xp.tiles_m * xp.tiles_n * (MODE == kXentSum ? xp.splits : 1);
    int n = resident[dev.device & 63];
    if (n > tiles) n = (int)tiles;
    cfg.gridDim = dim3(CG * n);
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    cfg.stream = stream;
    if (cudaLaunchKernelEx(&cfg, kern, xp) != cudaSuccess) return refused();
    note_launch();
    return kOk;
}

template <bool BF16>
int launch_xent(XentParams& xp, int mode, int cg, const DeviceInfo& dev, cudaStream_t s) {
    if (mode == kXentStats)
        return cg == 2 ? launch_xent_variant<kXentStats, 2, BF16>(xp, dev, s)
                       : launch_xent_variant<kXentStats, 1, BF16>(xp, dev, s);
    if (mode == kXentGrad)
        return cg == 2 ? launch_xent_variant<kXentGrad, 2, BF16>(xp, dev, s)
                       : launch_xent_variant<kXentGrad, 1, BF16>(xp, dev, s);
    if (mode == kXentGrad2)
        return cg == 2 ? launch_xent_variant<kXentGrad2, 2, BF16>(xp, dev, s)
                       : launch_xent_variant<kXentGrad2, 1, BF16>(xp, dev, s);
    if (mode == kXentTable) return launch_xent_variant<kXentTable, 2, BF16>(xp, dev, s);
    return cg == 2 ? launch_xent_variant<kXentSum, 2, BF16>(xp, dev, s)
                   : launch_xent_variant<kXentSum, 1, BF16>(xp, dev, s);
}

}  // namespace
}  // namespace libgemm
