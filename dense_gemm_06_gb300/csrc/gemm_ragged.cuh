// gemm_ragged.cuh -- the tcgen05 kernel of the products whose sizes live in
// device memory: gemm_grouped, gemm_grouped_k and the two launches of
// gemm_lora (see gemm_ragged.cu for the mathematics and the design).
//
// What bounds it (see gemm_ragged.cu for the cases): few rows per group, HBM --
// the weights stream through the ring once (1024 rows in 128 groups of 1536 x
// 2048: 119 us, 6.5 TB/s); many, the tensor pipe and its feed from L2 (one group
// of 8192^3: 556 us, 1.98 PFLOP/s, gemm() 548 us on the same GPU); the smallest
// calls, the chain of latencies from launch to last store (one row against 4096 x
// 4096 with an adapter: 11 us, of which the weights take 5).
//
// Times in these files are of short runs. In runs of seconds the large calls settle
// at the power limit's clocks and take 12 to 18% longer (cuBLAS: 10%).
//
// One orientation serves all four: the MMA's M side (128 TMEM lanes per CTA)
// is the feature side P -- the weights -- and its N side the row side Q -- the
// tokens --, so that a unit of work is as wide as it has rows, in steps of 16
// (32 for a CTA pair). A group of 40 rows costs 48 columns, not a 128-row tile.
#pragma once

#include "gemm_tc.cuh"
#include "policy.h"
#include "ptx_ragged.cuh"

namespace libgemm {

enum RaggedMode {
    kRagRows = 0,    // groups of rows, a weight matrix each        (gemm_grouped)
    kRagDepth = 1,   // groups of the summed dimension              (gemm_grouped_k)
    kRagShrink = 2,  // T = scale * X LA^T of a row tile's adapters (gemm_lora, 1st launch)
    kRagLora = 3,    // X W^T + T LB                                (gemm_lora, 2nd launch)
    kRagShrinkRows = 4,  // kRagShrink for few rows, by plain dot products
};

// Tensor maps by use. P operands are 3-D (group or adapter number last).
enum RaggedMap {
    kMapP = 0,    // weights / B of the depth product / LA
    kMapQ = 1,    // rows, a full unit's share per box
    kMapQ16 = 2,  // rows, 16 per box (units narrower than the tile)
    kMapLB = 3,   // lora: LB
    kMapT = 4, kMapT16 = 5,  // lora: T, as Q and Q16
    kMapC = 6,    // C, a staging tile per box (depth: 3-D), where c_tma
    kRaggedMaps = 7
};

struct RaggedParams {
    CUtensorMap map[kRaggedMaps];
    const int32_t* offsets;  // rows, depth: G + 1 group limits
    // in device memory; depth: P's and Q's map of each group and the order of the
    // groups; depth, and rows where units are many: the count of units taken
    const CUtensorMap* gmaps;
    const int32_t* order;
    unsigned int* ticket;
    int G;
    int rows;       // rows of C (depth: of each C_g)
    int feats;      // columns of C (shrink: of LB)
    int depth;      // depth: rows of A and B, over which the groups are (kRagShrinkRows: K)
    int num_kb;     // 64-deep k-blocks (depth: per group, from the offsets)
    int tile_w;     // rows of a full unit (shrink: divides list_w)
    int tiles_f;    // feature tiles
    int tiles_r;    // row tiles (depth: per group)
    int split;      // log2 of the CTAs that share a unit's depth (a cluster of single CTAs)
    void* C;
    int c_tma;        // a 16-bit C with 16-byte aligned rows: whole pieces go out by TMA
    int64_t ldc;
    int64_t stridec;  // depth: between the C_g
    EpiParams epi;
    // gemm_lora
    const int32_t* adapter;  // adapter number of each row
    const float* scale;      // one factor per adapter, or null
    const void* x;           // kRagShrinkRows: X and LA, row pitches ldx and ldla
    const void* lora_a;
    int64_t ldx, ldla;
    const void* lora_b;      // LB as the kernels read it, row pitch ldlb (padding zero)
    int64_t ldlb;
    int L, R, slot;          // adapters, rank, lanes per adapter (16, 32, 64 or 128)
    int list_w;              // rows that share one list of adapters (the expand's tile_w)
    int lanes;               // shrink: lanes per unit, 64 (narrow) or 128
    int chains;              // shrink: clusters that share a row tile's lists of lanes
                             // (kRagShrinkRows: blocks of dot products)
    int32_t* lists;          // per list tile: n, list_w adapter numbers, list_w slots, flags
    int list_pitch, flags;   // flags: of a list, one per warp (block) that looked
    void* T;                 // halves of T: 64 elements per 32 lanes, fp16: 128
    int64_t ldt;
    int pdl;                 // host only
    ErrWord* err;
    unsigned long long* check;
    ErrWord gen;
    unsigned long long wait_limit_ns;
    int fault_inject;
#ifdef LIBGEMM_TC_TRACE
    unsigned long long* trace;  // trace build: 64 timestamps for each of trace_ctas CTAs
    unsigned trace_ctas;
#endif
};

#ifdef LIBGEMM_TC_TRACE
unsigned long long* trace_buffer();  // the registered buffer (gemm_tc.cu)
#endif

// Launchers, one per element type (gemm_ragged_<in>_<out>.cu, gemm_lora_<t>.cu).
// cg: CTAs per unit; p_mn: the weights' features are contiguous.
int launch_ragged_f16_f32(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units,
                          const DeviceInfo& dev, cudaStream_t s);
int launch_ragged_bf16_f32(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units,
                           const DeviceInfo& dev, cudaStream_t s);
int launch_ragged_f16_f16(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units,
                          const DeviceInfo& dev, cudaStream_t s);
int launch_ragged_bf16_bf16(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units,
                            const DeviceInfo& dev, cudaStream_t s);
int launch_lora_f16(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units,
                    const DeviceInfo& dev, cudaStream_t s);
int launch_lora_bf16(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units,
                     const DeviceInfo& dev, cudaStream_t s);

namespace {

constexpr int UNIT_SLOTS = 4;  // units found ahead

// The ring: 128 features and up to 128 rows of 64 k each per CTA and stage.
// NARROW (the shrink of ranks up to 32): 64 of both, two k-blocks to a stage.
// With so little work in a block the loops' own latency (a wait, an election,
// a commit: 0.22 us) is what bounds it, not the bytes: 8192 rows of 4096 took
// 22 us with one block per stage however many stages there were. The MMA's
// other 64 lanes read whatever lies behind and are never stored.
template <bool NARROW>
struct RCfg {
    static constexpr int LANES = NARROW ? 64 : 128;
    static constexpr int SUB = NARROW ? 2 : 1;  // k-blocks per stage
    static constexpr int BLOCK_BYTES = LANES * BK * 2;
    static constexpr int P_BYTES = SUB * BLOCK_BYTES;
    static constexpr int Q_BYTES = SUB * BLOCK_BYTES;
    static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
    static constexpr int STAGES = 6;
    static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
    // Two 2 KB staging tiles per epilogue warp (shrink: its list instead --
    // ids[256], slots[256], list[256], warp sums[16])
    static constexpr int TILE_BYTES = 2048;
    static constexpr int EXTRA_BYTES = EPI_WARPS * 2 * TILE_BYTES;
    // Partial sums of a split unit of up to PARTS_ROWS rows: behind the list.
    static constexpr int PARTS_OFFSET = 4096;
    static constexpr int PARTS_ROWS = (EXTRA_BYTES - PARTS_OFFSET) / 512;
    // full[S], empty[S], acc_full[2], acc_empty[2], drain, never, ring_free, parts,
    // unit_ready[UNITS], unit_read[UNITS], unit_read_by_peer[UNITS]; then the TMEM
    // address and the units
    static constexpr int UNITS = UNIT_SLOTS;
    static constexpr int NUM_BARS = 2 * STAGES + 8 + 3 * UNITS;
    static constexpr int UNIT_OFFSET = NUM_BARS * 8 + 16;
    static constexpr int SMEM_BYTES = RING_BYTES + EXTRA_BYTES + UNIT_OFFSET + UNITS * 48 + 1024;
    static_assert(SMEM_BYTES <= 232448, "over the 227 KB of shared memory a CTA may use");
};
// Warps: 0 copies, 1 MMA, 2 units, 3 .. 10 epilogue.
constexpr int REPI_WARP0 = 3;
constexpr int RTHREADS = 32 * (REPI_WARP0 + EPI_WARPS);
// fp32 results: depth summed in one accumulator, in k-blocks. The tensor core
// cuts each addition to the accumulator off below 2^-23 of it, an error that
// grows with the depth (measured against 64 bits, 2-norm: 1.3e-6 of the result
// at a depth of 1037, 3.5e-6 at a few thousand), so sums of 704 are added up in
// registers with rounding (6e-7 at any depth; plain fp32 sums: 2.5e-7 to
// 5e-7). 16-bit results round off 2^-9 or 2^-12 anyway and sum whole. Sums of
// 512, 768 or 1024 take the same time (476-483 us, 64 gradients of 2816 x 2048).
constexpr int FOLD_KB = 11;
constexpr int EXT_K = 32;  // lanes of T (rows of LB) per extension block: hi | lo fill 64
// T in fp16. Below 2^-3 its low half runs out of exponents (its last step is
// 2^-24), so what hi + lo leave of t is kept too, times 2^24 and again as two
// halves: t = hi + lo + 2^-24 (hi2 + lo2), to 2^-22 of t down to 2^-25 and
// 2^-49 below. In a tile where some row's neighbouring ranks (a warp's 32, four
// in the dot products) are all below T_SMALL, the expand sums hi2 and lo2 into
// the other accumulator and the epilogue joins the two. Elsewhere hi + lo leave
// 2^-25, at most 2^-19 of the row's largest t nearby: 1/128 of C's own rounding.
// (bf16 has fp32's exponents: hi + lo do.) Measured, 48 rows and 24 adapters of
// 4096 x 4096: 16.3 us with hi and lo only, 16.6 us so, 18.1 us where the second
// accumulator is used; 8192 rows 179, 184 and 205 us. Rank 16, T about 1e-6, LB
// about 1e3: the adapters' part was off by 1.7e-2 with hi and lo only.
constexpr float T_SMALL = 0x1p-6f, T_UP = 0x1p24f, T_DOWN = 0x1p-24f;
// Elements of T per 32 lanes.
template <typename In>
constexpr int T_BLOCK = std::is_same_v<In, __half> ? 128 : 64;
// Bits of a list's flags.
constexpr int kListNonfinite = 1;  // an infinity or NaN in a listed LB
constexpr int kListSmallT = 2;     // small T: hi2 and lo2 count

// One unit of work: `width` rows of C from row0 (those before row_end are
// stored) by 128 features per CTA from feat0.
struct RUnit {
    int g;           // group (weight matrix)
    int row0, row_end;
    int feat0;       // first feature of the unit (of the pair)
    int width;       // MMA N: rows rounded up
    int k0, nkb;     // depth: first k-row and k-blocks; else 0 and num_kb
    int k_end;       // depth: the group's last k-row + 1
    int tile;        // lora: list tile
};

// An active epilogue that adds to C and does nothing else: an fp32 C takes it as
// global additions.
__host__ __device__ __forceinline__ bool adds(const EpiParams& e) {
    return e.beta == 1.f && !e.bias && e.act == 0;
}

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// rows mode: finds the group, row tile and feature tile of unit u. The whole
// warp takes part: a lane holds the limits of four consecutive groups, a scan
// gives the units before each lane, and 128 groups are searched at a time.
// Units are asked for in increasing order, so later chunks replace earlier
// ones. Limits are clamped to [0, M] and to the largest before them, so that
// whatever they hold, the groups do not overlap, no row outside A and C is ever
// addressed and there are no more units than the launch was sized for.
struct RowWalk {
    int g0, base, total, incl;
    int top;  // the largest limit before the chunk
    int off[5];

    __device__ __forceinline__ int units(const RaggedParams& p, int i) const {
        const int lane = threadIdx.x & 31;
        const int rows = off[i + 1] - off[i];
        return lane * 4 + i < p.G - g0 && rows > 0 ? ragged_units(rows, p.tile_w) * p.tiles_f : 0;
    }
    __device__ __forceinline__ void load(const RaggedParams& p) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            const int g = g0 + min(lane * 4 + i, p.G - g0);
            off[i] = clampi(__ldcg(p.offsets + g), 0, p.rows);
        }
        int most = max(max(off[0], off[1]), max(off[2], off[3]));
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, most, d);
            if (lane >= d) most = max(most, o);
        }
        int before = __shfl_up_sync(0xffffffffu, most, 1);
        before = lane > 0 ? max(before, top) : top;
#pragma unroll
        for (int i = 0; i < 5; ++i) before = off[i] = max(off[i], before);
        top = __shfl_sync(0xffffffffu, off[4], 31);
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) mine += units(p, i);
        incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        total = __shfl_sync(0xffffffffu, incl, 31);
    }
    __device__ __forceinline__ void start(const RaggedParams& p) {
        g0 = base = top = 0;
        load(p);
    }
    template <int CG>
    __device__ __forceinline__ bool find(const RaggedParams& p, int u, RUnit& un) {
        while (u >= base + total) {
            if (p.G - g0 <= 128) return false;
            base += total;
            g0 += 128;
            load(p);
        }
        const int lane = threadIdx.x & 31;
        const int r = u - base;
        const int who = __ffs(__ballot_sync(0xffffffffu, incl > r)) - 1;
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) mine += units(p, i);
        int rem = r - (incl - mine), g = g0 + lane * 4, lo = off[0], hi = off[1];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int n = units(p, i);
            if (g == g0 + lane * 4 + i && rem >= n) {
                rem -= n;
                ++g;
                lo = off[i + 1];
                hi = off[i + 2];
            }
        }
        un.g = __shfl_sync(0xffffffffu, g, who);
        rem = __shfl_sync(0xffffffffu, rem, who);
        lo = __shfl_sync(0xffffffffu, lo, who);
        hi = __shfl_sync(0xffffffffu, hi, who);
        const TileCoord tc = raster(rem, ragged_units(hi - lo, p.tile_w), p.tiles_f);
        un.row0 = lo + tc.tm * p.tile_w;
        un.row_end = hi;
        un.feat0 = tc.tn * 128 * CG;
        un.width = ragged_width(hi - un.row0, 16 * CG, p.tile_w);
        un.k0 = 0;
        un.k_end = 0;
        un.nkb = p.num_kb;
        un.tile = 0;
        return true;
    }
};

// The units of a role, in order: u = cluster, cluster + clusters, ...
template <int CG, int MODE>
struct Units {
    RowWalk walk;
    int u, step;
    bool started;

    __device__ __forceinline__ Units(const RaggedParams& p, int cluster, int clusters)
        : u(cluster), step(clusters), started(false) {
        if constexpr (MODE == kRagRows) walk.start(p);
    }
    __device__ __forceinline__ bool next(const RaggedParams& p, RUnit& un) {
        int t = u;
        u += step;
        if constexpr (MODE == kRagDepth || MODE == kRagRows) {
            // After its first unit a cluster takes the next one that nobody has:
            // the groups, and so the units, are of any size (see depth_maps_kernel
            // for their order in the depth product).
            if (started && (MODE == kRagDepth || p.ticket)) {
                if ((threadIdx.x & 31) == 0) t = step + (int)atomicAdd(p.ticket, 1u);
                t = __shfl_sync(0xffffffffu, t, 0);
            }
            started = true;
        }
        if constexpr (MODE == kRagRows) {
            return walk.template find<CG>(p, t, un);
        } else if constexpr (MODE == kRagDepth) {
            const int per = p.tiles_r * p.tiles_f;
            if (t >= p.G * per) return false;
            const int nth = t / per;
            un.g = __ldcg(p.order + nth);
            const TileCoord tc = raster(t - nth * per, p.tiles_r, p.tiles_f);
            un.row0 = tc.tm * p.tile_w;
            un.row_end = p.rows;
            un.feat0 = tc.tn * 128 * CG;
            un.width = ragged_width(p.rows - un.row0, 64 * CG, p.tile_w);
            un.k0 = clampi(__ldcg(p.offsets + un.g), 0, p.depth);
            un.k_end = clampi(__ldcg(p.offsets + un.g + 1), un.k0, p.depth);
            un.nkb = ragged_blocks(un.k0, un.k_end);
            un.tile = 0;
            return true;
        } else if constexpr (MODE == kRagLora) {
            if (t >= p.tiles_r * p.tiles_f) return false;
            const TileCoord tc = raster(t, p.tiles_r, p.tiles_f);
            un.g = 0;
            un.tile = tc.tm;
            un.row0 = tc.tm * p.tile_w;
            un.row_end = p.rows;
            un.feat0 = tc.tn * 128 * CG;
            un.width = ragged_width(p.rows - un.row0, 16 * CG, p.tile_w);
            un.k0 = un.k_end = 0;
            un.nkb = p.num_kb;
            return true;
        }
        return false;
    }
};

// shrink: the units of a cluster are the lane parts (`lanes` each) sg = chain, chain +
// chains, ... of its row tile's list (lane l of the list: rank index l % slot
// of its l / slot-th adapter); un.g = sg.
template <>
struct Units<1, kRagShrink> {
    int sg, parts, tile;
    __device__ __forceinline__ Units(const RaggedParams& p, int cluster, int n)
        : sg(cluster % p.chains), parts((n * p.slot + p.lanes - 1) / p.lanes),
          tile(cluster / p.chains) {}
    __device__ __forceinline__ bool next(const RaggedParams& p, RUnit& un) {
        if (sg >= parts || tile * p.tile_w >= p.rows) return false;
        un.g = sg;
        sg += p.chains;
        un.row0 = tile * p.tile_w;
        un.row_end = p.rows;
        un.feat0 = 0;
        un.width = ragged_width(p.rows - un.row0, 16, p.tile_w);
        un.k0 = un.k_end = 0;
        un.nkb = p.num_kb;
        un.tile = un.row0 / p.list_w;
        return true;
    }
};

// Bounded waits as in gemm_tc.cuh, for this kernel's parameters.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const RaggedParams& p) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, p.err, p.gen, p.wait_limit_ns);
}
__device__ __forceinline__ bool wait_bar_warp(uint32_t bar, uint32_t parity,
                                              const RaggedParams& p) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, p));
}

// A unit passed through shared memory (a shared::cluster address), 48 bytes per
// slot.
__device__ __forceinline__ void put_unit(uint32_t at, const RUnit& un, bool more) {
    st_cluster_v4(at, (uint32_t)un.g, (uint32_t)un.row0, (uint32_t)un.row_end,
                  (uint32_t)un.feat0);
    st_cluster_v4(at + 16, (uint32_t)un.width, (uint32_t)un.k0, (uint32_t)un.nkb,
                  (uint32_t)un.k_end);
    st_cluster_v4(at + 32, (uint32_t)un.tile, more ? 1u : 0u, 0u, 0u);
}
__device__ __forceinline__ bool get_unit(uint32_t at, RUnit& un) {
    const uint4 a = lds128(at), b = lds128(at + 16), c = lds128(at + 32);
    un.g = (int)a.x; un.row0 = (int)a.y; un.row_end = (int)a.z; un.feat0 = (int)a.w;
    un.width = (int)b.x; un.k0 = (int)b.y; un.nkb = (int)b.z; un.k_end = (int)b.w;
    un.tile = (int)c.x;
    return c.y != 0;
}

// A wait on the unit slots. It outlasts a timeout of another wait of the
// launch: every role goes on taking units after one, so that the clusters'
// barriers stay in step, and the slots keep moving.
__device__ __forceinline__ bool wait_unit(uint32_t bar, uint32_t parity, const RaggedParams& p) {
    if (!mbar_try_wait(bar, parity)) {
        const uint64_t t0 = globaltimer_ns(), limit = 2 * p.wait_limit_ns + 1000000000ull;
        while (!mbar_try_wait(bar, parity))
            if (globaltimer_ns() - t0 > limit) {
                gen_record_timeout(p.err, p.gen);
                return false;
            }
    }
    return true;
}

// The units of a role, in order, as warp 2 (a pair's leader's) finds them:
// finding one takes 0.5 to 1.4 us of searches, divisions and reads of the
// limits, which the MMA would otherwise wait for at every unit.
// (Each arrival here is local and of CTA scope: a release at cluster scope
// waits for the warp's outstanding stores of C, 1 to 2 us per unit.)
struct Feed {
    uint32_t ready, slots;  // the first ready barrier and slot
    int j;
    __device__ __forceinline__ Feed(uint32_t r, uint32_t s) : ready(r), slots(s), j(0) {}
    __device__ __forceinline__ bool next(const RaggedParams& p, RUnit& un) {
        const bool more = peek(p, un);
        done();
        return more;
    }
    // The next unit / its slot may be used again.
    __device__ __forceinline__ bool peek(const RaggedParams& p, RUnit& un) {
        const int s = j % UNIT_SLOTS;
        if (!__all_sync(0xffffffffu, wait_unit(ready + 8u * s, (uint32_t)(j / UNIT_SLOTS) & 1u, p)))
            return false;
        return get_unit(slots + 48u * s, un);
    }
    __device__ __forceinline__ void done() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            mbar_arrive_local(ready + 8u * (UNIT_SLOTS + j % UNIT_SLOTS));
        ++j;
    }
};

template <bool BF16>
__device__ __forceinline__ bool nonfinite16(uint32_t w) {
    constexpr uint32_t e = BF16 ? 0x7F80u : 0x7C00u;
    return (w & e) == e || ((w >> 16) & e) == e;
}

// Two packed 16-bit numbers.
template <bool BF16>
__device__ __forceinline__ float2 to_f32x2(uint32_t w) {
    if constexpr (BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// One element of C (feature f of row `row`), fused epilogue included.
template <typename OutT>
__device__ __forceinline__ void store_c(const RaggedParams& p, OutT* dst, float acc, float bias,
                                        bool epi) {
    float x = acc;
    if (epi) {
        x *= p.epi.alpha;
        if (p.epi.beta != 0.f) x = fmaf(p.epi.beta, to_f32(*dst), x);
        x = activate(x + bias, p.epi.act);
    }
    *dst = from_f32<OutT>(x);
}

// x, rounded to a 16-bit T, into shared memory.
template <typename T>
__device__ __forceinline__ void sts_as(uint32_t addr, float x) {
    const T t = from_f32<T>(x);
    asm volatile("st.shared.b16 [%0], %1;"
                 :: "r"(addr), "h"(*reinterpret_cast<const uint16_t*>(&t)) : "memory");
}

// t as two 16-bit numbers, 32 elements apart; fp16: and what they leave of it
// as two more.
template <typename In>
__device__ __forceinline__ void store_t(In* dst, float t) {
    const In hi = from_f32<In>(t);
    const float d = t - to_f32(hi);  // infinite or NaN where hi is: then hi says it all
    const In lo = from_f32<In>(isfinite(d) ? d : 0.f);
    dst[0] = hi;
    dst[32] = lo;
    if constexpr (std::is_same_v<In, __half>) {
        // (a large t leaves more than fp16 holds, and needs none of it)
        const float left = (d - to_f32(lo)) * T_UP, small = fabsf(left) < 1.f ? left : 0.f;
        const In hi2 = from_f32<In>(small);
        dst[64] = hi2;
        dst[96] = from_f32<In>(small - to_f32(hi2));
    }
}

// Is the largest of these numbers' magnitudes, given as bits, small but not zero?
__device__ __forceinline__ bool small_t(uint32_t largest) {
    return largest != 0u && largest < __float_as_uint(T_SMALL);
}

// sum_r T[row][r] LB[id][r][f] for a row whose adapter is the s-th of its list
// (the lanes of `t` in blocks of 32, as store_t leaves them); lb points at
// LB[id][0][f].
template <typename In>
__device__ __noinline__ float adapter_part(const In* t, const In* lb, int64_t ldlb, int lane0,
                                           int rank) {
    float v = 0.f;
    for (int r = 0; r < rank; ++r) {
        const In* tt = t + (lane0 + r) / 32 * T_BLOCK<In> + (lane0 + r) % 32;
        float x = to_f32(tt[0]) + to_f32(tt[32]);
        if constexpr (std::is_same_v<In, __half>)
            x = fmaf(T_DOWN, to_f32(tt[64]) + to_f32(tt[96]), x);
        v = fmaf(x, to_f32(lb[r * ldlb]), v);
    }
    return v;
}

// wait_bar_warp without a call: the folding epilogue waits with its sums live,
// and a call would spill them.
__device__ __forceinline__ bool wait_bar_inline(uint32_t bar, uint32_t parity,
                                                const RaggedParams& p) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t n = 1;; ++n) {
            ok = mbar_try_wait(bar, parity);
            if (ok || ((n & 31u) == 0 && gen_failed(p.err, p.gen))) break;
            if ((n & 31u) == 0 && globaltimer_ns() - t0 > p.wait_limit_ns) {
                gen_record_timeout(p.err, p.gen);
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// Debug build: true when element (row, f) lies inside C, else records it.
__device__ __forceinline__ bool c_checked(const RaggedParams& p, int row, int f) {
    return device_check(p.check, row >= 0 && row < p.rows && f >= 0 && f < p.feats, kCheckTcStore,
                        ((unsigned long long)(uint32_t)row << 24) | (uint32_t)f);
}

// The list of the distinct adapters of a row tile, in order of first use, by
// all threads of the CTA: ids[list_w] the adapter or -1 of each row, then
// slots[] each row's place in the list (-1: none), list[] the adapters.
// Returns their number. Rows of one warp find each other by match_any; the
// first of each set then looks for its adapter among the earlier warps' rows
// in shared memory (at most 224, four per load, no early exit: the loads
// pipeline, where a scalar loop that stops at the first hit waits for each).
template <int NTHREADS>
__device__ __forceinline__ int make_list(const RaggedParams& p, int row0, int* ids, int* slots,
                                         int* list, int* sums) {
    const int i = threadIdx.x, warp = i >> 5, lane = i & 31;
    int id = -1;
    if (i < p.list_w && row0 + i < p.rows) {
        id = __ldcg(p.adapter + row0 + i);
        if (id >= p.L) {
            gen_record_timeout(p.err + 1, 1);  // flags the bad value (see internal.h)
            id = -1;
        }
        if (id < 0) id = -1;
    }
    if (i < 256) ids[i] = id;
    __syncthreads();
    // the row's first equal within its warp, then (that row) among earlier warps
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    const int lead = __ffs(same) - 1;
    int first = warp * 32 + lead;
    if (id >= 0 && lead == lane && i < 256) {
        const int4* v = reinterpret_cast<const int4*>(ids);
#pragma unroll 8
        for (int j = warp * 8 - 1; j >= 0; --j) {
            const int4 x = v[j];
            if (x.w == id) first = 4 * j + 3;
            if (x.z == id) first = 4 * j + 2;
            if (x.y == id) first = 4 * j + 1;
            if (x.x == id) first = 4 * j;
        }
    }
    const bool mine = id >= 0 && first == i;
    const uint32_t b = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) sums[warp] = __popc(b);
    first = __shfl_sync(0xffffffffu, first, lead);
    __syncthreads();
    int place = __popc(b & ((1u << lane) - 1)), n = 0;
#pragma unroll
    for (int w = 0; w < NTHREADS / 32; ++w) {
        const int c = sums[w];
        if (w < warp) place += c;
        n += c;
    }
    if (mine) {
        slots[i] = place;
        list[place] = id;
    }
    __syncthreads();
    int s = -1;
    if (id >= 0) s = slots[first];
    __syncthreads();
    if (i < 256) slots[i] = s;
    __syncthreads();
    return n;
}

// Does the LB of a listed adapter hold an infinity or a NaN, in this thread's
// share (16-byte groups i, i + step, ... of the listed LBs one after the other;
// their rows' padding is zero)? Eight loads in flight.
template <bool BF16>
__device__ __forceinline__ bool scan_lb(const RaggedParams& p, const int* list, int n, uint32_t i,
                                        uint32_t step) {
    const uint32_t vecs = (uint32_t)((int64_t)p.R * p.ldlb / 8);
    const uint64_t total = (uint64_t)n * vecs;
    const uint4* lb = static_cast<const uint4*>(p.lora_b);
    bool bad = false;
    for (uint64_t at = i; at < total; at += 8ull * step) {
        uint4 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint64_t x = at + (uint64_t)j * step;
            w[j] = make_uint4(0u, 0u, 0u, 0u);
            if (x < total) {
                const uint32_t a = (uint32_t)x / vecs;  // total < 2^32: see lora()
                w[j] = __ldg(lb + (int64_t)list[a] * vecs + ((uint32_t)x - a * vecs));
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            bad |= nonfinite16<BF16>(w[j].x) | nonfinite16<BF16>(w[j].y) |
                   nonfinite16<BF16>(w[j].z) | nonfinite16<BF16>(w[j].w);
    }
    return bad;
}

// kRagShrinkRows: T of few rows without tensor cores. A block computes ROW_RANKS
// of a row's dot products sum_k x[k] LA_a[r][k], each of its 8 warps an eighth
// of K for all of them, straight from memory, and writes them (zeros for the
// list's other adapters). Little is read twice in a decoding batch, so there is
// nothing to tile; what counts is the chain of latencies: the row's adapter
// number, then all loads in flight at once while the list is made, then a
// shuffle and one exchange through shared memory -- where the tensor-core form
// goes through a ring, a cluster's exchange and its barriers (10.7 us for one
// row of 4096, 14 us for 48). The blocks past p.chains scan LB meanwhile, one
// flag each.
constexpr int kRowsThreads = 256, ROW_RANKS = 4;
template <bool BF16>
__global__ void __launch_bounds__(kRowsThreads)
    lora_rows_kernel(const __grid_constant__ RaggedParams p) {
    using In = std::conditional_t<BF16, __nv_bfloat16, __half>;
    constexpr int WARPS = kRowsThreads / 32;
    __shared__ __align__(16) int ids[256], slots[256], list[256], sums[16];
    __shared__ float partial[WARPS][ROW_RANKS];
    __shared__ int any_bad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) any_bad = 0;
    pdl_wait();  // and the expand relies on it, as after kRagShrink
    pdl_launch_dependents();
    if ((int)blockIdx.x >= p.chains) {
        const int n = make_list<kRowsThreads>(p, 0, ids, slots, list, sums);
        const int me = (int)blockIdx.x - p.chains;
        const int scans = (int)gridDim.x - p.chains;
        const bool bad = scan_lb<BF16>(p, list, n, (uint32_t)(me * kRowsThreads + threadIdx.x),
                                       (uint32_t)(scans * kRowsThreads));
        if (__any_sync(0xffffffffu, bad) && lane == 0) any_bad = 1;
        __syncthreads();
        if (threadIdx.x == 0) p.lists[1 + 2 * p.list_w + me] = any_bad ? kListNonfinite : 0;
        return;
    }
    const int per_row = p.slot / ROW_RANKS;  // blocks per row
    const int row = (int)blockIdx.x / per_row;
    const int r0 = (int)blockIdx.x % per_row * ROW_RANKS;
    const int a = __ldcg(p.adapter + row);
    const bool some = a >= 0 && a < p.L && r0 < p.R;
    float t[ROW_RANKS] = {};
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const In*>(p.x) +
                                                    (int64_t)row * p.ldx);
    const uint4* la[ROW_RANKS];
#pragma unroll
    for (int i = 0; i < ROW_RANKS; ++i)  // a rank past the last reads the last's row
        la[i] = reinterpret_cast<const uint4*>(
            static_cast<const In*>(p.lora_a) +
            ((int64_t)(some ? a : 0) * p.R + min(r0 + i, p.R - 1)) * p.ldla);
    const int vecs = p.depth / 8, rest = p.depth % 8;
    // vectors v, v + 32 and those of the other ranks, in flight across the list
    constexpr int U = 2, STEP = WARPS * 32;
    uint4 xv[U], av[U][ROW_RANKS];
    auto load = [&](int v) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = some && v + u * STEP < vecs;
            xv[u] = in ? __ldg(x + v + u * STEP) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < ROW_RANKS; ++i)
                av[u][i] = in ? __ldg(la[i] + v + u * STEP) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto dot = [](float acc, const uint4& u, const uint4& v) {
        const uint32_t a4[4] = {u.x, u.y, u.z, u.w}, b4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = to_f32x2<BF16>(a4[i]), g = to_f32x2<BF16>(b4[i]);
            acc = fmaf(f.x, g.x, acc);
            acc = fmaf(f.y, g.y, acc);
        }
        return acc;
    };
    int v = warp * 32 + lane;
    load(v);
    const int n = make_list<kRowsThreads>(p, 0, ids, slots, list, sums);
    for (; v - lane - warp * 32 < vecs; v += U * STEP) {
        if (v - lane - warp * 32 != 0) load(v);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < ROW_RANKS; ++i) t[i] = dot(t[i], xv[u], av[u][i]);
    }
    if (some && warp == 0 && lane < rest)
#pragma unroll
        for (int i = 0; i < ROW_RANKS; ++i)
            t[i] = fmaf(to_f32(reinterpret_cast<const In*>(x)[8 * vecs + lane]),
                        to_f32(reinterpret_cast<const In*>(la[i])[8 * vecs + lane]), t[i]);
#pragma unroll
    for (int i = 0; i < ROW_RANKS; ++i) {
#pragma unroll
        for (int d = 16; d > 0; d /= 2) t[i] += __shfl_xor_sync(0xffffffffu, t[i], d);
        if (lane == 0) partial[warp][i] = t[i];
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) p.lists[0] = n;
        if (threadIdx.x < n) p.lists[1 + threadIdx.x] = list[threadIdx.x];
        if (threadIdx.x < p.list_w) p.lists[1 + p.list_w + threadIdx.x] = slots[threadIdx.x];
    }
    if (!BF16 && threadIdx.x == 0) {  // this block's flag: behind those of the scan
        uint32_t largest = 0u;
#pragma unroll
        for (int i = 0; i < ROW_RANKS; ++i) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) sum += partial[w][i];
            if (p.scale && some) sum *= p.scale[a];
            if (some && r0 + i < p.R) largest = max(largest, __float_as_uint(fabsf(sum)));
        }
        p.lists[1 + 2 * p.list_w + (int)gridDim.x - p.chains + (int)blockIdx.x] =
            small_t(largest) ? kListSmallT : 0;
    }
    const int s = slots[row];
    In* out = static_cast<In*>(p.T) + (int64_t)row * p.ldt;
    for (int k = threadIdx.x; k < n * ROW_RANKS; k += kRowsThreads) {
        const int j = k / ROW_RANKS, i = k % ROW_RANKS;
        float sum = 0.f;
        if (j == s && r0 + i < p.R) {
#pragma unroll
            for (int w = 0; w < WARPS; ++w) sum += partial[w][i];
            if (p.scale) sum *= p.scale[a];
        }
        const int ll = j * p.slot + r0 + i;
        store_t<In>(out + ll / 32 * T_BLOCK<In> + ll % 32, sum);
    }
}

// CG: CTAs per unit (a pair halves P's features and Q's rows between its
// CTAs). P_MN: P's features are contiguous (weights N-major; always in the
// depth product); the shrink, whose P is always K-major, runs its narrow ring
// with it. With p.split > 0 (CG == 1) a cluster of 2^split CTAs shares
// each unit: every CTA sums its share of the k-blocks, and the partial sums
// meet in the shared memory of the CTA that owns the row, in rank order.
// EPI: the launch has a fused epilogue. A template argument where fp32 sums are
// folded (else always true): the 128 sums leave the plain kernel no registers
// for code that it does not run (511 us against 477 us, 64 weight gradients of
// 2816 x 2048).
template <int CG, int MODE, bool P_MN, bool BF16, typename OutT, bool EPI>
__global__ void __launch_bounds__(RTHREADS, 1)
    ragged_kernel(const __grid_constant__ RaggedParams p) {
    constexpr bool NARROW = MODE == kRagShrink && P_MN;
    constexpr bool PF_MN = P_MN && MODE != kRagShrink;  // P's features are contiguous
    using C_ = RCfg<NARROW>;
    using In = std::conditional_t<BF16, __nv_bfloat16, __half>;
    constexpr bool Q_MN = MODE == kRagDepth;
    // T in fp16 may need the second accumulator (see T_SMALL)
    constexpr bool SMALL_T = MODE == kRagLora && !BF16;
    constexpr bool FOLD = std::is_same_v<OutT, float> && MODE != kRagShrink;
    constexpr int CHUNKS = CG == 2 ? 4 : 2;  // of 32 rows that an epilogue warp stores
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);

    const uint32_t sP0 = base;
    const uint32_t sQ0 = base + C_::STAGES * C_::P_BYTES;
    const uint32_t bar0 = base + C_::RING_BYTES + C_::EXTRA_BYTES;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (C_::STAGES + s); };
    auto accf_bar = [&](int a) { return bar0 + 8u * (2 * C_::STAGES + a); };
    auto acce_bar = [&](int a) { return bar0 + 8u * (2 * C_::STAGES + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * C_::STAGES + 4);
    const uint32_t never_bar = bar0 + 8u * (2 * C_::STAGES + 5);
    const uint32_t free_bar = bar0 + 8u * (2 * C_::STAGES + 6);   // every CTA's ring is free
    const uint32_t parts_bar = bar0 + 8u * (2 * C_::STAGES + 7);  // partial sums have arrived
    const uint32_t ready_bar = bar0 + 8u * (2 * C_::STAGES + 8);  // [UNITS], then read[UNITS]
    const uint32_t unit_slots = bar0 + (uint32_t)C_::UNIT_OFFSET;
    int* sm_ids = reinterpret_cast<int*>(smem + C_::RING_BYTES);
    int* sm_slots = sm_ids + 256;
    int* sm_list = sm_ids + 512;
    int* sm_sums = sm_ids + 768;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C_::RING_BYTES + C_::EXTRA_BYTES +
                                                      8 * C_::NUM_BARS);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int S = CG == 1 && MODE != kRagDepth ? 1 << p.split : 1;  // depth: units by ticket
    const uint32_t crank = CG == 2 || S > 1 ? cluster_ctarank() : 0u;
    const uint32_t rank = CG == 2 ? crank : 0u;   // side of the pair
    const int part = S > 1 ? (int)crank : 0;      // share of the depth
    const bool leader = rank == 0;
    const int per_cluster = CG == 2 ? 2 : S;
    const int cluster = (int)blockIdx.x / per_cluster;
    const int nclusters = (int)gridDim.x / per_cluster;

    if (threadIdx.x == 0) TC_TRACE(p, 0);
    if constexpr (MODE == kRagShrink) {
        // Everything before this launch is complete past the wait, and the
        // expand, which may then start, relies on that: it reads X and W
        // without waiting for this grid.
        pdl_wait();
    }
    pdl_launch_dependents();

    if (threadIdx.x == 0) {
        if (MODE != kRagDepth && p.num_kb > 0) {  // no maps without a depth
            tma_prefetch_desc(&p.map[kMapP]);
            tma_prefetch_desc(&p.map[kMapQ]);
            tma_prefetch_desc(&p.map[kMapQ16]);
            if (MODE == kRagLora) {
                tma_prefetch_desc(&p.map[kMapLB]);
                tma_prefetch_desc(&p.map[kMapT]);
                tma_prefetch_desc(&p.map[kMapT16]);
            }
        }
        for (int s = 0; s < C_::STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(accf_bar(a), 1);
            mbar_init(acce_bar(a), CG * EPI_WARPS);
        }
        mbar_init(drain_bar, 1);
        mbar_init(never_bar, 1);
        mbar_init(free_bar, S);
        mbar_init(parts_bar, S * EPI_WARPS);
        for (int i = 0; i < C_::UNITS; ++i) {
            mbar_init(ready_bar + 8u * i, 1);
            // read by the producer, the epilogue warps and the leader's MMA warp
            mbar_init(ready_bar + 8u * (C_::UNITS + i), 1 + EPI_WARPS + (leader ? 1 : 0));
            mbar_init(ready_bar + 8u * (2 * C_::UNITS + i), 1);  // read in the pair's other CTA
        }
        fence_mbarrier_init_cluster();
    }
    if (warp == 1) {
        tmem_alloc<CG>(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish<CG>();
    }
    int n_list = 0;
    if constexpr (MODE == kRagShrink) {
        const int row0 = cluster / p.chains * p.tile_w;
        const int list_tile = row0 / p.list_w;
        n_list = make_list<RTHREADS>(p, list_tile * p.list_w, sm_ids, sm_slots, sm_list, sm_sums);
        if (cluster % p.chains == 0 && part == 0 && row0 % p.list_w == 0) {
            int32_t* out = p.lists + (int64_t)list_tile * p.list_pitch;
            if (threadIdx.x == 0) out[0] = n_list;
            if (threadIdx.x < n_list) out[1 + threadIdx.x] = sm_list[threadIdx.x];
            if (threadIdx.x < p.list_w) out[1 + p.list_w + threadIdx.x] = sm_slots[threadIdx.x];
        }
    }
    tc_fence_before_sync();
    if (CG == 2 || S > 1) cluster_sync_all(); else __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
    if (threadIdx.x == 0) TC_TRACE(p, 1);

    bool aborted = false;
    RUnit un;
    // k-blocks [kb0, kb1) of a unit are this CTA's (all of them but for a split)
    auto share = [&](int n, int& a, int& b) {
        const int sh = CG == 1 && MODE != kRagDepth ? p.split : 0;
        a = (n >> sh) * part + (((n & (S - 1)) * part) >> sh);
        b = (n >> sh) * (part + 1) + (((n & (S - 1)) * (part + 1)) >> sh);
    };
    // lora: those of n extension blocks that this CTA takes.
    auto blocks_of = [&](int n) {
        const int sh = CG == 1 ? p.split : 0;
        return part < n ? ((n - 1 - part) >> sh) + 1 : 0;
    };
    // lora: extension blocks of a unit's list tile; 0 when its flags tell the
    // epilogue to add the adapters' part itself. `ids`: its adapters.
    // `id`: this lane's entry of the list, read with the rest (one latency).
    // `two`: whether hi2 and lo2 count (fp16).
    auto ext_blocks = [&](int tile, int& n, const int32_t*& ids, int& id, bool& two) {
        const int32_t* l = p.lists + (int64_t)tile * p.list_pitch;
        n = __ldcg(l);
        ids = l + 1;
        id = __ldcg(ids + (lane & (p.list_w - 1)));
        int bad = 0;
        for (int i = lane; i < p.flags; i += 32) bad |= __ldcg(l + 1 + 2 * p.list_w + i);
        two = SMALL_T && __any_sync(0xffffffffu, (bad & kListSmallT) != 0);
        if (__any_sync(0xffffffffu, (bad & kListNonfinite) != 0)) return 0;
        return (n * p.slot + EXT_K - 1) / EXT_K;
    };
    const int list_arg = MODE == kRagShrink ? n_list : nclusters;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer --
        if constexpr (MODE == kRagRows || MODE == kRagDepth) pdl_wait();
        int stage = 0;
        uint32_t phase = 0;
        bool waited = false;
        int map_group = -1;
        Feed units(ready_bar, unit_slots);
        for (bool more = units.next(p, un); more;) {
            const int q_rows = un.width / CG;
            const int q_row = un.row0 + (int)rank * q_rows;
            const int f0 = un.feat0 + (int)rank * 128;
            int kb0, kb1;
            share(un.nkb, kb0, kb1);
            const CUtensorMap* gmaps = nullptr;
            if constexpr (MODE == kRagDepth) {
                gmaps = p.gmaps + 2 * (int64_t)un.g;
                if (un.nkb > 0 && un.g != map_group) {  // once per group, by the issuing lane
                    if (elect_one()) {
                        tma_desc_acquire(gmaps);
                        tma_desc_acquire(gmaps + 1);
                    }
                    __syncwarp();
                    map_group = un.g;
                }
            }
            // shrink: the adapters whose lanes this unit holds
            const int spu = MODE == kRagShrink ? C_::LANES / p.slot : 1;
            const int s0 = MODE == kRagShrink ? un.g * spu : 0;
            const int ns = MODE == kRagShrink ? min(spu, n_list - s0) : 1;
            for (int kb = kb0; kb < kb1 && !aborted; kb += C_::SUB) {
                if (!wait_bar_warp(empty_bar(stage), phase ^ 1u, p)) { aborted = true; break; }
                const uint32_t fb = CG == 2 ? mapa_shared(full_bar(stage), 0) : full_bar(stage);
                const uint32_t sp = sP0 + stage * C_::P_BYTES;
                const uint32_t sq = sQ0 + stage * C_::Q_BYTES;
                if constexpr (MODE == kRagDepth) {
                    const int k0 = un.k0 + kb * BK;
                    const int nq = q_rows / 64;  // 64-wide chunks of this CTA's rows
                    if (kb == kb0 && lane == 0) TC_TRACE(p, 2);
                    if (elect_one()) {
                        if (leader)
                            mbar_arrive_expect_tx(full_bar(stage),
                                                  (uint32_t)(CG * (2 + nq) * 64 * BK * 2));
                        // the group's own maps end at its last row: what its last
                        // block takes beyond is zeros, never another group's values
                        for (int j = 0; j < 2; ++j)
                            tma_load_2d<CG>(sp + j * 64 * BK * 2, gmaps, fb, f0 + 64 * j, k0);
                        for (int j = 0; j < nq; ++j)
                            tma_load_2d<CG>(sq + j * 64 * BK * 2, gmaps + 1, fb, q_row + 64 * j,
                                            k0);
                    }
                } else {
                    const int k0 = kb * BK;
                    const bool x_ok = device_check(p.check, (k0 & 7) == 0 && (f0 & 7) == 0,
                                                   kCheckTcTmaX, (unsigned long long)k0);
                    if (kb == kb0 && lane == 0) TC_TRACE(p, 2);
                    if (x_ok && elect_one()) {
                        const int p_bytes = MODE == kRagShrink ? ns * p.slot * BK * 2 : C_::P_BYTES;
                        const int subs = NARROW ? min(C_::SUB, kb1 - kb) : 1;
                        if (leader)
                            mbar_arrive_expect_tx(
                                full_bar(stage),
                                (uint32_t)(subs * CG * (p_bytes + q_rows * BK * 2)));
                        if constexpr (MODE == kRagShrink) {
                            for (int j = 0; j < ns; ++j)
                                for (int b = 0; b < subs; ++b)
                                    tma_load_3d<CG>(
                                        sp + b * C_::BLOCK_BYTES + j * p.slot * BK * 2,
                                        &p.map[kMapP], fb, k0 + b * BK, 0, sm_list[s0 + j]);
                        } else if constexpr (!P_MN) {
                            tma_load_3d<CG>(sp, &p.map[kMapP], fb, k0, f0, un.g);
                        } else {
                            for (int j = 0; j < 2; ++j)
                                tma_load_3d<CG>(sp + j * 64 * BK * 2, &p.map[kMapP], fb,
                                                f0 + 64 * j, k0, un.g);
                        }
                        for (int b = 0; b < subs; ++b) {
                            const uint32_t dst = sq + (uint32_t)(b * C_::BLOCK_BYTES);
                            if (un.width == p.tile_w) {
                                tma_load_2d<CG>(dst, &p.map[kMapQ], fb, k0 + b * BK, q_row);
                            } else {
                                for (int r = 0; r < q_rows; r += 16)
                                    tma_load_2d<CG>(dst + r * 128, &p.map[kMapQ16], fb, k0 + b * BK,
                                                    q_row + r);
                            }
                        }
                    }
                }
                __syncwarp();
                if (++stage == C_::STAGES) { stage = 0; phase ^= 1u; }
            }
            if constexpr (MODE == kRagLora) {
                // T and the lists are the first launch's: wait for it only here
                if (lane == 0) TC_TRACE(p, 3);
                if (!waited) pdl_wait();
                waited = true;
                if (lane == 0) TC_TRACE(p, 4);
                int n;
                const int32_t* ids;
                int lane_id;
                bool two;
                const int ne = ext_blocks(un.tile, n, ids, lane_id, two);
                // hi and lo of all adapters, then hi2 and lo2
                const int mine = blocks_of(ne);
                for (int nth = 0; nth < (two ? 2 * mine : mine) && !aborted; ++nth) {
                    if (!wait_bar_warp(empty_bar(stage), phase ^ 1u, p)) { aborted = true; break; }
                    const int e = part + (two && nth >= mine ? nth - mine : nth) * S;
                    const int x = e * T_BLOCK<In> + (nth < mine ? 0 : 64);  // T's elements
                    const uint32_t fb = CG == 2 ? mapa_shared(full_bar(stage), 0) : full_bar(stage);
                    const uint32_t sp = sP0 + stage * C_::P_BYTES;
                    const uint32_t sq = sQ0 + stage * C_::Q_BYTES;
                    const int k_rows = min(EXT_K, n * p.slot - e * EXT_K);
                    const int box = min(p.slot, EXT_K);  // LB rows per copy
                    const int pieces = k_rows / box;
                    // the (one or two) adapters' numbers, for the lane that issues
                    const int at0 = e * EXT_K / p.slot, at1 = at0 + 1;
                    int id0 = __shfl_sync(0xffffffffu, lane_id, at0 & 31);
                    int id1 = __shfl_sync(0xffffffffu, lane_id, at1 & 31);
                    if (at0 >= 32) id0 = __ldcg(ids + at0);
                    if (at1 >= 32 && at1 < n) id1 = __ldcg(ids + at1);
                    if (elect_one()) {
                        if (leader)
                            mbar_arrive_expect_tx(
                                full_bar(stage),
                                (uint32_t)(CG * (k_rows * 128 * 2 + q_rows * BK * 2)));
                        for (int i = 0; i < pieces; ++i)
                            for (int j = 0; j < 2; ++j)
                                tma_load_3d<CG>(sp + j * 64 * BK * 2 + i * box * 128,
                                                &p.map[kMapLB], fb, f0 + 64 * j,
                                                (e * EXT_K + i * box) % p.slot, i ? id1 : id0);
                        if (un.width == p.tile_w) {
                            tma_load_2d<CG>(sq, &p.map[kMapT], fb, x, q_row);
                        } else {
                            for (int r = 0; r < q_rows; r += 16)
                                tma_load_2d<CG>(sq + r * 128, &p.map[kMapT16], fb, x, q_row + r);
                        }
                    }
                    __syncwarp();
                    if (++stage == C_::STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            more = units.next(p, un);
            if (S > 1 && more) cluster_sync_all();  // the ring held partial sums until here
        }
        if (aborted) grace_period_ns(200000);  // let issued copies land
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer --
        if (leader) {
            if constexpr (MODE == kRagRows || MODE == kRagDepth) pdl_wait();
            constexpr uint32_t idesc0 =
                make_idesc_f16(BF16, PF_MN, Q_MN, (uint32_t)(128 * CG), 0u);
            constexpr uint32_t idesc_ext0 =
                make_idesc_f16(BF16, true, false, (uint32_t)(128 * CG), 0u);
            const uint64_t p_mn0 = make_sdesc_sw128(sP0, 64 * BK * 2, 1024);
            const uint64_t p_desc0 = PF_MN ? p_mn0 : make_sdesc_sw128(sP0, 16, 1024);
            const uint64_t q_desc0 = Q_MN ? make_sdesc_sw128(sQ0, 64 * BK * 2, 1024)
                                          : make_sdesc_sw128(sQ0, 16, 1024);
            constexpr int P_STEP = PF_MN ? UMMA_K * 128 : UMMA_K * 2;
            constexpr int Q_STEP = Q_MN ? UMMA_K * 128 : UMMA_K * 2;
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool waited = false;
            int nt = 0;  // units issued (trace slots)
            Feed units(ready_bar, unit_slots);
            for (bool more = units.next(p, un); more;) {
                const uint32_t width_bits = (uint32_t)(un.width >> 3) << 17;
                int kb0, kb1, n = 0, ne = 0;
                share(un.nkb, kb0, kb1);
                bool issued = false;  // into the accumulator acc: else the first MMA overwrites
                if (lane == 0) TC_TRACE(p, 20 + 4 * nt);
                const uint32_t idesc = idesc0 | width_bits;
                for (int kb = kb0; kb < kb1 && !aborted;) {
                    if (!wait_bar_warp(acce_bar(acc), acc_phase ^ 1u, p)) { aborted = true; break; }
                    tc_fence_after_sync();
                    if (kb == kb0 && lane == 0) TC_TRACE(p, 21 + 4 * nt);
                    const uint32_t d_tmem = tmem_base + (uint32_t)(acc * ACC_COLS);
                    const int first = kb;
                    const int last = FOLD ? min(kb + FOLD_KB, kb1) : kb1;
                    for (; kb < last; kb += C_::SUB) {
                        if (!wait_bar_warp(full_bar(stage), phase, p)) { aborted = true; break; }
                        tc_fence_after_sync();
                        if (kb == kb0 && lane == 0) TC_TRACE(p, 5);
                        if (kb == kb0 && lane == 0) TC_TRACE(p, 22 + 4 * nt);
                        const uint64_t pd = p_desc0 + (uint64_t)(stage * (C_::P_BYTES >> 4));
                        const uint64_t qd = q_desc0 + (uint64_t)(stage * (C_::Q_BYTES >> 4));
                        // depth: a group's last block stops at its last 16-deep step
                        const int left = MODE == kRagDepth ? un.k_end - un.k0 - kb * BK : BK;
                        if (elect_one()) {
                            if (MODE != kRagDepth || left > BK - UMMA_K) {
#pragma unroll
                                for (int j = 0; j < BK / UMMA_K; ++j)
                                    mma_f16<CG>(d_tmem, pd + (uint64_t)(j * (P_STEP >> 4)),
                                                qd + (uint64_t)(j * (Q_STEP >> 4)), idesc,
                                                ((kb - first) | j) != 0 ? 1u : 0u);
                                if (NARROW && kb + 1 < last) {  // the stage's second block
#pragma unroll
                                    for (int j = 0; j < BK / UMMA_K; ++j) {
                                        constexpr int at = C_::BLOCK_BYTES;
                                        mma_f16<CG>(d_tmem,
                                                    pd + (uint64_t)((at + j * P_STEP) >> 4),
                                                    qd + (uint64_t)((at + j * Q_STEP) >> 4),
                                                    idesc, 1u);
                                    }
                                }
                            } else {
                                for (int j = 0; j * UMMA_K < left; ++j)
                                    mma_f16<CG>(d_tmem, pd + (uint64_t)(j * (P_STEP >> 4)),
                                                qd + (uint64_t)(j * (Q_STEP >> 4)), idesc,
                                                ((kb - first) | j) != 0 ? 1u : 0u);
                            }
                            mma_commit<CG>(empty_bar(stage));
                        }
                        __syncwarp();
                        if (++stage == C_::STAGES) { stage = 0; phase ^= 1u; }
                    }
                    issued = true;
                    if (FOLD && kb < kb1 && !aborted) {
                        // hand over this part of the sum, go on in the other accumulator
                        if (elect_one()) mma_commit<CG>(accf_bar(acc));
                        __syncwarp();
                        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
                        issued = false;
                    }
                }
                if constexpr (MODE == kRagLora) {
                    if (!waited) pdl_wait();
                    waited = true;
                    const int32_t* ids;
                    int lane_id;
                    bool two;
                    ne = ext_blocks(un.tile, n, ids, lane_id, two);
                    const int mine = blocks_of(ne);
                    for (int nth = 0; nth < (two ? 2 * mine : mine) && !aborted; ++nth) {
                        const int e = part + (two && nth >= mine ? nth - mine : nth) * S;
                        if (two && nth == mine) {  // hi2 and lo2 go into the other accumulator
                            if (elect_one()) mma_commit<CG>(accf_bar(acc));
                            __syncwarp();
                            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
                            issued = false;
                        }
                        if (!issued && !wait_bar_warp(acce_bar(acc), acc_phase ^ 1u, p)) {
                            aborted = true;
                            break;
                        }
                        if (!wait_bar_warp(full_bar(stage), phase, p)) { aborted = true; break; }
                        tc_fence_after_sync();
                        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * ACC_COLS);
                        const uint64_t pd = p_mn0 + (uint64_t)(stage * (C_::P_BYTES >> 4));
                        const uint64_t qd = q_desc0 + (uint64_t)(stage * (C_::Q_BYTES >> 4));
                        const int steps = min(EXT_K, n * p.slot - e * EXT_K) / UMMA_K;
                        if (elect_one()) {
                            // both halves of T against the same rows of LB
                            for (int j = 0; j < steps; ++j)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    mma_f16<CG>(d_tmem, pd + (uint64_t)(j * (UMMA_K * 128 >> 4)),
                                                qd + (uint64_t)((j + 2 * h) * (UMMA_K * 2 >> 4)),
                                                idesc_ext0 | width_bits,
                                                issued || j + h != 0 ? 1u : 0u);
                            mma_commit<CG>(empty_bar(stage));
                        }
                        issued = true;
                        __syncwarp();
                        if (++stage == C_::STAGES) { stage = 0; phase ^= 1u; }
                    }
                }
                if (lane == 0) TC_TRACE(p, 6);
                if (lane == 0) TC_TRACE(p, 23 + 4 * nt);
                ++nt;
                if (issued && !aborted) {
                    if (elect_one()) mma_commit<CG>(accf_bar(acc));
                    __syncwarp();
                    if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
                }
                more = units.next(p, un);
                if (S > 1 && more) cluster_sync_all();
            }
            // Drain: wait (bounded) until every MMA issued above has completed.
            if (elect_one()) {
                if constexpr (CG == 2) mma_commit_pair(drain_bar, (uint16_t)1);
                else mma_commit_local(drain_bar);
            }
            __syncwarp();
            uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() - t0 < 1000000000ull) {
            }
        }
        __syncwarp();
    } else if (warp >= REPI_WARP0) {
        // ------------------------------------------------------ epilogue --
        const int q = warp & 3;  // TMEM lane quarter (hardware: warp % 4)
        const int half = (warp - REPI_WARP0) >> 2;
        int acc = 0;
        uint32_t acc_phase = 0, split_phase = 0, free_phase = 0;
        // 16-bit results leave in 32 x 32 chunks by TMA (rows K-major at a depth of
        // 2048: 323 us against 337 us by st.global, whose 64-byte rows take the
        // shared-memory port that the operands need); fp32 ones, with 128-byte rows,
        // row by row (2.4 us per unit against 3.0 us through staging tiles).
        constexpr bool BY_TMA = MODE != kRagShrink && sizeof(OutT) == 2;
        const uint32_t tiles =
            base + C_::RING_BYTES + (uint32_t)((warp - REPI_WARP0) * 2 * C_::TILE_BYTES);
        int tile_i = 0;
        int nt = 0;  // units stored (trace slots)
        pdl_wait();
        if (p.fault_inject == 1) {
            if (!__all_sync(0xffffffffu, wait_bar(never_bar, 0u, p))) aborted = true;
        }
        int list_flags = 0;       // shrink: what this warp saw, written at its end
        int32_t* flag = nullptr;
        if constexpr (MODE == kRagShrink) {
            // Does an adapter of the list hold an infinity or a NaN in LB? A
            // zero of T times it would be NaN in the other adapters' rows of the
            // tile, so the expand then adds this tile's adapters one by one.
            // The CTAs of a list tile share the scan, which also brings LB into
            // L2 for the expand.
            const int subs = p.list_w / p.tile_w;
            const int me = ((cluster / p.chains % subs) * p.chains + cluster % p.chains) * S + part;
            const int ctas = subs * p.chains * S;
            bool bad = scan_lb<BF16>(p, sm_list, n_list,
                                     (uint32_t)(me * (EPI_WARPS * 32) + threadIdx.x -
                                                REPI_WARP0 * 32),
                                     (uint32_t)(ctas * (EPI_WARPS * 32)));
            if (__any_sync(0xffffffffu, bad)) list_flags = kListNonfinite;
            flag = p.lists + (int64_t)(cluster / p.chains / subs) * p.list_pitch + 1 +
                   2 * p.list_w + me * EPI_WARPS + (warp - REPI_WARP0);
            if (warp == REPI_WARP0 && lane == 0) TC_TRACE(p, 7);
        }
        Feed units(ready_bar, unit_slots);
        for (bool more = units.peek(p, un); more;) {
            int kb0, kb1, n = 0, ne = 0;
            share(un.nkb, kb0, kb1);
            bool issued = kb1 > kb0;
            const int32_t* ids = nullptr;
            bool two = false;  // a second accumulator holds the sums of hi2 and lo2
            if constexpr (MODE == kRagLora) {
                int lane_id;
                ne = ext_blocks(un.tile, n, ids, lane_id, two);
                two = two && part < ne;
                issued = issued || part < ne;
            }
            const bool by_hand = MODE == kRagLora && n > 0 && ne == 0;
            const int l = q * 32 + lane;  // TMEM lane
            const int f = un.feat0 + (int)rank * 128 + l;
            const int n_rows = min(un.width, un.row_end - un.row0);
            const bool epi = EPI && MODE != kRagShrink && p.epi.active;
            const bool f_ok = f < p.feats;
            float bias = 0.f;
            if (epi && p.epi.bias && f_ok)
                bias = to_f32(static_cast<const OutT*>(p.epi.bias)[(int64_t)un.g * p.feats + f]);
            const bool accumulates = epi && adds(p.epi);
            OutT* c_col = nullptr;
            if constexpr (MODE != kRagShrink)
                c_col = static_cast<OutT*>(p.C) + (int64_t)un.row0 * p.ldc + f +
                        (MODE == kRagDepth ? (int64_t)un.g * p.stridec : 0);
            // shrink: this lane's adapter (place in the list, factor) and rank index
            int slot = 0, r_idx = 0;
            float factor = 1.f;
            In* t_col = nullptr;
            const int* row_slot = nullptr;  // the rows' places in the list
            int my_slot = 0;                // -2 for a lane past the rank: matches no row
            if constexpr (MODE == kRagShrink) {
                const int ll = un.g * C_::LANES + l;
                slot = l < C_::LANES ? ll / p.slot : n_list;  // n_list: nothing to store
                r_idx = ll % p.slot;
                if (slot < n_list && p.scale) factor = p.scale[sm_list[slot]];
                my_slot = r_idx < p.R ? slot : -2;
                row_slot = sm_slots + un.row0 % p.list_w;
                t_col = static_cast<In*>(p.T) + (int64_t)un.row0 * p.ldt +
                        (int64_t)(ll / 32) * T_BLOCK<In> + lane;
            }
            // shrink, fp16: notes a row of small T (all lanes of the warp).
            auto note_t = [&](float t) {
                if (MODE == kRagShrink && !BF16 &&
                    small_t(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(t)))))
                    list_flags |= kListSmallT;
            };
            // lora, by hand: what row j's adapter adds to this lane's feature.
            auto adapters = [&](int j) {
                const int s = __ldcg(ids + p.list_w + j);
                if (s < 0) return 0.f;
                const int id = __ldcg(ids + s);
                return adapter_part<In>(
                    static_cast<const In*>(p.T) + (int64_t)(un.row0 + j) * p.ldt,
                    static_cast<const In*>(p.lora_b) + (int64_t)id * p.R * p.ldlb + f, p.ldlb,
                    s * p.slot, p.R);
            };
            // One row j of the unit, value v of this lane (split depths).
            auto emit = [&](int j, float v) {
                if constexpr (MODE == kRagShrink) {
                    const float t = slot < n_list && row_slot[j] == my_slot ? v * factor : 0.f;
                    note_t(t);
                    if (slot < n_list) store_t<In>(t_col + (int64_t)j * p.ldt, t);
                } else if (f_ok && c_checked(p, un.row0 + j, f)) {
                    if (MODE == kRagLora && by_hand) v += adapters(j);
                    store_c<OutT>(p, c_col + (int64_t)j * p.ldc, v, bias, epi);
                }
            };
            // Rows 32 c .. of the unit, v[i] this lane's value of row 32 c + i (the
            // fused epilogue works in place).
            auto emit_chunk = [&](int c, float (&v)[32]) {
                const int left = n_rows - c * 32;
                if constexpr (MODE == kRagShrink) {
                    if (BF16 && slot >= n_list) return;
                    In* dst = t_col + (int64_t)(c * 32) * p.ldt;
                    int s[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[i] = row_slot[c * 32 + i];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float t = slot < n_list && s[i] == my_slot ? v[i] * factor : 0.f;
                        if (i < left) {
                            note_t(t);
                            if (BF16 || slot < n_list) store_t<In>(dst, t);
                        }
                        dst += p.ldt;
                    }
                    return;
                }
                OutT* dst = c_col + (int64_t)(c * 32) * p.ldc;
                const int row = un.row0 + c * 32;
                if constexpr (MODE == kRagLora) {
                    if (by_hand && f_ok) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < left) v[i] += adapters(c * 32 + i);
                    }
                }
                if constexpr (std::is_same_v<OutT, float>) {
                    if (accumulates) {
                        // C += alpha * sum, added in L2: nothing to wait for (each
                        // element gets one addition, so its order is no question).
                        // That addition takes numbers below 2^-126 as zero.
                        if (!f_ok) return;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (i < left && c_checked(p, row + i, f))
                                red_add_f32(dst, p.epi.alpha * v[i]);
                            dst += p.ldc;
                        }
                        return;
                    }
                }
                if (epi && f_ok) {
                    // the incoming C of OLD rows at a time: one latency for all of them
                    constexpr int OLD = FOLD ? 8 : 32;
#pragma unroll
                    for (int r = 0; r < 32; r += OLD) {
                        float old[OLD];
#pragma unroll
                        for (int i = 0; i < OLD; ++i)
                            old[i] = p.epi.beta != 0.f && r + i < left
                                         ? to_f32(dst[(int64_t)(r + i) * p.ldc]) : 0.f;
#pragma unroll
                        for (int i = 0; i < OLD; ++i) {
                            v[r + i] *= p.epi.alpha;
                            if (p.epi.beta != 0.f) v[r + i] = fmaf(p.epi.beta, old[i], v[r + i]);
                            v[r + i] += bias;
                        }
                    }
                    if (p.epi.act == 1) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = activate(v[i], 1);
                    } else if (p.epi.act == 2) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = activate(v[i], 2);
                    }
                }
                if constexpr (BY_TMA) {
                    if (p.c_tma && left >= 32 && p.feats - (f - lane) >= 32) {
                        // A whole chunk goes through one of the warp's two staging
                        // tiles, written while TMA still reads the other.
                        const uint32_t tile = tiles + (uint32_t)(tile_i * C_::TILE_BYTES);
                        tile_i ^= 1;
                        if (lane == 0) bulk_wait_read_1();
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            sts_as<OutT>(tile + (uint32_t)((i * 32 + lane) * 2), v[i]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && c_checked(p, row, f) && c_checked(p, row + 31, f + 31)) {
                            if constexpr (MODE == kRagDepth)
                                tma_store_3d(&p.map[kMapC], tile, f, row, un.g);
                            else
                                tma_store_2d(&p.map[kMapC], tile, f, row);
                            bulk_commit_group();
                        }
                        return;
                    }
                }
                if (!f_ok) return;
                // one store and one pointer step per row
                if (left >= 32) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (c_checked(p, row + i, f)) *dst = from_f32<OutT>(v[i]);
                        dst += p.ldc;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (i < left && c_checked(p, row + i, f)) *dst = from_f32<OutT>(v[i]);
                        dst += p.ldc;
                    }
                }
            };
            // Split depth: row j of the unit belongs to CTA j % S; this lane's
            // partial sums of the chunk go there.
            const int own = un.width >> (CG == 1 ? p.split : 0);  // rows per CTA
            // Up to PARTS_ROWS rows fit beside the ring; more take the ring itself,
            // once every CTA's MMAs have read theirs.
            const bool beside = un.width <= C_::PARTS_ROWS;
            const uint32_t parts_at =
                beside ? (uint32_t)(C_::RING_BYTES + C_::PARTS_OFFSET) : 0u;
            auto push_chunk = [&](int c, const float (&v)[32]) {
                const uint32_t at = base + parts_at + (uint32_t)((part * own * 128 + l) * 4);
                auto push = [&](int i) {
                    st_cluster_f32(mapa_shared(at, (uint32_t)(i & (S - 1))) +
                                       (uint32_t)(((c * 32 + i) >> p.split) * 512),
                                   v[i]);
                };
#pragma unroll
                for (int i = 0; i < 16; ++i) push(i);
                if (c * 32 + 16 < un.width) {
#pragma unroll
                    for (int i = 16; i < 32; ++i) push(i);
                }
            };
            // pair units' timeline (the leader's slots hold its MMA warp's)
            const bool stamp = CG == 2 && !leader && warp == REPI_WARP0 && lane == 0;
            if (stamp) TC_TRACE(p, 20 + 4 * nt);
            const uint32_t tlane = tmem_base + ((uint32_t)(q * 32) << 16);
            auto read_chunk = [&](int c, uint32_t (&u)[32]) {
                tmem_ld_32x32b_x32(tlane + (uint32_t)(acc * ACC_COLS + c * 32), u);
            };
            auto read_second = [&](int c, uint32_t (&u)[32]) {
                tmem_ld_32x32b_x32(tlane + (uint32_t)((acc ^ 1) * ACC_COLS + c * 32), u);
            };
            auto wait_acc = [&]() {
                if (!aborted && !wait_bar_inline(accf_bar(acc), acc_phase, p)) aborted = true;
                if (SMALL_T && two && !aborted &&
                    !wait_bar_inline(accf_bar(acc ^ 1), acc_phase ^ (uint32_t)acc, p))
                    aborted = true;
                tc_fence_after_sync();
            };
            // Relaxed: the accumulator's reads are complete (wait::ld) and nothing else
            // is handed over, so the arrival need not wait for the stores of C.
            bool held = false;
            auto free_acc = [&]() {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2)
                        mbar_arrive_cluster_relaxed(mapa_shared(acce_bar(acc), 0));
                    else
                        mbar_arrive_local(acce_bar(acc));
                }
                if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
                held = false;
            };
            auto free_accs = [&]() {
                free_acc();
                if (SMALL_T && two) free_acc();
            };
            // The unit's sums: the parts of a folded depth before the last add up
            // in registers; the last one (or the only one) is read from its
            // accumulator as the chunks are stored.
            float sum[FOLD ? CHUNKS : 1][32];
            bool folded = false;
            auto add_chunk = [&](int k) {
                uint32_t u[32];
                read_chunk(half + 2 * k, u);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[k][i] += __uint_as_float(u[i]);
            };
            if constexpr (FOLD) {
                if (kb1 - kb0 > FOLD_KB) {
                    folded = true;
#pragma unroll
                    for (int k = 0; k < CHUNKS; ++k)
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[k][i] = 0.f;
                    for (int kb = kb0; kb + FOLD_KB < kb1; kb += FOLD_KB) {
                        wait_acc();
#pragma unroll
                        for (int k = 0; k < CHUNKS; ++k)
                            if (!aborted && (half + 2 * k) * 32 < un.width) add_chunk(k);
                        free_acc();
                    }
                }
            }
            if (issued) wait_acc();
            held = issued;
            // Here, before this unit's stores and well after the last one's: even a
            // CTA-scope release waits for stores just issued.
            units.done();
            if (warp == REPI_WARP0 && lane == 0) TC_TRACE(p, 8);
            if (stamp) TC_TRACE(p, 22 + 4 * nt);
            auto each_chunk = [&](auto&& use) {
                if constexpr (FOLD) {
                    if (folded) {
#pragma unroll
                        for (int k = 0; k < CHUNKS; ++k)
                            if ((half + 2 * k) * 32 < un.width) {
                                add_chunk(k);
                                if (k == CHUNKS - 1) free_acc();
                                use(half + 2 * k, sum[k]);
                            }
                        return;
                    }
                }
#pragma unroll 1
                for (int c = half; c * 32 < un.width; c += 2) {
                    float v[32];
                    if (issued) {
                        uint32_t u[32];
                        read_chunk(c, u);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
                        if (SMALL_T && two) {
                            read_second(c, u);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] = fmaf(T_DOWN, __uint_as_float(u[i]), v[i]);
                        }
                        if ((c + 2) * 32 >= un.width) free_accs();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0.f;
                    }
                    use(c, v);
                }
            };

            if (S == 1) {
                if (!aborted) each_chunk(emit_chunk);
            } else {
                // Give every CTA the partial sums of its rows (through the ring: after
                // telling the peers that this CTA's MMAs have read it, and hearing
                // the same of theirs).
                if (!beside) {
                    if (!aborted && warp == REPI_WARP0 && lane < S)
                        mbar_arrive_cluster(mapa_shared(free_bar, (uint32_t)lane));
                    if (!aborted && !wait_bar_warp(free_bar, free_phase, p)) aborted = true;
                    free_phase ^= 1u;
                }
                if (warp == REPI_WARP0 && lane == 0) TC_TRACE(p, 9);
                if (!aborted) {
                    each_chunk(push_chunk);
                    __syncwarp();
                    if (lane < S) mbar_arrive_cluster(mapa_shared(parts_bar, (uint32_t)lane));
                    if (warp == REPI_WARP0 && lane == 0) TC_TRACE(p, 10);
                    if (!wait_bar_warp(parts_bar, split_phase, p)) aborted = true;
                }
                if (warp == REPI_WARP0 && lane == 0) TC_TRACE(p, 11);
                if (!aborted) {
                    // add the parts in rank order (a short loop: it runs once per call
                    // when decoding, and code that is not in the instruction cache
                    // costs more than the loads' latency)
                    const float* parts = reinterpret_cast<const float*>(smem + parts_at) + l;
#pragma unroll 1
                    for (int t = half; t < own; t += 2) {
                        const int j = t * S + part;
                        if (j >= n_rows) break;
                        float x[8], v = 0.f;
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            x[r] = r < S ? parts[(r * own + t) * 128] : 0.f;
#pragma unroll
                        for (int r = 0; r < 8; ++r) v += x[r];
                        emit(j, v);
                    }
                }
                split_phase ^= 1u;
                fence_proxy_async_all();  // the next unit's copies write where the parts were
            }
            if (held) free_accs();
            if (warp == REPI_WARP0 && lane == 0) TC_TRACE(p, 12);
            if (stamp) TC_TRACE(p, 23 + 4 * nt);
            ++nt;
            more = units.peek(p, un);
            if (S > 1 && more) cluster_sync_all();
        }
        units.done();
        if (MODE == kRagShrink && lane == 0) *flag = list_flags;
        if (BY_TMA && p.c_tma && lane == 0) bulk_wait_all();
        __syncwarp();
    } else {
        // Warp 2 finds the units and passes them on, up to UNITS ahead, and takes
        // part in the barrier between a split's units. The first CTA's looks over
        // the group limits too (all clamp what is wrong with them).
        if constexpr (MODE == kRagRows || MODE == kRagDepth) {
            pdl_wait();
            if (blockIdx.x == 0) {
                const int most = MODE == kRagRows ? p.rows : p.depth;
                bool bad = false;
                for (unsigned g = lane; g < (unsigned)p.G; g += 32) {
                    const int a = __ldcg(p.offsets + g), b = __ldcg(p.offsets + g + 1);
                    bad |= a < 0 || b > most || b < a;
                }
                if (bad) gen_record_timeout(p.err + 1, 1);
            }
            __syncwarp();
        }
        if (!leader) {
            // tells the leader's warp 2 that this CTA has read a unit
            bool more = true;
            for (int j = 0; more; ++j) {
                const int s = j % C_::UNITS;
                const uint32_t parity = (uint32_t)(j / C_::UNITS) & 1u;
                if (!__all_sync(0xffffffffu, wait_unit(ready_bar + 8u * s, parity, p))) break;
                more = get_unit(unit_slots + 48u * s, un);
                if (!__all_sync(0xffffffffu,
                                wait_unit(ready_bar + 8u * (C_::UNITS + s), parity, p)))
                    break;
                if (lane == 0)
                    mbar_arrive_cluster(mapa_shared(ready_bar + 8u * (2 * C_::UNITS + s), 0));
                __syncwarp();
            }
        } else {
            Units<CG, MODE> units(p, cluster, list_arg);
            bool more = true;
            for (int j = 0; more; ++j) {
                more = units.next(p, un);
                const int s = j % C_::UNITS;
                const uint32_t parity = (uint32_t)(j / C_::UNITS - 1) & 1u;
                if (j >= C_::UNITS) {
                    bool ok = wait_unit(ready_bar + 8u * (C_::UNITS + s), parity, p);
                    if (CG == 2)
                        ok = ok && wait_unit(ready_bar + 8u * (2 * C_::UNITS + s), parity, p);
                    if (!__all_sync(0xffffffffu, ok)) break;
                }
                if (lane < CG) {  // to each CTA of the pair
                    const uint32_t to = CG == 2 ? (uint32_t)lane : crank;
                    put_unit(mapa_shared(unit_slots + 48u * s, to), un, more);
                    mbar_arrive_cluster(mapa_shared(ready_bar + 8u * s, to));
                }
                __syncwarp();
                if (S > 1 && j > 0 && more) cluster_sync_all();
            }
        }
    }

    // ------------------------------------------------------------ teardown --
    // (Relaxed: no CTA reads what another wrote after this; it only must not
    // exit, or free its TMEM, while a peer still uses its memory.)
    tc_fence_before_sync();
    if (CG == 2 || S > 1) {
        __syncwarp();
        cluster_arrive_relaxed();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<CG>(tmem_base, TMEM_COLS);
        if (lane == 0) TC_TRACE(p, 13);
    }
}

// units: work units (an upper bound where only the device knows their number);
// the grid holds as many clusters as fit the GPU at once, at most one per unit.
template <int CG, int MODE, bool P_MN, bool BF16, typename OutT, bool EPI = true>
int launch_ragged_variant(RaggedParams& rp, int64_t units, const DeviceInfo& dev,
                          cudaStream_t stream) {
    if constexpr (EPI && std::is_same_v<OutT, float> && MODE != kRagShrink)
        if (!rp.epi.active)
            return launch_ragged_variant<CG, MODE, P_MN, BF16, OutT, false>(rp, units, dev, stream);
    auto kern = ragged_kernel<CG, MODE, P_MN, BF16, OutT, EPI>;
    static std::mutex mu;
    static uint64_t configured = 0;  // bit per device
    static int pairs[64];
    const int cl = CG == 2 ? 2 : 1 << rp.split;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.blockDim = dim3(RTHREADS);
    cfg.dynamicSmemBytes = RCfg<MODE == kRagShrink && P_MN>::SMEM_BYTES;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    {
        std::lock_guard<std::mutex> lock(mu);
        const uint64_t bit = 1ull << (dev.device & 63);
        if (!(configured & bit)) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     RCfg<MODE == kRagShrink && P_MN>::SMEM_BYTES) != cudaSuccess)
                return kCuda;
            int n = dev.sm_count / 2;
            if (CG == 2) {
                cfg.gridDim = dim3(2 * n);
                int m = 0;
                if (cudaOccupancyMaxActiveClusters(&m, kern, &cfg) == cudaSuccess && m > 0) n = m;
                else cudaGetLastError();
            }
            pairs[dev.device & 63] = n;
            configured |= bit;
        }
    }
    int64_t clusters = units;
    if (MODE != kRagShrink) {
        const int64_t fit = CG == 2 ? pairs[dev.device & 63] : dev.sm_count / cl;
        if (clusters > fit) clusters = fit;
    }
    if (clusters < 1) clusters = 1;
    cfg.gridDim = dim3((unsigned)(clusters * cl));
    if (rp.pdl) {
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
    }
    cfg.stream = stream;
    if (cudaLaunchKernelEx(&cfg, kern, rp) != cudaSuccess) {
        cudaGetLastError();
        return kCuda;
    }
    note_launch();
    return kOk;
}

// The grouped products of one element type.
template <bool BF16, typename OutT>
int dispatch_ragged(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units,
                    const DeviceInfo& dev, cudaStream_t s) {
    if (mode == kRagDepth)
        return cg == 2 ? launch_ragged_variant<2, kRagDepth, true, BF16, OutT>(rp, units, dev, s)
                       : launch_ragged_variant<1, kRagDepth, true, BF16, OutT>(rp, units, dev, s);
    if (cg == 2)
        return p_mn ? launch_ragged_variant<2, kRagRows, true, BF16, OutT>(rp, units, dev, s)
                    : launch_ragged_variant<2, kRagRows, false, BF16, OutT>(rp, units, dev, s);
    return p_mn ? launch_ragged_variant<1, kRagRows, true, BF16, OutT>(rp, units, dev, s)
                : launch_ragged_variant<1, kRagRows, false, BF16, OutT>(rp, units, dev, s);
}

template <bool BF16>
int launch_lora_rows(RaggedParams& rp, int64_t blocks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kRowsThreads);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    if (cudaLaunchKernelEx(&cfg, lora_rows_kernel<BF16>, rp) != cudaSuccess) {
        cudaGetLastError();
        return kCuda;
    }
    note_launch();
    return kOk;
}

// The two launches of gemm_lora of one element type.
template <bool BF16, typename OutT>
int dispatch_lora(RaggedParams& rp, int mode, int cg, bool p_mn, int64_t units,
                  const DeviceInfo& dev, cudaStream_t s) {
    if (mode == kRagShrinkRows) return launch_lora_rows<BF16>(rp, units, s);
    if (mode == kRagShrink)
        return rp.lanes == 64
                   ? launch_ragged_variant<1, kRagShrink, true, BF16, OutT>(rp, units, dev, s)
                   : launch_ragged_variant<1, kRagShrink, false, BF16, OutT>(rp, units, dev, s);
    if (cg == 2)
        return p_mn ? launch_ragged_variant<2, kRagLora, true, BF16, OutT>(rp, units, dev, s)
                    : launch_ragged_variant<2, kRagLora, false, BF16, OutT>(rp, units, dev, s);
    return p_mn ? launch_ragged_variant<1, kRagLora, true, BF16, OutT>(rp, units, dev, s)
                : launch_ragged_variant<1, kRagLora, false, BF16, OutT>(rp, units, dev, s);
}

}  // namespace
}  // namespace libgemm
