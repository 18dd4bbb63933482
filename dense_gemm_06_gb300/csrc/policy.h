// policy.h -- the host-side choices the library makes automatically, as plain
// C++ (no CUDA), so they can be compiled and checked on a machine without a
// GPU: the FFMA kernel's K-split of the tiles left after its last full round,
// whether a K-major fp32 operand is first transposed, the row panels
// gemm_host() pipelines its copies over, and the tensor-core kernel's tile
// shape and split of its last round.
#pragma once

#include <cstdint>
#include <numeric>

#ifdef __CUDACC__
#define LIBGEMM_BOTH __host__ __device__ __forceinline__
#else
#define LIBGEMM_BOTH inline
#endif

namespace libgemm {

// K-split of the FFMA kernel's tail. Tiles 0 .. dp_tiles-1 (raster order) run
// whole; every later tile is cut into `splits` K-slices of `kt_slice` k-tiles,
// one CTA each, summed in slice order by a fixup kernel.
struct TailSplit {
    int dp_tiles;
    int splits;
    int kt_slice;
};

// Model: an SM finishes the same tile work per unit of time whether it holds
// one CTA or two, so a launch takes (most tile-units on one SM) x (work of a
// unit). With P SMs and T tiles, q = T / P full rounds and r = T mod P tail
// tiles: whole, the tail adds one round; cut into s K-slices (one CTA each),
// it adds ceil(r s / P) / s. split_mode 0 (automatic): with no full round (the
// GPU under-filled) or at least two, the s in 2..8 (slices of at least 32
// k-tiles: shorter ones spend too much of their time filling the pipeline
// and writing partial sums) with the shortest time, if that saves at least
// 10% against no split. With exactly one full round the model fails
// (measured at 2048^3: 4 slices ran 12% slower than whole tiles), so that
// case is not split. split_mode 1: never. split_mode 2 (tests): always cut
// the last wave of `slots` resident CTAs (all tiles if T < slots) into 2-4
// slices. slots <= 0 (occupancy unknown) or sm_count <= 0: never.
inline TailSplit plan_tail_split(int64_t T, int slots, int sm_count, int nkt, int split_mode) {
    TailSplit t{(int)T, 1, nkt};
    if (split_mode == 1 || slots <= 0 || sm_count <= 0 || T <= 0) return t;
    if (split_mode == 2) {
        int64_t r = T % slots;
        if (r == 0) r = T < slots ? T : slots;
        int s = (int)(slots / r);
        s = s < 2 ? 2 : (s > 4 ? 4 : s);
        t.dp_tiles = (int)(T - r);
        t.splits = s;
        t.kt_slice = (nkt + s - 1) / s;
        return t;
    }
    const int64_t P = sm_count, q = T / P, r = T % P;
    if (r == 0 || q == 1) return t;
    const double whole = (double)(q + 1);
    double best = whole;
    int best_s = 1;
    for (int s = 2; s <= 8 && nkt >= 32 * s; ++s) {
        const double time = (double)q + (double)((r * s + P - 1) / P) / s;
        if (time < best - 1e-9) {
            best = time;
            best_s = s;
        }
    }
    if (best_s == 1 || best > 0.9 * whole) return t;
    t.dp_tiles = (int)(T - r);
    t.splits = best_s;
    t.kt_slice = (nkt + best_s - 1) / best_s;
    return t;
}

// Stream-K plan of the TMA-fed FFMA kernel: tiles 0 .. dp_tiles-1 (raster
// order) run whole, one CTA each; the k-iterations of the later tiles (tile
// t, k-tile k is iteration (t - dp_tiles) * nkt + k) are shared evenly by
// sk_ctas CTAs, each taking one contiguous range (at most one tile's worth,
// so at most two tile segments). sk_ctas == 0: no stream-K.
struct StreamK {
    int dp_tiles;
    int sk_ctas;
};

// Model: with P SMs, `slots` = 2 P resident CTAs (two per SM) and
// P <= T < 2 P tiles, whole tiles give some SMs two tiles, so the launch
// takes two tiles' time. Sharing every tile's k-iterations evenly over all
// `slots` CTAs gives every CTA, wherever the block scheduler places it, the
// same T / (2 P) tiles' worth, so every SM does T / P: split_mode 0
// (automatic) uses that when it saves at least 10% (T <= 1.8 P) and a tile
// has at least 32 k-tiles. (Mixing whole-tile CTAs with stream-K CTAs
// measured slower: co-resident CTAs come from neighbouring block indices,
// so two whole tiles could share an SM.) split_mode 3 (tests): stream-K
// whatever it saves, a third of the tiles whole and the rest shared by 3/2
// as many CTAs as tiles. Otherwise no stream-K.
inline StreamK plan_stream_k(int64_t T, int slots, int sm_count, int nkt, int split_mode) {
    StreamK s{(int)T, 0};
    if (T <= 0 || nkt <= 0) return s;
    if (split_mode == 3) {
        const int64_t dp = T / 3, rest = T - dp;
        const int64_t g = rest + (rest + 1) / 2;
        s.dp_tiles = (int)dp;
        s.sk_ctas = (int)(g < rest * nkt ? g : rest * nkt);  // no CTA without iterations
        return s;
    }
    if (split_mode != 0 || sm_count <= 0 || slots < 2 * sm_count || nkt < 32) return s;
    const int64_t P = sm_count;
    if (T < P || T >= 2 * P || 10 * T > 18 * P) return s;
    s.dp_tiles = 0;
    s.sk_ctas = (int)(2 * P);
    return s;
}

// Whether to give the FFMA kernel an MN-major copy of a K-major operand.
// The kernel reads MN-major tiles with 16-byte copies (or TMA) and K-major
// ones with transposing 4-byte copies (about 10% slower at 8192^3); a
// transpose costs two HBM passes over the operand, 48/n of the GEMM time for
// the other dimension n, so it pays when n >= 512 and the product is large
// enough for the extra launch not to matter. mode: 0 automatic, 1 never,
// 2 always.
inline bool want_transpose(int64_t other_dim, int64_t M, int64_t N, int64_t K, int mode) {
    if (mode == 1) return false;
    if (mode == 2) return true;
    return other_dim >= 512 && (double)M * (double)N * (double)K >= 2147483648.0;
}

// gemm_host(): with more than one row panel and an fp32 C, the first panel
// runs as host_k_pieces() GEMMs over consecutive ranges of K, each adding its
// product to C (fused epilogue, beta = 1), so the first one starts once a
// quarter of B (and of that panel's A) is in instead of all of it. A 16-bit C
// would be rounded between the pieces, and K below 4 x 256 would leave pieces
// too short to pay for their launches: those run whole (1 piece).
constexpr int kHostKPieces = 4;
inline int host_k_pieces(int64_t panels, int out_bytes, int64_t K) {
    return panels > 1 && out_bytes == 4 && K >= kHostKPieces * 256 ? kHostKPieces : 1;
}

// First k of piece j of `pieces` (j == pieces: K): K j / pieces rounded up to
// a multiple of 64, so every piece but the last covers whole 64-deep k-tiles.
inline int64_t host_k_bound(int64_t K, int pieces, int j) {
    if (j >= pieces) return K;
    const int64_t b = (K * j / pieces + 63) / 64 * 64;
    return b < K ? b : K;
}

// Rows of the normalised C per gemm_host() panel: a whole number of waves of
// the kernel that computes it (so no panel adds a partial wave), at most
// about 8 panels; M itself when the product is too small (M N K < 1e10) for
// overlapping the copies with compute to pay. f32: the FFMA kernel (128 x
// 128 tiles, `ctas_per_sm` resident CTAs per SM); otherwise the tensor-core
// kernel with CTA group `cta_group` (1: 128 x 256 tiles, one CTA each; 2:
// 256 x 256 tiles per CTA pair) and operand multicast (2: clusters of two
// pairs, 512 x 256).
inline int64_t host_panel_rows(int64_t M, int64_t N, int64_t K, bool f32, int ctas_per_sm,
                               int cta_group, int multicast, int sm_count) {
    if (K == 0 || (double)M * (double)N * (double)K < 1.0e10) return M;
    const bool one_cta = f32 || cta_group == 1;
    const int64_t tm = f32 ? 128 : (cta_group == 1 ? 128 : (multicast == 2 ? 512 : 256));
    const int64_t tn = f32 ? 128 : 256;
    int64_t slots = f32 ? (int64_t)sm_count * ctas_per_sm
                        : (int64_t)sm_count / (one_cta ? 1 : (multicast == 2 ? 4 : 2));
    if (slots < 1) slots = 1;
    const int64_t tiles_m = (M + tm - 1) / tm, tiles_n = (N + tn - 1) / tn;
    int64_t r = slots / std::gcd(slots, tiles_n);
    while (r * 8 < tiles_m) r *= 2;
    return r >= tiles_m ? M : r * tm;
}

// Tensor-core tile shape: the CTA group (1: a CTA per 128-row tile, 2: a
// CTA pair per 256-row tile) and the tile width in columns (64, 128 or 256;
// at least 64 per CTA of the group). cta_group / tile_n: the value asked for,
// or 0 for automatic. Automatic: a problem with fewer 256 x 256 pair tiles
// than a quarter of the SMs (fewer than half the CTA pairs would get one)
// runs one CTA per tile, in the narrowest width that still fits every tile
// into one round over the SMs, so its epilogue (the part of a short problem
// that takes longest) is spread over as many SMs as possible; everything
// else runs 256 x 256 pair tiles. Operand multicast always runs 256 x 256
// pair tiles.
struct TcShape {
    int cta_group;
    int tile_n;
};

inline TcShape plan_tc_shape(int64_t M, int64_t N, int cta_group, int tile_n, bool multicast,
                             int sm_count) {
    TcShape s{cta_group, tile_n};
    if (multicast) return TcShape{2, 256};
    if (s.cta_group != 1 && s.cta_group != 2) {
        const int64_t pair_tiles = ((M + 255) / 256) * ((N + 255) / 256);
        s.cta_group = pair_tiles * 4 < (int64_t)sm_count ? 1 : 2;
    }
    if (s.tile_n != 64 && s.tile_n != 128 && s.tile_n != 256) {
        s.tile_n = 256;
        if (s.cta_group == 1)
            for (int tn = 64; tn < 256; tn *= 2)
                if (((M + 127) / 128) * ((N + tn - 1) / tn) <= (int64_t)sm_count) {
                    s.tile_n = tn;
                    break;
                }
    }
    if (s.tile_n < 64 * s.cta_group) s.tile_n = 64 * s.cta_group;
    return s;
}

// The first tile (raster order) of a tensor-core launch that runs as two
// work units of half the width. With `slots` clusters resident at once and T
// tiles, the last round holds r = T mod slots tiles; when at least two rounds
// are needed and r is at most half the slots, splitting those r tiles makes
// the last round take half as long (2 r half units still fit in one round):
// at 8192^3 (1024 pair tiles on 76 pairs, r = 36) 14 rounds become 13.5.
// split_mode 0: automatic; 1: never; 2 (tests): split the last round's
// tiles (every tile when there is less than one round) whatever it saves.
// Half units need half the width to hold 64 columns per CTA; operand
// multicast never splits. Returns T for no split.
inline int64_t plan_tc_split(int64_t T, int64_t slots, int tile_n, int cta_group,
                             bool multicast, int split_mode) {
    if (split_mode == 1 || multicast || tile_n / 2 < 64 * cta_group || slots <= 0 || T <= 0)
        return T;
    int64_t r = T % slots;
    if (split_mode == 2) {
        if (r == 0) r = T < slots ? T : slots;
        return T - r;
    }
    if (T <= slots || r == 0 || 2 * r > slots) return T;
    return T - r;
}

// How a product over ragged groups runs: CTAs per unit (a CTA pair takes 256
// features, a single CTA 128), rows of a full unit, and CTAs that share a
// unit's depth as a cluster (single CTAs only).
struct RaggedShape {
    int cta_group;
    int tile_w;
    int split;
};

// The kernels' round-ups, in unsigned numbers: a group may have up to 2^31 - 1
// rows, whose round-up no longer fits an int. Units of a group of `rows` rows;
// rows that a unit spans when `rows` of its group are left; 64-deep blocks of
// the summed rows [k0, k_end).
LIBGEMM_BOTH int ragged_units(int rows, int tile_w) {
    return (int)(((unsigned)rows + (unsigned)tile_w - 1u) / (unsigned)tile_w);
}
LIBGEMM_BOTH int ragged_width(int rows, int step, int most) {
    const unsigned up = ((unsigned)rows + (unsigned)step - 1u) / (unsigned)step * (unsigned)step;
    return (int)(up < (unsigned)most ? up : (unsigned)most);
}
LIBGEMM_BOTH int ragged_blocks(int k0, int k_end) {
    return (int)(((unsigned)(k_end - k0) + 63u) / 64u);
}

// Largest power of two <= 8 that keeps units * split within the SMs (half of them
// for clusters of 8: a GPC holds few of those, and 16 no longer run at once) and
// six k-blocks for each CTA of the cluster. Measured, with and without a split:
// one row of 4096 x 4096 9.0 us and 17.7 us, 4 groups of 2 rows of 512 x 7168
// 11.7 and 28.0, 2 of 30 rows of 1024 x 2048 7.9 and 11.9. Clusters of 8 and of
// 4: 20 rows of 1024 x 4096 (8 units) 7.8 and 9.4, 8 groups of one row of 256 x
// 4096 (16 units) 14.5 and 9.2.
inline int plan_ragged_split(int64_t units, int64_t num_kb, int sm_count) {
    int s = 1;
    while (s < 8 && units * (2 * s) <= (s == 4 ? sm_count / 2 : sm_count) &&
           num_kb >= 6 * (2 * s))
        s *= 2;
    return s;
}

// What the epilogue of a grouped product does to C.
enum RaggedOut {
    kOut16,          // 16-bit, written
    kOut16Reads,     // 16-bit, read first (beta)
    kOut32,          // fp32, written as it is summed
    kOut32Epilogue,  // fp32, added to by global additions, or bias / activation, beta 0
    kOut32Reads,     // fp32, read first (any other beta)
};

// gemm_grouped: M rows in G groups (their sizes are known on the device only),
// N features, num_kb k-blocks. Pairs where a group has more than 64 rows on
// average and their units fill the SMs. Measured, 64 groups of 1536 x 2048,
// single CTAs and pairs: 8 rows each 70.2 and 71.4 us, 64 rows 75.0 and 75.4, 96
// rows 78.9 and 78.3, 256 rows 103.7 and 92.0. A fused epilogue on fp32 results
// takes a pair's warps, with twice the columns each, longer than it saves unless
// many rounds of units (and with C read first, a long depth) hide it: 3 rounds,
// 22 k-blocks (16 groups, 4096 rows, 2048 features) beta 1 41.0 and 51.6 us, other
// beta 43.1 and 71.6, bias and GELU 40.2 and 64.1; 7 rounds, 32 k-blocks 83.2 and
// 92.6, 85.3 and 115.1, 85.4 and 110.2; 15 rounds, 64 k-blocks 505 and 372, 513 and
// 473, 526 and 442; 37 rounds, 32 k-blocks 533 and 457, 578 and 688, 630 and 574.
// (16-bit results with the same epilogues: pairs at most 3% slower, up to 36%
// faster.)
inline RaggedShape plan_grouped(int64_t G, int64_t M, int64_t N, int64_t num_kb, int sm_count,
                                RaggedOut out = kOut16) {
    const int64_t groups = G < M ? G : M;  // at most this many have rows
    const int64_t avg = (M + groups - 1) / groups;
    const int64_t pair_units = (groups + M / 256) * ((N + 255) / 256);
    bool pairs = avg > 64 && pair_units * 2 > sm_count;
    if (out == kOut32Epilogue || out == kOut32Reads)
        pairs = pairs && pair_units * 2 / sm_count >= 12 && (out != kOut32Reads || num_kb >= 64);
    if (pairs) return RaggedShape{2, 256, 1};
    const int64_t units = (groups + M / 128) * ((N + 127) / 128);
    return RaggedShape{1, 128, plan_ragged_split(units, num_kb, sm_count)};
}

// gemm_grouped: whether CTA pairs count the units taken instead of walking every
// n-th one. The units' widths differ, so a fixed walk ends up to about a unit
// late; the count costs a 4-byte memset before the launch and the launch's
// overlap with what precedes it, 3 us in all. Measured, walked and counted, by
// k-blocks per unit: 64 groups, 49152 rows, 2816 features 16 203 and 207 us, 32
// 387 and 386, 64 804 and 795, 128 1567 and 1522, 224 2920 and 2790; 8 groups,
// 16384 rows, 4096 features 16 84 and 87, 64 320 and 321, 128 660 and 648, 224
// 1172 and 1164; 16 groups, 12288 rows, 2048 features 32 71 and 75, 64 132 and
// 136, 128 259 and 262, 224 501 and 486. So from 64 k-blocks on, with two rounds
// of units at least; between 64 and 128 neither is ahead by more than 3%.
inline bool plan_grouped_ticket(const RaggedShape& s, int64_t M, int64_t N, int64_t num_kb,
                                int sm_count) {
    return s.cta_group == 2 && num_kb >= 64 && (M / 256) * ((N + 255) / 256) >= sm_count;
}

// gemm_grouped_k: G results of M x N, `avg` summed rows each on average. Pairs
// move fewer operands per product; single CTAs store a result with half the
// columns per epilogue warp, which counts where C is read or the sums are short.
// Measured, single CTAs and pairs (us; rounds: pair units per pair):
//   kOut16          8 of 1536 x 1664, 64 to 1000 rows 20.4 to 46.5, 17.3 to 38.5; 77
//                   of 256 x 256 9.9 to 29.1, 10.3 to 30.5
//   kOut16Reads     3 rounds 44 and 55, 7 69 and 91, 16 275 and 308, 20 225 and
//                   270, 40 713 and 719, 74 1459 and 1444
//   kOut32          300 rows, 1 round 15.4 and 17.1, 3 24.4 and 28.2, 4 28.3 and
//                   30.2, 6 41.5 and 39.4, 13 68.8 and 60.8; 800 rows, 1 round 21.6
//                   and 22.5, 3 36.3 and 31.0, 4 43.2 and 41.1
//   kOut32Epilogue  beta 1, 40 rounds, 64, 300, 768 and 1500 rows 266 and 276, 285
//                   and 295, 365 and 336, 585 and 465; 768 rows, 13 rounds 126 and
//                   124, 7 73 and 78, 3 50 and 58. ReLU alike: 768 rows, 13 rounds
//                   107 and 102, 300 rows 73 and 86
//   kOut32Reads     74 rounds, 64, 768 and 1500 rows 765 and 1293, 849 and 1267,
//                   1146 and 1369; 3 rounds, 64 rows 30 and 51
inline RaggedShape plan_grouped_k(int64_t G, int64_t M, int64_t N, int sm_count,
                                  RaggedOut out = kOut16, int64_t avg = 0) {
    const RaggedShape pairs{2, 256, 1}, single{1, 128, 1};
    const int64_t pair_units = G * ((M + 255) / 256) * ((N + 255) / 256);
    if (pair_units * 2 <= sm_count) return single;
    const int64_t rounds = pair_units * 2 / sm_count;
    switch (out) {
        case kOut16: return pairs;
        case kOut16Reads: return rounds >= 32 ? pairs : single;
        case kOut32: return rounds >= 5 || (rounds >= 3 && avg >= 512) ? pairs : single;
        case kOut32Epilogue: return rounds >= 8 && avg >= 704 ? pairs : single;
        default: return single;
    }
}

// gemm_lora: the expand's shape, and the shrink's: rows_blocks > 0 -- few rows,
// plain dot products in that many blocks, beside scan_blocks that look over LB
// (whole calls on 4096 x 4096 with 24 adapters, dot products and tensor cores:
// 48 rows of rank 16 16.3 and 23.1 us, 128 rows of rank 16 21.1 and 28.3, 64
// rows of rank 64 31.2 and 31.5) --, else lanes per unit, rows per tile, split
// and chains (clusters that share the parts of a row tile's list). slot: lanes
// per adapter; ranks up to 32 run the narrow ring (64 lanes and rows, two
// k-blocks per stage: a tile of requests one after the other seldom has more
// than two adapters). listed: most adapters of a list.
struct LoraShape {
    RaggedShape expand;
    int lanes;
    int rows_blocks, scan_blocks;
    int shrink_w, shrink_split, chains;
};

inline LoraShape plan_lora(int64_t M, int64_t N, int64_t num_kb, int64_t listed, int slot,
                           int sm_count) {
    LoraShape s{};
    const int64_t pair_units = ((M + 255) / 256) * ((N + 255) / 256);
    if (M > 128 && pair_units * 2 > sm_count) {
        s.expand = RaggedShape{2, 256, 1};
    } else {
        int w = 16;
        while (w < 128 && w < M) w *= 2;
        // More rows than a unit: narrower units before a split of the depth. Which
        // is faster hangs on the rows' adapters, which only the device knows.
        // Requests one after the other (19 rows each, rank 24), units of 64 and of
        // 128 rows: 66 shapes of 129 to 900 rows, 65 of them faster with 64, by 4 to
        // 72% (611 rows of 1804 x 1544 26.2 and 37.4 us, 400 of 1024 x 4096 26.2 and
        // 30.6; 200 of 1804 x 4096 28.9 and 27.8). Another adapter in every row, 8
        // adapters of rank 16: 26.5 and 31.4, 26.9 and 25.3, 29.2 and 27.3; 40
        // adapters: 60.0 and 56.5, 57.9 and 54.1, 46.7 and 45.1.
        if (M > 128 && ((M + 127) / 128) * ((N + 127) / 128) * 2 <= sm_count) w = 64;
        const int64_t units = ((M + w - 1) / w) * ((N + 127) / 128);
        s.expand = RaggedShape{1, w, plan_ragged_split(units, num_kb, sm_count)};
    }
    s.lanes = slot <= 32 ? 64 : 128;
    s.shrink_w = s.expand.tile_w < s.lanes ? s.expand.tile_w : s.lanes;
    if (M > 128 && (M + 127) / 128 * 2 <= sm_count) s.shrink_w = 64;
    const int64_t parts = (listed * slot + s.lanes - 1) / s.lanes;
    const int64_t tiles = (M + s.shrink_w - 1) / s.shrink_w;
    s.shrink_split = plan_ragged_split(tiles, num_kb, sm_count);
    const int64_t chains = sm_count / (tiles * s.shrink_split);
    s.chains = (int)(chains < 1 ? 1 : (chains > parts ? parts : chains));
    if (M <= 128 && M * slot <= 4096) {
        s.rows_blocks = (int)(M * (slot / 4));
        // 16 blocks look over 512 KB of LB in one pass of their loads. Measured, 16
        // and 64 blocks (us): 1 row of rank 16 and 4096 features (128 KB) 13.1 and
        // 13.4, 1 of rank 128 (1 MB) 12.5 and 11.1, 16 of rank 16 (2 MB) 13.0 and
        // 12.4, 24 (3 MB) 16.9 and 14.1, 16 of rank 128 (16 MB) 58.9 and 29.6; 16 of
        // rank 16 and 1024 features (512 KB) 9.3 and 9.6, 24 (768 KB) 10.4 and 10.6
        s.scan_blocks = listed * slot * N * 2 < (1 << 20) ? 16 : 64;
    }
    return s;
}

}  // namespace libgemm
