// embed.cu -- embed_rows() and embed_rows_grad().
//
//   y_t = scale table[id_t]           (zeros where id_t is negative)
//   dtable_v = beta dtable_v + scale sum over the t with id_t = v of dy_t
//
// Both are bound by memory. The gradient sorts the tokens (a row of the table is
// then one run of the sorted list), so that every row of the table is written
// once, by one block, and its terms are added in the order of t: no atomics, and
// results that do not depend on timing.
//
// Sort: the 64-bit number (token, t) is unique, so its place in the sorted list is
// a count of smaller ones. Blocks sort 512 numbers each; then 16 runs at a time are
// merged, every number finding its place among the 15 other runs by binary
// search. 8192 tokens take two launches, 131072 three.
//
// Sums: the sorted list is cut into chunks of equal length, so that a frequent
// token's rows are shared by many blocks. A run that crosses chunks leaves one
// partial sum in each, which a last kernel adds in the order of the chunks.
//
// 8192 tokens of 32000 x 2048, bf16 to fp32, us: forward 11.5; sort 4, merge 8, list
// of pieces 4, sums and fill 47.5 (6.2 TB/s), crossing runs 8.5, some of it beside its
// neighbours: 82 together. (Filling a part of the rows beside the list of pieces and
// the crossing runs instead left the whole as it was.)
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gemm.h"
#include "internal.h"
#include "policy.h"
#include "rows.cuh"

namespace libgemm {
namespace {

bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// G elements of a row on their way: the aligned piece that begins with them, or
// (ALIGNED false) the one or two aligned pieces that hold them. The second one is
// read only where it holds one of them, else the first again, so that the reads of
// several groups are in flight together, without branches between them.
template <typename T, int G, bool ALIGNED>
struct Group {
    static constexpr int BYTES = G * (int)sizeof(T), WORDS = BYTES / 4;
    static_assert(BYTES == 8 || BYTES == 16, "whole words");
    Piece<BYTES> a, b;

    __device__ __forceinline__ void load(const T* p) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        const uint32_t off = ALIGNED ? 0 : (uint32_t)(at % BYTES);
        const Piece<BYTES>* from = reinterpret_cast<const Piece<BYTES>*>(at - off);
        a = from[0];
        if constexpr (!ALIGNED) b = from[off ? 1 : 0];
    }
    // The elements; p as in load().
    __device__ __forceinline__ void values(const T* p, float (&out)[G]) const {
        uint32_t r[WORDS];
        if constexpr (ALIGNED) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) r[i] = a.w[i];
        } else {
            uint32_t w[2 * WORDS];
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = a.w[i], w[WORDS + i] = b.w[i];
            const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) % BYTES);
            // selections, not branches: the groups of several pieces interleave
            const uint32_t skip = off / 4, bits = off % 4 * 8;
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                uint32_t lo = 0, hi = 0;
#pragma unroll
                for (int k = 0; k < WORDS; ++k) {
                    if (skip == (uint32_t)k) lo = w[i + k];
                    if (skip == (uint32_t)k && i + k + 1 < 2 * WORDS) hi = w[i + k + 1];
                }
                r[i] = __funnelshift_r(lo, hi, bits);
            }
        }
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < G; ++i) out[i] = __uint_as_float(r[i]);
        } else {
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const uint16_t h = (uint16_t)(r[i / 2] >> (i % 2 * 16));
                out[i] = to_f32(*reinterpret_cast<const T*>(&h));
            }
        }
    }
};

// G elements to a row at `p`, in one store where that is aligned.
template <typename T, int G>
__device__ __forceinline__ void store_group(T* p, const float (&v)[G]) {
    alignas(16) T o[G];
#pragma unroll
    for (int i = 0; i < G; ++i) o[i] = from_f32<T>(v[i]);
    constexpr int BYTES = G * (int)sizeof(T);
    if (reinterpret_cast<uintptr_t>(p) % (BYTES < 16 ? BYTES : 16) == 0) {
        if constexpr (BYTES == 8) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(o);
#pragma unroll
        for (int j = 0; j < BYTES / 16; ++j)
            reinterpret_cast<uint4*>(p)[j] = reinterpret_cast<uint4*>(o)[j];
    } else {
#pragma unroll
        for (int i = 0; i < G; ++i) p[i] = o[i];
    }
}

struct EmbedArgs {
    int64_t M, V, K;
    const int32_t* ids;
    const void* table;
    int64_t ldt;
    float scale;
    void* y;
    int64_t ldy;
    ErrWord* err;
};

// A warp takes a piece of a row: kPieces groups of G elements in each lane, all in
// flight at once (2 KB of a 16-bit row). Groups are aligned in y; the elements
// before the first and after the last whole group are copied one by one.
constexpr int kPieces = 4;
template <typename T, typename O, bool ALIGNED>
__global__ void __launch_bounds__(256) embed_kernel(const EmbedArgs a, int pieces) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int G = 16 / (int)sizeof(O) < 16 / (int)sizeof(T) ? 16 / (int)sizeof(O)
                                                                : 16 / (int)sizeof(T);
    const int lane = threadIdx.x & 31;
    const int64_t unit = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
    const int64_t t = unit / pieces, piece = unit - t * pieces;
    gemm_ptx::pdl_wait();
    if (t >= a.M) return;
    const int id = a.ids[t];
    if (id >= a.V && lane == 0) report_bad_value(a.err);
    const bool named = id >= 0 && id < a.V;
    const T* from = static_cast<const T*>(a.table) + (named ? (int64_t)id * a.ldt : 0);
    O* to = static_cast<O*>(a.y) + t * a.ldy;
    const int past = (int)(reinterpret_cast<uintptr_t>(to) % (G * sizeof(O))) / (int)sizeof(O);
    int64_t head = past ? G - past : 0;
    if (head > a.K) head = a.K;
    const int64_t tail = head + (a.K - head) / G * G;
    const int64_t c0 = head + (piece * kPieces * 32 + lane) * G;
    Group<T, G, ALIGNED> v[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j)
        if (named && c0 + j * 32 * G < tail) v[j].load(from + c0 + j * 32 * G);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        if (c0 + j * 32 * G >= tail) continue;
        float f[G] = {};
        if (named) v[j].values(from + c0 + j * 32 * G, f);
#pragma unroll
        for (int e = 0; e < G; ++e) f[e] *= a.scale;
        store_group<O, G>(to + c0 + j * 32 * G, f);
    }
    if (piece == 0)
        for (int64_t i = lane; i < head + (a.K - tail); i += 32) {
            const int64_t c = i < head ? i : tail + (i - head);
            to[c] = from_f32<O>(named ? a.scale * to_f32(from[c]) : 0.f);
        }
}

// ------------------------------------------------------------------ sort --
// The number of a token: its row of the table above its place in the list;
// tokens that do not count come last.
constexpr int kTile = 512;       // numbers that a block sorts
constexpr int kMerge = 16;       // runs merged in one pass
constexpr uint32_t kNone = 0xffffffffu;

__device__ __forceinline__ uint32_t token_of(uint64_t x) { return (uint32_t)(x >> 32); }

// Bitonic: a thread holds numbers i and i + kTile / 2; partners nearer than a warp
// are exchanged by shuffles, the others through shared memory.
__global__ void __launch_bounds__(kTile / 2)
    sort_tiles_kernel(const int32_t* __restrict__ ids, int64_t M, int64_t V,
                      uint64_t* __restrict__ out, uint32_t* __restrict__ counts, ErrWord* err) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int HALF = kTile / 2;
    __shared__ uint64_t x[kTile];
    gemm_ptx::pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x < 2) counts[threadIdx.x] = 0;  // for a later kernel
    const int64_t base = (int64_t)blockIdx.x * kTile;
    const int i0 = threadIdx.x;
    uint64_t v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t t = base + i0 + h * HALF;
        v[h] = ~0ull;  // past the list: after every number
        if (t >= M) continue;
        const int id = ids[t];
        if (id >= V) report_bad_value(err);
        v[h] = ((uint64_t)(id >= 0 && id < V ? (uint32_t)id : kNone) << 32) | (uint32_t)t;
    }
#pragma unroll
    for (int k = 2; k <= kTile; k *= 2) {
#pragma unroll
        for (int j = k / 2; j > 0; j /= 2) {
            if (j == HALF) {  // the thread's own two (k == kTile: ascending)
                const uint64_t lo = v[0] < v[1] ? v[0] : v[1];
                v[1] = v[0] < v[1] ? v[1] : v[0];
                v[0] = lo;
                continue;
            }
            uint64_t other[2];
            if (j < 32) {
                other[0] = __shfl_xor_sync(0xffffffffu, v[0], j);
                other[1] = __shfl_xor_sync(0xffffffffu, v[1], j);
            } else {
                __syncthreads();
                x[i0] = v[0];
                x[i0 + HALF] = v[1];
                __syncthreads();
                other[0] = x[i0 ^ j];
                other[1] = x[(i0 ^ j) + HALF];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = i0 + h * HALF;
                const bool small = ((i & j) == 0) == ((i & k) == 0);  // keeps the smaller
                v[h] = (other[h] < v[h]) == small ? other[h] : v[h];
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (base + i0 + h * HALF < M) out[base + i0 + h * HALF] = v[h];
}

// Each number finds its place in the 16 runs by binary searches side by side: first
// among a part of the run in shared memory (all of it up to kSamples numbers, else
// every (run / kFew)th), then, of long runs, in what lies between. In global memory
// alone, where every block starts at the same few numbers, 8192 numbers took 26 us.
constexpr int kMergeThreads = 128;
constexpr int kSamples = kTile, kFew = 128;
__global__ void __launch_bounds__(kMergeThreads)
    sort_merge_kernel(const uint64_t* __restrict__ in, uint64_t* __restrict__ out, int64_t M,
                      uint32_t run) {
    gemm_ptx::pdl_launch_dependents();
    extern __shared__ uint64_t sample[];  // kMerge x samples of a run
    gemm_ptx::pdl_wait();
    const uint32_t n = (uint32_t)M;
    const uint64_t group = (uint64_t)run * kMerge;
    const uint64_t i = (uint64_t)blockIdx.x * kMergeThreads + threadIdx.x;
    const uint64_t base = (uint64_t)blockIdx.x * kMergeThreads / group * group;
    const uint32_t each = run <= kSamples ? run : kFew, stride = run / each;
    // the last of each `stride` numbers, as if the list went on with larger ones
#pragma unroll 16
    for (uint32_t k = threadIdx.x; k < kMerge * each; k += kMergeThreads) {
        const uint64_t at = base + (uint64_t)k * stride + stride - 1;
        sample[k] = at < n ? in[at] : ~0ull;
    }
    __syncthreads();
    if (i >= n) return;
    const uint64_t x = in[i];
    uint32_t pos[kMerge];  // samples of each run that are below x
#pragma unroll
    for (int r = 0; r < kMerge; ++r) pos[r] = 0;
    for (uint32_t w = each / 2; w > 0; w /= 2)
#pragma unroll
        for (int r = 0; r < kMerge; ++r)
            if (sample[r * each + pos[r] + w - 1] < x) pos[r] += w;
    uint64_t at = base;
#pragma unroll
    for (int r = 0; r < kMerge; ++r) {
        if (sample[r * each + pos[r]] < x) ++pos[r];
        pos[r] *= stride;
    }
    // fewer than `stride` numbers more (none where a run's samples are all below)
    for (uint32_t w = stride / 2; w > 0; w /= 2) {
        uint64_t got[kMerge];
#pragma unroll
        for (int r = 0; r < kMerge; ++r) {
            const uint64_t p = base + (uint64_t)r * run + pos[r] + w - 1;
            got[r] = in[p < n ? p : n - 1];
        }
#pragma unroll
        for (int r = 0; r < kMerge; ++r)
            if (pos[r] < run && base + (uint64_t)r * run + pos[r] + w - 1 < n && got[r] < x)
                pos[r] += w;
    }
#pragma unroll
    for (int r = 0; r < kMerge; ++r) at += pos[r];
    out[at] = x;
}

// ------------------------------------------------------------------ sums --
struct EmbedGradArgs {
    int64_t M, V, K;
    const uint64_t* sorted;
    const void* dy;
    int64_t lddy;
    float scale, beta;
    void* dtable;
    int64_t lddt;
    float* part;      // chunks x 2 x kp: a crossing run's sum at the chunk's begin, and at its end
    int64_t kp;       // K rounded up to whole groups
    int chunk;        // sorted numbers of a chunk
    int chunks;
    int col_warps;    // warps that share a row's columns in the last kernel
    int col_blocks;   // and blocks (of 128 groups) before that
    const struct RunPiece* pieces;
    const uint32_t* crossing;
    const uint32_t* counts;  // of pieces and crossing
    int64_t sum_blocks;
};

constexpr int kSumThreads = 128, kSumWarps = kSumThreads / 32;
constexpr int kFillRows = 8;      // rows of the table that a block looks after: small pieces,
                                  // so that the last blocks end together

// The first place of the sorted list whose token is not below `token`; the whole
// warp calls it (32 places at a time: 4 steps for 2^20 numbers).
__device__ __forceinline__ int64_t first_at(const uint64_t* sorted, int64_t M, uint64_t token) {
    const uint64_t x = token << 32;
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, n = M;  // the place is lo .. lo + n
    while (n > 0) {
        const int64_t step = (n + 31) / 32;  // probes at the ends of 32 shares
        const int64_t at = lane * step + step - 1;
        const bool below = at < n && sorted[lo + at] < x;
        const int shares = __popc(__ballot_sync(0xffffffffu, below));
        lo += shares * step;
        n = n - shares * step < step - 1 ? n - shares * step : step - 1;
    }
    return lo;
}

// G sums of a run to its row of the table; the whole warp calls it.
template <typename O, int G>
__device__ __forceinline__ void write_sum(const EmbedGradArgs& a, uint32_t token, int64_t c,
                                          const float (&sum)[G]) {
    O* row = static_cast<O*>(a.dtable) + (int64_t)token * a.lddt;
    float v[G];
#pragma unroll
    for (int e = 0; e < G; ++e) v[e] = a.scale * sum[e];
    if (a.beta != 0.f) add_row<O, G>(row, a.K, c, a.beta, v);
    store_row<O, G>(row, a.K, c, v);
}

// The list of the pieces: runs of one token within a chunk, in any order (they are
// summed apart from each other, so results do not depend on it).
struct RunPiece {
    uint32_t token, row;    // row: of the piece's first number
    uint32_t at;            // its place in the sorted list
    uint32_t count_begins;  // numbers << 2 | goes on after the chunk << 1 | begins here
};

// counts: of the pieces, and of `crossing`, the chunks in which a run begins that
// goes on in the next one (one at most in a chunk).
__global__ void __launch_bounds__(256)
    embed_pieces_kernel(const uint64_t* __restrict__ sorted, int64_t M, int chunk,
                        RunPiece* __restrict__ pieces, uint32_t* __restrict__ crossing,
                        uint32_t* __restrict__ counts) {
    gemm_ptx::pdl_launch_dependents();
    __shared__ uint32_t first[9];
    gemm_ptx::pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const uint64_t x = p < M ? sorted[p] : ~0ull;
    const uint32_t token = token_of(x);
    const bool begins = token != kNone && (p == 0 || token_of(sorted[p - 1]) != token);
    const bool piece = token != kNone && (begins || p % chunk == 0);
    const uint32_t mask = __ballot_sync(0xffffffffu, piece);
    if (lane == 0) first[w] = __popc(mask);
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t sum = 0;
        for (int i = 0; i < 8; ++i) {
            const uint32_t n = first[i];
            first[i] = sum;
            sum += n;
        }
        const uint32_t base = sum ? atomicAdd(counts, sum) : 0;
        for (int i = 0; i < 8; ++i) first[i] += base;
    }
    __syncthreads();
    if (!piece) return;
    // the piece's end: the last number of the chunk that is not above the token's
    int64_t end = (p / chunk + 1) * chunk;
    if (end > M) end = M;
    int64_t lo = p + 1, hi = end;
    while (lo < hi) {
        const int64_t mid = lo + (hi - lo) / 2;
        if (token_of(sorted[mid]) == token) lo = mid + 1;
        else hi = mid;
    }
    const bool goes_on = lo == end && end < M && token_of(sorted[end]) == token;
    if (begins && goes_on) crossing[atomicAdd(counts + 1, 1u)] = (uint32_t)(p / chunk);
    pieces[first[w] + __popc(mask & ((1u << lane) - 1))] =
        RunPiece{token, (uint32_t)x, (uint32_t)p,
                 (uint32_t)(lo - p) << 2 | (goes_on ? 2u : 0u) | (begins ? 1u : 0u)};
}

// Two roles, side by side.
//
// Sums (the first a.sum_blocks blocks): a block takes a piece of the list and 128
// groups of columns at a time, every sum_blocks'th; it reads the next one's entry
// beside this one's rows. Few registers and little code, so that many pieces are
// in flight: most have a row or two. (A warp that walked through a chunk and wrote
// wherever a run ended took three times as long.)
//
// The others: the rows of the table that no token names become zeros, or beta times
// what they hold.
template <typename T, typename O, bool ALIGNED>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const EmbedGradArgs a) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int G = 16 / (int)sizeof(T), AHEAD = ALIGNED ? 4 : 2;  // rows in flight
    __shared__ uint32_t named;
    __shared__ int64_t range[2];
    gemm_ptx::pdl_wait();
    if (blockIdx.x < a.sum_blocks) {
        // every `stride`th piece, and always the same columns
        const uint32_t pieces = a.counts[0], stride = (uint32_t)a.sum_blocks / a.col_blocks;
        const int64_t c =
            ((int64_t)(blockIdx.x % (uint32_t)a.col_blocks) * kSumThreads + threadIdx.x) * G;
        const bool whole = c + G <= a.K;
        uint32_t at = blockIdx.x / (uint32_t)a.col_blocks;
        RunPiece next{};
        if (at < pieces) next = a.pieces[at];
        for (; at < pieces; at += stride) {
            const RunPiece piece = next;
            if (at + stride < pieces) next = a.pieces[at + stride];
            const int count = (int)(piece.count_begins >> 2);
            const bool begins = piece.count_begins & 1u, goes_on = piece.count_begins & 2u;
            float sum[G] = {};
            for (int j0 = 0; j0 < count; j0 += AHEAD) {
                Group<T, G, ALIGNED> v[AHEAD];
                const T* from[AHEAD];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    if (j0 + j >= count) continue;
                    const uint32_t row = j0 + j == 0 ? piece.row
                                                     : (uint32_t)a.sorted[piece.at + j0 + j];
                    from[j] = static_cast<const T*>(a.dy) + (int64_t)row * a.lddy + c;
                    if (whole) v[j].load(from[j]);
                }
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    if (j0 + j >= count) continue;
                    float f[G] = {};
                    if (whole) {
                        v[j].values(from[j], f);
                    } else {  // a group that the row's end cuts
                        for (int e = 0; e < G; ++e)
                            if (c + e < a.K) f[e] = to_f32(from[j][e]);
                    }
#pragma unroll
                    for (int e = 0; e < G; ++e) sum[e] += f[e];
                }
            }
            if (begins && !goes_on) {
                write_sum<O, G>(a, piece.token, c, sum);
            } else if (c < a.K) {
                const int64_t chunk = piece.at / (uint32_t)a.chunk;
                float4* to =
                    reinterpret_cast<float4*>(a.part + (chunk * 2 + (begins ? 1 : 0)) * a.kp + c);
#pragma unroll
                for (int k = 0; k < G / 4; ++k)
                    to[k] = make_float4(sum[4 * k], sum[4 * k + 1], sum[4 * k + 2],
                                        sum[4 * k + 3]);
            }
        }
        return;
    }
    // Rows without a token: which of these kFillRows have one stands in the sorted
    // list between the places of the first and the last.
    const int64_t v0 = (blockIdx.x - a.sum_blocks) * kFillRows;
    const int rows = a.V - v0 < kFillRows ? (int)(a.V - v0) : kFillRows;
    if (threadIdx.x == 0) named = 0;
    if (threadIdx.x < 64) {
        const int w = threadIdx.x >> 5;
        const int64_t at = first_at(a.sorted, a.M, v0 + w * rows);
        if ((threadIdx.x & 31) == 0) range[w] = at;
    }
    __syncthreads();
    for (int64_t p = range[0] + threadIdx.x; p < range[1]; p += kSumThreads) {
        const uint32_t bit = 1u << (token_of(a.sorted[p]) - (uint32_t)v0);
        if (!(named & bit)) atomicOr(&named, bit);
    }
    __syncthreads();
    constexpr int GO = 16 / (int)sizeof(O);
    for (int r = 0; r < rows; ++r) {
        if (named >> r & 1) continue;
        O* row = static_cast<O*>(a.dtable) + (v0 + r) * a.lddt;
        int64_t count = a.K;
        if (a.lddt == a.K)  // rows without gaps between them: as one
            for (; r + 1 < rows && !(named >> (r + 1) & 1); ++r) count += a.K;
        if (a.beta != 0.f) {
            for (int64_t c = threadIdx.x; c < count; c += kSumThreads)
                row[c] = from_f32<O>(a.beta * to_f32(row[c]));
            continue;
        }
        const int past = (int)(reinterpret_cast<uintptr_t>(row) % 16) / (int)sizeof(O);
        int64_t head = past ? GO - past : 0;
        if (head > count) head = count;
        const int64_t tail = head + (count - head) / GO * GO;
#pragma unroll 4
        for (int64_t c = head + (int64_t)threadIdx.x * GO; c < tail; c += kSumThreads * GO)
            *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
        for (int64_t i = threadIdx.x; i < head + (count - tail); i += kSumThreads)
            row[i < head ? i : tail + (i - head)] = from_f32<O>(0.f);
    }
}

// A run that crosses chunks: a block for each 32 groups of its columns adds its
// partial sums, each warp a quarter of the chunks in order, and then the quarters.
template <typename T, typename O>
__global__ void __launch_bounds__(kSumThreads) embed_cross_kernel(const EmbedGradArgs a) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int G = 16 / (int)sizeof(T), AHEAD = 64 / G;
    __shared__ float4 quarter[kSumWarps - 1][G / 4][32];
    gemm_ptx::pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const uint32_t runs = a.counts[1], stride = gridDim.x / (uint32_t)a.col_warps;
    const int64_t c = ((int64_t)(blockIdx.x % (uint32_t)a.col_warps) * 32 + lane) * G;
    for (uint32_t at = blockIdx.x / (uint32_t)a.col_warps; at < runs; at += stride) {
        const int64_t chunk = a.crossing[at];
        const uint32_t token = token_of(a.sorted[(chunk + 1) * a.chunk]);
        const int64_t end = first_at(a.sorted, a.M, (uint64_t)token + 1);
        const bool in = c < a.K;  // the other lanes only take part in the stores
        // chunk's own sum is its second one; those of the chunks after it their first
        const int64_t more = (end - 1) / a.chunk - chunk;
        const int64_t k0 = chunk + 1 + more * w / kSumWarps;
        const int64_t k1 = chunk + 1 + more * (w + 1) / kSumWarps;
        float sum[G] = {};
        auto add = [&](const float4 (&v)[G / 4]) {
#pragma unroll
            for (int q = 0; q < G / 4; ++q) {
                sum[4 * q] += v[q].x;
                sum[4 * q + 1] += v[q].y;
                sum[4 * q + 2] += v[q].z;
                sum[4 * q + 3] += v[q].w;
            }
        };
        auto load = [&](float4 (&v)[G / 4], int64_t slot) {
#pragma unroll
            for (int q = 0; q < G / 4; ++q)
                v[q] = in ? reinterpret_cast<const float4*>(a.part + slot * a.kp + c)[q]
                          : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        if (w == 0) {
            float4 v[G / 4];
            load(v, chunk * 2 + 1);
            add(v);
        }
        for (int64_t k = k0; k < k1; k += AHEAD) {
            float4 v[AHEAD][G / 4];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (k + j < k1) load(v[j], (k + j) * 2);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (k + j < k1) add(v[j]);
        }
        if (w > 0) {
#pragma unroll
            for (int q = 0; q < G / 4; ++q)
                quarter[w - 1][q][lane] =
                    make_float4(sum[4 * q], sum[4 * q + 1], sum[4 * q + 2], sum[4 * q + 3]);
        }
        __syncthreads();
        if (w == 0) {
            for (int o = 0; o < kSumWarps - 1; ++o) {
                float4 v[G / 4];
#pragma unroll
                for (int q = 0; q < G / 4; ++q) v[q] = quarter[o][q][lane];
                add(v);
            }
            write_sum<O, G>(a, token, c, sum);
        }
        __syncthreads();  // the next run's quarters go to the same place
    }
}

bool rows_ok(const void* p, int64_t rows, int64_t K, int64_t ld, int es) {
    return p && aligned_to(p, es) && ld >= K &&
           (__int128)(rows - 1) * ld + K <= (__int128)(INT64_MAX / es);
}

bool rows_aligned(const void* p, int64_t ld, int es) {
    return aligned_to(p, 16) && ld * es % 16 == 0;
}

int embed(int64_t M, int64_t V, int64_t K, const int32_t* ids, const void* table, int64_t ldt,
          float scale, void* y, int64_t ldy, int dtype, cudaStream_t s) {
    if (dtype < GEMM_F32 || dtype > GEMM_BF16_BF16) return kInvalidArg;
    if (M < 0 || V < 0 || K < 0 || M > INT32_MAX || V > INT32_MAX || K > INT32_MAX)
        return kInvalidArg;
    if (M == 0 || K == 0) return kOk;
    const int ts = dtype == GEMM_F32 ? 4 : 2, os = dtype <= GEMM_BF16_F32 ? 4 : 2;
    if (!ids || !aligned_to(ids, 4) || !rows_ok(y, M, K, ldy, os)) return kInvalidArg;
    if (V > 0 && !rows_ok(table, V, K, ldt, ts)) return kInvalidArg;
    DeviceInfo* dev = nullptr;
    int rc = current_device_info(&dev, nullptr);
    if (rc != kOk) return rc;
    const void* ptrs[3] = {ids, V > 0 ? table : nullptr, y};
    rc = check_device_pointers(ptrs, 3, dev->device);
    if (rc != kOk) return rc;
    const EmbedArgs a{M, V, K, ids, table, ldt, scale, y, ldy, dev->err_word};
    const int64_t group = 16 / (os > ts ? os : ts);
    const int64_t pieces = (K + group * 32 * kPieces - 1) / (group * 32 * kPieces);
    if (M * pieces > (int64_t)INT32_MAX * 8) return kUnsupported;
    const dim3 grid((unsigned)((M * pieces + 7) / 8));
    // groups start on 16-byte boundaries in both
    const bool aligned = rows_aligned(table, ldt, ts) && rows_aligned(y, ldy, os);
    auto run = [&](auto t, auto o) {
        using T = decltype(t);
        using O = decltype(o);
        return launch_dependent(aligned ? embed_kernel<T, O, true> : embed_kernel<T, O, false>,
                                grid, dim3(256), 0, s, a, (int)pieces);
    };
    switch (dtype) {
        case GEMM_F32: return run(float{}, float{});
        case GEMM_F16_F32: return run(__half{}, float{});
        case GEMM_BF16_F32: return run(__nv_bfloat16{}, float{});
        case GEMM_F16_F16: return run(__half{}, __half{});
        default: return run(__nv_bfloat16{}, __nv_bfloat16{});
    }
}

int embed_grad(int64_t M, int64_t V, int64_t K, const int32_t* ids, const void* dy, int64_t lddy,
               float scale, void* dtable, int64_t lddt, float beta, int dtype, cudaStream_t s) {
    if (dtype < GEMM_F32 || dtype > GEMM_BF16_BF16) return kInvalidArg;
    if (M < 0 || V < 0 || K < 0 || M > INT32_MAX || V > INT32_MAX || K > INT32_MAX)
        return kInvalidArg;
    if (V == 0 || K == 0) return kOk;
    const int ts = dtype == GEMM_F32 ? 4 : 2, os = dtype <= GEMM_BF16_F32 ? 4 : 2;
    if (!rows_ok(dtable, V, K, lddt, os)) return kInvalidArg;
    if (M > 0 && (!ids || !aligned_to(ids, 4) || !rows_ok(dy, M, K, lddy, ts))) return kInvalidArg;
    if (M == 0 && beta == 1.f) return kOk;
    DeviceInfo* dev = nullptr;
    cudaMemPool_t pool = nullptr;
    int rc = current_device_info(&dev, &pool);
    if (rc != kOk) return rc;
    const void* ptrs[3] = {M > 0 ? ids : nullptr, M > 0 ? dy : nullptr, dtable};
    rc = check_device_pointers(ptrs, 3, dev->device);
    if (rc != kOk) return rc;

    EmbedGradArgs a{};
    a.M = M;
    a.V = V;
    a.K = K;
    a.dy = dy;
    a.lddy = lddy;
    a.scale = scale;
    a.beta = beta;
    a.dtable = dtable;
    a.lddt = lddt;
    const int group = 16 / ts;
    a.kp = up(K, 16);
    a.chunk = embed_chunk(M);
    a.chunks = (int)((M + a.chunk - 1) / a.chunk);
    a.col_warps = (int)((K + (int64_t)group * 32 - 1) / ((int64_t)group * 32));
    a.col_blocks = (a.col_warps + kSumWarps - 1) / kSumWarps;
    // 32 for each SM, where there may be as many pieces: five times those that fit, so
    // that the blocks which meet a frequent token's pieces do not end last (8: 3 % of
    // the call's time more); as many for each of the columns
    const int64_t stride = (dev->sm_count * 32 + a.col_blocks - 1) / a.col_blocks;
    a.sum_blocks = (M < stride ? M : stride) * a.col_blocks;
    // of chunks, one run at most goes on from each
    const int64_t cross = (dev->sm_count * 8 + a.col_warps - 1) / a.col_warps;
    const int64_t cross_blocks = (a.chunks < cross ? a.chunks : cross) * a.col_warps;
    const int64_t fill = beta == 1.f ? 0 : (V + kFillRows - 1) / kFillRows;
    if (a.sum_blocks + fill > INT32_MAX || cross_blocks > INT32_MAX) return kUnsupported;
    Scratch scratch{pool, s, dev->device};
    const int64_t list = up(M * 8, 256);
    char* mem = nullptr;
    if (M > 0) {
        const int64_t part = up((int64_t)a.chunks * 2 * a.kp * 4, 256);
        const int64_t bytes = 4 * list + part + 8 + (int64_t)a.chunks * 4;
        mem = static_cast<char*>(scratch.get((size_t)bytes));
        if (!mem) return kCuda;
        uint64_t* in = reinterpret_cast<uint64_t*>(mem);
        uint64_t* out = reinterpret_cast<uint64_t*>(mem + list);
        uint32_t* counts = reinterpret_cast<uint32_t*>(mem + 4 * list + part);
        rc = launch_dependent(sort_tiles_kernel, dim3((unsigned)((M + kTile - 1) / kTile)),
                              dim3(kTile / 2), 0, s, ids, M, V, in, counts, dev->err_word);
        for (int64_t run = kTile; rc == kOk && run < M; run *= kMerge) {
            const int smem = kMerge * (run <= kSamples ? (int)run : kFew) * 8;
            rc = allow_smem(sort_merge_kernel, kMerge * kSamples * 8, *dev);
            if (rc == kOk)
                rc = launch_dependent(sort_merge_kernel,
                                      dim3((unsigned)((M + kMergeThreads - 1) / kMergeThreads)),
                                      dim3(kMergeThreads), smem, s, (const uint64_t*)in, out, M,
                                      (uint32_t)run);
            std::swap(in, out);
        }
        a.sorted = in;
        RunPiece* pieces = reinterpret_cast<RunPiece*>(mem + 2 * list);
        if (rc == kOk)
            rc = launch_dependent(embed_pieces_kernel, dim3((unsigned)((M + 255) / 256)),
                                  dim3(256), 0, s, a.sorted, M, a.chunk, pieces, counts + 2,
                                  counts);
        a.pieces = pieces;
        a.crossing = counts + 2;
        a.counts = counts;
        a.part = reinterpret_cast<float*>(mem + 4 * list);
    }
    const bool aligned = rows_aligned(dy, lddy, ts);
    auto run = [&](auto t, auto o) {
        using T = decltype(t);
        using O = decltype(o);
        int r = rc;
        if (r == kOk && a.sum_blocks + fill > 0)
            r = launch_dependent(aligned ? embed_sum_kernel<T, O, true>
                                         : embed_sum_kernel<T, O, false>,
                                 dim3((unsigned)(a.sum_blocks + fill)), dim3(kSumThreads), 0, s, a);
        if (r == kOk && a.chunks > 1)
            r = launch_dependent(embed_cross_kernel<T, O>, dim3((unsigned)cross_blocks),
                                 dim3(kSumThreads), 0, s, a);
        return r;
    };
    switch (dtype) {
        case GEMM_F32: rc = run(float{}, float{}); break;
        case GEMM_F16_F32: rc = run(__half{}, float{}); break;
        case GEMM_BF16_F32: rc = run(__nv_bfloat16{}, float{}); break;
        case GEMM_F16_F16: rc = run(__half{}, __half{}); break;
        default: rc = run(__nv_bfloat16{}, __nv_bfloat16{}); break;
    }
    scratch.release();
    return rc;
}

}  // namespace
}  // namespace libgemm

using namespace libgemm;

extern "C" {

int embed_rows(int64_t M, int64_t V, int64_t K, const int32_t* ids, const void* table, int64_t ldt,
               float scale, void* y, int64_t ldy, int dtype, void* stream) {
    try {
        return embed(M, V, K, ids, table, ldt, scale, y, ldy, dtype,
                     static_cast<cudaStream_t>(stream));
    } catch (...) {
        return kCuda;
    }
}

int embed_rows_grad(int64_t M, int64_t V, int64_t K, const int32_t* ids, const void* dy,
                    int64_t lddy, float scale, void* dtable, int64_t lddt, float beta, int dtype,
                    void* stream) {
    try {
        return embed_grad(M, V, K, ids, dy, lddy, scale, dtable, lddt, beta, dtype,
                          static_cast<cudaStream_t>(stream));
    } catch (...) {
        return kCuda;
    }
}

}  // extern "C"
