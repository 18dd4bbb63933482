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
// token's rows are shared by many blocks. A block adds up the runs within its
// chunk; a run that crosses chunks leaves one partial sum in each, which a last
// kernel adds in the order of the chunks.
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

// G elements of a row, from any alignment: the one or two aligned 16-byte (or
// smaller) pieces that hold them, shifted together. The second piece is read only
// when it holds one of them.
template <typename T, int G>
__device__ __forceinline__ void load_group(const T* p, float (&out)[G]) {
    constexpr int BYTES = G * (int)sizeof(T);  // 4, 8 or 16
    constexpr int WORDS = BYTES / 4;
    static_assert(BYTES == 8 || BYTES == 16, "whole words");
    struct alignas(BYTES) Piece { uint32_t w[WORDS]; };
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint32_t off = (uint32_t)(at % BYTES);
    const Piece* from = reinterpret_cast<const Piece*>(at - off);
    uint32_t w[2 * WORDS];
    const Piece a = from[0];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = a.w[i];
    if (off) {
        const Piece b = from[1];
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[WORDS + i] = b.w[i];
        uint32_t r[WORDS];
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
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = r[i];
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < G; ++i) out[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const uint16_t h = (uint16_t)(w[i / 2] >> (i % 2 * 16));
            out[i] = to_f32(*reinterpret_cast<const T*>(&h));
        }
    }
}

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
template <typename T, typename O>
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
    float v[kPieces][G];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
#pragma unroll
        for (int e = 0; e < G; ++e) v[j][e] = 0.f;
        if (named && c0 + j * 32 * G < tail) load_group<T, G>(from + c0 + j * 32 * G, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        if (c0 + j * 32 * G >= tail) continue;
#pragma unroll
        for (int e = 0; e < G; ++e) v[j][e] *= a.scale;
        store_group<O, G>(to + c0 + j * 32 * G, v[j]);
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
                      uint64_t* __restrict__ out, ErrWord* err) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int HALF = kTile / 2;
    __shared__ uint64_t x[kTile];
    gemm_ptx::pdl_wait();
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
    int col_blocks;   // blocks that share a chunk's columns
    int64_t sum_blocks;
};

constexpr int kSumThreads = 128;
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

// G elements of a row from column c on, held by each lane of a warp one group after
// the other (the whole warp calls it, lanes past the row's end too). Where the row
// starts on no 16-byte boundary, lanes hand the beginning of their groups to the
// lane before, so that all but the warp's first and last elements still leave in
// 16-byte stores (2-byte stores of rows of 1803 took two thirds of the kernel).
template <typename O, int G>
__device__ __forceinline__ void store_row(O* row, int64_t K, int64_t c, const float (&v)[G]) {
    constexpr int ES = (int)sizeof(O), WORDS = G * ES / 4, PER = 16 / ES;
    static_assert(WORDS % 4 == 0, "whole 16-byte pieces");
    alignas(16) O o[G];
#pragma unroll
    for (int e = 0; e < G; ++e) o[e] = from_f32<O>(v[e]);
    uint32_t w[WORDS + 4];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = reinterpret_cast<uint32_t*>(o)[i];
    const int lane = threadIdx.x & 31;
    // bytes up to the next 16-byte boundary: the same for every lane
    const uint32_t skip = (uint32_t)(-(intptr_t)reinterpret_cast<uintptr_t>(row + c)) & 15u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[WORDS + i] = __shfl_down_sync(0xffffffffu, w[i], 1);
    const uint32_t words = skip / 4, bits = skip % 4 * 8;
    uint32_t s[WORDS];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (words == (uint32_t)k) {
                lo = w[i + k];
                if (i + k + 1 < WORDS + 4) hi = w[i + k + 1];
            }
        s[i] = __funnelshift_r(lo, hi, bits);
    }
    const int ahead = (int)skip / ES;  // elements that the lane before takes
#pragma unroll
    for (int g = 0; g < WORDS / 4; ++g) {
        const int64_t c0 = c + ahead + g * PER;  // the piece's first element
        // of the last lane's last piece the next warp has the rest
        const int have = lane == 31 && g == WORDS / 4 - 1 ? PER - ahead : PER;
        if (c0 + PER <= K && have == PER) {
            *reinterpret_cast<uint4*>(row + c0) =
                make_uint4(s[4 * g], s[4 * g + 1], s[4 * g + 2], s[4 * g + 3]);
        } else {
            const O* piece = reinterpret_cast<const O*>(s + 4 * g);
#pragma unroll
            for (int e = 0; e < PER; ++e)
                if (e < have && c0 + e < K) row[c0 + e] = piece[e];
        }
    }
    if (lane == 0) {  // no lane before
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (e < ahead && c + e < K) row[c + e] = o[e];
    }
}

template <typename O, int G>
__device__ __forceinline__ void write_sum(const EmbedGradArgs& a, uint32_t token, int64_t c,
                                          const float (&sum)[G]) {
    O* row = static_cast<O*>(a.dtable) + (int64_t)token * a.lddt;
    float v[G];
#pragma unroll
    for (int e = 0; e < G; ++e) {
        v[e] = a.scale * sum[e];
        if (a.beta != 0.f && c + e < a.K) v[e] = fmaf(a.beta, to_f32(row[c + e]), v[e]);
    }
    __syncwarp();  // every lane has read what it adds to
    store_row<O, G>(row, a.K, c, v);
}

// The first a.sum_blocks blocks add up chunks; the others look after the rows of
// the table that no token names (zeros, or beta times what they hold).
template <typename T, typename O>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const EmbedGradArgs a) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int G = 16 / (int)sizeof(T);
    __shared__ uint32_t named;
    __shared__ int64_t range[2];
    gemm_ptx::pdl_wait();
    if (blockIdx.x < a.sum_blocks) {
        const int64_t chunk = blockIdx.x / a.col_blocks;
        const int64_t c = ((int64_t)(blockIdx.x % a.col_blocks) * kSumThreads + threadIdx.x) * G;
        const bool out = c >= a.K;  // such lanes only take part in the stores
        if (__all_sync(0xffffffffu, out)) return;
        const int64_t p0 = chunk * a.chunk;
        const int64_t p1 = p0 + a.chunk < a.M ? p0 + a.chunk : a.M;
        const uint32_t before = p0 > 0 ? token_of(a.sorted[p0 - 1]) : kNone;
        const uint32_t after = p1 < a.M ? token_of(a.sorted[p1]) : kNone;
        const bool whole = c + G <= a.K;
        float sum[G] = {};
        uint32_t token = token_of(a.sorted[p0]);
        bool crossing = p0 > 0 && before == token;  // the run began in an earlier chunk
        constexpr int AHEAD = 4;
        for (int64_t p = p0; p < p1; p += AHEAD) {
            uint32_t tok[AHEAD];
            float v[AHEAD][G];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                tok[j] = kNone;
                if (p + j >= p1) continue;
                const uint64_t x = a.sorted[p + j];
                tok[j] = token_of(x);
                if (tok[j] == kNone) continue;
                const T* row = static_cast<const T*>(a.dy) + (int64_t)(uint32_t)x * a.lddy + c;
                if (out) {
#pragma unroll
                    for (int e = 0; e < G; ++e) v[j][e] = 0.f;
                } else if (whole) {
                    load_group<T, G>(row, v[j]);
                } else {
#pragma unroll
                    for (int e = 0; e < G; ++e) v[j][e] = c + e < a.K ? to_f32(row[e]) : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                if (p + j >= p1) continue;
                if (tok[j] != token) {  // the run before ends here
                    if (token != kNone) {
                        if (crossing) {
                            float* to = a.part + chunk * 2 * a.kp + c;
                            if (!out)
#pragma unroll
                                for (int e = 0; e < G; ++e) to[e] = sum[e];
                        } else {
                            write_sum<O, G>(a, token, c, sum);
                        }
                    }
                    token = tok[j];
                    crossing = false;
#pragma unroll
                    for (int e = 0; e < G; ++e) sum[e] = 0.f;
                }
                if (token != kNone) {
#pragma unroll
                    for (int e = 0; e < G; ++e) sum[e] += v[j][e];
                }
            }
        }
        if (token == kNone) return;
        const bool goes_on = p1 < a.M && after == token;
        if (crossing || goes_on) {
            float* to = a.part + (chunk * 2 + (crossing ? 0 : 1)) * a.kp + c;
            if (!out)
#pragma unroll
                for (int e = 0; e < G; ++e) to[e] = sum[e];
        } else {
            write_sum<O, G>(a, token, c, sum);
        }
        return;
    }
    // Rows without a token: which of these kFillRows have one stands in the sorted
    // list between the places of the first and the last.
    const int64_t v0 = (int64_t)(blockIdx.x - a.sum_blocks) * kFillRows;
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

// A run that crosses chunks: the block of the chunk where it begins adds its
// partial sums in order.
template <typename T, typename O>
__global__ void __launch_bounds__(kSumThreads) embed_cross_kernel(const EmbedGradArgs a) {
    gemm_ptx::pdl_launch_dependents();
    constexpr int G = 16 / (int)sizeof(T);
    gemm_ptx::pdl_wait();
    const int64_t chunk = blockIdx.x / a.col_blocks;
    const int64_t c = ((int64_t)(blockIdx.x % a.col_blocks) * kSumThreads + threadIdx.x) * G;
    const int64_t p0 = chunk * a.chunk, p1 = p0 + a.chunk;
    if (p1 >= a.M) return;
    const uint32_t token = token_of(a.sorted[p1 - 1]);
    if (token == kNone || token_of(a.sorted[p1]) != token) return;   // no run goes on
    if (p0 > 0 && token_of(a.sorted[p0 - 1]) == token &&
        token_of(a.sorted[p0]) == token) return;                     // it began earlier
    const int64_t end = first_at(a.sorted, a.M, (uint64_t)token + 1);
    const bool out = c >= a.K;
    if (__all_sync(0xffffffffu, out)) return;
    const int64_t last = (end - 1) / a.chunk;
    float sum[G];
    const float* from = a.part + (chunk * 2 + 1) * a.kp + c;
#pragma unroll
    for (int e = 0; e < G; ++e) sum[e] = out ? 0.f : from[e];
    constexpr int AHEAD = 64 / G;
    for (int64_t k = chunk + 1; k <= last; k += AHEAD) {
        float4 more[AHEAD][G / 4];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
#pragma unroll
            for (int q = 0; q < G / 4; ++q)
                if (k + j <= last && !out)
                    more[j][q] =
                        reinterpret_cast<const float4*>(a.part + (k + j) * 2 * a.kp + c)[q];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (k + j <= last && !out) {
#pragma unroll
                for (int q = 0; q < G / 4; ++q) {
                    sum[4 * q] += more[j][q].x;
                    sum[4 * q + 1] += more[j][q].y;
                    sum[4 * q + 2] += more[j][q].z;
                    sum[4 * q + 3] += more[j][q].w;
                }
            }
    }
    write_sum<O, G>(a, token, c, sum);
}

bool rows_ok(const void* p, int64_t rows, int64_t K, int64_t ld, int es) {
    return p && aligned_to(p, es) && ld >= K &&
           (__int128)(rows - 1) * ld + K <= (__int128)(INT64_MAX / es);
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
    auto run = [&](auto kern) {
        return launch_dependent(kern, grid, dim3(256), 0, s, a, (int)pieces);
    };
    switch (dtype) {
        case GEMM_F32: return run(embed_kernel<float, float>);
        case GEMM_F16_F32: return run(embed_kernel<__half, float>);
        case GEMM_BF16_F32: return run(embed_kernel<__nv_bfloat16, float>);
        case GEMM_F16_F16: return run(embed_kernel<__half, __half>);
        default: return run(embed_kernel<__nv_bfloat16, __nv_bfloat16>);
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
    a.col_blocks = (int)((K + (int64_t)group * kSumThreads - 1) / ((int64_t)group * kSumThreads));
    a.sum_blocks = (int64_t)a.chunks * a.col_blocks;
    const int64_t fill = beta == 1.f ? 0 : (V + kFillRows - 1) / kFillRows;
    if (a.sum_blocks + fill > INT32_MAX) return kUnsupported;
    Scratch scratch{pool, s, dev->device};
    const int64_t list = up(M * 8, 256);
    char* mem = nullptr;
    if (M > 0) {
        mem = static_cast<char*>(scratch.get((size_t)(2 * list + (int64_t)a.chunks * 2 * a.kp * 4)));
        if (!mem) return kCuda;
        uint64_t* in = reinterpret_cast<uint64_t*>(mem);
        uint64_t* out = reinterpret_cast<uint64_t*>(mem + list);
        rc = launch_dependent(sort_tiles_kernel, dim3((unsigned)((M + kTile - 1) / kTile)),
                              dim3(kTile / 2), 0, s, ids, M, V, in, dev->err_word);
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
        a.part = reinterpret_cast<float*>(mem + 2 * list);
    }
    auto run = [&](auto sum, auto cross) {
        int r = rc;
        if (r == kOk && a.sum_blocks + fill > 0)
            r = launch_dependent(sum, dim3((unsigned)(a.sum_blocks + fill)), dim3(kSumThreads), 0,
                                 s, a);
        if (r == kOk && a.chunks > 1)
            r = launch_dependent(cross, dim3((unsigned)a.sum_blocks), dim3(kSumThreads), 0, s, a);
        return r;
    };
    switch (dtype) {
        case GEMM_F32: rc = run(embed_sum_kernel<float, float>, embed_cross_kernel<float, float>); break;
        case GEMM_F16_F32: rc = run(embed_sum_kernel<__half, float>, embed_cross_kernel<__half, float>); break;
        case GEMM_BF16_F32:
            rc = run(embed_sum_kernel<__nv_bfloat16, float>, embed_cross_kernel<__nv_bfloat16, float>);
            break;
        case GEMM_F16_F16: rc = run(embed_sum_kernel<__half, __half>, embed_cross_kernel<__half, __half>); break;
        default:
            rc = run(embed_sum_kernel<__nv_bfloat16, __nv_bfloat16>,
                     embed_cross_kernel<__nv_bfloat16, __nv_bfloat16>);
            break;
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
