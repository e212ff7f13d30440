// The embedding table's lookup and gradient for gfx950.  Formulas and
// conventions: lso_ops.h.
//
// Lookup: one wave per token and run of columns; bound by the rows it moves.
//
// Gradient: the positions are sorted by token (a stable radix sort, so the
// positions of a token stay in ascending order), then every table row is
// written once by the wave that owns it, which finds its run of positions in
// the sorted tokens: no atomics, and one rounding of an FP32 sum.  A token
// that occurs often would keep one wave busy for long, so runs longer than
// kRun positions are summed in parts of the sorted order, kRun positions
// each, and a second launch joins a run's parts in order.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>
#include <vector>

#include "lso_bf16.h"
#include "lso_launch.h"
#include "lso_ops.h"
#include "lso_runtime.h"

namespace lso {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kRun = 32;            // positions per part of a long run
constexpr uint32_t kMaxDigitBits = 10;
constexpr uint32_t kMaxBins = 1u << kMaxDigitBits;
constexpr uint32_t kSortThreads = 256;
constexpr uint32_t kMaxSortGroups = 64;  // every group reads all groups' counts
constexpr uint32_t kMinSortTile = 512;
constexpr uint32_t kRankSort = 4096;     // up to so many tokens are sorted by counting
constexpr uint64_t kMaxGroups = (1ull << 24) - 1;   // workgroups of a launch: 256 lanes each, under 2^32 in all

// What passes the caches (non-temporal).  Measured with outputs in turn, so
// that none is still cached: the gradient's table always (257 tokens of width
// 2048 33.0 against 40.5 us, 32768 of width 4096 161 against 168 us); where
// the rows of a call exceed the eight XCDs' L2s (4 MB each), the rows that a
// lookup writes (16384 tokens of width 2048 16.9 against 18.5 us) and a
// gradient reads (131072 of width 8192 827 against 852 us; small ones lose: 257
// tokens 46 against 34 us).  Not the table's rows that a lookup reads, which
// tokens share (29.6 us).
constexpr uint64_t kL2Bytes = 32ull << 20;

// The sorted positions do not change while a gradient kernel runs, and a
// wave reads the same one in every lane: scalar loads.
#define LSO_CONST __attribute__((address_space(4)))

struct Tokens {
    const void* p;
    uint32_t n, vocab;
    bool wide;   // 64-bit
};

// The sort key: the token, or vocab for padding.
__device__ __forceinline__ uint32_t token_key(const Tokens& t, uint32_t i)
{
    const int64_t v = t.wide ? static_cast<const int64_t*>(t.p)[i] : static_cast<const int32_t*>(t.p)[i];
    return v >= 0 && v < static_cast<int64_t>(t.vocab) ? static_cast<uint32_t>(v) : t.vocab;
}

// V consecutive values of a row.  kOnce: they are not read again soon, and
// pass the caches (non-temporal).
template <int V, bool kF32, bool kOnce>
__device__ __forceinline__ void load_values(const void* base, uint64_t i, float (&v)[V])
{
    if (kF32) {
        const float* p = static_cast<const float*>(base) + i;
        if (V == 1) {
            v[0] = *p;
        } else {
#pragma unroll
            for (int e = 0; e < V; e += 4) {
                const f32x4* q = reinterpret_cast<const f32x4*>(p + e);
                const f32x4 x = kOnce ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
                for (int k = 0; k < 4 && e + k < V; ++k) v[e + k] = x[k];
            }
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(base) + i;
        if (V == 1) {
            v[0] = bf16_widen(*p);
        } else {
            const u32x4* q = reinterpret_cast<const u32x4*>(p);
            const u32x4 x = kOnce ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
            for (int k = 0; k < 4 && 2 * k + 1 < V; ++k) {
                v[2 * k] = bf16_widen(x[k] & 0xFFFFu);
                v[2 * k + 1] = bf16_widen(x[k] >> 16);
            }
        }
    }
}

template <int V, bool kF32, bool kOnce>
__device__ __forceinline__ void store_values(void* base, uint64_t i, const float (&v)[V])
{
    if (kF32) {
        float* p = static_cast<float*>(base) + i;
        if (V == 1) {
            *p = v[0];
        } else {
#pragma unroll
            for (int e = 0; e + 3 < V; e += 4) {
                const f32x4 x = {v[e], v[e + 1], v[e + 2], v[e + 3]};
                if (kOnce) __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(p + e));
                else *reinterpret_cast<f32x4*>(p + e) = x;
            }
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(base) + i;
        if (V == 1) {
            *p = static_cast<uint16_t>(bf16_rne(v[0]));
        } else {
            u32x4 x;
#pragma unroll
            for (int k = 0; k < 4 && 2 * k + 1 < V; ++k) x[k] = bf16_rne(v[2 * k]) | (bf16_rne(v[2 * k + 1]) << 16);
            if (kOnce) __builtin_nontemporal_store(x, reinterpret_cast<u32x4*>(p));
            else *reinterpret_cast<u32x4*>(p) = x;
        }
    }
}

// ------------------------------------------------------------------ lookup

struct LookupArgs {
    Tokens tokens;
    const void* table;
    void* rows;
    uint64_t ld_table, ld_rows;
    uint32_t width;
    uint32_t steps;      // column steps of one wave
    uint32_t chunks;     // waves per token
    float scale;
};

template <int V, bool kTableF32, bool kRowsF32, bool kOnce>
__global__ void __launch_bounds__(256) embed_lookup_kernel(const LookupArgs a)
{
    const uint64_t job = static_cast<uint64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const uint64_t i = job / a.chunks;
    if (i >= a.tokens.n) return;
    const uint32_t key = token_key(a.tokens, static_cast<uint32_t>(i));
    const uint32_t c0 = static_cast<uint32_t>(job % a.chunks) * a.steps * 64 * V + (threadIdx.x & 63u) * V;
#pragma unroll 4
    for (uint32_t s = 0; s < a.steps; ++s) {
        const uint32_t c = c0 + s * 64 * V;
        if (c >= a.width) break;
        float v[V];
        if (key < a.tokens.vocab) {
            load_values<V, kTableF32, false>(a.table, key * a.ld_table + c, v);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] *= a.scale;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = 0.0f;
        }
        store_values<V, kRowsF32, kOnce>(a.rows, i * a.ld_rows + c, v);
    }
}

// -------------------------------------------------------------------- sort
//
// Least significant digit first, at most kMaxDigitBits bits a pass.  Each
// group of threads owns a consecutive part of the input; counts[group][bin]
// says how many of its keys fall into each bin.

struct SortArgs {
    Tokens tokens;            // first pass: keys come from here, positions are 0 .. n-1
    const uint32_t* keys;     // later passes
    const uint32_t* pos;
    uint32_t* keys_out;
    uint32_t* pos_out;
    uint32_t* counts;
    uint32_t tile, groups;    // tile: a multiple of kSortThreads
    uint32_t shift, bits;
    bool first;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint32_t i) { return a.first ? token_key(a.tokens, i) : a.keys[i]; }

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortArgs a)
{
    __shared__ uint32_t count[kMaxBins];
    const uint32_t bins = 1u << a.bits;
    for (uint32_t b = threadIdx.x; b < bins; b += kSortThreads) count[b] = 0;
    __syncthreads();
    const uint64_t begin = static_cast<uint64_t>(blockIdx.x) * a.tile;
    for (uint32_t k = threadIdx.x; k < a.tile; k += kSortThreads)
        if (begin + k < a.tokens.n)
            atomicAdd(&count[(sort_key(a, static_cast<uint32_t>(begin + k)) >> a.shift) & (bins - 1)], 1u);
    __syncthreads();
    for (uint32_t b = threadIdx.x; b < bins; b += kSortThreads) a.counts[blockIdx.x * bins + b] = count[b];
}

__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const SortArgs a)
{
    __shared__ uint32_t base[kMaxBins];
    __shared__ uint32_t in_wave[kSortThreads / 64][kMaxBins];
    __shared__ uint32_t wave_total[kSortThreads / 64];
    const uint32_t bins = 1u << a.bits, lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    // base[b]: keys of smaller bins, and of this bin in earlier groups
    uint32_t carry = 0;
    for (uint32_t b0 = 0; b0 < bins; b0 += kSortThreads) {
        const uint32_t b = b0 + threadIdx.x;
        uint32_t total = 0, before = 0;
        if (b < bins) {
#pragma unroll 8
            for (uint32_t g = 0; g < a.groups; ++g) {
                const uint32_t c = a.counts[g * bins + b];
                if (g < blockIdx.x) before += c;
                total += c;
            }
        }
        uint32_t scan = total;   // inclusive over the wave
#pragma unroll
        for (uint32_t off = 1; off < 64; off <<= 1) {
            const uint32_t up = __shfl_up(scan, off, 64);
            if (lane >= off) scan += up;
        }
        if (lane == 63) wave_total[wave] = scan;
        __syncthreads();
        uint32_t smaller = carry;
        for (uint32_t w = 0; w < kSortThreads / 64; ++w) {
            if (w < wave) smaller += wave_total[w];
            carry += wave_total[w];
        }
        if (b < bins) base[b] = smaller + scan - total + before;
        __syncthreads();
    }
    for (uint32_t b = threadIdx.x; b < bins * (kSortThreads / 64); b += kSortThreads) (&in_wave[0][0])[b / bins * kMaxBins + b % bins] = 0;
    __syncthreads();
    const uint64_t begin = static_cast<uint64_t>(blockIdx.x) * a.tile;
    for (uint32_t k = 0; k < a.tile && begin + k < a.tokens.n; k += kSortThreads) {
        const uint64_t i = begin + k + threadIdx.x;
        const bool in = i < a.tokens.n;
        const uint32_t key = in ? sort_key(a, static_cast<uint32_t>(i)) : 0;
        const uint32_t pos = in ? (a.first ? static_cast<uint32_t>(i) : a.pos[i]) : 0;
        const uint32_t d = (key >> a.shift) & (bins - 1);
        // lanes of this wave with the same digit
        uint64_t same = __ballot(in);
        for (uint32_t bit = 0; bit < a.bits; ++bit) {
            const uint64_t set = __ballot((d >> bit) & 1u);
            same &= ((d >> bit) & 1u) ? set : ~set;
        }
        const uint32_t rank = static_cast<uint32_t>(__popcll(same & ((1ull << lane) - 1)));
        if (in && rank == 0) in_wave[wave][d] = static_cast<uint32_t>(__popcll(same));
        __syncthreads();
        if (in) {
            uint32_t at = base[d] + rank;
            for (uint32_t w = 0; w < wave; ++w) at += in_wave[w][d];
            a.keys_out[at] = key;
            a.pos_out[at] = pos;
        }
        __syncthreads();
        if (in && rank == 0) {
            atomicAdd(&base[d], in_wave[wave][d]);
            in_wave[wave][d] = 0;
        }
        __syncthreads();
    }
}

// Up to kRankSort tokens, in one launch: an element's place is the number of
// smaller keys and of equal keys before it.  A workgroup places 64 elements,
// sixteen threads count for each.
struct RankArgs {
    Tokens tokens;
    uint32_t* keys_out;
    uint32_t* pos_out;
};

__global__ void __launch_bounds__(1024) sort_by_rank_kernel(const RankArgs a)
{
    __shared__ __attribute__((aligned(16))) uint32_t keys[kRankSort];
    __shared__ uint32_t count[16][64];
    const uint32_t n = a.tokens.n, padded = (n + 63) / 64 * 64;
    for (uint32_t i = threadIdx.x; i < padded; i += 1024) keys[i] = i < n ? token_key(a.tokens, i) : 0xFFFFFFFFu;
    __syncthreads();
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, i = blockIdx.x * 64 + lane, key = keys[i];
    // wave w counts in blocks w, w + 16, ... of 64 keys: in blocks before the
    // element's an equal key counts, in later ones it does not
    uint32_t smaller = 0;
    for (uint32_t b = wave; b < padded / 64; b += 16) {
        const uint32_t* block = keys + b * 64;
        if (b == blockIdx.x) {
            for (uint32_t j = 0; j < 64; ++j) smaller += (block[j] < key || (block[j] == key && j < lane)) ? 1u : 0u;
            continue;
        }
        const uint32_t limit = b < blockIdx.x ? key + 1 : key;   // a key is at most 2^31 (but for the padding's, unused)
#pragma unroll 4
        for (uint32_t j = 0; j < 64; j += 4) {
            const u32x4 k4 = *reinterpret_cast<const u32x4*>(block + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) smaller += k4[e] < limit ? 1u : 0u;
        }
    }
    count[wave][lane] = smaller;
    __syncthreads();
    if (wave == 0 && i < n) {
        uint32_t to = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) to += count[w][lane];
        a.keys_out[to] = key;
        a.pos_out[to] = i;
    }
}

// ---------------------------------------------------------------- gradient

struct GradArgs {
    const uint32_t* keys;    // sorted
    const uint32_t* pos;
    const void* rows;
    void* table;
    float* parts;            // [block of kRun positions][first or last run][width]
    uint64_t ld_rows, ld_table;
    uint32_t n, vocab, width;
    float scale;
    bool add;
};

// First sorted position whose key is >= v, by all lanes of a wave.
__device__ __forceinline__ uint32_t find_run(const uint32_t* keys, uint32_t n, uint32_t v)
{
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t lo = 0, hi = n;   // the answer is in [lo, hi]
    while (hi > lo) {
        const uint32_t step = (hi - lo + 63) / 64;
        const uint64_t at = lo + static_cast<uint64_t>(lane) * step + step - 1;   // last of this lane's piece
        const bool below = at < hi && keys[at] < v;
        const uint32_t pieces = static_cast<uint32_t>(__popcll(__ballot(below)));
        lo += pieces * step;
        if (step == 1) return lo;
        hi = lo + step - 1 < hi ? lo + step - 1 : hi;
    }
    return lo;
}

// A value that every lane of the wave holds.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v))); }

// Sum of the rows at sorted positions [first, first + count), at columns c
// and on; first and count are the same in every lane.
template <int V, bool kRowsF32, bool kOnce>
__device__ __forceinline__ void sum_rows(const GradArgs& a, uint32_t first, uint32_t count, uint32_t c, float (&sum)[V])
{
    const LSO_CONST uint32_t* pos = reinterpret_cast<const LSO_CONST uint32_t*>(reinterpret_cast<uintptr_t>(a.pos + first));
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = 0.0f;
    uint32_t k = 0;
    for (; k + 4 <= count; k += 4) {
        float v[4][V];
#pragma unroll
        for (int x = 0; x < 4; ++x) load_values<V, kRowsF32, kOnce>(a.rows, pos[k + x] * a.ld_rows + c, v[x]);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += v[x][e];
    }
    for (; k < count; ++k) {
        float v[V];
        load_values<V, kRowsF32, kOnce>(a.rows, pos[k] * a.ld_rows + c, v);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += v[e];
    }
}

template <int V, bool kTableF32>
__device__ __forceinline__ void put_gradient(const GradArgs& a, uint32_t v, uint32_t c, float (&sum)[V])
{
    const uint64_t i = v * a.ld_table + c;
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] *= a.scale;
    if (a.add) {
        float old[V];
        load_values<V, kTableF32, false>(a.table, i, old);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += old[e];
    }
    store_values<V, kTableF32, true>(a.table, i, sum);
}

// The runs at the two ends of block b of kRun sorted positions.  first_*:
// the run of its first key, last_*: of its last, when that is another run.
struct BlockRuns {
    uint32_t key[2];
    uint32_t begin[2], count[2];   // positions inside the block, relative to its start
    bool is_long[2];               // the whole run has more than kRun positions
    bool starts_here[2];           // its first position is in this block
};

__device__ __forceinline__ BlockRuns block_runs(const GradArgs& a, uint32_t b)
{
    // lanes look at positions from kRun before the block to kRun behind it
    const uint32_t lane = threadIdx.x & 63u;
    const uint64_t p0 = static_cast<uint64_t>(b) * kRun;
    const uint32_t size = static_cast<uint32_t>(a.n - p0 < kRun ? a.n - p0 : kRun);
    const uint32_t none = 0xFFFFFFFFu;
    // lanes 0 .. 31: before the block, 32 .. 63: the block
    const bool has0 = p0 + lane >= kRun && p0 + lane - kRun < a.n;
    const uint32_t k0 = has0 ? a.keys[p0 + lane - kRun] : none;
    const bool has1 = lane < kRun && p0 + kRun + lane < a.n;
    const uint32_t k1 = has1 ? a.keys[p0 + kRun + lane] : none;
    BlockRuns r;
    r.key[0] = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(k0), kRun));
    r.key[1] = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(k0), static_cast<int>(kRun + size - 1)));
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const uint64_t w = __ballot(has0 && k0 == r.key[x]);
        const uint32_t before = static_cast<uint32_t>(__popcll(w & 0xFFFFFFFFull));
        const uint32_t inside = static_cast<uint32_t>(__popcll(w >> 32));
        const uint32_t behind = static_cast<uint32_t>(__popcll(__ballot(has1 && k1 == r.key[x])));
        r.count[x] = inside;
        r.begin[x] = x == 0 ? 0 : size - inside;
        r.is_long[x] = r.key[x] < a.vocab && before + inside + behind > kRun;
        r.starts_here[x] = before == 0;
    }
    if (r.key[0] == r.key[1]) r.is_long[1] = false;   // one run, held as the first
    return r;
}

// A wave writes some table rows; rows of long runs are left to the join.
template <int V, bool kRowsF32, bool kTableF32, bool kOnce>
__device__ __forceinline__ void grad_rows(const GradArgs& a, uint32_t v0, uint32_t rows)
{
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t v1 = a.vocab - v0 < rows ? a.vocab : v0 + rows;
    uint32_t first = uniform(find_run(a.keys, a.n, v0));
    if (first >= a.n || uniform(a.keys[first]) >= v1) {
        // no token here: most waves of a short batch
        if (a.add) return;
        float zero[V];
#pragma unroll
        for (int e = 0; e < V; ++e) zero[e] = 0.0f;
        for (uint32_t v = v0; v < v1; ++v)
            for (uint32_t c = lane * V; c < a.width; c += 64 * V) store_values<V, kTableF32, true>(a.table, v * a.ld_table + c, zero);
        return;
    }
    for (uint32_t v = v0; v < v1; ++v) {
        const uint64_t at = static_cast<uint64_t>(first) + lane;
        const uint32_t key = at < a.n ? a.keys[at] : 0xFFFFFFFFu;
        uint32_t count = static_cast<uint32_t>(__popcll(__ballot(key == v)));
        if (count <= kRun && !(count == 0 && a.add)) {
            for (uint32_t c = lane * V; c < a.width; c += 64 * V) {
                float sum[V];
                sum_rows<V, kRowsF32, kOnce>(a, first, count, c, sum);
                put_gradient<V, kTableF32>(a, v, c, sum);
            }
        }
        if (count < 64) first += count;
        else if (v + 1 < v1) first = uniform(find_run(a.keys, a.n, v + 1));
    }
}

template <int V, bool kRowsF32, bool kOnce>
__device__ __forceinline__ void grad_parts(const GradArgs& a, uint64_t job, uint32_t chunks)
{
    static_assert(kRun == 32, "block_runs looks at half a wave");
    const uint64_t b = job / chunks;
    if (b * kRun >= a.n) return;
    const BlockRuns r = block_runs(a, static_cast<uint32_t>(b));
    const uint32_t lane = threadIdx.x & 63u, c = static_cast<uint32_t>(job % chunks) * 64 * V + lane * V;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        if (!r.is_long[x]) continue;
        const uint32_t first = uniform(static_cast<uint32_t>(b) * kRun + r.begin[x]), count = uniform(r.count[x]);
        if (c >= a.width) continue;
        float sum[V];
        sum_rows<V, kRowsF32, kOnce>(a, first, count, c, sum);
        store_values<V, true, false>(a.parts, (b * 2 + x) * static_cast<uint64_t>(a.width) + c, sum);
    }
}

// The rows of the table, and in the same launch the parts of long runs:
// part_groups workgroups of parts first, which take longest.
template <int V, bool kRowsF32, bool kTableF32, bool kOnce>
__global__ void __launch_bounds__(256) embed_grad_kernel(const GradArgs a, uint32_t part_groups, uint32_t chunks, uint32_t rows_per_wave)
{
    const uint32_t wave = uniform(threadIdx.x >> 6);
    if (blockIdx.x < part_groups) {
        grad_parts<V, kRowsF32, kOnce>(a, static_cast<uint64_t>(blockIdx.x) * 4 + wave, chunks);
        return;
    }
    const uint64_t v0 = (static_cast<uint64_t>(blockIdx.x - part_groups) * 4 + wave) * rows_per_wave;
    if (v0 < a.vocab) grad_rows<V, kRowsF32, kTableF32, kOnce>(a, static_cast<uint32_t>(v0), rows_per_wave);
}

// The parts of a long run, joined in order by the block it starts in: four
// waves take a quarter of its blocks each.
template <int V, bool kTableF32>
__global__ void __launch_bounds__(256) embed_grad_join_kernel(const GradArgs a, uint32_t chunks)
{
    __shared__ float quarter[4][64 * V];
    const uint32_t b = blockIdx.x / chunks;
    const BlockRuns r = block_runs(a, b);   // the same in every wave
    const int x = r.is_long[1] ? 1 : 0;     // a run that starts here and is long is the block's last
    if (!r.is_long[x] || !r.starts_here[x]) return;
    const uint32_t v = r.key[x], lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t c = (blockIdx.x % chunks) * 64 * V + lane * V;
    // blocks b + 1 .. last begin with v
    const uint32_t end = find_run(a.keys, a.n, v + 1), blocks = (end - 1) / kRun - b + 1;
    const uint32_t per = (blocks + 3) / 4, k0 = wave * per, k1 = k0 + per < blocks ? k0 + per : blocks;
    float sum[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = 0.0f;
    if (c < a.width) {
#pragma unroll 4
        for (uint32_t k = k0; k < k1; ++k) {
            float p[V];
            load_values<V, true, false>(a.parts, ((static_cast<uint64_t>(b) + k) * 2 + (k == 0 ? x : 0)) * a.width + c, p);
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += p[e];
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) quarter[wave][lane * V + e] = sum[e];
    __syncthreads();
    if (wave == 0 && c < a.width) {
#pragma unroll
        for (int w = 1; w < 4; ++w)
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += quarter[w][lane * V + e];
        put_gradient<V, kTableF32>(a, v, c, sum);
    }
}

// -------------------------------------------------------------------- host

constexpr uint64_t kMaxCount = (1ull << 31) - 2;

struct GradWork {
    uint64_t keys[2], pos[2], counts, parts, bytes;
};

GradWork grad_work(uint64_t n, uint64_t width)
{
    GradWork w{};
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) { const uint64_t o = at; at += (bytes + 255) / 256 * 256; return o; };
    if (n == 0) return w;
    for (int k = 0; k < 2; ++k) {
        w.keys[k] = take(4 * n);
        w.pos[k] = take(4 * n);
    }
    w.counts = take(4ull * kMaxBins * kMaxSortGroups);
    w.parts = n > kRun ? take((n + kRun - 1) / kRun * 2 * width * 4) : at;
    w.bytes = at;
    return w;
}

uint64_t elem_bytes(uint32_t dtype) { return dtype == LSO_DT_F32 || dtype == LSO_DT_I32 ? 4 : dtype == LSO_DT_I64 ? 8 : 2; }

lso_status check_embed(const lso_embed* e, bool gradient, std::vector<Interval>& iv, bool& empty)
{
    if (!e) return fail(LSO_E_INVALID, "the descriptor is NULL");
    if (e->token_dtype != LSO_DT_I32 && e->token_dtype != LSO_DT_I64) return fail(LSO_E_DTYPE, "tokens must be I32 or I64");
    for (const uint32_t d : {e->table_dtype, e->rows_dtype})
        if (d != LSO_DT_F32 && d != LSO_DT_BF16) return fail(LSO_E_DTYPE, "table and rows must be F32 or BF16");
    if ((e->flags & ~(gradient ? LSO_EMBED_ADD : 0u)) != 0) return fail(LSO_E_INVALID, "unknown flags");
    if (!std::isfinite(e->scale) || !std::isfinite(static_cast<float>(e->scale)))
        return fail(LSO_E_INVALID, "scale must be a finite FP32 number");
    if (e->n > kMaxCount || e->vocab > kMaxCount || e->width > kMaxCount || e->ld_table > kMaxCount || e->ld_rows > kMaxCount)
        return fail(LSO_E_INVALID, "n, vocab, width or a stride is too large");
    empty = e->width == 0 || e->vocab == 0 || (e->n == 0 && !gradient);
    if (empty) return LSO_OK;
    if (e->ld_table < e->width || (e->n > 0 && e->ld_rows < e->width)) return fail(LSO_E_INVALID, "a row stride is smaller than width");
    const uint64_t et = elem_bytes(e->table_dtype), er = elem_bytes(e->rows_dtype), ek = elem_bytes(e->token_dtype);
    const struct { const void* p; uint64_t count, elem; bool written; const char* name; } arr[3] = {
        {e->tokens, e->n, ek, false, "tokens"},
        {e->table, (e->vocab - 1) * e->ld_table + e->width, et, gradient, "table"},
        {e->rows, e->n ? (e->n - 1) * e->ld_rows + e->width : 0, er, !gradient, "rows"},
    };
    for (size_t i = 0; i < 3; ++i) {
        if (arr[i].count == 0) continue;
        if (!arr[i].p) return fail(LSO_E_INVALID, "%s is NULL", arr[i].name);
        const uintptr_t addr = reinterpret_cast<uintptr_t>(arr[i].p);
        if (addr % arr[i].elem != 0) return fail(LSO_E_ALIGN, "%s is not aligned to its elements", arr[i].name);
        if (!add_array(iv, addr, arr[i].count * arr[i].elem, arr[i].written, i))
            return fail(LSO_E_INVALID, "%s range wraps the address space", arr[i].name);
    }
    return LSO_OK;
}

Tokens tokens_of(const lso_embed& e)
{
    return {e.tokens, static_cast<uint32_t>(e.n), static_cast<uint32_t>(e.vocab), e.token_dtype == LSO_DT_I64};
}

// Table rows per wave of the gradient: several where most rows are empty
// (257 tokens, 32000 rows, cached: 1 row 33.6, 2 rows 30.6, 4 rows 30.0, 8 rows
// 34.8 us).
uint32_t rows_of_wave(uint64_t n, uint64_t vocab) { return n * 4 <= vocab ? 4 : 1; }

bool beyond_l2(const lso_embed& e) { return e.n * e.width * elem_bytes(e.rows_dtype) > kL2Bytes; }

// Eight values per lane, if every row starts on 16 bytes.
bool vectors(const lso_embed& e)
{
    return e.width % 8 == 0 && e.ld_table % 8 == 0 && e.ld_rows % 8 == 0 && reinterpret_cast<uintptr_t>(e.table) % 16 == 0 &&
           reinterpret_cast<uintptr_t>(e.rows) % 16 == 0;
}

lso_status too_large() { return fail(LSO_E_INVALID, "the call is too large: split it"); }

template <int V>
lso_status launch_lookup(const lso_embed& e, hipStream_t s)
{
    LookupArgs a{};
    a.tokens = tokens_of(e);
    a.table = e.table;
    a.rows = e.rows;
    a.ld_table = e.ld_table;
    a.ld_rows = e.ld_rows;
    a.width = static_cast<uint32_t>(e.width);
    a.scale = static_cast<float>(e.scale);
    const uint64_t columns = (e.width + 64 * V - 1) / (64 * V);
    a.steps = 1;
    while (a.steps < 4 && e.n * columns / (2 * a.steps) >= 8192) a.steps *= 2;
    a.chunks = static_cast<uint32_t>((columns + a.steps - 1) / a.steps);
    const uint64_t groups = (e.n * a.chunks + 3) / 4;
    if (groups > kMaxGroups) return too_large();
    const dim3 grid(static_cast<uint32_t>(groups)), threads(256);
    const bool t32 = e.table_dtype == LSO_DT_F32, r32 = e.rows_dtype == LSO_DT_F32;
    auto enqueue = [&](auto once) {
        constexpr bool kOnce = decltype(once)::value;
        const auto kernel = t32 ? (r32 ? embed_lookup_kernel<V, true, true, kOnce> : embed_lookup_kernel<V, true, false, kOnce>)
                                : (r32 ? embed_lookup_kernel<V, false, true, kOnce> : embed_lookup_kernel<V, false, false, kOnce>);
        return launch(kernel, grid, threads, s, a);
    };
    const hipError_t err = beyond_l2(e) ? enqueue(std::true_type{}) : enqueue(std::false_type{});
    return err == hipSuccess ? LSO_OK : hip_fail(err, "embedding lookup launch");
}

template <int V, bool kRowsF32, bool kTableF32>
hipError_t launch_grad_typed(const GradArgs& a, bool once, hipStream_t s)
{
    const dim3 threads(256);
    const uint32_t rows_per_wave = rows_of_wave(a.n, a.vocab), row_groups = (a.vocab + 4 * rows_per_wave - 1) / (4 * rows_per_wave);
    const uint32_t blocks = a.n > kRun ? (a.n + kRun - 1) / kRun : 0;   // a run of up to kRun is no long one
    const uint32_t chunks = (a.width + 64 * V - 1) / (64 * V);
    const uint32_t jobs = blocks * chunks, part_groups = (jobs + 3) / 4;
    const auto kernel = once ? embed_grad_kernel<V, kRowsF32, kTableF32, true> : embed_grad_kernel<V, kRowsF32, kTableF32, false>;
    hipError_t err = launch(kernel, dim3(part_groups + row_groups), threads, s, a, part_groups, chunks, rows_per_wave);
    if (err == hipSuccess && blocks > 0) err = launch(embed_grad_join_kernel<V, kTableF32>, dim3(jobs), threads, s, a, chunks);
    return err;
}

template <int V>
hipError_t launch_grad(const GradArgs& a, bool r32, bool t32, bool once, hipStream_t s)
{
    if (r32 && t32) return launch_grad_typed<V, true, true>(a, once, s);
    if (r32) return launch_grad_typed<V, true, false>(a, once, s);
    if (t32) return launch_grad_typed<V, false, true>(a, once, s);
    return launch_grad_typed<V, false, false>(a, once, s);
}

// Sort the tokens into workspace; sets a.keys and a.pos.
hipError_t launch_sort(const lso_embed& e, char* work, const GradWork& w, GradArgs& a, hipStream_t s)
{
    uint32_t bits = 1;
    while ((e.vocab >> bits) != 0) ++bits;   // the largest key is vocab
    if (e.n <= kRankSort) {
        RankArgs x{};
        x.tokens = tokens_of(e);
        x.keys_out = reinterpret_cast<uint32_t*>(work + w.keys[0]);
        x.pos_out = reinterpret_cast<uint32_t*>(work + w.pos[0]);
        a.keys = x.keys_out;
        a.pos = x.pos_out;
        return launch(sort_by_rank_kernel, dim3((x.tokens.n + 63) / 64), dim3(1024), s, x);
    }
    const uint32_t passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    SortArgs x{};
    x.tokens = tokens_of(e);
    x.counts = reinterpret_cast<uint32_t*>(work + w.counts);
    x.tile = kMinSortTile;
    if (e.n > static_cast<uint64_t>(kMinSortTile) * kMaxSortGroups)
        x.tile = static_cast<uint32_t>(((e.n + kMaxSortGroups - 1) / kMaxSortGroups + kSortThreads - 1) / kSortThreads * kSortThreads);
    x.groups = static_cast<uint32_t>((e.n + x.tile - 1) / x.tile);
    x.bits = (bits + passes - 1) / passes;
    hipError_t err = hipSuccess;
    for (uint32_t p = 0; p < passes && err == hipSuccess; ++p) {
        x.first = p == 0;
        x.shift = p * x.bits;
        x.keys = reinterpret_cast<const uint32_t*>(work + w.keys[(p + 1) & 1u]);
        x.pos = reinterpret_cast<const uint32_t*>(work + w.pos[(p + 1) & 1u]);
        x.keys_out = reinterpret_cast<uint32_t*>(work + w.keys[p & 1u]);
        x.pos_out = reinterpret_cast<uint32_t*>(work + w.pos[p & 1u]);
        err = launch(sort_count_kernel, dim3(x.groups), dim3(kSortThreads), s, x);
        if (err == hipSuccess) err = launch(sort_scatter_kernel, dim3(x.groups), dim3(kSortThreads), s, x);
    }
    a.keys = x.keys_out;
    a.pos = x.pos_out;
    return err;
}

lso_status lookup(const lso_embed* e, void* stream)
{
    clear_error();
    std::vector<Interval> iv;
    bool empty;
    lso_status st = check_embed(e, false, iv, empty);
    if (st != LSO_OK || empty) return st;
    st = check_overlap(iv);
    if (st != LSO_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return vectors(*e) ? launch_lookup<8>(*e, s) : launch_lookup<1>(*e, s);
}

lso_status gradient(const lso_embed* e, void* workspace, uint64_t workspace_bytes, void* stream)
{
    clear_error();
    std::vector<Interval> iv;
    bool empty;
    lso_status st = check_embed(e, true, iv, empty);
    if (st != LSO_OK || empty) return st;
    const GradWork w = grad_work(e->n, e->width);
    if (e->n > 0) {
        if (!workspace) return fail(LSO_E_INVALID, "workspace is NULL");
        if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return fail(LSO_E_ALIGN, "workspace must be 16-byte aligned");
        if (workspace_bytes < w.bytes)
            return fail(LSO_E_INVALID, "workspace of %llu bytes is smaller than the %llu this call needs",
                        static_cast<unsigned long long>(workspace_bytes), static_cast<unsigned long long>(w.bytes));
        if (!add_array(iv, reinterpret_cast<uintptr_t>(workspace), w.bytes, true, 3))
            return fail(LSO_E_INVALID, "workspace range wraps the address space");
    }
    st = check_overlap(iv);
    if (st != LSO_OK) return st;
    const bool vec = vectors(*e);
    const uint64_t columns = (e->width + (vec ? 511 : 63)) / (vec ? 512 : 64);   // column runs of a wave
    if (e->vocab / (4 * rows_of_wave(e->n, e->vocab)) + 1 + (e->n + kRun - 1) / kRun * columns > kMaxGroups) return too_large();
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* work = static_cast<char*>(workspace);
    GradArgs a{};
    a.rows = e->rows;
    a.table = e->table;
    a.parts = reinterpret_cast<float*>(work + w.parts);
    a.ld_rows = e->ld_rows;
    a.ld_table = e->ld_table;
    a.n = static_cast<uint32_t>(e->n);
    a.vocab = static_cast<uint32_t>(e->vocab);
    a.width = static_cast<uint32_t>(e->width);
    a.scale = static_cast<float>(e->scale);
    a.add = (e->flags & LSO_EMBED_ADD) != 0;
    hipError_t err = e->n > 0 ? launch_sort(*e, work, w, a, s) : hipSuccess;
    const bool r32 = e->rows_dtype == LSO_DT_F32, t32 = e->table_dtype == LSO_DT_F32;
    if (err == hipSuccess) err = vec ? launch_grad<8>(a, r32, t32, beyond_l2(*e), s) : launch_grad<1>(a, r32, t32, false, s);
    return err == hipSuccess ? LSO_OK : hip_fail(err, "embedding gradient launch");
}

template <typename F>
lso_status guarded(F f)
{
    try {
        return f();
    } catch (const std::exception& ex) {
        return fail(LSO_E_NOMEM, "host memory: %s", ex.what());
    }
}

}  // namespace
}  // namespace lso

extern "C" {

lso_status lso_embed_lookup(const lso_embed* e, void* stream)
{
    return lso::guarded([&] { return lso::lookup(e, stream); });
}

uint64_t lso_embed_grad_workspace_bytes(uint64_t n, uint64_t vocab, uint64_t width)
{
    if (n > lso::kMaxCount || vocab > lso::kMaxCount || width > lso::kMaxCount) return 0;
    return lso::grad_work(n, width).bytes;
}

lso_status lso_embed_grad(const lso_embed* e, void* workspace, uint64_t workspace_bytes, void* stream)
{
    return lso::guarded([&] { return lso::gradient(e, workspace, workspace_bytes, stream); });
}

int lso_embed_producer(void* user, size_t layer, void* dev_grad, uint64_t n, void* compute_stream)
{
    if (!user) return 1;
    const lso_embed_producer_args* p = static_cast<const lso_embed_producer_args*>(user);
    if (layer != p->embed_layer) return p->other ? p->other(p->other_user, layer, dev_grad, n, compute_stream) : 1;
    lso_embed e = p->grad;
    if (e.flags != 0 || e.vocab == 0 || e.width == 0 || e.vocab > UINT64_MAX / e.width || e.vocab * e.width != n) return 1;
    e.table = dev_grad;
    e.ld_table = e.width;
    return lso_embed_grad(&e, p->workspace, p->workspace_bytes, compute_stream) == LSO_OK ? 0 : 1;
}

}  // extern "C"
