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
#include <vector>

#include "lso_bf16.h"
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
constexpr uint32_t kMinSortTile = 2048;
constexpr uint64_t kMaxGroups = (1ull << 24) - 1;   // workgroups of a launch: 256 lanes each, under 2^32 in all

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

// V consecutive values of a row.
template <int V, bool kF32>
__device__ __forceinline__ void load_values(const void* base, uint64_t i, float (&v)[V])
{
    if (kF32) {
        const float* p = static_cast<const float*>(base) + i;
        if (V == 1) {
            v[0] = *p;
        } else {
#pragma unroll
            for (int e = 0; e < V; e += 4) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(p + e);
#pragma unroll
                for (int k = 0; k < 4 && e + k < V; ++k) v[e + k] = x[k];
            }
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(base) + i;
        if (V == 1) {
            v[0] = bf16_widen(*p);
        } else {
            const u32x4 x = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
            for (int k = 0; k < 4 && 2 * k + 1 < V; ++k) {
                v[2 * k] = bf16_widen(x[k] & 0xFFFFu);
                v[2 * k + 1] = bf16_widen(x[k] >> 16);
            }
        }
    }
}

template <int V, bool kF32>
__device__ __forceinline__ void store_values(void* base, uint64_t i, const float (&v)[V])
{
    if (kF32) {
        float* p = static_cast<float*>(base) + i;
        if (V == 1) {
            *p = v[0];
        } else {
#pragma unroll
            for (int e = 0; e + 3 < V; e += 4) *reinterpret_cast<f32x4*>(p + e) = f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]};
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(base) + i;
        if (V == 1) {
            *p = static_cast<uint16_t>(bf16_rne(v[0]));
        } else {
            u32x4 x;
#pragma unroll
            for (int k = 0; k < 4 && 2 * k + 1 < V; ++k) x[k] = bf16_rne(v[2 * k]) | (bf16_rne(v[2 * k + 1]) << 16);
            *reinterpret_cast<u32x4*>(p) = x;
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

template <int V, bool kTableF32, bool kRowsF32>
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
            load_values<V, kTableF32>(a.table, key * a.ld_table + c, v);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] *= a.scale;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = 0.0f;
        }
        store_values<V, kRowsF32>(a.rows, i * a.ld_rows + c, v);
    }
}

// -------------------------------------------------------------------- sort
//
// Least significant digit first, at most kMaxDigitBits bits a pass.  Each
// group of threads owns a consecutive part of the input; counts[bin][group]
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
    for (uint32_t b = threadIdx.x; b < bins; b += kSortThreads) a.counts[b * a.groups + blockIdx.x] = count[b];
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
        if (b < bins)
            for (uint32_t g = 0; g < a.groups; ++g) {
                const uint32_t c = a.counts[b * a.groups + g];
                if (g < blockIdx.x) before += c;
                total += c;
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
template <int V, bool kRowsF32>
__device__ __forceinline__ void sum_rows(const GradArgs& a, uint32_t first, uint32_t count, uint32_t c, float (&sum)[V])
{
    const LSO_CONST uint32_t* pos = reinterpret_cast<const LSO_CONST uint32_t*>(reinterpret_cast<uintptr_t>(a.pos + first));
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = 0.0f;
    uint32_t k = 0;
    for (; k + 4 <= count; k += 4) {
        float v[4][V];
#pragma unroll
        for (int x = 0; x < 4; ++x) load_values<V, kRowsF32>(a.rows, pos[k + x] * a.ld_rows + c, v[x]);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += v[x][e];
    }
    for (; k < count; ++k) {
        float v[V];
        load_values<V, kRowsF32>(a.rows, pos[k] * a.ld_rows + c, v);
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
        load_values<V, kTableF32>(a.table, i, old);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += old[e];
    }
    store_values<V, kTableF32>(a.table, i, sum);
}

// One wave per table row; rows of long runs are left to the join.
template <int V, bool kRowsF32, bool kTableF32>
__global__ void __launch_bounds__(256) embed_grad_rows_kernel(const GradArgs a)
{
    const uint32_t v = uniform(blockIdx.x * 4 + (threadIdx.x >> 6)), lane = threadIdx.x & 63u;
    if (v >= a.vocab) return;
    const uint32_t first = uniform(find_run(a.keys, a.n, v));
    const uint64_t at = static_cast<uint64_t>(first) + lane;
    const bool mine = at < a.n && a.keys[at] == v;
    const uint32_t count = static_cast<uint32_t>(__popcll(__ballot(mine)));
    if (count > kRun || (count == 0 && a.add)) return;
    for (uint32_t c = lane * V; c < a.width; c += 64 * V) {
        float sum[V];
        sum_rows<V, kRowsF32>(a, first, count, c, sum);
        put_gradient<V, kTableF32>(a, v, c, sum);
    }
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

template <int V, bool kRowsF32>
__global__ void __launch_bounds__(256) embed_grad_parts_kernel(const GradArgs a, uint32_t chunks)
{
    static_assert(kRun == 32, "block_runs looks at half a wave");
    const uint64_t job = static_cast<uint64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
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
        sum_rows<V, kRowsF32>(a, first, count, c, sum);
        store_values<V, true>(a.parts, (b * 2 + x) * static_cast<uint64_t>(a.width) + c, sum);
    }
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
            load_values<V, true>(a.parts, ((static_cast<uint64_t>(b) + k) * 2 + (k == 0 ? x : 0)) * a.width + c, p);
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
    if (t32 && r32) hipLaunchKernelGGL((embed_lookup_kernel<V, true, true>), grid, threads, 0, s, a);
    else if (t32) hipLaunchKernelGGL((embed_lookup_kernel<V, true, false>), grid, threads, 0, s, a);
    else if (r32) hipLaunchKernelGGL((embed_lookup_kernel<V, false, true>), grid, threads, 0, s, a);
    else hipLaunchKernelGGL((embed_lookup_kernel<V, false, false>), grid, threads, 0, s, a);
    const hipError_t err = hipGetLastError();
    return err == hipSuccess ? LSO_OK : hip_fail(err, "embedding lookup launch");
}

template <int V, bool kRowsF32, bool kTableF32>
void launch_grad_typed(const GradArgs& a, hipStream_t s)
{
    const dim3 threads(256);
    hipLaunchKernelGGL((embed_grad_rows_kernel<V, kRowsF32, kTableF32>), dim3((a.vocab + 3) / 4), threads, 0, s, a);
    if (a.n <= kRun) return;
    const uint32_t blocks = (a.n + kRun - 1) / kRun, chunks = (a.width + 64 * V - 1) / (64 * V);
    const uint64_t jobs = static_cast<uint64_t>(blocks) * chunks;
    hipLaunchKernelGGL((embed_grad_parts_kernel<V, kRowsF32>), dim3(static_cast<uint32_t>((jobs + 3) / 4)), threads, 0, s, a, chunks);
    hipLaunchKernelGGL((embed_grad_join_kernel<V, kTableF32>), dim3(static_cast<uint32_t>(jobs)), threads, 0, s, a, chunks);
}

template <int V>
void launch_grad(const GradArgs& a, bool r32, bool t32, hipStream_t s)
{
    if (r32 && t32) launch_grad_typed<V, true, true>(a, s);
    else if (r32) launch_grad_typed<V, true, false>(a, s);
    else if (t32) launch_grad_typed<V, false, true>(a, s);
    else launch_grad_typed<V, false, false>(a, s);
}

// Sort the tokens into workspace; sets a.keys and a.pos.
void launch_sort(const lso_embed& e, char* work, const GradWork& w, GradArgs& a, hipStream_t s)
{
    uint32_t bits = 1;
    while ((e.vocab >> bits) != 0) ++bits;   // the largest key is vocab
    const uint32_t passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    SortArgs x{};
    x.tokens = tokens_of(e);
    x.counts = reinterpret_cast<uint32_t*>(work + w.counts);
    x.tile = kMinSortTile;
    if (e.n > static_cast<uint64_t>(kMinSortTile) * kMaxSortGroups)
        x.tile = static_cast<uint32_t>(((e.n + kMaxSortGroups - 1) / kMaxSortGroups + kSortThreads - 1) / kSortThreads * kSortThreads);
    x.groups = static_cast<uint32_t>((e.n + x.tile - 1) / x.tile);
    x.bits = (bits + passes - 1) / passes;
    for (uint32_t p = 0; p < passes; ++p) {
        x.first = p == 0;
        x.shift = p * x.bits;
        x.keys = reinterpret_cast<const uint32_t*>(work + w.keys[(p + 1) & 1u]);
        x.pos = reinterpret_cast<const uint32_t*>(work + w.pos[(p + 1) & 1u]);
        x.keys_out = reinterpret_cast<uint32_t*>(work + w.keys[p & 1u]);
        x.pos_out = reinterpret_cast<uint32_t*>(work + w.pos[p & 1u]);
        hipLaunchKernelGGL(sort_count_kernel, dim3(x.groups), dim3(kSortThreads), 0, s, x);
        hipLaunchKernelGGL(sort_scatter_kernel, dim3(x.groups), dim3(kSortThreads), 0, s, x);
    }
    a.keys = x.keys_out;
    a.pos = x.pos_out;
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
    (void)hipGetLastError();   // an error left by other work is not this call's
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
    if (e->vocab / 4 + 1 > kMaxGroups || (e->n + kRun - 1) / kRun * columns > kMaxGroups) return too_large();
    hipStream_t s = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();   // an error left by other work is not this call's
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
    if (e->n > 0) launch_sort(*e, work, w, a, s);
    const bool r32 = e->rows_dtype == LSO_DT_F32, t32 = e->table_dtype == LSO_DT_F32;
    if (vec) launch_grad<8>(a, r32, t32, s);
    else launch_grad<1>(a, r32, t32, s);
    const hipError_t err = hipGetLastError();
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
