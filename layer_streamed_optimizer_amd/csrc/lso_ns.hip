// Newton-Schulz orthogonalisation and the orthogonalised-momentum update for
// gfx950.  Formulas and precisions: lso_ops.h.
//
// General path (smaller side above 32), all matrices of a call together, one
// launch per step below:
//   norm     u (for the update: m' and u), its sum of squares per tile
//   scale    1 / (|u|_F + eps) per matrix
//   split    X_0 = u / (|u|_F + eps) into FP16 operands, X and its transpose
//   per step: S = X X^T; P = a I + b S + c S^2; X' = P X
// and the last product writes y, or master and weight, itself.
//
// Operands.  A value v is held as h + l, h = fp16(v * 4096), l =
// fp16(v * 4096 - h): 22 significant bits.  A product of two such matrices
// is three matrix-core products, h h + h l + l h, summed in the same FP32
// registers (l l is below FP32's rounding); with one term it is one.  All
// operands are stored with the summed index contiguous, so X and X^T are
// both kept; h and l of 32 consecutive values sit next to each other (64 B
// each), so a row of a product's stage is always one 128-byte line.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "lso_bf16.h"
#include "lso_ns.h"

namespace lso {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#define LSO_CONST __attribute__((address_space(4)))

// ------------------------------------------------------------- the table

// Entries per writer launch: the kernel arguments stay under 4 KiB.
constexpr uint32_t kWriteMats = 38;
struct NsTablePart {
    NsMat* dst;
    uint32_t count;
    uint32_t pad;
    NsMat src[kWriteMats];
};
static_assert(sizeof(NsTablePart) <= 4000, "writer arguments");

__global__ void __launch_bounds__(64) ns_table_kernel(const NsTablePart part)
{
    if (threadIdx.x < part.count) part.dst[threadIdx.x] = part.src[threadIdx.x];
}

__device__ __forceinline__ NsMat load_mat(const NsMat* tab, uint32_t i)
{
    return *reinterpret_cast<const NsMat*>(reinterpret_cast<const char*>(tab) + static_cast<uint64_t>(i) * sizeof(NsMat));
}

// The last of n matrices whose first index (field F) is <= index.
template <uint32_t NsMat::*F>
__device__ __forceinline__ uint32_t find_mat(const NsMat* tab, uint32_t n, uint32_t index)
{
    uint32_t lo = 0, hi = n;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (tab[mid].*F <= index) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ------------------------------------------------------ elements of u

__device__ __forceinline__ float load_src(const NsMat& m, uint64_t r, uint32_t c)
{
    const uint64_t i = r * m.ld_src + c;
    return (m.flags & kNsSrcF32) ? static_cast<const float*>(m.src)[i]
                                 : bf16_widen(static_cast<const uint16_t*>(m.src)[i]);
}

__device__ __forceinline__ float new_momentum(const NsMat& m, float old, float g) { return fmaf(m.beta, old, m.c1 * g); }

__device__ __forceinline__ float lookahead(const NsMat& m, float m1, float g)
{
    return (m.flags & kNsNesterov) ? fmaf(m.beta, m1, m.c1 * g) : m1;
}

// u of element (r, c); kFirst: m holds the old momentum and takes the new.
template <bool kFirst>
__device__ __forceinline__ float load_u(const NsMat& m, uint32_t r, uint32_t c)
{
    const float g = load_src(m, r, c);
    if (!(m.flags & kNsMuon)) return g;
    float* p = m.m + static_cast<uint64_t>(r) * m.cols + c;
    float m1 = *p;
    if (kFirst) {
        m1 = new_momentum(m, m1, g);
        *p = m1;
    }
    return lookahead(m, m1, g);
}

// y of element (r, c): stored, or applied to master and weight.
__device__ __forceinline__ void put_result(const NsMat& m, uint32_t r, uint32_t c, float o)
{
    if (m.flags & kNsMuon) {
        const uint64_t i = static_cast<uint64_t>(r) * m.cols + c;
        const float p = fmaf(m.step, o, m.keep * m.master[i]);
        m.master[i] = p;
        if (m.dst) static_cast<uint16_t*>(m.dst)[i] = static_cast<uint16_t>(bf16_rne(p));
        return;
    }
    const uint64_t i = static_cast<uint64_t>(r) * m.ld_dst + c;
    if (m.flags & kNsDstF32) static_cast<float*>(m.dst)[i] = o;
    else static_cast<uint16_t*>(m.dst)[i] = static_cast<uint16_t>(bf16_rne(o));
}

// Sum over a workgroup of kN threads in a fixed order; valid in thread 0.
template <int kN>
__device__ __forceinline__ double group_sum(double v)
{
    __shared__ double per_wave[kN / 64];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    if ((threadIdx.x & 63) == 0) per_wave[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
        for (int k = 0; k < kN / 64; ++k) s += per_wave[k];
    return s;
}

// ------------------------------------------------------ general path: input

// Tile t of a matrix's padded kNsPrep tiles: first row and column of the
// natural (row-major, as given) matrix.
__device__ __forceinline__ void prep_tile(const NsMat& m, uint32_t t, uint32_t& r0, uint32_t& c0)
{
    const uint32_t across = ((m.flags & kNsTall) ? m.mp : m.np) / kNsPrep;
    r0 = t / across * kNsPrep;
    c0 = t % across * kNsPrep;
}

__global__ void __launch_bounds__(256) ns_norm_kernel(const NsMat* tab, uint32_t n, uint32_t gram_terms)
{
    const uint32_t i = find_mat<&NsMat::prep0>(tab, n, blockIdx.x);
    const NsMat m = load_mat(tab, i);
    uint32_t r0, c0;
    prep_tile(m, blockIdx.x - m.prep0, r0, c0);
    const uint32_t c = c0 + (threadIdx.x & 63u);
    double sum = 0.0;
    if (c < m.cols) {
#pragma unroll 4
        for (uint32_t k = threadIdx.x >> 6; k < kNsPrep; k += 4) {
            if (r0 + k < m.rows) {
                const double u = load_u<true>(m, r0 + k, c);
                sum = fma(u, u, sum);
            }
        }
    }
    sum = group_sum<256>(sum);
    if (threadIdx.x == 0) {
        const NsWork w = ns_work(m.mp, m.np, gram_terms);
        reinterpret_cast<double*>(m.work + w.partial)[blockIdx.x - m.prep0] = sum;
    }
}

// What X_0 is made with.  X_0 has the norm |u| / (|u| + eps), which is 1
// unless u is about as small as eps.  A small X_0 would leave FP16's range
// (its scale is fixed), so the path works on X 2^e with e >= 0 chosen to
// bring the norm of X_0 to [1/2, 2): with S' = S 2^2e the polynomial is
// a + b 2^-2e S' + c 2^-4e S'^2, and each step lowers e by as many powers of
// two as X can have grown by.
struct NsScaling {
    double inv;   // 2^e / (|u|_F + eps)
    int e;
};

// One workgroup per matrix.
__global__ void __launch_bounds__(1024) ns_scale_kernel(const NsMat* tab, uint32_t gram_terms, double eps)
{
    const NsMat m = load_mat(tab, blockIdx.x);
    const NsWork w = ns_work(m.mp, m.np, gram_terms);
    const uint32_t tiles = m.mp / kNsPrep * (m.np / kNsPrep);
    const double* part = reinterpret_cast<const double*>(m.work + w.partial);
    double sum = 0.0;
    for (uint32_t k = threadIdx.x; k < tiles; k += 1024) sum += part[k];
    sum = group_sum<1024>(sum);
    if (threadIdx.x != 0) return;
    const double norm = sqrt(sum), inv = 1.0 / (norm + eps);
    NsScaling s = {inv, 0};
    if (norm > 0.0 && norm * inv < 0.5) {
        int e = 0;
        frexp(norm * inv, &e);   // norm * inv in [2^(e-1), 2^e)
        s.e = 1 - e < 1000 ? 1 - e : 1000;
        s.inv = ldexp(inv, s.e);
    }
    *reinterpret_cast<NsScaling*>(m.work + w.inv) = s;
}

// Eight consecutive values v (already scaled) as FP16 terms into row `row`
// (of `ld` values) from column c (a multiple of 8) of an operand.
template <int kTerms>
__device__ __forceinline__ void put_terms(char* base, uint64_t row, uint64_t ld, uint32_t c, const float (&v)[8])
{
    f16x8 h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        h[e] = static_cast<_Float16>(v[e]);
        l[e] = static_cast<_Float16>(v[e] - static_cast<float>(h[e]));
    }
    if (kTerms == 1) {
        *reinterpret_cast<f16x8*>(base + (row * ld + c) * 2) = h;
    } else {
        char* p = base + (row * ld + (c & ~31u)) * 4 + (c & 31u) * 2;
        *reinterpret_cast<f16x8*>(p) = h;
        *reinterpret_cast<f16x8*>(p + 64) = l;
    }
}

__device__ __forceinline__ void put_terms_n(uint32_t terms, char* base, uint64_t row, uint64_t ld, uint32_t c, const float (&v)[8])
{
    if (terms == 1) put_terms<1>(base, row, ld, c, v);
    else put_terms<2>(base, row, ld, c, v);
}

// X_0 and its transpose from u, zeros in the padding.
__global__ void __launch_bounds__(256) ns_split_kernel(const NsMat* tab, uint32_t n, uint32_t gram_terms)
{
    __shared__ float tile[kNsPrep][kNsPrep + 1];
    const uint32_t i = find_mat<&NsMat::prep0>(tab, n, blockIdx.x);
    const NsMat m = load_mat(tab, i);
    const NsWork w = ns_work(m.mp, m.np, gram_terms);
    uint32_t r0, c0;
    prep_tile(m, blockIdx.x - m.prep0, r0, c0);
    const double inv = reinterpret_cast<const NsScaling*>(m.work + w.inv)->inv;
    const uint32_t cc = threadIdx.x & 63u;
#pragma unroll 4
    for (uint32_t k = threadIdx.x >> 6; k < kNsPrep; k += 4) {
        float x = 0.0f;
        if (r0 + k < m.rows && c0 + cc < m.cols)
            x = static_cast<float>(static_cast<double>(load_u<false>(m, r0 + k, c0 + cc)) * inv) * kNsScale;
        tile[k][cc] = x;
    }
    __syncthreads();
    const bool tall = (m.flags & kNsTall) != 0;
    char* xt = m.work + w.xt[0];
    char* x = m.work + w.x;
    // natural orientation: rows x cols is X, or X^T if tall
    for (uint32_t v = threadIdx.x; v < kNsPrep * kNsPrep / 8; v += 256) {
        const uint32_t r = v >> 3, c = (v & 7u) * 8;
        float a[8], b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[e] = tile[r][c + e];
            b[e] = tile[c + e][r];
        }
        if (tall) {
            put_terms<2>(xt, r0 + r, m.mp, c0 + c, a);
            put_terms_n(gram_terms, x, c0 + r, m.np, r0 + c, b);
        } else {
            put_terms_n(gram_terms, x, r0 + r, m.np, c0 + c, a);
            put_terms<2>(xt, c0 + r, m.mp, r0 + c, b);
        }
    }
}

// ------------------------------------------------------ general path: products
//
// D[i][j] = sum over k of A[i][k] B[j][k], a 128 x 128 tile per workgroup of
// four waves, 64 x 64 each (2 x 2 matrix-core tiles of 32 x 32).  A stage is
// 128 bytes of each row of a two-term operand (32 values, h and l) or of a
// one-term operand multiplied by one (64 values), 64 bytes of a one-term
// operand multiplied by a two-term one; two stages alternate in LDS, the
// next one loaded straight to LDS while the current one is multiplied.
// 16-byte pieces of a row are permuted by the row's number so that the eight
// lanes which read LDS together hit all banks; the permutation is made by
// the global address each lane loads from, since a load to LDS writes
// consecutive lanes to consecutive places.

constexpr uint32_t kPitch = kNsTile + 1;   // of the result tile in LDS

template <int kRowBytes>
__device__ __forceinline__ uint32_t swizzle(uint32_t row)
{
    return kRowBytes == 128 ? (row & 7u) : ((row >> 1) & 3u);
}

// Load stage rows [0, 128) x kRowBytes from g (row stride bytes) to lds.
template <int kRowBytes>
__device__ __forceinline__ void load_stage(const char* g, uint32_t stride, char* lds)
{
    constexpr uint32_t kPieces = kRowBytes / 16, kRowsPerLoad = 64 / kPieces, kLoads = kNsTile / kRowsPerLoad / 4;
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
#pragma unroll
    for (uint32_t q = 0; q < kLoads; ++q) {
        const uint32_t at = wave * kLoads + q;
        const uint32_t row = at * kRowsPerLoad + lane / kPieces;
        const uint32_t piece = (lane % kPieces) ^ swizzle<kRowBytes>(row);
        __builtin_amdgcn_global_load_lds(
            reinterpret_cast<const __attribute__((address_space(1))) uint32_t*>(
                reinterpret_cast<uintptr_t>(g + static_cast<uint64_t>(row) * stride + piece * 16)),
            (__attribute__((address_space(3))) uint32_t*)(lds + at * 1024), 16, 0, 0);
    }
}

template <int kRowBytes>
__device__ __forceinline__ f16x8 fragment(const char* lds, uint32_t row, uint32_t piece)
{
    return *reinterpret_cast<const f16x8*>(lds + row * kRowBytes + ((piece ^ swizzle<kRowBytes>(row)) * 16));
}

enum { kGram = 0, kPoly = 1, kApply = 2, kLast = 3 };

struct ProductArgs {
    const NsMat* tab;
    uint32_t n, tiles;
    uint32_t turn;       // which transpose of X is read
    double a, b, c;      // coefficients of the step (kPoly)
    int lowered, lower;  // by how much the steps before and this one lower e
};

__device__ __forceinline__ int left_of(int e, int lowered) { return e > lowered ? e - lowered : 0; }

// Value (row, c) of an operand, times kNsScale.
template <int kTerms>
__device__ __forceinline__ float get_term(const char* base, uint64_t row, uint64_t ld, uint32_t c)
{
    if (kTerms == 1) return static_cast<float>(*reinterpret_cast<const _Float16*>(base + (row * ld + c) * 2));
    const char* p = base + (row * ld + (c & ~31u)) * 4 + (c & 31u) * 2;
    return static_cast<float>(*reinterpret_cast<const _Float16*>(p)) + static_cast<float>(*reinterpret_cast<const _Float16*>(p + 64));
}

template <int kTermsA, int kTermsB, int kKind, int kGramTerms>
__global__ void __launch_bounds__(256, 2) ns_product_kernel(const ProductArgs args)
{
    constexpr int kValues = (kTermsA == 1 && kTermsB == 1) ? 64 : 32;   // of the summed index per stage
    constexpr int kRowA = kValues * 2 * kTermsA, kRowB = kValues * 2 * kTermsB;
    constexpr uint32_t kStage = kNsTile * (kRowA + kRowB);
    constexpr uint32_t kLds = 2 * kStage > kNsTile * kPitch * 4 ? 2 * kStage : kNsTile * kPitch * 4;
    __shared__ __attribute__((aligned(128))) char lds[kLds];

    // consecutive tiles go to one XCD (workgroups go round the eight in turn)
    const uint32_t per = (args.tiles + 7) / 8;
    const uint32_t t = (blockIdx.x & 7u) * per + (blockIdx.x >> 3);
    if (t >= args.tiles || (blockIdx.x >> 3) >= per) return;
    const uint32_t mi = kKind <= kPoly ? find_mat<&NsMat::sym0>(args.tab, args.n, t) : find_mat<&NsMat::apply0>(args.tab, args.n, t);
    const NsMat m = load_mat(args.tab, mi);
    const NsWork w = ns_work(m.mp, m.np, kGramTerms);
    uint32_t ti, tj;
    if (kKind <= kPoly) {
        const uint32_t k = t - m.sym0;
        ti = static_cast<uint32_t>((sqrtf(8.0f * static_cast<float>(k) + 1.0f) - 1.0f) * 0.5f);
        while (ti * (ti + 1) / 2 > k) --ti;
        while ((ti + 1) * (ti + 2) / 2 <= k) ++ti;
        tj = k - ti * (ti + 1) / 2;
    } else {
        const uint32_t k = t - m.apply0, across = m.mp / kNsTile;
        ti = k / across;
        tj = k % across;
    }
    const char* a;
    const char* b;
    uint32_t depth;
    if (kKind == kGram) {
        a = b = m.work + w.x;
        depth = m.np;
    } else if (kKind == kPoly) {
        a = b = m.work + w.s;
        depth = m.mp;
    } else {
        a = m.work + ((args.turn & 1u) ? w.xt[1] : w.xt[0]);
        b = m.work + w.p;
        depth = m.mp;
    }
    const uint32_t i0 = ti * kNsTile, j0 = tj * kNsTile;
    const uint32_t stride_a = depth * 2 * kTermsA, stride_b = depth * 2 * kTermsB;   // sides below 2^29
    a += static_cast<uint64_t>(i0) * stride_a;
    b += static_cast<uint64_t>(j0) * stride_b;

    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t wi = (wave >> 1) * 64, wj = (wave & 1u) * 64;
    f32x16 acc[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[x][y][e] = 0.0f;

    const uint32_t stages = depth / kValues;
    load_stage<kRowA>(a, stride_a, lds);
    load_stage<kRowB>(b, stride_b, lds + kNsTile * kRowA);
    __syncthreads();
    for (uint32_t s = 0; s < stages; ++s) {
        const char* now = lds + (s & 1u) * kStage;
        if (s + 1 < stages) {
            char* next = lds + ((s + 1) & 1u) * kStage;
            load_stage<kRowA>(a + (s + 1) * kRowA, stride_a, next);
            load_stage<kRowB>(b + (s + 1) * kRowB, stride_b, next + kNsTile * kRowA);
        }
#pragma unroll
        for (uint32_t kk = 0; kk < kValues / 16; ++kk) {
            f16x8 fa[2][kTermsA], fb[2][kTermsB];
#pragma unroll
            for (uint32_t x = 0; x < 2; ++x) {
#pragma unroll
                for (uint32_t p = 0; p < kTermsA; ++p)
                    fa[x][p] = fragment<kRowA>(now, wi + x * 32 + (lane & 31u), p * 4 + kk * 2 + (lane >> 5));
#pragma unroll
                for (uint32_t p = 0; p < kTermsB; ++p)
                    fb[x][p] = fragment<kRowB>(now + kNsTile * kRowA, wj + x * 32 + (lane & 31u), p * 4 + kk * 2 + (lane >> 5));
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[x][0], fb[y][0], acc[x][y], 0, 0, 0);
                    if (kTermsB == 2) acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[x][0], fb[y][kTermsB - 1], acc[x][y], 0, 0, 0);
                    if (kTermsA == 2) acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[x][kTermsA - 1], fb[y][0], acc[x][y], 0, 0, 0);
                }
        }
        __syncthreads();
    }

    // the tile through LDS, values times kNsScale (products carry its square)
    float* tile = reinterpret_cast<float*>(lds);
    float unscale = 1.0f / kNsScale, ca = 0.0f, cb = 0.0f, cc = 0.0f;
    if (kKind == kPoly || kKind == kLast) {
        const int e0 = reinterpret_cast<const NsScaling*>(m.work + w.inv)->e;
        const int before = left_of(e0, args.lowered), after = left_of(e0, args.lowered + args.lower), up = after - before;
        if (kKind == kLast) unscale = ldexpf(1.0f / (kNsScale * kNsScale), -after);
        ca = static_cast<float>(ldexp(args.a, up));
        cb = static_cast<float>(ldexp(args.b, up - 2 * before));
        cc = static_cast<float>(ldexp(args.c, up - 4 * before));
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t i = wi + x * 32 + 8 * (e / 4) + 4 * (lane >> 5) + (e & 3);
                const uint32_t j = wj + y * 32 + (lane & 31u);
                float v = acc[x][y][e] * unscale;
                if (kKind == kPoly) {
                    const float sv = get_term<kGramTerms>(m.work + w.s, i0 + i, m.mp, j0 + j);
                    v = fmaf(cc, v, cb * sv);
                    if (i0 + i == j0 + j) v += ca * kNsScale;
                }
                tile[i * kPitch + j] = v;
            }
    __syncthreads();

    if (kKind == kLast) {
        // D is X'^T: element (i, j) is X'(j, i); rows of the natural matrix
        // are i if tall, else j
        const bool tall = (m.flags & kNsTall) != 0;
        const uint32_t r0 = tall ? i0 : j0, c0 = tall ? j0 : i0;
        for (uint32_t v = threadIdx.x; v < kNsTile * kNsTile; v += 256) {
            const uint32_t r = v / kNsTile, c = v % kNsTile;
            if (r0 + r < m.rows && c0 + c < m.cols) put_result(m, r0 + r, c0 + c, tall ? tile[r * kPitch + c] : tile[c * kPitch + r]);
        }
        return;
    }
    char* out_rows;      // takes D
    char* out_cols;      // takes D transposed
    uint64_t ld_rows, ld_cols;
    if (kKind == kApply) {
        out_rows = m.work + ((args.turn & 1u) ? w.xt[0] : w.xt[1]);
        out_cols = m.work + w.x;
        ld_rows = m.mp;
        ld_cols = m.np;
    } else {
        out_rows = out_cols = m.work + (kKind == kGram ? w.s : w.p);
        ld_rows = ld_cols = m.mp;
    }
    for (uint32_t v = threadIdx.x; v < kNsTile * kNsTile / 8; v += 256) {
        const uint32_t r = v / (kNsTile / 8), c = v % (kNsTile / 8) * 8;
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = tile[r * kPitch + c + e];
        if (kKind == kApply) put_terms<2>(out_rows, i0 + r, ld_rows, j0 + c, d);
        else put_terms<kGramTerms>(out_rows, i0 + r, ld_rows, j0 + c, d);
        if (kKind == kApply || ti != tj) {
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = tile[(c + e) * kPitch + r];
            put_terms<kGramTerms>(out_cols, j0 + r, ld_cols, i0 + c, d);
        }
    }
}

// ------------------------------------------------------ small path
//
// k = the smaller side, at most kK.  X is k x l; the iterates are
// X_n = Q_n X_0 with Q_n a polynomial in S_0 = X_0 X_0^T, so everything but
// the first and last pass happens on k x k matrices:
//   S_{n+1} = P S_n P, Q_{n+1} = P Q_n, P = a I + b S_n + c S_n^2.
// S_0 squares the singular values' spread and each step multiplies the
// error of the small ones by a^2 (about 12), which FP32 would not survive
// over five steps; in FP64 it ends near 1e-11.  |u|_F^2 is the trace of the
// unscaled S.  Bound: two reads of u and launch latency.

template <int kK>
__device__ __forceinline__ void small_place(const NsMat& m, uint32_t p, uint32_t l, uint32_t& r, uint32_t& c)
{
    const bool tall = (m.flags & kNsTall) != 0;
    r = tall ? l : p;
    c = tall ? p : l;
}

// Stage u of long-side elements [l0, l0 + count) into u[p][l - l0].
template <int kK, bool kFirst>
__device__ __forceinline__ void stage_u(const NsMat& m, uint32_t k, uint32_t l0, uint32_t count, float (&u)[kK][kNsSmallChunk + 1])
{
    const bool tall = (m.flags & kNsTall) != 0;
    for (uint32_t v = threadIdx.x; v < k * count; v += 256) {
        // natural order: consecutive v are consecutive columns
        const uint32_t p = tall ? v % k : v / count, l = tall ? v / k : v % count;
        uint32_t r, c;
        small_place<kK>(m, p, l0 + l, r, c);
        u[p][l] = load_u<kFirst>(m, r, c);
    }
}

template <int kK>
__global__ void __launch_bounds__(256) ns_small_gram_kernel(const NsMat* tab, uint32_t n)
{
    __shared__ float u[kK][kNsSmallChunk + 1];
    __shared__ double part[256];
    const NsMat m = load_mat(tab, find_mat<&NsMat::prep0>(tab, n, blockIdx.x));
    const uint32_t chunk = blockIdx.x - m.prep0;
    const uint32_t k = m.rows < m.cols ? m.rows : m.cols, l = m.rows < m.cols ? m.cols : m.rows;
    const uint32_t l0 = chunk * kNsSmallChunk, count = l - l0 < kNsSmallChunk ? l - l0 : kNsSmallChunk;
    stage_u<kK, true>(m, k, l0, count, u);
    __syncthreads();
    double* out = reinterpret_cast<double*>(m.work) + static_cast<uint64_t>(chunk) * k * k;
    constexpr uint32_t kSlots = kK * kK;
    if (kSlots >= 256) {
        for (uint32_t s = threadIdx.x; s < kSlots; s += 256) {
            const uint32_t p = s / kK, q = s % kK;
            if (p >= k || q >= k) continue;
            double sum = 0.0;
            for (uint32_t x = 0; x < count; ++x) sum = fma(static_cast<double>(u[p][x]), static_cast<double>(u[q][x]), sum);
            out[p * k + q] = sum;
        }
    } else {
        // several threads per (p, q), each over its own part of the chunk
        constexpr uint32_t kParts = 256 / kSlots;
        const uint32_t s = threadIdx.x % kSlots, g = threadIdx.x / kSlots, p = s / kK, q = s % kK;
        double sum = 0.0;
        if (p < k && q < k)
            for (uint32_t x = g * (kNsSmallChunk / kParts); x < (g + 1) * (kNsSmallChunk / kParts) && x < count; ++x)
                sum = fma(static_cast<double>(u[p][x]), static_cast<double>(u[q][x]), sum);
        part[threadIdx.x] = sum;
        __syncthreads();
        if (g == 0 && p < k && q < k) {
            for (uint32_t x = 1; x < kParts; ++x) sum += part[x * kSlots + s];
            out[p * k + q] = sum;
        }
    }
}

struct SmallArgs {
    const NsMat* tab;
    uint32_t steps;
    double eps;
    double coef[3 * kNsMaxSteps];
};

// One workgroup of kK * kK threads per matrix, one element each.
template <int kK>
__global__ void __launch_bounds__(kK * kK) ns_small_iterate_kernel(const SmallArgs args)
{
    __shared__ double s[kK][kK + 1], t[kK][kK + 1], p[kK][kK + 1], q[kK][kK + 1];
    const NsMat m = load_mat(args.tab, blockIdx.x);
    const uint32_t k = m.rows < m.cols ? m.rows : m.cols, l = m.rows < m.cols ? m.cols : m.rows;
    const uint32_t chunks = (l + kNsSmallChunk - 1) / kNsSmallChunk;
    const uint32_t i = threadIdx.x / kK, j = threadIdx.x % kK;
    const bool in = i < k && j < k;
    const double* part = reinterpret_cast<const double*>(m.work);
    double sum = 0.0;
    if (in)
        for (uint32_t c = 0; c < chunks; ++c) sum += part[static_cast<uint64_t>(c) * k * k + i * k + j];
    s[i][j] = sum;
    __syncthreads();
    double trace = 0.0;
    for (uint32_t x = 0; x < k; ++x) trace += s[x][x];
    const double inv = 1.0 / (sqrt(trace) + args.eps);
    __syncthreads();
    s[i][j] = sum * inv * inv;
    q[i][j] = i == j ? inv : 0.0;   // Q_0 carries the scaling of u to X_0
    __syncthreads();
    auto product = [&](const double (&x)[kK][kK + 1], const double (&y)[kK][kK + 1]) {
        double v = 0.0;
        for (uint32_t e = 0; e < k; ++e) v = fma(x[i][e], y[e][j], v);
        return v;
    };
    for (uint32_t n = 0; n < args.steps; ++n) {
        const double a = args.coef[3 * n], b = args.coef[3 * n + 1], c = args.coef[3 * n + 2];
        const double s2 = product(s, s);
        p[i][j] = (i == j ? a : 0.0) + b * s[i][j] + c * s2;
        __syncthreads();
        const double qn = product(p, q);
        t[i][j] = product(p, s);
        __syncthreads();
        q[i][j] = qn;
        s[i][j] = product(t, p);
        __syncthreads();
    }
    if (in) reinterpret_cast<double*>(m.work)[static_cast<uint64_t>(chunks) * k * k + i * k + j] = q[i][j];
}

template <int kK>
__global__ void __launch_bounds__(256) ns_small_apply_kernel(const NsMat* tab, uint32_t n)
{
    __shared__ float u[kK][kNsSmallChunk + 1];
    __shared__ double q[kK * kK];
    const NsMat m = load_mat(tab, find_mat<&NsMat::prep0>(tab, n, blockIdx.x));
    const uint32_t chunk = blockIdx.x - m.prep0;
    const uint32_t k = m.rows < m.cols ? m.rows : m.cols, l = m.rows < m.cols ? m.cols : m.rows;
    const uint32_t l0 = chunk * kNsSmallChunk, count = l - l0 < kNsSmallChunk ? l - l0 : kNsSmallChunk;
    const uint32_t chunks = (l + kNsSmallChunk - 1) / kNsSmallChunk;
    stage_u<kK, false>(m, k, l0, count, u);
    const double* src = reinterpret_cast<const double*>(m.work) + static_cast<uint64_t>(chunks) * k * k;
    for (uint32_t v = threadIdx.x; v < k * k; v += 256) q[v] = src[v];
    __syncthreads();
    if (threadIdx.x < count) {
        float col[kK];
#pragma unroll
        for (int e = 0; e < kK; ++e) col[e] = e < static_cast<int>(k) ? u[e][threadIdx.x] : 0.0f;
        for (uint32_t p = 0; p < k; ++p) {
            double v = 0.0;
#pragma unroll
            for (int e = 0; e < kK; ++e)
                if (e < static_cast<int>(k)) v = fma(q[p * k + e], static_cast<double>(col[e]), v);
            u[p][threadIdx.x] = static_cast<float>(v);
        }
    }
    __syncthreads();
    const bool tall = (m.flags & kNsTall) != 0;
    for (uint32_t v = threadIdx.x; v < k * count; v += 256) {
        const uint32_t p = tall ? v % k : v / count, x = tall ? v / k : v % count;
        uint32_t r, c;
        small_place<kK>(m, p, l0 + x, r, c);
        put_result(m, r, c, u[p][x]);
    }
}

template <int kK>
hipError_t launch_small(const NsCall& c, const NsMat* tab, uint32_t n, uint32_t chunks, hipStream_t s)
{
    SmallArgs args{};
    args.tab = tab;
    args.steps = c.steps;
    args.eps = c.eps;
    for (uint32_t k = 0; k < 3 * c.steps; ++k) args.coef[k] = c.coef[k];
    hipLaunchKernelGGL(ns_small_gram_kernel<kK>, dim3(chunks), dim3(256), 0, s, tab, n);
    hipLaunchKernelGGL(ns_small_iterate_kernel<kK>, dim3(n), dim3(kK * kK), 0, s, args);
    hipLaunchKernelGGL(ns_small_apply_kernel<kK>, dim3(chunks), dim3(256), 0, s, tab, n);
    return hipGetLastError();
}

template <int kGramTerms>
hipError_t launch_big(const NsCall& c, const NsMat* tab, hipStream_t s)
{
    const uint32_t n = c.nbig;
    hipLaunchKernelGGL(ns_norm_kernel, dim3(c.prep_tiles), dim3(256), 0, s, tab, n, c.gram_terms);
    hipLaunchKernelGGL(ns_scale_kernel, dim3(n), dim3(1024), 0, s, tab, c.gram_terms, c.eps);
    hipLaunchKernelGGL(ns_split_kernel, dim3(c.prep_tiles), dim3(256), 0, s, tab, n, c.gram_terms);
    const dim3 sym((c.sym_tiles + 7) / 8 * 8), apply((c.apply_tiles + 7) / 8 * 8), threads(256);
    int lowered = 0;
    for (uint32_t k = 0; k < c.steps; ++k) {
        ProductArgs args{};
        args.tab = tab;
        args.n = n;
        args.turn = k;
        args.a = c.coef[3 * k];
        args.b = c.coef[3 * k + 1];
        args.c = c.coef[3 * k + 2];
        args.lowered = lowered;
        args.lower = static_cast<int>(c.shift[k]);
        lowered += args.lower;
        args.tiles = c.sym_tiles;
        hipLaunchKernelGGL((ns_product_kernel<kGramTerms, kGramTerms, kGram, kGramTerms>), sym, threads, 0, s, args);
        hipLaunchKernelGGL((ns_product_kernel<kGramTerms, kGramTerms, kPoly, kGramTerms>), sym, threads, 0, s, args);
        args.tiles = c.apply_tiles;
        if (k + 1 < c.steps)
            hipLaunchKernelGGL((ns_product_kernel<2, kGramTerms, kApply, kGramTerms>), apply, threads, 0, s, args);
        else
            hipLaunchKernelGGL((ns_product_kernel<2, kGramTerms, kLast, kGramTerms>), apply, threads, 0, s, args);
    }
    return hipGetLastError();
}

}  // namespace

int ns_launch(const NsCall& c, NsMat* device_table, void* stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();   // an error left by other work is not this call's
    uint32_t total = c.nbig;
    for (int k = 0; k < kNsClasses; ++k) total += c.nsmall[k];
    for (uint32_t k = 0; k < total; k += kWriteMats) {
        NsTablePart part{};
        part.dst = device_table + k;
        part.count = total - k < kWriteMats ? total - k : kWriteMats;
        for (uint32_t j = 0; j < part.count; ++j) part.src[j] = c.table[k + j];
        hipLaunchKernelGGL(ns_table_kernel, dim3(1), dim3(64), 0, s, part);
    }
    hipError_t err = hipGetLastError();
    const NsMat* tab = device_table;
    for (int k = 0; k < kNsClasses && err == hipSuccess; ++k) {
        if (c.nsmall[k] == 0) continue;
        err = k == 0 ? launch_small<8>(c, tab, c.nsmall[k], c.small_chunks[k], s)
            : k == 1 ? launch_small<16>(c, tab, c.nsmall[k], c.small_chunks[k], s)
                     : launch_small<32>(c, tab, c.nsmall[k], c.small_chunks[k], s);
        tab += c.nsmall[k];
    }
    if (err == hipSuccess && c.nbig > 0) err = c.gram_terms == 1 ? launch_big<1>(c, tab, s) : launch_big<2>(c, tab, s);
    return err;
}

}  // namespace lso
