// Newton-Schulz orthogonalisation and the orthogonalised-momentum update for
// gfx950.  Formulas and precisions: lso_ops.h.
//
// General path (smaller side above 64, or above 32 where a few of those come
// with larger matrices), all matrices of a call together, one launch per step
// below:
//   norm     u (for the update: m' and u), its sum of squares per tile
//   scale    1 / (|u|_F + eps) per matrix
//   split    X_0 = u / (|u|_F + eps) into FP16 operands, X and its transpose
//   per step: S = X X^T; P = a I + b S + c S^2; X' = P X
// and the last product writes y, or master and weight, itself.
//
// Operands.  A value v is held as h + l, h = fp16(v * 4096), l =
// fp16(v * 4096 - h): 22 significant bits.  A product of two such matrices
// is three matrix-core products, h h + h l + l h, summed in the same FP32
// registers (l l is below FP32's rounding); with one term it is one.  The
// summed index of every operand runs along its rows, so X and X^T are both
// kept.  An operand is stored in blocks of kT rows (the edge of a product's
// tile) by 16 values, 32 bytes a row and term, one after another along the
// rows: what a product loads at a time is one run of memory.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "lso_bf16.h"
#include "lso_launch.h"
#include "lso_ns.h"

namespace lso {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

#define LSO_CONST __attribute__((address_space(4)))

// ------------------------------------------------------------- the table

// Written by small kernels whose arguments carry the entries (nothing is read
// from host memory later): 32 KiB of arguments at a time, or 2 KiB for the
// few matrices of most calls.  308 matrices: one launch against nine of 4 KiB
// (20 us).
template <uint32_t kCount>
struct NsTablePart {
    NsMat* dst;
    uint32_t count;
    uint32_t pad;
    NsMat src[kCount];
};
constexpr uint32_t kWriteFew = 19, kWriteMany = 314;
static_assert(sizeof(NsTablePart<kWriteFew>) <= 2048 && sizeof(NsTablePart<kWriteMany>) <= 32768, "writer arguments");

template <uint32_t kCount>
__global__ void __launch_bounds__(64) ns_table_kernel(const NsTablePart<kCount> part)
{
    const uint32_t i = blockIdx.x * 64 + threadIdx.x;
    if (i < part.count) part.dst[i] = part.src[i];
}

template <uint32_t kCount>
hipError_t write_table(NsMat* dst, const NsMat* src, uint32_t count, hipStream_t s)
{
    NsTablePart<kCount> part;
    part.dst = dst;
    part.count = count;
    part.pad = 0;
    for (uint32_t j = 0; j < kCount; ++j) part.src[j] = src[j < count ? j : 0];
    return launch(ns_table_kernel<kCount>, dim3((count + 63) / 64), dim3(64), s, part);
}

__device__ __forceinline__ NsMat load_mat(const NsMat* tab, uint32_t i)
{
    return *reinterpret_cast<const NsMat*>(reinterpret_cast<const char*>(tab) + static_cast<uint64_t>(i) * sizeof(NsMat));
}

// The matrix that workgroup `index` of a launch belongs to: through the
// launch's runs of alike matrices, or else the last of n whose first index
// (field F) is <= index.
template <uint32_t NsMat::*F>
__device__ __forceinline__ uint32_t find_mat(const NsMat* tab, uint32_t n, const NsIndex& x, uint32_t index)
{
    if (x.runs > 0) {
        uint32_t first = x.first[0], mat = x.first_mat[0], each = x.each[0];
#pragma unroll
        for (int r = 1; r < kNsRuns; ++r)
            if (static_cast<uint32_t>(r) < x.runs && x.first[r] <= index) {
                first = x.first[r];
                mat = x.first_mat[r];
                each = x.each[r];
            }
        return mat + (index - first) / each;
    }
    uint32_t lo = 0, hi = n;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (tab[mid].*F <= index) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ------------------------------------------------------ elements of u

__device__ __forceinline__ float load_src(const NsMat& m, uint64_t i)
{
    return (m.flags & kNsSrcF32) ? static_cast<const float*>(m.src)[i]
                                 : bf16_widen(static_cast<const uint16_t*>(m.src)[i]);
}

__device__ __forceinline__ f32x4 load_src4(const NsMat& m, uint64_t i)
{
    if (m.flags & kNsSrcF32) return *reinterpret_cast<const f32x4*>(static_cast<const float*>(m.src) + i);
    const u32x2 h = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(m.src) + i);
    return f32x4{bf16_widen(h.x & 0xFFFFu), bf16_widen(h.x >> 16), bf16_widen(h.y & 0xFFFFu), bf16_widen(h.y >> 16)};
}

// The new momentum of the old one m and the gradient g, and u of the new one.
__device__ __forceinline__ float new_momentum(const NsMat& m, float old, float g) { return fmaf(m.beta, old, m.c1 * g); }

__device__ __forceinline__ float lookahead(const NsMat& m, float m1, float g)
{
    return (m.flags & kNsNesterov) ? fmaf(m.beta, m1, m.c1 * g) : m1;
}

// u of element (r, c); kFirst: m holds the old momentum and takes the new.
template <bool kFirst>
__device__ __forceinline__ float load_u(const NsMat& m, uint32_t r, uint32_t c)
{
    const float g = load_src(m, static_cast<uint64_t>(r) * m.ld_src + c);
    if (!(m.flags & kNsMuon)) return g;
    float* p = m.m + static_cast<uint64_t>(r) * m.cols + c;
    float m1 = *p;
    if (kFirst) {
        m1 = new_momentum(m, m1, g);
        *p = m1;
    }
    return lookahead(m, m1, g);
}

// u of elements (r, c .. c + 3), zeros outside the matrix.
template <bool kFirst>
__device__ __forceinline__ f32x4 load_u4(const NsMat& m, uint32_t r, uint32_t c)
{
    f32x4 u = {0.0f, 0.0f, 0.0f, 0.0f};
    if (r >= m.rows || c >= m.cols) return u;
    if (m.flags & kNsQuads) {
        const f32x4 g = load_src4(m, static_cast<uint64_t>(r) * m.ld_src + c);
        if (!(m.flags & kNsMuon)) return g;
        f32x4* p = reinterpret_cast<f32x4*>(m.m + static_cast<uint64_t>(r) * m.cols + c);
        f32x4 m1 = *p;
        if (kFirst) {
#pragma unroll
            for (int e = 0; e < 4; ++e) m1[e] = new_momentum(m, m1[e], g[e]);
            *p = m1;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = lookahead(m, m1[e], g[e]);
        return u;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (c + e < m.cols) u[e] = load_u<kFirst>(m, r, c + e);
    return u;
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

__device__ __forceinline__ u32x2 bf16_rne4(f32x4 v)
{
    return u32x2{bf16_rne(v.x) | (bf16_rne(v.y) << 16), bf16_rne(v.z) | (bf16_rne(v.w) << 16)};
}

// y of elements (r, c .. c + 3) as far as the matrix goes; old: their master
// weights, read before (update, kNsQuads).
__device__ __forceinline__ void put_result4(const NsMat& m, uint32_t r, uint32_t c, f32x4 o, f32x4 old)
{
    if (r >= m.rows || c >= m.cols) return;
    if (!(m.flags & kNsQuads)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < m.cols) put_result(m, r, c + e, o[e]);
        return;
    }
    if (m.flags & kNsMuon) {
        const uint64_t i = static_cast<uint64_t>(r) * m.cols + c;
        f32x4 p;
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = fmaf(m.step, o[e], m.keep * old[e]);
        *reinterpret_cast<f32x4*>(m.master + i) = p;
        if (m.dst) *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(m.dst) + i) = bf16_rne4(p);
        return;
    }
    const uint64_t i = static_cast<uint64_t>(r) * m.ld_dst + c;
    if (m.flags & kNsDstF32) *reinterpret_cast<f32x4*>(static_cast<float*>(m.dst) + i) = o;
    else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(m.dst) + i) = bf16_rne4(o);
}

__device__ __forceinline__ f32x4 old_master4(const NsMat& m, uint32_t r, uint32_t c)
{
    if ((m.flags & (kNsMuon | kNsQuads)) != (kNsMuon | kNsQuads) || r >= m.rows || c >= m.cols) return f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    return *reinterpret_cast<const f32x4*>(m.master + static_cast<uint64_t>(r) * m.cols + c);
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

__global__ void __launch_bounds__(256) ns_norm_kernel(const NsMat* tab, uint32_t n, NsIndex index, NsLayout layout, uint32_t* counters,
                                                      uint32_t ncounters)
{
    // the products' counters start at zero
    for (uint32_t k = blockIdx.x * 256 + threadIdx.x; k < ncounters; k += gridDim.x * 256) counters[k] = 0;
    const uint32_t i = find_mat<&NsMat::prep0>(tab, n, index, blockIdx.x);
    const NsMat m = load_mat(tab, i);
    uint32_t r0, c0;
    prep_tile(m, blockIdx.x - m.prep0, r0, c0);
    const uint32_t c = c0 + (threadIdx.x & 15u) * 4, r = r0 + (threadIdx.x >> 4);
    f32x4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = load_u4<true>(m, r + 16 * k, c);
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum = fma(static_cast<double>(u[k][e]), static_cast<double>(u[k][e]), sum);
    sum = group_sum<256>(sum);
    if (threadIdx.x == 0) {
        const NsWork w = ns_work(m.mp, m.np, layout);
        reinterpret_cast<double*>(m.work + w.partial)[blockIdx.x - m.prep0] = sum;
    }
}

// What X_0 is made with.  X_0 has the norm |u| / (|u| + eps), which is 1
// unless u is about as small as eps.  A small X_0 would leave FP16's range
// (its scale is fixed), so the path works on X 2^e with e >= 0 chosen to
// bring the norm of X_0 to [1/2, 2): with S' = S 2^2e the polynomial is
// a + b 2^-2e S' + c 2^-4e S'^2, and each step lowers e by as many powers of
// two as X can have grown by, or raises it by as many as X must have shrunk
// by (five steps of 0.02 X would leave FP16's range as well).
struct NsScaling {
    double inv;   // 2^e / (|u|_F + eps)
    int e;
};

// One workgroup per matrix.
__global__ void __launch_bounds__(1024) ns_scale_kernel(const NsMat* tab, NsLayout layout, double eps)
{
    const NsMat m = load_mat(tab, blockIdx.x);
    const NsWork w = ns_work(m.mp, m.np, layout);
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

// Where the 16 bytes of term `term` of values (row, c .. c + 7) of an operand
// are (c a multiple of 8, ld its padded row length).  The pieces of a row in
// a block are permuted by the row's number, so that the sixteen lanes which
// read LDS together (64 banks) hit all banks once a block has been copied
// there as it is.
template <int kTerms>
__device__ __forceinline__ uint32_t swizzle(uint32_t row)
{
    return kTerms == 2 ? ((row >> 2) & 3u) : ((row >> 3) & 1u);
}

template <int kT, int kTerms>
__device__ __forceinline__ uint64_t piece_at(uint32_t row, uint32_t ld, uint32_t c, uint32_t term)
{
    const uint32_t r = row % kT, piece = (term * 2 + (c % 16) / 8) ^ swizzle<kTerms>(r);
    return (static_cast<uint64_t>(row / kT) * (ld / 16) + c / 16) * (kT * 32 * kTerms) + r * (32 * kTerms) + piece * 16;
}

// Eight consecutive values v (already scaled) as FP16 terms.
template <int kT, int kTerms>
__device__ __forceinline__ void put_terms(char* base, uint32_t row, uint32_t ld, uint32_t c, const float (&v)[8])
{
    f16x8 h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        h[e] = static_cast<_Float16>(v[e]);
        l[e] = static_cast<_Float16>(v[e] - static_cast<float>(h[e]));
    }
    *reinterpret_cast<f16x8*>(base + piece_at<kT, kTerms>(row, ld, c, 0)) = h;
    if (kTerms == 2) *reinterpret_cast<f16x8*>(base + piece_at<kT, kTerms>(row, ld, c, 1)) = l;
}

// Eight consecutive values, times kNsScale.
template <int kT, int kTerms>
__device__ __forceinline__ void get_terms(const char* base, uint32_t row, uint32_t ld, uint32_t c, float (&v)[8])
{
    const f16x8 h = *reinterpret_cast<const f16x8*>(base + piece_at<kT, kTerms>(row, ld, c, 0));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(h[e]);
    if (kTerms == 2) {
        const f16x8 l = *reinterpret_cast<const f16x8*>(base + piece_at<kT, kTerms>(row, ld, c, 1));
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += static_cast<float>(l[e]);
    }
}

// X_0 and its transpose from u, zeros in the padding.
template <int kT, int kXTerms, int kXtTerms>
__global__ void __launch_bounds__(256) ns_split_kernel(const NsMat* tab, uint32_t n, NsIndex index, NsLayout layout)
{
    __shared__ float tile[kNsPrep][kNsPrep + 1];
    const uint32_t i = find_mat<&NsMat::prep0>(tab, n, index, blockIdx.x);
    const NsMat m = load_mat(tab, i);
    const NsWork w = ns_work(m.mp, m.np, layout);
    uint32_t r0, c0;
    prep_tile(m, blockIdx.x - m.prep0, r0, c0);
    const double inv = reinterpret_cast<const NsScaling*>(m.work + w.inv)->inv;
    const uint32_t cc = (threadIdx.x & 15u) * 4, rr = threadIdx.x >> 4;
    f32x4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = load_u4<false>(m, r0 + rr + 16 * k, c0 + cc);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            tile[rr + 16 * k][cc + e] = static_cast<float>(static_cast<double>(u[k][e]) * inv) * kNsScale;
    __syncthreads();
    const bool tall = (m.flags & kNsTall) != 0;
    char* xt = m.work + w.xt[0];
    char* x = m.work + w.x;
    // natural orientation: rows x cols is X, or X^T if tall; two lanes per row of a block
    for (uint32_t v = threadIdx.x; v < kNsPrep * kNsPrep / 8; v += 256) {
        const uint32_t c = (v & 1u) * 8 + v / (kNsPrep * 2) * 16, r = (v >> 1) % kNsPrep;
        float a[8], b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[e] = tile[r][c + e];
            b[e] = tile[c + e][r];
        }
        if (tall) {
            put_terms<kT, kXtTerms>(xt, r0 + r, m.mp, c0 + c, a);
            put_terms<kT, kXTerms>(x, c0 + r, m.np, r0 + c, b);
        } else {
            put_terms<kT, kXTerms>(x, r0 + r, m.np, c0 + c, a);
            put_terms<kT, kXtTerms>(xt, c0 + r, m.mp, r0 + c, b);
        }
    }
}

// ------------------------------------------------------ general path: products
//
// D[i][j] = sum over k of A[i][k] B[j][k], one tile of kT x kT per workgroup.
// kT = 64 or 128: four waves, a quarter each; kT = 256: eight waves, 128 x 64 each;
// in matrix-core tiles of 32 x 32.  A stage is one block of each operand (two
// where both have one term); stages go round four buffers in LDS, loaded
// straight to LDS three stages ahead of the one that is multiplied.
//
// Where a launch has too few tiles for the 256 CUs, the summed index of a tile
// is cut into parts, one workgroup each.  Each leaves its FP32 sums in the
// workspace and the last one to finish (a counter per tile) adds them up in
// the order of the parts, so the result does not depend on which that is.
// Nobody waits for another workgroup.

// Copy kBytes from g to lds, by all waves (where there is less than a load for
// each, several make the same one, so that all count alike).
template <uint32_t kWaves, uint32_t kBytes>
__device__ __forceinline__ void load_stage(const char* g, char* lds, uint32_t wave, uint32_t lane)
{
    constexpr uint32_t kAll = kBytes / 1024, kEach = kAll < kWaves ? 1 : kAll / kWaves;
    static_assert(kAll * 1024 == kBytes && (kAll < kWaves ? kWaves % kAll == 0 : kAll % kWaves == 0), "whole loads");
#pragma unroll
    for (uint32_t q = 0; q < kEach; ++q) {
        const uint32_t at = (wave * kEach + q) % kAll * 1024;
        __builtin_amdgcn_global_load_lds(
            reinterpret_cast<const __attribute__((address_space(1))) uint32_t*>(reinterpret_cast<uintptr_t>(g + at + lane * 16)),
            (__attribute__((address_space(3))) uint32_t*)(lds + at), 16, 0, 0);
    }
}

// Fragments of a stage: at LDS addresses a0 and a1 four, two or one of them
// each, kA bytes apart, likewise two or one at b0 (and b1).  The reads and
// the wait for them are one asm block, because the compiler would put a wait
// for the loads of later stages (which go to other buffers) before reads of
// LDS that it sees.
template <int kA, int kB>
__device__ __forceinline__ void read_4_2(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, f16x8 (&fa)[2][4], f16x8 (&fb)[2][2])
{
    asm volatile("ds_read_b128 %0, %12\n\tds_read_b128 %8, %14\n\tds_read_b128 %9, %14 offset:%17\n\t"
                 "ds_read_b128 %1, %12 offset:%16\n\tds_read_b128 %2, %12 offset:2*%16\n\tds_read_b128 %3, %12 offset:3*%16\n\t"
                 "ds_read_b128 %10, %15\n\tds_read_b128 %11, %15 offset:%17\n\t"
                 "ds_read_b128 %4, %13\n\tds_read_b128 %5, %13 offset:%16\n\t"
                 "ds_read_b128 %6, %13 offset:2*%16\n\tds_read_b128 %7, %13 offset:3*%16\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(fa[0][0]), "=&v"(fa[0][1]), "=&v"(fa[0][2]), "=&v"(fa[0][3]), "=&v"(fa[1][0]), "=&v"(fa[1][1]),
                   "=&v"(fa[1][2]), "=&v"(fa[1][3]), "=&v"(fb[0][0]), "=&v"(fb[0][1]), "=&v"(fb[1][0]), "=&v"(fb[1][1])
                 : "v"(a0), "v"(a1), "v"(b0), "v"(b1), "n"(kA), "n"(kB)
                 : "memory");
}

template <int kA, int kB>
__device__ __forceinline__ void read_4_1(uint32_t a0, uint32_t a1, uint32_t b0, f16x8 (&fa)[2][4], f16x8 (&fb)[1][2])
{
    asm volatile("ds_read_b128 %0, %10\n\tds_read_b128 %8, %12\n\tds_read_b128 %9, %12 offset:%14\n\t"
                 "ds_read_b128 %1, %10 offset:%13\n\tds_read_b128 %2, %10 offset:2*%13\n\tds_read_b128 %3, %10 offset:3*%13\n\t"
                 "ds_read_b128 %4, %11\n\tds_read_b128 %5, %11 offset:%13\n\t"
                 "ds_read_b128 %6, %11 offset:2*%13\n\tds_read_b128 %7, %11 offset:3*%13\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(fa[0][0]), "=&v"(fa[0][1]), "=&v"(fa[0][2]), "=&v"(fa[0][3]), "=&v"(fa[1][0]), "=&v"(fa[1][1]),
                   "=&v"(fa[1][2]), "=&v"(fa[1][3]), "=&v"(fb[0][0]), "=&v"(fb[0][1])
                 : "v"(a0), "v"(a1), "v"(b0), "n"(kA), "n"(kB)
                 : "memory");
}

template <int kA, int kB>
__device__ __forceinline__ void read_1_2(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, f16x8 (&fa)[2][1], f16x8 (&fb)[2][1])
{
    asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %2, %6\n\tds_read_b128 %3, %7\n\tds_read_b128 %1, %5\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(fa[0][0]), "=&v"(fa[1][0]), "=&v"(fb[0][0]), "=&v"(fb[1][0])
                 : "v"(a0), "v"(a1), "v"(b0), "v"(b1)
                 : "memory");
}

template <int kA, int kB>
__device__ __forceinline__ void read_1_1(uint32_t a0, uint32_t a1, uint32_t b0, f16x8 (&fa)[2][1], f16x8 (&fb)[1][1])
{
    asm volatile("ds_read_b128 %0, %3\n\tds_read_b128 %2, %5\n\tds_read_b128 %1, %4\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(fa[0][0]), "=&v"(fa[1][0]), "=&v"(fb[0][0])
                 : "v"(a0), "v"(a1), "v"(b0)
                 : "memory");
}

template <int kA, int kB>
__device__ __forceinline__ void read_2_2(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, f16x8 (&fa)[2][2], f16x8 (&fb)[2][2])
{
    asm volatile("ds_read_b128 %0, %8\n\tds_read_b128 %4, %10\n\tds_read_b128 %5, %10 offset:%13\n\tds_read_b128 %1, %8 offset:%12\n\t"
                 "ds_read_b128 %6, %11\n\tds_read_b128 %7, %11 offset:%13\n\tds_read_b128 %2, %9\n\tds_read_b128 %3, %9 offset:%12\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(fa[0][0]), "=&v"(fa[0][1]), "=&v"(fa[1][0]), "=&v"(fa[1][1]), "=&v"(fb[0][0]), "=&v"(fb[0][1]),
                   "=&v"(fb[1][0]), "=&v"(fb[1][1])
                 : "v"(a0), "v"(a1), "v"(b0), "v"(b1), "n"(kA), "n"(kB)
                 : "memory");
}

template <int kA, int kB>
__device__ __forceinline__ void read_2_1(uint32_t a0, uint32_t a1, uint32_t b0, f16x8 (&fa)[2][2], f16x8 (&fb)[1][2])
{
    asm volatile("ds_read_b128 %0, %6\n\tds_read_b128 %4, %8\n\tds_read_b128 %5, %8 offset:%10\n\tds_read_b128 %1, %6 offset:%9\n\t"
                 "ds_read_b128 %2, %7\n\tds_read_b128 %3, %7 offset:%9\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(fa[0][0]), "=&v"(fa[0][1]), "=&v"(fa[1][0]), "=&v"(fa[1][1]), "=&v"(fb[0][0]), "=&v"(fb[0][1])
                 : "v"(a0), "v"(a1), "v"(b0), "n"(kA), "n"(kB)
                 : "memory");
}

// Meetings of a workgroup's waves.  A wave's loads to LDS, or its reads of LDS,
// are waited for where the others go on to read, or overwrite, what they
// touch.  The empty asm keeps memory accesses on their side.
__device__ __forceinline__ void meet()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" : : : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Until at most kLeft loads of this wave are on their way, and its reads of
// LDS are done.
template <int kLeft>
__device__ __forceinline__ void wait_loads()
{
    static_assert(kLeft < 16, "the count's low bits");
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" : : : "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | kLeft);   // vmcnt(kLeft) lgkmcnt(0)
}

template <int kLeft>
__device__ __forceinline__ void wait_loads_and_meet()
{
    wait_loads<kLeft>();
    meet();
}

// What a product makes: S of X (kGram), a I + b S + c S^2 of S (kPoly), the
// product of two squares that commute (kSquare; symmetric like them), the
// next X and its transpose (kApply), or the result (kLast).
enum { kGram, kPoly, kSquare, kApply, kLast };

struct ProductArgs {
    const NsMat* tab;
    float* parts;        // sums of the parts, [unit][kT * kT]
    uint32_t* counters;  // finished parts, per tile of the launch; zero between launches
    uint32_t n;
    NsIndex index;
    NsLayout layout;
    uint32_t turn;       // which transpose of X is read
    uint32_t a_square, b_square, out_square;   // which squares are read and written
    uint32_t depth;      // stages per part
    double ca, cb, cc;   // coefficients of the step (kPoly)
    int16_t shift[kNsMaxSteps];   // each step's, as in NsCall
    uint32_t step;
};

// e behind a step; it stays at 0 or above.
__device__ __forceinline__ int step_scale(int e, int shift) { return e > shift ? e - shift : 0; }

// Tile number k of the tiles on and under the diagonal of tm x tm, in bands
// of four rows, down the columns of a band: tiles near each other in this
// order share their operands' rows.
__device__ __forceinline__ void lower_tile(uint32_t k, uint32_t tm, uint32_t& ti, uint32_t& tj)
{
    // band g starts at 8 g^2 + 2 g
    uint32_t g = static_cast<uint32_t>((sqrtf(1.0f + 8.0f * static_cast<float>(k)) - 1.0f) * 0.125f);
    while (8 * g * g + 2 * g > k) --g;
    while (8 * (g + 1) * (g + 1) + 2 * (g + 1) <= k) ++g;
    uint32_t at = k - (8 * g * g + 2 * g), left = tm - 4 * g < 4 ? tm - 4 * g : 4;
    const uint32_t whole = left * (4 * g + 1);   // columns up to the band's first row
    if (at < whole) {
        tj = at / left;
        ti = 4 * g + at % left;
        return;
    }
    at -= whole;
    tj = 4 * g + 1;
    for (--left; at >= left; --left, ++tj) at -= left;
    ti = tj + at;
}

// Tile number k of tn x tm, in bands of four rows, down the columns of a band.
__device__ __forceinline__ void band_tile(uint32_t k, uint32_t tn, uint32_t tm, uint32_t& ti, uint32_t& tj)
{
    const uint32_t g = k / (4 * tm), at = k - g * 4 * tm, left = tn - 4 * g < 4 ? tn - 4 * g : 4;
    tj = at / left;
    ti = 4 * g + at % left;
}

template <int kT, int kTermsA, int kTermsB, int kKind, int kTermsOut>
__global__ void __launch_bounds__(kT == 256 ? 512 : 256, 2) ns_product_kernel(const ProductArgs args)
{
    constexpr int kWaves = kT == 256 ? 8 : 4, kThreads = kWaves * 64;
    constexpr int kWm = kT / 2, kWn = kT == 256 ? 64 : kT / 2;            // a wave's part of the tile
    constexpr int kX = kWm / 32, kY = kWn / 32;                           // in matrix-core tiles
    // blocks of each operand in a stage (squares of small calls, whose stages
    // would be all meetings: 1000 x 777 and smaller 264 against 353 us; tiles of
    // X come in numbers and want the LDS for more workgroups)
    constexpr int kParts = ns_blocks(kT, kKind <= kSquare, kTermsA);
    constexpr int kValues = kParts * ((kTermsA == 1 && kTermsB == 1) ? 32 : 16);   // of the summed index per stage
    constexpr uint32_t kPartA = kT * 2 * kValues * kTermsA / kParts, kPartB = kT * 2 * kValues * kTermsB / kParts;
    constexpr int kRowA = 32 * kTermsA, kRowB = 32 * kTermsB;             // bytes of a row in a block
    constexpr uint32_t kStageA = kT * 2 * kValues * kTermsA, kStageB = kT * 2 * kValues * kTermsB, kStage = kStageA + kStageB;
    constexpr int kRing = 4;
    constexpr auto loads_of = [](uint32_t bytes) { return bytes / 1024 < kWaves ? 1 : static_cast<int>(bytes / 1024 / kWaves); };
    constexpr int kLoads = loads_of(kStageA) + loads_of(kStageB);         // of a wave per stage
    constexpr uint32_t kPitch = kT + 1, kStrip = kT < 128 ? kT : 128;                     // of the result tile in LDS
    constexpr uint32_t kLds = kRing * kStage > kStrip * kPitch * 4 ? kRing * kStage : kStrip * kPitch * 4;
    __shared__ __attribute__((aligned(128))) char lds[kLds];
    __shared__ uint32_t last_part;

    constexpr bool kSym = kKind <= kSquare;        // tiles on and under the diagonal, and their mirror images
    constexpr bool kOne = kTermsA == 1;            // of an apply: X^T has one term
    constexpr uint32_t NsMat::*kFirst = kKind == kGram ? &NsMat::gram0 : kSym ? &NsMat::square0 : kOne ? &NsMat::apply_one0 : &NsMat::apply0;
    const NsMat m = load_mat(args.tab, find_mat<kFirst>(args.tab, args.n, args.index, blockIdx.x));
    const NsWork w = ns_work(m.mp, m.np, args.layout);
    auto square = [&](uint32_t k) { return m.work + w.square + k * w.square_bytes; };
    const uint32_t tm = m.mp / kT, tn = m.np / kT, tiles = kSym ? tm * (tm + 1) / 2 : tm * tn, first = m.*kFirst;
    const uint32_t depth = kKind == kGram ? m.np : m.mp;
    const char* a = kKind == kGram ? m.work + w.x : kSym ? square(args.a_square) : m.work + ((args.turn & 1u) ? w.xt[1] : w.xt[0]);
    const char* b = kKind == kGram ? a : square(args.b_square);
    const uint32_t stages = depth / kValues, parts = (stages + args.depth - 1) / args.depth;
    // a matrix has a multiple of eight workgroups, which go round the eight
    // XCDs in turn; consecutive units of a matrix go to one XCD, neighbouring
    // tiles of the same part, which share rows
    const uint32_t units = tiles * parts, per = (units + 7) / 8, at = blockIdx.x - first;
    const uint32_t unit = (at & 7u) * per + (at >> 3);
    if (unit >= units) return;
    const uint32_t k = unit % tiles, part = unit / tiles;
    uint32_t ti, tj;
    if (kSym) lower_tile(k, tm, ti, tj);
    else band_tile(k, tn, tm, ti, tj);
    const uint32_t i0 = ti * kT, j0 = tj * kT;
    const uint32_t s0 = part * args.depth, s1 = s0 + args.depth < stages ? s0 + args.depth : stages;
    a += static_cast<uint64_t>(ti) * stages * kStageA;
    b += static_cast<uint64_t>(tj) * stages * kStageB;

    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)));
    const uint32_t wi = (kT == 256 ? wave >> 2 : wave >> 1) * kWm, wj = (kT == 256 ? wave & 3u : wave & 1u) * kWn;
    f32x16 acc[kX][kY];
#pragma unroll
    for (int x = 0; x < kX; ++x)
#pragma unroll
        for (int y = 0; y < kY; ++y)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[x][y][e] = 0.0f;

    // stage s (the last one again behind the end, so that the waits count alike)
    auto load_a = [&](uint32_t s) {
        load_stage<kWaves, kStageA>(a + static_cast<uint64_t>(s < s1 ? s : s1 - 1) * kStageA, lds + (s % kRing) * kStage, wave, lane);
    };
    auto load_b = [&](uint32_t s) {
        load_stage<kWaves, kStageB>(b + static_cast<uint64_t>(s < s1 ? s : s1 - 1) * kStageB, lds + (s % kRing) * kStage + kStageA, wave, lane);
    };
    // A stage is 16 values of two-term operands, whose second fragments are
    // the l terms, or 32 values of one-term operands, whose second fragments
    // are the second block.  A fragment is 32 rows by 16 values, eight per lane.
    constexpr int kNb = kTermsA == kTermsB ? 2 : 1;
    f16x8 fa[2][kX], fb[kNb][kY];
    const uint32_t row_a = wi + (lane & 31u), row_b = wj + (lane & 31u);
    // (the rows of a wave's other fragments are multiples of 32 further on: the same swizzle)
    const uint32_t pa = (lane >> 5) ^ swizzle<kTermsA>(row_a), pb = (lane >> 5) ^ swizzle<kTermsB>(row_b);
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds));
    const uint32_t at_a = lds0 + row_a * kRowA + pa * 16, at_b = lds0 + kStageA + row_b * kRowB + pb * 16;
    const uint32_t at_a1 = kTermsA == 2 ? lds0 + row_a * kRowA + (pa ^ 2u) * 16 : at_a + kT * kRowA;
    const uint32_t at_b1 = kTermsB == 2 ? lds0 + kStageA + row_b * kRowB + (pb ^ 2u) * 16 : at_b + kT * kRowB;
    auto read = [&](uint32_t s, uint32_t part) {
        const uint32_t in_a = (s % kRing) * kStage + part * kPartA, in_b = (s % kRing) * kStage + part * kPartB;
        if constexpr (kNb == 2) {
            if constexpr (kX == 4) read_4_2<32 * kRowA, 32 * kRowB>(in_a + at_a, in_a + at_a1, in_b + at_b, in_b + at_b1, fa, fb);
            else if constexpr (kX == 1) read_1_2<32 * kRowA, 32 * kRowB>(in_a + at_a, in_a + at_a1, in_b + at_b, in_b + at_b1, fa, fb);
            else read_2_2<32 * kRowA, 32 * kRowB>(in_a + at_a, in_a + at_a1, in_b + at_b, in_b + at_b1, fa, fb);
        } else {
            if constexpr (kX == 4) read_4_1<32 * kRowA, 32 * kRowB>(in_a + at_a, in_a + at_a1, in_b + at_b, fa, fb);
            else if constexpr (kX == 1) read_1_1<32 * kRowA, 32 * kRowB>(in_a + at_a, in_a + at_a1, in_b + at_b, fa, fb);
            else read_2_1<32 * kRowA, 32 * kRowB>(in_a + at_a, in_a + at_a1, in_b + at_b, fa, fb);
        }
    };
    auto product = [&](const f16x8 (&x8)[kX], const f16x8 (&y8)[kY]) {
#pragma unroll
        for (int x = 0; x < kX; ++x)
#pragma unroll
            for (int y = 0; y < kY; ++y) acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x8[x], y8[y], acc[x][y], 0, 0, 0);
    };
    // Multiply what has been read; in between, while the matrix cores are
    // busy, send for stage s.  Sent for beside the reads of LDS, the loads held
    // those up: the matrix cores were busy 58% of the time against 80% now,
    // the product of 8192 x 8192 and 8192 x 28672 took 10.0 against 8.7 ms.
    auto multiply = [&](uint32_t s, bool send) {
        product(fa[0], fb[0]);
        __builtin_amdgcn_sched_barrier(0);
        if (send) load_a(s);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (kTermsA == 1) {
            if (send) load_b(s);
            __builtin_amdgcn_sched_barrier(0);
            product(fa[1], fb[1]);                               // the second 16 values
        } else {
            if constexpr (kTermsB == 2) product(fa[0], fb[1]);   // h l
            __builtin_amdgcn_sched_barrier(0);
            if (send) load_b(s);
            __builtin_amdgcn_sched_barrier(0);
            product(fa[1], fb[0]);                               // l h
        }
    };
#pragma unroll
    for (uint32_t s = 0; s < 3; ++s) {
        load_a(s0 + s);
        load_b(s0 + s);
    }
    if (kT < 256) {
        for (uint32_t s = s0; s < s1; ++s) {
            wait_loads_and_meet<2 * kLoads>();   // stage s is here, stage s - 1 has been read
            for (int part = 0; part < kParts; ++part) {
                read(s, part);
                multiply(s + 3, part == 0);
            }
        }
    } else {
        // Two waves share a SIMD.  Waves 4 to 7 run one meeting behind waves 0
        // to 3, so that of the two one reads LDS while the other multiplies:
        // between two meetings a wave does one of the two for a stage.  A
        // buffer is loaded anew once both groups have read it; a stage has
        // arrived before the first group meets to read it.
        const bool second = wave >= 4;
        wait_loads_and_meet<2 * kLoads>();
        if (second) meet();
        for (uint32_t s = s0; s < s1; ++s) {
            read(s, 0);
            if (second) wait_loads<kLoads>();
            meet();
            __builtin_amdgcn_s_setprio(1);
            multiply(s + 3, true);
            __builtin_amdgcn_s_setprio(0);
            if (!second) wait_loads<2 * kLoads>();
            meet();
        }
        if (!second) meet();
    }
    wait_loads_and_meet<0>();

    if (parts > 1) {
        // This part's sums, in the registers' own order.  They go past the
        // XCD's L2 (device-scope stores and loads of 8 bytes): a fence that
        // writes the L2 back costs tens of microseconds here.
        typedef unsigned long long u64;
        u64* mine = reinterpret_cast<u64*>(args.parts) + (static_cast<uint64_t>(first) + unit) * (kT * kT / 2) + threadIdx.x;
#pragma unroll
        for (int x = 0; x < kX; ++x)
#pragma unroll
            for (int y = 0; y < kY; ++y)
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const u64 v = static_cast<u64>(__float_as_uint(acc[x][y][2 * q])) |
                                  (static_cast<u64>(__float_as_uint(acc[x][y][2 * q + 1])) << 32);
                    __hip_atomic_store(mine + ((x * kY + y) * 8 + q) * kThreads, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                }
        wait_loads_and_meet<0>();   // of every wave, its stores have reached memory
        if (threadIdx.x == 0) {
            uint32_t* counter = args.counters + first + k;
            const uint32_t done = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last_part = done == parts - 1;
            // for the next launch; nobody counts this tile any more
            if (done == parts - 1) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (!last_part) return;
        u64* all = mine - static_cast<uint64_t>(part) * tiles * (kT * kT / 2);
#pragma unroll
        for (int x = 0; x < kX; ++x)
#pragma unroll
            for (int y = 0; y < kY; ++y)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[x][y][e] = 0.0f;
        for (uint32_t p = 0; p < parts; ++p) {
            u64* from = all + static_cast<uint64_t>(p) * tiles * (kT * kT / 2);
#pragma unroll
            for (int x = 0; x < kX; ++x)
#pragma unroll
                for (int y = 0; y < kY; ++y) {
                    u64 v[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        v[q] = __hip_atomic_load(from + ((x * kY + y) * 8 + q) * kThreads, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        acc[x][y][2 * q] += __uint_as_float(static_cast<uint32_t>(v[q]));
                        acc[x][y][2 * q + 1] += __uint_as_float(static_cast<uint32_t>(v[q] >> 32));
                    }
                }
        }
    }

    // the tile through LDS, values times kNsScale (products carry its
    // square), kStrip rows at a time
    float unscale = 1.0f / kNsScale, ca = 0.0f, cb = 0.0f, cc = 0.0f;
    if (kKind == kPoly || kKind == kLast) {
        int before = reinterpret_cast<const NsScaling*>(m.work + w.inv)->e, after = 0;
#pragma unroll
        for (uint32_t k = 0; k < kNsMaxSteps; ++k) {
            if (k > args.step) break;
            if (k == args.step) after = step_scale(before, args.shift[k]);
            else before = step_scale(before, args.shift[k]);
        }
        const int up = after - before;
        if (kKind == kLast) unscale = ldexpf(1.0f / (kNsScale * kNsScale), -after);
        ca = static_cast<float>(ldexp(args.ca, up));
        cb = static_cast<float>(ldexp(args.cb, up - 2 * before));
        cc = static_cast<float>(ldexp(args.cc, up - 4 * before));
    }
    float* tile = reinterpret_cast<float*>(lds);
    for (uint32_t strip = 0; strip < kT; strip += kStrip) {
        __syncthreads();   // the stages, or the strip before, have been read
        if (wi / kStrip * kStrip == strip) {
#pragma unroll
            for (int x = 0; x < kX; ++x)
#pragma unroll
                for (int y = 0; y < kY; ++y)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const uint32_t i = wi + x * 32 + 8 * (e / 4) + 4 * (lane >> 5) + (e & 3);
                        const uint32_t j = wj + y * 32 + (lane & 31u);
                        tile[(i - strip) * kPitch + j] = acc[x][y][e] * unscale;
                    }
        }
        __syncthreads();
        const uint32_t is = i0 + strip;   // row of D that the strip starts at

        if (kKind == kLast) {
            // D is X'^T: element (i, j) is X'(j, i); rows of the natural
            // matrix are i if tall, else j
            const bool tall = (m.flags & kNsTall) != 0;
            constexpr uint32_t kQuads = kStrip * kT / 4 / kThreads;   // per thread, four at a time
            const uint32_t across = tall ? kT / 4 : kStrip / 4;
            const uint32_t rr = tall ? is : j0, cr = tall ? j0 : is;
            for (uint32_t q = 0; q < kQuads; q += 4) {
                uint32_t r[4], c[4];
                f32x4 old[4];
#pragma unroll
                for (uint32_t x = 0; x < 4; ++x) {
                    const uint32_t v = threadIdx.x + (q + x) * kThreads;
                    r[x] = v / across;
                    c[x] = v % across * 4;
                    old[x] = old_master4(m, rr + r[x], cr + c[x]);
                }
#pragma unroll
                for (uint32_t x = 0; x < 4; ++x) {
                    f32x4 o;
#pragma unroll
                    for (uint32_t e = 0; e < 4; ++e) o[e] = tall ? tile[r[x] * kPitch + c[x] + e] : tile[(c[x] + e) * kPitch + r[x]];
                    put_result4(m, rr + r[x], cr + c[x], o, old[x]);
                }
            }
            continue;
        }
        char* out_rows;      // takes D
        char* out_cols;      // takes D transposed
        uint32_t ld_rows, ld_cols;
        if (kSym) {
            out_rows = out_cols = square(args.out_square);
            ld_rows = ld_cols = m.mp;
        } else {
            out_rows = m.work + ((args.turn & 1u) ? w.xt[0] : w.xt[1]);
            out_cols = m.work + w.x;
            ld_rows = m.mp;
            ld_cols = m.np;
        }
        // a I + b S + c S^2 from S^2, at elements (row, c .. c + 7)
        auto polynomial = [&](uint32_t row, uint32_t c, float (&d)[8]) {
            float sv[8];
            get_terms<kT, kTermsA>(square(args.a_square), row, m.mp, c, sv);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                d[e] = fmaf(cc, d[e], cb * sv[e]);
                if (row == c + e) d[e] += ca * kNsScale;
            }
        };
        // two lanes per row of a block
        for (uint32_t v = threadIdx.x; v < kStrip * kT / 8; v += kThreads) {
            float d[8];
            {
                const uint32_t c = (v & 1u) * 8 + v / (kStrip * 2) * 16, r = (v >> 1) % kStrip;
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = tile[r * kPitch + c + e];
                if (kKind == kPoly) polynomial(is + r, j0 + c, d);
                put_terms<kT, kTermsOut>(out_rows, is + r, ld_rows, j0 + c, d);
            }
            if (!kSym || ti != tj) {
                const uint32_t c = (v & 1u) * 8 + v / (kT * 2) * 16, r = (v >> 1) % kT;
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = tile[(c + e) * kPitch + r];
                if (kKind == kPoly) polynomial(j0 + r, is + c, d);
                put_terms<kT, kSym ? kTermsOut : kTermsB>(out_cols, j0 + r, ld_cols, is + c, d);   // X in the polynomial's terms
            }
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
// unscaled S.  Bound: two reads of u and launch latency; for sides of 33 to
// 64 the FP64 matrix instructions.  Measured (us) for those, here and in the
// general path in full precision: 308 of 64 x 2048 411 / 915, 2000 of 64 x 512 862 /
// 3045, one of 64 x 4096 75 / 106, of 64 x 262144 447 / 827, two of 64 x 64 68 / 68.

constexpr uint32_t kSmallPitch = kNsSmallChunk + 1;

// Four columns of the natural matrix that thread number v stages: quads of a
// row after another.  Returns the row and column; (p, x) is the first
// element's place in u (smaller side, long side) and `step` the way to the
// next one.
template <int kK>
__device__ __forceinline__ void small_quad(bool tall, uint32_t v, uint32_t l0, uint32_t& r, uint32_t& c, uint32_t& at, uint32_t& step)
{
    const uint32_t across = tall ? kK / 4 : kNsSmallChunk / 4, i = v / across, j = v % across * 4;
    r = tall ? l0 + i : i;
    c = tall ? j : l0 + j;
    at = tall ? j * kSmallPitch + i : i * kSmallPitch + j;
    step = tall ? kSmallPitch : 1;
}

// Stage u of long-side elements [l0, l0 + kNsSmallChunk) as u[p][x], zeros
// outside the matrix.
template <int kK, bool kFirst>
__device__ __forceinline__ void stage_u(const NsMat& m, uint32_t l0, float* u)
{
    const bool tall = (m.flags & kNsTall) != 0;
    constexpr int kQuads = kK / 4;   // per thread
    f32x4 q[kQuads];
    uint32_t at[kQuads], step;
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
        uint32_t r, c;
        small_quad<kK>(tall, threadIdx.x + k * 256, l0, r, c, at[k], step);
        q[k] = load_u4<kFirst>(m, r, c);
    }
#pragma unroll
    for (int k = 0; k < kQuads; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[at[k] + e * step] = q[k][e];
}

template <int kK>
__global__ void __launch_bounds__(256) ns_small_gram_kernel(const NsMat* tab, uint32_t n, NsIndex index)
{
    // FP64 matrix instructions: 16 x 16 products of 16 rows by 4 values, the
    // same register for both operands.  With kK = 8 rows 8 to 15 are the
    // first eight again at the other half of the chunk; with 32 the tiles
    // are (0, 0), (0, 1) and (1, 1); with 64 a wave makes a row of four tiles
    // from the whole chunk.  (A thread per product, with FP64 vector
    // instructions, took 14.4 against 13.2 us for 308 adapters: two loads
    // and two conversions for each.)
    constexpr int kTiles = kK == 32 ? 3 : 1, kRows = kK == 32 ? 2 : 1;
    constexpr uint32_t kSpan = kK == 8 ? kNsSmallChunk / 2 : kNsSmallChunk;   // values per row
    __shared__ float u[kK * kSmallPitch];
    __shared__ double part[kK == 64 ? 1 : kTiles * 4 * 256];   // [tile][wave][row][column]
    const NsMat m = load_mat(tab, find_mat<&NsMat::prep0>(tab, n, index, blockIdx.x));
    const uint32_t chunk = blockIdx.x - m.prep0, k = m.rows < m.cols ? m.rows : m.cols;
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    stage_u<kK, true>(m, chunk * kNsSmallChunk, u);
    __syncthreads();
    double* out = reinterpret_cast<double*>(m.work) + static_cast<uint64_t>(chunk) * k * k;
    if constexpr (kK == 64) {
        f64x4 sum[4] = {};
        const float* from = u + (lane & 15u) * kSmallPitch + (lane >> 4);
        const float* mine = from + wave * 16 * kSmallPitch;
#pragma unroll 4
        for (uint32_t x = 0; x < kNsSmallChunk; x += 4) {
            const double row = mine[x];
#pragma unroll
            for (int y = 0; y < 4; ++y)
                sum[y] = __builtin_amdgcn_mfma_f64_16x16x4f64(row, static_cast<double>(from[y * 16 * kSmallPitch + x]), sum[y], 0, 0, 0);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t p = wave * 16 + 4 * e + (lane >> 4), q = y * 16 + (lane & 15u);
                if (p < k && q < k) out[p * k + q] = sum[y][e];
            }
        return;
    }
    f64x4 acc[kTiles] = {};
    const uint32_t row = lane & 15u, at = wave * (kSpan / 4) + (lane >> 4);
    const float* from = kK == 8 ? u + (row & 7u) * kSmallPitch + (row >> 3) * kSpan + at : u + row * kSmallPitch + at;
#pragma unroll 4
    for (uint32_t x = 0; x < kSpan / 4; x += 4) {
        double a[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) a[r] = from[r * 16 * kSmallPitch + x];
        acc[0] = __builtin_amdgcn_mfma_f64_16x16x4f64(a[0], a[0], acc[0], 0, 0, 0);
        if constexpr (kRows == 2) {
            acc[1] = __builtin_amdgcn_mfma_f64_16x16x4f64(a[0], a[1], acc[1], 0, 0, 0);
            acc[2] = __builtin_amdgcn_mfma_f64_16x16x4f64(a[1], a[1], acc[2], 0, 0, 0);
        }
    }
    // element e of lane l: row 4 e + l / 16, column l % 16
#pragma unroll
    for (int y = 0; y < kTiles; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[((y * 4 + wave) * 16 + 4 * e + (lane >> 4)) * 16 + (lane & 15u)] = acc[y][e];
    __syncthreads();
    for (uint32_t v = threadIdx.x; v < kK * kK; v += 256) {
        uint32_t p = v / kK, q = v % kK;
        if (p >= k || q >= k) continue;
        uint32_t y = 0, r = p, c = q;
        if (kK == 32) {
            if (p > q) {   // the mirror image
                r = q;
                c = p;
            }
            y = c < 16 ? 0 : r < 16 ? 1 : 2;
            r &= 15u;
            c &= 15u;
        }
        double sum = 0.0;
#pragma unroll
        for (uint32_t w = 0; w < 4; ++w) {
            sum += part[((y * 4 + w) * 16 + r) * 16 + c];
            if (kK == 8) sum += part[((y * 4 + w) * 16 + r + 8) * 16 + c + 8];
        }
        out[p * k + q] = sum;
    }
}

struct SmallArgs {
    const NsMat* tab;
    uint32_t steps;
    double eps;
    double coef[3 * kNsMaxSteps];
};

// Threads of a workgroup of it.
constexpr int small_threads(int k) { return k == 64 ? 640 : k == 32 ? 256 : 64; }

// One workgroup per matrix.  kK = 8: a thread per element.  kK = 16 to 64: a
// wave per 16 x 16 tile (of 64 x 64 on and under the diagonal, as all of these
// are polynomials in S), FP64 matrix instructions (32 x 32: 26 against 12 us
// with two by two elements per thread).
template <int kK>
__global__ void __launch_bounds__(small_threads(kK)) ns_small_iterate_kernel(const SmallArgs args)
{
    constexpr int kE = kK == 8 ? 1 : 4;   // elements per thread
    __shared__ double s[kK][kK + 1], t[kK][kK + 1], p[kK][kK + 1], q[kK][kK + 1];
    const NsMat m = load_mat(args.tab, blockIdx.x);
    const uint32_t k = m.rows < m.cols ? m.rows : m.cols, l = m.rows < m.cols ? m.cols : m.rows;
    const uint32_t chunks = (l + kNsSmallChunk - 1) / kNsSmallChunk;
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    // the wave's tile
    uint32_t ti = kK == 32 ? wave >> 1 : 0, tj = kK == 32 ? wave & 1u : wave;
    if (kK == 64) {
        for (; tj > ti; ++ti) tj -= ti + 1;
    }
    ti *= 16;
    tj *= 16;
    // element e of a thread: row i + e * 4, column j
    const uint32_t i = kK == 8 ? lane >> 3 : ti + (lane >> 4), j = kK == 8 ? lane & 7u : tj + (lane & 15u);
    const double* part = reinterpret_cast<const double*>(m.work);
    auto put = [&](double (&to)[kK][kK + 1], const double (&from)[kE]) {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            to[i + e * 4][j] = from[e];
            if (kK == 64 && ti != tj) to[j][i + e * 4] = from[e];
        }
    };
    double v[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const uint32_t ii = i + e * 4;
        double sum = 0.0;
        if (ii < k && j < k) {
            const double* from = part + ii * k + j;
#pragma unroll 8
            for (uint32_t c = 0; c < chunks; ++c) sum += from[static_cast<uint64_t>(c) * k * k];
        }
        v[e] = sum;
    }
    put(s, v);
    __syncthreads();
    double trace = 0.0;
#pragma unroll
    for (int x = 0; x < kK; ++x) trace += s[x][x];   // zeros from k on
    const double inv = 1.0 / (sqrt(trace) + args.eps);
    __syncthreads();
    auto product = [&](const double (&a)[kK][kK + 1], const double (&b)[kK][kK + 1], double (&out)[kE]) {
        if constexpr (kK == 8) {
            double sum = 0.0;
#pragma unroll
            for (int e = 0; e < kK; ++e) sum = fma(a[i][e], b[e][j], sum);
            out[0] = sum;
        } else {
            f64x4 sum = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
            for (uint32_t e = 0; e < kK; e += 4)
                sum = __builtin_amdgcn_mfma_f64_16x16x4f64(a[ti + (lane & 15u)][e + (lane >> 4)],
                                                           b[e + (lane >> 4)][j], sum, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < kE; ++e) out[e] = sum[e];
        }
    };
    double w[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        v[e] = v[e] * inv * inv;
        w[e] = i + e * 4 == j ? inv : 0.0;   // Q_0 carries the scaling of u to X_0
    }
    put(s, v);
    put(q, w);
    __syncthreads();
    for (uint32_t n = 0; n < args.steps; ++n) {
        const double a = args.coef[3 * n], b = args.coef[3 * n + 1], c = args.coef[3 * n + 2];
        product(s, s, w);
#pragma unroll
        for (int e = 0; e < kE; ++e) w[e] = (i + e * 4 == j ? a : 0.0) + b * s[i + e * 4][j] + c * w[e];
        put(p, w);
        __syncthreads();
        const bool more = n + 1 < args.steps;
        if (more) {
            product(p, s, w);
            put(t, w);
        }
        product(p, q, w);
        __syncthreads();
        put(q, w);
        if (more) {
            product(t, p, w);
            put(s, w);
        }
        __syncthreads();
    }
    double* out = reinterpret_cast<double*>(m.work) + static_cast<uint64_t>(chunks) * k * k;
    for (uint32_t x = threadIdx.x; x < kK * kK; x += small_threads(kK)) out[x] = q[x / kK][x % kK];   // zeros from k on
}

template <int kK>
__global__ void __launch_bounds__(256) ns_small_apply_kernel(const NsMat* tab, uint32_t n, NsIndex index)
{
    __shared__ float u[kK * kSmallPitch];
    const NsMat m = load_mat(tab, find_mat<&NsMat::prep0>(tab, n, index, blockIdx.x));
    const uint32_t l0 = (blockIdx.x - m.prep0) * kNsSmallChunk;
    const uint32_t k = m.rows < m.cols ? m.rows : m.cols, l = m.rows < m.cols ? m.cols : m.rows;
    const uint32_t chunks = (l + kNsSmallChunk - 1) / kNsSmallChunk;
    const bool tall = (m.flags & kNsTall) != 0;
    constexpr uint32_t kPitch = kK == 64 ? kK + 1 : kK;
    __shared__ double q[kK * kPitch];
    const double* src = reinterpret_cast<const double*>(m.work) + static_cast<uint64_t>(chunks) * k * k;
    for (uint32_t v = threadIdx.x; v < kK * kK; v += 256) q[v / kK * kPitch + v % kK] = src[v];
    constexpr int kQuads = kK / 4;
    f32x4 old[kQuads];
#pragma unroll
    for (int x = 0; x < kQuads; ++x) {
        uint32_t r, c, at, step;
        small_quad<kK>(tall, threadIdx.x + x * 256, l0, r, c, at, step);
        old[x] = old_master4(m, r, c);
    }
    stage_u<kK, false>(m, l0, u);
    __syncthreads();
    if constexpr (kK == 64) {
        // a wave's 64 columns of u, which no other wave touches: a tile of
        // four by four matrix instructions' results (a thread per column
        // would wait for LDS, two reads of q for each four products)
        const uint32_t lane = threadIdx.x & 63u, c0 = (threadIdx.x & ~63u) + (lane & 15u), e0 = lane >> 4;
        f64x4 sum[4][4] = {};
        for (uint32_t e = 0; e < kK; e += 4) {
            double a[4], b[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                a[y] = q[(y * 16 + (lane & 15u)) * kPitch + e + e0];
                b[y] = u[(e + e0) * kSmallPitch + c0 + y * 16];
            }
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int x = 0; x < 4; ++x) sum[y][x] = __builtin_amdgcn_mfma_f64_16x16x4f64(a[y], b[x], sum[y][x], 0, 0, 0);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) u[(y * 16 + 4 * e + e0) * kSmallPitch + c0 + x * 16] = static_cast<float>(sum[y][x][e]);
    } else {
        // one column of u per thread, four rows of the result at a time
        float col[kK];
#pragma unroll
        for (int e = 0; e < kK; ++e) col[e] = u[e * kSmallPitch + threadIdx.x];
        for (uint32_t p = 0; p < k; p += 4) {
            double v[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
            for (int e = 0; e < kK; ++e) {
                const double x = col[e];
#pragma unroll
                for (int y = 0; y < 4; ++y) v[y] = fma(q[(p + y) * kPitch + e], x, v[y]);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) u[(p + y) * kSmallPitch + threadIdx.x] = static_cast<float>(v[y]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kQuads; ++x) {
        uint32_t r, c, at, step;
        small_quad<kK>(tall, threadIdx.x + x * 256, l0, r, c, at, step);
        f32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = u[at + e * step];
        put_result4(m, r, c, o, old[x]);
    }
}

template <int kK>
hipError_t launch_small(const NsCall& c, const NsMat* tab, uint32_t n, uint32_t chunks, const NsIndex& index, hipStream_t s)
{
    SmallArgs args{};
    args.tab = tab;
    args.steps = c.steps;
    args.eps = c.eps;
    for (uint32_t k = 0; k < 3 * c.steps; ++k) args.coef[k] = c.coef[k];
    hipError_t err = launch(ns_small_gram_kernel<kK>, dim3(chunks), dim3(256), s, tab, n, index);
    if (err == hipSuccess) err = launch(ns_small_iterate_kernel<kK>, dim3(n), dim3(small_threads(kK)), s, args);
    if (err == hipSuccess) err = launch(ns_small_apply_kernel<kK>, dim3(chunks), dim3(256), s, tab, n, index);
    return err;
}

// The general path.  kTerms: of X as S reads it, and of what X is multiplied by.
template <int kT, int kTerms>
class BigLaunch {
public:
    BigLaunch(const NsCall& c, const NsMat* tab, hipStream_t s) : c_(c), s_(s)
    {
        args_.tab = tab;
        args_.parts = c.parts;
        args_.counters = c.counters;
        args_.n = c.nbig;
        args_.layout = c.layout;
        for (uint32_t k = 0; k < kNsMaxSteps; ++k) args_.shift[k] = c.shift[k];
    }

    hipError_t run()
    {
        const NsMat* tab = args_.tab;
        enqueue(ns_norm_kernel, c_.prep_tiles, 256, tab, c_.nbig, c_.prep_index, c_.layout, c_.counters, c_.ncounters);
        enqueue(ns_scale_kernel, c_.nbig, 1024, tab, c_.layout, c_.eps);
        enqueue(xt_terms(0) == 2 ? ns_split_kernel<kT, kTerms, 2> : ns_split_kernel<kT, kTerms, 1>, c_.prep_tiles, 256, tab, c_.nbig,
                c_.prep_index, c_.layout);
        for (uint32_t k = 0; k < c_.steps && err_ == hipSuccess;) {
            const bool pair = paired(k);
            gram();
            poly(k, 0, 1, !pair);
            if (pair) {
                square(1, 0, 2, false);        // P S
                square(2, 1, 0, false);        // S' = P S P
                poly(k + 1, 0, 3, false);      // P'
                square(3, 1, 2, true);         // Q = P' P
            }
            apply(k, pair ? k + 2 : k + 1, pair ? 2 : 1);
            k += pair ? 2 : 1;
        }
        return err_;
    }

private:
    // Nothing more is enqueued after an error.
    template <typename... P>
    void enqueue(void (*kernel)(P...), uint32_t groups, uint32_t threads, const typename as_is<P>::type&... args)
    {
        if (err_ == hipSuccess) err_ = lso::launch(kernel, dim3(groups), dim3(threads), s_, args...);
    }

    bool paired(uint32_t k) const { return c_.pairs && c_.pair[k]; }

    // Terms of X^T where step k reads it.  In half precision the last two
    // steps, taken singly, read one: what no later step magnifies is below
    // the rounding of S and the polynomial anyway.
    int xt_terms(uint32_t k) const { return kTerms == 2 || k + 2 < c_.steps || paired(k) ? 2 : 1; }

    template <int kA, int kB, int kKind, int kOut>
    void launch(const NsProduct& p)
    {
        args_.depth = p.depth;
        args_.index = p.index;
        enqueue(ns_product_kernel<kT, kA, kB, kKind, kOut>, p.units, kT == 256 ? 512 : 256, args_);
    }

    bool two_term_squares() const { return c_.layout.square_terms == 2; }

    void gram()
    {
        args_.out_square = 0;
        if (kTerms == 1 && !two_term_squares()) launch<kTerms, kTerms, kGram, 1>(c_.gram);
        else launch<kTerms, kTerms, kGram, 2>(c_.gram);
    }

    void squares(uint32_t a, uint32_t b, uint32_t out)
    {
        args_.a_square = a;
        args_.b_square = b;
        args_.out_square = out;
    }

    // The polynomial of step k in square `in`; multiplier: X is multiplied by it.
    void poly(uint32_t k, uint32_t in, uint32_t out, bool multiplier)
    {
        squares(in, in, out);
        args_.ca = c_.coef[3 * k];
        args_.cb = c_.coef[3 * k + 1];
        args_.cc = c_.coef[3 * k + 2];
        args_.step = k;
        if (!two_term_squares()) launch<1, 1, kPoly, 1>(c_.square);
        else if (multiplier) launch<2, 2, kPoly, kTerms>(c_.square);
        else launch<2, 2, kPoly, 2>(c_.square);
    }

    void square(uint32_t a, uint32_t b, uint32_t out, bool multiplier)
    {
        squares(a, b, out);
        if (multiplier) launch<2, 2, kSquare, kTerms>(c_.square);
        else launch<2, 2, kSquare, 2>(c_.square);
    }

    // X of step `next` from that of step k (the poly before has set what
    // kLast needs of the scaling).
    void apply(uint32_t k, uint32_t next, uint32_t by)
    {
        args_.b_square = by;
        const int from = xt_terms(k), to = next < c_.steps ? xt_terms(next) : 0;
        if constexpr (kTerms == 2) {
            if (to == 0) launch<2, 2, kLast, 1>(c_.apply);
            else launch<2, 2, kApply, 2>(c_.apply);
        } else if (from == 2) {
            if (to == 0) launch<2, 1, kLast, 1>(c_.apply);
            else if (to == 1) launch<2, 1, kApply, 1>(c_.apply);
            else launch<2, 1, kApply, 2>(c_.apply);
        } else {
            if (to == 0) launch<1, 1, kLast, 1>(c_.apply_one);
            else launch<1, 1, kApply, 1>(c_.apply_one);
        }
        ++args_.turn;
    }

    const NsCall& c_;
    hipStream_t s_;
    hipError_t err_ = hipSuccess;
    ProductArgs args_{};
};

template <int kT>
hipError_t launch_big(const NsCall& c, const NsMat* tab, hipStream_t s)
{
    return c.layout.x_terms == 1 ? BigLaunch<kT, 1>(c, tab, s).run() : BigLaunch<kT, 2>(c, tab, s).run();
}

}  // namespace

int ns_launch(const NsCall& c, NsMat* device_table, void* stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint32_t total = c.nbig;
    for (int k = 0; k < kNsClasses; ++k) total += c.nsmall[k];
    hipError_t err = hipSuccess;
    for (uint32_t k = 0; k < total && err == hipSuccess; k += kWriteMany) {
        if (total - k <= kWriteFew) err = write_table<kWriteFew>(device_table + k, c.table + k, total - k, s);
        else err = write_table<kWriteMany>(device_table + k, c.table + k, total - k < kWriteMany ? total - k : kWriteMany, s);
    }
    const NsMat* tab = device_table;
    for (int k = 0; k < kNsClasses && err == hipSuccess; ++k) {
        if (c.nsmall[k] == 0) continue;
        err = k == 0 ? launch_small<8>(c, tab, c.nsmall[k], c.small_chunks[k], c.small_index[k], s)
            : k == 1 ? launch_small<16>(c, tab, c.nsmall[k], c.small_chunks[k], c.small_index[k], s)
            : k == 2 ? launch_small<32>(c, tab, c.nsmall[k], c.small_chunks[k], c.small_index[k], s)
                     : launch_small<64>(c, tab, c.nsmall[k], c.small_chunks[k], c.small_index[k], s);
        tab += c.nsmall[k];
    }
    if (err == hipSuccess && c.nbig > 0) {
        err = c.tile == 256 ? launch_big<256>(c, tab, s) : c.tile == 128 ? launch_big<128>(c, tab, s) : launch_big<64>(c, tab, s);
    }
    return err;
}

}  // namespace lso
