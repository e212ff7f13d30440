// Internal types of the Newton-Schulz path, shared by its host side
// (lso_matrix.cpp) and its kernels (lso_ns.hip).
#pragma once

#include <cstdint>

namespace lso {

// Operands are FP16 numbers of the values times kNsScale (a power of two, so
// scaling is exact): a matrix of Frobenius norm 1 and some million elements
// has elements of about 2^-12, which the scale brings to the middle of
// FP16's range, and no element of an iterate (at most kNsMostValue) passes
// its end.
constexpr float kNsScale = 4096.0f;
constexpr double kNsMostValue = 15.9;

// Edge of the square tiles of the elementwise passes.
constexpr uint32_t kNsPrep = 64;
// Elements along the long side per workgroup of the small path.
constexpr uint32_t kNsSmallChunk = 256;
// The small path's kernels are built for smaller sides up to 8, 16, 32 and 64.
constexpr int kNsClasses = 4;
constexpr uint32_t kNsMaxSteps = 16;

enum : uint32_t {
    kNsSrcF32 = 1u,     // x or gradient is FP32 (else BF16)
    kNsDstF32 = 2u,     // y is FP32 (else BF16)
    kNsTall = 4u,       // rows > cols: the transpose is iterated on
    kNsMuon = 8u,       // update: src is the gradient, dst the weight (or null)
    kNsNesterov = 16u,
    kNsQuads = 32u,     // groups of four columns are whole, and aligned in every array
};

// One matrix of a call (an entry of the table in the workspace).
struct NsMat {
    const void* src;    // x, or the gradient
    void* dst;          // y, or the BF16 weight or null
    float* m;           // update only
    float* master;      // update only
    char* work;         // its part of the workspace
    uint32_t rows, cols;
    uint32_t ld_src, ld_dst;
    uint32_t flags;
    float beta, c1;     // beta, 1 - beta
    float keep, step;   // 1 - lr weight_decay, -lr scale
    uint32_t mp, np;    // padded smaller and larger side (general path)
    // first index of this matrix in the index space of each launch
    uint32_t prep0;     // kNsPrep tiles of the padded matrix; small path: chunks
    uint32_t gram0;     // units (tile, part of the summed index) of S, a multiple of 8 per matrix
    uint32_t square0;   // of a product of two squares
    uint32_t apply0;    // of X
    uint32_t apply_one0;   // of X where X^T has one term
};
static_assert(sizeof(NsMat) == 104, "NsMat layout");

// What a call's workspace holds per value: X (the smaller side by the larger,
// read by S = X X^T) in x_terms FP16 numbers, its transpose (read and written
// in turn by the product with the polynomial) in up to two, and `squares`
// matrices of the smaller side in square_terms.
struct NsLayout {
    uint32_t x_terms, square_terms, squares;
};

// Offsets of a general-path matrix inside its part of the workspace.
struct NsWork {
    uint64_t x, xt[2], square, square_bytes, partial, inv, bytes;
};
#if defined(__HIPCC__)
__host__ __device__
#endif
inline NsWork ns_work(uint64_t mp, uint64_t np, const NsLayout& l)
{
    const uint64_t xs = mp * np * 2;   // all of these are multiples of 256
    NsWork w{};
    w.x = 0;
    w.xt[0] = xs * l.x_terms;
    w.xt[1] = w.xt[0] + 2 * xs;
    w.square = w.xt[1] + 2 * xs;
    w.square_bytes = mp * mp * 2 * l.square_terms;
    w.inv = w.square + w.square_bytes * l.squares;
    w.partial = w.inv + 256;
    w.bytes = w.partial + (mp / kNsPrep * (np / kNsPrep) * 8 + 255) / 256 * 256;
    return w;
}

// Of a small-path matrix: the FP64 partial products of each chunk, and the
// k x k matrix that x is multiplied by, in rows of its class's size.
inline uint64_t ns_small_bytes(uint64_t k, uint64_t l)
{
    const uint64_t chunks = (l + kNsSmallChunk - 1) / kNsSmallChunk, side = k <= 8 ? 8 : k <= 16 ? 16 : k <= 32 ? 32 : 64;
    return (chunks * k * k * 8 + side * side * 8 + 255) / 256 * 256;
}

// Where a launch's workgroups belong: matrices first_mat[r] and on have `each`
// indices apiece from first[r] on, until the next run starts.  runs == 0: too
// many runs, the table is searched.
constexpr int kNsRuns = 8;
struct NsIndex {
    uint32_t runs;
    uint32_t first[kNsRuns], first_mat[kNsRuns], each[kNsRuns];
};

// Blocks of each operand per stage of a product with tiles of this edge.
constexpr int ns_blocks(uint32_t edge, bool symmetric, int terms) { return edge == 64 && symmetric && terms == 2 ? 2 : 1; }

// A product's launch: workgroups, and stages of the summed index per part.
struct NsProduct {
    uint32_t units, depth;
    NsIndex index;
};

// One call, as the launches need it.  The table holds the small-path
// matrices by class, then the others.
struct NsCall {
    const NsMat* table;                    // host copy
    uint32_t nsmall[kNsClasses], nbig;
    uint32_t small_chunks[kNsClasses];     // index spaces
    NsIndex small_index[kNsClasses];
    uint32_t prep_tiles;
    NsIndex prep_index;
    NsProduct gram, square, apply, apply_one;
    uint32_t tile;                         // edge of a product tile: 64, 128 or 256
    float* parts;                          // workspace of the parts' sums
    uint32_t* counters;
    uint32_t ncounters;
    NsLayout layout;
    bool pairs;                            // take steps two at a time where pair[] allows
    bool pair[kNsMaxSteps];                // step k and the next one may be taken together
    uint32_t steps;
    double eps;
    double coef[3 * kNsMaxSteps];
    int16_t shift[kNsMaxSteps];            // a step multiplies X by less than 2^shift (-255 at least)
};

// Enqueue the table's upload to device_table and every launch (lso_ns.hip).
// Returns the hipError_t.
int ns_launch(const NsCall& c, NsMat* device_table, void* stream);

}  // namespace lso
