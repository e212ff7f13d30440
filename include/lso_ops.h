/*
 * lso_ops.h -- operators around the update: orthogonalisation of matrices,
 * the orthogonalised-momentum update, and the embedding table's lookup and
 * gradient.  Same library (liblso.so) and the same conventions as lso.h:
 * a lso_status is returned, nothing throws, errors found before anything is
 * enqueued leave memory untouched, streams are hipStream_t passed as void*.
 *
 * None of these calls allocates device memory, synchronises or reads host
 * memory after it returns, so all of them may be captured into a HIP graph.
 * They run on the current device, which must be the stream's and the arrays'.
 * A workspace is device memory of the caller, 16-byte aligned, whose content
 * need not survive between calls: calls that run at the same time (other
 * streams, two graphs) need separate ones.  Every sum is taken in an order
 * that the shapes (and for the embedding gradient the tokens) fix, so equal
 * inputs give equal bits.
 */
#ifndef LSO_OPS_H
#define LSO_OPS_H

#include "lso.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------
 * Orthogonalisation by Newton-Schulz products.
 *
 *   X_0     = x / (|x|_F + eps)
 *   X_{k+1} = a X_k + (b S + c S^2) X_k,   S = X_k X_k^T   (k = 0 .. steps-1)
 *   y       = X_steps
 *
 * With rows > cols the same is done to the transpose, so S has the smaller
 * side.  Each singular value s of X goes through s -> a s + b s^3 + c s^5
 * and the singular vectors stay; the default coefficients (3.4445, -4.7750,
 * 2.0315) bring every s that is not tiny to about 1 in five steps.
 *
 * Arithmetic (precision):
 *   LSO_NS_FULL  operands of every product are held as a sum of two FP16
 *                numbers (22 significant bits), products are summed in FP32:
 *                results as accurate as FP32 products;
 *   LSO_NS_HALF  what X is multiplied by is rounded to FP16 (11 bits), X
 *                itself keeps 22 but for its last steps: errors of about
 *                1e-3 of |y|_F, below the rounding of a BF16 result, at less
 *                than half the time;
 *   LSO_NS_AUTO  FULL whatever the types: rounding to 11 bits is the caller's
 *                choice (22 of 256 x 2048 into BF16: 1.86e-3 off 64 bits against
 *                1.66e-3, which is the rounding of the result alone).
 * Two steps are taken as one product with X where that saves operations
 * (S of the next step follows from the polynomial and S).
 * Matrices whose smaller side is at most LSO_NS_SMALL_SIDE take another way
 * whatever the precision: S is iterated on in FP64 and x multiplied once.
 * (Those above 32 do not where a few of them come with larger matrices.)
 * A matrix with a NaN or an infinity gives NaNs (in that matrix only); a
 * zero matrix gives zeros.
 * ------------------------------------------------------------------- */
#define LSO_NS_AUTO 0u
#define LSO_NS_FULL 1u
#define LSO_NS_HALF 2u
#define LSO_NS_SMALL_SIDE 64u
#define LSO_NS_MAX_STEPS 16u

/* The iteration.  NULL in a call means the defaults.  steps: 1 to
 * LSO_NS_MAX_STEPS.  eps: finite, >= 0 (with 0 a zero matrix gives NaN).
 * coef: steps triples a, b, c, one for each step, or NULL for the default
 * ones in every step.  Coefficients under which a singular value, its
 * square or the polynomial a + b s^2 + c s^4 could pass 15.9 (starting
 * from s <= 1) are refused: the operands are held in FP16 scaled by 2^12. */
typedef struct lso_ns_params {
    uint32_t      steps;       /* default 5 */
    uint32_t      precision;   /* LSO_NS_*, default AUTO */
    double        eps;         /* default 1e-7 */
    const double* coef;        /* host memory, read before return */
} lso_ns_params;

/* One matrix, row-major.  ld_x, ld_y: elements from one row to the next
 * (>= cols).  x_dtype, y_dtype: LSO_DT_F32 or LSO_DT_BF16.  x and y need
 * their element's alignment; y may be x (same dtype and stride), any other
 * overlap of a y with an array of the call is refused (arrays taken as the
 * span from the first to the last element).  rows == 0 or cols == 0 is a
 * no-op.  rows, cols, ld below 2^31. */
typedef struct lso_matrix {
    const void* x;
    void*       y;
    uint64_t    rows, cols;
    uint64_t    ld_x, ld_y;
    uint32_t    x_dtype, y_dtype;
} lso_matrix;

/* lso_orthogonalize: every matrix of the call, in a fixed number of launches
 * (the matrices advance together).  Workspace: at least
 * lso_orthogonalize_workspace_bytes (0 if the arguments are not valid), which
 * depends on the sizes and the precision.
 * Errors: INVALID, ALIGN, DTYPE, OVERLAP (nothing enqueued), HIP. */
uint64_t   lso_orthogonalize_workspace_bytes(const lso_matrix* mats, size_t n, const lso_ns_params* params);
lso_status lso_orthogonalize(const lso_matrix* mats, size_t n, const lso_ns_params* params, void* workspace,
                             uint64_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------
 * The orthogonalised-momentum update of weight matrices.
 *
 *   m'      = beta m + (1 - beta) g
 *   u       = beta m' + (1 - beta) g   (LSO_MUON_NESTEROV), else m'
 *   O       = orthogonalize(u)
 *   master' = (1 - lr weight_decay) master - lr scale O    (the additive write-back)
 *   weight  = BF16 round-to-nearest-even of master'
 *
 * master and m are FP32, g BF16 or FP32 (grad_dtype), all rows x cols,
 * contiguous; the BF16 weight is written unless weight_dtype is
 * LSO_DT_NONE.  Addresses are base + off_*, as in lso_block; arrays need
 * only their element's alignment here (a matrix may start anywhere inside a
 * block).  Hyper-parameters are per matrix: lr, weight_decay and scale finite,
 * 0 <= beta < 1.  scale carries the shape factor that a run uses (for
 * instance sqrt(max(1, rows / cols)), or 0.2 sqrt(max(rows, cols)), which
 * gives updates the root mean square of Adam's).  The constants are
 * computed in FP64 and rounded once; the element arithmetic is FP32.  No
 * written array may overlap any other array of the call.  rows == 0 or
 * cols == 0 is a no-op.
 * Errors: as lso_orthogonalize.
 * ------------------------------------------------------------------- */
#define LSO_MUON_NESTEROV 1u

typedef struct lso_muon_block {
    void*    base;
    uint64_t rows, cols;
    uint64_t off_master;
    uint64_t off_m;
    uint64_t off_grad;
    uint64_t off_weight;
    uint32_t grad_dtype;     /* LSO_DT_BF16 or LSO_DT_F32 */
    uint32_t weight_dtype;   /* LSO_DT_BF16 or LSO_DT_NONE */
    uint32_t flags;          /* LSO_MUON_* */
    uint32_t reserved;       /* must be 0 */
    double   lr, beta, weight_decay, scale;
} lso_muon_block;

uint64_t   lso_muon_workspace_bytes(const lso_muon_block* blocks, size_t n, const lso_ns_params* params);
lso_status lso_muon_step(const lso_muon_block* blocks, size_t n, const lso_ns_params* params, void* workspace,
                         uint64_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------
 * The embedding table.
 *
 *   lookup:    rows[i]  = scale * table[tokens[i]]
 *   gradient:  table[v] = scale * sum over i with tokens[i] == v of rows[i]
 *              (LSO_EMBED_ADD: += that)
 *
 * table: vocab x width, row v at v * ld_table; rows: n x width, row i at
 * i * ld_rows (strides in elements, >= width).  In the lookup the table is
 * a block's BF16 weight (or an FP32 master) and is read; in the gradient it
 * is the block's gradient array, written whole: rows of tokens that do not
 * occur become zero, unless LSO_EMBED_ADD adds to what is there, which
 * leaves such rows untouched.  Elements between width and the stride are not
 * touched.  A token below 0 or >= vocab is padding: its looked-up row is
 * zero, its gradient row is not read.
 * Sums are in FP32 over the positions i in an order the tokens fix, scaled
 * and rounded once to the table's type.  dtypes: LSO_DT_F32 or LSO_DT_BF16
 * each; tokens LSO_DT_I32 or LSO_DT_I64, contiguous.  Arrays need their
 * element's alignment (16-byte aligned rows are the fast case).  scale is
 * finite and used in FP32.  n, vocab < 2^31 - 1; width, ld < 2^31; width == 0 or vocab == 0 is a
 * no-op; n == 0 writes nothing in the lookup, and a gradient of zeros.
 * The array written may not overlap the others (or the workspace).
 * ------------------------------------------------------------------- */
#define LSO_DT_I32 3u
#define LSO_DT_I64 4u
#define LSO_EMBED_ADD 1u

typedef struct lso_embed {
    const void* tokens;
    uint64_t    n;
    void*       table;
    uint64_t    vocab, width, ld_table;
    void*       rows;
    uint64_t    ld_rows;
    uint32_t    token_dtype, table_dtype, rows_dtype;
    uint32_t    flags;         /* LSO_EMBED_* (gradient only) */
    double      scale;
} lso_embed;

/* Errors: INVALID, ALIGN, DTYPE, OVERLAP (nothing enqueued), HIP. */
lso_status lso_embed_lookup(const lso_embed* e, void* stream);

/* Workspace: lso_embed_grad_workspace_bytes(n, vocab, width) bytes or more. */
uint64_t   lso_embed_grad_workspace_bytes(uint64_t n, uint64_t vocab, uint64_t width);
lso_status lso_embed_grad(const lso_embed* e, void* workspace, uint64_t workspace_bytes, void* stream);

/* A gradient producer of the layer stream (lso_grad_fn) whose layer
 * `embed_layer` is an embedding table of vocab * width parameters: for that
 * layer it enqueues lso_embed_grad into the slot's gradient buffer (table
 * and ld_table of `grad` are replaced, table_dtype must be the layer's
 * grad_dtype, LSO_EMBED_ADD is refused), for every other layer it calls
 * `other` with `other_user`.  Pass lso_embed_producer as the function and a
 * lso_embed_producer_args as its user pointer.  A layer stream's own streams
 * wait for no other stream: tokens and rows must be complete on the device
 * when lso_stream_layers or lso_stream_files is called. */
typedef struct lso_embed_producer_args {
    lso_embed   grad;
    size_t      embed_layer;
    void*       workspace;
    uint64_t    workspace_bytes;
    lso_grad_fn other;
    void*       other_user;
} lso_embed_producer_args;

int lso_embed_producer(void* user, size_t layer, void* dev_grad, uint64_t n, void* compute_stream);

#ifdef __cplusplus
}
#endif
#endif /* LSO_OPS_H */
