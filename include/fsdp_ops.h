/*
 * fsdp_ops.h - C ABI of the training operators that stand next to the
 * packing library (fsdp_pack.h): the feed-forward half of a transformer
 * block, whose gradients are what a fully_shard group packs.
 *
 *   fsdp_layer_norm_forward / _backward   layer norm with its parameter
 *                                         gradients
 *   fsdp_act8_store / _load               activation checkpoints in 8 bits
 *   fsdp_gated_ffn_forward / _backward    both projections, the activation
 *                                         and the product of a gated
 *                                         feed-forward block
 *
 * The backward calls read the 8-bit checkpoints in place of the tensors they
 * were taken from, and write gradients in the dtypes that
 * fsdp_pack_reduce_scatter reads (BF16 or FP32).
 *
 * Conventions, on top of those of fsdp_pack.h (device pointers, asynchronous
 * on the stream, arguments checked on the host before anything is launched,
 * one-line errors through fsdp_last_error()):
 *   - Matrices are row-major with unit column stride; `ld` is the distance
 *     between rows in elements and at least the number of columns.
 *   - Every pointer need only be aligned to its element size, except
 *     checkpoints and workspaces (16 bytes).  Rows whose start is 16-byte
 *     aligned take faster paths.
 *   - Of inputs, the whole 16-byte units that a row, or a checkpoint's scale
 *     bytes, lie in may be read: up to 15 bytes beside them, whose values are
 *     ignored.  They never leave an allocation's 16-byte unit.  Nothing is written
 *     outside a matrix.
 *   - Indexing is 64-bit throughout.
 *   - No call allocates device memory: calls that need scratch take a
 *     workspace, whose size the matching _workspace call gives.  A workspace
 *     holds nothing between calls, and one workspace serves one call at a
 *     time.
 *   - Results are the same, bit for bit, on every run: sums run in a fixed
 *     order and no result goes through an atomic.
 *   - rows may be 0: outputs of that many rows are empty, and gradients of
 *     parameters (sums over no rows) are written as 0.
 *   - NaN and infinities propagate as the formulas say.
 *   - Every wait inside the kernels is bounded; fsdp_ops_sync_status tells
 *     whether one gave up.  fsdp_debug_set_wait_fault (the limit and the test
 *     hook) holds for these kernels' pipelines too; fault = 1 + 256 * g starves
 *     the g-th group of rows of a layer norm's first block.
 */
#ifndef FSDP_OPS_H
#define FSDP_OPS_H

#include "fsdp_pack.h"

#ifdef __cplusplus
extern "C" {
#endif

/* In the activation dtype fields below, beside FSDP_DTYPE_F32 and
 * FSDP_DTYPE_BF16: the activation is given by its 8-bit checkpoint. */
#define FSDP_ACT8 2

/* Elements of a row that share one scale of an 8-bit checkpoint. */
#define FSDP_ACT8_GROUP 32

/*
 * Activation checkpoints in 8 bits.
 *
 * A checkpoint of a [rows, cols] matrix x is one buffer, 16-byte aligned:
 * int8 codes [rows, 32 G], then one scale byte per group [rows, G], with
 * G = ceil(cols / 32).  A group is 32 consecutive elements of a row (the last
 * one of a row may be shorter; its missing elements count and are stored as
 * 0).  With a = max |x| over the group and e the least integer >= -126 with
 * a <= 127 * 2^e:
 *   scale byte = e + 127,   code = x * 2^-e rounded to the nearest integer,
 *                                  ties to even (for e = 122 held to
 *                                  [-63, 63]: 64 * 2^122 is infinite)
 *   value read back = code * 2^(scale byte - 127)
 * A group that holds a NaN or an infinity has scale byte 255 and codes 0, and
 * reads back as NaN throughout, so that a check for overflowed gradients
 * still sees it.  Codes have 7 bits and the scale is a power of two, so every
 * value that reads back is exact in BF16 (and so on the tensor cores), and
 * storing what was read back gives the same checkpoint again.  The error of an
 * element is at most 2^(e-1), below a / 127 (2^e for e = 122).
 */

/* Bytes of the checkpoint of a [rows, cols] matrix: rows * 33 * G.
 * FSDP_EINVAL for NULL bytes, rows < 0 or cols < 1. */
fsdp_status_t fsdp_act8_bytes(int64_t rows, int64_t cols, int64_t *bytes);

/* x [rows, cols] (dtype FSDP_DTYPE_F32 or _BF16) -> ckpt. */
fsdp_status_t fsdp_act8_store(const void *x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, void *ckpt,
                              fsdp_stream_t stream);

/* ckpt -> y [rows, cols] (dtype FSDP_DTYPE_F32 or _BF16: exact in both). */
fsdp_status_t fsdp_act8_load(const void *ckpt, int64_t rows, int64_t cols, void *y, int32_t dtype, int64_t ld,
                             fsdp_stream_t stream);

/*
 * Layer norm over the rows of a [rows, cols] matrix.  For each row:
 *   mean = sum x / cols,  rstd = (sum (x - mean)^2 / cols + eps)^(-1/2),
 *   xh = (x - mean) * rstd,  y = xh * weight + bias
 * and for the backward pass, with g = dy * weight:
 *   dx = rstd * (g - mean(g) - xh * mean(g * xh)),
 *   dweight = sum over rows of dy * xh,  dbias = sum over rows of dy.
 * All arithmetic and sums are in binary32.
 */
typedef struct {
  int64_t rows;         /* >= 0 */
  int64_t cols;         /* 1 .. FSDP_NORM_MAX_COLS */
  int64_t ld_x;         /* row distance of x (ignored for a checkpoint) */
  int64_t ld_y;         /* row distance of y (forward) or dy (backward) */
  int64_t ld_dx;        /* row distance of dx (backward) */
  int32_t x_dtype;      /* FSDP_DTYPE_F32, FSDP_DTYPE_BF16 or FSDP_ACT8 */
  int32_t y_dtype;      /* dtype of y and dy: F32 or BF16 */
  int32_t dx_dtype;     /* dtype of dx: F32 or BF16 */
  int32_t param_dtype;  /* dtype of weight and bias: F32 or BF16 */
  int32_t grad_dtype;   /* dtype of dweight and dbias: F32 or BF16 */
  float eps;            /* >= 0 */
} fsdp_norm_desc_t;

#define FSDP_NORM_MAX_COLS 65536

/*
 *   x:          [rows, cols], or its checkpoint (x_dtype FSDP_ACT8).
 *   weight:     cols elements of param_dtype, or NULL for all ones.
 *   bias:       cols elements of param_dtype, or NULL for none.
 *   mean, rstd: rows binary32 values each, written for the backward pass; both
 *               may be NULL.
 *   keep:       NULL, or receives the 8-bit checkpoint of x in the same pass
 *               (x_dtype F32 or BF16 only).
 */
fsdp_status_t fsdp_layer_norm_forward(const fsdp_norm_desc_t *desc, const void *x, const void *weight,
                                      const void *bias, void *y, float *mean, float *rstd, void *keep,
                                      fsdp_stream_t stream);

/*
 *   x, weight:      as in the forward pass (x may be the checkpoint that the
 *                   forward pass kept); mean and rstd: what it wrote.
 *   dx:             [rows, cols] of dx_dtype, or NULL if not wanted.
 *   dweight, dbias: cols elements of grad_dtype each, written (not added to);
 *                   either may be NULL if not wanted.
 *   workspace:      fsdp_layer_norm_workspace bytes, 16-byte aligned; may be NULL
 *                   if that is 0.
 */
fsdp_status_t fsdp_layer_norm_backward(const fsdp_norm_desc_t *desc, const void *dy, const void *x,
                                       const void *weight, const float *mean, const float *rstd, void *dx,
                                       void *dweight, void *dbias, void *workspace, int64_t workspace_bytes,
                                       fsdp_stream_t stream);

/* Bytes of workspace that fsdp_layer_norm_backward needs on the current
 * device (a limit for any device when there is none). */
fsdp_status_t fsdp_layer_norm_workspace(const fsdp_norm_desc_t *desc, int64_t *bytes);

/*
 * Gated feed-forward block over rows of d features with f hidden features: both
 * projections, the activation and the product in one kernel.
 *   g = x w_gate^T,  u = x w_up^T,  h = act(g) * u        (forward)
 *   dg = dh * u * act'(g),  du = dh * act(g)
 *   dx = dg w_gate + du w_up,  dw_gate = dg^T x,  dw_up = du^T x   (backward)
 * with act(g) = g / (1 + e^-g) (FSDP_ACT_SILU) or g * Phi(g), Phi the normal
 * distribution (FSDP_ACT_GELU, the exact form).  Matrices are BF16 unless a
 * dtype field says otherwise; products run on the tensor cores with binary32
 * sums, whose additions may cut where binary32 units round, and activations,
 * their derivatives and products in binary32.  dg and du are rounded to BF16
 * once, as operands of the backward products; g and u are not rounded unless
 * they are kept.
 *
 * Kept for the backward pass (`keep`): nothing (the backward call computes g
 * and u again), the 8-bit checkpoints of g and u (33/32 byte an element), or
 * both in BF16.
 */
typedef enum { FSDP_ACT_SILU = 0, FSDP_ACT_GELU = 1 } fsdp_activation_t;
typedef enum { FSDP_KEEP_NONE = 0, FSDP_KEEP_ACT8 = 1, FSDP_KEEP_BF16 = 2 } fsdp_keep_t;

typedef struct {
  int64_t rows;        /* tokens, >= 0 */
  int64_t d, f;        /* features in and hidden, >= 1 */
  int64_t ld_x;        /* row distances; of matrices that a call is not given, ignored */
  int64_t ld_w_gate, ld_w_up;
  int64_t ld_h;        /* of h (forward) or dh (backward) */
  int64_t ld_kept;     /* of gate and up kept in BF16 */
  int64_t ld_dx, ld_dw_gate, ld_dw_up;
  int32_t activation;  /* fsdp_activation_t */
  int32_t keep;        /* fsdp_keep_t */
  int32_t x_dtype;     /* FSDP_DTYPE_BF16, or in the backward pass FSDP_ACT8 */
  int32_t dx_dtype;    /* F32 or BF16 */
  int32_t dw_dtype;    /* F32 or BF16 */
  int32_t unaligned;   /* which operands start off a 16-byte boundary: 1 x, 2 w_gate, 4 w_up */
} fsdp_ffn_desc_t;

/* Bytes of workspace of the forward (backward = 0) or backward call.  Operands
 * whose rows do not all start on 16-byte boundaries (by their row distance or
 * by `unaligned`) are copied there once per call, which costs their bytes.  The
 * backward call holds dg and du there in BF16, 4 bytes for each element of h,
 * and of an x given by its checkpoint a BF16 copy: it saves memory between the
 * passes, not during this one. */
fsdp_status_t fsdp_gated_ffn_workspace(const fsdp_ffn_desc_t *desc, int32_t backward, int64_t *bytes);

/*
 *   x [rows, d], w_gate and w_up [f, d], h [rows, f].
 *   gate, up: by `keep`, NULL; [rows, f] checkpoints of fsdp_act8_bytes(rows, f)
 *             bytes; or [rows, f] BF16 matrices.
 *   workspace: may be NULL if fsdp_gated_ffn_workspace gives 0.
 */
fsdp_status_t fsdp_gated_ffn_forward(const fsdp_ffn_desc_t *desc, const void *x, const void *w_gate,
                                     const void *w_up, void *h, void *gate, void *up, void *workspace,
                                     int64_t workspace_bytes, fsdp_stream_t stream);

/*
 *   dh [rows, f]; x as in the forward pass or its checkpoint; gate and up as kept
 *   (NULL for FSDP_KEEP_NONE).
 *   dx [rows, d], dw_gate and dw_up [f, d]: written (not added to); dx may be
 *   NULL, and dw_gate and dw_up together, where they are not wanted.
 */
fsdp_status_t fsdp_gated_ffn_backward(const fsdp_ffn_desc_t *desc, const void *dh, const void *x,
                                      const void *w_gate, const void *w_up, const void *gate, const void *up,
                                      void *dx, void *dw_gate, void *dw_up, void *workspace,
                                      int64_t workspace_bytes, fsdp_stream_t stream);

/* Synchronise `stream`, then say whether a wait of this header's kernels gave
 * up.  Failures are counted per device, for all streams and threads of the
 * process together, and the counts are never reset: FSDP_ETIMEOUT if one has
 * grown since this host thread last asked on this device (for a thread that
 * never asked: since the process began).  So every thread that asks is told of
 * every failure once, whoever else was told; a thread may be told of one on
 * another's stream. */
fsdp_status_t fsdp_ops_sync_status(fsdp_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FSDP_OPS_H */
