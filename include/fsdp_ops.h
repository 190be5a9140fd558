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
 *   fsdp_embedding_forward / _backward    embedding lookup, its gradient by
 *                                         sorted tokens
 *   fsdp_gated_scan_forward / _backward   gated linear recurrence over
 *                                         sequences
 *   fsdp_distill_loss_forward / _backward distillation from a teacher's top
 *                                         logits
 *   fsdp_policy_loss_forward / _backward  clipped policy loss with a KL term
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

/*
 * ---------------------------------------------------------------------------
 * Embedding lookup and its gradient.
 *   out[i] = scale * weight[tokens[i]]
 *   dweight[v] = (dweight[v] +) scale * sum over i with tokens[i] = v of dout[i]
 * A token outside [0, vocab) (padding) gives a row of zeros and no gradient.
 * The gradient's rows are summed in binary32 in the order of i, in pieces whose
 * length depends on the sizes alone, and rounded once.
 */
#define FSDP_INDEX_I32 0
#define FSDP_INDEX_I64 1

typedef struct {
  int64_t rows;         /* tokens, 0 .. 2^31 - 1 */
  int64_t vocab;        /* rows of weight, 1 .. 2^31 - 2 */
  int64_t cols;         /* features, >= 1 */
  int64_t ld_weight;    /* row distance of weight (forward) or dweight (backward) */
  int64_t ld_out;       /* row distance of out (forward) or dout (backward) */
  int32_t token_dtype;  /* FSDP_INDEX_I32 or _I64 */
  int32_t weight_dtype; /* F32 or BF16, of weight or dweight */
  int32_t out_dtype;    /* F32 or BF16, of out or dout */
  int32_t accumulate;   /* backward: 0 writes all of dweight, rows without tokens as 0;
                           1 adds to it and leaves those rows as they were (a tied output
                           layer's gradient is there already) */
  float scale;          /* finite */
} fsdp_embedding_desc_t;

/* tokens: rows indices; weight [vocab, cols]; out [rows, cols]. */
fsdp_status_t fsdp_embedding_forward(const fsdp_embedding_desc_t *desc, const void *tokens, const void *weight, void *out,
                                     fsdp_stream_t stream);

/* dout [rows, cols]; dweight [vocab, cols]; workspace: fsdp_embedding_workspace bytes. */
fsdp_status_t fsdp_embedding_backward(const fsdp_embedding_desc_t *desc, const void *tokens, const void *dout,
                                      void *dweight, void *workspace, int64_t workspace_bytes, fsdp_stream_t stream);

/* Bytes of workspace of the backward call: the tokens' order and partial sums of
 * rows that many tokens share. */
fsdp_status_t fsdp_embedding_workspace(const fsdp_embedding_desc_t *desc, int64_t *bytes);

/*
 * ---------------------------------------------------------------------------
 * Gated linear recurrence along the rows of each sequence, every column on its own:
 *   a_t = 1 / (1 + e^-(gate_t + bias)),   h_t = a_t h_(t-1) + (1 - a_t) x_t
 * from the sequence's initial state, and for the backward pass, with
 * D_t = dh_t + a_(t+1) D_(t+1) (at a sequence's last row dh_t + dfinal):
 *   dx_t = (1 - a_t) D_t,   dgate_t = D_t (h_(t-1) - x_t) a_t (1 - a_t),
 *   dbias = sum of dgate over the rows of all sequences,   dinitial = a_1 D_1
 * States and sums are binary32, and a and 1 - a each good to a few ulp of their own sizes (below
 * 2^-125 they count as 0): slow columns and gates that are nearly shut keep their precision, and
 * a sequence has the same states however it is cut into calls, but for roundings.  Gates below
 * -69 cost a little: the rows around them are taken twice.  One row a sequence is a step of
 * generation: pass the states in `initial` and receive them in `final`, which may be the same
 * buffer; no other output may overlap an input.
 *
 * The rows of a batch are its sequences one after another: `seqs` of `seq_len` rows each,
 * or with `packed` sequence s from row offsets[s] up to offsets[s + 1], where offsets has
 * seqs + 1 device values that do not decrease and lie in [0, rows].  Rows outside every
 * sequence (behind the last, say) are neither read into a result nor written, and a
 * sequence without rows passes its state on (final = initial, dinitial = dfinal).
 * Offsets that break this give unspecified results within the arrays, no other access.
 */
typedef struct {
  int64_t rows, cols;          /* of x; rows >= 0, cols >= 1 */
  int64_t seqs;                /* sequences, >= 0 */
  int64_t seq_len;             /* rows of each, with packed = 0: rows = seqs * seq_len */
  int64_t ld_x, ld_gate;       /* row distances */
  int64_t ld_h;                /* of h (forward) or dh (backward) */
  int64_t ld_dx, ld_dgate;
  int32_t packed;              /* 1: offsets say where sequences are; seq_len is ignored */
  int32_t offset_dtype;        /* FSDP_INDEX_I32 or _I64 */
  int32_t x_dtype;             /* F32 or BF16, of x and gate */
  int32_t h_dtype;             /* F32 or BF16, of h or dh */
  int32_t dx_dtype;            /* F32 or BF16, of dx and dgate */
  int32_t param_dtype;         /* F32 or BF16, of bias */
  int32_t grad_dtype;          /* F32 or BF16, of dbias */
} fsdp_scan_desc_t;

/* Rows of the matrix [n, cols] of binary32 that a forward call fills for the backward call
 * (states some rows apart, from which the backward call makes h again): n depends on rows
 * and cols alone. */
fsdp_status_t fsdp_gated_scan_states(int64_t rows, int64_t cols, int64_t *n);

/* Bytes of workspace of the forward (backward = 0) or backward call. */
fsdp_status_t fsdp_gated_scan_workspace(const fsdp_scan_desc_t *desc, int32_t backward, int64_t *bytes);

/*
 *   x, gate, h [rows, cols];  bias: cols elements, or NULL for 0.
 *   initial: [seqs, cols] binary32 without gaps, or NULL for 0;  final: the same, written,
 *            or NULL.
 *   offsets: seqs + 1 device values with packed, else NULL.
 *   states:  what the backward call needs, or NULL (of rows outside every sequence unspecified).
 */
fsdp_status_t fsdp_gated_scan_forward(const fsdp_scan_desc_t *desc, const void *x, const void *gate, const void *bias,
                                      const float *initial, const void *offsets, void *h, float *final,
                                      float *states, void *workspace, int64_t workspace_bytes, fsdp_stream_t stream);

/*
 *   x, gate, bias, initial, offsets: as in the forward call;  states: what it wrote.
 *   dh [rows, cols];  dfinal: [seqs, cols] binary32, or NULL for 0.
 *   dx, dgate [rows, cols], both written;  dbias (cols elements) and dinitial ([seqs, cols]
 *   binary32): written, or NULL if not wanted.  dinitial may not be dfinal: a sequence's first
 *   rows may be done before its last ones.
 */
fsdp_status_t fsdp_gated_scan_backward(const fsdp_scan_desc_t *desc, const void *dh, const void *x, const void *gate,
                                       const void *bias, const float *initial, const void *offsets,
                                       const float *states, const float *dfinal, void *dx, void *dgate, void *dbias,
                                       float *dinitial, void *workspace, int64_t workspace_bytes, fsdp_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Losses over rows of logits z [rows, vocab].  With p = softmax(z / T) of a row and
 * lse = log sum e^(z / T):
 *
 * Distillation from a teacher's top logits: entries j of a row name tokens and the
 * teacher's logits for them; q is the softmax of those logits / T over the row's entries.
 *   loss = weight T^2 sum_j q_j (log q_j - log p_(token j))
 *   dlogits_i = dloss weight T (p_i - sum of q_j over entries with token j = i)
 * Entries with a token outside [0, vocab), or a logit of -infinity, do not count; a row
 * without entries has loss and gradient 0.  A token may be named more than once.
 *
 * Clipped policy loss: token a was taken with log-probability old_logp and advantage A.
 * With logp = z_a / T - lse, r = e^(logp - old_logp), and k = ref_logp - logp:
 *   loss = weight (-min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl (e^k - k - 1))
 *   dlogits_i = dloss weight c / T ([i = a] - p_i),
 *   c = (r A <= clip(r) A ? -r A : 0) + kl (1 - e^k)
 * old_logp NULL: r is 1 (and its derivative r).  ref_logp NULL: no KL term.  A row whose token
 * is outside [0, vocab) has loss, logp and gradient 0 (and its lse).
 *
 * A row of weight 0 is not read: its loss, logp, lse and gradient are written as 0, whatever
 * its logits hold.  Sums are binary32.  Logits of -infinity have probability 0 (a row of nothing
 * else has no distribution: NaN); those of any finite value are values like others, masks of -1e10
 * or of the type's lowest value too.
 *
 * With dlogits given, the forward call also writes the gradient of the sum of the rows'
 * losses (dloss = 1), for which a row stays on the chip; the backward call computes it from
 * the lse (and logp) of a forward call, whose rounding it carries: 2^-24 |lse| in each
 * probability, relative, so that of a row masked with -1e10 throughout nothing is left (the
 * forward call's gradient is right there, too).  dlogits may be logits itself, with the same row
 * distance and dtype; no other overlap is allowed.
 */
#define FSDP_DISTILL_MAX_TOP 1024

typedef struct {
  int64_t rows, vocab;         /* rows >= 0, vocab 1 .. 2^31 - 64 */
  int64_t ld_logits, ld_dlogits;
  int64_t top;                 /* entries of a row, 0 .. FSDP_DISTILL_MAX_TOP */
  int64_t ld_tokens, ld_teacher;
  int32_t logits_dtype, dlogits_dtype, teacher_dtype; /* F32 or BF16 */
  int32_t token_dtype;         /* FSDP_INDEX_I32 or _I64 */
  float temperature;           /* T, finite and > 0 */
} fsdp_distill_desc_t;

/*
 *   logits [rows, vocab];  teacher_tokens, teacher_logits [rows, top];  weight: rows binary32
 *   values, or NULL for 1.
 *   loss, lse: rows binary32 values, written;  dlogits [rows, vocab], or NULL.
 */
fsdp_status_t fsdp_distill_loss_forward(const fsdp_distill_desc_t *desc, const void *logits, const void *teacher_tokens,
                                        const void *teacher_logits, const float *weight, float *loss, float *lse,
                                        void *dlogits, fsdp_stream_t stream);

/* dloss: rows binary32 values, or NULL for 1. */
fsdp_status_t fsdp_distill_loss_backward(const fsdp_distill_desc_t *desc, const void *logits, const void *teacher_tokens,
                                         const void *teacher_logits, const float *weight, const float *lse,
                                         const float *dloss, void *dlogits, fsdp_stream_t stream);

typedef struct {
  int64_t rows, vocab;         /* rows >= 0, vocab 1 .. 2^31 - 64 */
  int64_t ld_logits, ld_dlogits;
  int32_t logits_dtype, dlogits_dtype; /* F32 or BF16 */
  int32_t token_dtype;         /* FSDP_INDEX_I32 or _I64 */
  float temperature;           /* T, finite and > 0 */
  float clip_low, clip_high;   /* >= 0; infinity: no bound */
  float kl;                    /* weight of the KL term, finite, >= 0 */
} fsdp_policy_desc_t;

/*
 *   tokens: rows indices;  old_logp, ref_logp, advantage, weight: rows binary32 values each
 *   (old_logp, ref_logp and weight may be NULL).
 *   loss, logp, lse: rows binary32 values, written;  dlogits [rows, vocab], or NULL.
 */
fsdp_status_t fsdp_policy_loss_forward(const fsdp_policy_desc_t *desc, const void *logits, const void *tokens,
                                       const float *old_logp, const float *ref_logp, const float *advantage,
                                       const float *weight, float *loss, float *logp, float *lse, void *dlogits,
                                       fsdp_stream_t stream);

/* logp, lse: what the forward call wrote;  dloss: rows binary32 values, or NULL for 1. */
fsdp_status_t fsdp_policy_loss_backward(const fsdp_policy_desc_t *desc, const void *logits, const void *tokens,
                                        const float *old_logp, const float *ref_logp, const float *advantage,
                                        const float *weight, const float *logp, const float *lse, const float *dloss,
                                        void *dlogits, fsdp_stream_t stream);

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
