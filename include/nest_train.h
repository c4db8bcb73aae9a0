/*
 * nest_train.h - C ABI of the training-step operators beside the placement solver.
 *
 * Two numbers of the solver's instances (nest.h) come from the training step and not
 * from the shapes of a model: the all-to-all bytes of a mixture-of-experts layer, which
 * grow with the load of its fullest expert, and the optimizer-state bytes per weight
 * byte.  These entry points run the parts of the step that decide them:
 *   nest_route, nest_route_backward    gates, chosen experts, per-expert counts and the
 *                                      balance loss of a router, and its gradient;
 *   nest_grad_norm                     global norm of many gradient tensors, clip scale;
 *   nest_adamw, nest_adamw_values      one AdamW step over many tensors, with moments
 *                                      in 32 or in 8 bits, and the moments' values.
 *
 * As in nest.h the caller allocates every buffer, the library allocates nothing, and
 * each call only checks its arguments and enqueues kernels on the caller's stream, so
 * it can be captured in a CUDA graph.  It returns NEST_OK once the work is enqueued,
 * NEST_E_INVALID or NEST_E_LIMITS (nothing enqueued) on bad arguments,
 * NEST_E_WORKSPACE on a workspace that is too small or not 256-byte aligned, and
 * NEST_E_CUDA when a launch fails.  Results do not depend on timing: the same inputs
 * give the same bits.
 */
#ifndef NEST_TRAIN_H
#define NEST_TRAIN_H

#include "nest.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define NEST_F32  0
#define NEST_BF16 1
#define NEST_F16  2

/* ---- routing ------------------------------------------------------------------
 * Logits x[t][e] at logits + (t * row_stride + e * col_stride) elements.
 * A row t counts ("is live") when mask is NULL or mask[t] != 0 and some x[t][e] is not
 * minus infinity.  For live rows
 *   p[t][e] = exp(x[t][e]) / sum over e' of exp(x[t][e'])
 *   ids[t][0 .. k-1]: the experts of the k largest logits, largest first, the lower
 *     index where two are equal (-0 equals +0).  Logits of minus infinity (closed
 *     experts) and NaN are not chosen; slots left over hold id -1 and weight 0.
 *   weights[t][j] = p[t][ids[t][j]], divided by their sum over j when normalize is set
 * and with n the number of live rows and c[e] how often e was chosen
 *   mean_prob[e] = (1/n) sum over live t of p[t][e]
 *   loss = E / (k n) * sum over e of c[e] mean_prob[e]
 * which is 1 for a perfectly even router.  Rows that are not live hold id -1 and weight
 * 0 and whatever their logits are (NaN included) reaches no result; with n = 0
 * mean_prob and loss are 0.  NaN or plus infinity in a live row gives NaN gates in that
 * row, NaN means and a NaN loss; ids and counts stay valid.                        */
typedef struct {
    int64_t tokens;      /* T >= 0, with T * k < 2^31 */
    int32_t experts;     /* 1 <= E <= 1024 */
    int32_t k;           /* 1 <= k <= min(E, 32) */
    int64_t row_stride;  /* elements, >= 0 */
    int64_t col_stride;  /* elements, >= 0 */
    int32_t dtype;       /* NEST_F32, NEST_BF16 or NEST_F16 */
    int32_t normalize;   /* 0 or 1 */
} nest_route_desc;

/* Device workspace of nest_route in bytes, 0 when the description breaks a limit.  Its first
 * NEST_TRAIN_TICKET bytes are zero on entry - the caller clears them once - and zero again
 * when the call's work is done; the rest is scratch.  Calls that overlap need workspaces of
 * their own. */
#define NEST_TRAIN_TICKET 256
size_t nest_route_workspace_size(const nest_route_desc *desc);

/* DEVICE buffers: logits, mask (uint8 [T] or NULL), ids int32 [T][k], weights float
 * [T][k], counts int32 [E], live int32 [1] (n), mean_prob float [E], loss float [1]. */
int nest_route(const nest_route_desc *desc, const void *logits, const uint8_t *mask, int32_t *ids,
               float *weights, int32_t *counts, int32_t *live, float *mean_prob, float *loss,
               void *workspace, size_t ws_bytes, void *stream);

/* Gradient with respect to the logits, given the gradients of the loss (float [1], NULL
 * = 0) and of the weights (float [T][k], NULL = 0), with ids, weights, counts and live
 * as nest_route wrote them for the same logits, mask and description.  The counts are
 * constants of the gradient.  With
 *   d[t][e] = grad_loss * E c[e] / (k n^2) + (u[t][j] where e = ids[t][j])
 *   u[t][j] = grad_weights[t][j], or when normalize is set
 *             (grad_weights[t][j] - sum over j' of grad_weights[t][j'] weights[t][j'])
 *             / (sum over j' of p[t][ids[t][j']])
 * grad_logits[t][e] = p[t][e] (d[t][e] - sum over e' of p[t][e'] d[t][e']), rounded once
 * to the logits' type; rows that are not live hold 0.  Ids outside [0, E) count as -1.
 *   grad_logits   DEVICE [T][E] in the logits' type, rows grad_stride >= E elements apart */
int nest_route_backward(const nest_route_desc *desc, const void *logits, const uint8_t *mask,
                        const int32_t *ids, const float *weights, const int32_t *counts,
                        const int32_t *live, const float *grad_weights, const float *grad_loss,
                        void *grad_logits, int64_t grad_stride, void *stream);

/* ---- lists of tensors -----------------------------------------------------------
 * The optimizer's entry points work on a list of tensors through a table in device
 * memory, packed once on the host.  Elements are taken in blocks of NEST_OPT_BLOCK;
 * every tensor starts a new block, and the list's own buffers (master weights, moments,
 * scales) hold the blocks of all tensors back to back: tensor i's element j is element
 * NEST_OPT_BLOCK * (blocks of the tensors before i) + j, and what lies between the end
 * of a tensor and its last block's end is never written.                            */
#define NEST_OPT_BLOCK 256

typedef struct {
    void *weight;        /* DEVICE, contiguous; may be NULL in a list used for norms only */
    const void *grad;    /* DEVICE, contiguous, numel elements */
    int64_t numel;       /* >= 0; pointers of empty tensors are not read */
    float weight_decay;  /* of this tensor */
    float lr_scale;      /* this tensor's learning rate over the step's */
} nest_tensor;

typedef struct {
    int64_t table_bytes; /* of the packed table */
    int64_t blocks;      /* NEST_OPT_BLOCK-element blocks of the list, < 2^31 */
    int64_t items;       /* runs of blocks of one tensor that one worker takes */
    int32_t tensors;
    int32_t workers;     /* even shares of the blocks that the kernels are launched over */
} nest_table_info;

/* Sizes of the packed table of n >= 0 tensors (HOST array). */
int nest_table_query(const nest_tensor *tensors, int32_t n, nest_table_info *out);

/* Packs the table into HOST memory of info->table_bytes bytes; the caller copies it to
 * the device (16-byte aligned).  The table holds the tensors' addresses: it is packed
 * again when one of them moves. */
int nest_table_pack(const nest_tensor *tensors, int32_t n, const nest_table_info *info, void *table_host);

/* ---- gradient norm -----------------------------------------------------------------
 *   out[0] = sqrt(sum over all tensors of grad^2)
 *   out[1] = min(1, max_norm / (out[0] + 1e-6)), NaN when out[0] is not finite
 * Squares are summed in 32 bits, with the rounding errors of the long sums added up beside
 * them; gradients beyond 1.8e19 overflow to an infinite norm.
 *   out   DEVICE float [2];  max_norm > 0 (may be infinite: out[1] = 1)
 *   workspace   as nest_route's: its first NEST_TRAIN_TICKET bytes zero on entry and after */
size_t nest_grad_norm_workspace_size(const nest_table_info *info);
int nest_grad_norm(const nest_table_info *info, const void *table, int32_t grad_type, float max_norm,
                   float *out, void *workspace, size_t ws_bytes, void *stream);

/* ---- AdamW -------------------------------------------------------------------------
 * With t the number of steps including this one, g = grad_scale * grad, per element
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   w = w - lr lr_scale (m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps) + weight_decay w)
 * in 32 bits on the master weight, which the weight is the rounding of (32-bit weights
 * are their own master).  When *grad_scale is not finite the call changes nothing, the
 * step count included.
 *
 * Moments in 8 bits: each block holds its moments as 3-bit-mantissa floats times a power
 * of two 2^s chosen per block and moment so that the largest finite magnitude a of the
 * block is below 1.75 * 2^s, s in [-100, 120]:
 *   m   sign, 4 exponent bits, 3 mantissa bits, bias 7, of the value m * 2^(8-s)
 *       (largest 448, smallest 2^-9; 0x7F and 0xFF: NaN)
 *   v   5 exponent bits, 3 mantissa bits, bias 32, no sign, of the value v * 2^(-1-s)
 *       (largest 0.875, smallest 2^-34; 0xFF: NaN)
 * A moment that is not finite is held as NaN.  Rounding is stochastic, so that a moment
 * that changes by less than a step per call still moves in the mean: 16 bits of noise r
 * from (seed, t, block, position) are added below the last bit kept, which rounds up
 * with the probability (to 2^-16) of the part cut off.  The update of the weight uses
 * the moments before they are rounded.                                              */
typedef struct {
    double beta1_t, beta2_t;   /* beta1^t, beta2^t of the steps taken: 1, 1 at the start */
    int64_t step;              /* steps taken */
    uint32_t ticket;           /* 0 between calls */
    uint32_t reserved;
} nest_adamw_state;            /* DEVICE, 16-byte aligned; read and advanced by each call */

typedef struct {
    int32_t weight_type, grad_type;  /* NEST_F32, NEST_BF16 or NEST_F16 */
    int32_t state_bits;              /* 32 or 8 */
    uint32_t seed;                   /* of the stochastic rounding (8 bits) */
    double lr, beta1, beta2, eps;    /* 0 <= beta < 1, eps >= 0 */
    float *master;                   /* DEVICE float [blocks][256]; NULL iff weight_type is NEST_F32 */
    void *m, *v;                     /* DEVICE float or uint8 [blocks][256] */
    int8_t *m_exp, *v_exp;           /* DEVICE int8 [blocks] (s above); NULL with 32 bits */
    nest_adamw_state *state;         /* DEVICE */
    const float *grad_scale;         /* DEVICE float [1], e.g. out + 1 of nest_grad_norm; NULL = 1 */
} nest_adamw_args;                   /* the list's buffers are 256-byte aligned */

int nest_adamw(const nest_table_info *info, const void *table, const nest_adamw_args *args, void *stream);

/* The values that 8-bit moments stand for, as bf16 (exact: four significant bits and a
 * power of two).  m_out, v_out: DEVICE bf16 [blocks][256], 256-byte aligned. */
int nest_adamw_values(const nest_table_info *info, const void *m, const void *v, const int8_t *m_exp,
                      const int8_t *v_exp, void *m_out, void *v_out, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* NEST_TRAIN_H */
