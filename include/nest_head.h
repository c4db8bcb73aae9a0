/*
 * nest_head.h - C ABI of the losses at a model's output head, beside the training-step
 * operators of nest_train.h.
 *
 * The last stage of a pipeline ends in the product of its hidden states with the output
 * weights, whose logits are the largest activation of a model with a large vocabulary:
 * tokens * vocabulary numbers, against tokens * hidden of a layer's output.  These entry
 * points compute two losses of those logits, and the gradients of hidden states and
 * weights, without keeping them: the logits are made in tiles and reduced where they are
 * made, and made again for the gradients, whose workspace holds the losses' derivatives in 16
 * bits of a piece of the vocabulary (up to 256 MiB, or 8192 columns; tokens rounded up to 256).
 *
 * Conventions are those of nest_train.h: the caller allocates every buffer, a call only
 * checks its arguments and enqueues kernels on the caller's stream, and the same inputs
 * give the same bits.  Results and workspace share no memory with the inputs or with each other:
 * the kernels read the ones while they write the others (calls do not check it).
 */
#ifndef NEST_HEAD_H
#define NEST_HEAD_H

#include "nest_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- losses -------------------------------------------------------------------
 * z[t][v] = sum over d of hidden[t][d] weight[v][d], V = vocab, in 32 bits: the tensor cores add
 * 16 products at a time and cut the sum off towards zero.  Every z is multiplied by 1 + f ceil(D / 16)
 * 2^-24, f = 0.26 (NEST_BF16) or 0.30 (NEST_F16), which is what sums like a model's logits lose by
 * that in the mean.  Other sums differ: of products of one sign they lose up to 0.46, and a sum that
 * loses nothing (rows padded with zeros, rows of few numbers) comes out too large by the factor,
 * 1.1e-6 of z for every 1024 of D.
 *
 * Labels (k = 0): label[t] = index[t].  Token t counts ("is live") when its label is in
 * [0, V), and
 *   losses[t] = lse[t] - z[t][label[t]],   lse[t] = log(sum over v of exp(z[t][v]))
 *
 * A teacher's largest logits (k >= 1): index[t][j] are columns and teacher[t][j] the
 * teacher's logits of them, in any order.  A slot counts when mask is NULL or mask[t] != 0,
 * its index is in [0, V) and its logit is not minus infinity; a token is live when one of its slots
 * counts.  With the temperature h
 *   q[t][j]   = exp(teacher[t][j] / h) / sum over the row's slots that count
 *   lse[t]    = log(sum over v of exp(z[t][v] / h))
 *   losses[t] = h^2 sum over j of q[t][j] (log q[t][j] - z[t][index[t][j]] / h + lse[t])
 * A column that is listed twice has the sum of both shares in the gradients (each slot has
 * its own log q in the loss); one whose share is 0 in 32 bits adds nothing.
 *
 * Both: loss = the mean of losses over the n live tokens, 0 when n = 0; live = n.  Tokens
 * that are not live have losses and lse 0, and whatever their hidden states hold (NaN
 * included) reaches no result.  NaN in a live token's row gives it a NaN loss.  A logit of
 * minus infinity adds nothing to lse; as a target's it makes the loss infinite, and a row that
 * is nothing else has lse minus infinity and a NaN loss.  (Where z log2(e) / h of a row's
 * largest logit is beyond 32 bits, its results are not finite.)                          */
#define NEST_I32 0
#define NEST_I64 1

typedef struct {
    int64_t tokens;                      /* 0 <= T <= 2^24, with ceil(T / 256) ceil(V / 128) <= 2^30 */
    int64_t vocab;                       /* 1 <= V <= 2^24 */
    int64_t hidden;                      /* 1 <= D <= 2^16 */
    int64_t hidden_row, hidden_col;      /* strides in elements, >= 0 */
    int64_t weight_row, weight_col;      /* strides in elements, >= 0 */
    int32_t dtype;                       /* of hidden and weight: NEST_BF16 or NEST_F16 */
    int32_t index_type;                  /* NEST_I32 or NEST_I64 */
    int32_t k;                           /* 0: labels; 1 .. 256: listed teacher logits per token */
    int32_t teacher_type;                /* NEST_F32, NEST_BF16 or NEST_F16 (k >= 1) */
    float temperature;                   /* h in [2^-10, 2^10]; 1 with labels */
    int32_t reserved;                    /* 0 */
} nest_head_desc;

/* Device workspace in bytes of the two calls with these weights (their address decides
 * whether they are copied first: rows that are not contiguous or not 16-byte aligned), 0 when
 * the description breaks a limit.  Uninitialised memory will do, 256-byte aligned. */
size_t nest_head_loss_workspace_size(const nest_head_desc *desc, const void *weight);
size_t nest_head_backward_workspace_size(const nest_head_desc *desc, const void *weight);

/* DEVICE buffers: hidden [T][D], weight [V][D], index [T] or [T][k], teacher [T][k], mask
 * (uint8 [T] or NULL), loss float [1], losses float [T], lse float [T], live int32 [1].
 * teacher and mask are NULL with labels. */
int nest_head_loss(const nest_head_desc *desc, const void *hidden, const void *weight, const void *index,
                   const void *teacher, const uint8_t *mask, float *loss, float *losses, float *lse, int32_t *live,
                   void *workspace, size_t ws_bytes, void *stream);

/* Gradients of hidden states and weights from those of the mean (grad_loss, float [1], NULL =
 * 0) and of each token's loss (grad_losses, float [T], NULL = 0), with lse as nest_head_loss
 * wrote it for the same inputs.  With g[t] = grad_loss / n + grad_losses[t] and p the softmax
 * of z / h (h = 1 with labels), q of a label 1:
 *   dz[t][v]          = g[t] h (p[t][v] - sum over j with index[t][j] = v of q[t][j])
 *   grad_hidden[t][d] = sum over v of dz[t][v] weight[v][d]
 *   grad_weight[v][d] = sum over live t of dz[t][v] hidden[t][d]
 * dz is rounded once to the inputs' type - without grad_losses p - q, before the factor that
 * all rows share, else relative to a power of two above every finite |g[t] h| - and lifted by
 * 2^15 in NEST_F16, which would lose small p otherwise; the sums are in 32 bits and rounded
 * once to the inputs' type.  Tokens that are not live have gradient 0.
 *   grad_hidden   DEVICE [T][D], grad_weight DEVICE [V][D], contiguous; one of them may be
 *                 NULL, which leaves out its product                                     */
int nest_head_loss_backward(const nest_head_desc *desc, const void *hidden, const void *weight, const void *index,
                            const void *teacher, const uint8_t *mask, const float *lse, const float *grad_loss,
                            const float *grad_losses, void *grad_hidden, void *grad_weight, void *workspace,
                            size_t ws_bytes, void *stream);

/* Warps of these calls' kernels on the current device whose wait for a copy or a product gave
 * up after 2 s, since the library was loaded: 0 unless the GPU failed or stood still.  What
 * they did not see is NaN in the results, which NaN in the inputs would give too; the count
 * tells the two apart.  Unlike the calls above it waits for the work that is on the stream,
 * and cannot be captured. */
int nest_head_waits_given_up(int64_t *count, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* NEST_HEAD_H */
