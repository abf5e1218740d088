/*
 * muonstep_train.h -- C ABI of what a training step runs next to the Muon step
 * on MI355X (gfx950): the softmax cross entropy of the language-model head with
 * its gradients, and AdamW with 8-bit states.
 *
 * "Record: L_ParallelResiduals_UNetSkips_DepthRecur_Muon_ 1.0901" (PR #1893),
 * "Architecture and training stack", gives the model these serve (512 wide, a
 * vocabulary of 4096, AdamW on the embeddings and scalars); the page prints
 * neither operator's equations, which are stated at each entry below.
 *
 * The conventions, error codes and muon_last_error() of muonstep.h hold here:
 * device pointers, everything validated on the host before anything is
 * enqueued, work ordered on `stream`, no allocation, no synchronisation,
 * results that do not depend on scheduling (no atomics).
 */
#ifndef MUONSTEP_TRAIN_H
#define MUONSTEP_TRAIN_H

#include "muonstep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * AdamW with 8-bit states.
 *
 * One tensor of the update: numel contiguous values.  Either
 *   8-bit states (exp_avg_scale set): exp_avg and rms hold one OCP e4m3 code
 *     per value, in units of a float32 scale for each MUON_ADAMW8_BLOCK
 *     consecutive values (ceil(numel / MUON_ADAMW8_BLOCK) scales):
 *       m = exp_avg[i] * exp_avg_scale[i / 256],
 *       sqrt(v) = rms[i] * rms_scale[i / 256];
 *   or 32-bit states (both scales NULL): exp_avg holds m and rms holds v, as
 *     float32 (adamw_step's exp_avg and exp_avg_sq).
 * param (float32) and the states are updated in place; grad (float32 or
 * bfloat16, by grad_bf16) is read only; ema (float32) and copy (bfloat16) are
 * optional (NULL): the weight EMA on the updated parameter, and the updated
 * parameter rounded to bfloat16, which the next forward pass reads.
 * None of the buffers of any tensor of a call may overlap. */
#define MUON_ADAMW8_BLOCK 256
typedef struct adamw8_tensor_t {
    float* param;
    const void* grad;
    void* exp_avg;
    float* exp_avg_scale;
    void* rms;
    float* rms_scale;
    float* ema;
    void* copy;
    int64_t numel;
    int32_t grad_bf16;
} adamw8_tensor_t;

/* AdamW over n tensors.  Per value, every operation in float32 and rounded by
 * itself (no fused multiply-add), with t = step:
 *   m <- beta1 m + (1 - beta1) g;   v <- beta2 v + (1 - beta2) g^2
 *   p <- (1 - lr*wd) p - (m / (sqrt(v) / sqrt(1 - beta2^t) + eps)) lr / (1 - beta1^t)
 * then ema <- ema_decay ema + (1 - ema_decay) p and copy <- p where set.  8-bit
 * states are then written back per block: scale = top / 448 with top the
 * block's largest |m| (or sqrt(v)), code = |x| * (448 * (1 / top)) in e4m3:
 *   nearest     (dither == 0): to the nearest code, halves to the smaller;
 *   stochastic  (dither == 1): up with the probability of the part cut off
 *               (to 2^-16), from 32 mixed bits of (seed, step, tensor's place
 *               in the list, value's index): the moments' averages then keep
 *               increments below half a step on the average, and the same
 *               arguments give the same bits.  All tensors draw from one
 *               sequence of 2^32, each from a place of its own: long ones may
 *               share a stretch of it, and beyond 2^32 values it repeats.
 * A v above zero never becomes the zero code.  A block with a value that is
 * not finite gets a NaN scale: its states are lost as a whole, as the
 * parameters are.  Blocks whose largest value is below 2^-100 are written as zero
 * (sqrt(v): as the smallest code).
 * The scalars, step and seed among them, are arguments of the launches: a captured
 * graph repeats the step that was captured.
 * Argument limits as adamw_step; tensors with numel == 0 are skipped.  param,
 * exp_avg, rms, scales, ema: 4-byte aligned (8-bit codes: any); grad, copy: aligned to
 * their type.  Aligned to 16 bytes (codes: 4, bfloat16: 8) they take the
 * vector path, with the same results. */
int adamw8_step(const adamw8_tensor_t* tensors, int32_t n, float lr, float beta1, float beta2, float eps,
                float weight_decay, int32_t step, float ema_decay, int32_t dither, uint64_t seed, void* stream);

/* 8-bit states from float32 moments (to the nearest code) and back, for
 * checkpoints and for changing between adamw_step's states and these.
 * exp_avg_sq must not be negative; the two directions read their input only. */
int adamw8_encode(const float* exp_avg, const float* exp_avg_sq, void* exp_avg_codes, float* exp_avg_scale,
                  void* rms_codes, float* rms_scale, int64_t numel, void* stream);
int adamw8_decode(const void* exp_avg_codes, const float* exp_avg_scale, const void* rms_codes,
                  const float* rms_scale, float* exp_avg, float* exp_avg_sq, int64_t numel, void* stream);

/* ------------------------------------------------------------------------
 * Softmax cross entropy of the language-model head, without the logits.
 *
 * With z_ij = hidden_i . weight_j, l = softcap tanh(z / softcap) (softcap 0: l = z):
 *   lse_i = log sum_j exp l_ij;   nll_i = lse_i - l_i,targets[i]
 *   g_i = token_weights[i], or 1 / (counted tokens) where token_weights is NULL
 *   loss = sum_i g_i nll_i
 *   grad_hidden = d loss / d hidden;   grad_weight = d loss / d weight.
 * A token whose target is ignore_index is not counted: its nll and lse are 0,
 * its gradient row is 0, and whatever its hidden state holds (NaN, infinity)
 * reaches nothing.  With no counted token loss and gradients are 0.  A
 * target outside [0, vocab) that is not ignore_index gives a NaN nll (and
 * loss and gradients); nothing is read out of range.
 *
 *   hidden       tokens x dim, weight vocab x dim: 16-bit floats of type `dtype`,
 *                dim values contiguous, rows hidden_stride / weight_stride
 *                elements apart (>= dim; weight rows must not overlap).
 *   targets      int64 per token.
 *   token_weights  NULL or float32 per token (finite).
 *   nll          float32 per token.    lse   NULL or float32 per token.
 *   loss         NULL or one float32.
 *   grad_hidden, grad_weight   NULL or rows like hidden and weight, overwritten
 *                (not added to).  Each is computed only if given; with both and
 *                loss NULL the call only scores.
 *   A buffer reaches from its first element to its last, the gaps of strided
 *   rows included: what is written may overlap nothing else.
 *   tokens >= 0, vocab >= 1, dim >= 1 (limits below); softcap finite, >= 0.
 * Products take their 16-bit inputs as they are and sum in float32; the
 * probabilities are rounded to 16 bits once, before they are multiplied with
 * weight and hidden; gradients are rounded once.  Probabilities come from
 * exponentials kept in float16 in units of the largest of 32, 64 or 128
 * neighbours: they have 11 significant bits down to 2^-29 of it and end at
 * 2^-40.  Under a softcap l and the factor 1 - (l / softcap)^2 are off by a few ulp of
 * themselves, and the exponential is kept multiplied by the factor: the same bounds
 * hold for the two together.  nll and lse have the same bits
 * whatever else is asked for.  dim a multiple of 8 with
 * 16-byte aligned rows is read in place, anything else through a padded copy
 * in the workspace.
 * For gradients the tokens go through the workspace in pieces of at most
 * MUON_HEAD_PIECE_BYTES of 16-bit values (vocab x piece), never all logits of a
 * large batch at once. */
#define MUON_HEAD_BF16 0
#define MUON_HEAD_FP16 1
#define MUON_HEAD_MAX_TOKENS (1 << 24)
#define MUON_HEAD_MAX_VOCAB (1 << 22)
#define MUON_HEAD_MAX_DIM 65536
#define MUON_HEAD_PIECE_BYTES ((int64_t)2 << 30)
typedef struct head_loss_t {
    const void* hidden;
    const void* weight;
    const int64_t* targets;
    const float* token_weights;
    float* loss;
    float* nll;
    float* lse;
    void* grad_hidden;
    void* grad_weight;
    int64_t tokens, vocab, dim;
    int64_t hidden_stride, weight_stride, grad_hidden_stride, grad_weight_stride;
    int64_t ignore_index;
    float softcap;
    int32_t dtype;
} head_loss_t;

/* Bytes of device workspace head_loss needs for this problem: its sizes,
 * strides (<= 2^22), which outputs it has and the alignment of hidden and weight.  0 if the
 * arguments are invalid (see muon_last_error()). */
size_t head_loss_workspace_size(const head_loss_t* problem);

/* The loss (and gradients).  workspace: a device buffer of at least
 * head_loss_workspace_size(...) bytes, 256-byte aligned, that overlaps no
 * tensor; its contents on entry do not matter. */
int head_loss(const head_loss_t* problem, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MUONSTEP_TRAIN_H */
