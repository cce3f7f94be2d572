/*
 * bf16delta_step.h -- C ABI of libbf16delta, the trainer's side of a weight
 * update: the optimizer step that makes the new BF16 weights of a whole
 * checkpoint out of the old ones, and the gradient norm that it is clipped
 * by.  bf16d_compress (bf16delta.h) then takes (old, new).
 *
 * Conventions are those of bf16delta.h: the caller owns every buffer, device
 * pointers are 16-byte aligned, work is enqueued on `stream`, sizes are at
 * most 2^62, BF16D_EINVAL means that nothing was enqueued.  Both operators are
 * prepared once over fixed buffers and then run at every step:
 *   - *_prepare checks the jobs and uploads them into `table` (device memory
 *     of *_table_bytes, owned by the caller).  It waits for the upload, so the
 *     table may be used on any stream of the device afterwards, and it is refused
 *     (BF16D_EINVAL) on a stream that is being captured.  `plan` (host memory)
 *     receives what the later calls need; copying it is fine.
 *   - the run calls enqueue one kernel and nothing else: no copy, no
 *     allocation, no host synchronisation.  They may be captured into a HIP
 *     graph.  The current device must be the one that was current at
 *     *_prepare, and `stream` must belong to it (NULL: its null stream).
 * The table and every buffer of the jobs must stay valid, at the same
 * addresses, for as long as calls (or graphs that hold them) use the plan.
 * Calls that share a plan, a table or a written buffer must not overlap in
 * time; nor must replays of graphs that hold such calls.  A batch holds fewer
 * than 2^24 chunks of 4096 elements (6.8e10 elements).  BF16D_EHIP also reports a failed host allocation.
 */
#ifndef BF16DELTA_STEP_H
#define BF16DELTA_STEP_H

#include "bf16delta.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BF16D_GRAD_BF16 0u
#define BF16D_GRAD_F32  1u

/* What a prepared operator needs at every call; written by *_prepare. */
typedef struct bf16d_step_plan {
    uint64_t opaque[8];
} bf16d_step_plan;

/* ---- global gradient norm ------------------------------------------------ */

/* One gradient tensor: n elements of the type `dtype` (BF16D_GRAD_*).  grad
 * may be NULL when n == 0.  Types may differ from tensor to tensor. */
typedef struct bf16d_grad {
    const void *grad;
    uint64_t    n;
    uint32_t    dtype;
    uint32_t    reserved;   /* 0 */
} bf16d_grad;

/* Written by the device, 8-byte aligned device memory.
 *   norm      : |grad_scale| * sqrt(sum of grad^2 over all tensors); squares
 *               and sums are in 64 bits, so finite gradients of any size give
 *               a finite norm, and the order of the sums is fixed: equal
 *               inputs give equal bits.
 *   scale     : grad_scale * min(1, max_norm / norm): the factor that turns a
 *               gradient as stored into the one the step uses.
 *   nonfinite : 1 if any gradient, as stored, is infinite or NaN (norm and scale
 *               are then of no use), else 0.  scale is finite in any case, but
 *               scale * gradient, and its square in v, are formed in fp32: they
 *               can overflow from gradients of 3.4e38 and 1.8e19 on, which the
 *               flag does not cover (with a max_norm below 1.8e19 they cannot). */
typedef struct bf16d_norm_result {
    double   norm;
    float    scale;
    uint32_t nonfinite;
} bf16d_norm_result;

size_t bf16d_grad_norm_table_bytes(uint64_t total_n, uint32_t count);

/* `result` receives the outcome of every later call on this plan, and is not
 * written here: before the first call it holds what the caller put there (a
 * nonfinite of 1 makes a step that reads it too early one that is left out).  It
 * may not overlap the gradients or the table. */
int bf16d_grad_norm_prepare(const bf16d_grad *grads, uint32_t count, void *table,
                            size_t table_bytes, bf16d_norm_result *result, hipStream_t stream,
                            bf16d_step_plan *plan);

/* max_norm: above 0; infinity for no clipping.  grad_scale: finite in fp32; what a
 * stored gradient is multiplied by (1 / the number of accumulated batches,
 * for example). */
int bf16d_grad_norm(const bf16d_step_plan *plan, double max_norm, double grad_scale,
                    hipStream_t stream);

/* ---- AdamW --------------------------------------------------------------- */

/* One tensor of n elements.  With g = s * grad, s the norm result's scale (1
 * without one), t the step number and c_i = 1 - beta_i^t:
 *   m   = beta1 * m + (1 - beta1) * g
 *   v   = beta2 * v + (1 - beta2) * g^2
 *   p   = p - lr * lr_scale * (weight_decay * p + (m / c1) / (sqrt(v / c2) + eps))
 *   out = p in bf16
 * computed in 32 bits.
 *
 *   weights : the weights before the step.  Read only without a master copy
 *             (then p is the bf16 weight itself); may be NULL with one.
 *   out     : the weights after the step; may be `weights` (in place), or
 *             the other one of two working copies, so that the pair (weights,
 *             out) is what bf16d_compress takes.
 *   master  : fp32 master copy, updated in place, or NULL.
 *   grad    : gradient, of type grad_dtype.
 *   m, v    : state_bits 32: n floats each.  state_bits 8: n codes each, see
 *             below.
 *   m_scale, v_scale : state_bits 8: ceil(n / 32) bytes each.  state_bits 32:
 *             NULL.
 * With n == 0 the pointers may be NULL.  out, master, m, v and the scales are
 * written and may overlap nothing else of the batch (a tensor that two names
 * share is one job).
 *
 * Rounding of the weights: with a master copy to the nearest, ties to even.
 * Without one stochastically (the next bf16 value away from zero is taken with
 * the probability that the value's position between the two says, in steps of
 * 2^-16): most updates of a step are far smaller than half a bf16 step, and
 * rounding to the nearest would lose them all.
 *
 * 8-bit states: element i stands for e4m3(code[i]) * 2^(scale[i / 32] - 127),
 * e4m3 being the 4-exponent 3-mantissa-bit float (largest value 448, no
 * infinities, 0x7F and 0xFF NaN) and the scale byte an 8-bit exponent (255
 * stands for nothing).  Cleared states (all bytes 0) are zeros.  At each step a
 * block's scale is the smallest power of two, at least 2^-126, with which its
 * largest finite magnitude does not pass 448, and each magnitude is rounded
 * stochastically to the e4m3 grid.  A positive v is never rounded to 0 (the
 * smallest code stands for it): m may not be divided by eps alone because v
 * was lost.
 * Infinities and NaN are held as NaN, in their element only.
 * The rounding is stochastic because a step lowers v by at most 1 - beta2 of
 * itself, at beta2 = 0.999 far less than half a step of the e4m3 grid (3 to
 * 6 %): rounded to the nearest, v could never fall.  Its price is noise: against
 * 32-bit states on Gaussian gradients, v differs by 13, 18 and 21 % (rms) at beta2
 * = 0.95, 0.99 and 0.999 (a longer memory collects hardly more, since a small
 * change seldom moves a code: 33 % is a bound for all of these), m by 9 % at
 * beta1 = 0.9, and the update by 11, 13 and 14 % (its mean by 1 to 2 %).
 *
 * Random numbers: element i of job j has number e = start_j + i, start_j the
 * sum of the earlier jobs' n, each rounded up to a multiple of 512.  With
 * K = mix64(mix64(seed) + step) (mix64: the SplitMix64 finaliser), k0 and k1
 * its low and high halves, and all words 32 bits wide:
 *   x  = low(e) ^ k0
 *   x  = (x ^ x >> 16) * 0xBF58476D + k1 + high(e) * 0x9E3779B9
 *   x  = (x ^ x >> 15) * 0x94D049BB
 *   x ^= x >> 16
 * m is rounded with the low half of x, v with its high half, the weight with
 * the high half of x * 0x9E3779B1.  A fraction of a step, cut to 16 bits, plus
 * such a half rounds up where it reaches 2^16.  Batches of one model should
 * have seeds of their own. */
typedef struct bf16d_adamw_job {
    const uint16_t *weights;
    uint16_t       *out;
    float          *master;
    const void     *grad;
    void           *m;
    void           *v;
    uint8_t        *m_scale;
    uint8_t        *v_scale;
    uint64_t        n;
    float           lr_scale;       /* these two and their product: */
    float           weight_decay;   /*   finite, not negative */
    uint32_t        grad_dtype;     /* BF16D_GRAD_* */
    uint32_t        reserved;       /* 0 */
} bf16d_adamw_job;

/* lr: finite in fp32, not negative; beta1, beta2: in [0, 1); eps: from 2^-50 (8.9e-16;
 * beside a smaller one, the root of a v too small for fp32 would count) to
 * 2^100; step: from 1.  lr_device (4-byte aligned) and step_device (8-byte
 * aligned), where not NULL, are device words read by the kernel in place of
 * lr and step, for calls captured in a graph; a step word of 0 counts as 1. */
typedef struct bf16d_adamw_params {
    double          lr, beta1, beta2, eps;
    uint64_t        step;
    uint64_t        seed;
    const float    *lr_device;
    const uint64_t *step_device;
} bf16d_adamw_params;

size_t bf16d_adamw_table_bytes(uint64_t total_n, uint32_t count);

/* state_bits: 32 or 8, for all jobs of the plan. */
int bf16d_adamw_prepare(const bf16d_adamw_job *jobs, uint32_t count, uint32_t state_bits,
                        void *table, size_t table_bytes, hipStream_t stream,
                        bf16d_step_plan *plan);

/* One step over every job.  norm: a device result of bf16d_grad_norm whose
 * scale multiplies the gradients, or NULL.  If its nonfinite flag is set, the
 * step is left out: masters and states keep their values, and out receives the
 * weights as they are (bf16(master), or a copy of `weights`).  The caller
 * advances the step number, by 1 - nonfinite so that a step left out does not
 * count. */
int bf16d_adamw_step(const bf16d_step_plan *plan, const bf16d_adamw_params *params,
                     const bf16d_norm_result *norm, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* BF16DELTA_STEP_H */
