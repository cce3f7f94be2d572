/*
 * bf16delta_loss.h -- C ABI of libbf16delta, the losses of a policy update:
 * from a model's logits to the gradients that the optimizer step
 * (bf16delta_step.h) takes, and what a sampler reports for the tokens it drew.
 *   bf16d_logprob          : log probabilities of given tokens, with the
 *                            distributions' entropy and the top alternatives
 *   bf16d_policy_loss      : the clipped policy loss and its gradients
 *   bf16d_logprob_backward : the gradient of the logits
 *   bf16d_balance, bf16d_balance_backward : the balance loss of a router,
 *                            its per-expert counts and its gradient
 *
 * Conventions are those of bf16delta.h (the caller owns every buffer, work is
 * enqueued on `stream`, BF16D_EINVAL means that nothing was enqueued), with
 * these differences.  Every call enqueues one kernel and nothing else: no copy,
 * no allocation, no host synchronisation; it may be captured into a HIP
 * graph.  `stream` must belong to the current device (NULL: its null stream).
 * Logits, ids and gradients need the alignment of their type only; written
 * arrays and workspaces are 16-byte aligned.
 *
 * Workspaces: device memory of *_workspace_bytes, all zero before the first call
 * that uses them; every call leaves its counters zero again.  Calls that share a workspace
 * or a written buffer must not overlap in time; nor must replays of graphs that
 * hold such calls.
 *
 * A written range may overlap nothing else of its call, except where it is
 * said.  Sums, softmax statistics and losses are held in 32 bits or more; a
 * gradient of bf16 logits is rounded once, to the nearest, as it is stored.
 * Equal inputs give equal bits: no result depends on the order of atomics.
 */
#ifndef BF16DELTA_LOSS_H
#define BF16DELTA_LOSS_H

#include "bf16delta.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BF16D_LOGITS_BF16 0u
#define BF16D_LOGITS_F32  1u
#define BF16D_IDS_I64     0u
#define BF16D_IDS_I32     1u
#define BF16D_MAX_VOCAB   (1u << 28)
#define BF16D_MAX_TOP     64u
#define BF16D_MAX_EXPERTS 1024u

/* Rows in two levels: row r begins at data + (r / inner) * outer_stride +
 * (r % inner) * inner_stride elements (inner is the call's), and its elements
 * are adjacent.  So logits[:, :-1] of a (batch, length, vocab) tensor is one
 * set of rows.  Rows that are read may overlap each other, or be one (stride 0). */
typedef struct bf16d_rows {
    void    *data;
    uint64_t outer_stride, inner_stride;
} bf16d_rows;

/* ---- log probabilities of given tokens ------------------------------------ */

/* What the backward pass needs of a row; 16 bytes. */
typedef struct bf16d_row_stats {
    float max;        /* m, the largest logit */
    float log2_sum;   /* log2 of S = sum over j of e^((x_j - m) / temperature) */
    float entropy;    /* H, or NaN where it was not asked for */
    float scale;      /* log2(e) / temperature */
} bf16d_row_stats;

/* For every row x of `vocab` logits with its token y, p the softmax of x / temperature:
 *   logp       = ln p_y
 *   entropy    = H = -sum over j of p_j ln p_j          (NULL: not computed)
 *   top_ids    = the ids of the `top` largest logits, largest first, equal ones
 *                by their id, and top_logp = ln p of each   (top 0: NULL)
 * each of outer * inner rows (top values a row), and
 *   stats      : for the backward pass (NULL: not written).
 *
 * A logit of -infinity is a token that cannot occur: its p is 0, it adds nothing
 * to H, and it is no alternative (as a given token it has logp = -infinity).
 * Where fewer than `top` are left, the rest has id -1 and logp -infinity.
 *   - a negative token leaves its row out: whatever its logits are, logp and
 *     entropy are 0, and it has no alternatives;
 *   - a row of nothing but -infinity has logp = -infinity, entropy 0 and no
 *     alternatives;
 *   - NaN or +infinity among the logits makes the row's logp, entropy and
 *     top_logp NaN (NaN is no alternative);
 *   - a token from `vocab` on has logp = NaN.
 * Logits of any finite size are fine, a mask of the type's lowest value among
 * them.  A log probability below fp32's range (the lowest value over a temperature
 * below 1) is -infinity; as an alternative it keeps its id, and its p of 0 adds
 * nothing to H or to a gradient.
 *
 * temperature: from 2^-20 to 2^20.  outer * inner is below 2^24 (with alternatives
 * below 2^22), vocab from 1 to BF16D_MAX_VOCAB, top at most BF16D_MAX_TOP.  With no
 * rows, pointers may be NULL. */
typedef struct bf16d_logprob_job {
    bf16d_rows       logits;        /* of logits_dtype, BF16D_LOGITS_* */
    bf16d_rows       tokens;        /* of token_dtype, BF16D_IDS_*; one id a row */
    uint64_t         outer, inner;
    uint32_t         vocab, logits_dtype, token_dtype, top;
    double           temperature;
    float           *logp, *entropy;
    bf16d_row_stats *stats;
    int64_t         *top_ids;
    float           *top_logp;
} bf16d_logprob_job;

/* For every call of up to `rows` rows, and up to `top` alternatives. */
size_t bf16d_logprob_workspace_bytes(uint64_t rows, uint32_t vocab, uint32_t top);

int bf16d_logprob(const bf16d_logprob_job *job, void *workspace, size_t workspace_bytes,
                  hipStream_t stream);

/* The gradient of sum over the rows of grad_logp * logp + grad_entropy * entropy
 * by the logits, a = grad_logp and h = grad_entropy of the row:
 *   out_j = (a (1[j = y] - p_j) - h p_j (ln p_j + H)) / temperature
 * `stats` are those that bf16d_logprob wrote for these logits (with an entropy,
 * where grad_entropy is given; NULL: h = 0); the temperature is the one it
 * was given.
 *   - rows that are left out, rows of nothing but -infinity, and rows whose
 *     a and h are 0 receive zeros, whatever their logits hold;
 *   - else a token from `vocab` on, and NaN or +infinity among the logits, make
 *     the row NaN, which a gradient norm reports.
 * out: rows of the logits' type; its rows may not overlap each other.  It
 * may be the logits (the same address and strides), else nothing of it may
 * lie between the logits' first and last byte. */
typedef struct bf16d_logprob_grad_job {
    bf16d_rows             logits, tokens, out;
    uint64_t               outer, inner;
    uint32_t               vocab, logits_dtype, token_dtype, reserved;   /* 0 */
    const bf16d_row_stats *stats;
    const float           *grad_logp, *grad_entropy;
} bf16d_logprob_grad_job;

int bf16d_logprob_backward(const bf16d_logprob_grad_job *job, hipStream_t stream);

/* ---- clipped policy loss -------------------------------------------------- */

/* Means over the tokens by their weights, the loss aside; all 0 where the sum of
 * the weights is 0. */
typedef struct bf16d_policy_result {
    float    loss;       /* scale * sum of weight * l */
    float    weight;     /* sum of the weights */
    float    kl;         /* mean of r - 1 - ln r: how far the policy has moved from `old` */
    float    clipped;    /* share of the tokens whose ratio was clipped */
    float    entropy;    /* mean entropy (0 without entropies) */
    uint32_t reserved[3];
} bf16d_policy_result;

/* For each of n tokens, with r = e^(logp - old) and A its advantage:
 *   l = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
 *       + kl_coef (e^(ref - logp) - 1 - (ref - logp)) - entropy_coef entropy
 *   grad_logp    = scale weight dl/dlogp     (0 through a clipped ratio; one on
 *                                             the border is not clipped)
 *   grad_entropy = -scale weight entropy_coef
 * computed in 64 bits from the 32-bit inputs and rounded once.  A token of weight 0 adds nothing and
 * has gradients 0, whatever its other numbers are; weights NULL: all 1.  A of
 * 0 has r A = 0 and no gradient, for any r.  ref may be NULL
 * where kl_coef is 0, entropy where entropy_coef is 0 (it is then left out of the
 * result); grad_entropy may be NULL.
 * clip_low: from 0 to below 1; clip_high: from 0, infinity for none;
 * kl_coef, entropy_coef, scale: finite.  n is below 2^40.  The arrays are 4-byte
 * aligned; the gradients' 16-byte. */
typedef struct bf16d_policy_job {
    const float *logp, *old, *advantages, *weights, *ref, *entropy;
    float       *grad_logp, *grad_entropy;
    uint64_t     n;
    double       clip_low, clip_high, kl_coef, entropy_coef, scale;
} bf16d_policy_job;

size_t bf16d_policy_loss_workspace_bytes(void);

int bf16d_policy_loss(const bf16d_policy_job *job, bf16d_policy_result *result, void *workspace,
                      size_t workspace_bytes, hipStream_t stream);

/* ---- balance loss of a router ---------------------------------------------- */

typedef struct bf16d_balance_result {
    float    loss;       /* balance_coef * balance + z_coef * z */
    float    balance;
    float    z;
    uint32_t reserved;
    int64_t  tokens;     /* N */
} bf16d_balance_result;

/* Over the tokens t with mask[t] != 0 (mask NULL: all), N of them, p_t the
 * softmax of row t of the router's logits over `experts`, and c_e how often
 * their `chosen` ids name expert e (f_e = c_e / sum of c):
 *   balance = experts * sum over e of f_e * (mean over t of p_te)
 *   z       = mean over t of (ln sum over e of e^x_te)^2
 *   counts  = c
 * balance is 1 where either is even.  Its gradient goes through p; f is a constant.
 *   - a negative id is no choice; one from `experts` on makes loss and balance NaN
 *     (and counts hold the rest);
 *   - a row of nothing but -infinity adds nothing to the sums, and is a token;
 *   - NaN or +infinity in a row that counts makes loss, balance and z NaN;
 *   - with no tokens balance and z are 0, with no choices balance is.
 * rows is below 2^24; experts from 1 to BF16D_MAX_EXPERTS, choices from 1 to
 * experts.  Rows of logits and of chosen ids begin logits_stride and
 * chosen_stride elements apart. */
typedef struct bf16d_balance_job {
    const void    *logits;          /* of logits_dtype, BF16D_LOGITS_* */
    const void    *chosen;          /* of chosen_dtype, BF16D_IDS_* */
    const uint8_t *mask;
    uint64_t       rows, logits_stride, chosen_stride;
    uint32_t       experts, choices, logits_dtype, chosen_dtype;
    double         balance_coef, z_coef;    /* finite */
    int64_t       *counts;          /* experts numbers */
} bf16d_balance_job;

size_t bf16d_balance_workspace_bytes(uint32_t experts);

int bf16d_balance(const bf16d_balance_job *job, bf16d_balance_result *result, void *workspace,
                  size_t workspace_bytes, hipStream_t stream);

/* out = scale * (the gradient of the loss by the logits), of their type, rows
 * out_stride elements apart:
 *   out_te = scale p_te (balance_coef experts (f_e - sum over j of p_tj f_j)
 *                        + 2 z_coef ln(sum over j of e^x_tj)) / N
 * from `counts` and `tokens` (N) in device memory: those that bf16d_balance wrote, or,
 * where several ranks hold a part of the batch each, their sums.  N counts as at least 1.
 * Rows that do not count, and rows of nothing but -infinity, receive zeros.  NaN or
 * +infinity make their row NaN; where the loss of `result` (what bf16d_balance
 * wrote; NULL: it is not looked at) is NaN, every row that counts becomes NaN, so
 * that an id out of range reaches the gradient norm, too.  out may be the
 * logits (the same address and stride). */
typedef struct bf16d_balance_grad_job {
    const void    *logits;
    void          *out;
    const uint8_t *mask;
    uint64_t       rows, logits_stride, out_stride;
    uint32_t       experts, logits_dtype;
    double         balance_coef, z_coef, scale;    /* finite, and their products */
    const int64_t *counts, *tokens;
    const bf16d_balance_result *result;
} bf16d_balance_grad_job;

int bf16d_balance_backward(const bf16d_balance_grad_job *job, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* BF16DELTA_LOSS_H */
