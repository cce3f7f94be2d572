// loss_api.hip -- host side of the losses' C ABI (see include/bf16delta_loss.h):
// checks the arguments of a call, chooses how it is cut into workgroups, and
// launches its one kernel.
#include <cmath>

#include "host_checks.hpp"
#include "loss.hpp"

using namespace bf16d;

namespace {

constexpr uint64_t kMaxRows = 1ull << 24;      // below this: a workgroup each, 2^32 threads
constexpr uint64_t kMaxWideRows = kMaxRows * kThreads / kLogprobWide;
constexpr uint64_t kMaxTokens = 1ull << 40;

bool aligned(const void *p, uint64_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
uint64_t logits_size(uint32_t dtype) { return dtype == BF16D_LOGITS_F32 ? 4 : 2; }
uint64_t id_size(uint32_t dtype) { return dtype == BF16D_IDS_I32 ? 4 : 8; }

// x * y + z, or false beyond 2^62
bool mul_add(uint64_t x, uint64_t y, uint64_t z, uint64_t &out) {
    const unsigned __int128 v = (unsigned __int128)x * y + z;
    out = (uint64_t)v;
    return v <= kMaxSize;
}

// The bytes from the first element of `rows` rows of `width` to behind the last
// one; false where that passes 2^62.
bool extent(const bf16d_rows &r, uint64_t outer, uint64_t inner, uint64_t width, uint64_t size,
            uint64_t &bytes) {
    uint64_t e = 0;
    return mul_add(outer - 1, r.outer_stride, 0, e) && mul_add(inner - 1, r.inner_stride, e, e) &&
           mul_add(e + width, size, 0, bytes);
}

// Whether no two rows share an element: the rows of one level lie within the
// steps of the other.
bool rows_apart(const bf16d_rows &r, uint64_t outer, uint64_t inner, uint64_t width) {
    auto nested = [&](uint64_t n_small, uint64_t small, uint64_t n_large, uint64_t large) {
        uint64_t span = width;
        if (n_small > 1 && (small < width || !mul_add(n_small - 1, small, width, span)))
            return false;
        return n_large <= 1 || large >= span;
    };
    return nested(inner, r.inner_stride, outer, r.outer_stride) ||
           nested(outer, r.outer_stride, inner, r.inner_stride);
}

// whether every row starts at a 16-byte address
bool rows_aligned(const bf16d_rows &r, uint64_t outer, uint64_t inner, uint64_t size) {
    return aligned16(r.data) && (outer <= 1 || r.outer_stride * size % 16 == 0) &&
           (inner <= 1 || r.inner_stride * size % 16 == 0);
}

RowSet row_set(const bf16d_rows &r) { return RowSet{r.data, r.outer_stride, r.inner_stride}; }

// rows = outer * inner; false where there are too many
bool count_rows(uint64_t outer, uint64_t inner, uint64_t &rows) {
    return mul_add(outer, inner, 0, rows) && rows < kMaxRows && outer < kMaxRows &&
           inner < kMaxRows;
}

// How rows are cut: into `parts` workgroups each, of part_turns turns, enough for
// kLogprobGroups in all.  With alternatives for no more than that: two on a CU take
// longer than one that reads on (200 rows of 50021 bf16, 20 alternatives: 14.8 us whole, cut
// in two 17.8; 96 of 131072 fp32 cut in two 20.3, in three 22.4).
struct Cut {
    uint32_t parts, part_turns;
};
Cut cut_rows(uint64_t rows, uint32_t turns, bool alternatives) {
    const uint64_t wanted = alternatives ? std::max<uint64_t>(1, kLogprobGroups / rows)
                                         : (kLogprobGroups + rows - 1) / rows;
    const uint32_t parts = uint32_t(std::min<uint64_t>(wanted, turns));
    const uint32_t each = (turns + parts - 1) / parts;
    return Cut{(turns + each - 1) / each, each};   // whole turns each: fewer parts may do
}

// counters (rows in parts are fewer than kLogprobGroups), then the parts' words
constexpr size_t kCounterBytes = 4 * size_t(kLogprobGroups);
size_t logprob_workspace(uint64_t rows, uint32_t turns, uint32_t top) {
    if (rows == 0 || turns <= 1) return 0;
    // rows * ceil(groups / rows) is below groups + rows, and nothing is cut from
    // `groups` rows on
    const uint64_t cut = std::min<uint64_t>(rows, kLogprobGroups - 1);
    const uint64_t words = std::min<uint64_t>(cut * turns, kLogprobGroups + cut) * (2 + top);
    return kCounterBytes + 8 * words;
}
static_assert(kLogprobWide >= kThreads, "a wide workgroup's turns are fewer");

bool finite(double x) { return std::isfinite(x); }

int logprob(const bf16d_logprob_job *job, void *workspace, size_t workspace_bytes,
            hipStream_t stream) {
    if (!job) return BF16D_EINVAL;
    const bf16d_logprob_job &J = *job;
    uint64_t rows = 0;
    if (!count_rows(J.outer, J.inner, rows) || J.vocab == 0 || J.vocab > BF16D_MAX_VOCAB ||
        J.logits_dtype > BF16D_LOGITS_F32 || J.token_dtype > BF16D_IDS_I32 ||
        J.top > BF16D_MAX_TOP || (J.top > 0 && rows >= kMaxWideRows) ||
        !(J.temperature >= 0x1p-20) || !(J.temperature <= 0x1p20))
        return BF16D_EINVAL;
    if (!aligned16(J.logp) || !aligned16(J.entropy) || !aligned16(J.stats) ||
        !aligned16(J.top_ids) || !aligned16(J.top_logp) || !aligned16(workspace) ||
        !aligned(J.logits.data, logits_size(J.logits_dtype)) ||
        !aligned(J.tokens.data, id_size(J.token_dtype)))
        return BF16D_EINVAL;
    const uint64_t size = logits_size(J.logits_dtype);
    const bool at16 = rows_aligned(J.logits, J.outer, J.inner, size);
    const uint32_t turns = turns_of(J.vocab, J.logits_dtype, at16, kThreads);
    if (rows > 0) {
        if (!J.logits.data || !J.tokens.data || !J.logp) return BF16D_EINVAL;
        if ((J.top > 0) != (J.top_ids != nullptr) || (J.top > 0) != (J.top_logp != nullptr))
            return BF16D_EINVAL;
        uint64_t logits_bytes = 0, token_bytes = 0;
        if (!extent(J.logits, J.outer, J.inner, J.vocab, size, logits_bytes) ||
            !extent(J.tokens, J.outer, J.inner, 1, id_size(J.token_dtype), token_bytes))
            return BF16D_EINVAL;
        const size_t need = logprob_workspace(rows, turns, J.top);
        if (workspace_bytes < need || (need && !workspace)) return BF16D_EINVAL;
        std::vector<Range> ranges;
        add_range(ranges, J.logits.data, logits_bytes, false);
        add_range(ranges, J.tokens.data, token_bytes, false);
        add_range(ranges, J.logp, 4 * rows, true);
        if (J.entropy) add_range(ranges, J.entropy, 4 * rows, true);
        if (J.stats) add_range(ranges, J.stats, sizeof(bf16d_row_stats) * rows, true);
        add_range(ranges, J.top_ids, 8 * rows * J.top, true);
        add_range(ranges, J.top_logp, 4 * rows * J.top, true);
        add_range(ranges, workspace, need, true);
        if (!ranges_disjoint(ranges)) return BF16D_EINVAL;
    }
    int32_t dev = -1;
    const int rc = stream_on_current(stream, dev);
    if (rc != BF16D_OK || rows == 0) return rc;
    LogprobArgs a{};
    a.logits = row_set(J.logits);
    a.tokens = row_set(J.tokens);
    a.rows = uint32_t(rows);
    a.inner = uint32_t(J.inner);
    a.vocab = J.vocab;
    a.token_i32 = J.token_dtype == BF16D_IDS_I32;
    a.top = J.top;
    // see kLogprobWide
    const uint32_t wide_turns = turns_of(J.vocab, J.logits_dtype, at16, kLogprobWide);
    const bool wide = J.top > 0 || (turns > 1 && wide_turns == 1 && rows <= kLogprobGroups);
    const Cut cut = cut_rows(rows, wide ? wide_turns : turns, J.top > 0);
    a.parts = cut.parts;
    a.part_turns = cut.part_turns;
    const bool keep = J.stats && rows * J.vocab * size <= kLogprobKept;
    a.scale = float(1.4426950408889634 / J.temperature);
    a.inv_t = float(1.0 / J.temperature);
    a.logp = J.logp;
    a.entropy = J.entropy;
    a.stats = J.stats;
    a.top_ids = J.top_ids;
    a.top_logp = J.top_logp;
    a.done = static_cast<uint32_t *>(workspace);
    a.partial = reinterpret_cast<uint64_t *>(static_cast<uint8_t *>(workspace) + kCounterBytes);
    return launch_logprob(a, J.logits_dtype == BF16D_LOGITS_F32, wide, keep, stream) == hipSuccess
               ? BF16D_OK
               : BF16D_EHIP;
}

int logprob_backward(const bf16d_logprob_grad_job *job, hipStream_t stream) {
    if (!job) return BF16D_EINVAL;
    const bf16d_logprob_grad_job &J = *job;
    uint64_t rows = 0;
    if (!count_rows(J.outer, J.inner, rows) || J.vocab == 0 || J.vocab > BF16D_MAX_VOCAB ||
        J.logits_dtype > BF16D_LOGITS_F32 || J.token_dtype > BF16D_IDS_I32 || J.reserved != 0)
        return BF16D_EINVAL;
    const uint64_t size = logits_size(J.logits_dtype);
    if (!aligned(J.logits.data, size) || !aligned(J.out.data, size) ||
        !aligned(J.tokens.data, id_size(J.token_dtype)) || !aligned16(J.stats) ||
        !aligned(J.grad_logp, 4) || !aligned(J.grad_entropy, 4))
        return BF16D_EINVAL;
    if (rows > 0) {
        if (!J.logits.data || !J.tokens.data || !J.out.data || !J.stats || !J.grad_logp)
            return BF16D_EINVAL;
        uint64_t logits_bytes = 0, token_bytes = 0, out_bytes = 0;
        if (!extent(J.logits, J.outer, J.inner, J.vocab, size, logits_bytes) ||
            !extent(J.tokens, J.outer, J.inner, 1, id_size(J.token_dtype), token_bytes) ||
            !extent(J.out, J.outer, J.inner, J.vocab, size, out_bytes) ||
            !rows_apart(J.out, J.outer, J.inner, J.vocab))
            return BF16D_EINVAL;
        // strides of a level with one row do not matter
        const bool in_place =
            J.out.data == J.logits.data &&
            (J.outer == 1 || J.out.outer_stride == J.logits.outer_stride) &&
            (J.inner == 1 || J.out.inner_stride == J.logits.inner_stride);
        std::vector<Range> ranges;
        if (!in_place) add_range(ranges, J.logits.data, logits_bytes, false);
        add_range(ranges, J.tokens.data, token_bytes, false);
        add_range(ranges, J.stats, sizeof(bf16d_row_stats) * rows, false);
        add_range(ranges, J.grad_logp, 4 * rows, false);
        if (J.grad_entropy) add_range(ranges, J.grad_entropy, 4 * rows, false);
        add_range(ranges, J.out.data, out_bytes, true);
        if (!ranges_disjoint(ranges)) return BF16D_EINVAL;
    }
    int32_t dev = -1;
    const int rc = stream_on_current(stream, dev);
    if (rc != BF16D_OK || rows == 0) return rc;
    const uint32_t turns = turns_of(J.vocab, J.logits_dtype,
                                    rows_aligned(J.logits, J.outer, J.inner, size), kThreads);
    LogprobGradArgs a{};
    a.logits = row_set(J.logits);
    a.tokens = row_set(J.tokens);
    a.out = row_set(J.out);
    a.rows = uint32_t(rows);
    a.inner = uint32_t(J.inner);
    a.vocab = J.vocab;
    a.token_i32 = J.token_dtype == BF16D_IDS_I32;
    // a turn each, or as many as the grid's limit asks for
    const uint64_t most = std::max<uint64_t>(1, (kMaxTiles - 1) / rows);
    a.part_turns = uint32_t((turns + most - 1) / most);
    a.parts = (turns + a.part_turns - 1) / a.part_turns;
    a.stats = J.stats;
    a.grad_logp = J.grad_logp;
    a.grad_entropy = J.grad_entropy;
    return launch_logprob_backward(a, J.logits_dtype == BF16D_LOGITS_F32, stream) == hipSuccess
               ? BF16D_OK
               : BF16D_EHIP;
}

// partial sums, then the counters
constexpr size_t kPolicyPartial = 8 * size_t(kPolicyGrid) * kPolicySums;

int policy_loss(const bf16d_policy_job *job, bf16d_policy_result *result, void *workspace,
                size_t workspace_bytes, hipStream_t stream) {
    if (!job || !result || !aligned16(result) || !workspace || !aligned16(workspace) ||
        workspace_bytes < bf16d_policy_loss_workspace_bytes())
        return BF16D_EINVAL;
    const bf16d_policy_job &J = *job;
    if (J.n >= kMaxTokens || !(J.clip_low >= 0.0) || !(J.clip_low < 1.0) ||
        !(J.clip_high >= 0.0) || !finite(J.kl_coef) || !finite(J.entropy_coef) ||
        !finite(J.scale))
        return BF16D_EINVAL;
    const float *const read[] = {J.logp, J.old, J.advantages, J.weights, J.ref, J.entropy};
    for (const float *p : read)
        if (!aligned(p, 4)) return BF16D_EINVAL;
    if (!aligned16(J.grad_logp) || !aligned16(J.grad_entropy)) return BF16D_EINVAL;
    if (J.n > 0 && (!J.logp || !J.old || !J.advantages || !J.grad_logp ||
                    (J.kl_coef != 0.0 && !J.ref) || (J.entropy_coef != 0.0 && !J.entropy)))
        return BF16D_EINVAL;
    std::vector<Range> ranges;
    for (const float *p : read)
        if (p) add_range(ranges, p, 4 * J.n, false);
    if (J.grad_logp) add_range(ranges, J.grad_logp, 4 * J.n, true);
    if (J.grad_entropy) add_range(ranges, J.grad_entropy, 4 * J.n, true);
    add_range(ranges, result, sizeof *result, true);
    add_range(ranges, workspace, bf16d_policy_loss_workspace_bytes(), true);
    if (!ranges_disjoint(ranges)) return BF16D_EINVAL;
    int32_t dev = -1;
    const int rc = stream_on_current(stream, dev);
    if (rc != BF16D_OK) return rc;
    PolicyArgs a{};
    a.logp = J.logp;
    a.old = J.old;
    a.advantages = J.advantages;
    a.weights = J.weights;
    a.ref = J.ref;
    a.entropy = J.entropy;
    a.grad_logp = J.grad_logp;
    a.grad_entropy = J.grad_entropy;
    a.n = J.n;
    a.low = 1.0 - J.clip_low;
    a.high = 1.0 + J.clip_high;
    a.log_low = std::log1p(-J.clip_low);
    a.log_high = std::log1p(J.clip_high);
    a.kl_coef = J.kl_coef;
    a.entropy_coef = J.entropy_coef;
    a.scale = J.scale;
    a.result = result;
    a.partial = static_cast<uint64_t *>(workspace);
    a.done = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(workspace) + kPolicyPartial);
    return launch_policy_loss(a, stream) == hipSuccess ? BF16D_OK : BF16D_EHIP;
}

// accumulators (counts, sums of p, three more; in copies), partial sums, the counters
struct BalanceSpace {
    size_t partial, done, total;
};
BalanceSpace balance_space(uint32_t experts) {
    BalanceSpace s;
    s.partial = align_up(8 * kBalanceCopies * (2 * size_t(experts) + 3), 16);
    s.done = s.partial + 8 * size_t(kBalanceGrid);
    s.total = s.done + 4 * kDoneWords;
    return s;
}

// rows of `width`, `stride` apart
bf16d_rows flat(const void *p, uint64_t stride) {
    return bf16d_rows{const_cast<void *>(p), 0, stride};
}

int balance(const bf16d_balance_job *job, bf16d_balance_result *result, void *workspace,
            size_t workspace_bytes, hipStream_t stream) {
    if (!job || !result || !aligned16(result) || !workspace || !aligned16(workspace))
        return BF16D_EINVAL;
    const bf16d_balance_job &J = *job;
    if (J.rows >= kMaxRows || J.experts == 0 || J.experts > BF16D_MAX_EXPERTS ||
        J.choices == 0 || J.choices > J.experts || J.logits_dtype > BF16D_LOGITS_F32 ||
        J.chosen_dtype > BF16D_IDS_I32 || !finite(J.balance_coef) || !finite(J.z_coef))
        return BF16D_EINVAL;
    const BalanceSpace space = balance_space(J.experts);
    if (workspace_bytes < space.total || !J.counts || !aligned16(J.counts) ||
        !aligned(J.logits, logits_size(J.logits_dtype)) ||
        !aligned(J.chosen, id_size(J.chosen_dtype)))
        return BF16D_EINVAL;
    std::vector<Range> ranges;
    if (J.rows > 0) {
        uint64_t logits_bytes = 0, chosen_bytes = 0;
        if (!J.logits || !J.chosen ||
            !extent(flat(J.logits, J.logits_stride), 1, J.rows, J.experts,
                    logits_size(J.logits_dtype), logits_bytes) ||
            !extent(flat(J.chosen, J.chosen_stride), 1, J.rows, J.choices,
                    id_size(J.chosen_dtype), chosen_bytes))
            return BF16D_EINVAL;
        add_range(ranges, J.logits, logits_bytes, false);
        add_range(ranges, J.chosen, chosen_bytes, false);
        if (J.mask) add_range(ranges, J.mask, J.rows, false);
    }
    add_range(ranges, J.counts, 8 * uint64_t(J.experts), true);
    add_range(ranges, result, sizeof *result, true);
    add_range(ranges, workspace, space.total, true);
    if (!ranges_disjoint(ranges)) return BF16D_EINVAL;
    int32_t dev = -1;
    const int rc = stream_on_current(stream, dev);
    if (rc != BF16D_OK) return rc;
    auto *base = static_cast<uint8_t *>(workspace);
    BalanceArgs a{};
    a.logits = J.logits;
    a.chosen = J.chosen;
    a.mask = J.mask;
    a.logits_stride = J.logits_stride;
    a.chosen_stride = J.chosen_stride;
    a.rows = uint32_t(J.rows);
    a.experts = J.experts;
    a.choices = J.choices;
    a.chosen_i32 = J.chosen_dtype == BF16D_IDS_I32;
    a.balance_coef = J.balance_coef;
    a.z_coef = J.z_coef;
    a.counts = J.counts;
    a.result = result;
    a.sums = reinterpret_cast<uint64_t *>(base);
    a.partial = reinterpret_cast<uint64_t *>(base + space.partial);
    a.done = reinterpret_cast<uint32_t *>(base + space.done);
    return launch_balance(a, J.logits_dtype == BF16D_LOGITS_F32, stream) == hipSuccess
               ? BF16D_OK
               : BF16D_EHIP;
}

int balance_backward(const bf16d_balance_grad_job *job, hipStream_t stream) {
    if (!job) return BF16D_EINVAL;
    const bf16d_balance_grad_job &J = *job;
    if (J.rows >= kMaxRows || J.experts == 0 || J.experts > BF16D_MAX_EXPERTS ||
        J.logits_dtype > BF16D_LOGITS_F32 || !finite(J.balance_coef) || !finite(J.z_coef) ||
        !finite(J.scale) || !std::isfinite(float(J.scale * J.balance_coef * J.experts)) ||
        !std::isfinite(float(2.0 * J.scale * J.z_coef)))
        return BF16D_EINVAL;
    const uint64_t size = logits_size(J.logits_dtype);
    if (!aligned(J.logits, size) || !aligned(J.out, size) || !aligned(J.counts, 8) ||
        !aligned(J.tokens, 8) || !aligned(J.result, 8))
        return BF16D_EINVAL;
    if (J.rows > 0) {
        uint64_t logits_bytes = 0, out_bytes = 0;
        if (!J.logits || !J.out || !J.counts || !J.tokens ||
            !extent(flat(J.logits, J.logits_stride), 1, J.rows, J.experts, size, logits_bytes) ||
            !extent(flat(J.out, J.out_stride), 1, J.rows, J.experts, size, out_bytes) ||
            (J.rows > 1 && J.out_stride < J.experts))
            return BF16D_EINVAL;
        const bool in_place =
            J.out == J.logits && (J.rows == 1 || J.out_stride == J.logits_stride);
        std::vector<Range> ranges;
        if (!in_place) add_range(ranges, J.logits, logits_bytes, false);
        if (J.mask) add_range(ranges, J.mask, J.rows, false);
        add_range(ranges, J.counts, 8 * uint64_t(J.experts), false);
        add_range(ranges, J.tokens, 8, false);
        if (J.result) add_range(ranges, J.result, sizeof *J.result, false);
        add_range(ranges, J.out, out_bytes, true);
        if (!ranges_disjoint(ranges)) return BF16D_EINVAL;
    }
    int32_t dev = -1;
    const int rc = stream_on_current(stream, dev);
    if (rc != BF16D_OK || J.rows == 0) return rc;
    BalanceGradArgs a{};
    a.logits = J.logits;
    a.out = J.out;
    a.mask = J.mask;
    a.logits_stride = J.logits_stride;
    a.out_stride = J.out_stride;
    a.rows = uint32_t(J.rows);
    a.experts = J.experts;
    a.balance_coef = J.balance_coef;
    a.z_coef = J.z_coef;
    a.scale = J.scale;
    a.counts = J.counts;
    a.tokens = J.tokens;
    a.result = J.result;
    return launch_balance_backward(a, J.logits_dtype == BF16D_LOGITS_F32, stream) == hipSuccess
               ? BF16D_OK
               : BF16D_EHIP;
}

// a C entry lets no exception out (host memory)
template <typename F>
int guarded(F f) {
    try {
        return f();
    } catch (...) {
        return BF16D_EHIP;
    }
}

}  // namespace

extern "C" {

size_t bf16d_logprob_workspace_bytes(uint64_t rows, uint32_t vocab, uint32_t top) {
    if (vocab == 0) return 0;
    // fp32 rows have more turns
    const uint32_t turns =
        turns_of(std::min(vocab, BF16D_MAX_VOCAB), BF16D_LOGITS_F32, false, kThreads);
    return logprob_workspace(rows, turns, std::min(top, BF16D_MAX_TOP));
}

int bf16d_logprob(const bf16d_logprob_job *job, void *workspace, size_t workspace_bytes,
                  hipStream_t stream) {
    return guarded([&] { return logprob(job, workspace, workspace_bytes, stream); });
}

int bf16d_logprob_backward(const bf16d_logprob_grad_job *job, hipStream_t stream) {
    return guarded([&] { return logprob_backward(job, stream); });
}

size_t bf16d_policy_loss_workspace_bytes(void) { return kPolicyPartial + 4 * kDoneWords; }

int bf16d_policy_loss(const bf16d_policy_job *job, bf16d_policy_result *result, void *workspace,
                      size_t workspace_bytes, hipStream_t stream) {
    return guarded([&] { return policy_loss(job, result, workspace, workspace_bytes, stream); });
}

size_t bf16d_balance_workspace_bytes(uint32_t experts) {
    return balance_space(std::min(experts, BF16D_MAX_EXPERTS)).total;
}

int bf16d_balance(const bf16d_balance_job *job, bf16d_balance_result *result, void *workspace,
                  size_t workspace_bytes, hipStream_t stream) {
    return guarded([&] { return balance(job, result, workspace, workspace_bytes, stream); });
}

int bf16d_balance_backward(const bf16d_balance_grad_job *job, hipStream_t stream) {
    return guarded([&] { return balance_backward(job, stream); });
}

}  // extern "C"
