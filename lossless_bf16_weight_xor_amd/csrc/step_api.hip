// step_api.hip -- host side of the optimizer step's C ABI (see
// include/bf16delta_step.h): checks the jobs once, uploads them with the
// chunk -> job map, and launches one kernel per call.
#include <cmath>
#include <cstring>

#include "host_checks.hpp"
#include "step.hpp"

using namespace bf16d;

namespace {

// What bf16d_step_plan holds.
struct Plan {
    uint64_t magic;     // which operator prepared it
    const void *jobs;
    const uint32_t *map;
    uint64_t chunks;
    void *partial;      // norm: partial sums, then the counter
    bf16d_norm_result *result;
    int32_t device;
    uint32_t state_bits;
    uint32_t lds_bytes, kept;
};
static_assert(sizeof(Plan) == sizeof(bf16d_step_plan), "the plan is opaque words");
constexpr uint64_t kNormMagic = 0x4D524F4E44363146ull;    // "F16DNORM"
constexpr uint64_t kAdamMagic = 0x4D41444144363146ull;    // "F16DADAM"

// jobs, the chunk -> job map, and the norm's partial sums and counter
struct Table {
    size_t map, partial, done, total;
};
Table table_layout(size_t job_bytes, uint32_t count, uint64_t chunks, bool norm) {
    Table t;
    t.map = align_up(job_bytes * count, 256);
    t.partial = align_up(t.map + 4 * chunks, 256);
    t.done = t.partial + (norm ? 8 * size_t(kNormGrid) : 0);
    t.total = t.done + (norm ? 256 : 0);
    return t;
}
uint64_t chunks_of(uint64_t n, uint32_t chunk) { return (n + chunk - 1) / chunk; }

// The table's content, uploaded and there when the call returns.
int upload(void *table, const std::vector<uint8_t> &host, hipStream_t stream) {
    if (hipMemcpyAsync(table, host.data(), host.size(), hipMemcpyHostToDevice, stream) !=
        hipSuccess)
        return BF16D_EHIP;
    return hipStreamSynchronize(stream) == hipSuccess ? BF16D_OK : BF16D_EHIP;
}

// a prepare waits for its upload, which a capture does not allow
int prepare_stream(hipStream_t stream, int32_t &dev) {
    const int rc = stream_on_current(stream, dev);
    if (rc != BF16D_OK) return rc;
    hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(stream, &st) != hipSuccess) return BF16D_EHIP;
    return st == hipStreamCaptureStatusNone ? BF16D_OK : BF16D_EINVAL;
}

int norm_prepare(const bf16d_grad *grads, uint32_t count, void *table, size_t table_bytes,
                 bf16d_norm_result *result, hipStream_t stream, bf16d_step_plan *plan) {
    if (!grads || count == 0 || !table || !aligned16(table) || !result || !plan ||
        (reinterpret_cast<uintptr_t>(result) & 7u) != 0)
        return BF16D_EINVAL;
    std::vector<Range> ranges;
    ranges.reserve(size_t(count) + 2);
    uint64_t chunks = 0, bytes = 0, kept = 0;
    for (uint32_t j = 0; j < count; ++j) {
        const bf16d_grad &G = grads[j];
        if (G.n > kMaxSize / 4 || G.dtype > BF16D_GRAD_F32 || G.reserved != 0 ||
            (G.n > 0 && (!G.grad || !aligned16(G.grad))))
            return BF16D_EINVAL;
        const uint64_t size = G.dtype == BF16D_GRAD_F32 ? 4 : 2;
        chunks += chunks_of(G.n, kNormChunk);
        if (chunks >= kMaxTiles) return BF16D_EINVAL;
        // the chunks that begin within the first kNormKept bytes
        if (bytes < kNormKept)
            kept += std::min(chunks_of(G.n, kNormChunk),
                             chunks_of(kNormKept - bytes, uint32_t(kNormChunk * size)));
        bytes += G.n * size;
        add_range(ranges, G.grad, G.n * size, false);
    }
    const Table t = table_layout(sizeof(NormJob), count, chunks, true);
    if (table_bytes < t.total) return BF16D_EINVAL;
    add_range(ranges, table, t.total, true);
    add_range(ranges, result, sizeof *result, true);
    if (!ranges_disjoint(ranges)) return BF16D_EINVAL;
    Plan p{};
    const int rc = prepare_stream(stream, p.device);
    if (rc != BF16D_OK) return rc;

    std::vector<uint8_t> host(t.total, 0);
    auto *dj = reinterpret_cast<NormJob *>(host.data());
    auto *map = reinterpret_cast<uint32_t *>(host.data() + t.map);
    uint64_t c = 0;
    for (uint32_t j = 0; j < count; ++j) {
        dj[j].grad = (BF16D_GMEM const void *)grads[j].grad;
        dj[j].chunk0 = uint32_t(c);
        dj[j].full_chunks = uint32_t(grads[j].n / kNormChunk);
        dj[j].tail = uint32_t(grads[j].n % kNormChunk);
        dj[j].dtype = grads[j].dtype;
        for (const uint64_t end = c + chunks_of(grads[j].n, kNormChunk); c < end; ++c) map[c] = j;
    }
    auto *base = static_cast<uint8_t *>(table);
    p.magic = kNormMagic;
    p.jobs = base;
    p.map = reinterpret_cast<const uint32_t *>(base + t.map);
    p.chunks = chunks;
    p.partial = base + t.partial;
    p.result = result;
    p.kept = bytes <= kNormKeptTotal ? uint32_t(kept) : 0;
    const int up = upload(table, host, stream);
    if (up == BF16D_OK) std::memcpy(plan, &p, sizeof p);
    return up;
}

// The LDS a workgroup (one wave) of the step asks for, to limit how many run on
// a CU at once: kAdamFlight bytes of loads in flight, by the batch's mean.
uint32_t flight_lds(uint64_t loaded, uint64_t total) {
    if (total == 0) return 0;
    const double wave = double(loaded) / double(total) * kAdamGroup;   // bytes a wave loads
    const double waves = kAdamFlight / wave;
    return waves >= 31.0 ? 0 : uint32_t(kLdsBytes / waves) & ~1023u;
}

bool rate_ok(float x) { return std::isfinite(x) && x >= 0.0f; }

int adamw_prepare(const bf16d_adamw_job *jobs, uint32_t count, uint32_t state_bits, void *table,
                  size_t table_bytes, hipStream_t stream, bf16d_step_plan *plan) {
    if (!jobs || count == 0 || (state_bits != 32 && state_bits != 8) || !table ||
        !aligned16(table) || !plan)
        return BF16D_EINVAL;
    const bool bits8 = state_bits == 8;
    std::vector<Range> ranges;
    ranges.reserve(8 * size_t(count) + 1);
    uint64_t chunks = 0, number = 0, total = 0, loaded = 0;
    for (uint32_t j = 0; j < count; ++j) {
        const bf16d_adamw_job &J = jobs[j];
        if (J.n > kMaxSize / 4 || J.grad_dtype > BF16D_GRAD_F32 || J.reserved != 0 ||
            !rate_ok(J.lr_scale) || !rate_ok(J.weight_decay) ||
            !rate_ok(J.lr_scale * J.weight_decay))
            return BF16D_EINVAL;
        if (!aligned16(J.weights) || !aligned16(J.out) || !aligned16(J.master) ||
            !aligned16(J.grad) || !aligned16(J.m) || !aligned16(J.v) || !aligned16(J.m_scale) ||
            !aligned16(J.v_scale))
            return BF16D_EINVAL;
        if (J.n > 0) {
            if (!J.out || !J.grad || !J.m || !J.v || (!J.master && !J.weights))
                return BF16D_EINVAL;
            if (bits8 != (J.m_scale != nullptr) || bits8 != (J.v_scale != nullptr))
                return BF16D_EINVAL;
        }
        chunks += chunks_of(J.n, kAdamChunk);
        if (chunks >= kMaxTiles) return BF16D_EINVAL;
        total += J.n;
        loaded += J.n * ((J.master ? 4 : 2) + (J.grad_dtype == BF16D_GRAD_F32 ? 4 : 2) +
                         (bits8 ? 2 : 8));
        const uint64_t state = bits8 ? J.n : 4 * J.n;
        const uint64_t scales = bits8 ? chunks_of(J.n, kScaleBlock) : 0;
        // without a master copy the weights may be updated in place: each
        // thread stores the elements it has loaded, and no others
        if (!J.master && J.weights != J.out) add_range(ranges, J.weights, 2 * J.n, false);
        add_range(ranges, J.out, 2 * J.n, true);
        if (J.master) add_range(ranges, J.master, 4 * J.n, true);
        add_range(ranges, J.grad, J.n * (J.grad_dtype == BF16D_GRAD_F32 ? 4 : 2), false);
        add_range(ranges, J.m, state, true);
        add_range(ranges, J.v, state, true);
        add_range(ranges, J.m_scale, scales, true);
        add_range(ranges, J.v_scale, scales, true);
    }
    const Table t = table_layout(sizeof(AdamJob), count, chunks, false);
    if (table_bytes < t.total) return BF16D_EINVAL;
    add_range(ranges, table, t.total, true);
    if (!ranges_disjoint(ranges)) return BF16D_EINVAL;
    Plan p{};
    const int rc = prepare_stream(stream, p.device);
    if (rc != BF16D_OK) return rc;

    std::vector<uint8_t> host(t.total, 0);
    auto *dj = reinterpret_cast<AdamJob *>(host.data());
    auto *map = reinterpret_cast<uint32_t *>(host.data() + t.map);
    uint64_t c = 0;
    for (uint32_t j = 0; j < count; ++j) {
        const bf16d_adamw_job &J = jobs[j];
        dj[j].weights = (BF16D_GMEM const uint16_t *)J.weights;
        dj[j].out = (BF16D_GMEM uint16_t *)J.out;
        dj[j].master = (BF16D_GMEM float *)J.master;
        dj[j].grad = (BF16D_GMEM const void *)J.grad;
        dj[j].m = (BF16D_GMEM void *)J.m;
        dj[j].v = (BF16D_GMEM void *)J.v;
        dj[j].m_scale = (BF16D_GMEM uint8_t *)J.m_scale;
        dj[j].v_scale = (BF16D_GMEM uint8_t *)J.v_scale;
        dj[j].number0 = number;
        dj[j].chunk0 = uint32_t(c);
        dj[j].full_chunks = uint32_t(J.n / kAdamChunk);
        dj[j].tail = uint32_t(J.n % kAdamChunk);
        dj[j].lr_scale = J.lr_scale;
        dj[j].decay = J.lr_scale * J.weight_decay;
        dj[j].grad_dtype = J.grad_dtype;
        number += align_up(J.n, kNumberSpan);
        for (const uint64_t end = c + chunks_of(J.n, kAdamChunk); c < end; ++c) map[c] = j;
    }
    auto *base = static_cast<uint8_t *>(table);
    p.magic = kAdamMagic;
    p.jobs = base;
    p.map = reinterpret_cast<const uint32_t *>(base + t.map);
    p.chunks = chunks;
    p.state_bits = state_bits;
    p.lds_bytes = flight_lds(loaded, total);
    const int up = upload(table, host, stream);
    if (up == BF16D_OK) std::memcpy(plan, &p, sizeof p);
    return up;
}

// The plan's content, if it is one of this operator; its device must be the
// current one and `stream`'s.
int read_plan(const bf16d_step_plan *plan, uint64_t magic, Plan &p) {
    if (!plan) return BF16D_EINVAL;
    std::memcpy(&p, plan, sizeof p);
    return p.magic == magic ? BF16D_OK : BF16D_EINVAL;
}
int check_device(const Plan &p, hipStream_t stream) {
    int32_t dev = -1;
    const int rc = stream_on_current(stream, dev);
    if (rc != BF16D_OK) return rc;
    return dev == p.device ? BF16D_OK : BF16D_EINVAL;
}

bool beta_ok(double b) { return b >= 0.0 && b < 1.0; }

}  // namespace

extern "C" {

size_t bf16d_grad_norm_table_bytes(uint64_t total_n, uint32_t count) {
    return table_layout(sizeof(NormJob), count, chunks_of(total_n, kNormChunk) + count, true)
        .total;
}

size_t bf16d_adamw_table_bytes(uint64_t total_n, uint32_t count) {
    return table_layout(sizeof(AdamJob), count, chunks_of(total_n, kAdamChunk) + count, false)
        .total;
}

int bf16d_grad_norm_prepare(const bf16d_grad *grads, uint32_t count, void *table,
                            size_t table_bytes, bf16d_norm_result *result, hipStream_t stream,
                            bf16d_step_plan *plan) {
    try {
        return norm_prepare(grads, count, table, table_bytes, result, stream, plan);
    } catch (...) {   // host memory
        return BF16D_EHIP;
    }
}

int bf16d_grad_norm(const bf16d_step_plan *plan, double max_norm, double grad_scale,
                    hipStream_t stream) {
    Plan p;
    int rc = read_plan(plan, kNormMagic, p);
    if (rc != BF16D_OK) return rc;
    // The step multiplies by the scale in fp32.  Clipping only makes it smaller, so
    // where grad_scale is finite there, the scale is.
    if (!(max_norm > 0.0) || !std::isfinite(float(grad_scale))) return BF16D_EINVAL;
    rc = check_device(p, stream);
    if (rc != BF16D_OK) return rc;
    NormArgs a{};
    a.jobs = static_cast<const NormJob *>(p.jobs);
    a.map = p.map;
    a.partial = static_cast<uint64_t *>(p.partial);
    a.done = reinterpret_cast<uint32_t *>(a.partial + kNormGrid);
    a.result = p.result;
    a.chunks = uint32_t(p.chunks);
    a.kept = p.kept;
    a.max_norm = max_norm;
    a.grad_scale = grad_scale;
    return launch_grad_norm(a, stream) == hipSuccess ? BF16D_OK : BF16D_EHIP;
}

int bf16d_adamw_prepare(const bf16d_adamw_job *jobs, uint32_t count, uint32_t state_bits,
                        void *table, size_t table_bytes, hipStream_t stream,
                        bf16d_step_plan *plan) {
    try {
        return adamw_prepare(jobs, count, state_bits, table, table_bytes, stream, plan);
    } catch (...) {   // host memory
        return BF16D_EHIP;
    }
}

int bf16d_adamw_step(const bf16d_step_plan *plan, const bf16d_adamw_params *params,
                     const bf16d_norm_result *norm, hipStream_t stream) {
    Plan p;
    int rc = read_plan(plan, kAdamMagic, p);
    if (rc != BF16D_OK) return rc;
    if (!params || (reinterpret_cast<uintptr_t>(norm) & 7u) != 0 ||
        (reinterpret_cast<uintptr_t>(params->lr_device) & 3u) != 0 ||
        (reinterpret_cast<uintptr_t>(params->step_device) & 7u) != 0)
        return BF16D_EINVAL;
    const bf16d_adamw_params &P = *params;
    // below 2^-50 the root of a v that fp32 cannot hold would count, and a 1 / d
    // of a larger eps than 2^100 would be denormal
    if (!beta_ok(P.beta1) || !beta_ok(P.beta2) || !(P.eps >= 0x1p-50) || !(P.eps <= 0x1p100))
        return BF16D_EINVAL;
    if (!P.lr_device && !rate_ok(float(P.lr))) return BF16D_EINVAL;
    if (!P.step_device && P.step == 0) return BF16D_EINVAL;
    rc = check_device(p, stream);
    if (rc != BF16D_OK) return rc;
    AdamArgs a{};
    a.jobs = static_cast<const AdamJob *>(p.jobs);
    a.map = p.map;
    a.norm = norm;
    a.lr_device = P.lr_device;
    a.step_device = P.step_device;
    a.lr = P.lr;
    // beta 0 has logarithm -infinity, and 1 - beta^t = -expm1(-infinity) = 1
    a.log_beta1 = std::log(P.beta1);
    a.log_beta2 = std::log(P.beta2);
    a.numbers = step_numbers(P.lr, P.step, P.seed, a.log_beta1, a.log_beta2);
    a.beta1 = float(P.beta1);
    a.beta2 = float(P.beta2);
    a.rest1 = float(1.0 - P.beta1);
    a.rest2 = float(1.0 - P.beta2);
    a.eps = float(P.eps);
    a.seed = P.seed;
    a.step = P.step;
    a.groups = uint32_t(p.chunks) * kAdamSplit;
    return launch_adamw(a, p.state_bits, p.lds_bytes, stream) == hipSuccess ? BF16D_OK
                                                                            : BF16D_EHIP;
}

}  // extern "C"
