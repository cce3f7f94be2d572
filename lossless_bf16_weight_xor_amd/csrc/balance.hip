// balance.hip -- the balance loss of a router, the tokens each expert was
// chosen for, and the gradient of the router's logits.
//
// The gradient of balance = E sum f_e P_e needs every f_e, so it is a pass of
// its own: the first one sums p and counts, the second one computes p again.
// A row is held by the next power of two of `experts` lanes (at most 64), each with
// every 64th expert, so softmax sums are a few lane steps, and a lane's sums
// of p over its rows stay in registers.  Workgroups add up in integers (counts,
// and sums of p in steps of 2^-32), so the order of the atomics does not matter.
#include "loss.hpp"

namespace bf16d {
namespace {

constexpr float kLog2E = 1.44269504088896340736f;
constexpr double kFixed = 4294967296.0;   // steps of a sum of p, of which rows < 2^24 give < 2^56

// what the accumulators after the 2 * experts counts and sums are
enum { kSumTokens = 0, kSumBadIds = 1, kSumBadRows = 2, kSumWords = 3 };

__device__ __forceinline__ uint32_t lanes_of(uint32_t experts) {
    return experts > 32 ? 64u : experts > 1 ? 1u << (32 - __clz(experts - 1)) : 1u;
}
// over the `lanes` (a power of two) lanes that share a row
__device__ __forceinline__ float row_max(float v, uint32_t lanes) {
    for (uint32_t d = lanes >> 1; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, (int)d, 64));
    return v;
}
__device__ __forceinline__ float row_sum(float v, uint32_t lanes) {
    for (uint32_t d = lanes >> 1; d >= 1; d >>= 1) v += __shfl_xor(v, (int)d, 64);
    return v;
}

// A row's softmax: e^(x - m) of the lane's experts, their sum over the row
// (0: nothing but -infinity), and m.
template <int kEach>
struct RowSoftmax {
    float e[kEach], sum, m;
};
template <bool kF32, int kEach>
__device__ __forceinline__ RowSoftmax<kEach> row_softmax(const uint8_t *row, bool live,
                                                         uint32_t sub, uint32_t lanes,
                                                         uint32_t experts) {
    RowSoftmax<kEach> r;
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const uint32_t e = sub + 64 * k;
        r.e[k] = -INFINITY;
        if (live && e < experts) {
            if constexpr (kF32) r.e[k] = ((const float *)row)[e];
            else r.e[k] = __uint_as_float((uint32_t)((const uint16_t *)row)[e] << 16);
        }
        m = fmaxf(m, r.e[k]);
    }
    m = row_max(m, lanes);
    r.m = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        r.e[k] = __builtin_amdgcn_exp2f((r.e[k] - r.m) * kLog2E);
        s += r.e[k];
    }
    r.sum = row_sum(s, lanes);
    return r;
}

template <bool kF32, int kEach>
__global__ __launch_bounds__(kThreads) void balance_kernel(BalanceArgs a) {
    __shared__ uint32_t s_count[64 * kEach];
    __shared__ float s_p[kWaves][64 * kEach];
    __shared__ double s_sum[kWaves];
    __shared__ uint32_t s_tokens, s_bad;
    for (uint32_t e = threadIdx.x; e < a.experts; e += kThreads) s_count[e] = 0;
    if (threadIdx.x == 0) s_tokens = s_bad = 0;
    __syncthreads();
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t lanes = lanes_of(a.experts), sub = lane & (lanes - 1);
    const uint32_t held = 64 / lanes;   // rows of a wave
    float p[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) p[k] = 0.0f;
    double squares = 0.0;
    uint32_t tokens = 0, bad = 0;
    for (uint32_t first = (blockIdx.x * kWaves + wave) * held; first < a.rows;
         first += gridDim.x * kWaves * held) {
        const uint32_t row = first + lane / lanes;
        const bool live = row < a.rows && (!a.mask || a.mask[row]);
        const RowSoftmax<kEach> r = row_softmax<kF32, kEach>(
            (const uint8_t *)a.logits + row * a.logits_stride * (kF32 ? 4 : 2), live, sub, lanes,
            a.experts);
        if (r.sum != 0.0f) {   // else nothing, or nothing that counts
            const float inv = 1.0f / r.sum;
#pragma unroll
            for (int k = 0; k < kEach; ++k) p[k] += r.e[k] * inv;
            const float lse = r.m + logf(r.sum);
            if (sub == 0) squares += (double)lse * lse;
        }
        if (!live) continue;
        tokens += sub == 0;
        for (uint32_t j = sub; j < a.choices; j += lanes) {
            const int64_t id = load_id((const uint8_t *)a.chosen +
                                           (row * a.chosen_stride + j) * (a.chosen_i32 ? 4 : 8),
                                       a.chosen_i32);
            if (id >= (int64_t)a.experts) bad = 1;
            else if (id >= 0) atomicAdd(&s_count[id], 1u);
        }
    }
    if (tokens) atomicAdd(&s_tokens, tokens);
    if (bad) atomicOr(&s_bad, 1u);
    // rows of a wave, then the waves, in a fixed order
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        for (uint32_t d = lanes; d < 64; d <<= 1) p[k] += __shfl_xor(p[k], (int)d, 64);
        if (lane < lanes) s_p[wave][lane + 64 * k] = p[k];
    }
    squares = wave_sum(squares);
    if (lane == 0) s_sum[wave] = squares;
    __syncthreads();
    uint64_t dep = 0;
    auto add = [&](uint32_t at, uint64_t v) {
        dep ^= __hip_atomic_fetch_add(a.sums + at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    bool nan = false;
    for (uint32_t e = threadIdx.x; e < a.experts; e += kThreads) {
        float all = 0.0f;
#pragma unroll
        for (uint32_t w = 0; w < kWaves; ++w) all += s_p[w][e];
        nan |= !(all < INFINITY);
        if (s_count[e]) add(e, s_count[e]);
        if (all > 0.0f && all < INFINITY)
            add(a.experts + e, (uint64_t)__double2ll_rn((double)all * kFixed));
    }
    if (nan) add(2 * a.experts + kSumBadRows, 1);
    if (threadIdx.x == 0) {
        if (s_tokens) add(2 * a.experts + kSumTokens, s_tokens);
        if (s_bad) add(2 * a.experts + kSumBadIds, 1);
        double all = 0.0;
#pragma unroll
        for (uint32_t w = 0; w < kWaves; ++w) all += s_sum[w];
        dep ^= __hip_atomic_exchange(a.partial + blockIdx.x, (uint64_t)__double_as_longlong(all),
                                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!last_of(a.done, gridDim.x, dep)) return;

    // the accumulators are read and cleared
    __shared__ double s_tmp[kWaves];
    auto take = [&](uint32_t at) {
        return __hip_atomic_exchange(a.sums + at, (uint64_t)0, __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_AGENT);
    };
    double choices = 0.0, product = 0.0, z = 0.0;
    for (uint32_t e = threadIdx.x; e < a.experts; e += kThreads) {
        const uint64_t c = take(e);
        a.counts[e] = (int64_t)c;
        choices += (double)c;
        product += (double)c * ((double)take(a.experts + e) / kFixed);
    }
    static_assert(kBalanceGrid <= kThreads, "a thread takes one workgroup's sum");
    if (threadIdx.x < gridDim.x)
        z = __longlong_as_double((long long)ld_relaxed_agent(a.partial + threadIdx.x));
    choices = group_total(choices, s_tmp);
    product = group_total(product, s_tmp);
    z = group_total(z, s_tmp);
    if (threadIdx.x == 0) {
        const uint64_t n = take(2 * a.experts + kSumTokens);
        const bool bad_ids = take(2 * a.experts + kSumBadIds) != 0;
        const bool bad_rows = take(2 * a.experts + kSumBadRows) != 0;
        const double over = n ? 1.0 / (double)n : 0.0;
        double balance = choices > 0.0 ? (double)a.experts * product / choices * over : 0.0;
        if (bad_ids || bad_rows) balance = NAN;
        z *= over;
        if (bad_rows) z = NAN;
        a.result->balance = (float)balance;
        a.result->z = (float)z;
        a.result->loss = (float)(a.balance_coef * balance + a.z_coef * z);
        a.result->tokens = (int64_t)n;
        __hip_atomic_store(a.done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

template <bool kF32>
__device__ __forceinline__ void store_element(uint8_t *row, uint32_t e, float v) {
    if constexpr (kF32) ((float *)row)[e] = v;
    else ((__bf16 *)row)[e] = (__bf16)v;
}

template <bool kF32, int kEach>
__global__ __launch_bounds__(kThreads) void balance_grad_kernel(BalanceGradArgs a) {
    __shared__ double s_tmp[kWaves];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t lanes = lanes_of(a.experts), sub = lane & (lanes - 1);
    const uint32_t held = 64 / lanes;
    double choices = 0.0;
    for (uint32_t e = threadIdx.x; e < a.experts; e += kThreads) choices += (double)a.counts[e];
    choices = group_total(choices, s_tmp);
    const double n = *a.tokens > 1 ? (double)*a.tokens : 1.0;
    const float by_share = (float)(a.scale * a.balance_coef * a.experts / n);
    const float by_lse = (float)(2.0 * a.scale * a.z_coef / n);
    const float spoilt = a.result && a.result->loss != a.result->loss ? NAN : 0.0f;
    float share[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const uint32_t e = sub + 64 * k;
        share[k] = e < a.experts && choices > 0.0 ? (float)((double)a.counts[e] / choices) : 0.0f;
    }
    constexpr uint32_t kSize = kF32 ? 4 : 2;
    for (uint32_t first = (blockIdx.x * kWaves + wave) * held; first < a.rows;
         first += gridDim.x * kWaves * held) {
        const uint32_t row = first + lane / lanes;
        const bool live = row < a.rows && (!a.mask || a.mask[row]);
        const RowSoftmax<kEach> r = row_softmax<kF32, kEach>(
            (const uint8_t *)a.logits + row * a.logits_stride * kSize, live, sub, lanes, a.experts);
        const float inv = r.sum != 0.0f ? 1.0f / r.sum : 0.0f;
        float inner = 0.0f;
#pragma unroll
        for (int k = 0; k < kEach; ++k) inner += r.e[k] * share[k];
        inner = row_sum(inner, lanes) * inv;
        const float same = (r.sum != 0.0f ? by_lse * (r.m + logf(r.sum)) : 0.0f) - by_share * inner;
        if (row >= a.rows) continue;
        uint8_t *out = (uint8_t *)a.out + row * a.out_stride * kSize;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const uint32_t e = sub + 64 * k;
            const float g = live ? r.e[k] * inv * (by_share * share[k] + same) + spoilt : 0.0f;
            if (e < a.experts) store_element<kF32>(out, e, g);
        }
    }
}

// lane steps of 64 experts, and the workgroups: `most`, or one for each four waves of rows
uint32_t grid_of(uint32_t rows, uint32_t experts, uint32_t most) {
    uint32_t held = 64;
    while (held > 1 && 64 / held < experts) held >>= 1;
    const uint32_t groups = (rows + kWaves * held - 1) / (kWaves * held);
    return groups < most ? (groups ? groups : 1) : most;
}

template <bool kF32>
hipError_t launch_forward(const BalanceArgs &a, uint32_t grid, hipStream_t stream) {
    auto *kernel = a.experts <= 64    ? balance_kernel<kF32, 1>
                   : a.experts <= 128 ? balance_kernel<kF32, 2>
                   : a.experts <= 256 ? balance_kernel<kF32, 4>
                   : a.experts <= 512 ? balance_kernel<kF32, 8>
                                      : balance_kernel<kF32, 16>;
    return launch_one(kernel, grid, kThreads, a, 0, stream);
}
template <bool kF32>
hipError_t launch_backward(const BalanceGradArgs &a, uint32_t grid, hipStream_t stream) {
    auto *kernel = a.experts <= 64    ? balance_grad_kernel<kF32, 1>
                   : a.experts <= 128 ? balance_grad_kernel<kF32, 2>
                   : a.experts <= 256 ? balance_grad_kernel<kF32, 4>
                   : a.experts <= 512 ? balance_grad_kernel<kF32, 8>
                                      : balance_grad_kernel<kF32, 16>;
    return launch_one(kernel, grid, kThreads, a, 0, stream);
}

}  // namespace

hipError_t launch_balance(const BalanceArgs &a, bool f32, hipStream_t stream) {
    const uint32_t grid = grid_of(a.rows, a.experts, kBalanceGrid);
    return f32 ? launch_forward<true>(a, grid, stream) : launch_forward<false>(a, grid, stream);
}

hipError_t launch_balance_backward(const BalanceGradArgs &a, bool f32, hipStream_t stream) {
    const uint32_t grid = grid_of(a.rows, a.experts, 2048);
    return f32 ? launch_backward<true>(a, grid, stream) : launch_backward<false>(a, grid, stream);
}

}  // namespace bf16d
