// policy.hip -- the clipped policy loss over the tokens of a batch, with its
// gradients by the log probabilities and entropies, in one launch.
//
// A token is 12 to 24 bytes read, 4 or 8 written and two exponentials.  All of
// it is in 64 bits: near r = 1, where most tokens are, e^u - 1 - u and the
// distance to the clip range are differences of nearly equal numbers, and the
// arithmetic costs nothing beside the launch.  The clip range is compared as
// logarithms, logp - old being exact in 64 bits.
#include "loss.hpp"

namespace bf16d {
namespace {

// e^u - 1 - u, at least 0; v: e^u - 1
__device__ __forceinline__ double excess(double v, double u) {
    return v == INFINITY ? (double)INFINITY : v - u;
}

__device__ __forceinline__ void group_sums(double (&v)[kPolicySums],
                                           double (*s_tmp)[kPolicySums]) {
#pragma unroll
    for (uint32_t k = 0; k < kPolicySums; ++k) {
        v[k] = wave_sum(v[k]);
        if ((threadIdx.x & 63) == 0) s_tmp[threadIdx.x >> 6][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (uint32_t k = 0; k < kPolicySums; ++k) {
        v[k] = 0.0;
#pragma unroll
        for (uint32_t w = 0; w < kWaves; ++w) v[k] += s_tmp[w][k];
    }
    __syncthreads();
}

__global__ __launch_bounds__(kThreads) void policy_loss_kernel(PolicyArgs a) {
    __shared__ double s_tmp[kWaves][kPolicySums];
    double sum[kPolicySums] = {0.0, 0.0, 0.0, 0.0, 0.0};
    for (uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x; i < a.n;
         i += (uint64_t)gridDim.x * kThreads) {
        const double w = a.weights ? a.weights[i] : 1.0f;
        double slope = 0.0;
        if (w != 0.0) {
            const double lp = a.logp[i], adv = a.advantages[i];
            const double u = lp - a.old[i], v = expm1(u);
            const bool cut =
                (adv > 0.0 && u > a.log_high) || (adv < 0.0 && u < a.log_low);
            double each = 0.0;
            if (cut) {
                each = -(adv > 0.0 ? a.high : a.low) * adv;
            } else if (adv != 0.0) {
                each = slope = -(v + 1.0) * adv;
            }
            if (a.kl_coef != 0.0) {
                const double away = a.ref[i] - lp, grow = expm1(away);
                each += a.kl_coef * excess(grow, away);
                slope -= a.kl_coef * grow;
            }
            if (a.entropy) {
                const double h = a.entropy[i];
                if (a.entropy_coef != 0.0) each -= a.entropy_coef * h;
                sum[4] += w * h;
            }
            sum[0] += w * each;
            sum[1] += w;
            sum[2] += w * excess(v, u);
            sum[3] += cut ? w : 0.0;
            slope *= a.scale * w;
        }
        a.grad_logp[i] = (float)slope;
        if (a.grad_entropy)
            a.grad_entropy[i] = w != 0.0 ? (float)(-a.scale * w * a.entropy_coef) : 0.0f;
    }
    group_sums(sum, s_tmp);
    // handed over by returning device-scope atomics, as last_of asks
    uint64_t dep = 0;
    if (threadIdx.x < kPolicySums) {
        double mine = sum[0];
#pragma unroll
        for (uint32_t k = 1; k < kPolicySums; ++k) mine = threadIdx.x == k ? sum[k] : mine;
        dep = __hip_atomic_exchange(a.partial + blockIdx.x * kPolicySums + threadIdx.x,
                                    (uint64_t)__double_as_longlong(mine), __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!last_of(a.done, gridDim.x, dep)) return;
    static_assert(kPolicyGrid <= kThreads, "a thread takes one workgroup's sums");
#pragma unroll
    for (uint32_t k = 0; k < kPolicySums; ++k)
        sum[k] = threadIdx.x < gridDim.x
                     ? __longlong_as_double((long long)ld_relaxed_agent(
                           a.partial + threadIdx.x * kPolicySums + k))
                     : 0.0;
    group_sums(sum, s_tmp);
    if (threadIdx.x == 0) {
        const double over = sum[1] != 0.0 ? 1.0 / sum[1] : 0.0;
        a.result->loss = (float)(a.scale * sum[0]);
        a.result->weight = (float)sum[1];
        a.result->kl = (float)(sum[2] * over);
        a.result->clipped = (float)(sum[3] * over);
        a.result->entropy = (float)(sum[4] * over);
        __hip_atomic_store(a.done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

}  // namespace

hipError_t launch_policy_loss(const PolicyArgs &a, hipStream_t stream) {
    const uint64_t groups = (a.n + kThreads - 1) / kThreads;
    const uint32_t grid = groups < kPolicyGrid ? (groups ? (uint32_t)groups : 1) : kPolicyGrid;
    return launch_one(policy_loss_kernel, grid, kThreads, a, 0, stream);
}

}  // namespace bf16d
