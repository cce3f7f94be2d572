// policy.hip -- the clipped policy loss over the tokens of a batch, with its
// gradients by the log probabilities and entropies, in one launch.
//
// A token is 12 to 24 bytes read, 8 written (4 for a caller who leaves grad_entropy out)
// and two exponentials.  All of it is in 64 bits: near r = 1, where most tokens are, e^u - 1 - u and the
// distance to the clip range are differences of nearly equal numbers, and the
// arithmetic costs next to nothing beside the launch (4096 tokens 6.3 us, with the library's
// expm1 6.4, with its exp as well 6.5).  The clip range is compared as logarithms, logp - old
// being exact in 64 bits.  4096 tokens take 6.4 us, of which launch and joining
// the workgroups' sums are 5; 1e6 tokens 10.2, with reference and entropy 11.7 (2.4
// TB/s of what they read and write).
#include "loss.hpp"

namespace bf16d {
namespace {

// e^u and e^u - 1, each with its own digits: near u = 0 they are lost to one of 1 + (e^u - 1),
// far below it to the other.  u = k ln 2 + f with |f| at most ln 2 / 2 (k times the first part of
// ln 2 is exact), and the series of e^f without its 1, to f^13 / 13!: what is left out is
// below 2^-56 of f.
struct Exponential {
    double r, less;
    __device__ __forceinline__ explicit Exponential(double u) {
        u = u < -800.0 ? -800.0 : u > 800.0 ? 800.0 : u;   // 0 and infinity
        const double k = u == u ? rint(u * 1.4426950408889634074) : 0.0;   // not of NaN
        const double f = fma(k, -1.9082149292705877e-10, fma(k, -0.69314718036912382, u));
        double p = 1.0 / 6227020800.0;
        const double of[] = {479001600.0, 39916800.0, 3628800.0, 362880.0, 40320.0, 5040.0,
                             720.0, 120.0, 24.0, 6.0, 2.0};
#pragma unroll
        for (int j = 0; j < 11; ++j) p = fma(p, f, 1.0 / of[j]);
        const double q = fma(f * f, p, f);
        r = ldexp(1.0 + q, (int)k);
        less = k == 0.0 ? q : r - 1.0;
    }
};

// e^u - 1 - u, at least 0; v: e^u - 1
__device__ __forceinline__ double excess(double v, double u) {
    return v == INFINITY ? (double)INFINITY : v - u;
}

constexpr uint32_t kPolicyWaves = kPolicyThreads / 64;

// the sums over the workgroup, in a fixed order, in the first wave's lanes
__device__ __forceinline__ void group_sums(double (&v)[kPolicySums],
                                           double (*s_tmp)[kPolicyWaves]) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (uint32_t k = 0; k < kPolicySums; ++k) {
        v[k] = lanes_reduce<Add>(v[k]);
        if (lane == 0) s_tmp[k][wave] = v[k];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (uint32_t k = 0; k < kPolicySums; ++k)
            v[k] = lanes_reduce<Add>(s_tmp[k][lane & (kPolicyWaves - 1)], kPolicyWaves);
    }
    __syncthreads();
}

// A token's numbers, loaded ahead of their use.
struct Token {
    float w, lp, old, adv, ref, entropy;
};
__device__ __forceinline__ Token load_token(const PolicyArgs &a, uint64_t i) {
    Token t = {1.0f, a.logp[i], a.old[i], a.advantages[i], 0.0f, 0.0f};
    if (a.weights) t.w = a.weights[i];
    if (a.kl_coef != 0.0) t.ref = a.ref[i];
    if (a.entropy) t.entropy = a.entropy[i];
    return t;
}

// Adds the token to the sums and stores its gradients.
__device__ __forceinline__ void add_token(double (&sum)[kPolicySums], const PolicyArgs &a,
                                          const Token &t, uint64_t i) {
    const double w = t.w;
    double slope = 0.0;
    if (w != 0.0) {
        const double lp = t.lp, adv = t.adv;
        const double u = lp - t.old;
        const Exponential e(u);
        const double v = e.less;
        const bool cut = (adv > 0.0 && u > a.log_high) || (adv < 0.0 && u < a.log_low);
        double each = 0.0;
        if (cut) {
            each = -(adv > 0.0 ? a.high : a.low) * adv;
        } else if (adv != 0.0) {
            each = slope = -e.r * adv;
        }
        if (a.kl_coef != 0.0) {
            const double away = t.ref - lp, grow = Exponential(away).less;
            each += a.kl_coef * excess(grow, away);
            slope -= a.kl_coef * grow;
        }
        if (a.entropy) {
            const double h = t.entropy;
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

__global__ __launch_bounds__(kPolicyThreads) void policy_loss_kernel(PolicyArgs a) {
    __shared__ double s_tmp[kPolicySums][kPolicyWaves];
    double sum[kPolicySums] = {0.0, 0.0, 0.0, 0.0, 0.0};
    const uint64_t step = (uint64_t)gridDim.x * kPolicyThreads;
    uint64_t i = (uint64_t)blockIdx.x * kPolicyThreads + threadIdx.x;
    Token next = {};
    if (i < a.n) next = load_token(a, i);
    while (i < a.n) {
        const Token t = next;
        const uint64_t at = i;
        i += step;
        if (i < a.n) next = load_token(a, i);
        add_token(sum, a, t, at);
    }
    group_sums(sum, s_tmp);
    if (gridDim.x > 1) {
        // handed over by returning device-scope atomics, as last_of_launch asks
        uint64_t dep = 0;
        if (threadIdx.x < kPolicySums) {
            double mine = sum[0];
#pragma unroll
            for (uint32_t k = 1; k < kPolicySums; ++k) mine = threadIdx.x == k ? sum[k] : mine;
            dep = __hip_atomic_exchange(a.partial + blockIdx.x * kPolicySums + threadIdx.x,
                                        (uint64_t)__double_as_longlong(mine), __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
        }
        if (!last_of_launch(a.done, dep)) return;
        static_assert(kPolicyGrid <= kPolicyThreads, "a thread takes one workgroup's sums");
#pragma unroll
        for (uint32_t k = 0; k < kPolicySums; ++k)
            sum[k] = threadIdx.x < gridDim.x
                         ? __longlong_as_double((long long)ld_relaxed_agent(
                               a.partial + threadIdx.x * kPolicySums + k))
                         : 0.0;
        group_sums(sum, s_tmp);
    }
    if (threadIdx.x == 0) {
        const double over = sum[1] != 0.0 ? 1.0 / sum[1] : 0.0;
        a.result->loss = (float)(a.scale * sum[0]);
        a.result->weight = (float)sum[1];
        a.result->kl = (float)(sum[2] * over);
        a.result->clipped = (float)(sum[3] * over);
        a.result->entropy = (float)(sum[4] * over);
    }
}

}  // namespace

hipError_t launch_policy_loss(const PolicyArgs &a, hipStream_t stream) {
    const uint64_t turns = (a.n + kPolicyThreads - 1) / kPolicyThreads;
    const uint32_t grid =
        turns <= kPolicyAlone ? 1 : turns < kPolicyGrid ? (uint32_t)turns : kPolicyGrid;
    return launch_one(policy_loss_kernel, grid, kPolicyThreads, a, 0, stream);
}

}  // namespace bf16d
