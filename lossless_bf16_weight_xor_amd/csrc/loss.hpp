// loss.hpp -- shared definitions of the loss kernels and the host code that
// launches them (include/bf16delta_loss.h).
#pragma once

#include <math.h>

#include "bf16delta_loss.h"
#include "internal.hpp"
#include "step.hpp"

namespace bf16d {

// ---- log probabilities --------------------------------------------------------
// A row is read in turns, four 16-byte vectors a thread, by one workgroup where
// there are at least kLogprobGroups rows (one for each CU), else cut into parts of
// whole turns so that there are as many workgroups.  More of them gain less than
// the joining costs: 256 rows of 131072 bf16 logits 13.4 us, cut for 512 and
// 1024 workgroups 15.1 and 16.1; one row 4.6, 4.6 and 4.5.
constexpr uint32_t kTurnVectors = 4;   // of a thread
constexpr uint32_t kLogprobGroups = 256;
// Workgroups of 16 waves hold a row of up to 32768 bf16 or 16384 fp32 logits in one
// turn and need no join: 96 rows of 32000 bf16 5.2 us, in parts 6.2; 8000 fp32 4.3
// and 5.1.  A row of more than that is faster in parts (one of 50021 bf16 5.5 and
// 6.3), except with alternatives, which are found by such workgroups.
constexpr uint32_t kLogprobWide = 1024;        // threads
constexpr uint32_t vector_elems(uint32_t dtype) { return dtype == BF16D_LOGITS_F32 ? 4 : 8; }
// The most turns of a row for workgroups of `threads`; aligned: all rows start at
// 16-byte addresses.
inline uint32_t turns_of(uint32_t vocab, uint32_t dtype, bool aligned, uint32_t threads) {
    const uint32_t per = kTurnVectors * threads * vector_elems(dtype);
    return (vocab + (aligned ? 0 : vector_elems(dtype) - 1) + per - 1) / per;
}
// Logits of up to this many bytes are left in the last-level cache for the
// backward pass; more are read with non-temporal loads (fp32, 16384 x 32000: 305
// us, plain 343).  Forward and backward of bf16 logits with and without: 66 MB 38.9
// and 42.1 us, 131 MB 72.5 and 75.1; of 262 MB in fp32 131.6 and 127.3, and the
// forward pass alone 47.8 and 42.2.
constexpr uint64_t kLogprobKept = 128u << 20;
// Turns whose sums a thread adds up in 32 bits: rows of up to 262144 bf16 or 131072 fp32
// logits, of 2^20 and 2^19 with alternatives.  Sums in 64 bits of every turn took the registers of
// the eighth wave of a SIMD (2039 rows of 100003 bf16 with entropy 72.5 us, 79.2).
constexpr uint32_t kLogprobChain = 32;

// Rows of a call, as the device sees them.
struct RowSet {
    void *data;
    uint64_t outer_stride, inner_stride;
};

struct LogprobArgs {
    RowSet logits, tokens;
    uint32_t rows, inner, vocab, token_i32, top;
    uint32_t parts, part_turns;   // workgroups of a row, turns of each
    float scale;                  // log2(e) / temperature
    float inv_t;
    float *logp, *entropy;
    bf16d_row_stats *stats;
    int64_t *top_ids;
    float *top_logp;
    uint64_t *partial;   // (2 + top) words of each part of each row
    uint32_t *done;      // of each row
};
// wide: workgroups of kLogprobWide threads (with alternatives: always); keep: the
// logits may stay in the caches (with wide: always)
hipError_t launch_logprob(const LogprobArgs &a, bool f32, bool wide, bool keep,
                          hipStream_t stream);

struct LogprobGradArgs {
    RowSet logits, tokens, out;
    uint32_t rows, inner, vocab, token_i32;
    uint32_t parts, part_turns;
    const bf16d_row_stats *stats;
    const float *grad_logp, *grad_entropy;
};
hipError_t launch_logprob_backward(const LogprobGradArgs &a, bool f32, hipStream_t stream);

// ---- policy loss ----------------------------------------------------------------
// A workgroup of 16 waves for each CU at most: 1e6 tokens 10.2 us, with 4 waves 14.1.
constexpr uint32_t kPolicyGrid = 256;
constexpr uint32_t kPolicyThreads = 1024;
constexpr uint32_t kPolicyAlone = 2;   // turns that one workgroup takes sooner than joining sums
constexpr uint32_t kPolicySums = 5;   // loss, weight, kl, clipped, entropy
struct PolicyArgs {
    const float *logp, *old, *advantages, *weights, *ref, *entropy;
    float *grad_logp, *grad_entropy;
    uint64_t n;
    double low, high;              // clip range of the ratio
    double log_low, log_high;      // and of its logarithm
    double kl_coef, entropy_coef, scale;
    bf16d_policy_result *result;
    uint64_t *partial;             // kPolicySums words a workgroup
    uint32_t *done;                // kDoneWords
};
hipError_t launch_policy_loss(const PolicyArgs &a, hipStream_t stream);

// ---- balance loss ------------------------------------------------------------------
// A workgroup of 16 waves for each CU: as many rows in flight as with small ones,
// and fewer that add to the shared sums at the end (with 512 workgroups 65536 rows of
// 64 fp32 experts took 16.6 us instead of 11.7).
constexpr uint32_t kBalanceGrid = 256;
constexpr uint32_t kBalanceThreads = 1024;
constexpr uint32_t kBalanceAlone = 4;        // turns that one takes sooner than joining sums
// of the sums that workgroups add to: 16384 rows of 64 fp32 experts 9.7 us, with one
// copy 13.8
constexpr uint32_t kBalanceCopies = 8;
// Turns of a wave whose p a lane adds up in 32 bits before they go on as integers: in one
// chain 2^24 rows of 1024 equal logits drift by 5e-5.  Kernels of their own do so (in all
// of them 65536 rows of 64 fp32 experts took 12.25 us instead of 11.75); 2^21 rows of 1024 bf16
// experts, 512 turns, take 907 us, in one chain 893.
constexpr uint32_t kBalanceChain = 64;
// of four waves, where a lane holds up to 8 experts (262144 rows of 64 bf16 experts 15.5 us,
// with 1024 17.2), else half of them (262144 of 1024: 209 us, with 2048 241)
constexpr uint32_t kBalanceGradGrid = 2048;
struct BalanceArgs {
    const void *logits, *chosen;
    const uint8_t *mask;
    uint64_t logits_stride, chosen_stride;
    uint32_t rows, experts, choices, chosen_i32, lane_bits;
    double balance_coef, z_coef;
    int64_t *counts;
    bf16d_balance_result *result;
    uint64_t *sums;      // kBalanceCopies times 2 * experts + 3, zero between calls
    uint64_t *partial;   // a workgroup's sum of squares
    uint32_t *done;      // kDoneWords
};
hipError_t launch_balance(BalanceArgs a, bool f32, hipStream_t stream);

struct BalanceGradArgs {
    const void *logits;
    void *out;
    const uint8_t *mask;
    uint64_t logits_stride, out_stride;
    uint32_t rows, experts, lane_bits;
    double balance_coef, z_coef, scale;
    const int64_t *counts, *tokens;
    const bf16d_balance_result *result;
};
hipError_t launch_balance_backward(BalanceGradArgs a, bool f32, hipStream_t stream);

// ---- device helpers -----------------------------------------------------------------
typedef uint32_t word4 __attribute__((ext_vector_type(4)));
// 16 bytes at an address of a 2- or 4-byte type's alignment
typedef word4 word4_any __attribute__((aligned(2)));

// a / b of uniform numbers, as one: there is no scalar division, and the quotient would
// stay in vector registers, with all that is computed from it
__device__ __forceinline__ uint32_t scalar_div(uint32_t a, uint32_t b) {
    return b == 1 ? a : first_lane(a / b);
}
__device__ __forceinline__ const uint8_t *row_ptr(const RowSet &s, uint32_t row, uint32_t inner,
                                                  uint32_t size) {
    const uint32_t o = scalar_div(row, inner), i = row - o * inner;
    return static_cast<const uint8_t *>(s.data) +
           (o * s.outer_stride + i * s.inner_stride) * size;
}
__device__ __forceinline__ int64_t load_id(const uint8_t *p, uint32_t i32) {
    return i32 ? (int64_t)*(const int32_t *)p : *(const int64_t *)p;
}

// Whether this is the last of `count` workgroups that call it on one counter
// (as last_workgroup, whose count is the grid's).
__device__ __forceinline__ bool last_of(uint32_t *done, uint32_t count, uint64_t dep) {
    __shared__ bool s_last;
    asm volatile("" ::"v"(dep) : "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        s_last = __hip_atomic_fetch_add(done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                 count - 1;
    __syncthreads();
    return s_last;
}

// The same for all workgroups of a launch, in two levels: additions to one address
// take some 10 to 20 ns each (1e6 tokens of the policy loss, 256 workgroups: 10.2 us, in
// one level 11.7).  done: kDoneWords counters.
constexpr uint32_t kDoneGroups = 16, kDoneStride = 32;   // words: a line each
constexpr uint32_t kDoneWords = (kDoneGroups + 1) * kDoneStride;
__device__ __forceinline__ bool last_of_launch(uint32_t *done, uint64_t dep) {
    __shared__ bool s_last;
    asm volatile("" ::"v"(dep) : "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        auto arrive = [&](uint32_t *at, uint32_t count) {
            const bool last = __hip_atomic_fetch_add(at, 1u, __ATOMIC_RELAXED,
                                                     __HIP_MEMORY_SCOPE_AGENT) == count - 1;
            if (last) __hip_atomic_store(at, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            return last;
        };
        uint32_t *all = done + kDoneGroups * kDoneStride;
        const uint32_t group = blockIdx.x % kDoneGroups;
        if (gridDim.x <= kDoneGroups)
            s_last = arrive(all, gridDim.x);
        else
            s_last = arrive(done + group * kDoneStride,
                            (gridDim.x - group + kDoneGroups - 1) / kDoneGroups) &&
                     arrive(all, kDoneGroups);
    }
    __syncthreads();
    return s_last;
}

// ---- reductions over the lanes of a wave ------------------------------------------
// v combined with the value of another lane, step by step, over groups of `lanes`
// (a power of two, the same in the whole wave) neighbouring lanes, all of which
// get the result.  DPP moves and lane swaps take a few cycles where a shuffle
// through LDS takes a hundred.  The order is fixed.
struct Add {
    template <typename T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
template <int kCtrl>
__device__ __forceinline__ float dpp_value(float v) {
    return __uint_as_float(dpp_src<kCtrl>(__float_as_uint(v)));
}
template <int kCtrl>
__device__ __forceinline__ double dpp_value(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)((uint64_t)dpp_src<kCtrl>((uint32_t)(b >> 32)) << 32 |
                                            dpp_src<kCtrl>((uint32_t)b)));
}
// (v of the even 16- or 32-lane half in both halves, v of the odd one in both)
template <int kHalf>
__device__ __forceinline__ void both_halves(float v, float &even, float &odd) {
    const uint32_t b = __float_as_uint(v);
    auto r = kHalf == 16 ? __builtin_amdgcn_permlane16_swap(b, b, false, false)
                         : __builtin_amdgcn_permlane32_swap(b, b, false, false);
    even = __uint_as_float(r[0]);
    odd = __uint_as_float(r[1]);
}
template <int kHalf>
__device__ __forceinline__ void both_halves(double v, double &even, double &odd) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t l = (uint32_t)b, h = (uint32_t)(b >> 32);
    auto lo = kHalf == 16 ? __builtin_amdgcn_permlane16_swap(l, l, false, false)
                          : __builtin_amdgcn_permlane32_swap(l, l, false, false);
    auto hi = kHalf == 16 ? __builtin_amdgcn_permlane16_swap(h, h, false, false)
                          : __builtin_amdgcn_permlane32_swap(h, h, false, false);
    even = __longlong_as_double((long long)((uint64_t)hi[0] << 32 | lo[0]));
    odd = __longlong_as_double((long long)((uint64_t)hi[1] << 32 | lo[1]));
}
// v of the lane whose number differs in the bits of kMask
template <int kMask>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
    constexpr int kLow = kMask & 15;
    static_assert(kLow == 0 || kLow == 1 || kLow == 2 || kLow == 3 || kLow == 4 || kLow == 7 ||
                      kLow == 8 || kLow == 15,
                  "one or two moves within a row of 16 lanes");
    if constexpr (kLow == 1) v = dpp_src<0xB1>(v);
    if constexpr (kLow == 2) v = dpp_src<0x4E>(v);
    if constexpr (kLow == 3) v = dpp_src<0x1B>(v);                   // quad_perm 3 2 1 0
    if constexpr (kLow == 4) v = dpp_src<0x1B>(dpp_src<0x141>(v));   // 7, then 3
    if constexpr (kLow == 7) v = dpp_src<0x141>(v);
    if constexpr (kLow == 8) v = dpp_src<0x128>(v);                  // row_ror:8
    if constexpr (kLow == 15) v = dpp_src<0x140>(v);
    if constexpr ((kMask & 16) != 0) {
        auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = threadIdx.x & 16 ? r[0] : r[1];
    }
    if constexpr ((kMask & 32) != 0) {
        auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = threadIdx.x & 32 ? r[0] : r[1];
    }
    return v;
}

template <typename Op, typename T>
__device__ __forceinline__ T lanes_reduce(T v, uint32_t lanes = 64) {
    const Op op;
    T even, odd;
    if (lanes > 1) v = op(v, dpp_value<0xB1>(v));     // quad_perm 1 0 3 2
    if (lanes > 2) v = op(v, dpp_value<0x4E>(v));     // quad_perm 2 3 0 1
    if (lanes > 4) v = op(v, dpp_value<0x141>(v));    // row_half_mirror
    if (lanes > 8) v = op(v, dpp_value<0x140>(v));    // row_mirror
    if (lanes > 16) {
        both_halves<16>(v, even, odd);
        v = op(even, odd);
    }
    if (lanes > 32) {
        both_halves<32>(v, even, odd);
        v = op(even, odd);
    }
    return v;
}

// the sum over a workgroup of kCount waves, in a fixed order; every thread gets it
template <uint32_t kCount>
__device__ __forceinline__ double group_total(double v, double (&s_tmp)[kCount]) {
    v = lanes_reduce<Add>(v);
    if ((threadIdx.x & 63) == 0) s_tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (uint32_t w = 0; w < kCount; ++w) t += s_tmp[w];
    __syncthreads();
    return t;
}

// Element k (known at compile time) of a vector of logits.
template <bool kF32>
__device__ __forceinline__ float element(const word4 &w, int k) {
    if constexpr (kF32) return __uint_as_float(w[k]);
    else return __uint_as_float(k & 1 ? w[k >> 1] & 0xFFFF0000u : w[k >> 1] << 16);
}

// two floats to bf16, nearest even
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef float pair __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16_pair __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(pair{lo, hi}, bf16_pair));
}

}  // namespace bf16d
