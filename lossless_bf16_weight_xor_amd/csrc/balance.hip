// balance.hip -- the balance loss of a router, the tokens each expert was
// chosen for, and the gradient of the router's logits.
//
// The gradient of balance = E sum f_e P_e needs every f_e, so it is a pass of
// its own: the first one sums p and counts, the second one computes p again.
// A lane holds 16 bytes of neighbouring experts (a row of more than 64 such
// pieces: two or four), a row the next power of two of lanes, a wave 64 / lanes rows.
// So softmax sums are a few lane steps, and a lane's sums of p over its rows stay
// in registers.  Lanes and workgroups add up in integers (counts, and sums of p
// in steps of 2^-36), so the order of their atomics does not matter.
#include "loss.hpp"

namespace bf16d {
namespace {

constexpr float kLog2E = 1.44269504088896340736f;
constexpr double kFixed = 68719476736.0;   // 2^36: sums of p stay below 2^24 rows * 2^36

// what the accumulators after the 2 * experts counts and sums are
enum { kSumTokens = 0, kSumBadIds = 1, kSumBadRows = 2, kSumWords = 3 };

// Which experts a lane holds: kVec pieces of kPer neighbours, piece v from
// start[v] on, of which the ones from lo[v] to hi - 1 count.  (The last piece of
// a row ends where the row ends, so that all pieces are whole loads; what it shares
// with the one before counts there.)
template <bool kF32, int kVec>
struct Pieces {
    static constexpr uint32_t kPer = kF32 ? 4 : 8, kSize = kF32 ? 4 : 2;
    uint32_t lanes, sub, held;   // of a row, this lane among them, rows of a wave
    uint32_t experts, hi;
    uint32_t start[kVec], lo[kVec];

    __device__ __forceinline__ explicit Pieces(uint32_t n) : experts(n) {
        const uint32_t pieces = (n + kPer - 1) / kPer;
        lanes = pieces >= 64 ? 64u : pieces > 1 ? 1u << (32 - __clz(pieces - 1)) : 1u;
        sub = threadIdx.x & (lanes - 1);
        held = 64 / lanes;
        hi = n < kPer ? n : kPer;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const uint32_t first = (sub + 64 * v) * kPer;
            const uint32_t last = n < kPer ? 0 : n - kPer;
            start[v] = first < last ? first : last;
            lo[v] = first < n ? first - start[v] : kPer;
        }
    }
    __device__ __forceinline__ bool holds(int v, uint32_t k) const { return k >= lo[v] && k < hi; }
};

// A row's pieces as they are in memory, at any alignment of their type.
template <bool kF32, int kVec>
__device__ __forceinline__ void load_row(word4 (&w)[kVec], const Pieces<kF32, kVec> &P,
                                         const uint8_t *row) {
    constexpr uint32_t kPer = Pieces<kF32, kVec>::kPer, kSize = Pieces<kF32, kVec>::kSize;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
        const uint8_t *p = row + P.start[v] * kSize;
        if (P.experts >= kPer) {
            if (P.lo[v] < kPer) w[v] = *(const word4_any *)p;
            continue;
        }
#pragma unroll
        for (uint32_t k = 0; k < kPer; ++k) {   // one lane holds the whole row
            if (k >= P.hi) continue;
            if constexpr (kF32) w[v][k] = ((const uint32_t *)p)[k];
            else w[v][k >> 1] = (k & 1 ? w[v][k >> 1] & 0xFFFFu : 0u) |
                                (uint32_t)((const uint16_t *)p)[k] << (16 * (k & 1));
        }
    }
}

// e^(x - m) of the lane's experts, their sum over the row (0: nothing but
// -infinity, or a row that does not count), and m.
template <bool kF32, int kVec>
struct RowSoftmax {
    static constexpr int kPer = kF32 ? 4 : 8;
    float e[kVec][kPer];
    float sum, m;

    __device__ __forceinline__ RowSoftmax(const Pieces<kF32, kVec> &P, const word4 (&w)[kVec],
                                          bool live) {
        m = -INFINITY;
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                e[v][k] = live && k < (int)P.hi && P.lo[v] < P.kPer ? element<kF32>(w[v], k)
                                                                   : -INFINITY;
                m = fmaxf(m, e[v][k]);
            }
        m = lanes_reduce<Max>(m, P.lanes);
        if (m == -INFINITY) m = 0.0f;
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                e[v][k] = __builtin_amdgcn_exp2f((e[v][k] - m) * kLog2E);
                s += P.holds(v, k) ? e[v][k] : 0.0f;
            }
        sum = lanes_reduce<Add>(s, P.lanes);
    }
};

// What the rows of a wave's turn hold.  Whatever a row that is not there or does
// not count holds is not looked at.
template <bool kF32, int kVec>
struct Turn {
    word4 w[kVec];
    bool there, live;

    __device__ __forceinline__ void load(const Pieces<kF32, kVec> &P, const void *logits,
                                         uint64_t stride, const uint8_t *mask, uint32_t row,
                                         uint32_t rows) {
        there = row < rows;
        live = false;
        if (!there) return;
        live = !mask || mask[row];
        load_row(w, P, (const uint8_t *)logits + row * stride * P.kSize);
    }
};

template <bool kF32, int kVec>
__global__ __launch_bounds__(kBalanceThreads) void balance_kernel(BalanceArgs a) {
    constexpr int kPer = kF32 ? 4 : 8;
    constexpr uint32_t kGroupWaves = kBalanceThreads / 64;
    constexpr uint32_t kMost = 64 * kVec * kPer;
    __shared__ uint32_t s_count[kMost];
    __shared__ unsigned long long s_p[kMost];
    __shared__ double s_sum[kGroupWaves];
    __shared__ uint32_t s_tokens, s_bad_ids, s_bad_rows;
    for (uint32_t e = threadIdx.x; e < a.experts; e += kBalanceThreads) {
        s_count[e] = 0;
        s_p[e] = 0;
    }
    if (threadIdx.x == 0) s_tokens = s_bad_ids = s_bad_rows = 0;
    __syncthreads();
    const Pieces<kF32, kVec> P(a.experts);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float p[kVec][kPer] = {};
    double squares = 0.0;
    uint32_t tokens = 0;
    bool bad_id = false, bad_row = false;
    const uint32_t step = gridDim.x * kGroupWaves * P.held;
    uint32_t row = (blockIdx.x * kGroupWaves + wave) * P.held + lane / P.lanes;
    const uint32_t turns = row - lane / P.lanes < a.rows
                               ? (a.rows - (row - lane / P.lanes) + step - 1) / step
                               : 0;   // the same in the whole wave
    auto id_at = [&](uint32_t r, uint32_t j) {
        return load_id((const uint8_t *)a.chosen +
                           (r * a.chosen_stride + j) * (a.chosen_i32 ? 4 : 8),
                       a.chosen_i32);
    };
    Turn<kF32, kVec> next;
    int64_t next_id = -1;
    auto fetch = [&](uint32_t r) {
        next.load(P, a.logits, a.logits_stride, a.mask, r, a.rows);
        next_id = r < a.rows && P.sub < a.choices ? id_at(r, P.sub) : -1;
    };
    auto count = [&](int64_t id) {
        if (id >= (int64_t)a.experts) bad_id = true;
        else if (id >= 0) atomicAdd(&s_count[id], 1u);
    };
    if (turns) fetch(row);
    for (uint32_t t = 0; t < turns; ++t, row += step) {
        const Turn<kF32, kVec> now = next;
        const int64_t id = next_id;
        if (t + 1 < turns) fetch(row + step);
        const RowSoftmax<kF32, kVec> r(P, now.w, now.live);
        if (r.sum != 0.0f) {   // else nothing, or nothing that counts
            const float inv = 1.0f / r.sum;
#pragma unroll
            for (int v = 0; v < kVec; ++v)
#pragma unroll
                for (int k = 0; k < kPer; ++k) p[v][k] += r.e[v][k] * inv;
            const float lse = r.m + logf(r.sum);
            if (P.sub == 0) squares += (double)lse * lse;
            bad_row |= !(r.sum < INFINITY);
        }
        if (!now.live) continue;
        tokens += P.sub == 0;
        count(id);
        for (uint32_t j = P.sub + P.lanes; j < a.choices; j += P.lanes) count(id_at(row, j));
    }
    if (tokens) atomicAdd(&s_tokens, tokens);
    if (bad_id) s_bad_ids = 1;
    if (bad_row) s_bad_rows = 1;
#pragma unroll
    for (int v = 0; v < kVec; ++v)
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (P.holds(v, k) && p[v][k] > 0.0f && p[v][k] < INFINITY)
                atomicAdd(&s_p[P.start[v] + k],
                          (unsigned long long)__double2ll_rn((double)p[v][k] * kFixed));
    squares = lanes_reduce<Add>(squares);
    if (lane == 0) s_sum[wave] = squares;
    __syncthreads();
    uint64_t dep = 0;
    auto add = [&](uint32_t at, uint64_t v) {
        if (v)
            dep ^= __hip_atomic_fetch_add(a.sums + at, v, __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT);
    };
    for (uint32_t e = threadIdx.x; e < a.experts; e += kBalanceThreads) {
        add(e, s_count[e]);
        add(a.experts + e, s_p[e]);
    }
    if (threadIdx.x == 0) {
        add(2 * a.experts + kSumTokens, s_tokens);
        add(2 * a.experts + kSumBadIds, s_bad_ids);
        add(2 * a.experts + kSumBadRows, s_bad_rows);
        double all = 0.0;
#pragma unroll
        for (uint32_t w = 0; w < kGroupWaves; ++w) all += s_sum[w];
        dep ^= __hip_atomic_exchange(a.partial + blockIdx.x, (uint64_t)__double_as_longlong(all),
                                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!last_of(a.done, gridDim.x, dep)) return;

    // the accumulators are read and cleared
    auto take = [&](uint32_t at) {
        return __hip_atomic_exchange(a.sums + at, (uint64_t)0, __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_AGENT);
    };
    double choices = 0.0, product = 0.0, z = 0.0;
    for (uint32_t e = threadIdx.x; e < a.experts; e += kBalanceThreads) {
        const uint64_t c = take(e);
        a.counts[e] = (int64_t)c;
        choices += (double)c;
        product += (double)c * ((double)take(a.experts + e) / kFixed);
    }
    static_assert(kBalanceGrid <= kBalanceThreads, "a thread takes one workgroup's sum");
    if (threadIdx.x < gridDim.x)
        z = __longlong_as_double((long long)ld_relaxed_agent(a.partial + threadIdx.x));
    choices = group_total(choices, s_sum);
    product = group_total(product, s_sum);
    z = group_total(z, s_sum);
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

// A row's pieces from its values.  Two lanes that share experts at a row's end store
// the same values there.
template <bool kF32, int kVec, int kPer>
__device__ __forceinline__ void store_row(const float (&g)[kVec][kPer],
                                          const Pieces<kF32, kVec> &P, uint8_t *row) {
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
        uint8_t *p = row + P.start[v] * P.kSize;
        word4 w;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (kF32) w[k] = __float_as_uint(g[v][k]);
            else w[k] = pack_bf16(g[v][2 * k], g[v][2 * k + 1]);
        }
        if (P.experts >= P.kPer) {
            if (P.lo[v] < P.kPer) *(word4_any *)p = w;
            continue;
        }
#pragma unroll
        for (uint32_t k = 0; k < P.kPer; ++k) {
            if (k >= P.hi) continue;
            if constexpr (kF32) ((uint32_t *)p)[k] = w[k];
            else ((uint16_t *)p)[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
        }
    }
}

template <bool kF32, int kVec>
__global__ __launch_bounds__(kThreads) void balance_grad_kernel(BalanceGradArgs a) {
    constexpr int kPer = kF32 ? 4 : 8;
    __shared__ double s_tmp[kWaves];
    const Pieces<kF32, kVec> P(a.experts);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t step = gridDim.x * kWaves * P.held;
    uint32_t row = (blockIdx.x * kWaves + wave) * P.held + lane / P.lanes;
    const uint32_t turns = row - lane / P.lanes < a.rows
                               ? (a.rows - (row - lane / P.lanes) + step - 1) / step
                               : 0;
    Turn<kF32, kVec> next;
    if (turns) next.load(P, a.logits, a.logits_stride, a.mask, row, a.rows);
    double choices = 0.0;
    for (uint32_t e = threadIdx.x; e < a.experts; e += kThreads) choices += (double)a.counts[e];
    choices = group_total(choices, s_tmp);
    const double n = *a.tokens > 1 ? (double)*a.tokens : 1.0;
    const float by_share = (float)(a.scale * a.balance_coef * a.experts / n);
    const float by_lse = (float)(2.0 * a.scale * a.z_coef / n);
    const float spoilt = a.result && a.result->loss != a.result->loss ? NAN : 0.0f;
    float share[kVec][kPer];
#pragma unroll
    for (int v = 0; v < kVec; ++v)
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            share[v][k] = P.lo[v] < P.kPer && k < (int)P.hi && choices > 0.0
                              ? (float)((double)a.counts[P.start[v] + k] / choices)
                              : 0.0f;
    for (uint32_t t = 0; t < turns; ++t, row += step) {
        const Turn<kF32, kVec> now = next;
        if (t + 1 < turns) next.load(P, a.logits, a.logits_stride, a.mask, row + step, a.rows);
        const RowSoftmax<kF32, kVec> r(P, now.w, now.live);
        const float inv = r.sum != 0.0f ? 1.0f / r.sum : 0.0f;
        float inner = 0.0f;
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                inner += P.holds(v, k) ? r.e[v][k] * share[v][k] : 0.0f;
        inner = lanes_reduce<Add>(inner, P.lanes) * inv;
        const float same = (r.sum != 0.0f ? by_lse * (r.m + logf(r.sum)) : 0.0f) - by_share * inner;
        if (!now.there) continue;
        float g[kVec][kPer];
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                g[v][k] = now.live ? r.e[v][k] * inv * (by_share * share[v][k] + same) + spoilt
                                   : 0.0f;
        store_row(g, P, (uint8_t *)a.out + row * a.out_stride * P.kSize);
    }
}

// workgroups of `waves` waves for the rows: `most`, or a turn each
uint32_t grid_of(uint32_t rows, uint32_t experts, bool f32, uint32_t waves, uint32_t most) {
    const uint32_t per = f32 ? 4 : 8, pieces = (experts + per - 1) / per;
    uint32_t lanes = 1;
    while (lanes < 64 && lanes < pieces) lanes *= 2;
    const uint32_t turn = waves * (64 / lanes);
    const uint32_t groups = (rows + turn - 1) / turn;
    return groups < most ? (groups ? groups : 1) : most;
}

}  // namespace

hipError_t launch_balance(const BalanceArgs &a, bool f32, hipStream_t stream) {
    const uint32_t grid =
        grid_of(a.rows, a.experts, f32, kBalanceThreads / 64, kBalanceGrid);
    auto *kernel = f32 ? (a.experts <= 256   ? balance_kernel<true, 1>
                          : a.experts <= 512 ? balance_kernel<true, 2>
                                             : balance_kernel<true, 4>)
                       : (a.experts <= 512 ? balance_kernel<false, 1> : balance_kernel<false, 2>);
    return launch_one(kernel, grid, kBalanceThreads, a, 0, stream);
}

hipError_t launch_balance_backward(const BalanceGradArgs &a, bool f32, hipStream_t stream) {
    const uint32_t grid = grid_of(a.rows, a.experts, f32, kWaves, kBalanceGradGrid);
    auto *kernel =
        f32 ? (a.experts <= 256   ? balance_grad_kernel<true, 1>
               : a.experts <= 512 ? balance_grad_kernel<true, 2>
                                  : balance_grad_kernel<true, 4>)
            : (a.experts <= 512 ? balance_grad_kernel<false, 1> : balance_grad_kernel<false, 2>);
    return launch_one(kernel, grid, kThreads, a, 0, stream);
}

}  // namespace bf16d
