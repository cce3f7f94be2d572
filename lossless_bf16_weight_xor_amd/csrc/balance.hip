// balance.hip -- the balance loss of a router, the tokens each expert was
// chosen for, and the gradient of the router's logits.
//
// The gradient of balance = E sum f_e P_e needs every f_e, so it is a pass of
// its own: the first one sums p and counts, the second one computes p again.
// A row is cut into pieces of 16 bytes of neighbouring experts.  A lane holds one to
// four of them, a row a power of two of lanes, a wave 64 / lanes rows.  So softmax sums
// are a few lane steps for several rows at once, and a lane's sums of p over its rows
// stay in registers.  Lanes and workgroups add up in integers (counts, and sums of p
// in steps of 2^-36), so the order of their atomics does not matter.
//
// 65536 rows of 64 fp32 experts: 11.7 us forward, of which launch and join are 8, and
// 8.6 backward (3.9 TB/s); 32768 rows of 257 bf16 experts 16.2 and 11.5 (1024 of them:
// 10.4 and 3.8), 131072 of them 29.5 and 29 (2.5 and 4.7 TB/s).
#include "loss.hpp"

namespace bf16d {
namespace {

constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr double kFixed = 68719476736.0;   // 2^36: sums of p stay below 2^24 rows * 2^36

// what the accumulators after the 2 * experts counts and sums are
enum { kSumTokens = 0, kSumBadIds = 1, kSumBadRows = 2, kSumWords = 3 };

// Which experts a lane holds: kVec pieces of kPer neighbours, piece v from
// start[v] on, 2^bits pieces apart.  The last piece of a row ends where the row ends, so
// that all pieces are whole loads; what it shares with the one before has weight 0
// in sums, and both lanes store the same values there.  A row has more than kVec - 1
// pieces for each lane, so only a lane's last one can be that piece, or none.
template <bool kF32, int kVec>
struct Pieces {
    static constexpr int kPer = kF32 ? 4 : 8;
    static constexpr uint32_t kSize = kF32 ? 4 : 2;
    uint32_t bits, lanes, sub, held;   // lanes = 2^bits of a row, this one, rows of a wave
    uint32_t experts;
    uint32_t start[kVec];
    bool any;              // whether the lane holds a last one
    float weight[kPer];    // of that: 1 or 0

    __device__ __forceinline__ Pieces(uint32_t n, uint32_t lane_bits) : bits(lane_bits), experts(n) {
        lanes = 1u << bits;
        sub = threadIdx.x & (lanes - 1);
        held = 64u >> bits;
#pragma unroll
        for (int v = 0; v < kVec - 1; ++v) start[v] = (sub + lanes * v) * kPer;
        const uint32_t first = (sub + lanes * (kVec - 1)) * kPer;
        const uint32_t last = n < kPer ? 0 : n - kPer;
        start[kVec - 1] = first < last ? first : last;
        any = first < n;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            weight[k] =
                start[kVec - 1] + k >= first && start[kVec - 1] + k < n ? 1.0f : 0.0f;
    }
    __device__ __forceinline__ bool holds(int v) const { return v < kVec - 1 || any; }
    // x[v][k] times a factor of its own, summed over the lane's experts in short chains
    template <typename F>
    __device__ __forceinline__ float total(const float (&x)[kVec][kPer], F factor) const {
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            float a = x[v][0] * factor(v, 0), b = x[v][1] * factor(v, 1);
#pragma unroll
            for (int k = 2; k < kPer; k += 2) {
                a = fmaf(x[v][k], factor(v, k), a);
                b = fmaf(x[v][k + 1], factor(v, k + 1), b);
            }
            sum = v ? sum + (a + b) : a + b;
        }
        return sum;
    }
};

// What the rows of a wave's turn hold, as it is in memory (at any alignment of its
// type), and -infinity where a lane holds nothing.
template <bool kF32, int kVec>
struct Turn {
    static constexpr int kPer = kF32 ? 4 : 8;
    word4 w[kVec];
    bool there, live;

    __device__ __forceinline__ void clear() {
        constexpr uint32_t kFill = kF32 ? 0xFF800000u : 0xFF80FF80u;
#pragma unroll
        for (int v = 0; v < kVec; ++v) w[v] = word4{kFill, kFill, kFill, kFill};
    }
    __device__ __forceinline__ Turn() : there(false), live(false) { clear(); }

    __device__ __forceinline__ void load(const Pieces<kF32, kVec> &P, const void *logits,
                                         uint64_t stride, const uint8_t *mask, uint32_t row,
                                         uint32_t rows) {
        there = row < rows;
        live = there && (!mask || mask[row]);
        if (!there) return;
        const uint8_t *at = (const uint8_t *)logits + row * stride * P.kSize;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const uint8_t *p = at + P.start[v] * P.kSize;
            if (P.experts >= kPer) {
                if (P.holds(v)) w[v] = *(const word4_any *)p;
                continue;
            }
#pragma unroll
            for (int k = 0; k < kPer; ++k) {   // one lane holds the whole row
                if (k >= (int)P.experts) continue;
                if constexpr (kF32) {
                    w[v][k] = ((const uint32_t *)p)[k];
                } else {
                    const uint32_t e = ((const uint16_t *)p)[k];
                    w[v][k >> 1] = k & 1 ? (w[v][k >> 1] & 0xFFFFu) | e << 16
                                         : (w[v][k >> 1] & 0xFFFF0000u) | e;
                }
            }
        }
    }
    // Whatever a row that does not count holds is not looked at.
    __device__ __forceinline__ void hide() {
        if (__ballot(!live) && !live) clear();
    }
};

// e^(x - m) of the lane's experts, their sum over the row (0: nothing but
// -infinity, or a row that does not count), and m.
template <bool kF32, int kVec>
struct RowSoftmax {
    static constexpr int kPer = kF32 ? 4 : 8;
    float e[kVec][kPer];
    float sum, m;

    __device__ __forceinline__ RowSoftmax(const Pieces<kF32, kVec> &P, const word4 (&w)[kVec]) {
        m = -INFINITY;
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
            for (int k = 0; k < kPer; ++k) m = fmaxf(m, element<kF32>(w[v], k));
        m = lanes_reduce<Max>(m, P.lanes);
        if (m == -INFINITY) m = 0.0f;
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                e[v][k] = __builtin_amdgcn_exp2f((element<kF32>(w[v], k) - m) * kLog2E);
        sum = lanes_reduce<Add>(
            P.total(e, [&](int v, int k) { return v < kVec - 1 ? 1.0f : P.weight[k]; }), P.lanes);
    }
    // the hardware's log2, good to one unit in the last place
    __device__ __forceinline__ float lse() const { return m + kLn2 * __builtin_amdgcn_logf(sum); }
};

// kLong: waves of more than kBalanceChain turns.
template <bool kF32, int kVec, bool kLong>
__global__ __launch_bounds__(kBalanceThreads) void balance_kernel(BalanceArgs a) {
    constexpr int kPer = kF32 ? 4 : 8;
    constexpr uint32_t kGroupWaves = kBalanceThreads / 64;
    constexpr uint32_t kMost = BF16D_MAX_EXPERTS;
    constexpr uint32_t kWordsEach = (2 * kMost + kSumWords + kBalanceThreads - 1) / kBalanceThreads;
    // counts, sums of p, and what else is summed
    __shared__ unsigned long long s_words[2 * kMost + kSumWords];
    __shared__ double s_sum[kGroupWaves][3];
    const uint32_t words = 2 * a.experts + kSumWords;
    unsigned long long *const s_more = s_words + 2 * a.experts;
    auto clear = [&] {
        for (uint32_t i = threadIdx.x; i < words; i += kBalanceThreads) s_words[i] = 0;
        __syncthreads();
    };
    const Pieces<kF32, kVec> P(a.experts, a.lane_bits);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float p[kVec][kPer] = {};
    double squares = 0.0;
    uint32_t tokens = 0;
    bool bad_id = false, bad_row = false;
    const uint32_t step = gridDim.x * kGroupWaves * P.held;
    const uint32_t base = (blockIdx.x * kGroupWaves + first_lane(wave)) * P.held;
    uint32_t row = base + (lane >> P.bits);
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
        else if (id >= 0) atomicAdd(&s_words[id], 1ull);
    };
    // The lane's sums of p, as integers to the workgroup's.
    // Rows of up to 16 lanes: the sums of a wave's four quarters are added up first, and
    // each quarter hands over a fourth of them.
    const uint32_t quarter = lane >> 4;
    auto add_p = [&](int v, uint32_t k, float x, float weight) {
        if (weight != 0.0f && x > 0.0f && x < INFINITY)
            atomicAdd(&s_words[a.experts + P.start[v] + k],
                      (unsigned long long)__double2ll_rn((double)x * kFixed));
    };
    auto weight = [&](int v, int k) { return v < kVec - 1 ? 1.0f : P.weight[k]; };
    auto hand_over_p = [&] {
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
            for (int k = 0; k < kPer; k += 4) {
                if (P.bits > 4) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) add_p(v, k + j, p[v][k + j], weight(v, k + j));
                    continue;
                }
                float x = 0.0f, of = 0.0f;
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) {
                    float even, odd;
                    both_halves<32>(p[v][k + j], even, odd);
                    both_halves<16>(even + odd, even, odd);
                    x = quarter == j ? even + odd : x;
                    of = quarter == j ? weight(v, k + j) : of;
                }
                add_p(v, k + quarter, x, of);
            }
    };
    if (base < a.rows) fetch(row);   // while the sums are cleared
    clear();
    uint32_t at = base;
    auto take = [&](uint32_t end) {   // a wave's rows up to there
        for (; at < end; at += step, row += step) {
            Turn<kF32, kVec> now = next;
            const int64_t id = next_id;
            if (at + step < a.rows) fetch(row + step);
            now.hide();
            const RowSoftmax<kF32, kVec> r(P, now.w);
            if (r.sum != 0.0f) {   // else nothing, or nothing that counts
                const float inv = __builtin_amdgcn_rcpf(r.sum);
#pragma unroll
                for (int v = 0; v < kVec; ++v)
#pragma unroll
                    for (int k = 0; k < kPer; ++k) p[v][k] = fmaf(r.e[v][k], inv, p[v][k]);
                const float lse = r.lse();
                if (P.sub == 0) squares += (double)lse * lse;
                bad_row |= !(r.sum < INFINITY);
            }
            if (!now.live) continue;
            tokens += P.sub == 0;
            count(id);
            for (uint32_t j = P.sub + P.lanes; j < a.choices; j += P.lanes) count(id_at(row, j));
        }
    };
    if constexpr (kLong) {
        while (at < a.rows) {
            const uint32_t turns = kBalanceChain * step;   // their rows, at most 2^24
            take(a.rows - at > turns ? at + turns : a.rows);
            if (at >= a.rows) break;
            hand_over_p();
#pragma unroll
            for (int v = 0; v < kVec; ++v)
#pragma unroll
                for (int k = 0; k < kPer; ++k) p[v][k] = 0.0f;
        }
    } else {
        take(a.rows);
    }
    if (tokens) atomicAdd(&s_more[kSumTokens], (unsigned long long)tokens);
    if (bad_id) s_more[kSumBadIds] = 1;
    if (bad_row) s_more[kSumBadRows] = 1;
    hand_over_p();
    // sums over the workgroup, a value a lane, in a fixed order
    auto totals = [&](double (&x)[3]) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            x[k] = lanes_reduce<Add>(x[k]);
            if (lane == 0) s_sum[wave][k] = x[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k)
            x[k] = lanes_reduce<Add>(s_sum[lane & (kGroupWaves - 1)][k], kGroupWaves);
        __syncthreads();
    };
    double x[3] = {squares, 0.0, 0.0};
    __syncthreads();
    if (gridDim.x > 1) {
        totals(x);
        // Every workgroup adds to one of kBalanceCopies copies of the sums: additions
        // to one address by all 256 take 4 us.
        uint64_t *copy = a.sums + (uint64_t)(blockIdx.x % kBalanceCopies) * words;
        uint64_t dep = 0, was[kWordsEach] = {};
#pragma unroll
        for (uint32_t k = 0; k < kWordsEach; ++k) {
            const uint32_t i = threadIdx.x + k * kBalanceThreads;
            if (i < words && s_words[i])
                was[k] = __hip_atomic_fetch_add(copy + i, (uint64_t)s_words[i], __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (uint32_t k = 0; k < kWordsEach; ++k) dep ^= was[k];
        if (threadIdx.x == kBalanceThreads - 1)
            dep ^= __hip_atomic_exchange(a.partial + blockIdx.x,
                                         (uint64_t)__double_as_longlong(x[0]), __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
        if (!last_of_launch(a.done, dep)) return;
        clear();
        // The copies are read and cleared, kAhead words of a thread at once: 1024 rows of 1024
        // bf16 experts 15.6 us, one word at a time 19.2 (257 experts 10.4 and 11.0).
        const uint32_t copies = gridDim.x < kBalanceCopies ? gridDim.x : kBalanceCopies;
        constexpr uint32_t kAhead = 6;
        for (uint32_t i = threadIdx.x; i < copies * words; i += kAhead * kBalanceThreads) {
            uint64_t v[kAhead] = {};
#pragma unroll
            for (uint32_t k = 0; k < kAhead; ++k)
                if (i + k * kBalanceThreads < copies * words)
                    v[k] = __hip_atomic_exchange(a.sums + i + k * kBalanceThreads, (uint64_t)0,
                                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (uint32_t k = 0; k < kAhead; ++k)
                if (v[k])
                    atomicAdd(&s_words[(i + k * kBalanceThreads) % words],
                              (unsigned long long)v[k]);
        }
        static_assert(kBalanceGrid <= kBalanceThreads, "a thread takes one workgroup's sum");
        x[0] = threadIdx.x < gridDim.x
                   ? __longlong_as_double((long long)ld_relaxed_agent(a.partial + threadIdx.x))
                   : 0.0;
        __syncthreads();
    }
    // x: the squares, the choices, and sum of c_e sum of p_te
    for (uint32_t e = threadIdx.x; e < a.experts; e += kBalanceThreads) {
        const uint64_t c = s_words[e];
        a.counts[e] = (int64_t)c;
        x[1] += (double)c;
        x[2] += (double)c * ((double)s_words[a.experts + e] * (1.0 / kFixed));
    }
    totals(x);
    if (threadIdx.x == 0) {
        const uint64_t n = s_more[kSumTokens];
        const double over = n ? 1.0 / (double)n : 0.0;
        double balance = x[1] > 0.0 ? (double)a.experts * x[2] / x[1] * over : 0.0;
        double z = x[0] * over;
        if (s_more[kSumBadIds] || s_more[kSumBadRows]) balance = NAN;
        if (s_more[kSumBadRows]) z = NAN;
        a.result->balance = (float)balance;
        a.result->z = (float)z;
        a.result->loss = (float)(a.balance_coef * balance + a.z_coef * z);
        a.result->tokens = (int64_t)n;
    }
}

// A row's pieces from its values.
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
        if (P.experts >= kPer) {
            if (P.holds(v)) *(word4_any *)p = w;
            continue;
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (k >= (int)P.experts) continue;
            if constexpr (kF32) ((uint32_t *)p)[k] = w[k];
            else ((uint16_t *)p)[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
        }
    }
}

template <bool kF32, int kVec>
__global__ __launch_bounds__(kThreads) void balance_grad_kernel(BalanceGradArgs a) {
    constexpr int kPer = kF32 ? 4 : 8;
    __shared__ double s_tmp[kWaves];
    __shared__ float s_by[BF16D_MAX_EXPERTS];
    const Pieces<kF32, kVec> P(a.experts, a.lane_bits);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t step = gridDim.x * kWaves * P.held;
    const uint32_t base = (blockIdx.x * kWaves + first_lane(wave)) * P.held;
    uint32_t row = base + (lane >> P.bits);
    Turn<kF32, kVec> next;
    if (base < a.rows) next.load(P, a.logits, a.logits_stride, a.mask, row, a.rows);
    constexpr uint32_t kShare = BF16D_MAX_EXPERTS / kThreads;
    double chosen[kShare], choices = 0.0;
#pragma unroll
    for (uint32_t i = 0; i < kShare; ++i) {
        const uint32_t e = i * kThreads + threadIdx.x;
        chosen[i] = e < a.experts ? (double)a.counts[e] : 0.0;
        choices += chosen[i];
    }
    choices = group_total(choices, s_tmp);
    const double n = *a.tokens > 1 ? (double)*a.tokens : 1.0;
    // of one choice
    const double by_share =
        choices > 0.0 ? a.scale * a.balance_coef * a.experts / n / choices : 0.0;
    const float by_lse = (float)(2.0 * a.scale * a.z_coef / n);
    const float spoilt = a.result && a.result->loss != a.result->loss ? NAN : 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < kShare; ++i)
        s_by[i * kThreads + threadIdx.x] = (float)(by_share * chosen[i]);
    __syncthreads();
    float by[kVec][kPer], held[kPer];   // an expert's factor; of the last piece, weighted
#pragma unroll
    for (int v = 0; v < kVec; ++v)
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const uint32_t e = P.start[v] + k;
            by[v][k] = P.holds(v) && e < a.experts ? s_by[e] : 0.0f;
            if (v == kVec - 1) held[k] = by[v][k] * P.weight[k];
        }
    for (uint32_t at = base; at < a.rows; at += step, row += step) {   // a wave's rows
        Turn<kF32, kVec> now = next;
        if (at + step < a.rows) next.load(P, a.logits, a.logits_stride, a.mask, row + step, a.rows);
        now.hide();
        const RowSoftmax<kF32, kVec> r(P, now.w);
        const float inv = r.sum != 0.0f ? __builtin_amdgcn_rcpf(r.sum) : 0.0f;
        const float inner = inv * lanes_reduce<Add>(
            P.total(r.e, [&](int v, int k) { return v < kVec - 1 ? by[v][k] : held[k]; }), P.lanes);
        float same = r.sum != 0.0f ? (by_lse * r.lse() - inner) * inv : 0.0f;
        if (now.live) same += spoilt;
        if (!now.there) continue;
        float g[kVec][kPer];
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
            for (int k = 0; k < kPer; ++k) g[v][k] = r.e[v][k] * fmaf(by[v][k], inv, same);
        store_row(g, P, (uint8_t *)a.out + row * a.out_stride * P.kSize);
    }
}

// How a row is held: by 2^bits lanes of `vec` pieces each.
struct Hold {
    uint32_t bits, vec;
};
uint32_t pieces_of(uint32_t experts, bool f32) {
    const uint32_t per = f32 ? 4 : 8;
    return (experts + per - 1) / per;
}
// Few lanes take fewer steps to join, for more rows at once, and leave fewer lanes idle:
// 131072 rows of 257 bf16 experts 30 us forward and 29 backward, with a piece a lane 53 and 48;
// of 64 fp32 experts 15.7 and 13.6, 17.2 and 13.3.  Fewer than 8 lanes load too
// scattered (65536 rows of 64, 4 lanes: 17 and 17), and four pieces of 8 do not fit into the
// registers of a workgroup of 16 waves.
Hold fewest_lanes(uint32_t pieces, bool f32) {
    uint32_t bits = 0;
    auto most = [&] { return bits < 3 ? 1u : bits == 3 ? 2u : f32 ? 4u : 3u; };
    while (bits < 6 && pieces > most() << bits) ++bits;
    return Hold{bits, (pieces + (1u << bits) - 1) >> bits};
}
// The same with more lanes, as long as there are so many in all: 4096 rows of 257 bf16
// experts 12.2 us forward and 5.1 backward, with the fewest 13.9 and 6.5.
Hold more_lanes(Hold h, uint32_t pieces, uint32_t rows, uint32_t threads) {
    while (h.bits < 6 && pieces > 1u << h.bits && (uint64_t)rows << (h.bits + 1) <= threads)
        ++h.bits;
    return Hold{h.bits, (pieces + (1u << h.bits) - 1) >> h.bits};
}
// workgroups of `waves` waves for the rows: `most`, or a turn each, or one for up to
// `alone` turns
uint32_t grid_of(uint32_t rows, uint32_t lane_bits, uint32_t waves, uint32_t most,
                 uint32_t alone) {
    const uint32_t turn = waves * (64u >> lane_bits);
    const uint32_t turns = (rows + turn - 1) / turn;
    return turns <= alone ? 1 : turns < most ? turns : most;
}

template <bool kF32, bool kLong>
auto kernel_of(uint32_t vec) {
    return vec == 1   ? balance_kernel<kF32, 1, kLong>
           : vec == 2 ? balance_kernel<kF32, 2, kLong>
           : vec == 3 ? balance_kernel<kF32, 3, kLong>
                      : balance_kernel<kF32, kF32 ? 4 : 3, kLong>;
}
template <bool kF32>
auto grad_kernel_of(uint32_t vec) {
    return vec == 1   ? balance_grad_kernel<kF32, 1>
           : vec == 2 ? balance_grad_kernel<kF32, 2>
           : vec == 3 ? balance_grad_kernel<kF32, 3>
                      : balance_grad_kernel<kF32, kF32 ? 4 : 3>;
}

}  // namespace

hipError_t launch_balance(BalanceArgs a, bool f32, hipStream_t stream) {
    constexpr uint32_t kGroupWaves = kBalanceThreads / 64;
    const uint32_t pieces = pieces_of(a.experts, f32);
    Hold hold = fewest_lanes(pieces, f32);
    if (grid_of(a.rows, hold.bits, kGroupWaves, kBalanceGrid, kBalanceAlone) > 1)
        hold = more_lanes(hold, pieces, a.rows, kBalanceGrid * kBalanceThreads);
    a.lane_bits = hold.bits;
    const uint32_t grid = grid_of(a.rows, hold.bits, kGroupWaves, kBalanceGrid, kBalanceAlone);
    const uint64_t chain = (uint64_t)grid * kGroupWaves * (64u >> hold.bits) * kBalanceChain;
    auto *kernel = a.rows > chain
                       ? (f32 ? kernel_of<true, true>(hold.vec) : kernel_of<false, true>(hold.vec))
                       : f32 ? kernel_of<true, false>(hold.vec)
                             : kernel_of<false, false>(hold.vec);
    return launch_one(kernel, grid, kBalanceThreads, a, 0, stream);
}

hipError_t launch_balance_backward(BalanceGradArgs a, bool f32, hipStream_t stream) {
    const uint32_t pieces = pieces_of(a.experts, f32);
    Hold hold = fewest_lanes(pieces, f32);
    // as many workgroups as are resident at once: with more than 8 experts a lane half of them
    const uint32_t most = kBalanceGradGrid >> (hold.vec * (f32 ? 4 : 8) > 8);
    hold = more_lanes(hold, pieces, a.rows, most * kThreads);
    a.lane_bits = hold.bits;
    const uint32_t grid = grid_of(a.rows, hold.bits, kWaves, most, 1);
    return launch_one(f32 ? grad_kernel_of<true>(hold.vec) : grad_kernel_of<false>(hold.vec), grid,
                      kThreads, a, 0, stream);
}

}  // namespace bf16d
