// logprob.hip -- log probabilities of given tokens, the entropy and the top
// alternatives of their distributions, and the gradient of the logits.
//
// With c = log2(e) / temperature, m a running maximum and t_j = (x_j - m) c,
// every thread keeps S = sum 2^t_j and W = sum 2^t_j t_j of the elements it has
// seen; a new maximum m' shifts t by d = (m - m') c:
//   S' = 2^d S,   W' = 2^d (W + d S)
// Then ln p_y = (x_y - m) / T - ln S, and H = ln2 (log2 S - W / S): a sum of
// terms of one sign, so nothing cancels.  One pass over the logits.
//
// Differences are formed before anything is scaled, so logits at the ends of
// fp32 neither overflow nor lose their distance from the maximum.
#include "loss.hpp"

namespace bf16d {
namespace {

constexpr float kNone = -1e4f;   // a t below which 2^t is 0: keeps 0 * infinity out of W
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// ---- softmax sums ----------------------------------------------------------------
struct Sums {
    float m, s, w;
};
// what differences are taken from: the maximum, or 0 where there is none yet
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : m; }

// the same sums by a maximum of at least their own
__device__ __forceinline__ void shift(Sums &a, float m, float c) {
    const float d = (a.m - reference(m)) * c;
    const float f = exp2_fast(d);
    a.w = f * (a.w + fmaxf(d, kNone) * a.s);
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ void merge(Sums &a, Sums b, float c) {
    const float m = fmaxf(a.m, b.m);
    shift(a, m, c);
    shift(b, m, c);
    a.s += b.s;
    a.w += b.w;
}
// the sums of the whole workgroup, in every thread
__device__ __forceinline__ Sums group_sums(Sums a, float c, float (*s_tmp)[3]) {
    shift(a, lanes_reduce<Max>(a.m), c);
    a.s = lanes_reduce<Add>(a.s);
    a.w = lanes_reduce<Add>(a.w);
    const uint32_t wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
        s_tmp[wave][0] = a.m;
        s_tmp[wave][1] = a.s;
        s_tmp[wave][2] = a.w;
    }
    __syncthreads();
    Sums all = {s_tmp[0][0], s_tmp[0][1], s_tmp[0][2]};
#pragma unroll
    for (uint32_t v = 1; v < kWaves; ++v)
        merge(all, Sums{s_tmp[v][0], s_tmp[v][1], s_tmp[v][2]}, c);
    __syncthreads();
    return all;
}

// ---- the largest elements -------------------------------------------------------------
// A wave keeps the largest it has seen as one key a lane, sorted from lane 0
// down: the value's order in the high word, the complement of its id in the
// low one, so that no two are equal and the lower id of equal values is the
// larger key.  0 is no element.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t id) {
    if (!(x > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(x + 0.0f);   // -0 counts as 0
    const uint32_t order = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return (uint64_t)order << 32 | (uint32_t)~id;
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t shfl_key(uint64_t k, uint32_t lane) {
    return __shfl((unsigned long long)k, (int)lane, 64);
}
__device__ __forceinline__ uint64_t readlane_key(uint64_t k, uint32_t lane) {
    return (uint64_t)readlane_u32((uint32_t)k, lane) |
           (uint64_t)readlane_u32((uint32_t)(k >> 32), lane) << 32;
}
// the 64 largest of two sorted lists, sorted
__device__ __forceinline__ uint64_t merge_lists(uint64_t a, uint64_t b) {
    const uint32_t lane = threadIdx.x & 63;
    const uint64_t r = shfl_key(b, 63 - lane);
    uint64_t c = a > r ? a : r;   // falls and rises, or rises and falls
#pragma unroll
    for (uint32_t d = 32; d >= 1; d >>= 1) {
        const uint64_t o = shfl_key(c, lane ^ d);
        const bool keep_larger = (lane & d) == 0;
        c = (c > o) == keep_larger ? c : o;
    }
    return c;
}
// the value of rank `rank` (from 0) among the lanes' values, NaN aside
__device__ __forceinline__ float ranked_value(float v, uint32_t rank) {
    const uint32_t lane = threadIdx.x & 63;
    v = v > -INFINITY ? v : -INFINITY;
#pragma unroll
    for (uint32_t size = 2; size <= 64; size <<= 1) {
#pragma unroll
        for (uint32_t d = size >> 1; d >= 1; d >>= 1) {
            const float o = __shfl_xor(v, (int)d, 64);
            const bool falling = (lane & size) == 0;   // (lane & 64) is 0 at the last size
            const bool keep_larger = ((lane & d) == 0) == falling;
            v = keep_larger ? fmaxf(v, o) : fminf(v, o);
        }
    }
    return __uint_as_float(readlane_u32(__float_as_uint(v), rank));
}

struct TopList {
    uint64_t key;        // this lane's
    uint64_t last;       // the key of the last place that counts, 0 while it is free
    float least;         // what an element has to reach
};
// one candidate a lane (0: none), of any number
__device__ __forceinline__ void insert(TopList &l, uint64_t key, uint32_t top) {
    const uint32_t lane = threadIdx.x & 63;
    uint64_t todo = __ballot(key > l.last);
    while (todo) {
        const uint32_t from = (uint32_t)__builtin_ctzll(todo);
        const uint64_t k = readlane_key(key, from);
        const uint32_t place = (uint32_t)__popcll(__ballot(l.key > k));
        const uint64_t before = (uint64_t)wave_shr1((uint32_t)l.key) |
                                (uint64_t)wave_shr1((uint32_t)(l.key >> 32)) << 32;
        l.key = lane < place ? l.key : lane == place ? k : before;
        l.last = readlane_key(l.key, top - 1);
        todo &= todo - 1;
        todo &= __ballot(key > l.last);
    }
    if (l.last) l.least = fmaxf(l.least, key_value(l.last));
}

// ---- forward ---------------------------------------------------------------------------
// A row is cut into vectors at 16-byte addresses: vector i holds its elements from
// i * kPer - skip on, skip being how many elements lie between such an address
// and the row's start.  Only the first and the last vector can be partial.
// (Vectors counted from the row's own start read 10 to 20 % slower where that is odd.)
template <bool kF32>
struct RowVectors {
    static constexpr uint32_t kPer = kF32 ? 4 : 8, kSize = kF32 ? 4 : 2;
    const uint8_t *row;
    uint32_t skip, vocab;

    __device__ __forceinline__ RowVectors(const uint8_t *at, uint32_t n)
        : row(at), skip(((uint32_t)(uintptr_t)at & 15u) / kSize), vocab(n) {}
    // the id of vector i's first element (below 0 in a partial first one, as uint32_t)
    __device__ __forceinline__ uint32_t first(uint32_t i) const { return i * kPer - skip; }
    __device__ __forceinline__ const uint8_t *at(uint32_t i) const {
        return row + (int64_t)(int32_t)first(i) * kSize;
    }
    __device__ __forceinline__ bool whole(uint32_t i) const {
        return first(i) < vocab && vocab - first(i) >= kPer;
    }
    // whether every vector of the turn is
    __device__ __forceinline__ bool whole_turn(uint32_t turn) const {
        return (turn > 0 || skip == 0) && (turn + 1) * kTurnVectors * kPer <= vocab + skip;
    }
    __device__ __forceinline__ uint32_t turns() const {
        return (vocab + skip + kTurnVectors * kPer - 1) / (kTurnVectors * kPer);
    }
};

// what is no token is -infinity
template <bool kF32>
__device__ __forceinline__ word4 load_partial(const RowVectors<kF32> &r, uint32_t i) {
    constexpr uint32_t kPer = RowVectors<kF32>::kPer;
    const uint32_t first = r.first(i);
    word4 w;
    if constexpr (kF32) w = word4{0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u};
    else w = word4{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u};
#pragma unroll
    for (uint32_t k = 0; k < kPer; ++k) {
        if (first + k >= r.vocab) continue;
        if constexpr (kF32) {
            w[k] = ((const uint32_t *)r.row)[first + k];
        } else {
            const uint32_t e = ((const uint16_t *)r.row)[first + k];
            w[k >> 1] = k & 1 ? (w[k >> 1] & 0xFFFFu) | e << 16 : (w[k >> 1] & 0xFFFF0000u) | e;
        }
    }
    return w;
}

// The thread's vectors of a turn (vector q * kThreads + threadIdx.x of it).  kKeep: they
// may stay in the caches.
template <bool kKeep, bool kF32>
__device__ __forceinline__ void load_turn(word4 (&v)[4], const RowVectors<kF32> &r,
                                          uint32_t turn) {
    const uint32_t first = turn * kTurnVectors + threadIdx.x;
    if (r.whole_turn(turn)) {
        const auto *p = (const word4 *)r.at(first);
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
            if constexpr (kKeep) v[q] = p[q * kThreads];
            else v[q] = __builtin_nontemporal_load(p + q * kThreads);
        }
        return;
    }
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
        const uint32_t i = first + q * kThreads;
        v[q] = r.whole(i) ? *(const word4 *)r.at(i) : load_partial(r, i);
    }
}

template <bool kF32, bool kEntropy>
__device__ __forceinline__ void add_turn(Sums &a, const word4 (&v)[4], float m, float c) {
    constexpr int kPer = kF32 ? 4 : 8;
    shift(a, fmaxf(a.m, m), c);
    const float ref = reference(a.m);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const float t = (element<kF32>(v[q], k) - ref) * c;
            const float e = exp2_fast(t);
            a.s += e;
            if constexpr (kEntropy) a.w += e * fmaxf(t, kNone);
        }
}

// The outputs of a row that is left out, or of one whose sums are complete.
__device__ __forceinline__ void write_left_out(const LogprobArgs &a, uint32_t row) {
    if (threadIdx.x == 0) {
        a.logp[row] = 0.0f;
        if (a.entropy) a.entropy[row] = 0.0f;
        if (a.stats) a.stats[row] = bf16d_row_stats{0.0f, 0.0f, 0.0f, a.scale};
    }
    if (threadIdx.x < a.top) {
        a.top_ids[(uint64_t)row * a.top + threadIdx.x] = -1;
        a.top_logp[(uint64_t)row * a.top + threadIdx.x] = -INFINITY;
    }
}
// `key`: the list of the first wave
template <bool kEntropy>
__device__ __forceinline__ void write_row(const LogprobArgs &a, uint32_t row, const Sums &s,
                                          int64_t token, float x, uint64_t key) {
    const bool empty = s.s == 0.0f;   // the maximum itself adds 1
    const float ln_s = logf(s.s), log2_s = log2f(s.s);
    if (threadIdx.x == 0) {
        const float h = empty ? 0.0f : kLn2 * (log2_s - s.w / s.s);
        a.logp[row] = token >= (int64_t)a.vocab ? NAN
                      : empty                   ? -INFINITY
                                                : (x - s.m) * a.inv_t - ln_s;
        if (kEntropy) a.entropy[row] = h;
        if (a.stats)
            a.stats[row] = bf16d_row_stats{s.m, empty ? 0.0f : log2_s, kEntropy ? h : NAN, a.scale};
    }
    if (threadIdx.x < a.top) {
        const uint64_t at = (uint64_t)row * a.top + threadIdx.x;
        a.top_ids[at] = key ? (int64_t)(uint32_t)~(uint32_t)key : -1;
        a.top_logp[at] = key ? (key_value(key) - s.m) * a.inv_t - ln_s : -INFINITY;
    }
}

template <bool kF32, bool kEntropy, bool kTop, bool kKeep>
__global__ __launch_bounds__(kThreads) void logprob_kernel(LogprobArgs a) {
    __shared__ float s_tmp[kWaves][3];
    __shared__ uint64_t s_list[kTop ? kWaves : 1][64];
    constexpr uint32_t kPer = kF32 ? 4 : 8, kSize = kF32 ? 4 : 2;
    const uint32_t row = blockIdx.x / a.parts, part = blockIdx.x - row * a.parts;
    const int64_t token =
        load_id(row_ptr(a.tokens, row, a.inner, a.token_i32 ? 4 : 8), a.token_i32);
    if (token < 0) {
        if (part == 0) write_left_out(a, row);
        return;
    }
    const uint8_t *x = row_ptr(a.logits, row, a.inner, kSize);
    float own = 0.0f;   // the token's logit
    if (threadIdx.x == 0 && token < (int64_t)a.vocab) {
        if constexpr (kF32) own = ((const float *)x)[token];
        else own = __uint_as_float((uint32_t)((const uint16_t *)x)[token] << 16);
    }
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const RowVectors<kF32> r(x, a.vocab);
    const uint32_t turns = r.turns();
    const uint32_t begin = part * a.part_turns;
    const uint32_t end = begin + a.part_turns < turns ? begin + a.part_turns : turns;
    Sums mine = {-INFINITY, 0.0f, 0.0f};
    TopList best = {0, 0, -INFINITY};
    word4 v[4], next[4];
    if (begin < end) load_turn<kKeep>(next, r, begin);
    for (uint32_t turn = begin; turn < end; ++turn) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = next[q];
        if (turn + 1 < end) load_turn<kKeep>(next, r, turn + 1);
        float m = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int k = 0; k < (int)kPer; ++k) m = fmaxf(m, element<kF32>(v[q], k));
        if constexpr (kTop) {
            if (__ballot(m >= best.least && m > -INFINITY)) {
                // at least `top` elements reach the maximum of that rank
                if (!best.last) best.least = fmaxf(best.least, ranked_value(m, a.top - 1));
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int k = 0; k < (int)kPer; ++k) {
                        const float e = element<kF32>(v[q], k);
                        if (!__ballot(e >= best.least)) continue;
                        const uint32_t id =
                            r.first(turn * kTurnVectors + q * kThreads + threadIdx.x) + k;
                        insert(best, e >= best.least ? key_of(e, id) : 0, a.top);
                    }
            }
        }
        add_turn<kF32, kEntropy>(mine, v, m, a.scale);
    }
    Sums all = group_sums(mine, a.scale, s_tmp);
    uint64_t key = 0;
    if constexpr (kTop) {
        s_list[wave][lane] = best.key;
        __syncthreads();
        key = s_list[0][lane];
#pragma unroll
        for (uint32_t v = 1; v < kWaves; ++v) key = merge_lists(key, s_list[v][lane]);
    }
    if (a.parts == 1) {
        write_row<kEntropy>(a, row, all, token, own, key);
        return;
    }
    // the part's sums and list are handed over by returning device-scope atomics
    const uint32_t words = 2 + a.top;
    uint64_t *mine_at = a.partial + (uint64_t)blockIdx.x * words;
    uint64_t dep = 0;
    auto hand = [&](uint32_t at, uint64_t v) {
        return __hip_atomic_exchange(mine_at + at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    if (wave == 0) {
        if (lane == 0)
            dep = hand(0, (uint64_t)__float_as_uint(all.m) << 32 | __float_as_uint(all.s));
        if (lane == 1) dep = hand(1, __float_as_uint(all.w));
        if (kTop && lane < a.top) dep += hand(2 + lane, key);
    }
    if (!last_of(a.done + row, a.parts, dep)) return;
    const uint64_t *row_at = a.partial + (uint64_t)row * a.parts * words;
    mine = Sums{-INFINITY, 0.0f, 0.0f};
    for (uint32_t p = threadIdx.x; p < a.parts; p += kThreads) {
        const uint64_t ms = ld_relaxed_agent(row_at + (uint64_t)p * words);
        const uint64_t w = ld_relaxed_agent(row_at + (uint64_t)p * words + 1);
        merge(mine, Sums{__uint_as_float((uint32_t)(ms >> 32)), __uint_as_float((uint32_t)ms),
                         __uint_as_float((uint32_t)w)}, a.scale);
    }
    all = group_sums(mine, a.scale, s_tmp);
    if constexpr (kTop) {
        key = 0;
        for (uint32_t p = wave; p < a.parts; p += kWaves)
            key = merge_lists(key, lane < a.top ? ld_relaxed_agent(row_at + (uint64_t)p * words +
                                                                   2 + lane)
                                                : 0);
        s_list[wave][lane] = key;
        __syncthreads();
        key = s_list[0][lane];
#pragma unroll
        for (uint32_t v = 1; v < kWaves; ++v) key = merge_lists(key, s_list[v][lane]);
    }
    write_row<kEntropy>(a, row, all, token, own, key);
    if (threadIdx.x == 0)
        __hip_atomic_store(a.done + row, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---- backward ------------------------------------------------------------------------------
// The vectors of a turn, as they were loaded, into another row.
template <bool kF32>
__device__ __forceinline__ void store_turn(const word4 (&v)[4], uint8_t *out,
                                           const RowVectors<kF32> &r, uint32_t turn) {
    constexpr uint32_t kPer = RowVectors<kF32>::kPer, kSize = RowVectors<kF32>::kSize;
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
        const uint32_t i = turn * kTurnVectors + threadIdx.x + q * kThreads;
        const uint32_t first = r.first(i);
        if (r.whole(i)) {
            __builtin_nontemporal_store(v[q], (word4_any *)(out + (uint64_t)first * kSize));
        } else {
#pragma unroll
            for (uint32_t k = 0; k < kPer; ++k) {
                if (first + k >= r.vocab) continue;
                if constexpr (kF32) ((uint32_t *)out)[first + k] = v[q][k];
                else ((uint16_t *)out)[first + k] = (uint16_t)(v[q][k >> 1] >> (16 * (k & 1)));
            }
        }
    }
}

// One part of a row.  g_j = -p_j (A + B t_j) with t_j = log2 p_j, A = (a + h H) / T
// and B = h ln2 / T, and a / T more at the token.
template <bool kF32, bool kEntropy>
__global__ __launch_bounds__(kThreads) void logprob_grad_kernel(LogprobGradArgs g) {
    constexpr uint32_t kPer = kF32 ? 4 : 8, kSize = kF32 ? 4 : 2;
    const uint32_t row = blockIdx.x / g.parts, part = blockIdx.x - row * g.parts;
    const int64_t token =
        load_id(row_ptr(g.tokens, row, g.inner, g.token_i32 ? 4 : 8), g.token_i32);
    uint8_t *out = const_cast<uint8_t *>(row_ptr(g.out, row, g.inner, kSize));
    const RowVectors<kF32> r(row_ptr(g.logits, row, g.inner, kSize), g.vocab);
    const uint32_t turns = r.turns();
    const uint32_t begin = part * g.part_turns;
    const uint32_t end = begin + g.part_turns < turns ? begin + g.part_turns : turns;
    const float a = g.grad_logp[row], h = kEntropy ? g.grad_entropy[row] : 0.0f;
    const bf16d_row_stats s = g.stats[row];
    const bool zero = token < 0 || (a == 0.0f && h == 0.0f) ||
                      (s.max == -INFINITY && s.log2_sum == 0.0f);
    if (zero || token >= (int64_t)g.vocab) {
        const uint32_t fill = zero ? 0u : kF32 ? 0x7FC00000u : 0x7FC07FC0u;
        const word4 v[4] = {word4{fill, fill, fill, fill}, word4{fill, fill, fill, fill},
                            word4{fill, fill, fill, fill}, word4{fill, fill, fill, fill}};
        for (uint32_t turn = begin; turn < end; ++turn) store_turn(v, out, r, turn);
        return;
    }
    const float inv_t = s.scale * kLn2;
    const float add = a * inv_t;
    const float A = kEntropy ? -(a + h * s.entropy) * inv_t : -add;
    const float B = -h * inv_t * kLn2;
    for (uint32_t turn = begin; turn < end; ++turn) {
        word4 v[4];
        load_turn<false>(v, r, turn);
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
            const uint32_t id = r.first(turn * kTurnVectors + q * kThreads + threadIdx.x);
            const uint32_t hit = (uint32_t)token - id;   // below kPer: the token is here
            float d[kPer];
#pragma unroll
            for (uint32_t k = 0; k < kPer; ++k) {
                const float t = (element<kF32>(v[q], k) - s.max) * s.scale - s.log2_sum;
                const float p = exp2_fast(t);
                d[k] = kEntropy ? p * (A + B * fmaxf(t, kNone)) : p * A;
                if (k == hit) d[k] += add;
            }
            if constexpr (kF32) {
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) v[q][k] = __float_as_uint(d[k]);
            } else {
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) v[q][k] = pack_bf16(d[2 * k], d[2 * k + 1]);
            }
        }
        store_turn(v, out, r, turn);
    }
}

template <bool kF32, bool kEntropy>
hipError_t launch_forward(const LogprobArgs &a, bool keep, hipStream_t stream) {
    // few rows have alternatives: they stay in the caches in any case
    auto *kernel = a.top  ? logprob_kernel<kF32, kEntropy, true, true>
                   : keep ? logprob_kernel<kF32, kEntropy, false, true>
                          : logprob_kernel<kF32, kEntropy, false, false>;
    return launch_one(kernel, a.rows * a.parts, kThreads, a, 0, stream);
}
}  // namespace

hipError_t launch_logprob(const LogprobArgs &a, bool f32, bool keep, hipStream_t stream) {
    if (f32)
        return a.entropy ? launch_forward<true, true>(a, keep, stream)
                         : launch_forward<true, false>(a, keep, stream);
    return a.entropy ? launch_forward<false, true>(a, keep, stream)
                     : launch_forward<false, false>(a, keep, stream);
}

hipError_t launch_logprob_backward(const LogprobGradArgs &a, bool f32, hipStream_t stream) {
    auto *kernel = f32 ? (a.grad_entropy ? logprob_grad_kernel<true, true>
                                         : logprob_grad_kernel<true, false>)
                       : (a.grad_entropy ? logprob_grad_kernel<false, true>
                                         : logprob_grad_kernel<false, false>);
    return launch_one(kernel, a.rows * a.parts, kThreads, a, 0, stream);
}

}  // namespace bf16d
