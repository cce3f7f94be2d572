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
//
// Forward: 2 or 4 bytes and 8 to 10 vector instructions an element.  fp32 is bound
// by the read, at 6.2 to 6.9 TB/s (16384 x 32000: 305 us); bf16 by the read and
// the vector units (16384 x 32000: 161 us, 6.5 TB/s; with entropy 177 us, 91 % of
// the issue slots).  One fma an element instead of a difference and a product was
// no faster: the registers it took cost as much.
// Backward: a read and a write of every element, at 5.7 to 6.3 TB/s (4096 x 32000
// bf16 84 us; a plain copy of them runs at 5.4).  One turn a workgroup, as the loads
// and stores of neighbours then stay close together, and non-temporal stores: with plain
// ones the forward pass of the next batch waits for them to be written back (75
// instead of 52 us after the backward pass of 4096 x 32000).
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
template <uint32_t kCount>
__device__ __forceinline__ Sums group_sums(Sums a, float c, float (&s_tmp)[kCount][3]) {
    auto reduce = [&](Sums &x, uint32_t lanes) {
        shift(x, lanes_reduce<Max>(x.m, lanes), c);
        x.s = lanes_reduce<Add>(x.s, lanes);
        x.w = lanes_reduce<Add>(x.w, lanes);
    };
    reduce(a, 64);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane == 0) {
        s_tmp[wave][0] = a.m;
        s_tmp[wave][1] = a.s;
        s_tmp[wave][2] = a.w;
    }
    __syncthreads();
    const float *of = s_tmp[lane & (kCount - 1)];
    Sums all = {of[0], of[1], of[2]};
    reduce(all, kCount);
    __syncthreads();
    return all;
}

// ---- rows of logits ---------------------------------------------------------------------
// A row is cut into vectors at 16-byte addresses: vector i holds its elements from
// i * kPer - skip on, skip being how many elements lie between such an address
// and the row's start.  Only the first and the last vector can be partial.
// (Vectors counted from the row's own start were read at 4.8 instead of 5.9 TB/s where
// that is odd: 2039 rows of 100003.)
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
    // whether every vector of a turn of kBlock threads is
    template <uint32_t kBlock>
    __device__ __forceinline__ bool whole_turn(uint32_t turn) const {
        return (turn > 0 || skip == 0) && (turn + 1) * kTurnVectors * kBlock * kPer <= vocab + skip;
    }
    __device__ __forceinline__ uint32_t vectors() const { return (vocab + skip + kPer - 1) / kPer; }
    template <uint32_t kBlock>
    __device__ __forceinline__ uint32_t turns() const {
        constexpr uint32_t kTurn = kTurnVectors * kBlock;
        return (vectors() + kTurn - 1) / kTurn;
    }
};

// The same vector, as one the compiler has not seen: it widens bf16 elements again
// where they are used, and does not keep them widened, so that 64 registers
// are enough for two workgroups of 16 waves on a CU.
__device__ __forceinline__ word4 fresh(word4 w) {
    asm volatile("" : "+v"(w));
    return w;
}

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

// The thread's vectors of a turn (vector q * kBlock + threadIdx.x of it).  kKeep: they
// may stay in the caches.
template <uint32_t kBlock, bool kKeep, bool kF32>
__device__ __forceinline__ void load_turn(word4 (&v)[4], const RowVectors<kF32> &r,
                                          uint32_t turn) {
    const uint32_t first = turn * kTurnVectors * kBlock + threadIdx.x;
    if (r.template whole_turn<kBlock>(turn)) {
        const auto *p = (const word4 *)r.at(first);
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
            if constexpr (kKeep) v[q] = p[q * kBlock];
            else v[q] = __builtin_nontemporal_load(p + q * kBlock);
        }
        return;
    }
    constexpr uint32_t kFill = kF32 ? 0xFF800000u : 0xFF80FF80u;
    bool partial = false;
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
        const uint32_t i = first + q * kBlock;
        v[q] = word4{kFill, kFill, kFill, kFill};
        if (r.whole(i)) v[q] = *(const word4 *)r.at(i);
        else partial |= i < r.vectors();
    }
    if (!partial) return;
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
        const uint32_t i = first + q * kBlock;
        if (i < r.vectors() && !r.whole(i)) v[q] = fresh(load_partial(r, i));   // one at a time
    }
}

// ---- the largest elements -------------------------------------------------------------
// An element as one key: the value's order in the high word, the complement of
// its id in the low one, so that no two are equal and the lower id of equal
// values is the larger key.  0 is no element.  Lists are a wave's lanes, the largest
// key in lane 0.
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
__device__ __forceinline__ uint64_t readlane_key(uint64_t k, uint32_t lane) {
    return (uint64_t)readlane_u32((uint32_t)k, lane) |
           (uint64_t)readlane_u32((uint32_t)(k >> 32), lane) << 32;
}

// One comparison of a sorting network: the lower lane of a pair keeps the larger.
template <int kMask>
__device__ __forceinline__ bool lower_lane() {
    return (threadIdx.x & (1u << (31 - __builtin_clz(kMask)))) == 0;
}
template <int kMask>
__device__ __forceinline__ void exchange(float &v) {
    const float o = __uint_as_float(lane_xor<kMask>(__float_as_uint(v)));
    v = lower_lane<kMask>() ? fmaxf(v, o) : fminf(v, o);
}
template <int kMask>
__device__ __forceinline__ uint64_t xor_key(uint64_t v) {
    return (uint64_t)lane_xor<kMask>((uint32_t)(v >> 32)) << 32 | lane_xor<kMask>((uint32_t)v);
}
template <int kMask>
__device__ __forceinline__ void exchange(uint64_t &v) {
    const uint64_t o = xor_key<kMask>(v);
    v = (v > o) == lower_lane<kMask>() ? v : o;
}
// sorts what first rises and then falls, or the other way round, over kSize lanes
template <int kSize, typename T>
__device__ __forceinline__ void merge_halves(T &v) {
    if constexpr (kSize > 1) {
        exchange<kSize / 2>(v);
        merge_halves<kSize / 2>(v);
    }
}
// sorts the values of kSize lanes (not NaN)
template <int kSize = 64, typename T>
__device__ __forceinline__ void sort_lanes(T &v) {
    if constexpr (kSize > 1) {
        sort_lanes<kSize / 2>(v);
        exchange<kSize - 1>(v);
        merge_halves<kSize / 2>(v);
    }
}
// the 64 largest of two lists
__device__ __forceinline__ uint64_t merge_lists(uint64_t a, uint64_t b) {
    const uint64_t r = xor_key<63>(b);
    uint64_t c = a > r ? a : r;
    merge_halves<64>(c);
    return c;
}

// Inserts one candidate a lane (0: none), of any number; `last`: the key of the
// list's last place that counts, 0 while it is free.
__device__ __forceinline__ void insert(uint64_t &list, uint64_t &last, uint64_t key, uint32_t top) {
    const uint32_t lane = threadIdx.x & 63;
    uint64_t todo = __ballot(key > last);
    while (todo) {
        const uint32_t from = (uint32_t)__builtin_ctzll(todo);
        const uint64_t k = readlane_key(key, from);
        const uint32_t place = (uint32_t)__popcll(__ballot(list > k));
        const uint64_t before = (uint64_t)wave_shr1((uint32_t)list) |
                                (uint64_t)wave_shr1((uint32_t)(list >> 32)) << 32;
        list = lane < place ? list : lane == place ? k : before;
        last = readlane_key(list, top - 1);
        todo &= todo - 1;
        todo &= __ballot(key > last);
    }
}

// A workgroup's largest elements.  In each turn the lanes' maxima are joined to 16, 32
// or 64 groups; the group maximum of rank `top` is a bound that `top` elements
// reach.  Those that reach it (hardly more, unless many are equal or `top` is near
// 64) are collected and put in order.  A turn takes 2.5 us more with 5 alternatives
// than without, 3 with 20 (one row of 32000: 7.0 and 7.6 us).
constexpr uint32_t kFound = 1024;
template <uint32_t kCount>   // waves
struct TopShared {
    float named[64];
    float bound;
    uint32_t count[2];   // of the found ones, for even and odd turns
    float least;         // what an element has to reach to be among the largest so far
    uint64_t found[kFound];
    uint64_t lists[kCount][64];
};
// One wave: the list of the keys of its first `count` lanes, which s.found holds, too
// (the others' are 0).  A key's place is how many are larger; a sorting network
// takes twice as long for the 10 to 30 keys that there are as a rule.
template <uint32_t kCount>
__device__ __forceinline__ uint64_t in_order(TopShared<kCount> &s, uint64_t key, uint32_t count) {
    const uint32_t lane = threadIdx.x & 63;
    uint32_t place = 0;
#pragma unroll 4
    for (uint32_t j = 0; j < count; ++j) place += s.found[j] > key;
    if (lane < count) s.lists[0][place] = key;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // a wave's LDS accesses are in order
    return lane < count ? s.lists[0][lane] : 0;
}
// v: the thread's vectors of the turn, m: their maxima; begin: the first turn
template <uint32_t kCount, bool kF32>
__device__ __forceinline__ void add_largest(uint64_t &list, TopShared<kCount> &s,
                                            const word4 (&v)[4], const float (&m)[4],
                                            const RowVectors<kF32> &r, uint32_t turn,
                                            bool begin, uint32_t top) {
    constexpr int kPer = kF32 ? 4 : 8;
    constexpr uint32_t kBlock = 64 * kCount;
    static_assert(kBlock == 1024 && kFound <= kBlock, "groups of 16 to 64 lanes");
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, even = turn & 1;
    const uint32_t first = turn * kTurnVectors * kBlock + threadIdx.x;
    // With 64 groups of a row in no order and top 20, 24 elements reach the bound;
    // with 16 and 8, 11.  A turn with fewer vectors than threads has groups of fewer
    // lanes, enough of them for `top`.
    const uint32_t groups = top <= 8 ? 16 : top <= 16 ? 32 : 64;
    const uint32_t vectors = r.vectors() - turn * kTurnVectors * kBlock;
    uint32_t group = kBlock / groups;
    while (group > 1 && vectors < group * umax32(top, groups / 2)) group >>= 1;
    float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    most = most > -INFINITY ? most : -INFINITY;   // no NaN
    const float joined = lanes_reduce<Max>(most, group);
    if (threadIdx.x < groups * group && (threadIdx.x & (group - 1)) == 0)
        s.named[threadIdx.x / group] = joined;
    if (threadIdx.x == 0) s.count[even] = 0;
    __syncthreads();
    if (wave == 0) {   // a sort by all waves takes 0.7 us longer
        float x = lane < groups ? s.named[lane] : -INFINITY;
        if (groups == 16) sort_lanes<16>(x);
        else if (groups == 32) sort_lanes<32>(x);
        else sort_lanes<64>(x);
        const float bound = __uint_as_float(readlane_u32(__float_as_uint(x), top - 1));
        if (lane == 0) s.bound = begin ? bound : fmaxf(bound, s.least);
    }
    __syncthreads();
    const float bound = s.bound;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (!__ballot(m[q] >= bound)) continue;
        const word4 w = fresh(v[q]);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const float e = element<kF32>(w, k);
            if (!(e >= bound && e > -INFINITY)) continue;
            const uint32_t place = atomicAdd(&s.count[even], 1u);
            if (place < kFound) s.found[place] = key_of(e, r.first(first + q * kBlock) + k);
        }
    }
    __syncthreads();
    const uint32_t count = s.count[even];
    if (count <= 64) {
        if (wave == 0) {
            const uint64_t sorted = in_order(s, lane < count ? s.found[lane] : 0, count);
            list = begin ? sorted : merge_lists(list, sorted);
        }
    } else {
        uint64_t mine = 0;
        if (count <= kFound) {
            if (64 * wave < count) {
                mine = threadIdx.x < count ? s.found[threadIdx.x] : 0;
                sort_lanes(mine);
            }
        } else {   // more than that are equal, or nearly: each wave keeps a list
            uint64_t last = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const word4 w = fresh(v[q]);
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    const float e = element<kF32>(w, k);
                    if (!__ballot(e >= bound)) continue;
                    insert(mine, last,
                           e >= bound ? key_of(e, r.first(first + q * kBlock) + k) : 0, top);
                }
            }
        }
        s.lists[wave][lane] = mine;
        __syncthreads();
        if (wave == 0)
            for (uint32_t w = 0; w < kCount && (64 * w < count || count > kFound); ++w)
                list = merge_lists(list, s.lists[w][lane]);
    }
    if (wave == 0) {
        const uint64_t last = readlane_key(list, top - 1);
        if (lane == 0) s.least = last ? key_value(last) : -INFINITY;
    }
}

// ---- forward ---------------------------------------------------------------------------
// 2^d for a d of at most 0.  Close to 1 by its distance from it (a series of 2^d - 1), so that
// shifts of a row that rises all the way lose no more than one shift of the same height.
__device__ __forceinline__ double shift_by(float d) {
    const bool near = d > -1.0f / 32;
    const float less =
        d * fmaf(d, fmaf(d, fmaf(d, 9.61812911e-3f, 5.55041087e-2f), 0.240226507f), kLn2);
    return (double)(near ? less : exp2_fast(d)) + (near ? 1.0 : 0.0);
}
// The sums of threads of more than kLogprobChain turns, in 64 bits.  In LDS, as they are
// needed once in so many turns.
template <uint32_t kBlock>
struct LongSums {
    double s[kBlock], w[kBlock];
    float m[kBlock];

    // takes the thread's sums and leaves their maximum, by which they go on
    __device__ __forceinline__ void add(Sums &a, bool first, float c) {
        const uint32_t i = threadIdx.x;
        double ls = 0.0, lw = 0.0;
        if (!first) {
            const float d = (m[i] - reference(a.m)) * c;
            const double f = shift_by(d);
            ls = s[i];
            lw = f * fma((double)fmaxf(d, kNone), ls, w[i]);
            ls *= f;
        }
        s[i] = ls + a.s;
        w[i] = lw + a.w;
        m[i] = a.m;
        a.s = a.w = 0.0f;
    }
    __device__ __forceinline__ Sums sums() const {
        return Sums{m[threadIdx.x], (float)s[threadIdx.x], (float)w[threadIdx.x]};
    }
};
// A row's terms in one chain of fp32 drift where many are alike (in ln S 1e-5 for 131072 logits,
// 1e-2 for 2^28).  So they are added up by their vectors, those by their turn, the turns
// to the thread's sums, and these, after kLogprobChain of them (kLong), to LongSums.
template <bool kF32, bool kEntropy>
__device__ __forceinline__ void add_turn(Sums &a, const word4 (&v)[4], float m, float c) {
    constexpr int kPer = kF32 ? 4 : 8;
    shift(a, fmaxf(a.m, m), c);
    const float ref = reference(a.m);
    float s = 0.0f, w = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float vs = 0.0f, vw = 0.0f;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const float t = (element<kF32>(v[q], k) - ref) * c;
            const float e = exp2_fast(t);
            vs = k ? vs + e : e;
            if constexpr (kEntropy) vw = k ? vw + e * fmaxf(t, kNone) : e * fmaxf(t, kNone);
        }
        s = q ? s + vs : vs;
        if constexpr (kEntropy) w = q ? w + vw : vw;
    }
    a.s += s;
    if constexpr (kEntropy) a.w += w;
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

template <uint32_t kBlock, bool kF32, bool kEntropy, bool kTop, bool kKeep, bool kLong>
__global__ __launch_bounds__(kBlock, kTop ? 8 : 1) void logprob_kernel(LogprobArgs a) {
    constexpr uint32_t kCount = kBlock / 64;
    __shared__ float s_tmp[kCount][3];
    __shared__ TopShared<kTop ? kCount : 1> s_top;
    __shared__ LongSums<kLong ? kBlock : 1> s_long;
    constexpr uint32_t kPer = kF32 ? 4 : 8, kSize = kF32 ? 4 : 2;
    const uint32_t row = scalar_div(blockIdx.x, a.parts), part = blockIdx.x - row * a.parts;
    const RowVectors<kF32> r(row_ptr(a.logits, row, a.inner, kSize), a.vocab);
    const uint32_t turns = r.template turns<kBlock>();
    const uint32_t begin = part * a.part_turns;
    const uint32_t end = begin + a.part_turns < turns ? begin + a.part_turns : turns;
    // Few rows, hardly more than a turn each: the first one is not kept waiting for the
    // token.  Many: a row that is left out is not read, and a turn's vectors are
    // loaded a turn ahead.
    constexpr bool kWide = kBlock > kThreads;
    word4 v[4], next[4];
    auto load = [&](uint32_t turn) { load_turn<kBlock, kKeep>(kWide ? v : next, r, turn); };
    if (kWide && begin < end) load(begin);
    const int64_t token =
        load_id(row_ptr(a.tokens, row, a.inner, a.token_i32 ? 4 : 8), a.token_i32);
    if (token < 0) {
        if (part == 0) write_left_out(a, row);
        return;
    }
    if (!kWide && begin < end) load(begin);
    float own = 0.0f;   // the token's logit
    if (threadIdx.x == 0 && token < (int64_t)a.vocab) {
        if constexpr (kF32) own = ((const float *)r.row)[token];
        else own = __uint_as_float((uint32_t)((const uint16_t *)r.row)[token] << 16);
    }
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Sums mine = {-INFINITY, 0.0f, 0.0f};
    uint64_t list = 0;   // the first wave's
    for (uint32_t turn = begin; turn < end; ++turn) {
        if constexpr (!kWide) {
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = next[q];
            if (turn + 1 < end) load(turn + 1);
        }
        float m[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            m[q] = -INFINITY;
#pragma unroll
            for (int k = 0; k < (int)kPer; ++k) m[q] = fmaxf(m[q], element<kF32>(v[q], k));
        }
        if constexpr (kTop) add_largest(list, s_top, v, m, r, turn, turn == begin, a.top);
        const float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
        if constexpr (kTop) {
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = fresh(v[q]);
        }
        add_turn<kF32, kEntropy>(mine, v, most, a.scale);
        if constexpr (kWide) {
            if (turn + 1 < end) load(turn + 1);
        }
        if constexpr (kLong) {
            const uint32_t had = turn + 1 - begin;
            if (had % kLogprobChain == 0 || turn + 1 == end) {
                s_long.add(mine, had <= kLogprobChain, a.scale);
                if (turn + 1 == end) mine = s_long.sums();
            }
        }
    }
    Sums all = group_sums(mine, a.scale, s_tmp);
    if (a.parts == 1) {
        write_row<kEntropy>(a, row, all, token, own, list);
        return;
    }
    // the part's sums and list are handed over by returning device-scope atomics
    const uint32_t words = 2 + a.top;
    uint64_t *mine_at = a.partial + (uint64_t)blockIdx.x * words;
    uint64_t dep = 0;
    if (threadIdx.x < words) {   // the first wave, and two lanes more
        uint64_t w = list;
        if (threadIdx.x >= a.top)
            w = threadIdx.x == a.top ? (uint64_t)__float_as_uint(all.m) << 32 | __float_as_uint(all.s)
                                     : __float_as_uint(all.w);
        dep = __hip_atomic_exchange(mine_at + threadIdx.x, w, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!last_of(a.done + row, a.parts, dep)) return;
    const uint64_t *row_at = a.partial + (uint64_t)row * a.parts * words;
    mine = Sums{-INFINITY, 0.0f, 0.0f};
    for (uint32_t p = threadIdx.x; p < a.parts; p += kBlock) {
        const uint64_t *at = row_at + (uint64_t)p * words + a.top;
        const uint64_t ms = ld_relaxed_agent(at), w = ld_relaxed_agent(at + 1);
        merge(mine, Sums{__uint_as_float((uint32_t)(ms >> 32)), __uint_as_float((uint32_t)ms),
                         __uint_as_float((uint32_t)w)}, a.scale);
    }
    if constexpr (kTop) {
        // the parts' keys, 64 a wave in turn
        const uint32_t keys = a.parts * a.top;
        list = 0;
        for (uint32_t k = 64 * wave; k < keys; k += kBlock) {
            uint64_t key = 0;
            if (k + lane < keys) {
                const uint32_t p = (k + lane) / a.top;
                key = ld_relaxed_agent(row_at + (uint64_t)p * words + (k + lane - p * a.top));
            }
            sort_lanes(key);
            list = merge_lists(list, key);
        }
        s_top.lists[wave][lane] = list;
        __syncthreads();
        if (wave == 0)
            for (uint32_t w = 1; w < kCount && 64 * w < keys; ++w)
                list = merge_lists(list, s_top.lists[w][lane]);
    }
    all = group_sums(mine, a.scale, s_tmp);
    write_row<kEntropy>(a, row, all, token, own, list);
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
        const uint32_t i = turn * kTurnVectors * kThreads + threadIdx.x + q * kThreads;
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
    const uint32_t row = scalar_div(blockIdx.x, g.parts), part = blockIdx.x - row * g.parts;
    const int64_t token =
        load_id(row_ptr(g.tokens, row, g.inner, g.token_i32 ? 4 : 8), g.token_i32);
    uint8_t *out = const_cast<uint8_t *>(row_ptr(g.out, row, g.inner, kSize));
    const RowVectors<kF32> r(row_ptr(g.logits, row, g.inner, kSize), g.vocab);
    const uint32_t turns = r.template turns<kThreads>();
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
        load_turn<kThreads, false>(v, r, turn);
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
            const uint32_t id = r.first((turn * kTurnVectors + q) * kThreads + threadIdx.x);
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
hipError_t launch_forward(const LogprobArgs &a, bool wide, bool keep, hipStream_t stream) {
    // a long row is read with non-temporal loads; a wide one without alternatives is not long
    const bool lengthy = a.part_turns > kLogprobChain;
    auto *kernel =
        a.top ? (lengthy ? logprob_kernel<kLogprobWide, kF32, kEntropy, true, true, true>
                         : logprob_kernel<kLogprobWide, kF32, kEntropy, true, true, false>)
        : wide    ? logprob_kernel<kLogprobWide, kF32, kEntropy, false, true, false>
        : lengthy ? logprob_kernel<kThreads, kF32, kEntropy, false, false, true>
        : keep    ? logprob_kernel<kThreads, kF32, kEntropy, false, true, false>
                  : logprob_kernel<kThreads, kF32, kEntropy, false, false, false>;
    return launch_one(kernel, a.rows * a.parts, wide ? kLogprobWide : kThreads, a, 0, stream);
}

}  // namespace

hipError_t launch_logprob(const LogprobArgs &a, bool f32, bool wide, bool keep,
                          hipStream_t stream) {
    if (f32)
        return a.entropy ? launch_forward<true, true>(a, wide, keep, stream)
                         : launch_forward<true, false>(a, wide, keep, stream);
    return a.entropy ? launch_forward<false, true>(a, wide, keep, stream)
                     : launch_forward<false, false>(a, wide, keep, stream);
}

hipError_t launch_logprob_backward(const LogprobGradArgs &a, bool f32, hipStream_t stream) {
    auto *kernel = f32 ? (a.grad_entropy ? logprob_grad_kernel<true, true>
                                         : logprob_grad_kernel<true, false>)
                       : (a.grad_entropy ? logprob_grad_kernel<false, true>
                                         : logprob_grad_kernel<false, false>);
    return launch_one(kernel, a.rows * a.parts, kThreads, a, 0, stream);
}

}  // namespace bf16d
