// adamw.hip -- the AdamW step of every tensor of a checkpoint in one launch:
// new moments, new master weights and the new bf16 working copy from the old
// ones and the gradients (the formulas are in include/bf16delta_step.h).
//
// One pass, nothing is read twice: a lane holds four consecutive elements of
// every array, so each access of a wave is one contiguous run (1 KiB of an
// fp32 array, 512 bytes of a bf16 one, 256 of a code array).  With master
// copies and bf16 gradients 17 vector instructions an element against 28 bytes
// (32-bit states), or 37 against 16 (8-bit ones): bound by HBM, at 6.6 and
// 6.3 TB/s for a 7B-shaped layer of 2.0e8 elements (860 and 519 us).  Without
// master copies 8-bit states leave 10 bytes for 40 instructions: 6.4 TB/s, with
// 83 % of the vector issue slots taken.
//
// 8-bit states: a block of 32 elements is 8 neighbouring lanes, so its
// largest magnitude is three DPP steps inside a row of lanes, and no LDS is
// used.  The scale is a power of two: scaling and unscaling are exact, and
// only the rounding to the 3 mantissa bits of e4m3 loses anything.  gfx950
// converts both ways with the scale, and rounds stochastically to e4m3 and
// bf16, in one instruction an element.  Written out in integer instructions
// (with correctly rounded root and quotient, and no separate path for full
// groups) the 8-bit step of that layer took 859 us.
#include "step.hpp"

namespace bf16d {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// Every array is read once and written once: non-temporal accesses (5 to 10 %
// faster than plain ones).
template <typename T>
__device__ __forceinline__ T load_once(BF16D_GMEM const void *p) {
    return __builtin_nontemporal_load((BF16D_GMEM const T *)p);
}
template <typename T>
__device__ __forceinline__ void store_once(BF16D_GMEM void *p, const T &x) {
    __builtin_nontemporal_store(x, (BF16D_GMEM T *)p);
}

// The step's numbers, the same in every thread of a workgroup.
struct Scalars {
    float beta1, rest1, beta2, rest2;
    float root2;    // 1 / sqrt(c2)
    float eps;
    float rate;     // lr / c1
    float decay;    // lr * the tensor's decay
    float grad;     // the norm's scale, or 1
    uint32_t key0, key1;
};

// 32 random bits for each of the lane's four elements, numbered
// first + 4 * lane + q.  first is a multiple of 256 and the same in the whole
// wave, so the bits of a number from the 8th on are, and with them the shifted
// word of the first mixing step; what q adds to its product is a scalar, too.
__device__ __forceinline__ void random_bits(uint32_t (&r)[4], uint64_t first, const Scalars &s) {
    static_assert(kAdamGroup == 256 && kNumberSpan % 256 == 0 && kAdamChunk % 256 == 0,
                  "a workgroup's first number is a multiple of 256");
    constexpr uint32_t kMul = 0xBF58476Du;
    const uint32_t x = (uint32_t)first ^ s.key0;
    const uint32_t y = x ^ (x >> 16);   // of element 0; element i has y ^ i
    const uint32_t add = s.key1 + (uint32_t)(first >> 32) * 0x9E3779B9u;
    const uint32_t product = (y ^ (4 * threadIdx.x)) * kMul;
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
        // kept apart by first_lane: the compiler would multiply for each element
        const uint32_t more = first_lane(add + (((y ^ q) & 3) - (y & 3)) * kMul);
        uint32_t z = product + more;
        z = (z ^ (z >> 15)) * 0x94D049BBu;
        r[q] = z ^ (z >> 16);
    }
}

// Four elements at p, of which the first `valid` exist (the others read 0, and
// are not stored); kFull: all four do.
template <bool kFull>
__device__ __forceinline__ f32x4 load_f32(BF16D_GMEM const float *p, uint32_t valid) {
    if (kFull || valid >= 4) return load_once<f32x4>(p);
    f32x4 r = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
        if (k < valid) r[k] = p[k];
    return r;
}
template <bool kFull>
__device__ __forceinline__ u32x2 load_16(BF16D_GMEM const uint16_t *p, uint32_t valid) {
    if (kFull || valid >= 4) return load_once<u32x2>(p);
    u32x2 r = {0, 0};
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
        if (k < valid) r[k >> 1] |= (uint32_t)p[k] << (16 * (k & 1));
    return r;
}
template <bool kFull>
__device__ __forceinline__ uint32_t load_codes(BF16D_GMEM const uint8_t *p, uint32_t valid) {
    if (kFull || valid >= 4) return load_once<uint32_t>(p);
    uint32_t r = 0;
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
        if (k < valid) r |= (uint32_t)p[k] << (8 * k);
    return r;
}
template <bool kFull>
__device__ __forceinline__ void store_f32(BF16D_GMEM float *p, const f32x4 &x, uint32_t valid) {
    if (kFull || valid >= 4) {
        store_once<f32x4>(p, x);
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
        if (k < valid) p[k] = x[k];
}
template <bool kFull>
__device__ __forceinline__ void store_16(BF16D_GMEM uint16_t *p, const u32x2 &w, uint32_t valid) {
    if (kFull || valid >= 4) {
        store_once<u32x2>(p, w);
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
        if (k < valid) p[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
}
template <bool kFull>
__device__ __forceinline__ void store_codes(BF16D_GMEM uint8_t *p, uint32_t c, uint32_t valid) {
    if (kFull || valid >= 4) {
        store_once<uint32_t>(p, c);
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
        if (k < valid) p[k] = (uint8_t)(c >> (8 * k));
}

__device__ __forceinline__ f32x4 widen(const u32x2 &w) {
    f32x4 r = {__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u),
               __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xFFFF0000u)};
    return r;
}
// four floats to bf16, nearest even
__device__ __forceinline__ u32x2 nearest_bf16(const f32x4 &x) {
    return __builtin_bit_cast(u32x2, __builtin_convertvector(x, bf16x4));
}
// four floats to bf16, up where a float's low half and the high half of its
// random word carry (the instruction adds just that half; NaN stays NaN)
__device__ __forceinline__ u32x2 random_bf16(const f32x4 &x, const uint32_t (&random)[4]) {
    bf16x2 lo = {}, hi = {};
    lo = __builtin_amdgcn_cvt_sr_bf16_f32(lo, x[0], random[0], false);
    lo = __builtin_amdgcn_cvt_sr_bf16_f32(lo, x[1], random[1], true);
    hi = __builtin_amdgcn_cvt_sr_bf16_f32(hi, x[2], random[2], false);
    hi = __builtin_amdgcn_cvt_sr_bf16_f32(hi, x[3], random[3], true);
    u32x2 r = {__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
    return r;
}

// e4m3 codes times the block's scale, exact for every byte from 0 to 254 whose
// value fp32 holds (2^128, the code of 256 under byte 247, and more become infinite)
__device__ __forceinline__ f32x4 decode(uint32_t codes, uint32_t scale_byte) {
    const float s = __uint_as_float(scale_byte << 23);
    const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, s, false);
    const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, s, true);
    f32x4 r = {lo[0], lo[1], hi[0], hi[1]};
    return r;
}

// the largest value of the 8 lanes of a block, in all of them
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
    v = umax32(v, dpp_src<0xB1>(v));    // quad_perm 1 0 3 2
    v = umax32(v, dpp_src<0x4E>(v));    // quad_perm 2 3 0 1
    v = umax32(v, dpp_src<0x141>(v));   // row_half_mirror
    return v;
}

constexpr uint32_t kInfBits = 0x7F800000u;

// The scale byte of a block whose largest finite magnitude has the bits `top`:
// the smallest b >= 1 with max |x| <= 448 * 2^(b - 127).  448 is 1.75 * 2^8, so b is
// the exponent field less 8, and one more where the mantissa field passes
// that of 1.75 (0x600000): a carry of the sum.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    const int b = (int)((top + 0x1FFFFFu) >> 23) - 8;
    return (uint32_t)(b > 1 ? b : 1);
}
__device__ __forceinline__ uint32_t finite_bits(uint32_t b) { return b < kInfBits ? b : 0u; }

// The conversion divides by the scale and adds the highest 20 bits of its
// random word below the 3 mantissa bits it keeps (in a number below 2^-6,
// below its last step of 2^-9); with 16 random bits above zeros that is the
// rounding of the definition.  Infinities and NaN become NaN.
__device__ __forceinline__ uint32_t to_codes(const f32x4 &x, const uint32_t (&r)[4], uint32_t byte) {
    const float scale = __uint_as_float(byte << 23);
    int c = 0;
    c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, x[0], r[0], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, x[1], r[1], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, x[2], r[2], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, x[3], r[3], scale, 3);
    return (uint32_t)c;
}

// Four of each moment to codes and the blocks' scale bytes.  Every lane of the
// wave takes part.  v has no signs (NaN aside); one above 0 gets at least
// code 1.
__device__ __forceinline__ void encode(const f32x4 &m, const f32x4 &v, const uint32_t (&random)[4],
                                       uint32_t &mc, uint32_t &vc, uint32_t &mb, uint32_t &vb) {
    uint32_t av[4], r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) av[k] = __float_as_uint(v[k]);
    // the largest |m| leaves NaN out by itself; as bits, for v, NaN is the largest
    uint32_t mt = block_max(__float_as_uint(
        fmaxf(fmaxf(fabsf(m[0]), fabsf(m[1])), fmaxf(fabsf(m[2]), fabsf(m[3])))));
    uint32_t vt = block_max(umax32(umax32(av[0], av[1]), umax32(av[2], av[3])));
    if (__ballot(umax32(mt, vt) >= kInfBits)) {   // wave-uniform, rare: leave them out
        mt = vt = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            mt = umax32(mt, finite_bits(__float_as_uint(m[k]) & 0x7FFFFFFFu));
            vt = umax32(vt, finite_bits(av[k]));
        }
        mt = block_max(mt);
        vt = block_max(vt);
    }
    mb = scale_byte(mt);
    vb = scale_byte(vt);
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = random[k] << 16;
    mc = to_codes(m, r, mb);
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = random[k] & 0xFFFF0000u;
    vc = to_codes(v, r, vb);
    if (__ballot(((vc - 0x01010101u) & ~vc & 0x80808080u) != 0)) {   // some code is 0
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (av[k] != 0 && ((vc >> (8 * k)) & 0xFFu) == 0) vc |= 1u << (8 * k);
    }
}

// A job's arrays from the first element of a workgroup's on.
struct Group {
    BF16D_GMEM const uint8_t *grad;
    BF16D_GMEM const uint16_t *weights;
    BF16D_GMEM uint16_t *out;
    BF16D_GMEM float *master;
    BF16D_GMEM uint8_t *m, *v, *m_scale, *v_scale;
    uint64_t number;   // of its first element
    uint32_t count;    // elements left in the tensor, at most kAdamGroup
};

// A thread's four elements.  kFull: they and everybody else's exist.
template <int kBits, bool kExact, bool kF32, bool kMaster, bool kFull>
__device__ __forceinline__ void step_four(const Group &c, const Scalars &s) {
    uint32_t i = 4 * threadIdx.x, valid = 4;
    if constexpr (!kFull) {
        valid = i < c.count ? (c.count - i < 4 ? c.count - i : 4u) : 0u;
        i = valid ? i : 0;   // an address inside the arrays
    }
    f32x4 p, g, m, v;
    u32x2 ph, gh;
    uint32_t mc, vc, ms, vs;
    if constexpr (kF32) g = load_f32<kFull>((BF16D_GMEM const float *)c.grad + i, valid);
    else gh = load_16<kFull>((BF16D_GMEM const uint16_t *)c.grad + i, valid);
    if constexpr (kMaster) p = load_f32<kFull>(c.master + i, valid);
    else ph = load_16<kFull>(c.weights + i, valid);
    if constexpr (kBits == 8) {
        mc = load_codes<kFull>(c.m + i, valid);
        vc = load_codes<kFull>(c.v + i, valid);
        ms = c.m_scale[i / kScaleBlock];
        vs = c.v_scale[i / kScaleBlock];
    } else {
        m = load_f32<kFull>((BF16D_GMEM const float *)c.m + i, valid);
        v = load_f32<kFull>((BF16D_GMEM const float *)c.v + i, valid);
    }
    uint32_t random[4];
    if constexpr (kBits == 8 || !kMaster) random_bits(random, c.number, s);
    if constexpr (!kF32) g = widen(gh);
    if constexpr (!kMaster) p = widen(ph);
    if constexpr (kBits == 8) {
        m = decode(mc, ms);
        v = decode(vc, vs);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float gq = g[q] * s.grad;
        m[q] = s.beta1 * m[q] + s.rest1 * gq;
        v[q] = s.beta2 * v[q] + s.rest2 * gq * gq;
        const float root = kExact ? sqrtf(v[q]) : __builtin_amdgcn_sqrtf(v[q]);
        const float d = root * s.root2 + s.eps;
        // one rounding of p: decay and update are summed first
        p[q] -= s.decay * p[q] + s.rate * (m[q] * __builtin_amdgcn_rcpf(d));
    }
    u32x2 w;
    if constexpr (kMaster) {
        w = nearest_bf16(p);
    } else {
        uint32_t r[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) r[q] = random[q] * 0x9E3779B1u;
        w = random_bf16(p, r);
    }
    store_16<kFull>(c.out + i, w, valid);
    if constexpr (kMaster) store_f32<kFull>(c.master + i, p, valid);
    if constexpr (kBits == 8) {
        uint32_t mb, vb;
        // lanes past the end hold zeros
        encode(m, v, random, mc, vc, mb, vb);
        store_codes<kFull>(c.m + i, mc, valid);
        store_codes<kFull>(c.v + i, vc, valid);
        if ((threadIdx.x & 7) == 0 && (kFull || valid != 0)) {
            c.m_scale[i / kScaleBlock] = (uint8_t)mb;
            c.v_scale[i / kScaleBlock] = (uint8_t)vb;
        }
    } else {
        store_f32<kFull>((BF16D_GMEM float *)c.m + i, m, valid);
        store_f32<kFull>((BF16D_GMEM float *)c.v + i, v, valid);
    }
}

template <int kBits, bool kExact, bool kF32, bool kMaster>
__device__ __forceinline__ void step_group(const AdamJob &J, uint64_t first, uint32_t count,
                                           const Scalars &s) {
    Group c;
    c.grad = (BF16D_GMEM const uint8_t *)J.grad + first * (kF32 ? 4 : 2);
    c.weights = J.weights + first;
    c.out = J.out + first;
    c.master = J.master + first;
    c.m = (BF16D_GMEM uint8_t *)J.m + first * (kBits / 8);
    c.v = (BF16D_GMEM uint8_t *)J.v + first * (kBits / 8);
    c.m_scale = J.m_scale + first / kScaleBlock;
    c.v_scale = J.v_scale + first / kScaleBlock;
    c.number = J.number0 + first;
    c.count = count;
    if (count == kAdamGroup) step_four<kBits, kExact, kF32, kMaster, true>(c, s);
    else step_four<kBits, kExact, kF32, kMaster, false>(c, s);
}

// A step that is left out: out gets the weights as they are.
__device__ __forceinline__ void copy_group(const AdamJob &J, uint64_t first, uint32_t count) {
    if (!J.master && (uintptr_t)J.out == (uintptr_t)J.weights) return;
    const uint32_t i = 4 * threadIdx.x;
    if (i >= count) return;
    const uint32_t valid = count - i < 4 ? count - i : 4u;
    const uint64_t at = first + i;
    const u32x2 w = J.master ? nearest_bf16(load_f32<false>(J.master + at, valid))
                             : load_16<false>(J.weights + at, valid);
    store_16<false>(J.out + at, w, valid);
}

template <int kBits, bool kExact>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(AdamArgs a) {
    uint32_t b = blockIdx.x;
    AdamJob J = load_constant(a.jobs + load_constant(a.map + b / kAdamSplit));
    Scalars s;
    s.grad = 1.0f;
    bool left_out = false;
    if (a.norm) {
        left_out = a.norm->nonfinite != 0;
        s.grad = a.norm->scale;
    }
    // Numbers in device words cost every wave its own double-precision arithmetic,
    // which shows where the vector units are nearly full: 2.0e8 elements with 8-bit
    // states and no master copies take 444 us for 329, in the other forms 1 to 3 %
    // more.
    StepNumbers n = a.numbers;
    if (a.lr_device || a.step_device) {
        uint64_t step = a.step;
        if (a.step_device) step = *a.step_device ? *a.step_device : 1;
        n = step_numbers(a.lr_device ? (double)*a.lr_device : a.lr, step, a.seed, a.log_beta1,
                         a.log_beta2);
    }
    s.beta1 = a.beta1;
    s.rest1 = a.rest1;
    s.beta2 = a.beta2;
    s.rest2 = a.rest2;
    s.eps = a.eps;
    s.root2 = n.root2;
    s.key0 = n.key0;
    s.key1 = n.key1;
    for (;;) {
        const uint32_t chunk = b / kAdamSplit - J.chunk0;   // of the tensor
        const uint32_t in_chunk = b % kAdamSplit * kAdamGroup;
        uint32_t count = kAdamGroup;
        if (chunk == J.full_chunks)
            count = in_chunk >= J.tail ? 0u
                    : J.tail - in_chunk < kAdamGroup ? J.tail - in_chunk : kAdamGroup;
        const uint64_t first = (uint64_t)chunk * kAdamChunk + in_chunk;
        s.rate = n.rate * J.lr_scale;
        s.decay = n.lr * J.decay;
        const bool f32 = J.grad_dtype == BF16D_GRAD_F32;
        if (count == 0) {
            // behind the tensor's end
        } else if (left_out) {
            copy_group(J, first, count);
        } else if (J.master) {
            if (f32) step_group<kBits, kExact, true, true>(J, first, count, s);
            else step_group<kBits, kExact, false, true>(J, first, count, s);
        } else {
            if (f32) step_group<kBits, kExact, true, false>(J, first, count, s);
            else step_group<kBits, kExact, false, false>(J, first, count, s);
        }
        // one turn is all, except beyond kAdamGrid workgroups
        b += gridDim.x;
        if (b >= a.groups) return;
        J = load_constant(a.jobs + load_constant(a.map + b / kAdamSplit));
    }
}

hipError_t launch_adamw(const AdamArgs &a, uint32_t state_bits, uint32_t lds_bytes,
                        hipStream_t stream) {
    if (a.groups == 0) return hipSuccess;
    const uint32_t grid = a.groups < kAdamGrid ? a.groups : kAdamGrid;
    // v_sqrt_f32 takes a denormal v for 0.  Its root, below 2^-63, times root2,
    // which 1 / sqrt(rest2) bounds, is then lost beside eps: less than u = 2^-24
    // of eps unless eps is tiny.
    const bool exact = a.eps * 0x1p39 < 1.0 / sqrt((double)a.rest2);
    auto *kernel = state_bits == 8 ? (exact ? adamw_kernel<8, true> : adamw_kernel<8, false>)
                                   : (exact ? adamw_kernel<32, true> : adamw_kernel<32, false>);
    return launch_one(kernel, grid, kAdamThreads, a, lds_bytes, stream);
}

}  // namespace bf16d
