// adamw.hip -- the AdamW step of every tensor of a checkpoint in one launch:
// new moments, new master weights and the new bf16 working copy from the old
// ones and the gradients (the formulas are in include/bf16delta_step.h).
//
// One pass, nothing is read twice: a thread holds four consecutive elements
// of every array at a time, so each access of a wave is one contiguous run (1 KiB of
// an fp32 array, 512 bytes of a bf16 one, 256 of a code array).  About 30
// flops against 10 to 30 bytes an element: bound by HBM.
//
// 8-bit states: a block of 32 elements is 8 neighbouring lanes, so its
// largest magnitude is three DPP steps inside a row of lanes, and no LDS is
// used.  The scale is a power of two: scaling and unscaling are exact, and
// only the rounding to the 3 mantissa bits of e4m3 loses anything.
#include "step.hpp"

namespace bf16d {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// The step's numbers, the same in every thread of a workgroup.
struct Scalars {
    float beta1, rest1, beta2, rest2;
    float root2;    // 1 / sqrt(c2)
    float eps;
    float rate;     // lr / c1
    float decay;    // lr * weight_decay
    float grad;     // the norm's scale, or 1
    uint32_t key0, key1;
};

// 32 random bits of the element numbered e
__device__ __forceinline__ uint32_t random_bits(uint64_t e, const Scalars &s) {
    uint32_t x = (uint32_t)e ^ s.key0;
    x = (x ^ (x >> 16)) * 0xBF58476Du + (s.key1 + (uint32_t)(e >> 32) * 0x9E3779B9u);
    x = (x ^ (x >> 15)) * 0x94D049BBu;
    return x ^ (x >> 16);
}

// Four elements at p, of which the first `valid` exist (the others read 0, and
// are not stored).
__device__ __forceinline__ f32x4 load_f32(BF16D_GMEM const float *p, uint32_t valid) {
    if (valid >= 4) return *(BF16D_GMEM const f32x4 *)p;
    f32x4 r = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
        if (k < valid) r[k] = p[k];
    return r;
}
__device__ __forceinline__ f32x4 load_bf16(BF16D_GMEM const uint16_t *p, uint32_t valid) {
    f32x4 r = {0, 0, 0, 0};
    if (valid >= 4) {
        const u32x2 w = *(BF16D_GMEM const u32x2 *)p;
        r[0] = __uint_as_float(w[0] << 16);
        r[1] = __uint_as_float(w[0] & 0xFFFF0000u);
        r[2] = __uint_as_float(w[1] << 16);
        r[3] = __uint_as_float(w[1] & 0xFFFF0000u);
        return r;
    }
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
        if (k < valid) r[k] = __uint_as_float((uint32_t)p[k] << 16);
    return r;
}
__device__ __forceinline__ uint32_t load_codes(BF16D_GMEM const uint8_t *p, uint32_t valid) {
    if (valid >= 4) return *(BF16D_GMEM const uint32_t *)p;
    uint32_t r = 0;
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
        if (k < valid) r |= (uint32_t)p[k] << (8 * k);
    return r;
}
__device__ __forceinline__ void store_f32(BF16D_GMEM float *p, const f32x4 &x, uint32_t valid) {
    if (valid >= 4) {
        *(BF16D_GMEM f32x4 *)p = x;
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
        if (k < valid) p[k] = x[k];
}
__device__ __forceinline__ void store_bf16(BF16D_GMEM uint16_t *p, const u32x2 &w,
                                           uint32_t valid) {
    if (valid >= 4) {
        *(BF16D_GMEM u32x2 *)p = w;
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
        if (k < valid) p[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
}
__device__ __forceinline__ void store_codes(BF16D_GMEM uint8_t *p, uint32_t c, uint32_t valid) {
    if (valid >= 4) {
        *(BF16D_GMEM uint32_t *)p = c;
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
        if (k < valid) p[k] = (uint8_t)(c >> (8 * k));
}

// four floats to bf16, nearest even
__device__ __forceinline__ u32x2 nearest_bf16(const f32x4 &x) {
    return __builtin_bit_cast(u32x2, __builtin_convertvector(x, bf16x4));
}
// one float to bf16, up where its low half and r carry; a NaN stays one (the
// carry could reach its sign bit)
__device__ __forceinline__ uint32_t random_bf16(float x, uint32_t r) {
    const uint32_t b = __float_as_uint(x);
    return x == x ? (b + r) >> 16 : (b >> 16) | 0x40u;
}

// e4m3 codes times the block's scale.  A scale byte of 0 reads as 0.
__device__ __forceinline__ f32x4 decode(uint32_t codes, uint32_t scale_byte) {
    const float s = __uint_as_float(scale_byte << 23);
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
    f32x4 r = {lo[0] * s, lo[1] * s, hi[0] * s, hi[1] * s};
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
constexpr uint32_t kCodeNaN = 0x7Fu;

// Four moments to codes.  Returns the codes, and the block's scale byte in
// `byte`: the smallest b >= 1 with max |x| <= 448 * 2^(b - 127).  448 is 1.75 * 2^8, so b
// is the exponent field of max |x| less 8, and one more where the mantissa
// field passes that of 1.75 (0x600000): a carry of the sum below.
// A magnitude t = |x| / scale of at least 2^-6 is a normal e4m3 number: its
// code is the top of the float's bits, rounded up where the 20 bits below
// the 3 mantissa bits and the 16 random bits above the last 4 of them carry
// (into the exponent where need be).  Below 2^-6 the step is 2^-9, and t is
// rounded in fixed point with 16 fraction bits.
// kPositive: a value above 0 gets at least code 1.
template <bool kPositive, int kRandomShift>
__device__ __forceinline__ uint32_t encode(const f32x4 &x, const uint32_t (&random)[4],
                                           uint32_t &byte) {
    uint32_t a[4], top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        a[k] = __float_as_uint(x[k]) & 0x7FFFFFFFu;
        top = umax32(top, a[k] < kInfBits ? a[k] : 0u);
    }
    top = block_max(top);
    const int b = (int)((top + 0x1FFFFFu) >> 23) - 8;
    byte = (uint32_t)(b > 1 ? b : 1);
    const float inverse = __uint_as_float((254u - byte) << 23);
    uint32_t codes = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float t = __uint_as_float(a[k]) * inverse;
        const uint32_t r = (random[k] >> kRandomShift) & 0xFFFFu;
        const uint32_t normal = ((__float_as_uint(t) + (r << 4)) >> 20) - (120u << 3);
        const uint32_t small = ((uint32_t)(fminf(t, 0.015625f) * 33554432.0f) + r) >> 16;
        uint32_t c = t >= 0.015625f ? normal : small;
        if constexpr (kPositive) c = (c == 0 && a[k] != 0) ? 1u : c;
        c = a[k] < kInfBits ? c : kCodeNaN;
        if constexpr (!kPositive) c |= (__float_as_uint(x[k]) >> 31) << 7;
        codes |= c << (8 * k);
    }
    return codes;
}

// The elements [first, first + 4 * kThreads * kVecs) of a job, four a thread
// and turn; those from J.n on do not exist.
template <int kBits, bool kF32, bool kMaster>
__device__ __forceinline__ void step_chunk(const AdamJob &J, uint64_t first, const Scalars &s) {
    constexpr uint32_t kVecs = 2;   // turns whose loads are in flight together
    for (uint32_t turn = 0; turn < kAdamChunk; turn += kVecs * 4 * kThreads) {
        f32x4 p[kVecs], g[kVecs], m[kVecs], v[kVecs];
        uint32_t mc[kVecs], vc[kVecs], ms[kVecs], vs[kVecs], valid[kVecs];
        uint64_t at[kVecs];
#pragma unroll
        for (uint32_t k = 0; k < kVecs; ++k) {
            at[k] = first + turn + 4 * (k * kThreads + threadIdx.x);
            const uint64_t left = at[k] < J.n ? J.n - at[k] : 0;
            valid[k] = left < 4 ? (uint32_t)left : 4u;
            const uint64_t i = valid[k] ? at[k] : 0;   // an address inside the arrays
            if constexpr (kF32)
                g[k] = load_f32((BF16D_GMEM const float *)J.grad + i, valid[k]);
            else
                g[k] = load_bf16((BF16D_GMEM const uint16_t *)J.grad + i, valid[k]);
            if constexpr (kMaster) p[k] = load_f32(J.master + i, valid[k]);
            else p[k] = load_bf16(J.weights + i, valid[k]);
            if constexpr (kBits == 8) {
                mc[k] = load_codes((BF16D_GMEM const uint8_t *)J.m + i, valid[k]);
                vc[k] = load_codes((BF16D_GMEM const uint8_t *)J.v + i, valid[k]);
                ms[k] = J.m_scale[i / kScaleBlock];
                vs[k] = J.v_scale[i / kScaleBlock];
            } else {
                m[k] = load_f32((BF16D_GMEM const float *)J.m + i, valid[k]);
                v[k] = load_f32((BF16D_GMEM const float *)J.v + i, valid[k]);
            }
        }
#pragma unroll
        for (uint32_t k = 0; k < kVecs; ++k) {
            if constexpr (kBits == 8) {
                m[k] = decode(mc[k], ms[k]);
                v[k] = decode(vc[k], vs[k]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float gq = g[k][q] * s.grad;
                m[k][q] = s.beta1 * m[k][q] + s.rest1 * gq;
                v[k][q] = s.beta2 * v[k][q] + s.rest2 * gq * gq;
                const float d = sqrtf(v[k][q]) * s.root2 + s.eps;
                // one rounding of p: decay and update are summed first
                p[k][q] -= s.decay * p[k][q] + s.rate * m[k][q] / d;
            }
            uint32_t random[4] = {0, 0, 0, 0};
            if constexpr (kBits == 8 || !kMaster) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    random[q] = random_bits(J.number0 + at[k] + q, s);
            }
            u32x2 w;
            if constexpr (kMaster) {
                w = nearest_bf16(p[k]);
            } else {
                uint32_t h[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    h[q] = random_bf16(p[k][q], (random[q] * 0x9E3779B1u) >> 16);
                w[0] = h[0] | h[1] << 16;
                w[1] = h[2] | h[3] << 16;
            }
            uint32_t mb = 0, vb = 0;
            if constexpr (kBits == 8) {
                // every lane takes part: lanes past the end hold zeros
                mc[k] = encode<false, 0>(m[k], random, mb);
                vc[k] = encode<true, 16>(v[k], random, vb);
            }
            store_bf16(J.out + at[k], w, valid[k]);
            if constexpr (kMaster) store_f32(J.master + at[k], p[k], valid[k]);
            if constexpr (kBits == 8) {
                store_codes((BF16D_GMEM uint8_t *)J.m + at[k], mc[k], valid[k]);
                store_codes((BF16D_GMEM uint8_t *)J.v + at[k], vc[k], valid[k]);
                if ((threadIdx.x & 7) == 0 && valid[k] != 0) {
                    J.m_scale[at[k] / kScaleBlock] = (uint8_t)mb;
                    J.v_scale[at[k] / kScaleBlock] = (uint8_t)vb;
                }
            } else {
                store_f32((BF16D_GMEM float *)J.m + at[k], m[k], valid[k]);
                store_f32((BF16D_GMEM float *)J.v + at[k], v[k], valid[k]);
            }
        }
    }
}

// A step that is left out: out gets the weights as they are.
__device__ void copy_chunk(const AdamJob &J, uint64_t first) {
    if (!J.master && (uintptr_t)J.out == (uintptr_t)J.weights) return;
    for (uint32_t turn = 0; turn < kAdamChunk; turn += 4 * kThreads) {
        const uint64_t at = first + turn + 4 * threadIdx.x;
        if (at >= J.n) return;
        const uint32_t valid = J.n - at < 4 ? (uint32_t)(J.n - at) : 4u;
        if (J.master) {
            store_bf16(J.out + at, nearest_bf16(load_f32(J.master + at, valid)), valid);
        } else {
            for (uint32_t k = 0; k < valid; ++k) J.out[at + k] = J.weights[at + k];
        }
    }
}

template <int kBits>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamArgs a) {
    const uint64_t c = blockIdx.x;
    const AdamJob &J = a.jobs[a.map[c]];
    const uint64_t first = (c - J.chunk0) * kAdamChunk;
    Scalars s;
    s.grad = 1.0f;
    if (a.norm) {
        if (a.norm->nonfinite) {
            copy_chunk(J, first);
            return;
        }
        s.grad = a.norm->scale;
    }
    double c1 = a.c1, c2 = a.c2, lr = a.lr;
    uint64_t step = a.step;
    if (a.lr_device) lr = (double)*a.lr_device;
    if (a.step_device) {
        step = *a.step_device ? *a.step_device : 1;
        c1 = -expm1((double)step * a.log_beta1);
        c2 = -expm1((double)step * a.log_beta2);
    }
    lr *= (double)J.lr_scale;
    s.beta1 = a.beta1;
    s.rest1 = a.rest1;
    s.beta2 = a.beta2;
    s.rest2 = a.rest2;
    s.root2 = (float)(1.0 / sqrt(c2));
    s.eps = a.eps;
    s.rate = (float)(lr / c1);
    s.decay = (float)(lr * (double)J.weight_decay);
    const uint64_t key = mix64(mix64(a.seed) + step);
    s.key0 = (uint32_t)key;
    s.key1 = (uint32_t)(key >> 32);
    const bool f32 = J.grad_dtype == BF16D_GRAD_F32;
    if (J.master) {
        if (f32) step_chunk<kBits, true, true>(J, first, s);
        else step_chunk<kBits, false, true>(J, first, s);
    } else {
        if (f32) step_chunk<kBits, true, false>(J, first, s);
        else step_chunk<kBits, false, false>(J, first, s);
    }
}

void launch_adamw(const AdamArgs &a, uint32_t chunks, uint32_t state_bits, hipStream_t stream) {
    if (chunks == 0) return;
    if (state_bits == 8) adamw_kernel<8><<<chunks, kThreads, 0, stream>>>(a);
    else adamw_kernel<32><<<chunks, kThreads, 0, stream>>>(a);
}

}  // namespace bf16d
