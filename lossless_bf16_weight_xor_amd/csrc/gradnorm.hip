// gradnorm.hip -- the global L2 norm of a list of gradients, the factor that
// clips them to max_norm, and the non-finite flag, in one launch.
//
// norm = |c| sqrt(sum g^2).  One pass over the gradients, 2 or 4 bytes and
// one 64-bit multiply-add an element: bound by the read (7.1 TB/s for 1.75e9
// bf16 gradients, 6.8 to 7.1 for 9.7e8 fp32 ones).  The loads are non-temporal, 8 % faster than plain ones in a large
// batch, but for what the step that follows can find in the caches; the next
// turn's table entry is fetched a turn ahead.
#include "step.hpp"

namespace bf16d {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void add_square(double &s, uint32_t f32_bits) {
    const double d = (double)__uint_as_float(f32_bits);
    s = fma(d, d, s);
}

// kF32: 4 elements of a 16-byte word, else 8
template <bool kF32>
__device__ __forceinline__ void add_word(double (&s)[2], const u32x4 &w) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (kF32) {
            add_square(s[k & 1], w[k]);
        } else {
            add_square(s[0], w[k] << 16);
            add_square(s[1], w[k] & 0xFFFF0000u);
        }
    }
}

template <bool kKeep>
__device__ __forceinline__ u32x4 load_word(BF16D_GMEM const u32x4 *p) {
    if constexpr (kKeep) return *p;
    else return __builtin_nontemporal_load(p);
}

// kKeep: the words may stay in the caches
template <bool kF32, bool kKeep>
__device__ __forceinline__ void add_chunk(double (&s)[2], BF16D_GMEM const void *grad,
                                          uint64_t first, bool full, uint32_t count) {
    constexpr uint32_t kPer = kF32 ? 4 : 8;                       // elements of a word
    constexpr uint32_t kWords = kNormChunk / kPer / kThreads;     // words of a thread
    BF16D_GMEM const uint8_t *p =
        (BF16D_GMEM const uint8_t *)grad + first * (kF32 ? 4 : 2);
    if (full) {
        u32x4 w[kWords];
#pragma unroll
        for (uint32_t k = 0; k < kWords; ++k)
            w[k] = load_word<kKeep>((BF16D_GMEM const u32x4 *)p + k * kThreads + threadIdx.x);
#pragma unroll
        for (uint32_t k = 0; k < kWords; ++k) add_word<kF32>(s, w[k]);
        return;
    }
    const uint32_t words = count / kPer;
    for (uint32_t k = threadIdx.x; k < words; k += kThreads)
        add_word<kF32>(s, *((BF16D_GMEM const u32x4 *)p + k));
    // the last word's elements, one a thread
    const uint32_t i = words * kPer + threadIdx.x;
    if (threadIdx.x < kPer && i < count) {
        if constexpr (kF32) add_square(s[0], ((BF16D_GMEM const uint32_t *)p)[i]);
        else add_square(s[0], (uint32_t)((BF16D_GMEM const uint16_t *)p)[i] << 16);
    }
}

// the sum over the workgroup, in a fixed order; every thread gets it
__device__ __forceinline__ double group_sum(double v, double *s_tmp) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) s_tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) t += s_tmp[w];
    __syncthreads();
    return t;
}

// kKept: the batch's first chunks are left in the caches (its own kernel: the
// other one is 2 % slower with the choice in it)
template <bool kKept>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(NormArgs a) {
    __shared__ double s_tmp[kWaves];
    double s[2] = {0.0, 0.0};
    // turn t reads the t-th chunk, from the end where some are kept
    auto chunk_of = [&](uint32_t t) { return kKept ? a.chunks - 1 - t : t; };
    uint32_t t = blockIdx.x;
    uint32_t j = t < a.chunks ? load_constant(a.map + chunk_of(t)) : 0;
    while (t < a.chunks) {
        const NormJob J = load_constant(a.jobs + j);
        const uint32_t c = chunk_of(t);
        const uint32_t chunk = c - J.chunk0;   // of the tensor
        t += gridDim.x;
        if (t < a.chunks) j = load_constant(a.map + chunk_of(t));
        const uint64_t first = (uint64_t)chunk * kNormChunk;
        const bool full = chunk < J.full_chunks;
        if (J.dtype == BF16D_GRAD_F32) {
            if (kKept && c < a.kept) add_chunk<true, true>(s, J.grad, first, full, J.tail);
            else add_chunk<true, false>(s, J.grad, first, full, J.tail);
        } else {
            if (kKept && c < a.kept) add_chunk<false, true>(s, J.grad, first, full, J.tail);
            else add_chunk<false, false>(s, J.grad, first, full, J.tail);
        }
    }
    const double mine = group_sum(s[0] + s[1], s_tmp);
    // the partial sum is handed over by a returning device-scope atomic, as
    // last_workgroup asks
    uint64_t dep = 0;
    if (threadIdx.x == 0)
        dep = __hip_atomic_exchange(a.partial + blockIdx.x,
                                    (uint64_t)__double_as_longlong(mine), __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT);
    if (!last_workgroup(a.done, dep)) return;
    double all = 0.0;
    for (uint32_t b = threadIdx.x; b < gridDim.x; b += kThreads)
        all += __longlong_as_double((long long)ld_relaxed_agent(a.partial + b));
    const double sum = group_sum(all, s_tmp);
    if (threadIdx.x == 0) {
        const double norm = fabs(a.grad_scale) * sqrt(sum);
        a.result->norm = norm;
        a.result->scale =
            (float)(norm > a.max_norm ? a.grad_scale * (a.max_norm / norm) : a.grad_scale);
        // squares of finite floats and their sums stay far below the largest
        // double: the sum is infinite or NaN only where a gradient is
        a.result->nonfinite = !(sum <= 1.7976931348623157e308) ? 1u : 0u;
        __hip_atomic_store(a.done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

hipError_t launch_grad_norm(const NormArgs &a, hipStream_t stream) {
    const uint32_t grid =
        (uint32_t)(a.chunks < kNormGrid ? (a.chunks ? a.chunks : 1) : kNormGrid);
    auto *kernel = a.kept ? grad_norm_kernel<true> : grad_norm_kernel<false>;
    return launch_one(kernel, grid, kThreads, a, 0, stream);
}

}  // namespace bf16d
