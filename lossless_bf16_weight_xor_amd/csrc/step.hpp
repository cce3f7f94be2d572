// step.hpp -- shared definitions of the optimizer step's kernels and the host
// code that launches them (include/bf16delta_step.h).
#pragma once

#include <math.h>

#include "bf16delta_step.h"
#include "internal.hpp"

namespace bf16d {

// ---- gradient norm -------------------------------------------------------------
// Elements a workgroup reads per turn (32 bytes a thread in bf16, 64 in fp32),
// and workgroups at most, four for each of the 256 CUs.  Workgroup b takes turns
// b, b + grid, ..., counted from the first chunk, or from the last one where some
// are kept, and leaves one partial sum, so the grouping of the sums depends on
// the sizes alone.  1.75e9 bf16 gradients: 490 us (7.1 TB/s);
// with 2048 workgroups 536, with 768 569, with 512 814; with 8192 elements a
// turn 502 (1024 workgroups) and 484 (768), which leaves fewer turns to share
// out in smaller batches; with 2048 elements 741.  These were chosen on large
// batches.  In middle ones a fixed time shows that grows with the workgroups up
// to their most: 4.7 us for 2.7e5 bf16 elements (66 workgroups), 9.5 for 2e6
// (489), 17 for 8e6 and 23 for 3.2e7 (1024), where the launch and the read take
// 5, 5, 7 and 14.
constexpr uint32_t kNormChunk = 4096;
constexpr uint32_t kNormGrid = 1024;
// In batches up to kNormKeptTotal the chunks are read from the last one back to
// the first, and the first kNormKept bytes (the last-level cache's size) with
// loads that leave them in the caches, where the step that follows begins.
// Norm and step together, with and without: 6e7 bf16 gradients 276 and 291 us
// with 32-bit states, 179 and 191 with 8-bit ones; 2e8 fp32 ones 686 and 699.
// Larger batches keep too little of them, and are read faster from the first
// chunk on without (1.6 GB in bf16, 8-bit states: 1577 us, with 1600).
constexpr uint64_t kNormKept = 256u << 20;
constexpr uint64_t kNormKeptTotal = 1u << 30;

struct alignas(32) NormJob {
    BF16D_GMEM const void *grad;
    uint32_t chunk0;             // first chunk of this tensor
    uint32_t full_chunks, tail;  // full chunks, and the elements of the one after them
    uint32_t dtype;
};

struct NormArgs {
    const NormJob *jobs;
    const uint32_t *map;     // chunk -> job
    uint64_t *partial;       // kNormGrid bit patterns of doubles
    uint32_t *done;          // workgroups that have finished; 0 between calls
    bf16d_norm_result *result;
    uint32_t chunks;
    uint32_t kept;           // chunks from the first one that are left in the caches
    double max_norm, grad_scale;
};

// ---- AdamW ---------------------------------------------------------------------
constexpr uint32_t kAdamChunk = 4096;   // elements of an entry of the chunk -> job map
// A workgroup is one wave and does one turn, four elements a lane.  The step
// has up to four streams to read and four to write, and DRAM is fastest when
// the whole chip works close together in each of them: larger workgroups
// (128, 256 threads: 2 and 4 % slower on a 7B-shaped layer with 32-bit
// states) and ones that take several turns with their next loads in flight
// (4 to 8 % slower than 256 threads without) spread it further.
constexpr uint32_t kAdamThreads = 64;
constexpr uint32_t kAdamGroup = 4 * kAdamThreads;          // elements of a workgroup's turn
constexpr uint32_t kAdamSplit = kAdamChunk / kAdamGroup;   // workgroups of a chunk
constexpr uint32_t kAdamGrid = 1u << 25;   // workgroups at most: 2^31 threads
// For the same reason no more waves run on a CU than it takes to keep this many
// bytes of loads in flight there; the launch asks for LDS that it does not
// use, so that no more fit.  A 7B-shaped layer with 32-bit states, bf16
// gradients and master copies: 938 us without the limit, 914 with 64 KiB,
// 864 with 48, 886 with 40; four of them with fp32 gradients and their norm
// 4592, 4411, 4234 and 4350.  With 8-bit states the limit is worth 1 %, and
// without master copies it does not bind.
constexpr uint32_t kAdamFlight = 48 << 10;
constexpr uint32_t kLdsBytes = 160 << 10;   // of a CU
constexpr uint32_t kScaleBlock = 32;     // elements that share a scale byte
constexpr uint32_t kNumberSpan = 512;    // a job's element numbers start on a multiple of this

struct alignas(128) AdamJob {
    BF16D_GMEM const uint16_t *weights;
    BF16D_GMEM uint16_t *out;
    BF16D_GMEM float *master;
    BF16D_GMEM const void *grad;
    BF16D_GMEM void *m;
    BF16D_GMEM void *v;
    BF16D_GMEM uint8_t *m_scale;
    BF16D_GMEM uint8_t *v_scale;
    uint64_t number0;   // number of the tensor's first element
    uint32_t chunk0;    // its first chunk
    // Full chunks, and the elements of the one after them.  (Not n: ROCm 7.2's
    // compiler turns `left < chunk ? (uint32_t)left : chunk` of a uniform 64-bit
    // `left` into a scalar select on the carry of the subtraction before it,
    // which takes `chunk` for a tensor's end.  32-bit compares are selected as
    // they should.)
    uint32_t full_chunks, tail;
    float lr_scale, decay;   // decay: lr_scale * weight_decay
    uint32_t grad_dtype;
    uint64_t pad[2];
};
static_assert(sizeof(AdamJob) == 128, "AdamJob is one line");

// The numbers of a step that its rate and number decide.
struct StepNumbers {
    float rate;     // lr / c1, c_i = 1 - beta_i^step
    float lr;
    float root2;    // 1 / sqrt(c2)
    uint32_t key0, key1;   // of the random numbers
};
inline __host__ __device__ StepNumbers step_numbers(double lr, uint64_t step, uint64_t seed,
                                                    double log_beta1, double log_beta2) {
    StepNumbers n;
    n.lr = (float)lr;
    n.rate = (float)(lr / -expm1((double)step * log_beta1));
    n.root2 = (float)(1.0 / sqrt(-expm1((double)step * log_beta2)));
    auto mix = [](uint64_t z) {   // the SplitMix64 finaliser
        z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
        z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
        return z ^ (z >> 31);
    };
    const uint64_t key = mix(mix(seed) + step);
    n.key0 = (uint32_t)key;
    n.key1 = (uint32_t)(key >> 32);
    return n;
}

struct AdamArgs {
    const AdamJob *jobs;
    const uint32_t *map;    // chunk -> job
    const bf16d_norm_result *norm;
    const float *lr_device;
    const uint64_t *step_device;
    StepNumbers numbers;    // of the host's rate and step
    float beta1, beta2, rest1, rest2, eps;   // rest_i = 1 - beta_i
    // for numbers computed on the device
    double lr, log_beta1, log_beta2;
    uint64_t seed, step;
    uint32_t groups;   // chunks * kAdamSplit
};

// The table does not change while kernels run, so its entries are read as
// constants (scalar loads, though the kernel stores through other pointers).
template <typename T>
__device__ __forceinline__ T load_constant(const T *p) {
    struct Words {
        uint32_t w[sizeof(T) / 4];
    } x;
    auto *q = (const __attribute__((address_space(4))) uint32_t *)(uintptr_t)p;
#pragma unroll
    for (uint32_t k = 0; k < sizeof(T) / 4; ++k) x.w[k] = q[k];
    return __builtin_bit_cast(T, x);
}

// Launches a kernel of one argument and gives back the launch's own status:
// hipGetLastError would report an error that some earlier call left behind, of
// a step that has been enqueued.
template <typename Args>
hipError_t launch_one(void (*kernel)(Args), uint32_t grid, uint32_t threads, const Args &a,
                      uint32_t lds_bytes, hipStream_t stream) {
    void *args[] = {const_cast<Args *>(&a)};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3(grid), dim3(threads), args,
                           lds_bytes, stream);
}

hipError_t launch_grad_norm(const NormArgs &a, hipStream_t stream);
hipError_t launch_adamw(const AdamArgs &a, uint32_t state_bits, uint32_t lds_bytes,
                        hipStream_t stream);

}  // namespace bf16d
