// step.hpp -- shared definitions of the optimizer step's kernels and the host
// code that launches them (include/bf16delta_step.h).
#pragma once

#include "bf16delta_step.h"
#include "internal.hpp"

namespace bf16d {

// ---- gradient norm -------------------------------------------------------------
// Elements a workgroup reads per turn: 64 bytes a thread in bf16 (four
// 16-byte loads in flight), 128 in fp32.
constexpr uint32_t kNormChunk = 8192;
// Workgroups at most: 8 for each of the 256 CUs.  Each leaves one partial
// sum, and workgroup b always takes chunks b, b + grid, ..., so the grouping
// of the sums depends on the sizes alone.
constexpr uint32_t kNormGrid = 2048;

struct alignas(32) NormJob {
    BF16D_GMEM const void *grad;
    uint64_t n;
    uint64_t chunk0;   // first chunk of this tensor
    uint32_t dtype;
    uint32_t pad;
};

struct NormArgs {
    const NormJob *jobs;
    const uint32_t *map;     // chunk -> job
    uint64_t *partial;       // kNormGrid bit patterns of doubles
    uint32_t *done;          // workgroups that have finished; 0 between calls
    bf16d_norm_result *result;
    uint64_t chunks;
    double max_norm, grad_scale;
};

// ---- AdamW ---------------------------------------------------------------------
constexpr uint32_t kAdamChunk = 4096;    // elements of one workgroup: 16 a thread
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
    uint64_t n;
    uint64_t chunk0;    // first chunk of this tensor
    uint64_t number0;   // number of its first element
    float lr_scale, weight_decay;
    uint32_t grad_dtype, pad;
};
static_assert(sizeof(AdamJob) == 128, "AdamJob is one line");

struct AdamArgs {
    const AdamJob *jobs;
    const uint32_t *map;    // chunk -> job
    const bf16d_norm_result *norm;
    const float *lr_device;
    const uint64_t *step_device;
    double lr, log_beta1, log_beta2, c1, c2;   // c_i = 1 - beta_i^step
    float beta1, beta2, rest1, rest2, eps;     // rest_i = 1 - beta_i
    uint64_t seed, step;
};

void launch_grad_norm(const NormArgs &a, hipStream_t stream);
void launch_adamw(const AdamArgs &a, uint32_t chunks, uint32_t state_bits, hipStream_t stream);

}  // namespace bf16d
