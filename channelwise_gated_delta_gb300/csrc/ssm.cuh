// ssm.cuh -- what the kernels of the state space scan share.
#pragma once

#include "common.cuh"
#include "packed.cuh"

namespace gdr {

struct SsmArgs {
    const void *x, *b, *c, *z;              // z may be null
    const float *dt, *A, *D, *dt_bias, *h0;  // D, dt_bias, h0 may be null
    void *out;
    float *ht;                               // null: not stored
    // a walk cut into segments (units of a sequence): each unit's end state
    // from zero (the first one's from h0) and the log of its decay
    float *seg_state, *seg_log;
    long long ldx, ldb, ldc, ldz;
    int N, T, HK, HV, dk, dv;
    const int *cu;   // host
    int seg_rows;    // rows of a unit; INT_MAX: not cut
    int softplus;
    int bf16;
    int z_tma;  // z can be read by TMA (set by launch_ssm_chunks)
};

// step = softplus(dt + bias) (or dt + bias as it is)
__device__ __forceinline__ float ssm_step(float dt, float bias, int softplus) {
    const float r = dt + bias;
    return softplus ? fmaxf(r, 0.f) + log1pf(expf(-fabsf(r))) : r;
}
__device__ __forceinline__ float ssm_gate(float y, float z) { return y * (z / (1.f + expf(-z))); }

// pass 0: whole walks; 1: each unit's end state, no outputs; 2: the units
// with their outputs, from the starts that pass 1's states give
cudaError_t launch_ssm_walk(const SsmArgs &a, int pass, cudaStream_t stream);

// The same on the tensor cores, by chunks of 64 tokens (ssm_tc.cu): bf16, rows
// that TMA can read.
bool ssm_chunks_supported(const SsmArgs &a);
cudaError_t launch_ssm_chunks(const SsmArgs &a, int pass, cudaStream_t stream);

}  // namespace gdr
