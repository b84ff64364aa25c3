// state_cache.cu -- gdr_state_store / gdr_state_load: states in and out of an
// 8-bit cache.
//
// A row of a state (one key channel, dv values) has one scale: with a the
// row's largest magnitude, code = round(x 127 / a) and x' = code a / 127.
// 8 bits are a choice of the cache alone: the step of a row is 1/127 of its
// largest value, and what the recurrence runs on stays float32.
#include <math_constants.h>
#include <stdint.h>

#include "common.cuh"
#include "gdr.h"
#include "host_checks.h"

namespace gdr {
namespace {

constexpr float kInv127 = 1.f / 127.f;
constexpr float kTiny = 1e-30f;  // rows up to this are zeros: 127 / a stays finite

// One warp per row.
__global__ void gdr_state_store_kernel(const float *__restrict__ state,
                                       const int *__restrict__ slots,
                                       signed char *__restrict__ cache, float *__restrict__ scale,
                                       int n_slots, int HV, int dk, int dv, long long rows) {
    const long long row = (long long)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const long long per = (long long)HV * dk;  // rows of a state
    const int slot = slots[row / per];
    if (slot < 0 || slot >= n_slots) return;
    const float *x = state + row * dv;
    const long long out = (long long)slot * per + row % per;
    float top = 0.f;
    bool finite = true;
    for (int j = lane; j < dv; j += 32) {
        top = fmaxf(top, fabsf(x[j]));
        finite = finite && isfinite(x[j]);
    }
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    finite = __all_sync(0xffffffffu, finite);
    const bool held = finite && top > kTiny;
    const float inv = held ? __fmul_rn(127.f, __frcp_rn(top)) : 0.f;
    for (int j = lane; j < dv; j += 32)
        cache[out * dv + j] = held ? (signed char)__float2int_rn(__fmul_rn(x[j], inv)) : 0;
    if (lane == 0) scale[out] = !finite ? CUDART_NAN_F : held ? __fmul_rn(top, kInv127) : 0.f;
}

__global__ void gdr_state_load_kernel(const signed char *__restrict__ cache,
                                      const float *__restrict__ scale,
                                      const int *__restrict__ slots, float *__restrict__ state,
                                      int n_slots, int HV, int dk, int dv, long long rows) {
    const long long row = (long long)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const long long per = (long long)HV * dk;
    const int slot = slots[row / per];
    const bool known = slot >= 0 && slot < n_slots;
    const long long in = (long long)slot * per + row % per;
    for (int j = lane; j < dv; j += 32)
        state[row * dv + j] = known ? __fmul_rn((float)cache[in * dv + j], scale[in]) : 0.f;
}

gdr_status check(const void *state, const int *slots, const void *cache, const float *scale, int N,
                 int n_slots, int HV, int dk, int dv, bool store) {
    if (N < 0 || n_slots < 0 || HV <= 0) return GDR_ERR_SHAPE;
    if (!supported_dim(dk) || !supported_dim(dv)) return GDR_ERR_UNSUPPORTED;
    if ((long long)N * HV > (1LL << 30) || (long long)n_slots * HV > (1LL << 40))
        return GDR_ERR_SHAPE;
    if (N == 0) return GDR_OK;
    if (!state || !slots || (n_slots > 0 && (!cache || !scale))) return GDR_ERR_NULL;
    if (!aligned16(state) || !aligned16(cache) || !aligned4(slots) || !aligned4(scale))
        return GDR_ERR_ALIGN;
    const size_t rows = (size_t)HV * dk;
    const Range st = range_of(state, N * rows * dv * 4), sl = range_of(slots, (size_t)N * 4);
    const Range ca = range_of(cache, n_slots * rows * dv), sc = range_of(scale, n_slots * rows * 4);
    const bool clash = store ? overlap(ca, st) || overlap(ca, sl) || overlap(sc, st) ||
                                   overlap(sc, sl) || overlap(ca, sc)
                             : overlap(st, ca) || overlap(st, sc) || overlap(st, sl);
    return clash ? GDR_ERR_ALIAS : GDR_OK;
}

gdr_status done(cudaError_t e) {
    if (e == cudaSuccess) return GDR_OK;
    record_cuda_error(e);
    return GDR_ERR_CUDA;
}

constexpr int kWarps = 8;

}  // namespace
}  // namespace gdr

extern "C" GDR_API gdr_status gdr_state_store(const float *state, const int *slots,
                                              signed char *cache, float *scale, int N, int n_slots,
                                              int HV, int dk, int dv, void *stream) {
    using namespace gdr;
    const gdr_status st = check(state, slots, cache, scale, N, n_slots, HV, dk, dv, true);
    if (st != GDR_OK || N == 0 || n_slots == 0) return st;
    const long long rows = (long long)N * HV * dk;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    trace_begin(kKernStateStore, s);
    gdr_state_store_kernel<<<(unsigned)((rows + kWarps - 1) / kWarps), 32 * kWarps, 0, s>>>(
        state, slots, cache, scale, n_slots, HV, dk, dv, rows);
    trace_end(kKernStateStore, s);
    return done(cudaGetLastError());
}

extern "C" GDR_API gdr_status gdr_state_load(const signed char *cache, const float *scale,
                                             const int *slots, float *state, int N, int n_slots,
                                             int HV, int dk, int dv, void *stream) {
    using namespace gdr;
    const gdr_status st = check(state, slots, cache, scale, N, n_slots, HV, dk, dv, false);
    if (st != GDR_OK || N == 0) return st;
    const long long rows = (long long)N * HV * dk;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    trace_begin(kKernStateLoad, s);
    gdr_state_load_kernel<<<(unsigned)((rows + kWarps - 1) / kWarps), 32 * kWarps, 0, s>>>(
        cache, scale, slots, state, n_slots, HV, dk, dv, rows);
    trace_end(kKernStateLoad, s);
    return done(cudaGetLastError());
}
