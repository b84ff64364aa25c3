// state_cache.cu -- gdr_state_store / gdr_state_load: states in and out of an
// 8-bit cache.
//
// A row of a state (one key channel, dv values) has one scale: with a the
// row's largest magnitude, code = round(x 127 / a) and x' = code a / 127.
// 8 bits are a choice of the cache alone: the step of a row is 1/127 of its
// largest value, and what the recurrence runs on stays float32.
//
// Both directions are one pass over memory (5 bytes an element), and bound by
// it.  A lane holds four columns of a row, dv / 4 lanes the row, and a warp
// kSteps such groups of rows, whose loads are all in flight at once.
// Measured for states of 128 x 128 on the device: storing 64 x 32 heads and
// loading them again 48.3 us (338 MB at 7.0 TB/s: the codes are still in L2
// when they are loaded), loading 128 x 32 heads, 17 of them new, 49.4 us (328 MB at
// 6.6 TB/s, 0.98 of a copy's rate).  With one row in flight a warp they took 97
// and 74 us.
#include <stdint.h>

#include "common.cuh"
#include "gdr.h"
#include "host_checks.h"

namespace gdr {
namespace {

constexpr float kInv127 = 1.f / 127.f;
constexpr float kTiny = 1e-30f;  // rows up to this are zeros: 127 / a stays finite
constexpr int kWarps = 8;
constexpr int kSteps = 8;

// Largest bit pattern over the L lanes that hold a row.
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
    if constexpr (L == 32) {
        x = __reduce_max_sync(0xffffffffu, x);
    } else {
#pragma unroll
        for (int off = L / 2; off; off >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, off));
    }
    return x;
}

// Four values within [-127, 127] rounded to whole numbers (ties to even) and
// packed as bytes: added to 1.5 * 2^23 a value's rounding is the addition's,
// and its two's complement the sum's low byte.
__device__ __forceinline__ uint32_t pack4(float4 x, float inv) {
    constexpr float kMagic = 12582912.f;
    const uint32_t a = __float_as_uint(__fadd_rn(__fmul_rn(x.x, inv), kMagic));
    const uint32_t b = __float_as_uint(__fadd_rn(__fmul_rn(x.y, inv), kMagic));
    const uint32_t c = __float_as_uint(__fadd_rn(__fmul_rn(x.z, inv), kMagic));
    const uint32_t d = __float_as_uint(__fadd_rn(__fmul_rn(x.w, inv), kMagic));
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Byte e of four codes as a float: with its top bit flipped the byte is
// code + 128, and the low byte of 2^23 + code + 128.
__device__ __forceinline__ float unpack1(uint32_t flipped, int e) {
    return __fadd_rn(__uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7440 | e)), -8388736.f);
}

// A warp: kSteps groups of 32 / L rows, all of one state (dk is a multiple of
// the rows of a warp).
template <int DV>
struct Rows {
    static constexpr int L = DV / 4;            // lanes of a row
    static constexpr int kGroup = 32 / L;       // rows of a load
    static constexpr int kWarpRows = kGroup * kSteps;
};

template <int DV>
__global__ void __launch_bounds__(32 * kWarps)
    gdr_state_store_kernel(const float *__restrict__ state, const int *__restrict__ slots,
                           signed char *__restrict__ cache, float *__restrict__ scale, int n_slots,
                           unsigned state_warps, unsigned warps) {
    using R = Rows<DV>;
    const int lane = threadIdx.x & 31, sub = lane / R::L;
    const unsigned w = blockIdx.x * kWarps + threadIdx.x / 32, n = w / state_warps;
    if (w >= warps) return;
    const size_t row0 = (size_t)w * R::kWarpRows;
    const float *x = state + (row0 + sub) * DV + 4 * (lane % R::L);
    float4 v[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) v[s] = ldg_stream4(x + s * R::kGroup * DV);
    const int slot = slots[n];
    if (slot < 0 || slot >= n_slots) return;
    const size_t out = ((size_t)slot * state_warps + (w - n * state_warps)) * R::kWarpRows + sub;
    signed char *c = cache + out * DV + 4 * (lane % R::L);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        // magnitudes as bit patterns: ordered like the numbers, infinities
        // and NaN above all of them
        const uint32_t m = 0x7fffffffu;
        const uint32_t top = row_max<R::L>(
            max(max(__float_as_uint(v[s].x) & m, __float_as_uint(v[s].y) & m),
                max(__float_as_uint(v[s].z) & m, __float_as_uint(v[s].w) & m)));
        const float a = __uint_as_float(top);
        const bool finite = top < 0x7f800000u, held = finite && a > kTiny;
        const float inv = held ? __fmul_rn(127.f, __frcp_rn(a)) : 0.f;
        const uint32_t codes = held ? pack4(v[s], inv) : 0u;
        *reinterpret_cast<uint32_t *>(c + s * R::kGroup * DV) = codes;
        if (lane % R::L == 0)
            scale[out + s * R::kGroup] = !finite ? __uint_as_float(0x7fffffffu)
                                         : held  ? __fmul_rn(a, kInv127)
                                                 : 0.f;
    }
}

template <int DV>
__global__ void __launch_bounds__(32 * kWarps)
    gdr_state_load_kernel(const signed char *__restrict__ cache, const float *__restrict__ scale,
                          const int *__restrict__ slots, float *__restrict__ state, int n_slots,
                          unsigned state_warps, unsigned warps) {
    using R = Rows<DV>;
    const int lane = threadIdx.x & 31, sub = lane / R::L;
    const unsigned w = blockIdx.x * kWarps + threadIdx.x / 32, n = w / state_warps;
    if (w >= warps) return;
    const size_t row0 = (size_t)w * R::kWarpRows;
    const int slot = slots[n];
    float *x = state + (row0 + sub) * DV + 4 * (lane % R::L);
    if (slot < 0 || slot >= n_slots) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            stg_stream4(x + s * R::kGroup * DV, make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }
    const size_t in = ((size_t)slot * state_warps + (w - n * state_warps)) * R::kWarpRows + sub;
    const signed char *c = cache + in * DV + 4 * (lane % R::L);
    uint32_t codes[kSteps];
    float sc[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        codes[s] = __ldg(reinterpret_cast<const uint32_t *>(c + s * R::kGroup * DV));
        sc[s] = __ldg(scale + in + s * R::kGroup);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const uint32_t f = codes[s] ^ 0x80808080u;
        float4 y;
        y.x = __fmul_rn(unpack1(f, 0), sc[s]);
        y.y = __fmul_rn(unpack1(f, 1), sc[s]);
        y.z = __fmul_rn(unpack1(f, 2), sc[s]);
        y.w = __fmul_rn(unpack1(f, 3), sc[s]);
        stg_stream4(x + s * R::kGroup * DV, y);
    }
}

template <int DV>
cudaError_t launch_store(const float *state, const int *slots, signed char *cache, float *scale,
                         int N, int n_slots, int HV, int dk, cudaStream_t stream) {
    const unsigned state_warps = (unsigned)((long long)HV * dk / Rows<DV>::kWarpRows);
    const unsigned warps = (unsigned)N * state_warps;  // at most 2^30 (check())
    trace_begin(kKernStateStore, stream);
    gdr_state_store_kernel<DV><<<(warps + kWarps - 1) / kWarps, 32 * kWarps, 0, stream>>>(
        state, slots, cache, scale, n_slots, state_warps, warps);
    trace_end(kKernStateStore, stream);
    return cudaGetLastError();
}

template <int DV>
cudaError_t launch_load(const signed char *cache, const float *scale, const int *slots,
                        float *state, int N, int n_slots, int HV, int dk, cudaStream_t stream) {
    const unsigned state_warps = (unsigned)((long long)HV * dk / Rows<DV>::kWarpRows);
    const unsigned warps = (unsigned)N * state_warps;  // at most 2^30 (check())
    trace_begin(kKernStateLoad, stream);
    gdr_state_load_kernel<DV><<<(warps + kWarps - 1) / kWarps, 32 * kWarps, 0, stream>>>(
        cache, scale, slots, state, n_slots, state_warps, warps);
    trace_end(kKernStateLoad, stream);
    return cudaGetLastError();
}

gdr_status check(const void *state, const int *slots, const void *cache, const float *scale, int N,
                 int n_slots, int HV, int dk, int dv, bool store) {
    if (N < 0 || n_slots < 0 || HV <= 0) return GDR_ERR_SHAPE;
    if (!supported_dim(dk) || !supported_dim(dv)) return GDR_ERR_UNSUPPORTED;
    // states of at least 4 KB: no device holds 2^26 heads; their warps then fit 32 bits
    if ((long long)N * HV > (1LL << 26) || (long long)n_slots * HV > (1LL << 40))
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

}  // namespace
}  // namespace gdr

extern "C" GDR_API gdr_status gdr_state_store(const float *state, const int *slots,
                                              signed char *cache, float *scale, int N, int n_slots,
                                              int HV, int dk, int dv, void *stream) {
    using namespace gdr;
    const gdr_status st = check(state, slots, cache, scale, N, n_slots, HV, dk, dv, true);
    if (st != GDR_OK || N == 0 || n_slots == 0) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dv) {
        case 32: return done(launch_store<32>(state, slots, cache, scale, N, n_slots, HV, dk, s));
        case 64: return done(launch_store<64>(state, slots, cache, scale, N, n_slots, HV, dk, s));
        default: return done(launch_store<128>(state, slots, cache, scale, N, n_slots, HV, dk, s));
    }
}

extern "C" GDR_API gdr_status gdr_state_load(const signed char *cache, const float *scale,
                                             const int *slots, float *state, int N, int n_slots,
                                             int HV, int dk, int dv, void *stream) {
    using namespace gdr;
    const gdr_status st = check(state, slots, cache, scale, N, n_slots, HV, dk, dv, false);
    if (st != GDR_OK || N == 0) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dv) {
        case 32: return done(launch_load<32>(cache, scale, slots, state, N, n_slots, HV, dk, s));
        case 64: return done(launch_load<64>(cache, scale, slots, state, N, n_slots, HV, dk, s));
        default: return done(launch_load<128>(cache, scale, slots, state, N, n_slots, HV, dk, s));
    }
}
