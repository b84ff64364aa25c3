// short_conv.cu -- gdr_short_conv: a causal convolution of every channel with
// W taps over sequences of rows, with the state that the next rows need.
//
// out[t] = act(bias + sum_j w[:, j] x[t - W + 1 + j]).  A value is read and
// written once for 2 W + 4 operations: memory bounds it.  A thread holds VEC
// channels (16 bytes of a row in f32, 8 in bf16, whose 16 would take twice the
// registers), their taps and the last W - 1 rows in registers and walks `rows`
// rows of a sequence; kStep rows are in flight at a time.  The rows before its
// first are read again (W - 1 of `rows`).  65536 rows of 8192 channels in bf16
// take 328 us, 6.5 TB/s (468 us without the rows ahead; a copy runs at 6.8), where
// the issue slots are 62 % busy.  Channels in odd numbers or rows at odd distances
// are taken one a thread: 8192 rows of 8192 take 92 us so, 51 us by four.
#include <stdint.h>

#include "common.cuh"
#include "gdr.h"
#include "packed.cuh"
#include "sm100_ptx.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 128;
constexpr int kStep = 8;
constexpr int kMostRows = 64;

template <typename T, int VEC>
struct Vec;
template <>
struct Vec<float, 4> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(Raw r, float (&f)[4]) {
        f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y);
        f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ Raw pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
};
template <>
struct Vec<__nv_bfloat16, 4> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(Raw r, float (&f)[4]) {
        f[0] = __uint_as_float(r.x << 16);
        f[1] = __uint_as_float(r.x & 0xffff0000u);
        f[2] = __uint_as_float(r.y << 16);
        f[3] = __uint_as_float(r.y & 0xffff0000u);
    }
    static __device__ __forceinline__ Raw pack(const float (&f)[4]) {
        __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
        return make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
    }
    static __device__ __forceinline__ Raw zero() { return make_uint2(0, 0); }
};
template <>
struct Vec<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ void unpack(Raw r, float (&f)[1]) { f[0] = r; }
    static __device__ __forceinline__ Raw pack(const float (&f)[1]) { return f[0]; }
    static __device__ __forceinline__ Raw zero() { return 0.f; }
};
template <>
struct Vec<__nv_bfloat16, 1> {
    using Raw = __nv_bfloat16;
    static __device__ __forceinline__ void unpack(Raw r, float (&f)[1]) { f[0] = to_f32(r); }
    static __device__ __forceinline__ Raw pack(const float (&f)[1]) {
        return from_f32<__nv_bfloat16>(f[0]);
    }
    static __device__ __forceinline__ Raw zero() { return from_f32<__nv_bfloat16>(0.f); }
};

template <typename T, int W, int VEC, bool SILU>
__global__ void __launch_bounds__(kThreads)
    gdr_short_conv_kernel(const T *__restrict__ x, const float *__restrict__ w,
                          const float *__restrict__ bias, const T *s0, T *__restrict__ out, T *st,
                          int D, long long ldx, long long ldo, int rows, bool w16,
                          const __grid_constant__ SeqTable table) {
    using V = Vec<T, VEC>;
    using Raw = typename V::Raw;
    const int c = (blockIdx.y * kThreads + threadIdx.x) * VEC;
    if (c >= D) return;
    const SeqUnit u = find_unit(table, blockIdx.x);
    // rows count from the unit's first: a sequence may end where an int does
    const int r0 = u.unit * rows, n = min(u.len - r0, rows);
    x += (u.row0 + r0) * ldx + c;
    out += (u.row0 + r0) * ldo + c;
    const size_t state = (size_t)u.seq * (W - 1) * D + c;
    auto row = [&](int t) { return __ldg(reinterpret_cast<const Raw *>(x + t * ldx)); };

    // the rows before r0: units hold at least W - 1 rows, so that only the
    // first one looks into the state
    Raw before[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        if (r0 > 0)
            before[j] = row(j - (W - 1));
        else
            before[j] = s0 ? *reinterpret_cast<const Raw *>(s0 + state + (size_t)j * D) : V::zero();
    }
    float win[W - 1][VEC], tap[W][VEC], b[VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) V::unpack(before[j], win[j]);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        const float *q = w + (size_t)(c + v) * W;
        if (W == 4 && w16) {  // a channel's taps at once
            const float4 t = __ldg(reinterpret_cast<const float4 *>(q));
            tap[0][v] = t.x;
            tap[1][v] = t.y;
            tap[2][v] = t.z;
            tap[W - 1][v] = t.w;
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) tap[j][v] = __ldg(q + j);
        }
        b[v] = bias ? __ldg(bias + c + v) : 0.f;
    }
    // the new state: written by the thread that has read the old one, which it may replace
    if (st && u.unit == 0) {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int t = u.len - (W - 1) + i;
            Raw r = before[W - 2];
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                if (W - 1 + t == j) r = before[j];
            if (t >= 0) r = row(t);
            *reinterpret_cast<Raw *>(st + state + (size_t)i * D) = r;
        }
    }
    // kStep rows at a time, the next ones on their way meanwhile
    Raw in[kStep];
#pragma unroll
    for (int k = 0; k < kStep; ++k) in[k] = k < n ? row(k) : V::zero();
    for (int t0 = 0; t0 < n; t0 += kStep) {
        Raw next[kStep];
        const bool whole = t0 + 2 * kStep <= n;
#pragma unroll
        for (int k = 0; k < kStep; ++k)
            next[k] = whole || t0 + kStep + k < n ? row(t0 + kStep + k) : V::zero();
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            float f[VEC], y[VEC];
            V::unpack(in[k], f);
            if constexpr (VEC % 2 == 0) {
#pragma unroll
                for (int v = 0; v < VEC; v += 2) {
                    float2 q = make_float2(b[v], b[v + 1]);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j)
                        q = sm100::fma2(make_float2(tap[j][v], tap[j][v + 1]),
                                        make_float2(win[j][v], win[j][v + 1]), q);
                    q = sm100::fma2(make_float2(tap[W - 1][v], tap[W - 1][v + 1]),
                                    make_float2(f[v], f[v + 1]), q);
                    if (SILU) q = sm100::silu2(q);
                    y[v] = q.x;
                    y[v + 1] = q.y;
                }
            } else {
                y[0] = b[0];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) y[0] = fmaf(tap[j][0], win[j][0], y[0]);
                y[0] = fmaf(tap[W - 1][0], f[0], y[0]);
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (SILU && VEC % 2) y[v] = sm100::silu(y[v]);
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) win[j][v] = win[j + 1][v];
                win[W - 2][v] = f[v];
            }
            if (t0 + k < n) *reinterpret_cast<Raw *>(out + (t0 + k) * ldo) = V::pack(y);
        }
#pragma unroll
        for (int k = 0; k < kStep; ++k) in[k] = next[k];
    }
}

struct ConvArgs {
    const void *x, *s0;
    const float *w, *bias;
    void *out, *st;
    const int *cu;
    int N, T, D;
    long long ldx, ldo;
    bool silu;
};

template <typename T, int W, int VEC, bool SILU>
cudaError_t launch(const ConvArgs &a, int rows, cudaStream_t stream) {
    const unsigned ny = (unsigned)((a.D / VEC + kThreads - 1) / kThreads);
    return for_sequences(a.cu, a.N, a.T, rows, [&](const SeqTable &t, long long units) {
        trace_begin(kKernShortConv, stream);
        gdr_short_conv_kernel<T, W, VEC, SILU><<<dim3((unsigned)units, ny), kThreads, 0, stream>>>(
            static_cast<const T *>(a.x), a.w, a.bias, static_cast<const T *>(a.s0),
            static_cast<T *>(a.out), static_cast<T *>(a.st), a.D, a.ldx, a.ldo, rows,
            aligned16(a.w), t);
        trace_end(kKernShortConv, stream);
        return cudaGetLastError();
    });
}

template <typename T, int VEC>
cudaError_t by_width(const ConvArgs &a, int W, int rows, cudaStream_t s) {
    switch (W) {
        case 2: return a.silu ? launch<T, 2, VEC, true>(a, rows, s) : launch<T, 2, VEC, false>(a, rows, s);
        case 3: return a.silu ? launch<T, 3, VEC, true>(a, rows, s) : launch<T, 3, VEC, false>(a, rows, s);
        default: return a.silu ? launch<T, 4, VEC, true>(a, rows, s) : launch<T, 4, VEC, false>(a, rows, s);
    }
}

}  // namespace
}  // namespace gdr

extern "C" GDR_API gdr_status gdr_short_conv(const void *x, const float *w, const float *bias,
                                             const void *s0, void *out, void *st,
                                             const int *cu_seqlens, int N, int T, int D, int W,
                                             long long ldx, long long ldo, void *stream, int dtype,
                                             unsigned flags) {
    using namespace gdr;
    if (N < 0 || (!cu_seqlens && T < 0) || D <= 0 || ldx < D || ldo < D) return GDR_ERR_SHAPE;
    if (W < 2 || W > 4 || (dtype != GDR_F32 && dtype != GDR_BF16) || (flags & ~GDR_FLAG_SILU))
        return GDR_ERR_UNSUPPORTED;
    if (N == 0) return GDR_OK;
    if (cu_seqlens && check_offsets(cu_seqlens, N) != GDR_OK) return GDR_ERR_SHAPE;
    const long long total = cu_seqlens ? cu_seqlens[N] : (long long)N * T;
    const size_t es = dtype == GDR_BF16 ? 2 : 4;
    if (!rows_fit(total, ldx) || !rows_fit(total, ldo)) return GDR_ERR_SHAPE;
    if (!w || (total > 0 && (!x || !out))) return GDR_ERR_NULL;
    if (total == 0 && !st) return GDR_OK;
    const uintptr_t any = (uintptr_t)x | (uintptr_t)out | (uintptr_t)s0 | (uintptr_t)st;
    if ((any & (es - 1)) || !aligned4(w) || !aligned4(bias)) return GDR_ERR_ALIGN;
    const size_t state = (size_t)N * (W - 1) * D * es;
    const RowSet in = {x, D * es, ldx * es, total}, o = {out, D * es, ldo * es, total};
    const RowSet wr = packed_rows(w, (size_t)D * W * 4), br = packed_rows(bias, (size_t)D * 4);
    const RowSet r0 = packed_rows(s0, state), r1 = packed_rows(st, state);
    if (rows_overlap(o, in) || rows_overlap(o, wr) || rows_overlap(o, br) || rows_overlap(o, r0) ||
        rows_overlap(o, r1) || rows_overlap(r1, in) || rows_overlap(r1, wr) ||
        rows_overlap(r1, br) || (s0 != st && rows_overlap(r1, r0)))
        return GDR_ERR_ALIAS;
    const int vec = 4;
    const bool wide = D % vec == 0 && ldx % vec == 0 && ldo % vec == 0 && (any & (vec * es - 1)) == 0;
    // Rows of a thread: as many as leave every SM eight CTAs, at least W - 1.
    // 65536 rows of 8192 channels: 331 us by 64 (503 by 8, 347 by 32, 330 by 128);
    // 1141 rows of 1157: 4.7 us by 8 to 32, 6.3 by 64.
    const long long ny = (D / (wide ? vec : 1) + kThreads - 1) / kThreads;
    if (ny > 65535) return GDR_ERR_SHAPE;
    int rows = kMostRows;
    while (rows > kStep && count_units(cu_seqlens, N, T, rows) * ny < 152 * 8) rows /= 2;
    if (count_units(cu_seqlens, N, T, rows) > 0x7fffffffLL) return GDR_ERR_SHAPE;
    const ConvArgs a = {x, s0, w, bias, out, st, cu_seqlens, N, T, D, ldx, ldo,
                        (flags & GDR_FLAG_SILU) != 0};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == GDR_BF16)
        e = wide ? by_width<__nv_bfloat16, 4>(a, W, rows, s) : by_width<__nv_bfloat16, 1>(a, W, rows, s);
    else
        e = wide ? by_width<float, 4>(a, W, rows, s) : by_width<float, 1>(a, W, rows, s);
    if (e == cudaSuccess) return GDR_OK;
    record_cuda_error(e);
    return GDR_ERR_CUDA;
}
