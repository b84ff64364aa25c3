// qk_norm.cu -- gdr_qk_norm: norms of the heads of q and k, with the rotation
// of their first channels by the token's position in the same pass.
//
// A head of d values is held by d / 8 lanes, eight adjacent values each; the
// sum of squares is a shuffle reduction, the partner of a rotated channel (d_rot
// / 2 away, or its neighbour) another lane's value or the lane's own; where the
// whole head is rotated a lane holds four values and the four half a head on, and
// no pair is split.  Every value is read and written once: memory bounds it.
// 65536 rows of 2 x 16 heads of 128 in bf16 take 157 us, 6.8 TB/s (289 us with
// one group's loads in flight in place of kBatch, pairs in two lanes and an exact
// root; a copy runs at 6.8).  One token takes 2.1 us, which is a launch.
//
// Angles: a frequency is given in 2^-64 turns, and position times frequency
// in 64-bit integers wraps at whole turns, so that the angle's reduction is
// exact at any position; its top 32 bits as a float give sine and cosine to
// float accuracy.  A warp forms them once for a token and uses them for the
// heads that it walks.
#include <stdint.h>

#include <type_traits>

#include "common.cuh"
#include "gdr.h"
#include "packed.cuh"
#include "sm100_ptx.cuh"

namespace gdr {
namespace {

constexpr int kWarps = 4;
constexpr int kBatch = 4;  // groups of heads whose loads are in flight together

struct NormArgs {
    const void *q, *k;
    void *oq, *ok;
    const float *wq, *wk;
    const int *pos;
    const unsigned long long *freq;
    long long rows, ldq, ldk, ldoq, ldok;
    int HQ, HK, d_rot;
    int per_warp, parts;  // groups of heads a warp walks; warps of a row
    float eps, q_scale, inv_n;
};

// ROT: 0 none, 1 channel i with i + d_rot / 2, 2 channel 2 i with 2 i + 1,
// 3 as 1 with d_rot = d.  A lane holds 8 adjacent channels; in 3 it holds four
// and the four half a head on, so that pairs are its own.
template <typename T, int D, int ROT>
struct Lane {
    static constexpr int kSplit = ROT == 3 ? D / 2 : 4;
    static __device__ __forceinline__ int first(int l) { return ROT == 3 ? 4 * l : 8 * l; }
    using Raw = typename std::conditional<sizeof(T) == 2, uint2, float4>::type;
    Raw a, b;
    __device__ __forceinline__ void load(const T *p) {
        a = *reinterpret_cast<const Raw *>(p);
        b = *reinterpret_cast<const Raw *>(p + kSplit);
    }
    __device__ __forceinline__ void zero() { a = b = Raw{}; }
    static __device__ __forceinline__ void unpack4(uint2 r, float *f) {
        f[0] = __uint_as_float(r.x << 16);
        f[1] = __uint_as_float(r.x & 0xffff0000u);
        f[2] = __uint_as_float(r.y << 16);
        f[3] = __uint_as_float(r.y & 0xffff0000u);
    }
    static __device__ __forceinline__ void unpack4(float4 r, float *f) {
        f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
    }
    static __device__ __forceinline__ void pack4(const float *f, uint2 *r) {
        __nv_bfloat162 x = __floats2bfloat162_rn(f[0], f[1]), y = __floats2bfloat162_rn(f[2], f[3]);
        *r = make_uint2(*reinterpret_cast<uint32_t *>(&x), *reinterpret_cast<uint32_t *>(&y));
    }
    static __device__ __forceinline__ void pack4(const float *f, float4 *r) {
        *r = make_float4(f[0], f[1], f[2], f[3]);
    }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
        unpack4(a, f);
        unpack4(b, f + 4);
    }
    static __device__ __forceinline__ void store(T *p, const float (&f)[8]) {
        Raw x, y;
        pack4(f, &x);
        pack4(f + 4, &y);
        *reinterpret_cast<Raw *>(p) = x;
        *reinterpret_cast<Raw *>(p + kSplit) = y;
    }
};

// sine and cosine of t half turns, |t| <= 1: for bf16 outputs by the special
// function unit (off by 2^-21)
template <typename T>
__device__ __forceinline__ void turn(float t, float *sn, float *cs) {
    if (sizeof(T) == 2)
        __sincosf(t * 3.14159265358979f, sn, cs);
    else
        sincospif(t, sn, cs);
}

template <typename T, int D, int ROT>
__global__ void __launch_bounds__(32 * kWarps) gdr_qk_norm_kernel(const NormArgs a) {
    using V = Lane<T, D, ROT>;
    constexpr int L = D / 8, G = 32 / L;  // lanes of a head, heads of a warp's step
    const int lane = threadIdx.x & 31, sub = lane / L, l = lane % L;
    const long long w = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
    const long long row = w / a.parts;
    if (row >= a.rows) return;
    const int c = V::first(l);

    constexpr int P = ROT == 1 ? 8 : 4;  // pairs that this lane needs
    float cs[P], sn[P];
    const int half = a.d_rot / 2;
    const bool turned = ROT == 3 || (ROT && c < a.d_rot), upper = ROT == 1 && c >= half;
    if (ROT && turned) {
        const long long p = a.pos[row];
#pragma unroll
        for (int e = 0; e < P; ++e) {
            const int i = ROT == 1 ? (upper ? c - half : c) + e : ROT == 2 ? c / 2 + e : c + e;
            const unsigned long long turns = (unsigned long long)p * __ldg(a.freq + i);
            // the nearest 2^-32 of a turn, in half turns within [-1, 1)
            const int t = (int)(unsigned)((turns + 0x80000000ull) >> 32);
            turn<T>((float)t * 0x1p-31f, &sn[e], &cs[e]);
            if (ROT == 1 && !upper) sn[e] = -sn[e];
        }
    }
    const int from = upper ? l - half / 8 : l + half / 8;
    const int partner = sub * L + (ROT == 1 && turned ? from : l);

    // the warp's groups of heads: some of q, then some of k
    const int nq = (a.HQ + G - 1) / G, nk = (a.HK + G - 1) / G;
    const int g0 = (int)(w % a.parts) * a.per_warp, g1 = min(g0 + a.per_warp, nq + nk);
    auto walk = [&](const T *src, T *dst, const float *weight, int heads, float scale, int first,
                    int last) {
        if (first >= last) return;
        float wt[8];
        if (weight) {
#pragma unroll
            for (int e = 0; e < 8; ++e) wt[e] = __ldg(weight + c + (e < 4 ? e : V::kSplit + e - 4));
        }
        src += c;
        dst += c;
        for (int g = first; g < last; g += kBatch) {
            V v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int head = (g + k) * G + sub;
                if (g + k < last && head < heads)
                    v[k].load(src + head * D);
                else
                    v[k].zero();
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (g + k >= last) break;
                const int head = (g + k) * G + sub;
                float x[8];
                v[k].unpack(x);
                float2 q = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 y = make_float2(x[e], x[e + 1]);
                    q = sm100::fma2(y, y, q);
                }
                float s = q.x + q.y;
#pragma unroll
                for (int off = L / 2; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
                s = fmaf(s, a.inv_n, a.eps);
                // the approximate root, one step nearer; a head of zeros without
                // eps stays zeros, one whose sum is infinite becomes zeros
                float r = rsqrtf(s);
                r = fmaf(0.5f * r, fmaf(-s * r, r, 1.f), r);
                const float inv = s == 0.f || s == INFINITY ? 0.f : scale * r;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] *= inv;
                    if (weight) x[e] *= wt[e];
                }
                if (ROT == 1) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y = __shfl_sync(0xffffffffu, x[e], partner);
                        if (turned) x[e] = fmaf(x[e], cs[e % P], y * sn[e % P]);
                    }
                } else if (ROT == 2 && turned) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = x[2 * e], y = x[2 * e + 1];
                        x[2 * e] = fmaf(p, cs[e], -y * sn[e]);
                        x[2 * e + 1] = fmaf(y, cs[e], p * sn[e]);
                    }
                } else if (ROT == 3) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = x[e], y = x[4 + e];
                        x[e] = fmaf(p, cs[e], -y * sn[e]);
                        x[4 + e] = fmaf(y, cs[e], p * sn[e]);
                    }
                }
                if (head < heads) V::store(dst + head * D, x);
            }
        }
    };
    walk(static_cast<const T *>(a.q) + row * a.ldq, static_cast<T *>(a.oq) + row * a.ldoq, a.wq, a.HQ,
         a.q_scale, g0, min(g1, nq));
    walk(static_cast<const T *>(a.k) + row * a.ldk, static_cast<T *>(a.ok) + row * a.ldok, a.wk, a.HK,
         1.f, max(g0 - nq, 0), g1 - nq);
}

template <typename T, int D, int ROT>
cudaError_t launch(NormArgs a, cudaStream_t stream) {
    constexpr int G = 256 / D;
    const int groups = (a.HQ + G - 1) / G + (a.HK + G - 1) / G;
    // A warp walks all groups of a row where there are rows enough for eight warps an
    // SM, some of them otherwise (us, 24 groups of 128 / 4 of 64): 64 rows 2.7 / 2.5
    // in parts, 5 / 2.9 whole; 1141 rows 6.3 / 3.7 so, 6.5 / 4.6 in parts of one
    // group; 65536 rows 157 whole, 435 in parts (each forms the angles again).
    int parts = 1;
    while (parts < groups && a.rows * parts < 152 * 8) parts *= 2;
    if (parts > groups) parts = groups;
    a.per_warp = (groups + parts - 1) / parts;
    a.parts = (groups + a.per_warp - 1) / a.per_warp;
    const long long ctas = (a.rows * a.parts + kWarps - 1) / kWarps;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    trace_begin(kKernQkNorm, stream);
    gdr_qk_norm_kernel<T, D, ROT><<<(unsigned)ctas, 32 * kWarps, 0, stream>>>(a);
    trace_end(kKernQkNorm, stream);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t by_rotation(const NormArgs &a, bool interleaved, cudaStream_t s) {
    if (a.d_rot == 0) return launch<T, D, 0>(a, s);
    if (!interleaved && a.d_rot == D) return launch<T, D, 3>(a, s);
    return interleaved ? launch<T, D, 2>(a, s) : launch<T, D, 1>(a, s);
}

template <typename T>
cudaError_t by_dim(const NormArgs &a, int d, bool interleaved, cudaStream_t s) {
    switch (d) {
        case 32: return by_rotation<T, 32>(a, interleaved, s);
        case 64: return by_rotation<T, 64>(a, interleaved, s);
        case 128: return by_rotation<T, 128>(a, interleaved, s);
        default: return by_rotation<T, 256>(a, interleaved, s);
    }
}

}  // namespace
}  // namespace gdr

extern "C" GDR_API gdr_status gdr_qk_norm(const void *q, const void *k, const float *weight_q,
                                          const float *weight_k, const int *positions,
                                          const unsigned long long *freqs, void *out_q, void *out_k,
                                          long long rows, int HQ, int HK, int d, int d_rot,
                                          long long ldq, long long ldk, long long ldoq,
                                          long long ldok, float eps, float q_scale, void *stream,
                                          int dtype, unsigned flags) {
    using namespace gdr;
    if (rows < 0 || HQ <= 0 || HK <= 0 || !(eps >= 0.f)) return GDR_ERR_SHAPE;
    if ((d != 32 && d != 64 && d != 128 && d != 256) || (dtype != GDR_F32 && dtype != GDR_BF16) ||
        (flags & ~(GDR_FLAG_RMS_NORM | GDR_FLAG_ROPE_INTERLEAVED)))
        return GDR_ERR_UNSUPPORTED;
    if (d_rot < 0 || d_rot > d || d_rot % 16 != 0) return GDR_ERR_UNSUPPORTED;
    const long long wq = (long long)HQ * d, wk = (long long)HK * d;
    if (wq > 0x7fffffffLL || wk > 0x7fffffffLL || ldq < wq || ldk < wk || ldoq < wq || ldok < wk ||
        !rows_fit(rows, ldq) || !rows_fit(rows, ldk) || !rows_fit(rows, ldoq) ||
        !rows_fit(rows, ldok) || rows > (1LL << 40))
        return GDR_ERR_SHAPE;
    if (rows == 0) return GDR_OK;
    if (!q || !k || !out_q || !out_k || (d_rot > 0 && (!positions || !freqs))) return GDR_ERR_NULL;
    const int vec = dtype == GDR_BF16 ? 8 : 4;
    const size_t es = dtype == GDR_BF16 ? 2 : 4;
    if (!aligned16(q) || !aligned16(k) || !aligned16(out_q) || !aligned16(out_k) ||
        !aligned4(weight_q) || !aligned4(weight_k) || !aligned4(positions) ||
        ((uintptr_t)freqs & 7u) || ldq % vec || ldk % vec || ldoq % vec || ldok % vec)
        return GDR_ERR_ALIGN;
    const RowSet in[2] = {{q, wq * es, ldq * es, rows}, {k, wk * es, ldk * es, rows}};
    const RowSet out[2] = {{out_q, wq * es, ldoq * es, rows}, {out_k, wk * es, ldok * es, rows}};
    const RowSet other[4] = {packed_rows(weight_q, d * 4), packed_rows(weight_k, d * 4),
                             d_rot ? packed_rows(positions, rows * 4) : RowSet{},
                             d_rot ? packed_rows(freqs, d_rot / 2 * 8) : RowSet{}};
    if (rows_overlap(out[0], out[1])) return GDR_ERR_ALIAS;
    for (int i = 0; i < 2; ++i) {
        for (int j = 0; j < 2; ++j) {
            const bool in_place = i == j && in[j].p == out[i].p && in[j].ld == out[i].ld;
            if (!in_place && rows_overlap(out[i], in[j])) return GDR_ERR_ALIAS;
        }
        for (int j = 0; j < 4; ++j)
            if (rows_overlap(out[i], other[j])) return GDR_ERR_ALIAS;
    }
    const NormArgs a = {q, k, out_q, out_k, weight_q, weight_k, positions, freqs, rows, ldq, ldk,
                        ldoq, ldok, HQ, HK, d_rot, 0, 0, eps, q_scale,
                        (flags & GDR_FLAG_RMS_NORM) ? 1.f / d : 1.f};
    const bool il = (flags & GDR_FLAG_ROPE_INTERLEAVED) != 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == GDR_BF16 ? by_dim<__nv_bfloat16>(a, d, il, s)
                                            : by_dim<float>(a, d, il, s);
    if (e == cudaSuccess) return GDR_OK;
    record_cuda_error(e);
    return GDR_ERR_CUDA;
}
