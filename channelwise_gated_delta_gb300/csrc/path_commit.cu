// path_commit.cu -- gdr_commit_path: the state after the accepted nodes of a
// draft.
//
// Each node on the path takes the token recurrence's step without its output:
//     s_ij <- a_i s_ij            a_i = exp(g_i)
//     d_j   = beta (v_j - sum_i k_i s_ij)
//     s_ij <- s_ij + k_i d_j
// The columns j of a state never meet, so the state is cut along them and
// stays in registers over the whole path: read once, written once, which is
// what bounds the call for paths of up to about ten nodes (three operations an element
// and node against eight bytes an element).
//
// A warp owns 16 columns of a head's state: lane (cq = lane % 4, rg = lane /
// 4) holds columns 4 cq .. 4 cq + 3 of the rows rg + 8 m.  A row's 16 columns
// are 64 contiguous bytes, the sum over the rows stays inside the warp, and
// between the nodes no warp waits for another.  The arithmetic is on pairs of
// columns (fma.rn.f32x2: two roundings as by two fma).  k and exp(g) of a
// batch of nodes are staged in shared memory as (k, k, a, a), the pairs' form.
#include <stdint.h>

#include "common.cuh"
#include "gdr.h"
#include "host_checks.h"

namespace gdr {
namespace {

constexpr int kNodes = 8;      // nodes staged at a time
constexpr int kWarpCols = 16;  // columns of a warp

struct Pair {
    unsigned long long v;
};
__device__ __forceinline__ Pair pair(float x, float y) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ float2 split(Pair p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p.v));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// One CTA: BV columns of one head (BV / 16 warps).
template <typename Tin, int DK, int BV, bool GS>
__global__ void __launch_bounds__(2 * BV, BV == 64 ? 4 : 8)
    gdr_commit_kernel(const Tin *__restrict__ k, const Tin *__restrict__ v,
                      const float *__restrict__ g, const float *__restrict__ beta,
                      const float *h0, float *ht, const int *__restrict__ path,
                      const int *__restrict__ n_path, int T, int HK, int HV, int dv,
                      int max_path) {
    constexpr int NT = 2 * BV, RM = DK / 8;
    __shared__ float4 s_ka[kNodes][DK];  // k, k, a, a
    __shared__ float s_v[kNodes][BV];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tiles = dv / BV, tile = blockIdx.x % tiles, head = blockIdx.x / tiles;
    const int b = head / HV, hv = head - b * HV, hk = hv / (HV / HK);
    const int cq = lane & 3, rg = lane >> 2;
    const int col = tile * BV + warp * kWarpCols;  // the warp's first column
    const size_t base = ((size_t)head * DK + rg) * dv + col + 4 * cq;

    const int n = min(n_path[b], max_path);
    if (n <= 0 && h0 == ht) return;
    Pair s[RM][2];
    const float *from = h0 + base;
#pragma unroll
    for (int m = 0; m < RM; ++m, from += 8 * dv) {
        const float4 x = h0 ? ldg_stream4(from) : make_float4(0.f, 0.f, 0.f, 0.f);
        s[m][0] = pair(x.x, x.y);
        s[m][1] = pair(x.z, x.w);
    }
    for (int at = 0; at < n; at += kNodes) {
        // the nodes of this batch, one per lane; the path ends before the first invalid one
        int node = -1;
        if (lane < kNodes && at + lane < n) node = path[(size_t)b * max_path + at + lane];
        const unsigned bad = __ballot_sync(0xffffffffu, node < 0 || node >= T);
        const int cnt = min(kNodes, __ffs(bad) - 1);  // lanes past kNodes are bad
        if (at > 0) __syncthreads();  // the batch before has been used
#pragma unroll 4
        for (int i = 0; i < kNodes * DK / NT; ++i) {
            const int idx = i * NT + tid, c = idx / DK, r = idx % DK;
            const int t = __shfl_sync(0xffffffffu, node, c);
            if (c < cnt) {
                const size_t row = (size_t)b * T + t;
                const float kk = to_f32(k[(row * HK + hk) * DK + r]);
                const float a = expf(GS ? g[row * HV + hv] : g[(row * HV + hv) * DK + r]);
                s_ka[c][r] = make_float4(kk, kk, a, a);
            }
        }
#pragma unroll
        for (int i = 0; i < kNodes * BV / NT; ++i) {
            const int idx = i * NT + tid, c = idx / BV, j = idx % BV;
            const int t = __shfl_sync(0xffffffffu, node, c);
            if (c < cnt)
                s_v[c][j] = to_f32(v[(((size_t)b * T + t) * HV + hv) * dv + tile * BV + j]);
        }
        float bt = 0.f;
        if (lane < cnt) bt = beta[((size_t)b * T + node) * HV + hv];
        __syncthreads();
        for (int c = 0; c < cnt; ++c) {
            // decay, and the columns' sums over this lane's rows
            Pair acc[2][2];
#pragma unroll
            for (int m = 0; m < RM; ++m) {
                const ulonglong2 ka =
                    *reinterpret_cast<const ulonglong2 *>(&s_ka[c][rg + 8 * m]);
                const Pair kk{ka.x}, aa{ka.y};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s[m][h] = mul2(s[m][h], aa);
                    acc[m & 1][h] = m < 2 ? mul2(kk, s[m][h]) : fma2(kk, s[m][h], acc[m & 1][h]);
                }
            }
            const float2 x = split(add2(acc[0][0], acc[1][0])), y = split(add2(acc[0][1], acc[1][1]));
            // over the eight row groups: halving the columns twice, then one
            // sum left per lane, that of column 4 cq + 2 (rg & 1) + (rg >> 1 & 1)
            const bool odd = rg & 1, high = rg & 2;
            float p0 = odd ? y.x : x.x, p1 = odd ? y.y : x.y;
            p0 += __shfl_xor_sync(0xffffffffu, odd ? x.x : y.x, 4);
            p1 += __shfl_xor_sync(0xffffffffu, odd ? x.y : y.y, 4);
            float sum = high ? p1 : p0;
            sum += __shfl_xor_sync(0xffffffffu, high ? p0 : p1, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            const int mine = 4 * cq + (odd ? 2 : 0) + (high ? 1 : 0);
            const float b_t = __shfl_sync(0xffffffffu, bt, c);
            const float d = b_t * (s_v[c][warp * kWarpCols + mine] - sum);
            const Pair d0 = pair(__shfl_sync(0xffffffffu, d, cq), __shfl_sync(0xffffffffu, d, cq + 8));
            const Pair d1 =
                pair(__shfl_sync(0xffffffffu, d, cq + 4), __shfl_sync(0xffffffffu, d, cq + 12));
#pragma unroll
            for (int m = 0; m < RM; ++m) {
                const Pair kk{*reinterpret_cast<const unsigned long long *>(&s_ka[c][rg + 8 * m])};
                s[m][0] = fma2(kk, d0, s[m][0]);
                s[m][1] = fma2(kk, d1, s[m][1]);
            }
        }
        if (cnt < kNodes) break;
    }
    float *to = ht + base;
#pragma unroll
    for (int m = 0; m < RM; ++m, to += 8 * dv) {
        const float2 x = split(s[m][0]), y = split(s[m][1]);
        stg_stream4(to, make_float4(x.x, x.y, y.x, y.y));
    }
}

struct CommitArgs {
    const void *k, *v;
    const float *g, *beta, *h0;
    float *ht;
    const int *path, *n_path;
    int B, T, HK, HV, dk, dv, max_path;
};

template <typename Tin, int DK, int BV, bool GS>
cudaError_t launch_bv(const CommitArgs &a, cudaStream_t stream) {
    const long long ctas = (long long)a.B * a.HV * (a.dv / BV);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    trace_begin(kKernCommit, stream);
    gdr_commit_kernel<Tin, DK, BV, GS><<<(unsigned)ctas, 2 * BV, 0, stream>>>(
        static_cast<const Tin *>(a.k), static_cast<const Tin *>(a.v), a.g, a.beta, a.h0, a.ht,
        a.path, a.n_path, a.T, a.HK, a.HV, a.dv, a.max_path);
    trace_end(kKernCommit, stream);
    return cudaGetLastError();
}

// 64 columns per CTA, so that k and exp(g) are staged twice a head; 32 where
// dv is 32 or where 64 would give fewer CTAs than the device has SMs.
template <typename Tin, int DK, bool GS>
cudaError_t launch(const CommitArgs &a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (a.dv < 64 || (long long)a.B * a.HV * (a.dv / 64) < sms)
        return launch_bv<Tin, DK, 32, GS>(a, stream);
    return launch_bv<Tin, DK, 64, GS>(a, stream);
}

template <typename Tin, bool GS>
cudaError_t launch_dk(const CommitArgs &a, cudaStream_t stream) {
    switch (a.dk) {
        case 32: return launch<Tin, 32, GS>(a, stream);
        case 64: return launch<Tin, 64, GS>(a, stream);
        default: return launch<Tin, 128, GS>(a, stream);
    }
}

}  // namespace
}  // namespace gdr

extern "C" GDR_API gdr_status gdr_commit_path(const void *k, const void *v, const float *g,
                                              const float *beta, const float *h0, float *ht,
                                              const int *path, const int *n_path, int B, int T,
                                              int HK, int HV, int dk, int dv, int max_path,
                                              void *stream, int kv_dtype, unsigned flags) {
    using namespace gdr;
    if (B < 0 || T < 1 || max_path < 0 || HK <= 0 || HV <= 0 || HV % HK != 0) return GDR_ERR_SHAPE;
    if (kv_dtype != GDR_F32 && kv_dtype != GDR_BF16) return GDR_ERR_UNSUPPORTED;
    if (!supported_dim(dk) || !supported_dim(dv) || (flags & ~GDR_FLAG_SCALAR_GATE))
        return GDR_ERR_UNSUPPORTED;
    const long long BT = (long long)B * T;
    if (BT > (1LL << 40) || (long long)B * HV > (1LL << 30)) return GDR_ERR_SHAPE;
    if (B == 0) return GDR_OK;
    const bool gs = (flags & GDR_FLAG_SCALAR_GATE) != 0;
    if (!k || !v || !g || !beta || !ht || !n_path || (max_path > 0 && !path)) return GDR_ERR_NULL;
    const void *vectors[] = {k, v, g, h0, ht};
    for (const void *x : vectors)
        if (x && !aligned16(x)) return GDR_ERR_ALIGN;
    if (!aligned4(beta) || !aligned4(n_path) || (path && !aligned4(path))) return GDR_ERR_ALIGN;
    const size_t es = kv_dtype == GDR_BF16 ? 2 : 4, state = (size_t)B * HV * dk * dv * 4;
    const Range ins[] = {range_of(k, (size_t)BT * HK * dk * es),
                         range_of(v, (size_t)BT * HV * dv * es),
                         range_of(g, (size_t)BT * HV * (gs ? 1 : dk) * 4),
                         range_of(beta, (size_t)BT * HV * 4),
                         path ? range_of(path, (size_t)B * max_path * 4) : Range{0, 0},
                         range_of(n_path, (size_t)B * 4),
                         h0 && h0 != ht ? range_of(h0, state) : Range{0, 0}};
    if (overlaps_any(range_of(ht, state), ins, 7)) return GDR_ERR_ALIAS;
    const CommitArgs a{k, v, g, beta, h0, ht, path, n_path, B, T, HK, HV, dk, dv, max_path};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        kv_dtype == GDR_BF16
            ? (gs ? launch_dk<__nv_bfloat16, true>(a, s) : launch_dk<__nv_bfloat16, false>(a, s))
            : (gs ? launch_dk<float, true>(a, s) : launch_dk<float, false>(a, s));
    if (e == cudaSuccess) return GDR_OK;
    record_cuda_error(e);
    return GDR_ERR_CUDA;
}
