// path_commit.cu -- gdr_commit_path: the state after the accepted nodes of a
// draft.
//
// Each node on the path takes the token recurrence's step without its output:
//     s_ij <- a_i s_ij            a_i = exp(g_i)
//     d_j   = beta (v_j - sum_i k_i s_ij)
//     s_ij <- s_ij + k_i d_j
// The columns j of a state never meet, so the state is cut along them and
// stays in registers over the whole path: read once, written once.
#include <stdint.h>

#include "common.cuh"
#include "gdr.h"
#include "host_checks.h"

namespace gdr {
namespace {

// One CTA per (sequence, value head), one thread per value column.
template <typename Tin, int DK, bool GS>
__global__ void gdr_commit_kernel(const Tin *__restrict__ k, const Tin *__restrict__ v,
                                  const float *__restrict__ g, const float *__restrict__ beta,
                                  const float *h0, float *ht, const int *__restrict__ path,
                                  const int *__restrict__ n_path, int T, int HK, int HV, int dv,
                                  int max_path) {
    __shared__ float s_k[DK], s_a[DK];
    const int head = blockIdx.x, b = head / HV, hv = head % HV, hk = hv / (HV / HK);
    const int j = threadIdx.x;
    float s[DK];
    const size_t base = (size_t)head * DK * dv + j;
#pragma unroll
    for (int i = 0; i < DK; ++i) s[i] = h0 ? h0[base + (size_t)i * dv] : 0.f;
    const int n = min(n_path[b], max_path);
    for (int step = 0; step < n; ++step) {
        const int t = path[(size_t)b * max_path + step];
        if (t < 0 || t >= T) break;
        const size_t row = (size_t)b * T + t;
        __syncthreads();
        for (int i = j; i < DK; i += blockDim.x) {
            s_k[i] = to_f32(k[(row * HK + hk) * DK + i]);
            s_a[i] = expf(GS ? g[row * HV + hv] : g[(row * HV + hv) * DK + i]);
        }
        __syncthreads();
        float seen = 0.f;
#pragma unroll
        for (int i = 0; i < DK; ++i) {
            s[i] *= s_a[i];
            seen = fmaf(s_k[i], s[i], seen);
        }
        const float d = beta[row * HV + hv] * (to_f32(v[(row * HV + hv) * dv + j]) - seen);
#pragma unroll
        for (int i = 0; i < DK; ++i) s[i] = fmaf(s_k[i], d, s[i]);
    }
#pragma unroll
    for (int i = 0; i < DK; ++i) ht[base + (size_t)i * dv] = s[i];
}

struct CommitArgs {
    const void *k, *v;
    const float *g, *beta, *h0;
    float *ht;
    const int *path, *n_path;
    int B, T, HK, HV, dk, dv, max_path;
};

template <typename Tin, int DK, bool GS>
cudaError_t launch(const CommitArgs &a, cudaStream_t stream) {
    trace_begin(kKernCommit, stream);
    gdr_commit_kernel<Tin, DK, GS><<<a.B * a.HV, a.dv, 0, stream>>>(
        static_cast<const Tin *>(a.k), static_cast<const Tin *>(a.v), a.g, a.beta, a.h0, a.ht,
        a.path, a.n_path, a.T, a.HK, a.HV, a.dv, a.max_path);
    trace_end(kKernCommit, stream);
    return cudaGetLastError();
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
