// draft_verify.cu -- gdr_verify_drafts: which drafted tokens stand, and the
// token after them.
//
// A tree is walked from its root: the children of the node reached are tried
// in order, and where none is accepted the next token is drawn from the
// residual weights of that node's rows (include/gdr.h has the rule).  Mass
// is summed in whole numbers of 2^-40, so that every order of summation
// gives the same sums; each other operation is one float32 operation,
// written with its rounding so that no contraction changes it.
#include <stdint.h>

#include "common.cuh"
#include "gdr.h"
#include "host_checks.h"

namespace gdr {
namespace {

constexpr int kMaxNodes = 512;
constexpr int kMaxVocab = 1 << 22;  // 2^22 weights of at most 2^40 each: sums below 2^63
constexpr int kThreads = 512;
constexpr float kUnit = 1099511627776.f;         // 2^40
constexpr float kUnitInv = 9.094947017729282e-13f;  // 2^-40
constexpr int kUBits = 24;

// A probability as it counts: NaN and negative 0, above 1 at most 1.
template <typename Tp>
__device__ __forceinline__ float probability(Tp x) {
    return fminf(fmaxf(to_f32(x), 0.f), 1.f);  // fmaxf(NaN, 0) = 0
}
__device__ __forceinline__ long long fix(float x) { return __float2ll_rz(__fmul_rn(x, kUnit)); }
__device__ __forceinline__ float mass_of(long long sum) {
    return __fmul_rn(__ll2float_rn(sum), kUnitInv);
}

struct Residual {
    float scaled;  // R: what the next child is tried against
    float weight;  // r of the last refusal that left something (P before any)
};
// An element of the rows after n refusals with q; norm[s]: mass of residual
// s, 0 where it had none.
__device__ __forceinline__ Residual residual(float P, float Q, const float *norm, int n) {
    Residual x{P, P};
    for (int s = 0; s < n; ++s) {
        if (norm[s] == 0.f) continue;
        x.weight = fmaxf(__fsub_rn(x.scaled, Q), 0.f);
        x.scaled = __fdiv_rn(x.weight, norm[s]);
    }
    return x;
}

template <typename Tp>
__global__ void __launch_bounds__(kThreads)
    gdr_verify_kernel(const Tp *__restrict__ p, const Tp *__restrict__ q,
                      const int *__restrict__ tokens, const int *__restrict__ parent,
                      const float *__restrict__ coins, const float *__restrict__ u,
                      int *__restrict__ path, int *__restrict__ n_path,
                      int *__restrict__ next_token, int T, int V, long long ldp, long long ldq,
                      long long parent_sb, long long parent_st, int max_path) {
    __shared__ int s_parent[kMaxNodes], s_token[kMaxNodes];
    __shared__ float s_coin[kMaxNodes], s_p[kMaxNodes], s_q[kMaxNodes];
    __shared__ float s_norm[kMaxNodes];   // with q: the mass of each residual
    __shared__ int s_refused[kMaxNodes];  // without q: the tokens refused
    __shared__ long long s_sum[kThreads];
    __shared__ int s_here, s_tried, s_out, s_state;
    const int b = blockIdx.x, tid = threadIdx.x;

    for (int t = tid; t < T; t += kThreads) {
        const size_t at = (size_t)b * T + t;
        const int par = t > 0 ? parent[b * parent_sb + t * parent_st] : -1, tok = t > 0 ? tokens[at] : -1;
        const bool ok = par >= 0 && par < t && tok >= 0 && tok < V;
        const size_t row = (size_t)b * T + (ok ? par : 0);
        s_parent[t] = ok ? par : -1;
        s_token[t] = tok;
        s_coin[t] = coins[at];
        s_p[t] = ok ? probability(p[row * ldp + tok]) : 0.f;
        s_q[t] = ok && q ? probability(q[row * ldq + tok]) : 0.f;
    }
    if (tid == 0) {
        s_here = 0;   // the node reached
        s_tried = 0;  // nodes up to this one have been tried
        s_out = 0;    // refusals at s_here
        path[(size_t)b * max_path] = 0;
    }
    __syncthreads();

    // sums the weights of this thread's part of the rows of the node reached
    const int per = (V + kThreads - 1) / kThreads;
    const int lo = min(V, tid * per), hi = min(V, lo + per);
    auto weight = [&](int i, int n, bool all) -> float {
        const size_t row = (size_t)b * T + s_here;
        const float P = probability(p[row * ldp + i]);
        if (q) return residual(P, probability(q[row * ldq + i]), s_norm, n).weight;
        if (!all)
            for (int s = 0; s < n; ++s)
                if (s_refused[s] == i) return 0.f;
        return P;
    };
    auto sum_row = [&](int n, bool all) -> long long {  // exclusive sums in s_sum, total returned
        long long part = 0;
        for (int i = lo; i < hi; ++i) part += fix(weight(i, n, all));
        s_sum[tid] = part;
        __syncthreads();
        long long total = 0;
        for (int i = 0; i < kThreads; ++i) total += s_sum[i];
        __syncthreads();
        return total;
    };

    int n = 1;  // thread 0: nodes on the path
    long long left = (long long)kUnit;
    while (true) {
        if (tid == 0) {
            // tries children until one is refused with q (state 1) or the path ends (state 0)
            s_state = 0;
            int t = s_tried;
            while (n < max_path) {
                for (++t; t < T && s_parent[t] != s_here; ++t) {
                }
                if (t >= T) break;
                float a, bar;
                if (q) {
                    a = residual(s_p[t], s_q[t], s_norm, s_out).scaled;
                    bar = __fmul_rn(s_coin[t], s_q[t]);
                } else {
                    a = s_p[t];
                    for (int s = 0; s < s_out; ++s)
                        if (s_refused[s] == s_token[t]) a = 0.f;
                    bar = __fmul_rn(s_coin[t], mass_of(left));
                }
                if (a > 0.f && bar < a) {
                    s_here = t;
                    s_out = 0;
                    left = (long long)kUnit;
                    path[(size_t)b * max_path + n++] = t;
                } else if (q) {
                    s_norm[s_out++] = 1.f;  // its mass follows
                    s_state = 1;
                    break;
                } else {
                    left = max(left - fix(a), 0ll);
                    s_refused[s_out++] = s_token[t];
                }
            }
            s_tried = t;
        }
        __syncthreads();
        if (s_state == 0) break;
        const long long total = sum_row(s_out, false);
        if (tid == 0) s_norm[s_out - 1] = mass_of(total);
        __syncthreads();
    }

    long long total = sum_row(s_out, false);
    bool all = false;
    if (total == 0 && !q && s_out > 0) {  // nothing left: the row as it was
        all = true;
        total = sum_row(s_out, true);
    }
    if (tid == 0) {
        for (int i = n; i < max_path; ++i) path[(size_t)b * max_path + i] = -1;
        n_path[b] = n;
        if (total == 0) next_token[b] = -1;
    }
    if (total == 0) return;
    const float top = 1.f - 1.f / (1 << kUBits);
    const long long m =
        (long long)__fmul_rn(fminf(fmaxf(u[b], 0.f), top), (float)(1 << kUBits));
    const long long low = (1 << kUBits) - 1;
    const long long goal = (total >> kUBits) * m + (((total & low) * m) >> kUBits);
    long long run = 0;
    for (int i = 0; i < tid; ++i) run += s_sum[i];
    if (run <= goal && goal < run + s_sum[tid]) {
        for (int i = lo; i < hi; ++i) {
            run += fix(weight(i, s_out, all));
            if (run > goal) {
                next_token[b] = i;
                break;
            }
        }
    }
}

template <typename Tp>
cudaError_t launch(const void *p, const void *q, const int *tokens, const int *parent,
                   const float *coins, const float *u, int *path, int *n_path, int *next_token,
                   int B, int T, int V, long long ldp, long long ldq, long long parent_sb,
                   long long parent_st, int max_path, cudaStream_t stream) {
    trace_begin(kKernVerify, stream);
    gdr_verify_kernel<Tp><<<B, kThreads, 0, stream>>>(
        static_cast<const Tp *>(p), static_cast<const Tp *>(q), tokens, parent, coins, u, path,
        n_path, next_token, T, V, ldp, ldq, parent_sb, parent_st, max_path);
    trace_end(kKernVerify, stream);
    return cudaGetLastError();
}

// Whether `rows` rows `ld` apart are addressable (element offsets below 2^58).
bool rows_fit(long long rows, long long ld) { return ld <= 0 || rows <= (1LL << 58) / ld; }

}  // namespace
}  // namespace gdr

extern "C" GDR_API gdr_status gdr_verify_drafts(const void *p, const void *q, const int *tokens,
                                                const int *parent, const float *coins,
                                                const float *u, int *path, int *n_path,
                                                int *next_token, int B, int T, int V,
                                                long long ldp, long long ldq,
                                                long long parent_sb, long long parent_st,
                                                int max_path, void *stream, int prob_dtype) {
    using namespace gdr;
    if (B < 0 || T < 1 || V < 1 || max_path < 1 || max_path > T) return GDR_ERR_SHAPE;
    if (prob_dtype != GDR_F32 && prob_dtype != GDR_BF16) return GDR_ERR_UNSUPPORTED;
    if (T > kMaxNodes || V > kMaxVocab) return GDR_ERR_UNSUPPORTED;
    if (ldp < V || (q && ldq < V)) return GDR_ERR_SHAPE;
    const long long rows = (long long)B * T;
    if (!rows_fit(rows, ldp) || (q && !rows_fit(rows, ldq))) return GDR_ERR_SHAPE;
    if (parent_sb < 0 || parent_st < 0 || !rows_fit(B, parent_sb) || !rows_fit(T, parent_st))
        return GDR_ERR_SHAPE;
    if (B == 0) return GDR_OK;
    if (!p || !tokens || !parent || !coins || !u || !path || !n_path || !next_token)
        return GDR_ERR_NULL;
    if (!aligned16(p) || (q && !aligned16(q))) return GDR_ERR_ALIGN;
    const void *words[] = {tokens, parent, coins, u, path, n_path, next_token};
    for (const void *x : words)
        if (!aligned4(x)) return GDR_ERR_ALIGN;
    const size_t es = prob_dtype == GDR_BF16 ? 2 : 4, words4 = (size_t)rows * 4;
    const Range args[] = {range_of(p, ((size_t)(rows - 1) * ldp + V) * es),
                          q ? range_of(q, ((size_t)(rows - 1) * ldq + V) * es) : Range{0, 0},
                          range_of(tokens, words4),
                          range_of(parent, ((size_t)(B - 1) * parent_sb +
                                            (size_t)(T - 1) * parent_st + 1) * 4),
                          range_of(coins, words4),
                          range_of(u, (size_t)B * 4),
                          range_of(path, (size_t)B * max_path * 4),
                          range_of(n_path, (size_t)B * 4),
                          range_of(next_token, (size_t)B * 4)};
    for (int o = 6; o < 9; ++o)  // an output against the inputs and the outputs before it
        if (overlaps_any(args[o], args, o)) return GDR_ERR_ALIAS;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        prob_dtype == GDR_BF16
            ? launch<__nv_bfloat16>(p, q, tokens, parent, coins, u, path, n_path, next_token, B, T,
                                    V, ldp, ldq, parent_sb, parent_st, max_path, s)
            : launch<float>(p, q, tokens, parent, coins, u, path, n_path, next_token, B, T, V, ldp,
                            ldq, parent_sb, parent_st, max_path, s);
    if (e == cudaSuccess) return GDR_OK;
    record_cuda_error(e);
    return GDR_ERR_CUDA;
}
