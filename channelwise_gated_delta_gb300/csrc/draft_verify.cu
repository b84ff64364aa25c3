// draft_verify.cu -- gdr_verify_drafts: which drafted tokens stand, and the
// token after them.
//
// A tree is walked from its root: the children of the node reached are tried
// in order, and where none is accepted the next token is drawn from the
// residual weights of that node's rows (include/gdr.h has the rule).  Mass
// is summed in whole numbers of 2^-40, so that every order of summation
// gives the same sums; each other operation is one float32 operation,
// written with its rounding so that no contraction changes it.
//
// Only the last node's rows are read whole (and those of a node that was
// passed after refusals with q): the walk itself needs two elements per
// drafted token, which all are gathered at once.  What bounds the call is
// the latency of that chain -- tokens and parents, the gathered elements,
// the rows, the totals, the token's neighbourhood -- and for large batches
// the bandwidth of the rows.  A tree is therefore one cluster of CTAs, each
// of which walks the tree for itself (the same numbers, so the same walk)
// and sums its part of the rows; the totals meet in shared memory across
// the cluster, and the CTA in whose part the goal lies finds the token.
#include <stdint.h>

#include "common.cuh"
#include "gdr.h"
#include "host_checks.h"
#include "sm100_ptx.cuh"

namespace gdr {
namespace {

constexpr int kMaxNodes = 512;
constexpr int kMaxVocab = 1 << 22;  // 2^22 weights of at most 2^40 each: sums below 2^63
constexpr int kMaxCluster = 8;  // the portable limit
constexpr int kAheadF32 = 4;    // 16-byte loads a lane has in flight per row (bf16: half)
constexpr float kUnit = 1099511627776.f;            // 2^40
constexpr float kUnitInv = 9.094947017729282e-13f;  // 2^-40
constexpr int kUBits = 24;

// A probability as it counts: NaN and negative 0, above 1 at most 1.
__device__ __forceinline__ float probability(float x) { return __saturatef(x); }

// Sums of fix(x) = floor(2^40 x) for 0 <= x < 4.  A conversion to 64-bit whole
// numbers runs at the FP64 pipe's rate (it took two thirds of the call), so x
// is taken apart by float operations, all of them exact: added to 2^23 and
// rounded towards zero, a number below 2^23 leaves its whole part in the
// low bits of the sum.  floor(2^40 x) = 2^20 hi + lo with hi = floor(2^20 x)
// and lo the same of what is left of it.
struct Mass {
    uint32_t hi = 0, lo = 0;  // of at most 1024 elements
    long long sum = 0;
    __device__ __forceinline__ void add(float x) {
        constexpr float kTwo20 = 1048576.f, kTwo23 = 8388608.f;
        const float y = __fmul_rn(x, kTwo20);
        const float whole = __fadd_rz(y, kTwo23);
        const float rest = __fsub_rn(y, __fsub_rn(whole, kTwo23));
        hi += __float_as_uint(whole) - 0x4b000000u;
        lo += __float_as_uint(__fmaf_rz(rest, kTwo20, kTwo23)) - 0x4b000000u;
    }
    __device__ __forceinline__ void flush() {
        sum += ((long long)hi << 20) + lo;
        hi = lo = 0;
    }
};
__device__ __forceinline__ long long fix(float x) {
    Mass m;
    m.add(x);
    m.flush();
    return m.sum;
}
__device__ __forceinline__ float mass_of(long long sum) {
    return __fmul_rn(__ll2float_rn(sum), kUnitInv);
}

// w / mass for a residual's w >= 0.  Half of a residual is zeros, and a
// zero would take the division's slow path.
__device__ __forceinline__ float divided(float w, float mass) {
    const float x = __fdiv_rn(w > 0.f ? w : mass, mass);
    return w > 0.f ? x : 0.f;
}
// The weights of M elements after n refusals with q, given P in w and Q in x:
// the residual of the last refusal that left something (P before any);
// norm[s] is the mass of residual s, 0 where it had none.  All elements take
// a refusal together, for the latency of the division.
template <int M>
__device__ __forceinline__ void residuals(float (&w)[M], const float (&x)[M], const float *norm,
                                          int n) {
    float scale = 1.f;  // of the refusal before
    for (int s = 0; s < n; ++s) {
        const float mass = norm[s];
        if (mass == 0.f) continue;
        if (scale != 1.f) {
#pragma unroll
            for (int e = 0; e < M; ++e) w[e] = divided(w[e], scale);
        }
#pragma unroll
        for (int e = 0; e < M; ++e) w[e] = fmaxf(__fsub_rn(w[e], x[e]), 0.f);
        scale = mass;
    }
}

// ---- a row of V elements, addressed by j = i + shift, shift being the
// elements between the 16-byte boundary at or before the row and its start:
// vectors of VEC elements at multiples of VEC are aligned for every row.
template <typename Tp>
struct Vec {
    static constexpr int N = 16 / (int)sizeof(Tp);
};
template <typename Tp>
__device__ __forceinline__ int row_shift(const Tp *row) {
    return (int)(((uintptr_t)row & 15u) / sizeof(Tp));
}
__device__ __forceinline__ void unpack(uint4 r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(uint4 r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t bits_of(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }

// Elements i0 .. i0 + VEC - 1 of a row one by one, 0 outside of it: for the
// ends of a row, and for rows of q that do not lie to 16 bytes as p's do.
template <typename Tp>
__device__ __forceinline__ uint4 load_elements(const Tp *row, int i0, int V) {
    constexpr int N = Vec<Tp>::N;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int i = i0 + e;
        if (i >= 0 && i < V) w[e * 4 / N] |= bits_of(row[i]) << (N == 8 ? 16 * (e & 1) : 0);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename Tp>
__device__ __forceinline__ uint4 load_vec(const Tp *row, int i0) {
    return __ldg(reinterpret_cast<const uint4 *>(row + i0));
}

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// ---- the cluster
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores x to the same variable of CTA `rank` of the cluster.
__device__ __forceinline__ void store_remote(long long *var, int rank, long long x) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
        "st.shared::cluster.b64 [a], %2;\n\t}" ::"r"(sm100::smem_u32(var)),
        "r"(rank), "l"(x)
        : "memory");
}

// KEEP: a lane's part of the rows is at most kAhead vectors and stays in
// registers while the walk is at their node, for further refusals and for the
// search.  THREADS threads per CTA, 1024 / THREADS CTAs per SM.
template <typename Tp, bool HAS_Q, bool KEEP, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    gdr_verify_kernel(const Tp *__restrict__ p, const Tp *__restrict__ q,
                      const int *__restrict__ tokens, const int *__restrict__ parent,
                      const float *__restrict__ coins, const float *__restrict__ u,
                      int *__restrict__ path, int *__restrict__ n_path,
                      int *__restrict__ next_token, int T, int V, long long ldp, long long ldq,
                      long long parent_sb, long long parent_st, int max_path, int cluster) {
    constexpr int kThreads = THREADS, kWarps = THREADS / 32;
    constexpr int N = Vec<Tp>::N;
    constexpr int kWide = 32 * N;  // elements of a warp's load: a unit of the row
    constexpr int kAhead = kAheadF32 * 4 / N;
    __shared__ int s_parent[kMaxNodes], s_token[kMaxNodes];
    __shared__ float s_coin[kMaxNodes], s_p[kMaxNodes], s_q[kMaxNodes];
    __shared__ float s_norm[kMaxNodes];   // with q: the mass of each residual
    __shared__ int s_refused[kMaxNodes];  // without q: the nodes refused
    __shared__ long long s_warp[kWarps];
    __shared__ long long s_total[2][kMaxCluster];
    __shared__ int s_here, s_out, s_more, s_summed;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / cluster, rank = blockIdx.x - b * cluster;
    cluster_arrive();  // (1) this CTA runs: its shared memory may be written

    // ---- this warp's part of the rows of the node reached
    const Tp *prow = nullptr, *qrow = nullptr;
    int shift = 0, u0 = 0, u1 = 0, c0 = 0, per_warp = 0, units = 0;
    int f0 = 0, f1 = 0;  // the units whose vectors are aligned and inside the row
    auto take_rows = [&](int node) {
        const size_t row = (size_t)b * T + node;
        prow = p + row * ldp;
        shift = row_shift(prow);
        f0 = shift > 0 ? 1 : 0;
        f1 = (V + shift) / kWide;
        if (HAS_Q) {
            qrow = q + row * ldq;
            if (row_shift(qrow) != shift) f1 = f0;
        }
        units = (V + shift + kWide - 1) / kWide;
        const int per_cta = (units + cluster - 1) / cluster;
        per_warp = (per_cta + kWarps - 1) / kWarps;
        c0 = rank * per_cta;  // this CTA's units: c0 .. min(c0 + per_cta, units) - 1
        const int c1 = min(c0 + per_cta, units);
        u0 = min(c0 + warp * per_warp, c1);
        u1 = min(u0 + per_warp, c1);
    };
    // the weights of K vectors of a lane; refusals without q are taken off elsewhere
    auto weights = [&](const auto &pv, const auto &qv, int n, auto &w) {
        constexpr int K = sizeof(pv) / sizeof(uint4);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float y[N];
            unpack(pv[k], y);
#pragma unroll
            for (int e = 0; e < N; ++e) w[k * N + e] = probability(y[e]);
        }
        if (HAS_Q && n > 0) {
            float x[K * N];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float y[N];
                unpack(qv[k], y);
#pragma unroll
                for (int e = 0; e < N; ++e) x[k * N + e] = probability(y[e]);
            }
            if (n == 1 && s_norm[0] != 0.f) {  // nearly every row that is read whole
#pragma unroll
                for (int e = 0; e < K * N; ++e) w[e] = __saturatef(__fsub_rn(w[e], x[e]));
            } else {
                residuals(w, x, s_norm, n);
            }
        }
    };
    // a lane's vectors of unit `unit`, zeros behind unit `end`
    auto load_unit = [&](int unit, int end, bool with_q, uint4 &pv, uint4 &qv) {
        const int i0 = unit * kWide + lane * N - shift;
        pv = qv = make_uint4(0u, 0u, 0u, 0u);
        if (unit >= f0 && unit < min(end, f1)) {
            pv = load_vec(prow, i0);
            if (with_q) qv = load_vec(qrow, i0);
        } else if (unit < end) {  // at the ends of the row one by one
            pv = load_elements(prow, i0, V);
            if (with_q) qv = load_elements(qrow, i0, V);
        }
    };
    // the weights of this lane's elements of a unit
    auto unit_weights = [&](int unit, int n, float (&w)[N]) {
        uint4 pv[1], qv[1];
        load_unit(unit, units, HAS_Q && n > 0, pv[0], qv[0]);
        weights(pv, qv, n, w);
    };
    // KEEP: the rows of node `held`
    uint4 kept_p[KEEP ? kAhead : 1], kept_q[KEEP ? kAhead : 1];
    int held = -1;
    auto hold = [&](int node) {
        if (!KEEP || node == held) return;
        held = node;
        take_rows(node);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) load_unit(u0 + k, u1, HAS_Q, kept_p[KEEP ? k : 0], kept_q[KEEP ? k : 0]);
    };
    // mass of units lo .. hi - 1 after n refusals, in every lane of the warp
    auto mass = [&](int lo, int hi, int n) -> long long {
        Mass part;
        if (KEEP) {  // lo .. hi - 1 are this warp's own units
            float w[(KEEP ? kAhead : 1) * N];
            weights(kept_p, kept_q, n, w);
#pragma unroll
            for (int e = 0; e < (KEEP ? kAhead : 1) * N; ++e) part.add(w[e]);
            part.flush();
        }
        for (int at = lo; !KEEP && at < hi; at += kAhead) {
            uint4 pv[kAhead], qv[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const bool whole = at + k < hi && at + k >= f0 && at + k < f1;
                const int i0 = (at + k) * kWide + lane * N - shift;
                pv[k] = whole ? load_vec(prow, i0) : make_uint4(0u, 0u, 0u, 0u);
                qv[k] = HAS_Q && n > 0 && whole ? load_vec(qrow, i0) : make_uint4(0u, 0u, 0u, 0u);
            }
            if (at < f0 || min(at + kAhead, hi) > f1) {  // the ends of the row, one by one
                for (int k = 0; k < kAhead; ++k) {
                    if (at + k >= hi || (at + k >= f0 && at + k < f1)) continue;
                    float w[N];
                    unit_weights(at + k, n, w);
#pragma unroll
                    for (int e = 0; e < N; ++e) part.add(w[e]);
                }
            }
            float w[kAhead * N];
            weights(pv, qv, n, w);
#pragma unroll
            for (int e = 0; e < kAhead * N; ++e) part.add(w[e]);
            part.flush();
        }
        if (!HAS_Q)
            for (int s = lane; s < n; s += 32) {
                const int unit = (s_token[s_refused[s]] + shift) / kWide;
                if (unit >= lo && unit < hi) part.sum -= fix(s_p[s_refused[s]]);
            }
        return warp_sum(part.sum);
    };
    if (KEEP) hold(0);  // in flight with the nodes: the walk may well end at the root
    for (int t = tid; t < T; t += kThreads) {
        const size_t at = (size_t)b * T + t;
        int par = -1, tok = -1;
        if (t > 0) {
            par = parent[b * parent_sb + t * parent_st];
            tok = tokens[at];
        }
        const float coin = coins[at];
        const bool ok = par >= 0 && par < t && tok >= 0 && tok < V;
        const size_t row = (size_t)b * T + (ok ? par : 0);
        s_p[t] = ok ? probability(to_f32(p[row * ldp + tok])) : 0.f;
        s_q[t] = ok && HAS_Q ? probability(to_f32(q[row * ldq + tok])) : 0.f;
        s_parent[t] = ok ? par : -1;
        s_token[t] = tok;
        s_coin[t] = coin;
    }
    const float uu = u[b];
    __syncthreads();

    int round = 0;
    // total mass of the node's rows after n refusals; each warp's in s_warp,
    // each CTA's in s_total[round & 1]
    auto total_mass = [&](int n) -> long long {
        const long long mine = mass(u0, u1, n);
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        ++round;
        long long *totals = s_total[round & 1];
        if (round == 1) cluster_wait();  // (1)
        if (warp == 0) {
            const long long all = warp_sum(lane < kWarps ? s_warp[lane] : 0);
            if (lane < cluster) store_remote(totals + rank, lane, all);
            __syncwarp();
        }
        cluster_arrive();
        cluster_wait();
        long long sum = 0;
        for (int r = 0; r < cluster; ++r) sum += totals[r];
        return sum;
    };

    // ---- the walk, by warp 0 of each CTA: until the path ends, or with q
    // until a refusal's mass is wanted
    int here = 0, tried = 0, out = 0, n = 1;
    long long total = 0;
    bool summed = false;  // total is that of the weights after `out` refusals at `here`
    long long left = (long long)kUnit;
    const bool writer = rank == 0 && tid == 0;
    int *my_path = path + (size_t)b * max_path;
    if (writer) my_path[0] = 0;
    while (true) {
        if (warp == 0) {
            bool more = false;
            while (n < max_path) {
                // the next child of `here` behind node `tried`
                int t = T;
                for (int base = (tried + 1) & ~31; base < T; base += 32) {
                    const int at = base + lane;
                    const unsigned hit = __ballot_sync(
                        0xffffffffu, at > tried && at < T && s_parent[min(at, T - 1)] == here);
                    if (hit) {
                        t = base + __ffs(hit) - 1;
                        break;
                    }
                }
                if (t >= T) break;
                tried = t;
                float a, bar;
                if (HAS_Q) {
                    a = s_p[t];
                    for (int s = 0; s < out; ++s)
                        if (s_norm[s] != 0.f)
                            a = divided(fmaxf(__fsub_rn(a, s_q[t]), 0.f), s_norm[s]);
                    bar = __fmul_rn(s_coin[t], s_q[t]);
                } else {
                    bool again = false;
                    for (int s = lane; s < out; s += 32)
                        again = again || s_token[s_refused[s]] == s_token[t];
                    a = __any_sync(0xffffffffu, again) ? 0.f : s_p[t];
                    bar = __fmul_rn(s_coin[t], mass_of(left));
                }
                if (a > 0.f && bar < a) {
                    here = t;
                    out = 0;
                    summed = false;
                    left = (long long)kUnit;
                    if (writer) my_path[n] = t;
                    ++n;
                } else if (HAS_Q) {
                    if (lane == 0) s_norm[out] = 1.f;  // its mass follows
                    ++out;
                    more = true;
                    break;
                } else if (a > 0.f) {  // what has no mass need not be taken off
                    left = max(left - fix(a), 0ll);
                    __syncwarp();
                    if (lane == 0) s_refused[out] = t;
                    ++out;
                    __syncwarp();
                }
            }
            if (lane == 0) {
                s_here = here;
                s_out = out;
                s_more = more;
                s_summed = summed;
            }
        }
        __syncthreads();
        here = s_here;
        out = s_out;
        summed = s_summed;
        if (!HAS_Q || !s_more) break;
        if (KEEP)
            hold(here);
        else
            take_rows(here);
        total = total_mass(out);
        summed = total > 0;  // without mass the weights stay those of before
        if (tid == 0) s_norm[out - 1] = mass_of(total);
        __syncthreads();
    }
    if (writer) {
        for (int i = n; i < max_path; ++i) my_path[i] = -1;
        n_path[b] = n;
    }

    // ---- the next token
    if (!HAS_Q || !summed) {
        if (KEEP)
            hold(here);
        else
            take_rows(here);
        total = total_mass(out);
    }
    if (!HAS_Q && total == 0 && out > 0) {  // nothing left: the row as it was
        out = 0;
        total = total_mass(0);
    }
    if (total == 0) {
        if (writer) next_token[b] = -1;
        return;
    }
    const float top = 1.f - 1.f / (1 << kUBits);
    const long long m = (long long)__fmul_rn(fminf(fmaxf(uu, 0.f), top), (float)(1 << kUBits));
    const long long low = (1 << kUBits) - 1;
    long long goal = (total >> kUBits) * m + (((total & low) * m) >> kUBits);  // floor(total m / 2^24)
    const long long *totals = s_total[round & 1];
    for (int r = 0; r < rank; ++r) goal -= totals[r];
    if (goal < 0 || goal >= totals[rank]) return;
    int w = 0;
    for (; goal >= s_warp[w]; ++w) goal -= s_warp[w];
    // looks for the goal among a unit's elements, of weights x; takes the unit's mass off it
    auto in_unit = [&](int unit, float (&x)[N]) -> bool {
        const int i0 = unit * kWide + lane * N - shift;
        if (!HAS_Q)
            for (int s = 0; s < out; ++s) {
                const int e = s_token[s_refused[s]] - i0;
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (k == e) x[k] = 0.f;
            }
        Mass own;
#pragma unroll
        for (int e = 0; e < N; ++e) own.add(x[e]);
        own.flush();
        long long upto = own.sum;  // of the lanes up to this one
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += y;
        }
        if (upto - own.sum <= goal && goal < upto) {
            long long run = upto - own.sum;
            int found = -1;  // the first element whose running sum is above
#pragma unroll
            for (int e = 0; e < N; ++e) {
                run += fix(x[e]);
                if (found < 0 && run > goal) found = e;
            }
            next_token[b] = i0 + found;
        }
        const long long all = __shfl_sync(0xffffffffu, upto, 31);
        const bool hit = goal < all;
        goal -= all;
        return hit;
    };
    if (KEEP) {
        if (w != warp) return;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const uint4 pv[1] = {kept_p[KEEP ? k : 0]}, qv[1] = {kept_q[KEEP ? k : 0]};
            float x[N];
            weights(pv, qv, out, x);
            if (in_unit(u0 + k, x)) return;
        }
        return;
    }
    // the warp's units divided among all warps of the CTA, then one by one
    const int per_cta = (units + cluster - 1) / cluster, c1 = min(c0 + per_cta, units);
    const int w0 = min(c0 + w * per_warp, c1), w1 = min(w0 + per_warp, c1);
    const int step = (w1 - w0 + kWarps - 1) / kWarps;
    const int m0 = min(w0 + warp * step, w1), m1 = min(m0 + step, w1);
    __syncthreads();
    const long long mine = mass(m0, m1, out);
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    w = 0;
    for (; goal >= s_warp[w]; ++w) goal -= s_warp[w];
    if (w != warp) return;
    for (int at = m0; at < m1; ++at) {
        float x[N];
        unit_weights(at, out, x);
        if (in_unit(at, x)) return;
    }
}

struct VerifyArgs {
    const void *p, *q;
    const int *tokens, *parent;
    const float *coins, *u;
    int *path, *n_path, *next_token;
    int B, T, V;
    long long ldp, ldq, parent_sb, parent_st;
    int max_path;
};

template <typename Tp, bool HAS_Q, bool KEEP, int THREADS>
cudaError_t launch_clusters(const VerifyArgs &a, int c, cudaStream_t stream) {
    if ((long long)a.B * c > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * c));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    trace_begin(kKernVerify, stream);
    const cudaError_t e = cudaLaunchKernelEx(
        &cfg, gdr_verify_kernel<Tp, HAS_Q, KEEP, THREADS>, static_cast<const Tp *>(a.p),
        static_cast<const Tp *>(a.q), a.tokens, a.parent, a.coins, a.u, a.path, a.n_path,
        a.next_token, a.T, a.V, a.ldp, a.ldq, a.parent_sb, a.parent_st, a.max_path, c);
    trace_end(kKernVerify, stream);
    return e;
}

// CTAs per tree, a power of two up to the cluster limit.  Few trees: as many
// as SMs and row allow (a CTA has a vector at least for each of 256 threads),
// with the fewest threads whose lanes can keep their part of the row.  Clusters
// of 8 do not fill the device (a cluster keeps to one processing cluster of
// SMs), so 7 of 8 SMs are counted.  Otherwise CTAs of 256 threads that stream
// the rows, doubled while the trees' CTAs would leave the device's slots (4
// a SM) empty and each would keep 1024 elements.
template <typename Tp, bool HAS_Q>
cudaError_t launch_q(const VerifyArgs &a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    constexpr int N = Vec<Tp>::N, kKeep = kAheadF32 * 4 / N;
    int c = 1;
    while (c < kMaxCluster && (long long)a.B * 2 * c <= sms * 7 / 8 && a.V >= 2 * c * 256 * N)
        c *= 2;
    if (a.B <= sms) {
        // the units of a warp, of a row that may begin anywhere in a vector
        const int units = (a.V + N - 1 + 32 * N - 1) / (32 * N), per_cta = (units + c - 1) / c;
        if ((per_cta + 7) / 8 <= kKeep) return launch_clusters<Tp, HAS_Q, true, 256>(a, c, stream);
        if ((per_cta + 15) / 16 <= kKeep)
            return launch_clusters<Tp, HAS_Q, true, 512>(a, c, stream);
        if ((per_cta + 31) / 32 <= kKeep)
            return launch_clusters<Tp, HAS_Q, true, 1024>(a, c, stream);
    }
    c = 1;
    while (c < kMaxCluster && (long long)a.B * c < 4LL * sms && a.V / (2 * c) >= 1024) c *= 2;
    return launch_clusters<Tp, HAS_Q, false, 256>(a, c, stream);
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
    const VerifyArgs a{p,   q,   tokens,    parent,    coins,   u, path, n_path, next_token, B, T, V,
                       ldp, ldq, parent_sb, parent_st, max_path};
    const cudaError_t e =
        prob_dtype == GDR_BF16
            ? (q ? launch_q<__nv_bfloat16, true>(a, s) : launch_q<__nv_bfloat16, false>(a, s))
            : (q ? launch_q<float, true>(a, s) : launch_q<float, false>(a, s));
    if (e == cudaSuccess) return GDR_OK;
    record_cuda_error(e);
    return GDR_ERR_CUDA;
}
