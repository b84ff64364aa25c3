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
// the cluster, and the warp in whose part the goal lies finds the token.
//
// Measured on the device (chains of 8 nodes, f32 with q, 131,072 elements):
// 64 trees 16.0 us, the 67 MB of their last rows at 4.2 TB/s (0.62 of a
// copy's rate); bf16 13.0, f32 without q 11.6, bf16 without q 9.3.  By time
// stamps 2 us go to the nodes and their elements, 0.5 to 3 to the walk, 8 to 9
// to the rows, 1 to the totals and 1.3 to the search.  One tree over 32,768
// elements: 4.8 us.
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
constexpr int kKeepAhead = 4, kStreamAhead = 8;  // 16-byte loads a lane has in flight per row
constexpr float kUnit = 1099511627776.f;            // 2^40
constexpr float kUnitInv = 9.094947017729282e-13f;  // 2^-40
constexpr int kUBits = 24;

// A probability as it counts: NaN and negative 0, above 1 at most 1.
__device__ __forceinline__ float probability(float x) { return __saturatef(x); }

// Sums of fix(x) = floor(2^40 x) for 0 <= x < 4.  A conversion to 64-bit whole
// numbers runs at the FP64 pipe's rate (with it 64 trees took 27 us instead of
// 18, that pipe two thirds of the time), so x is taken apart by float
// operations, all of them exact: added to 2^23 and rounded towards zero, a
// number below 2^23 leaves its whole part in the low bits of the sum.
// floor(2^40 x) = 2^20 hi + lo with hi = floor(2^20 x) and lo the same of what is
// left of it.
struct Mass {
    uint32_t hi = 0, lo = 0;  // of at most 64 elements: a warp's sums fit 32 bits
    __device__ __forceinline__ void add(float x) {
        constexpr float kTwo20 = 1048576.f, kTwo23 = 8388608.f;
        const float y = __fmul_rn(x, kTwo20);
        const float whole = __fadd_rz(y, kTwo23);
        const float rest = __fsub_rn(y, __fsub_rn(whole, kTwo23));
        hi += __float_as_uint(whole) - 0x4b000000u;
        lo += __float_as_uint(__fmaf_rz(rest, kTwo20, kTwo23)) - 0x4b000000u;
    }
    __device__ __forceinline__ long long own() const { return ((long long)hi << 20) + lo; }
    __device__ __forceinline__ long long of_warp() const {
        const uint32_t h = __reduce_add_sync(0xffffffffu, hi);
        return ((long long)h << 20) + __reduce_add_sync(0xffffffffu, lo);
    }
};
__device__ __forceinline__ long long fix(float x) {
    Mass m;
    m.add(x);
    return m.own();
}
__device__ __forceinline__ float mass_of(long long sum) {
    return __fmul_rn(__ll2float_rn(sum), kUnitInv);
}

// w / mass for a residual's w >= 0.  Half of a residual is zeros, and a
// zero would take the division's slow path (16 trees of 32 nodes, up to three
// siblings drawn from q, 50,001 elements: 32 us, 17 without it).
__device__ __forceinline__ float divided(float w, float mass) {
    const float x = __fdiv_rn(w > 0.f ? w : mass, mass);
    return w > 0.f ? x : 0.f;
}
// The weights of M elements after n refusals with q, given P in w and Q in x:
// the residual of the last refusal that left something (P before any);
// norm[s] is the mass of residual s, 0 where it had none.  All elements take
// a refusal together, for the latency of the division.  Every refusal starts from P
// again, so that those of one node cost by the square of their number: one
// tree over 30,000 elements, 1 / 4 / 16 / 64 / 511 siblings all refused: 4.4 / 15
// / 115 / 1,490 / 89,300 us.
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
// ends of a row, and for rows of q that do not lie to 16 bytes as p's do (64
// chains over 131,072 elements: 36 us, 15 where they do).
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
// Stores x to the same variable of CTA `rank` of the cluster and counts its 8
// bytes on that CTA's barrier.
__device__ __forceinline__ void store_remote(long long *var, uint64_t *bar, int rank, long long x) {
    asm volatile(
        "{\n\t.reg .b32 a, b;\n\t"
        "mapa.shared::cluster.u32 a, %0, %2;\n\t"
        "mapa.shared::cluster.u32 b, %1, %2;\n\t"
        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [a], %3, [b];\n\t}" ::"r"(
            sm100::smem_u32(var)),
        "r"(sm100::smem_u32(bar)), "r"(rank), "l"(x)
        : "memory");
}
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s

// A lane takes its part of the rows in batches of AHEAD 16-byte vectors (of
// f32; half as many of bf16), whose loads are in flight together.  KEEP: that
// part is one batch at most and stays in registers while the walk is at its
// node, for further refusals and for the search.
template <typename Tp, bool HAS_Q, bool KEEP, int THREADS, int AHEAD>
__global__ void __launch_bounds__(THREADS, KEEP ? 1 : 2)
    gdr_verify_kernel(const Tp *__restrict__ p, const Tp *__restrict__ q,
                      const int *__restrict__ tokens, const int *__restrict__ parent,
                      const float *__restrict__ coins, const float *__restrict__ u,
                      int *__restrict__ path, int *__restrict__ n_path,
                      int *__restrict__ next_token, int T, int V, long long ldp, long long ldq,
                      long long parent_sb, long long parent_st, int max_path, int log_cluster,
                      int *dev_error) {
    constexpr int kThreads = THREADS, kWarps = THREADS / 32;
    constexpr int N = Vec<Tp>::N;
    constexpr int kWide = 32 * N;  // elements of a warp's load: a unit of the row
    constexpr int kAhead = AHEAD * 4 / N;
    __shared__ int s_parent[kMaxNodes], s_token[kMaxNodes];
    __shared__ int s_first[kMaxNodes];         // a node's first child
    __shared__ uint8_t s_first_yes[kMaxNodes];  // whether a node is accepted if it is tried first
    __shared__ float s_coin[kMaxNodes], s_p[kMaxNodes], s_q[kMaxNodes];
    __shared__ float s_norm[kMaxNodes];   // with q: the mass of each residual
    __shared__ int s_refused[kMaxNodes];  // without q: the nodes refused
    __shared__ long long s_warp[kWarps], s_before[kWarps];  // a warp's mass, those before it
    __shared__ long long s_total[2][kMaxCluster];
    __shared__ uint64_t s_bar[2];
    __shared__ int s_here, s_out, s_more, s_summed;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x >> log_cluster, cluster = 1 << log_cluster;
    const int rank = blockIdx.x - (b << log_cluster);
    if (tid == 0) {
        sm100::mbar_init(&s_bar[0], 1);
        sm100::mbar_init(&s_bar[1], 1);
        sm100::fence_mbar_init();
    }
    __syncwarp();
    cluster_arrive();  // (1) this CTA runs and its barriers are there: others may write to it

    // ---- this warp's part of the rows of the node reached
    const Tp *prow = nullptr, *qrow = nullptr;
    int shift = 0, u0 = 0, u1 = 0;
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
        const int units = (V + shift + kWide - 1) / kWide;
        const int per_cta = (units + cluster - 1) >> log_cluster;
        const int per_warp = (per_cta + kWarps - 1) / kWarps;
        const int c0 = rank * per_cta, c1 = min(c0 + per_cta, units);
        u0 = min(c0 + warp * per_warp, c1);
        u1 = min(u0 + per_warp, c1);
    };
    // the weights of K vectors of a lane; refusals without q are taken off elsewhere
    auto weights = [&](const uint4 *pv, const uint4 *qv, int n, auto &w) {
        constexpr int M = sizeof(w) / sizeof(float), K = M / N;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float y[N];
            unpack(pv[k], y);
#pragma unroll
            for (int e = 0; e < N; ++e) w[k * N + e] = probability(y[e]);
        }
        if (HAS_Q && n > 0) {
            float x[M];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float y[N];
                unpack(qv[k], y);
#pragma unroll
                for (int e = 0; e < N; ++e) x[k * N + e] = probability(y[e]);
            }
            if (n == 1 && s_norm[0] != 0.f) {  // nearly every row that is read whole
#pragma unroll
                for (int e = 0; e < M; ++e) w[e] = __saturatef(__fsub_rn(w[e], x[e]));
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
    // KEEP: the rows of node `held`
    uint4 kept_p[kAhead], kept_q[kAhead];
    int held = -1;
    auto hold = [&](int node) {
        if (node == held) return;
        held = node;
        take_rows(node);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) load_unit(u0 + k, u1, HAS_Q, kept_p[k], kept_q[k]);
    };
    // Mass of this warp's units after n refusals, in every lane.  Lane i also
    // keeps that of the i-th group of per_group batches of kAhead units, for the search.
    long long group = 0;
    int per_group = 1;
    auto add_all = [&](const auto &w) {
        constexpr int M = sizeof(w) / sizeof(float);
        Mass part;
#pragma unroll
        for (int e = 0; e < M; ++e) part.add(w[e]);
        return part;
    };
    auto mass = [&](int n) -> long long {
        const int batches = (u1 - u0 + kAhead - 1) / kAhead;
        per_group = max(1, (batches + 31) / 32);
        group = 0;
        if constexpr (KEEP) {
            float w[kAhead * N];
            weights(kept_p, kept_q, n, w);
            const long long sum = add_all(w).of_warp();
            if (lane == 0) group = sum;
        }
        for (int i = 0, to = 0, left = per_group; !KEEP && i < batches; ++i) {
            const int at = u0 + i * kAhead;
            uint4 pv[kAhead], qv[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const bool whole = at + k < u1 && at + k >= f0 && at + k < f1;
                const int i0 = (at + k) * kWide + lane * N - shift;
                pv[k] = whole ? load_vec(prow, i0) : make_uint4(0u, 0u, 0u, 0u);
                qv[k] = HAS_Q && n > 0 && whole ? load_vec(qrow, i0) : make_uint4(0u, 0u, 0u, 0u);
            }
            long long sum = 0;
            if (at < f0 || min(at + kAhead, u1) > f1) {  // the ends of the row, one by one
                for (int k = 0; k < kAhead; ++k) {
                    if (at + k >= u1 || (at + k >= f0 && at + k < f1)) continue;
                    uint4 ep, eq;
                    load_unit(at + k, u1, HAS_Q && n > 0, ep, eq);
                    float w[N];
                    weights(&ep, &eq, n, w);
                    sum += add_all(w).of_warp();
                }
            }
            float w[kAhead * N];
            weights(pv, qv, n, w);
            sum += add_all(w).of_warp();
            if (lane == to) group += sum;
            if (--left == 0) {
                left = per_group;
                ++to;
            }
        }
        if (!HAS_Q)
            for (int s = 0; s < n; ++s) {
                const int unit = (s_token[s_refused[s]] + shift) / kWide;
                if (unit >= u0 && unit < u1 && lane == (unit - u0) / kAhead / per_group)
                    group -= fix(s_p[s_refused[s]]);
            }
        return warp_sum(group);
    };
    // ---- the nodes, every CTA for itself: this thread's first one is loaded
    // at once, the others (T > kThreads) after it
    const float uu = u[b];
    const int *my_parent = parent + b * parent_sb;
    auto node_of = [&](int t, int &par, int &tok, float &coin) {
        par = tok = -1;
        coin = 0.f;
        if (t > 0 && t < T) {
            par = my_parent[t * parent_st];
            tok = tokens[(size_t)b * T + t];
            coin = coins[(size_t)b * T + t];
        }
    };
    int par, tok;
    float coin;
    node_of(tid, par, tok, coin);
    if (KEEP) hold(0);  // in flight with the nodes: the walk may well end at the root
    for (int t = tid; t < T; t += kThreads) s_first[t] = T;
    __syncthreads();
    for (int t = tid; t < T; t += kThreads) {
        if (t != tid) node_of(t, par, tok, coin);
        const bool ok = par >= 0 && par < t && tok >= 0 && tok < V;
        const size_t row = (size_t)b * T + (ok ? par : 0);
        const float P = ok ? probability(to_f32(p[row * ldp + tok])) : 0.f;
        const float Q = ok && HAS_Q ? probability(to_f32(q[row * ldq + tok])) : 0.f;
        if (ok) atomicMin(&s_first[par], t);
        s_first_yes[t] = P > 0.f && __fmul_rn(coin, HAS_Q ? Q : 1.f) < P;
        s_p[t] = P;
        s_q[t] = Q;
        s_parent[t] = ok ? par : -1;
        s_token[t] = tok;
        s_coin[t] = coin;
    }
    __syncthreads();

    int round = 0;
    bool ok = true;
    long long before = 0;  // mass of the CTAs before this one
    // Total mass of the node's rows after n refusals.  Each CTA's goes to all
    // others by a store that counts on their barriers (a cluster barrier took
    // 1.5 us); round r's barrier and totals are used again in round r + 2,
    // which no CTA enters before every other one has left round r.
    auto total_mass = [&](int n) -> long long {
        const long long mine = mass(n);
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        ++round;
        long long *totals = s_total[round & 1];
        uint64_t *bar = &s_bar[round & 1];
        if (round == 1) cluster_wait();  // (1)
        bool got = true;
        if (warp == 0) {
            const long long own = lane < kWarps ? s_warp[lane] : 0;
            long long upto = own;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += y;
            }
            if (lane < kWarps) s_before[lane] = upto - own;
            const long long all = __shfl_sync(0xffffffffu, upto, 31);
            if (lane == 0) sm100::mbar_arrive_expect_tx(bar, 8 * cluster);
            __syncwarp();
            if (lane < cluster) store_remote(totals + rank, bar, lane, all);
            got = sm100::mbar_wait_bounded(bar, (uint32_t)(round - 1) >> 1 & 1u, kWaitNs);
        }
        ok = __syncthreads_and(got) != 0;
        long long sum = 0;
        before = 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
            const long long x = r < cluster ? totals[r] : 0;
            sum += x;
            if (r < rank) before += x;
        }
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
                // first children one after the other, as far as they are accepted
                int t = T;
                if (out == 0 && tried == here) {
                    t = s_first[here];
                    if (t < T && s_first_yes[t]) {
                        here = tried = t;
                        summed = false;
                        if (writer) my_path[n] = t;
                        ++n;
                        continue;
                    }
                }
                // the next child of `here` behind node `tried`
                for (int base = (tried + 1) & ~31; t == T && base < T; base += 32) {
                    const int at = base + lane;
                    const unsigned hit = __ballot_sync(
                        0xffffffffu, at > tried && at < T && s_parent[min(at, T - 1)] == here);
                    if (hit) t = base + __ffs(hit) - 1;
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
        if (!ok) break;
        summed = total > 0;  // without mass the weights stay those of before
        if (tid == 0) s_norm[out - 1] = mass_of(total);
        __syncthreads();
    }
    if (writer) {
        for (int i = n; i < max_path; ++i) my_path[i] = -1;
        n_path[b] = n;
    }

    // ---- the next token
    if (ok && (!HAS_Q || !summed)) {
        if (KEEP)
            hold(here);
        else
            take_rows(here);
        total = total_mass(out);
    }
    if (!HAS_Q && ok && total == 0 && out > 0) {  // nothing left: the row as it was
        out = 0;
        total = total_mass(0);
    }
    if (!ok) {  // a total did not come: never leave with others' stores on their way here
        if (tid == 0) {
            atomicOr(dev_error, 1);
            sm100::mbar_wait_bounded(&s_bar[round & 1], (uint32_t)(round - 1) >> 1 & 1u, kWaitNs);
        }
        return;
    }
    if (total == 0) {
        if (writer) next_token[b] = -1;
        return;
    }
    const float top = 1.f - 1.f / (1 << kUBits);
    const long long m = (long long)__fmul_rn(fminf(fmaxf(uu, 0.f), top), (float)(1 << kUBits));
    const long long low = (1 << kUBits) - 1;
    // floor(total m / 2^24)
    long long goal = (total >> kUBits) * m + (((total & low) * m) >> kUBits);
    goal -= before + s_before[warp];
    if (goal < 0 || goal >= s_warp[warp]) return;  // in another warp's part
    // the group of batches, the batch, the unit, the lane, the element
    long long upto = group;  // of the lanes up to this one
    auto scan = [&]() {
        const long long own = upto;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += y;
        }
        return own;
    };
    const long long mine = scan();
    const int to = __ffs(__ballot_sync(0xffffffffu, goal < upto)) - 1;
    goal -= __shfl_sync(0xffffffffu, upto - mine, to);
    // a batch from unit `at` on; whether the goal was in it, else its mass is taken off the goal
    auto in_batch = [&](int at, const uint4 *pv, const uint4 *qv) -> bool {
        float x[kAhead * N];
        weights(pv, qv, out, x);
        const int i0 = at * kWide + lane * N - shift;  // of the first unit
        if (!HAS_Q)
            for (int s = 0; s < out; ++s) {
                const int gone = s_token[s_refused[s]] - i0;
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (gone == k * kWide + e) x[k * N + e] = 0.f;
            }
        int unit = -1;
        float y[N] = {};
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            Mass part;
#pragma unroll
            for (int e = 0; e < N; ++e) part.add(x[k * N + e]);
            const long long sum = part.of_warp();
            if (unit < 0 && goal < sum) {
                unit = k;
                upto = part.own();
#pragma unroll
                for (int e = 0; e < N; ++e) y[e] = x[k * N + e];
            }
            if (unit < 0) goal -= sum;
        }
        if (unit < 0) return false;
        const long long own = scan();
        long long run = upto - own;  // of the lanes before this one
        if (run <= goal && goal < upto) {
            int found = -1;  // the first element whose running sum is above
#pragma unroll
            for (int e = 0; e < N; ++e) {
                run += fix(y[e]);
                if (found < 0 && run > goal) found = e;
            }
            next_token[b] = i0 + unit * kWide + found;
        }
        return true;
    };
    if constexpr (KEEP) {
        in_batch(u0, kept_p, kept_q);
    } else {
        for (int at = u0 + to * per_group * kAhead; at < u1; at += kAhead) {
            uint4 pv[kAhead], qv[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                load_unit(at + k, u1, HAS_Q && out > 0, pv[k], qv[k]);
            if (in_batch(at, pv, qv)) return;
        }
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

template <typename Tp, bool HAS_Q, bool KEEP, int THREADS, int AHEAD>
cudaError_t launch_clusters(const VerifyArgs &a, int c, cudaStream_t stream) {
    int *err = nullptr, log_c = 0;
    cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return e;
    while (1 << log_c < c) ++log_c;
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
    e = cudaLaunchKernelEx(
        &cfg, gdr_verify_kernel<Tp, HAS_Q, KEEP, THREADS, AHEAD>, static_cast<const Tp *>(a.p),
        static_cast<const Tp *>(a.q), a.tokens, a.parent, a.coins, a.u, a.path, a.n_path,
        a.next_token, a.T, a.V, a.ldp, a.ldq, a.parent_sb, a.parent_st, a.max_path, log_c, err);
    trace_end(kKernVerify, stream);
    return e;
}

// CTAs per tree (a power of two up to the cluster limit) and variant, by the
// number of trees and the length of a row.  Figures: us on the device, chains
// of 8 nodes, f32 with q.
// Where a lane's part of the row fits one batch, it is kept, with the fewest
// threads that suffice: 32,000 elements, one tree: 4.8 kept by 256 threads, 5.3 by 512, 6.0
// streamed; 60,000: 5.4 kept by 512, 6.5 streamed.  (Two batches a lane kept:
// 7.0 at 131,072 elements, the same as streamed.)  There every tree gets as
// many CTAs as SMs and row allow (32,000 elements, one tree: 8.6 / 6.6 / 5.5 /
// 4.8 with 1 / 2 / 4 / 8), each with a vector at least for each of 256 threads.
// Clusters of 8 do not fill the device (a cluster keeps to one processing
// cluster of SMs): 7 of 8 SMs are counted (2,000 elements, 64 trees: 10.3
// with 8 CTAs each, 5.6 with 1).
// Otherwise CTAs of 256 threads, two a SM, stream the rows, as many per tree as
// the device's slots (two a SM) hold with 2048 elements each (131,072 elements, 64
// trees: 25.3 / 18.2 / 16.4 / 20.7 with 1 / 2 / 4 / 8; one tree: 17.6 / 11.9 / 8.7 /
// 7.0).  Powers of two leave slots empty in between, and at the last batch of a size
// its clusters do not all find room at once: 32 / 38 trees with 8 CTAs each 11.1 / 17.2, 39
// / 45 / 50 / 60 / 64 / 76 with 4 each 13.6 / 14.5 / 14.9 / 16.0 / 16.4 / 25.1, 77 with 2 each
// 20.1.
template <typename Tp, bool HAS_Q>
cudaError_t launch_q(const VerifyArgs &a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    constexpr int N = Vec<Tp>::N, kBatch = kKeepAhead * 4 / N;  // units
    int c = 1;
    while (c < kMaxCluster && (long long)a.B * 2 * c <= sms * 7 / 8 && a.V >= 2 * c * 256 * N)
        c *= 2;
    if (a.B <= sms) {
        // the units of a warp, of a row that may begin anywhere in a vector
        const int units = (a.V + N - 1 + 32 * N - 1) / (32 * N), per_cta = (units + c - 1) / c;
        if ((per_cta + 7) / 8 <= kBatch)
            return launch_clusters<Tp, HAS_Q, true, 256, kKeepAhead>(a, c, stream);
        if ((per_cta + 15) / 16 <= kBatch)
            return launch_clusters<Tp, HAS_Q, true, 512, kKeepAhead>(a, c, stream);
    }
    c = 1;
    while (c < kMaxCluster && (long long)a.B * 2 * c <= 2LL * sms && a.V / (2 * c) >= 2048) c *= 2;
    return launch_clusters<Tp, HAS_Q, false, 256, kStreamAhead>(a, c, stream);
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
    const VerifyArgs a{p, q, tokens, parent, coins, u, path, n_path, next_token,
                       B, T, V, ldp, ldq, parent_sb, parent_st, max_path};
    const cudaError_t e =
        prob_dtype == GDR_BF16
            ? (q ? launch_q<__nv_bfloat16, true>(a, s) : launch_q<__nv_bfloat16, false>(a, s))
            : (q ? launch_q<float, true>(a, s) : launch_q<float, false>(a, s));
    if (e == cudaSuccess) return GDR_OK;
    record_cuda_error(e);
    return GDR_ERR_CUDA;
}
