// path_commit.cu -- gdr_commit_path: the state after the accepted nodes of a
// draft.
//
// Each node on the path takes the token recurrence's step without its output:
//     s_ij <- a_i s_ij            a_i = exp(g_i)
//     d_j   = beta (v_j - sum_i k_i s_ij)
//     s_ij <- s_ij + k_i d_j
// The columns j of a state never meet, so the state is cut along them and
// stays in registers over the whole path: read once, written once, which is
// what bounds the call for paths of up to about ten nodes (three operations
// an element and node against eight bytes an element).
//
// Measured on the device: 64 x 32 heads of 128 x 128, paths of 1 to 8 nodes,
// 50.2 us (277 MB at 5.5 TB/s, 0.81 of a copy's rate), of one node 45.7 us (0.86), of 64
// nodes 283 us (0.29 us a head and node on an SM, bound by its FMA pipes).  With few
// heads an SM their lengths do not even out: 16 x 32 heads 20.4 us (0.50 of a
// copy's rate), of one node 13.6 us (0.74).  Other dims, paths of 1 to 5 nodes:
// 64 x 32 heads of 64 x 64 18 us (0.57; 16 x 32 heads 0.41), of 128 x 64 30 us (0.68),
// in f32 41 us (0.50).
//
// The kernel for heads other than 128 x 128: a warp owns 16 columns of a head's
// state; lane (cq = lane % 4, rg = lane / 4) holds columns 4 cq .. 4 cq + 3 of
// the rows rg + 8 m.  A row's 16 columns are 64 contiguous bytes, the sum over
// the rows stays inside the warp, and between the nodes no warp waits for
// another.  The arithmetic is on pairs of columns (fma.rn.f32x2: two roundings
// as by two fma).  k and exp(g) of a batch of nodes are staged in shared memory
// as (k, k, a, a), the pairs' form.  What bounds it is a chain in front of every
// tile (path length, path, nodes, with nothing of the next tile in flight).  The
// next batch of nodes waits in registers; with f32 nodes and dk = 128 they do not all
// fit beside the state (172 bytes of spills; dk = 64: 20, bf16 dk = 128: 12).
#include <stdint.h>

#include "common.cuh"
#include "gdr.h"
#include "host_checks.h"
#include "sm100_ptx.cuh"

namespace gdr {
namespace {

constexpr int kNodes = 8;      // nodes staged at a time
constexpr int kWarpCols = 16;  // columns of a warp
constexpr int kCols = 32;      // of a CTA

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

// One CTA: kCols columns of one head, two warps.  (Four warps, which stage k
// and exp(g) half as often: 2 x 32 heads of 64 x 64, paths of up to 6 nodes,
// 3.3 us either way; 64 x 32 heads 18.3 against 18.6, of 128 x 64 31.4
// against 31.5.)
template <typename Tin, int DK, bool GS>
__global__ void __launch_bounds__(2 * kCols, DK == 128 ? 6 : 8)
    gdr_commit_kernel(const Tin *__restrict__ k, const Tin *__restrict__ v,
                      const float *__restrict__ g, const float *__restrict__ beta,
                      const float *h0, float *ht, const int *__restrict__ path,
                      const int *__restrict__ n_path, int T, int HK, int HV, int dv,
                      int max_path) {
    constexpr int BV = kCols, NT = 2 * BV, RM = DK / 8;
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
    // The nodes of a batch are loaded while the batch before is worked through.
    // Element i of a thread's loads is that of node (i NT + tid) / DK (of k
    // and g; v: / BV); `entry` holds the path's entries at & ~31 + lane.
    constexpr int kK = kNodes * DK / NT, kV = kNodes * BV / NT;
    Tin kx[kK], vx[kV];
    float gx[kK], bt = 0.f;
    int entry = -1, cnt = 0;
    auto load = [&](int at) {
        if ((at & 31) == 0)
            entry = at + lane < n ? path[(size_t)b * max_path + at + lane] : -1;
        // the path ends before the first invalid entry
        const unsigned good = __ballot_sync(0xffffffffu, entry >= 0 && entry < T);
        cnt = min(kNodes, __ffs(~(good >> (at & 31) & ((1u << kNodes) - 1))) - 1);
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            const int c = (i * NT + tid) / DK, r = (i * NT + tid) % DK;
            const int t = __shfl_sync(0xffffffffu, entry, (at & 31) + c);
            if (c < cnt) {
                const size_t row = (size_t)b * T + t;
                kx[i] = k[(row * HK + hk) * DK + r];
                gx[i] = GS ? g[row * HV + hv] : g[(row * HV + hv) * DK + r];
            }
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int c = (i * NT + tid) / BV, j = (i * NT + tid) % BV;
            const int t = __shfl_sync(0xffffffffu, entry, (at & 31) + c);
            if (c < cnt) vx[i] = v[(((size_t)b * T + t) * HV + hv) * dv + tile * BV + j];
        }
        const int t = __shfl_sync(0xffffffffu, entry, (at & 31) + lane % kNodes);
        if (lane < cnt) bt = beta[((size_t)b * T + t) * HV + hv];
    };
    if (n > 0) load(0);
    for (int at = 0; at < n; at += kNodes) {
        if (at > 0) __syncthreads();  // the batch before has been used
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            const int c = (i * NT + tid) / DK, r = (i * NT + tid) % DK;
            const float kk = to_f32(kx[i]), a = expf(gx[i]);
            if (c < cnt) s_ka[c][r] = make_float4(kk, kk, a, a);
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int c = (i * NT + tid) / BV, j = (i * NT + tid) % BV;
            if (c < cnt) s_v[c][j] = to_f32(vx[i]);
        }
        const float b_batch = bt;
        const int steps = cnt;
        __syncthreads();
        if (steps == kNodes && at + kNodes < n) load(at + kNodes);
        for (int c = 0; c < steps; ++c) {
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
            const float2 x = split(add2(acc[0][0], acc[1][0]));
            const float2 y = split(add2(acc[0][1], acc[1][1]));
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
            const float b_t = __shfl_sync(0xffffffffu, b_batch, c);
            const float d = b_t * (s_v[c][warp * kWarpCols + mine] - sum);
            const Pair d0 =
                pair(__shfl_sync(0xffffffffu, d, cq), __shfl_sync(0xffffffffu, d, cq + 8));
            const Pair d1 =
                pair(__shfl_sync(0xffffffffu, d, cq + 4), __shfl_sync(0xffffffffu, d, cq + 12));
#pragma unroll
            for (int m = 0; m < RM; ++m) {
                const Pair kk{*reinterpret_cast<const unsigned long long *>(&s_ka[c][rg + 8 * m])};
                s[m][0] = fma2(kk, d0, s[m][0]);
                s[m][1] = fma2(kk, d1, s[m][1]);
            }
        }
        if (steps < kNodes) break;
    }
    float *to = ht + base;
#pragma unroll
    for (int m = 0; m < RM; ++m, to += 8 * dv) {
        const float2 x = split(s[m][0]), y = split(s[m][1]);
        stg_stream4(to, make_float4(x.x, x.y, y.x, y.y));
    }
}

// ---- dk = dv = 128: persistent, the 64 KB states by bulk copies.
//
// One CTA per SM walks heads blockIdx.x, + gridDim.x, ...  The kernel above
// waits for a chain of loads (path length, path, k / g / v of its nodes)
// before a head's first step and has nothing else to do meanwhile.  Here a
// head belongs to one of two groups of four warps in turn; two or four producer
// warps per group bring its heads' nodes (k, exp(g), v, beta as float32, one or
// two nodes each of a slot of four, the next slot's loads in flight), the first
// of them also the states (three 64 KB buffers, which the groups share in the order
// of the heads).  A group copies its state into registers, frees the buffer
// at once and stores from the registers, so that all three buffers are
// reads ahead.
//
// Warp w of a group owns columns 32 w .. + 31: lane (cq = lane % 8, rg = lane
// / 8) holds columns 4 cq .. + 3 of the rows 4 rg + 16 m .. + 3 (m < 8) as
// pairs of rows, so that k and a are pairs as they lie in shared memory.
//
// Against the kernel above at 128 x 128 (32 heads / 64 x 32 heads, all paths of
// one length): one node 4.2 / 45.7 us against 3.9 / 46.7, 8 nodes 7.2 / 55
// against 8.8 / 73, 64 nodes 29 / 283 against 60 / 443.  One producer warp per
// group instead of two: 67 us for 64 x 32 heads with paths of 1 to 8 nodes,
// against 50.  Taking four nodes in one step, with the decays multiplied out, saves a
// quarter of the operations and costs the producers more: 261 us for 64
// nodes, but 5.2 / 47.4 for one and 54 for 1 to 8.
constexpr int kD = 128;
constexpr int kBufs = 3;
constexpr int kSlots = 2;
constexpr int kSlotNodes = 4;
constexpr int kGroups = 2;
constexpr int kGroupWarps = 4;
// Producer warps per group, and the registers of a thread: the warpgroups of
// the states are given some that the producers' were launched with.  float32
// nodes are twice the bytes and want twice the warps (64 x 32 heads, paths of 1
// to 8 nodes: 51 us, 58 with two; bf16: 50 and 50, at 1 to 20 nodes 82 and 75).
template <typename Tin>
struct Producers {  // 384 threads of 168 registers: 2 x 128 x 208 + 128 x 88
    static constexpr int kWarps = 2, kStateRegs = 208, kRegs = 88;
};
template <>
struct Producers<float> {  // 512 threads of 128 registers: 2 x 128 x 184 + 2 x 128 x 72
    static constexpr int kWarps = 4, kStateRegs = 184, kRegs = 72;
};
template <typename Tin>
constexpr int kBulkThreads = kGroups * (kGroupWarps + Producers<Tin>::kWarps) * 32;
constexpr uint32_t kStateBytes = kD * kD * 4;
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s

static_assert(kBufs == 3 && kGroups == 2, "the order of the waits goes by these");

struct Slot {
    float k[kSlotNodes][kD], a[kSlotNodes][kD], v[kSlotNodes][kD];
    float beta[kSlotNodes];
    int count, last, pad[2];
};
struct BulkShared {
    float state[kBufs][kD * kD];
    Slot slot[kGroups][kSlots];
    uint64_t state_full[kBufs], state_empty[kBufs];
    uint64_t full[kGroups][kSlots], empty[kGroups][kSlots];
};

// Four elements of a row as they lie in memory.
template <typename Tin>
struct Raw4;
template <>
struct Raw4<float> {
    float4 x;
    __device__ __forceinline__ void load(const float *p) { x = load4(p); }
    __device__ __forceinline__ float4 f32() const { return x; }
};
template <>
struct Raw4<__nv_bfloat16> {
    uint2 x;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        x = *reinterpret_cast<const uint2 *>(p);
    }
    __device__ __forceinline__ float4 f32() const {
        return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                           __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
    }
};

// Whether the phase with that parity has completed; returns at once.
__device__ __forceinline__ bool test_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(sm100::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// A wait of a whole warp, with the same answer in every lane.  A group polls,
// looking at the clock every 1024 polls; a producer sleeps in the barrier, so
// as not to take issue slots from the groups it waits for.
template <bool SLEEP>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    if (SLEEP)
        return __all_sync(0xffffffffu, sm100::mbar_wait_bounded(bar, parity, kWaitNs));
    if (__all_sync(0xffffffffu, sm100::mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = sm100::global_timer_ns();
    for (int n = 0;; ++n) {
        if (__all_sync(0xffffffffu, sm100::mbar_try_wait(bar, parity))) return true;
        if ((n & 1023) == 1023 &&
            __any_sync(0xffffffffu, sm100::global_timer_ns() - t0 > kWaitNs))
            return false;
    }
}

template <typename Tin, bool GS>
__global__ void __launch_bounds__(kBulkThreads<Tin>, 1)
    gdr_commit_bulk_kernel(const Tin *__restrict__ k, const Tin *__restrict__ v,
                           const float *__restrict__ g, const float *__restrict__ beta,
                           const float *h0, float *ht, const int *__restrict__ path,
                           const int *__restrict__ n_path, int T, int HK, int HV, int max_path,
                           int nheads, int *dev_error) {
    constexpr int kProducers = Producers<Tin>::kWarps;
    constexpr int kOwn = kSlotNodes / kProducers;  // nodes of a slot per producer warp
    extern __shared__ __align__(128) unsigned char smem_raw[];
    BulkShared &sh = *reinterpret_cast<BulkShared *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < kBufs; ++i) {
            sm100::mbar_init(&sh.state_full[i], 1);
            sm100::mbar_init(&sh.state_empty[i], kGroupWarps);
        }
        for (int i = 0; i < kGroups; ++i)
            for (int j = 0; j < kSlots; ++j) {
                sm100::mbar_init(&sh.full[i][j], kProducers);
                sm100::mbar_init(&sh.empty[i][j], kGroupWarps);
            }
        sm100::fence_mbar_init();
    }
    __syncthreads();
    // the CTA's heads: number i is head blockIdx.x + i gridDim.x, in buffer i % kBufs
    const int my = (nheads - 1 - (int)blockIdx.x) / (int)gridDim.x + 1;
    bool ok = true;

    if (warp >= kGroups * kGroupWarps) {
        // ---- producers of group grp: heads grp, grp + 2, ...
        // Warp number `part` brings kOwn nodes of each slot; the first also
        // asks for the states and writes the slot's count.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Producers<Tin>::kRegs));
        const int producer = warp - kGroups * kGroupWarps;
        const int grp = producer / kProducers, part = producer % kProducers;
        int next_state = grp;  // the group's next head whose state has not been asked for
        // Asks for the states of heads up to `upto`, waiting for their buffers,
        // and up to `may` where that needs no wait.  A buffer's barriers tell
        // a phase only from the one before it, so head i's state may be asked for only once
        // head i - 6, the user of its buffer two uses ago, is known to have been
        // read: head i - 6 is this group's, every head takes at least one
        // slot, and a slot is filled again only after the group has
        // worked through it.  Before the wait for the slot of a head's
        // nodes that is known for the head itself, after it for the next one.
        auto states = [&](int upto, int may) {
            while (part == 0 && ok && h0 && next_state < my && next_state <= may) {
                const int buf = next_state % kBufs, use = next_state / kBufs;
                if (use > 0) {
                    const uint32_t parity = (uint32_t)(use - 1) & 1u;
                    if (next_state <= upto)
                        ok = warp_wait<true>(&sh.state_empty[buf], parity);
                    else if (!__all_sync(0xffffffffu, test_wait(&sh.state_empty[buf], parity)))
                        break;
                }
                if (ok && lane == 0) {
                    sm100::mbar_arrive_expect_tx(&sh.state_full[buf], kStateBytes);
                    const size_t head = (size_t)blockIdx.x + (size_t)next_state * gridDim.x;
                    sm100::bulk_load_1d(sh.state[buf], h0 + head * kD * kD, kStateBytes,
                                        &sh.state_full[buf]);
                }
                __syncwarp();
                if (ok) next_state += kGroups;
            }
        };
        // sequence, value head and key head of the head whose nodes are loaded;
        // the group's heads are kGroups gridDim.x apart
        const int step_b = kGroups * (int)gridDim.x / HV, step_h = kGroups * (int)gridDim.x % HV;
        const int first = blockIdx.x + grp * gridDim.x;
        const int per_key = HV / HK;
        int b = first / HV, hv = first % HV, hk = hv / per_key;
        // a head's path: its length and entry `from + lane` (of sequence bb)
        auto entries = [&](int bb, int from, int &len) -> int {
            len = n_path[bb];  // held to max_path where it is used: no wait for it here
            return from + lane < max_path ? path[(size_t)bb * max_path + from + lane] : -1;
        };
        struct Nodes {
            Raw4<Tin> k[kOwn], v[kOwn];
            float4 g[kOwn];
            float beta, gate;  // of node `lane`
            int count, last;
        };
        int head_i = grp, at = 0, n = 0, n_next = 0, entry = -1, entry_next = -1;
        if (head_i < my) entry = entries(b, 0, n);
        states(grp, grp + kGroups);
        auto next_b = [&]() { return b + step_b + (hv + step_h >= HV ? 1 : 0); };
        if (head_i + kGroups < my) entry_next = entries(next_b(), 0, n_next);
        // loads this warp's nodes of at .. at + 3 of head head_i, up to the path's end
        auto load = [&](Nodes &x) {
            n = min(n, max_path);
            const unsigned good =
                __ballot_sync(0xffffffffu, (at & ~31) + lane < n && entry >= 0 && entry < T);
            x.count = min(kSlotNodes, __ffs(~(good >> (at & 31) & ((1u << kSlotNodes) - 1))) - 1);
            x.last = x.count < kSlotNodes || at + kSlotNodes >= n;
            const size_t row = (size_t)b * T;
#pragma unroll
            for (int c = 0; c < kOwn; ++c) {
                const int node = part * kOwn + c;
                const int t = __shfl_sync(0xffffffffu, entry, (at & 31) + node);
                if (node < x.count) {
                    const size_t krow = (row + t) * HK + hk, vrow = (row + t) * HV + hv;
                    x.k[c].load(k + krow * kD + 4 * lane);
                    x.v[c].load(v + vrow * kD + 4 * lane);
                    if (!GS) x.g[c] = load4(g + vrow * kD + 4 * lane);
                    if (lane == node) x.beta = beta[vrow];
                    if (GS && lane == node) x.gate = g[vrow];
                }
            }
        };
        // to the next nodes; false behind the last head
        auto advance = [&](bool last) -> bool {
            if (!last) {
                at += kSlotNodes;
                if ((at & 31) == 0) entry = entries(b, at, n);
                return true;
            }
            head_i += kGroups;
            if (head_i >= my) return false;
            b = next_b();
            hv += step_h;
            if (hv >= HV) hv -= HV;
            hk = hv / per_key;
            at = 0;
            n = n_next;
            entry = entry_next;
            if (head_i + kGroups < my) entry_next = entries(next_b(), 0, n_next);
            return true;
        };
        // puts nodes x, of head this_head, into the group's slot number `number`
        auto place = [&](const Nodes &x, int this_head, int number) {
            states(this_head, this_head);  // the group may wait for it before it frees a slot
            const int to = number % kSlots;
            Slot &slot = sh.slot[grp][to];
            if (ok && number >= kSlots)
                ok = warp_wait<true>(&sh.empty[grp][to], (uint32_t)(number / kSlots - 1) & 1u);
            if (!ok) return;
            states(this_head, this_head + kGroups);
#pragma unroll
            for (int c = 0; c < kOwn; ++c) {
                const int j = part * kOwn + c;
                const float gate = GS ? __shfl_sync(0xffffffffu, x.gate, j) : 0.f;
                if (j < x.count) {
                    store4(&slot.k[j][4 * lane], x.k[c].f32());
                    store4(&slot.v[j][4 * lane], x.v[c].f32());
                    float4 a;
                    if (GS) {
                        a.x = a.y = a.z = a.w = expf(gate);
                    } else {
                        a = make_float4(expf(x.g[c].x), expf(x.g[c].y), expf(x.g[c].z),
                                        expf(x.g[c].w));
                    }
                    store4(&slot.a[j][4 * lane], a);
                }
            }
            if (lane / kOwn == part && lane < x.count) slot.beta[lane] = x.beta;
            if (part == 0 && lane == 0) {
                slot.count = x.count;
                slot.last = x.last;
            }
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&sh.full[grp][to]);
        };
        // the loads of one slot's nodes are in flight while the one before is placed
        Nodes x, y;
        int x_head = head_i, y_head = 0;
        bool x_more = head_i < my, y_more = false;
        if (x_more) load(x);
        for (int c = 0; ok && x_more; c += 2) {
            y_more = advance(x.last);
            y_head = head_i;
            if (y_more) load(y);
            place(x, x_head, c);
            if (!ok || !y_more) break;
            x_more = advance(y.last);
            x_head = head_i;
            if (x_more) load(x);
            place(y, y_head, c + 1);
        }
        if (!ok) {
            if (lane == 0) atomicOr(dev_error, 1);
            // never leave with loads in flight into this CTA: the last
            // states asked for, one per buffer at most
            for (int i = next_state - kGroups, j = 0; part == 0 && h0 && i >= 0 && j < kBufs;
                 i -= kGroups, ++j)
                sm100::mbar_wait_bounded(&sh.state_full[i % kBufs], (uint32_t)(i / kBufs) & 1u,
                                         kWaitNs);
        }
        return;
    }

    // ---- group grp
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Producers<Tin>::kStateRegs));
    const int grp = warp / kGroupWarps, cq = lane & 7, rg = lane >> 3;
    const int col = 32 * (warp % kGroupWarps) + 4 * cq;
    const bool odd = rg & 1, high = rg & 2;
    const int mine = col + (odd ? 2 : 0) + (high ? 1 : 0);  // the column whose sum ends here
    int chunk = 0;
    for (int i = grp; i < my; i += kGroups) {
        // The head's nodes first: they are there only after its state was
        // asked for, before which its buffer's barrier would still tell of the
        // use before.
        ok = warp_wait<false>(&sh.full[grp][chunk % kSlots], (uint32_t)(chunk / kSlots) & 1u);
        if (!ok) break;
        Pair s[8][2][4];  // [m][pair of rows][column]
        if (h0) {
            const int buf = i % kBufs;
            ok = warp_wait<false>(&sh.state_full[buf], (uint32_t)(i / kBufs) & 1u);
            if (!ok) break;
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float *row = &sh.state[buf][(4 * rg + 16 * m + 2 * r) * kD + col];
                    const float4 x = load4(row), y = load4(row + kD);
                    s[m][r][0] = pair(x.x, y.x);
                    s[m][r][1] = pair(x.y, y.y);
                    s[m][r][2] = pair(x.z, y.z);
                    s[m][r][3] = pair(x.w, y.w);
                }
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&sh.state_empty[buf]);
        } else {
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[m][r][e] = pair(0.f, 0.f);
        }
        int steps = 0;
        for (bool last = false; !last; ++chunk) {
            const int at = chunk % kSlots;
            ok = warp_wait<false>(&sh.full[grp][at], (uint32_t)(chunk / kSlots) & 1u);
            if (!ok) break;
            const Slot &slot = sh.slot[grp][at];
            const int count = slot.count;
            last = slot.last;
            steps += count;
            for (int c = 0; c < count; ++c) {
                const float *kr = &slot.k[c][4 * rg], *ar = &slot.a[c][4 * rg];
                Pair acc[4];
                ulonglong2 keys[8];
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    const ulonglong2 kk = keys[m] =
                        *reinterpret_cast<const ulonglong2 *>(kr + 16 * m);
                    const ulonglong2 aa = *reinterpret_cast<const ulonglong2 *>(ar + 16 * m);
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[m][r][e] = mul2(s[m][r][e], Pair{r ? aa.y : aa.x});
                            acc[e] = m + r == 0 ? mul2(Pair{kk.x}, s[m][r][e])
                                                : fma2(Pair{r ? kk.y : kk.x}, s[m][r][e], acc[e]);
                        }
                }
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 p = split(acc[e]);
                    x[e] = p.x + p.y;
                }
                // over the four row groups, halving the columns each time
                float p0 = odd ? x[2] : x[0], p1 = odd ? x[3] : x[1];
                p0 += __shfl_xor_sync(0xffffffffu, odd ? x[0] : x[2], 8);
                p1 += __shfl_xor_sync(0xffffffffu, odd ? x[1] : x[3], 8);
                float sum = high ? p1 : p0;
                sum += __shfl_xor_sync(0xffffffffu, high ? p0 : p1, 16);
                const float d = slot.beta[c] * (slot.v[c][mine] - sum);
                Pair dd[4];  // column e is in row group 2 (e & 1) + (e >> 1)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y = __shfl_sync(0xffffffffu, d, cq + 8 * (2 * (e & 1) + (e >> 1)));
                    dd[e] = pair(y, y);
                }
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    const ulonglong2 kk = keys[m];
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[m][r][e] = fma2(Pair{r ? kk.y : kk.x}, dd[e], s[m][r][e]);
                }
            }
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&sh.empty[grp][at]);
        }
        if (!ok) break;
        if (steps == 0 && h0 == ht) continue;
        float *to = ht + ((size_t)blockIdx.x + (size_t)i * gridDim.x) * kD * kD + 4 * rg * kD + col;
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float2 x = split(s[m][r][0]), y = split(s[m][r][1]), z = split(s[m][r][2]),
                             w = split(s[m][r][3]);
                stg_stream4(to + (16 * m + 2 * r) * kD, make_float4(x.x, y.x, z.x, w.x));
                stg_stream4(to + (16 * m + 2 * r + 1) * kD, make_float4(x.y, y.y, z.y, w.y));
            }
    }
    if (!ok && lane == 0) atomicOr(dev_error, 1);
}

struct CommitArgs {
    const void *k, *v;
    const float *g, *beta, *h0;
    float *ht;
    const int *path, *n_path;
    int B, T, HK, HV, dk, dv, max_path;
};

template <typename Tin, bool GS>
cudaError_t launch_bulk(const CommitArgs &a, cudaStream_t stream) {
    int *err = nullptr, dev = 0, sms = 0;
    cudaError_t e = device_error_word(&err);
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int nheads = a.B * a.HV;  // at most 2^30
    const int grid = nheads < sms ? nheads : sms;
    const auto kernel = gdr_commit_bulk_kernel<Tin, GS>;
    // The groups wait for registers that the block has to have been launched with.
    static const int launched = [kernel] {
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, kernel) == cudaSuccess ? f.numRegs : 0;
    }();
    using P = Producers<Tin>;
    constexpr int kWanted =
        kGroups * 32 * (kGroupWarps * P::kStateRegs + P::kWarps * P::kRegs);
    if (launched * kBulkThreads<Tin> < kWanted) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(BulkShared));
    if (e != cudaSuccess) return e;
    trace_begin(kKernCommit, stream);
    kernel<<<grid, kBulkThreads<Tin>, sizeof(BulkShared), stream>>>(
        static_cast<const Tin *>(a.k), static_cast<const Tin *>(a.v), a.g, a.beta, a.h0, a.ht,
        a.path, a.n_path, a.T, a.HK, a.HV, a.max_path, nheads, err);
    trace_end(kKernCommit, stream);
    return cudaGetLastError();
}

template <typename Tin, int DK, bool GS>
cudaError_t launch(const CommitArgs &a, cudaStream_t stream) {
    const long long ctas = (long long)a.B * a.HV * (a.dv / kCols);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    trace_begin(kKernCommit, stream);
    gdr_commit_kernel<Tin, DK, GS><<<(unsigned)ctas, 2 * kCols, 0, stream>>>(
        static_cast<const Tin *>(a.k), static_cast<const Tin *>(a.v), a.g, a.beta, a.h0, a.ht,
        a.path, a.n_path, a.T, a.HK, a.HV, a.dv, a.max_path);
    trace_end(kKernCommit, stream);
    return cudaGetLastError();
}

template <typename Tin, bool GS>
cudaError_t launch_dk(const CommitArgs &a, cudaStream_t stream) {
    if (a.dk == kD && a.dv == kD) return launch_bulk<Tin, GS>(a, stream);
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
