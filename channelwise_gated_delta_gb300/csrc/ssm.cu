// ssm.cu -- gdr_ssm_forward: the selective state space recurrence on states
// [dk][dv], per token
//     step = softplus(dt + dt_bias),  S <- exp(step A) S + step b x^T,
//     out = S^T c + D x, times silu(z).
//
// gdr_ssm_walk_kernel runs it token by token, in float32 throughout, for
// every type and size.  One CTA per (unit of a sequence, value head, 32 or 64
// columns); warp w holds the rows w dk / 4 .. of the columns of its lanes in
// registers, so that a token is three operations an element of the state (two
// elements at a time) and no exchange: the four warps' partial outputs meet in
// shared memory once every kTok tokens, and the next ones' inputs (z too: read
// where it is used it cost 565 us in place of 394) are on their way meanwhile.
// 4 x 1024 tokens of 32 gated heads of 128 x 128, f32: 394 us, where the operations
// at two a lane and cycle take 172 on all SMs and 205 as its 256 CTAs lie; the
// rest is latency, of the loads of b and c from shared memory before all.
// gdr_ssm_step_kernel is one pass over the states of single tokens, bound by
// memory; bf16 sequences take the chunks of ssm_tc.cu.
#include <limits.h>
#include <stdint.h>

#include "gdr.h"
#include "sm100_ptx.cuh"
#include "ssm.cuh"

namespace gdr {
namespace {

using sm100::fma2;
using sm100::mul2;

constexpr int kTok = 16;
constexpr int kThreads = 128;
constexpr int kWideSms = 152;

template <typename T, int DK, int PASS, int COLS>
__global__ void __launch_bounds__(kThreads)
    gdr_ssm_walk_kernel(const __grid_constant__ SsmArgs a, const __grid_constant__ SeqTable table) {
    constexpr int R = DK / 4;          // rows of a warp
    constexpr int kCols = 32 * COLS;   // columns of the CTA, a lane's 32 apart
    __shared__ __align__(16) float sb[kTok][DK], sc[kTok][DK];
    __shared__ float sx[kTok][kCols], part[4][kTok][kCols], sstep[kTok], sdec[kTok], slog[kTok];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tiles = a.dv / kCols;
    const int tile = blockIdx.x % tiles, rest = blockIdx.x / tiles;
    const int hv = rest % a.HV, hk = hv / (a.HV / a.HK);
    const SeqUnit u = find_unit(table, rest / a.HV);
    const int unit = table.unit0 + rest / a.HV;
    const long long cut = a.seg_rows;
    const int t0 = (int)(u.unit * cut), t1 = (int)min((long long)u.len, t0 + cut);
    if (PASS == 1 && t1 == u.len) return;  // no unit follows
    const size_t per = (size_t)DK * a.dv;

    float2 S[COLS][R / 2];  // rows 2 i and 2 i + 1 of the warp's, two operations at a time
    const size_t at = (size_t)(warp * R) * a.dv + tile * kCols + lane;
#pragma unroll
    for (int j = 0; j < COLS; ++j)
#pragma unroll
        for (int i = 0; i < R / 2; ++i) S[j][i] = make_float2(0.f, 0.f);
    auto rows = [&](const float *p, float keep) {  // S <- keep S + what stands at p
#pragma unroll
        for (int j = 0; j < COLS; ++j)
#pragma unroll
            for (int i = 0; i < R / 2; ++i)
                S[j][i] = fma2(make_float2(keep, keep), S[j][i],
                               make_float2(p[(size_t)(2 * i) * a.dv + 32 * j],
                                           p[(size_t)(2 * i + 1) * a.dv + 32 * j]));
    };
    if (a.h0 && u.unit == 0) rows(a.h0 + ((size_t)u.seq * a.HV + hv) * per + at, 0.f);
    if (PASS == 2)
        for (int i = 0; i < u.unit; ++i) {
            const size_t s = (size_t)(unit - u.unit + i) * a.HV + hv;
            rows(a.seg_state + s * per + at, expf(a.seg_log[s]));
        }

    const T *x = static_cast<const T *>(a.x) + u.row0 * a.ldx + (size_t)hv * a.dv + tile * kCols;
    const T *b = static_cast<const T *>(a.b) + u.row0 * a.ldb + (size_t)hk * DK;
    const T *c = static_cast<const T *>(a.c) + u.row0 * a.ldc + (size_t)hk * DK;
    const T *z = a.z ? static_cast<const T *>(a.z) + u.row0 * a.ldz + (size_t)hv * a.dv + tile * kCols : nullptr;
    const float *dt = a.dt + u.row0 * a.HV + hv;
    const float A = a.A[hv], bias = a.dt_bias ? a.dt_bias[hv] : 0.f, D = a.D ? a.D[hv] : 0.f;
    float total = 0.f;

    constexpr int NB = kTok * DK / kThreads, NX = kTok * kCols / kThreads;
    float rb[NB], rc[NB], rx[NX], rz[NX], gate[NX], rdt = 0.f;
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int e = tid + kThreads * i, k = e / DK, ch = e % DK;
            const bool in = t + k < t1;
            rb[i] = in ? to_f32(b[(t + k) * a.ldb + ch]) : 0.f;
            rc[i] = in && PASS != 1 ? to_f32(c[(t + k) * a.ldc + ch]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int e = tid + kThreads * i, k = e / kCols;
            rx[i] = t + k < t1 ? to_f32(x[(t + k) * a.ldx + e % kCols]) : 0.f;
            if (PASS != 1) rz[i] = a.z && t + k < t1 ? to_f32(z[(t + k) * a.ldz + e % kCols]) : 0.f;
        }
        if (tid < kTok && t + tid < t1) rdt = dt[(long long)(t + tid) * a.HV];
    };
    fetch(t0);
    for (int t = t0; t < t1; t += kTok) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int e = tid + kThreads * i;
            sb[e / DK][e % DK] = rb[i];
            sc[e / DK][e % DK] = rc[i];
        }
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int e = tid + kThreads * i;
            sx[e / kCols][e % kCols] = rx[i];
            if (PASS != 1) gate[i] = rz[i];
        }
        if (tid < kTok) {
            const float step = t + tid < t1 ? ssm_step(rdt, bias, a.softplus) : 0.f;
            sstep[tid] = step;
            slog[tid] = step * A;
            sdec[tid] = expf(step * A);
        }
        __syncthreads();
        if (t + kTok < t1) fetch(t + kTok);
        const int n = min(kTok, t1 - t);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float keep = sdec[k];
            if (PASS == 1) total += slog[k];
            const float2 keep2 = make_float2(keep, keep);
            float2 xs[COLS], y[COLS], y2[COLS];
#pragma unroll
            for (int j = 0; j < COLS; ++j) {
                const float q = sstep[k] * sx[k][lane + 32 * j];
                xs[j] = make_float2(q, q);
                y[j] = y2[j] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int r = 0; r < R; r += 4) {
                const float4 bv = *reinterpret_cast<const float4 *>(&sb[k][warp * R + r]);
                float4 cv = make_float4(0.f, 0.f, 0.f, 0.f);
                if (PASS != 1) cv = *reinterpret_cast<const float4 *>(&sc[k][warp * R + r]);
#pragma unroll
                for (int j = 0; j < COLS; ++j) {
                    float2 &s0 = S[j][r / 2], &s1 = S[j][r / 2 + 1];
                    s0 = fma2(keep2, s0, mul2(make_float2(bv.x, bv.y), xs[j]));
                    s1 = fma2(keep2, s1, mul2(make_float2(bv.z, bv.w), xs[j]));
                    if (PASS != 1) {
                        y[j] = fma2(make_float2(cv.x, cv.y), s0, y[j]);
                        y2[j] = fma2(make_float2(cv.z, cv.w), s1, y2[j]);
                    }
                }
            }
            if (PASS != 1)
#pragma unroll
                for (int j = 0; j < COLS; ++j) part[warp][k][lane + 32 * j] = (y[j].x + y[j].y) + (y2[j].x + y2[j].y);
        }
        __syncthreads();
        if (PASS != 1) {
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const int e = tid + kThreads * i, k = e / kCols, col = e % kCols;
                if (k >= n) continue;
                float y = (part[0][k][col] + part[1][k][col]) + (part[2][k][col] + part[3][k][col]);
                y = fmaf(D, sx[k][col], y);
                const size_t row = (size_t)(u.row0 + t + k);
                const size_t o = (size_t)hv * a.dv + tile * kCols + col;
                if (a.z) y = ssm_gate(y, gate[i]);
                static_cast<T *>(a.out)[row * a.HV * a.dv + o] = from_f32<T>(y);
            }
            __syncthreads();
        }
    }
    float *end = nullptr;
    if (PASS == 1) {
        const size_t s = (size_t)unit * a.HV + hv;
        end = a.seg_state + s * per;
        if (tid == 0 && tile == 0) a.seg_log[s] = total;
    } else if (a.ht && t1 == u.len) {
        end = a.ht + ((size_t)u.seq * a.HV + hv) * per;
    }
    if (end)
#pragma unroll
        for (int j = 0; j < COLS; ++j)
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
                end[at + (size_t)(2 * i) * a.dv + 32 * j] = S[j][i].x;
                end[at + (size_t)(2 * i + 1) * a.dv + 32 * j] = S[j][i].y;
            }
}

// Sequences of one token (or none): one CTA per (sequence, value head) passes
// its state through registers once, 16 bytes a thread and row; a warp's row
// or rows are adjacent, and all of a thread's loads are in flight together.
// 64 sequences of 32 heads of 128 x 128: 42 us, 6.4 TB/s (the walk takes 86).
constexpr int kStepWarps = 8;

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(32 * kStepWarps)
    gdr_ssm_step_kernel(const __grid_constant__ SsmArgs a, const __grid_constant__ SeqTable table) {
    constexpr int L = DV / 4, RW = 32 / L;              // lanes of a row, rows of a warp's access
    constexpr int N = DK / (RW * kStepWarps);           // accesses of a thread
    __shared__ float sb[DK], sc[DK];
    __shared__ __align__(16) float part[kStepWarps][DV];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane / L, col = 4 * (lane % L);
    const int hv = blockIdx.x % a.HV, hk = hv / (a.HV / a.HK);
    const SeqUnit u = find_unit(table, blockIdx.x / a.HV);
    const size_t state = ((size_t)u.seq * a.HV + hv) * DK * DV + (size_t)(warp * RW + sub) * DV + col;
    constexpr int kHop = kStepWarps * RW * DV;
    float4 S[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        S[i] = a.h0 ? ldg_stream4(a.h0 + state + i * kHop) : make_float4(0.f, 0.f, 0.f, 0.f);
    float keep = 1.f, step = 0.f;
    float4 xs = make_float4(0.f, 0.f, 0.f, 0.f);
    if (u.len > 0) {
        const T *x = static_cast<const T *>(a.x) + u.row0 * a.ldx + (size_t)hv * DV + col;
        const float x0 = to_f32(x[0]), x1 = to_f32(x[1]), x2 = to_f32(x[2]), x3 = to_f32(x[3]);
        const float raw = a.dt[u.row0 * a.HV + hv];
        if (tid < DK)
            sb[tid] = to_f32(static_cast<const T *>(a.b)[u.row0 * a.ldb + (size_t)hk * DK + tid]);
        else if (tid < 2 * DK)
            sc[tid - DK] = to_f32(static_cast<const T *>(a.c)[u.row0 * a.ldc + (size_t)hk * DK + tid - DK]);
        step = ssm_step(raw, a.dt_bias ? a.dt_bias[hv] : 0.f, a.softplus);
        keep = expf(step * a.A[hv]);
        xs = make_float4(step * x0, step * x1, step * x2, step * x3);
    } else if (tid < DK) {
        sb[tid] = sc[tid] = 0.f;
    }
    __syncthreads();
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = (i * kStepWarps + warp) * RW + sub;
        const float b = sb[r], c = sc[r];
        S[i].x = fmaf(keep, S[i].x, b * xs.x);
        S[i].y = fmaf(keep, S[i].y, b * xs.y);
        S[i].z = fmaf(keep, S[i].z, b * xs.z);
        S[i].w = fmaf(keep, S[i].w, b * xs.w);
        y.x = fmaf(c, S[i].x, y.x);
        y.y = fmaf(c, S[i].y, y.y);
        y.z = fmaf(c, S[i].z, y.z);
        y.w = fmaf(c, S[i].w, y.w);
        if (a.ht) stg_stream4(a.ht + state + i * kHop, S[i]);
    }
    if (u.len == 0) return;
#pragma unroll
    for (int off = L; off < 32; off <<= 1) {
        y.x += __shfl_xor_sync(0xffffffffu, y.x, off);
        y.y += __shfl_xor_sync(0xffffffffu, y.y, off);
        y.z += __shfl_xor_sync(0xffffffffu, y.z, off);
        y.w += __shfl_xor_sync(0xffffffffu, y.w, off);
    }
    if (sub == 0) *reinterpret_cast<float4 *>(&part[warp][col]) = y;
    __syncthreads();
    if (tid < DV) {
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w) o += part[w][tid];
        const size_t at = (size_t)hv * DV + tid;
        if (a.D) o = fmaf(a.D[hv], to_f32(static_cast<const T *>(a.x)[u.row0 * a.ldx + at]), o);
        if (a.z) o = ssm_gate(o, to_f32(static_cast<const T *>(a.z)[u.row0 * a.ldz + at]));
        static_cast<T *>(a.out)[u.row0 * a.HV * DV + at] = from_f32<T>(o);
    }
}

template <typename T, int DK, int DV>
cudaError_t launch_step(const SsmArgs &a, cudaStream_t stream) {
    return for_sequences(a.cu, a.N, a.T, INT_MAX, [&](const SeqTable &t, long long units) {
        trace_begin(kKernSsm, stream);
        gdr_ssm_step_kernel<T, DK, DV><<<(unsigned)(units * a.HV), 32 * kStepWarps, 0, stream>>>(a, t);
        trace_end(kKernSsm, stream);
        return cudaGetLastError();
    });
}
template <typename T, int DK>
cudaError_t step_by_dv(const SsmArgs &a, cudaStream_t s) {
    return a.dv == 32 ? launch_step<T, DK, 32>(a, s)
                      : a.dv == 64 ? launch_step<T, DK, 64>(a, s) : launch_step<T, DK, 128>(a, s);
}
template <typename T>
cudaError_t step_by_dk(const SsmArgs &a, cudaStream_t s) {
    return a.dk == 32 ? step_by_dv<T, 32>(a, s)
                      : a.dk == 64 ? step_by_dv<T, 64>(a, s) : step_by_dv<T, 128>(a, s);
}

template <typename T, int DK, int PASS, int COLS>
cudaError_t launch_cols(const SsmArgs &a, cudaStream_t stream) {
    return for_sequences(a.cu, a.N, a.T, a.seg_rows, [&](const SeqTable &t, long long units) {
        const long long ctas = units * a.HV * (a.dv / (32 * COLS));
        if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
        trace_begin(kKernSsm, stream);
        gdr_ssm_walk_kernel<T, DK, PASS, COLS><<<(unsigned)ctas, kThreads, 0, stream>>>(a, t);
        trace_end(kKernSsm, stream);
        return cudaGetLastError();
    });
}
// Two columns a lane read each row of b and c half as often: f32, 4 x 1024
// tokens of 32 gated heads of 128 x 128, 394 us against 485.  Below a CTA for each of
// kWideSms SMs the narrow ones are twice as many and no slower each.
template <typename T, int DK, int PASS>
cudaError_t launch_walk(const SsmArgs &a, cudaStream_t stream) {
    const long long wide = count_units(a.cu, a.N, a.T, a.seg_rows) * a.HV * (a.dv / 64);
    return a.dv % 64 == 0 && wide >= kWideSms ? launch_cols<T, DK, PASS, 2>(a, stream)
                                              : launch_cols<T, DK, PASS, 1>(a, stream);
}
template <typename T, int DK>
cudaError_t by_pass(const SsmArgs &a, int pass, cudaStream_t s) {
    return pass == 0 ? launch_walk<T, DK, 0>(a, s)
                     : pass == 1 ? launch_walk<T, DK, 1>(a, s) : launch_walk<T, DK, 2>(a, s);
}
template <typename T>
cudaError_t by_dk(const SsmArgs &a, int pass, cudaStream_t s) {
    return a.dk == 32 ? by_pass<T, 32>(a, pass, s)
                      : a.dk == 64 ? by_pass<T, 64>(a, pass, s) : by_pass<T, 128>(a, pass, s);
}

struct Plan {
    int longest;       // rows of the longest sequence
    int seg_rows;      // INT_MAX: walks are not cut
    long long units;   // units of the batch
    size_t bytes;      // workspace
    size_t off_log, off_h0;
};

// SMs of the current device; 0 without one.
int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return sms;
}

// Rows of a segment: few heads leave SMs idle while a long sequence is walked,
// so walks are cut where that is estimated to be faster.  Costs are in rows of
// a full walk; a walk to the end state alone, the second launch and the start
// from the segments before were measured.  An SM takes `full` CTAs of 32 columns
// before they slow one another down: of the chunk kernel one, of the walk as many
// as have 256 rows of states.  One sequence of 32 gated heads of 128 x 128, bf16, us a
// call whole / cut: 1024 tokens 50 / 40 (by three), 4096 174 / 83 (by four, the
// best of up to twelve), 16384 663 / 257 (by four; 254 by nine); two of 4096 174 / 136
// (by two, the best).  f32, us on the device: 4096 tokens 670 / 537 (by eight; 520 by
// 24); two of 2048 485 / 490 (by eight), not cut; 9 heads of 64 x 32, 4096
// tokens 502 / 45.
int choose_segment(const int *cu, int N, int T, int HV, int dk, int dv, int longest, bool chunks) {
    const int sms = sm_count(), grain = chunks ? 64 : 16, full = chunks ? 1 : 256 / dk;
    const long long per = (long long)HV * (chunks ? 1 : dv / 32);
    if (sms == 0 || longest < 4 * grain || N * per >= (long long)sms * full) return INT_MAX;
    const double state_only = 0.5, launch = chunks ? 256 : 32, start = chunks ? 24 : 4;
    auto slower = [&](long long ctas) {
        const double on_an_sm = (double)((ctas + sms - 1) / sms);
        return on_an_sm > full ? on_an_sm / full : 1.0;
    };
    double best = 0.9 * longest;  // cut for a tenth at least
    int rows = INT_MAX, r = longest;
    for (int cut = 2; cut <= 64 && r > grain; ++cut) {
        const int last = r;
        r = ((longest + cut - 1) / cut + grain - 1) / grain * grain;
        if (r >= longest || r == last) continue;
        const long long units = count_units(cu, N, T, r), after = units - N;
        const double cost = (slower(units * per) + state_only * slower(after * per)) * r + launch +
                            start * (longest / r);
        if (cost < best) {
            best = cost;
            rows = r;
        }
    }
    return rows;
}

Plan make_plan(const int *cu, int N, int T, int HV, int dk, int dv, int dtype, unsigned flags) {
    Plan p = {cu ? 0 : T, INT_MAX, N, 0, 0, 0};
    const int forced = (int)((flags >> 8) & 0xffu);
    int &longest = p.longest;
    for (int n = 0; cu && n < N; ++n) longest = longest > cu[n + 1] - cu[n] ? longest : cu[n + 1] - cu[n];
    if (!(flags & GDR_FLAG_NO_SEGMENTS) && longest > 64) {
        if (forced >= 2) {
            const int rows = ((longest + forced - 1) / forced + 63) / 64 * 64;
            if (rows < longest) p.seg_rows = rows;
        } else if (forced == 0) {
            p.seg_rows = choose_segment(cu, N, T, HV, dk, dv, longest,
                                        dtype == GDR_BF16 && !(flags & GDR_FLAG_FORCE_GENERIC));
        }
    }
    if (p.seg_rows != INT_MAX) {
        p.units = count_units(cu, N, T, p.seg_rows);
        const size_t state = (size_t)HV * dk * dv * 4;
        p.off_log = p.units * state;
        p.off_h0 = (p.off_log + (size_t)p.units * HV * 4 + 255) / 256 * 256;
        p.bytes = p.off_h0 + (size_t)N * state;
    }
    return p;
}

// Whether bf16 sequences are so short that walking them token by token is
// faster than chunks, by what both cost (microseconds): a CTA of the chunk
// kernel 9 for itself and 1.5 a chunk, one an SM; the walk its operations at 20
// TFLOP/s and its states at memory's rate.  64 sequences of 32 heads of 128 x
// 128: chunks 146 (2 to 16 tokens), walk 97 (2), 113 (4), 142 (8), 174 (16); of
// 64 x 64, 16 tokens: chunks 90, walk 40.
bool walk_is_faster(const SsmArgs &a, const Plan &plan) {
    const int sms = sm_count();
    if (sms == 0) return false;
    const double rows = a.cu ? a.cu[a.N] : (double)a.N * a.T, state = (double)a.dk * a.dv;
    const double waves = (double)((plan.units * a.HV + sms - 1) / sms);
    const double chunks = waves * (9.0 + 1.5 * (rows / 64 / plan.units < 1 ? 1 : rows / 64 / plan.units));
    const double walk = rows * a.HV * 5 * state / 20e6 + a.N * a.HV * state * 8 / 6e6 + 0.2 * plan.longest;
    return walk < chunks;
}

gdr_status check_shape(const int *cu, int N, int T, int HK, int HV, int dk, int dv, int dtype,
                       unsigned flags) {
    if (N < 0 || (!cu && T < 0) || HK <= 0 || HV <= 0 || HV % HK) return GDR_ERR_SHAPE;
    if (!supported_dim(dk) || !supported_dim(dv) || (dtype != GDR_F32 && dtype != GDR_BF16) ||
        (flags & ~(GDR_FLAG_DT_SOFTPLUS | GDR_FLAG_FORCE_GENERIC | GDR_FLAG_NO_SEGMENTS | 0xff00u)))
        return GDR_ERR_UNSUPPORTED;
    if (N > 0 && cu && check_offsets(cu, N) != GDR_OK) return GDR_ERR_SHAPE;
    // heads of the states, CTAs of a launch and element offsets
    if ((long long)N * HV > (1LL << 28) || (long long)HV * dv > 0x7fffffffLL ||
        (long long)HK * dk > 0x7fffffffLL)
        return GDR_ERR_SHAPE;
    return GDR_OK;
}

}  // namespace

cudaError_t launch_ssm_walk(const SsmArgs &a, int pass, cudaStream_t stream) {
    return a.bf16 ? by_dk<__nv_bfloat16>(a, pass, stream) : by_dk<float>(a, pass, stream);
}

}  // namespace gdr

extern "C" GDR_API size_t gdr_ssm_workspace_bytes(const int *cu_seqlens, int N, int T, int HK,
                                                  int HV, int dk, int dv, int dtype,
                                                  unsigned flags) {
    using namespace gdr;
    if (check_shape(cu_seqlens, N, T, HK, HV, dk, dv, dtype, flags) != GDR_OK || N == 0) return 0;
    return make_plan(cu_seqlens, N, T, HV, dk, dv, dtype, flags).bytes;
}

extern "C" GDR_API gdr_status gdr_ssm_forward(
    const void *x, const void *b, const void *c, const float *dt, const float *A, const float *D,
    const void *z, const float *dt_bias, const float *h0, void *out, float *ht,
    const int *cu_seqlens, int N, int T, int HK, int HV, int dk, int dv, long long ldx,
    long long ldb, long long ldc, long long ldz, void *stream, int dtype, void *workspace,
    size_t workspace_bytes, unsigned flags) {
    using namespace gdr;
    gdr_status st = check_shape(cu_seqlens, N, T, HK, HV, dk, dv, dtype, flags);
    if (st != GDR_OK) return st;
    const long long wx = (long long)HV * dv, wb = (long long)HK * dk;
    const long long total = N == 0 ? 0 : cu_seqlens ? cu_seqlens[N] : (long long)N * T;
    if (ldx < wx || ldb < wb || ldc < wb || (z && ldz < wx) || !rows_fit(total, ldx) ||
        !rows_fit(total, ldb) || !rows_fit(total, ldc) || (z && !rows_fit(total, ldz)))
        return GDR_ERR_SHAPE;
    if (N == 0) return GDR_OK;
    if (!A || (total > 0 && (!x || !b || !c || !dt || !out))) return GDR_ERR_NULL;
    if (total == 0 && !ht) return GDR_OK;
    const size_t es = dtype == GDR_BF16 ? 2 : 4;
    const uintptr_t any = (uintptr_t)x | (uintptr_t)b | (uintptr_t)c | (uintptr_t)z;
    if ((any & (es - 1)) || !aligned4(dt) || !aligned4(A) || !aligned4(D) || !aligned4(dt_bias) ||
        !aligned16(out) || !aligned16(h0) || !aligned16(ht))
        return GDR_ERR_ALIGN;
    const size_t state = (size_t)HV * dk * dv * 4;
    const RowSet o = packed_rows(out, total * wx * es), e = packed_rows(ht, N * state);
    const RowSet in[] = {{x, wx * es, ldx * es, total}, {b, wb * es, ldb * es, total},
                         {c, wb * es, ldc * es, total}, {z, wx * es, ldz * es, total},
                         packed_rows(dt, total * HV * 4), packed_rows(A, (size_t)HV * 4),
                         packed_rows(D, (size_t)HV * 4), packed_rows(dt_bias, (size_t)HV * 4)};
    const RowSet h = packed_rows(h0, N * state);
    for (const RowSet &r : in)
        if (rows_overlap(o, r) || rows_overlap(e, r)) return GDR_ERR_ALIAS;
    if (rows_overlap(o, h) || rows_overlap(o, e) || (h0 != ht && rows_overlap(e, h)))
        return GDR_ERR_ALIAS;
    const Plan plan = make_plan(cu_seqlens, N, T, HV, dk, dv, dtype, flags);
    if (plan.bytes) {
        if (!workspace || workspace_bytes < plan.bytes) return GDR_ERR_WORKSPACE;
        if ((uintptr_t)workspace & 255u) return GDR_ERR_ALIGN;
    }
    if (plan.units * HV * (dv / 32) > 0x7fffffffLL) return GDR_ERR_SHAPE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    SsmArgs a = {x, b, c, z, dt, A, D, dt_bias, h0, out, ht, nullptr, nullptr, ldx, ldb, ldc, ldz,
                 N, T, HK, HV, dk, dv, cu_seqlens, plan.seg_rows,
                 (flags & GDR_FLAG_DT_SOFTPLUS) ? 1 : 0, dtype == GDR_BF16 ? 1 : 0, 0};
    const bool chunks = !(flags & GDR_FLAG_FORCE_GENERIC) && ssm_chunks_supported(a) &&
                        (plan.bytes || !walk_is_faster(a, plan));
    const auto walk = chunks ? launch_ssm_chunks : launch_ssm_walk;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (plan.bytes) {
        a.seg_state = reinterpret_cast<float *>(ws);
        a.seg_log = reinterpret_cast<float *>(ws + plan.off_log);
        if (h0 && h0 == ht) {
            // a sequence's last unit may write ht before its first one has read h0
            float *copy = reinterpret_cast<float *>(ws + plan.off_h0);
            err = cudaMemcpyAsync(copy, h0, N * state, cudaMemcpyDeviceToDevice, s);
            a.h0 = copy;
        }
        if (err == cudaSuccess) err = walk(a, 1, s);
        if (err == cudaSuccess) err = walk(a, 2, s);
    } else if (plan.longest <= 1 && !(flags & GDR_FLAG_FORCE_GENERIC)) {
        err = dtype == GDR_BF16 ? step_by_dk<__nv_bfloat16>(a, s) : step_by_dk<float>(a, s);
    } else {
        err = walk(a, 0, s);
    }
    if (err == cudaSuccess) return GDR_OK;
    record_cuda_error(err);
    return GDR_ERR_CUDA;
}
