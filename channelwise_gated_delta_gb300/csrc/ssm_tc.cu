// ssm_tc.cu -- gdr_ssm_forward's walk on the tensor cores: bf16 x, b and c,
// by chunks of 64 tokens, one warp-specialised CTA per (unit of a sequence,
// value head), the state in registers.
//
// With cum the prefix sums of step A within a chunk (kept in log2 units), S
// the state at its start, r a reference near half of the chunk's decay, all
// per value head:
//     M[t][s] = (c_t . b_s) exp(r - cum_s) step_s   (s <= t),  M[t][t] += D exp(r - cum_t)
//     out^T   = (x^T M^T + (exp(r) S)^T c^T) exp(cum_t - r)
//     S^T    <- exp(cum_end) S^T + (w x)^T b,   w_s = exp(cum_end - cum_s) step_s
// so that both parts of an output meet in one accumulator, and M needs no
// exponential of its own.  That holds while no |cum - r| is above 80 (log2
// units; a decay of more than 1.7 nats a token).  In a chunk beyond that M
// takes every pair's own decay, the part from the state is formed first and
// rescaled in tensor memory, and the rest is added to it.
// A chunk within it holds its outputs times up to 2^80 and the state times down to
// 2^-80, so values from 2^47 on may overflow there and states below 2^-46 be lost;
// with a limit of 40 in place of 80 those were 2^87 and 2^-86, but every chunk of 0.9
// nats a token would go the slow way (4 x 16384 tokens of 32 heads: 629 us for 402).
//
// Everything is transposed so that dv fills the 128 rows of an MMA.  Four
// products a chunk:
//     G  = c b^T            both tiles as TMA brought them (128-byte swizzle)
//     Y  = S^T c^T          S^T as bf16 in tensor memory
//     Y += x^T M^T          x as it came (M-major A), M from the score warps
//     dS = (w x)^T b        (w x)^T in tensor memory, b as it came
// x, b and c are exact.  w x goes in as three bf16 numbers (see weigh3), off by
// 8e-7 of it: the state, which is float32 in registers and never rounded itself,
// keeps float32's accuracy but for that.  (A pair is off by 4e-6, and took 406 us
// where three take 400: the products are not what the kernel waits for.)  M goes
// in as a pair hi + lo, off by 2^-16.  The copy of S that Y reads is rounded
// once to bf16: its error is averaged over dk products and adds 1 to 27 % to
// what the output's own rounding leaves (M rounded the same way would add 26
// to 48 %).  A second number for it, in the place of one of Y's buffers, took 553 us
// for 395.
//
// The walk's only serial part is S <- g S + dS in the chain warps: dS does not
// depend on S.  Tensor memory, full: G 64 columns, Y 2 x 64, S 64, dS 128, w x
// 96.  So w x has one buffer, in two halves of 32 tokens that are written as
// soon as the last chunk's products have read them.
//     0-7    chain: lane = value column, 64 of the dk columns each; S in
//            registers, its bf16 copy into tensor memory
//     8-15   (w x)^T of 32 columns and 32 tokens into tensor memory
//     16-19  outputs: Y exp(cum - r), times silu(z)
//     20, 21, 24, 25  scores: rows of G to rows of M (G's 64 rows are TMEM lanes
//            0-63, which only warps 4 n and 4 n + 1 can read)
//     22     the chunk's scalars (steps, prefix sums, decays), two tokens a lane
//     27     TMA of x, b and c, up to three chunks ahead
//     23, 26 issue the MMAs (one thread each): G and dS; Y.  An MMA takes its
//            thread as long as the tensor cores (32 to 64 cycles each, some eight
//            ahead), and a thread that waits for one product's inputs feeds no other
// The chain's registers (112 a thread) come from the others (56).
//
// What bounds it: 4 x 16384 tokens of 32 heads of 128 take 395 us, 3000 cycles a
// chunk (629 where every chunk of a head is beyond r's range).  Its products take 1790 of them, its bytes 1820 (at 6.8 TB/s).
// The rest is one chunk's way around: products of dS 770, its read 200, S 600 to
// 900, the next products' start 200, with the other products in between.  With
// all arithmetic of the warps taken out it takes 380.
// Every wait is bounded (one second, of which a role may make three before it
// looks): a timeout sets the CTA's abort flag and the library's error word, and
// everyone runs out its loop.  Few instructions a wait: the warps run eight
// different programs out of one instruction cache.
#include <cuda.h>
#include <limits.h>

#include <type_traits>

#include "gdr.h"
#include "sm100_ptx.cuh"
#include "ssm.cuh"
#include "tma_host.h"

namespace gdr {
namespace {

using namespace sm100;

constexpr int kC = 64;
constexpr int kWarps = 28;
constexpr int kThreads = 32 * kWarps;
constexpr int kWx0 = 8, kOut0 = 16, kScore0 = 20, kScalars = 22, kIssueState = 23, kIssueY = 26,
              kLoads = 27;
// registers: 72 a thread at launch, of which the chain's two warpgroups take 112
// and the others keep 56
constexpr int kRegsLaunch = 72, kRegsChain = 112, kRegsOther = 56;
static_assert(2 * kRegsChain + 5 * kRegsOther == 7 * kRegsLaunch && kThreads * kRegsLaunch <= 65536, "registers");
constexpr int kStages = 3;
constexpr int kRing = 8;  // chunks whose scalars are held
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;

// shared memory, from a 1024-byte aligned base
constexpr uint32_t kTile = 16384;  // 64 rows of up to 128, two boxes of 64 columns
constexpr uint32_t kX = 0, kB = kTile, kCm = 2 * kTile, kStage = 3 * kTile;
constexpr uint32_t kM = kStages * kStage;           // [2] x {hi, lo} [64 t][64 s]
constexpr uint32_t kScal = kM + 2 * 16384;          // [kRing] of the following
// of a chunk, 64 numbers each: exp(cum - r), exp(r - cum) step, D exp(r - cum);
// in a chunk beyond r's range kCum the sums up to a token from its 16 tokens'
// first, and the steps; of every two tokens w's three parts and a gap; then
// exp(cum_end), exp(r) and whether the chunk is beyond r's range
constexpr uint32_t kE = 0, kV = 256, kDiag = 512, kCum = 768, kStep = 1024, kW = 1280, kEnd = 1792;
constexpr uint32_t kScalBytes = 1808;
constexpr float kRange = 80.f;
constexpr uint32_t kOut = (kScal + kRing * kScalBytes + 1023) / 1024 * 1024;  // [2][4 warps] [64 t][32]
                                                                              // z, then outputs
constexpr uint32_t kBad = kOut + 2 * 16384;  // [kRing][2][128] a column's first token, of either half's,
                                             // that is not finite
constexpr uint32_t kBadAt = kBad + kRing * 256;  // [kRing][4 x 32 columns][2] whether there is any
constexpr uint32_t kBars = kBadAt + kRing * 8;
enum {
    FULL = 0,               // [3] x, b, c of a chunk in, and its scalars
    EMPTY = FULL + kStages,  // [3] its last product done
    FIX = EMPTY + kStages,   // rows behind the sequence's end zeroed
    GRAM,                    // G done
    GFREE,                   // G read
    MFULL,                   // [2] M written, x looked through
    MFREE = MFULL + 2,       // [2] M read
    WX = MFREE + 2,          // [2 x 32 tokens] (w x)^T written
    WFREE = WX + 2,          // [2] (w x)^T read
    DELTA = WFREE + 2,       // dS done
    DFREE,                   // dS read
    SFULL,                   // S copied
    SFREE,                   // that copy read
    YDONE,                   // [2] Y done
    YFREE = YDONE + 2,       // [2] Y read
    YSCALED = YFREE + 2,     // in a chunk beyond r's range YDONE is the part from the state;
    YPART,                   // that is rescaled, and the rest added to it
    LAST,                    // [2] all done
    ZFULL = LAST + 2,        // [2][4 warps] z in
    kNumBars = ZFULL + 8
};
constexpr uint32_t kSlot = kBars + 8 * kNumBars;
constexpr uint32_t kAbort = kSlot + 4;
constexpr uint32_t kSmem = kAbort + 4 + 1024;
static_assert(kSmem <= 232448 && kOut % 16 == 0 && kBars % 8 == 0, "shared memory");

// tensor memory columns
constexpr uint32_t kTmG = 0, kTmY = 64, kTmS = 192, kTmD = 256, kTmW = 384, kTmCols = 512;

struct Maps {
    CUtensorMap x, b, c, z, out;
};

__device__ __forceinline__ void tma_load_2d(void *dst, const void *map, int c0, int c1,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_store_2d(const void *map, const void *src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(smem_u32(src))
                 : "memory");
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}
// (a, b) as hi + lo, two bf16 numbers each
__device__ __forceinline__ void pair2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack2(a, b);
    const float2 r = fma2(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)),
                          make_float2(-1.f, -1.f), make_float2(a, b));
    lo = pack2(r.x, r.y);
}
// A float32 weight as w0 + w1 + w2: the nearest power of two, and what is left
// of it as two bf16 numbers.
__device__ __forceinline__ void split_weight(float w, float &w0, float &w1, float &w2) {
    w0 = __uint_as_float((__float_as_uint(w) + 0x400000u) & 0xff800000u);
    const float d = w - w0;
    w1 = __bfloat162float(__float2bfloat16_rn(d));
    w2 = d - w1;
}
// x w of two bf16 numbers x and their weights as the sum of three bf16 numbers:
// x w0, which is exact, x w1 rounded, and x w2 with what that rounding left
// (eight bits, so exact).  The last one's own rounding stays: w0 leaves a
// third of w at the most, which makes that 8e-7 of x w (rms over weights of any
// size), where a pair of bf16 numbers leaves 4e-6 of it and three parts of the
// float32 product, exact, take eleven instructions in place of four.
__device__ __forceinline__ void weigh3(uint32_t x, uint4 w, uint32_t &q0, uint32_t &q1, uint32_t &q2) {
    asm("{\n\t.reg .b32 n, r;\n\t"
        "mul.rn.bf16x2 %0, %3, %4;\n\t"
        "mul.rn.bf16x2 %1, %3, %5;\n\t"
        "neg.bf16x2 n, %1;\n\t"
        "fma.rn.bf16x2 r, %3, %5, n;\n\t"
        "fma.rn.bf16x2 %2, %3, %6, r;\n\t}"
        : "=&r"(q0), "=&r"(q1), "=r"(q2)
        : "r"(x), "r"(w.x), "r"(w.y), "r"(w.z));
}

// Four 8 x 8 matrices of 16-bit numbers between shared memory and registers,
// transposed: a lane's address is that of row lane % 8 of matrix lane / 8, and
// register i holds rows 2 (lane % 4) and + 1 of column lane / 4 of matrix i.
__device__ __forceinline__ void ldsm4_t(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void stsm4_t(uint32_t at, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
// Tensor memory in the same arrangement, 16 lanes at a time: 32 columns of
// float32 (registers 4 j + {0, 1}: lane / 4 of the 16, columns 8 j + 2 (lane %
// 4) + {0, 1}; + 2: eight lanes on), and 16 columns of pairs (register 2 j:
// lane / 4, column 4 j + lane % 4; + 1: eight lanes on).
__device__ __forceinline__ void tmem_ld_16x256(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}
// what such a load has brought, once it is there
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                   "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st_16x128(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}
// waits until all but the latest of the thread's bulk stores have read shared memory
__device__ __forceinline__ void bulk_wait_read_but_one() {
    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
// `steps` products of 16 along K, the operands' descriptors (of which only the
// address, in the low half, moves) in steps of their own; one of A's is
// tensor memory where TS.  A step that ends a box of 64 columns moves by
// `jump` more.
template <bool TS>
__device__ __forceinline__ void products(uint32_t d, uint64_t a, int a_step, int a_jump, uint64_t b,
                                         int b_step, int b_jump, uint32_t idesc, int steps,
                                         uint32_t accumulate) {
    uint32_t al = (uint32_t)a, bl = (uint32_t)b;
    const uint64_t ah = a & 0xffffffff00000000ull, bh = b & 0xffffffff00000000ull;
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
        if (TS)
            mma_bf16_ts(d, al, bh | bl, idesc, accumulate);
        else
            mma_bf16(d, ah | al, bh | bl, idesc, accumulate);
        accumulate = 1;
        al += (uint32_t)(a_step + (k == 3 ? a_jump : 0));
        bl += (uint32_t)(b_step + (k == 3 ? b_jump : 0));
    }
}
// one lane of a converged warp, the same each time
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}
// 0 times a value that is not finite is no 0: such values of a column of x are
// taken out of the tile that Y1 reads (of its rows r0 to r0 + 31), so that they
// do not reach the outputs of the tokens before them, and the first one's place
// is kept for the outputs.
__device__ __noinline__ void mask_odd(unsigned char *smem, int stage, int r0, unsigned char *bad, int p) {
    unsigned char *x = smem + stage * kStage + kX + (p >> 6) * 8192 + (p & 7) * 2;
    int first = kC;
    for (int r = r0 + 31; r >= r0; --r) {
        uint16_t *v = reinterpret_cast<uint16_t *>(x + r * 128 + ((((p & 63) >> 3) ^ (r & 7)) << 4));
        if ((*v & 0x7f80u) == 0x7f80u) {
            first = r;
            *v = 0;
        }
    }
    bad[p] = (unsigned char)first;
    fence_async_smem();
}
// Such outputs of a column from there on, in the tile that leaves.
__device__ __noinline__ void spoil(unsigned char *tile, const unsigned char *any, const unsigned char *bad,
                                   int lane) {
    int from = any[0] ? bad[0] : kC;
    if (from == kC && any[1]) from = bad[128];
    for (int r = from; r < kC; ++r)
        *reinterpret_cast<uint16_t *>(tile + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) +
                                      (lane & 7) * 2) = 0x7fff;
}

template <int DK, int PASS>
__global__ void __launch_bounds__(kThreads, 1)
    gdr_ssm_chunk_kernel(const __grid_constant__ SsmArgs a, const __grid_constant__ SeqTable table,
                         const __grid_constant__ Maps maps, int *err) {
    constexpr bool OUT = PASS != 1;
    constexpr int kChain = DK > 64 ? 8 : 4;  // warps
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kBars);
    uint32_t *slot = reinterpret_cast<uint32_t *>(smem + kSlot);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kAbort);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int hv = blockIdx.x % a.HV, hk = hv / (a.HV / a.HK);
    const SeqUnit u = find_unit(table, blockIdx.x / a.HV);
    const int unit = table.unit0 + blockIdx.x / a.HV;
    const long long first = (long long)u.unit * a.seg_rows;
    const int T = (int)min((long long)u.len - first, (long long)a.seg_rows);
    const bool last = first + T == u.len;
    if (PASS == 1 && last) return;  // no unit follows
    const long long row0 = u.row0 + first;
    const int NC = (T + kC - 1) / kC;
    const int dv = a.dv;
    const size_t per = (size_t)DK * dv;

    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            const int n = i >= WX && i < WX + 2 || i == GFREE || i == YFREE || i == YFREE + 1 || i == YSCALED ? 128
                          : i == MFULL || i == MFULL + 1              ? 256 + 128
                          : i == DFREE || i == SFULL                  ? 32 * kChain
                          : i < EMPTY || (i < EMPTY + kStages && OUT) ? 2
                                                                      : 1;
            mbar_init(&bars[i], n);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(slot, kTmCols);
    // the blocks of M above the diagonal (rows below 32, columns from 32 on) stay zero
#pragma unroll 1
    for (int i = tid; i < 4 * 32 * 4; i += kThreads)
        *reinterpret_cast<uint4 *>(smem + kM + (i >> 7) * 8192 +
                                   kmajor_off((i >> 2) & 31, 32 + 8 * (i & 3), kC)) =
            make_uint4(0, 0, 0, 0);
    fence_async_smem();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *slot;
    const uint32_t bar0 = smem_u32(bars), abort0 = smem_u32(smem + kAbort);
    // one second at most; every warp looks at the abort flag once a chunk
    auto wait = [&](int id, uint32_t parity) { mbar_wait_cycles(bar0 + 8 * id, parity & 1, abort0); };
    // Two or three at once, a lane each: a wait whose phase has long ended still
    // takes some 180 cycles of this busy kernel.  (The phase before a barrier's
    // first counts as ended.)
    auto wait2 = [&](int i0, uint32_t p0, int i1, uint32_t p1) {
        wait(lane & 1 ? i1 : i0, lane & 1 ? p1 : p0);
        __syncwarp();
    };
    auto wait3 = [&](int i0, uint32_t p0, int i1, uint32_t p1, int i2, uint32_t p2) {
        wait2(lane & 2 ? i2 : i0, lane & 2 ? p2 : p0, i1, p1);
    };
    auto scal = [&](int c, uint32_t what) {
        return reinterpret_cast<float *>(smem + kScal + (c & (kRing - 1)) * kScalBytes + what);
    };
    auto rows_in = [&](int c) { return min(kC, T - c * kC); };
    // a chunk's stage and the parity of that stage's barriers
    struct Stage {
        int st = 0;
        uint32_t ph = 0;
        __device__ __forceinline__ void next() {
            if (++st == kStages) {
                st = 0;
                ph ^= 1;
            }
        }
    };
    Stage at;

    if (warp < kWx0)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsChain));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp < kChain) {
        // ================= chain
        constexpr int NH = 4 * DK / kChain;
        const int p = 32 * (warp & 3) + lane, n0 = NH * (warp >> 2);
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const bool on = 32 * (warp & 3) < dv;  // dv is a multiple of 32
        float dec = 0.f, ref = 0.f;
        if (NC > 0) {
            wait(FULL, 0);
            dec = scal(0, kEnd)[0];
            ref = scal(0, kEnd)[1];
        }
        at.next();
        mbar_arrive(&bars[DFREE]);
        float S[NH];
#pragma unroll
        for (int i = 0; i < NH; ++i) S[i] = 0.f;
        if (on && a.h0 && u.unit == 0) {
            const float *h = a.h0 + ((size_t)u.seq * a.HV + hv) * per + n0 * dv + p;
#pragma unroll
            for (int i = 0; i < NH; ++i, h += dv) S[i] = *h;
        }
        if (PASS == 2 && on)
#pragma unroll 1
            for (int k = 0; k < u.unit; ++k) {
                const size_t s = (size_t)(unit - u.unit + k) * a.HV + hv;
                const float keep = expf(a.seg_log[s]);
                const float *e = a.seg_state + s * per + n0 * dv + p;
#pragma unroll
                for (int i = 0; i < NH; ++i, e += dv) S[i] = fmaf(keep, S[i], *e);
            }
        for (int c = 0; c < NC && !*abort_flag; ++c, at.next()) {
            if (OUT) {
                wait(SFREE, c - 1);
                if (on) {
#pragma unroll
                    for (int g = 0; g < NH / 16; ++g) {
                        uint32_t h[8];
#pragma unroll
                        for (int m = 0; m < 8; ++m) {
                            const float2 q = mul2(make_float2(ref, ref),
                                                  make_float2(S[16 * g + 2 * m], S[16 * g + 2 * m + 1]));
                            h[m] = pack2(q.x, q.y);
                        }
                        tmem_st8(tl + kTmS + n0 / 2 + 8 * g, h);
                    }
                    tmem_st_wait();
                }
                tc_fence_before_sync();
                mbar_arrive(&bars[SFULL]);
            }
            const float now = dec;
            if (c + 1 < NC) wait(FULL + at.st, at.ph);
            if (c + 1 < NC) {
                dec = scal(c + 1, kEnd)[0];
                ref = scal(c + 1, kEnd)[1];
            }
            wait(DELTA, c);
            tc_fence_after_sync();
            if (on) {
                constexpr int W = 16;
#pragma unroll
                for (int g = 0; g < NH / W; ++g) {
                    float d[W];
                    tmem_ld16(tl + kTmD + n0 + W * g, d);
                    if (g == NH / W - 1) {  // dS is free before the last of it is added
                        tc_fence_before_sync();
                        mbar_arrive(&bars[DFREE]);
                    }
#pragma unroll
                    for (int m = 0; m < W; m += 2) {
                        const float2 q = fma2(make_float2(now, now),
                                              make_float2(S[W * g + m], S[W * g + m + 1]),
                                              make_float2(d[m], d[m + 1]));
                        S[W * g + m] = q.x;
                        S[W * g + m + 1] = q.y;
                    }
                }
            }
            if (!on) mbar_arrive(&bars[DFREE]);
        }
        float *end = PASS == 1 ? a.seg_state + ((size_t)unit * a.HV + hv) * per
                     : a.ht && last ? a.ht + ((size_t)u.seq * a.HV + hv) * per
                                    : nullptr;
        if (on && end && !*abort_flag) {
            end += n0 * dv + p;
#pragma unroll
            for (int i = 0; i < NH; ++i, end += dv) *end = S[i];
        }
    } else if (warp < kWx0) {
        // no columns for these
    } else if (warp < kOut0) {
        // ================= (w x)^T: value columns over the lanes, two tokens a column
        const int wq = warp & 3, half = (warp >> 2) & 1, p0 = 32 * wq, t0 = 32 * half;
        const uint32_t tw = tmem + ((uint32_t)p0 << 16) + kTmW + 48 * half;
        const bool on = p0 < dv;
        // this lane's row of the 8 x 8 blocks (tokens 8 j + row, columns p0 + 8 i ..):
        // matrices 0 and 1 of a load are adjacent columns, 2 and 3 the next tokens
        const int row = lane & 7;
        const uint32_t x0 = smem_u32(smem) + kX + (p0 >> 6) * 8192 + (t0 + (lane >> 4) * 8 + row) * 128;
        const int unit = ((p0 & 63) >> 3) + ((lane >> 3) & 1);
        for (int c = 0; c < NC && !*abort_flag; ++c, at.next()) {
            const int st = at.st;
            if (OUT)  // the last for the arrival below
                wait3(FULL + st, at.ph, WFREE + half, c - 1, MFREE + (c & 1), (c >> 1) - 1);
            else
                wait2(FULL + st, at.ph, WFREE + half, c - 1);
            if (rows_in(c) < kC) wait(FIX, 0);
            tc_fence_after_sync();
            bool any = false;
            if (on) {
                const uint4 *w = reinterpret_cast<const uint4 *>(scal(c, kW)) + 16 * half + (lane & 3);
                uint32_t odd = 0;  // NaN where a value is not finite
#pragma unroll 1
                for (int hh = 0; hh < 2; ++hh) {  // half of the columns
                    const uint32_t x = x0 + st * kStage + (((unit + 2 * hh) ^ row) << 4);
                    uint32_t q[8], h[8], m[8], l[8];
                    ldsm4_t(x, *reinterpret_cast<uint32_t (*)[4]>(q));
                    ldsm4_t(x + 2048, *reinterpret_cast<uint32_t (*)[4]>(q + 4));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 ww = w[4 * j];
                        if (OUT)
                            asm("fma.rn.bf16x2 %0, %1, %3, %0;\n\tfma.rn.bf16x2 %0, %2, %3, %0;"
                                : "+r"(odd)
                                : "r"(q[2 * j]), "r"(q[2 * j + 1]), "r"(0));
                        weigh3(q[2 * j], ww, h[2 * j], m[2 * j], l[2 * j]);
                        weigh3(q[2 * j + 1], ww, h[2 * j + 1], m[2 * j + 1], l[2 * j + 1]);
                    }
                    const uint32_t to = tw + ((uint32_t)(16 * hh) << 16);
                    tmem_st_16x128(to, h);
                    tmem_st_16x128(to + 16, m);
                    tmem_st_16x128(to + 32, l);
                }
                if (OUT) any = __any_sync(0xffffffffu, (odd & 0x7fff7fffu) != 0);
                tmem_st_wait();
            }
            tc_fence_before_sync();
            mbar_arrive(&bars[WX + half]);
            if (OUT) {
                if (on) {
                    unsigned char *bad = smem + kBad + (c & (kRing - 1)) * 256 + 128 * half;
                    if (any) mask_odd(smem, st, t0, bad, p0 + lane);
                    if (lane == 0) smem[kBadAt + (c & (kRing - 1)) * 8 + 2 * wq + half] = any;
                }
                mbar_arrive(&bars[MFULL + (c & 1)]);
            }
        }
    } else if (warp < kScore0) {
        // ================= outputs
        if (OUT) {
            const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
            const bool on = 32 * (warp & 3) < dv;
            // The warp's 32 columns of a chunk pass through shared memory: z comes
            // in and the outputs that take its place go out by TMA.  Rows of 64
            // bytes under the 64-byte swizzle (a row's four 16 bytes XORed with
            // half the row's number): eight rows of 8 x 8 blocks fall in different
            // banks.  Where TMA cannot go (z not 16-byte aligned, the rows of a
            // sequence's last chunk), lane = row lane / 4 of eight, 16 bytes lane % 4.
            const int r8 = lane >> 2, mine = r8 * 64 + (((lane & 3) ^ ((r8 >> 1) & 3)) << 4);
            const int wq = warp & 3, col0 = hv * dv + 32 * wq;
            const size_t col = (size_t)col0 + 8 * (lane & 3);
            const size_t ldo = (size_t)a.HV * dv;
            const uint16_t *z = static_cast<const uint16_t *>(a.z) + (row0 + r8) * a.ldz + col;
            uint16_t *out = static_cast<uint16_t *>(a.out) + (row0 + r8) * ldo + col;
            unsigned char *so = smem + kOut + wq * 4096;
            const bool gated = a.z != nullptr && on;
            // this lane's row of the 8 x 8 blocks (tokens, columns) of two loads or stores:
            // matrices 0 and 1 are adjacent columns, 2 and 3 the next eight tokens
            const int xr = (lane & 7) >> 1;
            const uint32_t blk = smem_u32(so) + ((lane >> 4) * 8 + (lane & 7)) * 64;
            int armed = -1;
            auto fetch = [&](int c) {
                unsigned char *sz = so + (c & 1) * 16384;
                if (a.z_tma) {
                    if (lane == 0) {
                        bulk_wait_read_all();  // the outputs that were there have gone
                        uint64_t *bar = &bars[ZFULL + 4 * (c & 1) + wq];
                        mbar_arrive_expect_tx(bar, 4096);
                        tma_load_2d(sz, &maps.z, col0, (int)(row0 + c * kC), bar);
                    }
                    armed = c;
                } else {
                    if (lane == 0) bulk_wait_read_all();
                    __syncwarp();
                    const int L = rows_in(c);
                    const uint16_t *q = z + (long long)c * kC * a.ldz;
#pragma unroll 1
                    for (int k = 0; k < 64; ++k) {
                        const int r = k & 56;  // eight rows at a time, element k & 7
                        if (r + r8 < L)
                            *reinterpret_cast<uint16_t *>(sz + mine + 64 * r + 2 * (k & 7)) =
                                __ldg(q + r * a.ldz + (k & 7));
                    }
                    __syncwarp();
                }
            };
            if (gated && NC > 0) fetch(0);
            uint32_t beyond = 0;  // chunks beyond r's range so far
            for (int c = 0; c < NC && !*abort_flag; ++c) {
                const int L = rows_in(c);
                const uint32_t ty = tl + kTmY + 64 * (c & 1);
                wait(YDONE + (c & 1), c >> 1);
                tc_fence_after_sync();
                const float *e = scal(c, kE);
                if (scal(c, kEnd)[2] != 0.f) {
                    // that was the part from the state alone: times exp(cum_t)
                    if (on)
#pragma unroll 1
                        for (int g = 0; g < 4; ++g) {
                            float y[16];
                            uint32_t q[16];
                            tmem_ld16(ty + 16 * g, y);
#pragma unroll
                            for (int m = 0; m < 16; ++m) q[m] = __float_as_uint(y[m] * e[16 * g + m]);
                            tmem_st16(ty + 16 * g, q);
                        }
                    tmem_st_wait();
                    tc_fence_before_sync();
                    mbar_arrive(&bars[YSCALED]);
                    wait(YPART, beyond++);
                    tc_fence_after_sync();
                    e = scal(c, kDiag);  // ones
                }
                auto combine = [&](auto with_z) {
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        const int hh = k & 1, t32 = k >> 1;  // half of the columns, of the tokens
                        const uint32_t at =
                            blk + (c & 1) * 16384 + t32 * 2048 + (((lane >> 3 & 1) + 2 * hh) ^ xr) * 16;
                        uint32_t y[16];
                        tmem_ld_16x256(ty + ((uint32_t)(16 * hh) << 16) + 32 * t32, y);
                        // meanwhile the factors: exp(cum - r), times silu(z)
                        float2 f[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            f[2 * j] = f[2 * j + 1] = *reinterpret_cast<const float2 *>(
                                e + 32 * t32 + 8 * j + 2 * (lane & 3));
                        if (with_z) {
                            uint32_t zt[8];
                            ldsm4_t(at, *reinterpret_cast<uint32_t (*)[4]>(zt));
                            ldsm4_t(at + 1024, *reinterpret_cast<uint32_t (*)[4]>(zt + 4));
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                f[i] = mul2(f[i], silu2(make_float2(__uint_as_float(zt[i] << 16),
                                                                    __uint_as_float(zt[i] & 0xffff0000u))));
                            }
                        }
                        tmem_ld_wait(y);
                        uint32_t o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 q = mul2(f[i], make_float2(__uint_as_float(y[2 * i]),
                                                                    __uint_as_float(y[2 * i + 1])));
                            o[i] = pack2(q.x, q.y);
                        }
                        stsm4_t(at, *reinterpret_cast<const uint32_t (*)[4]>(o));
                        stsm4_t(at + 1024, *reinterpret_cast<const uint32_t (*)[4]>(o + 4));
                    }
                };
                if (gated) {
                    if (c + 1 < NC) fetch(c + 1);
                    if (a.z_tma) wait(ZFULL + 4 * (c & 1) + wq, c >> 1);
                    combine(std::true_type{});
                } else if (on) {
                    // the outputs of two chunks before have gone
                    if (lane == 0) bulk_wait_read_but_one();
                    __syncwarp();
                    combine(std::false_type{});
                }
                tc_fence_before_sync();
                mbar_arrive(&bars[YFREE + (c & 1)]);
                if (on) {
                    unsigned char *sc = so + (c & 1) * 16384;
                    const unsigned char *any = smem + kBadAt + (c & (kRing - 1)) * 8 + 2 * wq;
                    if (*reinterpret_cast<const uint16_t *>(any)) {
                        // from a value of x on that is not finite
                        __syncwarp();
                        spoil(sc, any, smem + kBad + (c & (kRing - 1)) * 256 + 32 * wq + lane, lane);
                    }
                    if (L == kC) {
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(&maps.out, sc, col0, (int)(row0 + c * kC));
                            bulk_commit_group();
                        }
                    } else {
                        __syncwarp();
                        uint16_t *o = out + (size_t)c * kC * ldo;
#pragma unroll 1
                        for (int k = 0; k < 8; ++k, o += 8 * ldo)
                            if (8 * k + r8 < L)
                                *reinterpret_cast<uint4 *>(o) =
                                    *reinterpret_cast<const uint4 *>(sc + 512 * k + mine);
                    }
                }
            }
            if (lane == 0) {
                bulk_wait_all();
                if (*abort_flag)  // copies in flight land before the CTA leaves
#pragma unroll 1
                    for (int c = armed < 2 ? 0 : armed - 1; c <= armed; ++c)
                        mbar_wait_bounded(&bars[ZFULL + 4 * (c & 1) + wq], (c >> 1) & 1, kWaitNs);
            }
        }
    } else if (warp != kScalars && warp != kIssueState && warp != kIssueY && warp != kLoads) {
        // ================= scores: lane = token t of the chunk
        if (OUT) {
            const int sw = warp & 1, t = 32 * sw + lane;
            // 16 columns at a time, up to the row's own half; two warps take turns.  (A row
            // behind the sequence's end makes outputs that go nowhere.)
            const int g0 = (warp - kScore0) >> 2;
            const uint32_t tl = tmem + ((uint32_t)(32 * sw) << 16);
            const float D = a.D ? a.D[hv] : 0.f, A2 = a.A[hv] * kLog2e;
            for (int c = 0; c < NC && !*abort_flag; ++c, at.next()) {
                wait3(FULL + at.st, at.ph, GRAM, c, MFREE + (c & 1), (c >> 1) - 1);
                tc_fence_after_sync();
                unsigned char *m = smem + kM + (c & 1) * 16384 + kmajor_off(t, 0, kC);
                const bool far = scal(c, kEnd)[2] != 0.f;
                const float diag = far ? D : scal(c, kDiag)[t];
#pragma unroll 1
                for (int g = g0; g < 2 * sw + 2; g += 2) {
                    float d[16], w[16];
                    if (!far) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<float4 *>(w + e) =
                                *reinterpret_cast<const float4 *>(scal(c, kV) + 16 * g + e);
                    } else {
                        // exp(cum_t - cum_s) step_s, its exponent the sum of the tokens behind
                        // s up to t, from t's end on: what stands behind these 16 tokens,
                        // then one more of them a column.  (A difference of two sums would
                        // lose the slow decays beside a token that is large: 2^-24 of the sums.)
                        const float *step = scal(c, kStep) + 16 * g, *up = scal(c, kCum);
                        const int mine = t - 16 * g, quarter = t >> 4;
                        float sum = quarter > g ? up[t] : 0.f;
                        if (g < 1 && quarter > 1) sum += up[31];
                        if (g < 2 && quarter > 2) sum += up[47];
                        w[15] = fast_exp2(sum) * step[15];
#pragma unroll
                        for (int e = 14; e >= 0; --e) {
                            if (e < mine) sum = fmaf(step[e + 1], A2, sum);
                            w[e] = fast_exp2(sum) * step[e];
                        }
                    }
                    tmem_ld16(tl + kTmG + 16 * g, d);
                    if (g >= 2 * sw) {  // the warp's last: G is free again
                        tc_fence_before_sync();
                        mbar_arrive(&bars[GFREE]);
                    }
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 q = mul2(make_float2(d[e], d[e + 1]), make_float2(w[e], w[e + 1]));
                        d[e] = q.x;
                        d[e + 1] = q.y;
                    }
                    if (g >= 2 * sw) {  // columns of the row's own half
                        const int mine = t - 16 * g;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (e == mine) d[e] += diag;
                            d[e] = e <= mine ? d[e] : 0.f;
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 16; h += 8) {
                        uint4 hi, lo;
                        pair2(d[h], d[h + 1], hi.x, lo.x);
                        pair2(d[h + 2], d[h + 3], hi.y, lo.y);
                        pair2(d[h + 4], d[h + 5], hi.z, lo.z);
                        pair2(d[h + 6], d[h + 7], hi.w, lo.w);
                        *reinterpret_cast<uint4 *>(m + 256 * g + 16 * h) = hi;
                        *reinterpret_cast<uint4 *>(m + 8192 + 256 * g + 16 * h) = lo;
                    }
                }
                fence_async_smem();
                mbar_arrive(&bars[MFULL + (c & 1)]);
            }
        }
    } else if (warp == kLoads) {
        // ================= TMA
        const int nx = dv > 64 ? 2 : 1, nb = DK > 64 ? 2 : 1;
        int armed = -1;
        for (int c = 0; c < NC && !*abort_flag; ++c, at.next()) {
            const int st = at.st;
            if (c >= kStages) wait(EMPTY + st, at.ph ^ 1);
            if (*abort_flag) break;
            if (lane == 0) {
                uint64_t *bar = &bars[FULL + st];
                unsigned char *to = smem + st * kStage;
                mbar_arrive_expect_tx(bar, (uint32_t)(nx + (OUT ? 2 : 1) * nb) * 8192u);
                const int row = (int)(row0 + c * kC);
#pragma unroll 1
                for (int k = 0; k < nx; ++k)
                    tma_load_2d(to + kX + 8192 * k, &maps.x, hv * dv + 64 * k, row, bar);
#pragma unroll 1
                for (int k = 0; k < nb; ++k) {
                    tma_load_2d(to + kB + 8192 * k, &maps.b, hk * DK + 64 * k, row, bar);
                    if (OUT) tma_load_2d(to + kCm + 8192 * k, &maps.c, hk * DK + 64 * k, row, bar);
                }
                armed = c;
            }
            __syncwarp();
            const int L = rows_in(c);
            if (L < kC) {
                // the last chunk's rows behind the end hold other sequences'
                // values: zeros, since 0 times those may not be 0
                wait(FULL + st, at.ph);
#pragma unroll 1
                for (int k = lane; k < (kC - L) * 16; k += 32) {
                    const int r = L + k / 16;
                    const uint32_t o = ((k >> 3) & 1) * 8192 + r * 128 + (k & 7) * 16;
                    *reinterpret_cast<uint4 *>(smem + st * kStage + kX + o) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(smem + st * kStage + kB + o) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[FIX]);
            }
        }
        if (*abort_flag && lane == 0)  // copies in flight land before the CTA leaves
#pragma unroll 1
            for (int c = armed < kStages ? 0 : armed - kStages + 1; c <= armed; ++c)
                mbar_wait_bounded(&bars[FULL + c % kStages], (c / kStages) & 1, kWaitNs);
    } else if (warp == kScalars) {
        // ================= scalars: tokens 2 lane and 2 lane + 1
        const float A2 = a.A[hv] * kLog2e, bias = a.dt_bias ? a.dt_bias[hv] : 0.f;
        const float D = a.D ? a.D[hv] : 0.f;
        const float *dt = a.dt + row0 * a.HV + hv;
        auto dt_at = [&](int t) { return t < T ? __ldg(dt + (long long)t * a.HV) : 0.f; };
        float d0 = dt_at(2 * lane), d1 = dt_at(2 * lane + 1);
        double total = 0.0;  // log2 of the unit's decay
        for (int c = 0; c < NC && !*abort_flag; ++c, at.next()) {
            const int t = c * kC + 2 * lane;
            float s0 = ssm_step(d0, bias, a.softplus), s1 = ssm_step(d1, bias, a.softplus);
            s0 = t < T ? s0 : 0.f;
            s1 = t + 1 < T ? s1 : 0.f;
            d0 = dt_at(t + kC);
            d1 = dt_at(t + kC + 1);
            const float l0 = s0 * A2, l1 = s1 * A2;
            // sums within the half chunk of 16 lanes, of the tokens up to each
            // and of those behind it: no difference of long sums
            float up = l0 + l1, down = up;
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) {
                const float o = __shfl_up_sync(0xffffffffu, up, off, 16);
                const float q = __shfl_down_sync(0xffffffffu, down, off, 16);
                if ((lane & 15) >= off) up += o;
                if ((lane & 15) + off < 16) down += q;
            }
            float c0 = __shfl_up_sync(0xffffffffu, up, 1, 16);
            float f1 = __shfl_down_sync(0xffffffffu, down, 1, 16);
            c0 = ((lane & 15) ? c0 : 0.f) + l0;
            f1 = (lane & 15) < 15 ? f1 : 0.f;
            const float c1 = c0 + l1, f0 = f1 + l1;
            const float all0 = __shfl_sync(0xffffffffu, c1, 15), all1 = __shfl_sync(0xffffffffu, c1, 31);
            if (PASS == 1) total += (double)all0 + all1;
            float *q = scal(c, 0) + 2 * lane;
            auto put = [&](uint32_t what, float x, float y) {
                *reinterpret_cast<float2 *>(q + what / 4) = make_float2(x, y);
            };
            const float before = lane < 16 ? 0.f : all0, behind = lane < 16 ? all1 : 0.f;
            // r a whole number, so that exp(r) S is S but for its exponent
            float r = rintf(0.5f * (all0 + all1));
            const float p0 = before + c0, p1 = before + c1;
            // (a sum that is not a number counts as beyond: it would reach all of r's chunk)
            const bool far = __any_sync(0xffffffffu, !(fabsf(p0 - r) <= kRange && fabsf(p1 - r) <= kRange));
            float w0[3], w1[3];
            split_weight(fast_exp2(behind + f0) * s0, w0[0], w0[1], w0[2]);
            split_weight(fast_exp2(behind + f1) * s1, w1[0], w1[1], w1[2]);
            *reinterpret_cast<uint4 *>(scal(c, kW) + 4 * lane) =
                make_uint4(pack2(w0[0], w1[0]), pack2(w0[1], w1[1]), pack2(w0[2], w1[2]), 0);
            if (!far) {
                const float v0 = fast_exp2(r - p0), v1 = fast_exp2(r - p1);
                put(kE, fast_exp2(p0 - r), fast_exp2(p1 - r));
                put(kV, v0 * s0, v1 * s1);
                put(kDiag, D * v0, D * v1);
            } else {
                // kE rescales the part from the state; M is as it is, without D:
                // its columns of ones are what the outputs are scaled by
                r = 0.f;
                float in = l0 + l1;
#pragma unroll
                for (int off = 1; off < 8; off <<= 1) {
                    const float o = __shfl_up_sync(0xffffffffu, in, off, 8);
                    if ((lane & 7) >= off) in += o;
                }
                in = __shfl_up_sync(0xffffffffu, in, 1, 8);
                in = ((lane & 7) ? in : 0.f) + l0;
                put(kE, fast_exp2(p0), fast_exp2(p1));
                put(kCum, in, in + l1);
                put(kStep, s0, s1);
                put(kDiag, 1.f, 1.f);
            }
            if (lane == 0) {
                float *end = scal(c, kEnd);
                end[0] = fast_exp2(all0 + all1);
                end[1] = fast_exp2(r);
                end[2] = far ? 1.f : 0.f;
            }
            // there are as many more of these than stages as the outputs may lag
            // behind, but a stage's barrier counts one chunk at a time
            if (c >= kStages) wait(EMPTY + at.st, at.ph ^ 1);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[FULL + at.st]);
        }
        if (PASS == 1 && lane == 0) {
            a.seg_log[(size_t)unit * a.HV + hv] = (float)(total * 0.6931471805599453);
        }
    } else if (warp == kIssueState) {
        // ================= MMA issue: G and dS.  The warp waits as one, one lane issues
        constexpr uint32_t idG = idesc_bf16(128, kC, false, false, false);
        constexpr uint32_t idD = idesc_bf16(128, DK, false, true, false);
        // descriptors of stage 0; the stage, a box of 64 columns and a step's
        // 16 columns (K-major) or rows (MN-major) are added
        const uint32_t sb = smem_u32(smem);
        const uint64_t dB = smem_desc_sw128(sb + kB, 16, 1024), dC = smem_desc_sw128(sb + kCm, 16, 1024);
        const uint64_t dBt = smem_desc_sw128(sb + kB, 8192, 1024);
        auto gram = [&](int st) {
            const uint64_t o = (uint64_t)(st * (kStage >> 4));
            if (elect_one()) {
                products<false>(tmem + kTmG, dC + o, 2, 504, dB + o, 2, 504, idG, DK / 16, 0);
                mma_commit(&bars[GRAM]);
            }
            __syncwarp();
        };
        if (OUT && NC > 0) {
            wait(FULL, 0);
            gram(0);
        }
        for (int c = 0; c < NC && !*abort_flag; ++c) {
            const int st = at.st;
            const uint64_t o = (uint64_t)(st * (kStage >> 4));
            at.next();
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {  // 32 tokens at a time: three numbers against the same rows
                if (h == 0)
                    wait2(DFREE, c, WX, c);
                else
                    wait(WX + 1, c);
                tc_fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 6; ++k)
                        mma_bf16_ts(tmem + kTmD, tmem + kTmW + 48 * h + 8 * k,
                                    dBt + o + 256 * h + 128 * (k & 1), idD, h + k > 0);
                    mma_commit(&bars[WFREE + h]);
                    if (h) {
                        mma_commit(&bars[DELTA]);
                        mma_commit(&bars[EMPTY + st]);
                    }
                }
                __syncwarp();
            }
            if (OUT && c + 1 < NC) {
                wait2(FULL + at.st, at.ph, GFREE, c);
                tc_fence_after_sync();
                gram(at.st);
            }
        }
        // every MMA is done before the tensor memory goes
        if (elect_one()) mma_commit(&bars[LAST]);
        __syncwarp();
        mbar_wait_bounded(&bars[LAST], 0, kWaitNs);
    } else if (OUT) {
        // ================= MMA issue: Y
        constexpr uint32_t idY2 = idesc_bf16(128, kC, false, false, false);
        constexpr uint32_t idY1 = idesc_bf16(128, kC, true, false, false);
        const uint32_t sb = smem_u32(smem);
        const uint64_t dC = smem_desc_sw128(sb + kCm, 16, 1024), dXt = smem_desc_sw128(sb + kX, 8192, 1024);
        const uint64_t dM = smem_desc(sb + kM, 128, kC * 16);
        uint32_t beyond = 0;
        for (int c = 0; c < NC && !*abort_flag; ++c, at.next()) {
            const uint64_t o = (uint64_t)(at.st * (kStage >> 4)), m = dM + (uint64_t)((c & 1) * 1024);
            const uint32_t y = tmem + kTmY + 64 * (c & 1);
            wait3(FULL + at.st, at.ph, SFULL, c, YFREE + (c & 1), (c >> 1) - 1);
            const bool far = scal(c, kEnd)[2] != 0.f;
            tc_fence_after_sync();
            if (elect_one()) {
                products<true>(y, tmem + kTmS, 8, 0, dC + o, 2, 504, idY2, DK / 16, 0);
                mma_commit(&bars[SFREE]);
                if (far) mma_commit(&bars[YDONE + (c & 1)]);
            }
            __syncwarp();
            if (far) wait(YSCALED, beyond++);
            wait(MFULL + (c & 1), c >> 1);
            tc_fence_after_sync();
            if (elect_one()) {
                // M's hi, then its lo (8192 bytes on), against the same x
                products<false>(y, dXt + o, 128, -512, m, 16, 448, idY1, 8, 1);
                mma_commit(&bars[MFREE + (c & 1)]);
                mma_commit(far ? &bars[YPART] : &bars[YDONE + (c & 1)]);
                mma_commit(&bars[EMPTY + at.st]);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(&bars[LAST + 1]);
        __syncwarp();
        mbar_wait_bounded(&bars[LAST + 1], 0, kWaitNs);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (tid == 0 && *abort_flag && err) atomicExch(err, 1);
    if (warp == 0) tmem_dealloc(tmem, kTmCols);
}

// A tensor as [rows][width], rows ld elements apart: boxes of 64 rows of
// `cols`, swizzled over that many bytes.
bool encode(EncodeTiledFn fn, CUtensorMap *m, const void *p, long long width, long long rows,
            long long ld, int cols) {
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {(cuuint32_t)cols, 64}, one[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int PASS>
cudaError_t launch(const SsmArgs &a, const Maps &maps, int *err, cudaStream_t stream) {
    auto k = gdr_ssm_chunk_kernel<DK, PASS>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    return for_sequences(a.cu, a.N, a.T, a.seg_rows, [&](const SeqTable &t, long long units) {
        trace_begin(kKernSsm, stream);
        k<<<(unsigned)(units * a.HV), kThreads, kSmem, stream>>>(a, t, maps, err);
        trace_end(kKernSsm, stream);
        return cudaGetLastError();
    });
}

}  // namespace

bool ssm_chunks_supported(const SsmArgs &a) {
    const long long rows = a.cu ? a.cu[a.N] : (long long)a.N * a.T;
    const uintptr_t any = (uintptr_t)a.x | (uintptr_t)a.b | (uintptr_t)a.c;
    return a.bf16 && rows <= INT_MAX - kC && (any & 15u) == 0 && a.ldx % 8 == 0 && a.ldb % 8 == 0 &&
           a.ldc % 8 == 0 && a.ldx < (1LL << 38) && a.ldb < (1LL << 38) && a.ldc < (1LL << 38);
}

cudaError_t launch_ssm_chunks(const SsmArgs &given, int pass, cudaStream_t stream) {
    int *err = nullptr;
    cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return e;
    const EncodeTiledFn fn = tma_encode_fn(&e);
    if (e != cudaSuccess) return e;
    SsmArgs a = given;
    const long long rows = a.cu ? a.cu[a.N] : (long long)a.N * a.T;
    const long long wx = (long long)a.HV * a.dv, wb = (long long)a.HK * a.dk;
    a.z_tma = a.z && ((uintptr_t)a.z & 15u) == 0 && a.ldz % 8 == 0 && a.ldz < (1LL << 38);
    Maps m = {};
    if (!encode(fn, &m.x, a.x, wx, rows, a.ldx, 64) || !encode(fn, &m.b, a.b, wb, rows, a.ldb, 64) ||
        !encode(fn, &m.c, a.c, wb, rows, a.ldc, 64) || !encode(fn, &m.out, a.out, wx, rows, wx, 32) ||
        (a.z_tma && !encode(fn, &m.z, a.z, wx, rows, a.ldz, 32)))
        return cudaErrorInvalidValue;
    switch (a.dk) {
        case 32: return pass == 0 ? launch<32, 0>(a, m, err, stream)
                        : pass == 1 ? launch<32, 1>(a, m, err, stream) : launch<32, 2>(a, m, err, stream);
        case 64: return pass == 0 ? launch<64, 0>(a, m, err, stream)
                        : pass == 1 ? launch<64, 1>(a, m, err, stream) : launch<64, 2>(a, m, err, stream);
        default: return pass == 0 ? launch<128, 0>(a, m, err, stream)
                        : pass == 1 ? launch<128, 1>(a, m, err, stream) : launch<128, 2>(a, m, err, stream);
    }
}

}  // namespace gdr
