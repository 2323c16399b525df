// prefill_bf16.cu -- attention of several new tokens over the uncompressed cache
// (rq_prefill_attn_window on RQ_FMT_BF16): causal, with an optional sliding
// window and sinks.  The query at position p sees (p - window, p] and
// [0, sinks).
//
//   z = q K^T scale,  out = sum_t 2^(z_t - m) v_t / sum_t 2^(z_t - m)
// in one pass over the keys, with a running maximum m that is raised only when
// a row's maximum grows by more than 2^8 (then the row's accumulated output is
// rescaled).
//
// CTA = (split of the tokens, kv head, sequence x block of QT * 128 query rows,
// row = query token x head of the group).  Per 128-token tile and 128 rows, on
// the tcgen05 tensor cores:
//   S = Q K^T   8 MMAs of 128x128x16, both operands from shared memory
//   O += P V    8 MMAs of 128x128x16 with P from tensor memory, for each of P's
//               PP BF16 parts: one for BF16 output (half a step, 2^-9 of each
//               weight, is as small as the output's own rounding), a high and
//               a low one for fp32 output (2^-18; a third one did not lower what
//               the tensor cores' sums leave: they are cut off, not rounded,
//               which makes a row smaller by 2e-9 of itself for every token that
//               its split sums: 3e-6 for 1500, 2e-5 for 8192)
// P overwrites S in tensor memory; O is beside it (128 columns each).  Two S
// buffers keep the tensor cores and the softmax busy at once: with QT = 2 one
// per row tile -- one tile's MMAs run while the other's softmax does, and both
// share every K and V tile, which halves the L2 traffic (a 128 x 128 tile pair
// is 64 KB for 2 x 1024 tensor cycles); with QT = 1 (few rows) one per parity
// of the token tile.
// Several splits' partials are merged by a launch of its own.
//
// Warps: 4 QT softmax warps (a thread per row: tensor-memory lane = row), then
// one that issues the TMA loads (K and V tiles alternate in a ring of
// 128-byte-swizzled 32 KB stages) and one that issues the MMAs.
// Hand-offs, all bounded waits (error word, abort flag):
//   full[s]   TMA -> MMA          stage s loaded
//   empty[s]  MMA commit -> TMA   stage s read
//   sfull[i]  MMA commit -> softmax   S buffer i complete, and with it all MMAs
//             issued before (QT = 2: the values of the tile before among them)
//   pfull[i]  softmax -> MMA      P written over S buffer i
//   odone[q]  MMA commit -> softmax   values of a tile complete (before O is
//             rescaled with QT = 1, and at the end)
//
// RB: the same over a compressed cache.  A first launch (rebuild.cu) writes the
// tokens that the chunk sees, committed and tail, into a workspace, once for all
// the chunk's rows, as BF16 numbers: K and V as pairs for fp32 output, V as one
// number (2^-9, as small as the output's own rounding) for BF16 output:
//   S = Q (Khi + Klo)^T,  O += (Phi + Plo) Vhi + Phi Vlo.
// What is left out of a number is relative to it, whatever its size.  FP16
// operands would be faster (11 bits in one part each: 37, 38 and 54 us for the
// cases below), but under any one scale small values, and weights below 2^-25 of
// the largest, would be lost.  BF16 output with one part of P too: 39, 40 and 60
// us, relative error of the rows 2.2 to 2.7e-3 instead of 1.7 to 2.4e-3 (1.65e-3
// is the output's rounding); with one of P and two of V: 45, 54 and 70 us.  (P's
// high part is then cut off rather than rounded, which takes fewer operations: 41
// instead of 42 us for the first case.)
//
// What bounds it: the chain of a tile -- logits, maximum, exponentials, P handed
// over -- in a thread per row, a warp or two per scheduler; no unit is busy: 8192
// causal tokens, 16 heads, 313 us = 878 TFLOP/s, tensor pipe 36%, special-function
// pipe 37%, issue slots 26% in a 4096-token run.  Few rows over a short window
// also pay for launches and the pipeline's filling: 511 tokens in two sequences of
// 4 kv heads of 4, window 1024 (8.6 GFLOP), fp32 output, 30 us (tensor pipe 27%).
// Over compressed caches (all launches, BF16 output): 16 tokens of 4 x 16 heads,
// window 1024, 41 us; 500 tokens in two sequences of 4 kv heads of 4 heads, window
// 2000, 48 us; 2048 tokens of 16 heads, window 1024, 70 us (tensor pipe 44%).
//
// A V row that only some rows see may hold NaN or infinities, which 0 * NaN
// would carry into the other rows.  The store kernel notes in the arena when it
// was ever given such a V (a.nonfinite); only then, the first softmax warps look
// every V tile over before its values are formed, zero such rows and flag them,
// and rows that do see one get a NaN weight.  (A NaN in K stays in the token's
// own logits, which the rows that do not see it replace.)
#include <cuda.h>
#include <math_constants.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "combine.cuh"
#include "common.cuh"
#include "prefill.h"
#include "read.h"
#include "sync.cuh"
#include "tc.cuh"

namespace rq {
namespace {

constexpr int kTileT = 128;                          // tokens per tile
constexpr int kTileR = 128;                          // rows per row tile
constexpr int kBlkBytes = 128 * 128;                 // 128 rows of 64 BF16 columns
constexpr int kStageBytes = 2 * kBlkBytes;           // a K or V tile, or a Q row tile
constexpr float kRaiseLog2 = 8.f;
constexpr int kMerge = 8;                            // split partials of a row loaded at once

template <int QT>
struct Cfg {
    static constexpr int STAGES = 7 - QT;
    static constexpr int THREADS = 32 * (4 * QT + 2);
    static constexpr int SMEM = (QT + STAGES) * kStageBytes + 1024;   // + alignment of the base
    static constexpr uint32_t COLS = 512;            // S buffers at columns 0 and 128, O of row tile q at 256 + 128 q
};

// ---------------------------------------------------------------- PTX helpers
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]: A is M lanes x K / 2 columns of BF16 pairs.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
#define RQ_R32(v) \
    "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), \
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), \
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), \
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
#define RQ_W32(c, v) \
    c(v[0]), c(v[1]), c(v[2]), c(v[3]), c(v[4]), c(v[5]), c(v[6]), c(v[7]), c(v[8]), c(v[9]), c(v[10]), c(v[11]), \
        c(v[12]), c(v[13]), c(v[14]), c(v[15]), c(v[16]), c(v[17]), c(v[18]), c(v[19]), c(v[20]), c(v[21]), c(v[22]), \
        c(v[23]), c(v[24]), c(v[25]), c(v[26]), c(v[27]), c(v[28]), c(v[29]), c(v[30]), c(v[31])
#define RQ_OUT_REG(x) "=r"(x)
#define RQ_INOUT_REG(x) "+r"(x)
// 32 consecutive columns of the warp's 32 lanes (usable after wait_ld / settle)
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : RQ_W32(RQ_OUT_REG, v)
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        RQ_R32(v)
        : "memory");
}
__device__ __forceinline__ void wait_ld32(uint32_t *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : RQ_W32(RQ_INOUT_REG, v)::"memory");
}
// no use of v is scheduled before this point (and so not before a wait above it)
__device__ __forceinline__ void settle32(uint32_t *v) { asm volatile("" : RQ_W32(RQ_INOUT_REG, v)::"memory"); }

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float x0, float x1) {   // x0 in the low half
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(x1), "f"(x0));
    return d;
}
// bits [lo, hi) of a 32-bit word (clamped)
__device__ __forceinline__ uint32_t range_bits(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 32);
    return hi <= lo ? 0u : (0xFFFFFFFFu >> (32 - (hi - lo))) << lo;
}

struct Bf16Args {
    const uint16_t *q;      // [B][n][Hq][d]
    float *partials;        // [B][n][Hq][S][kPartialStride]
    float *out;             // [B][n][Hq][d] fp32, or
    uint16_t *out16;        // BF16
    int *err;
    const int *nonfinite;   // a V that is not finite was ever stored
    SeqLens seqT;
    int B, H, Hq, G, n, n_tail, S, nqb;   // n_tail: tokens after the committed ones (RB)
    int h0;                 // RB: the launch's first kv head; z counts the launch's heads
    int heads;              // of the launch
    int window, sinks;
    float scale_log2;
};

// Tensor maps: K and V (RB: the rebuilt rows' high parts, and their low ones).
struct Maps {
    CUtensorMap k, v, k_lo, v_lo;
};

// The token runs that rows of query tokens [i0, i1] read of a sequence of `end`
// tokens, in tiles of 128: the sinks', the window's.
struct Runs {
    int sink_tiles, sink_end, w_tile, tiles;
    __host__ __device__ Runs(int end, int n, int i0, int i1, int window, int sinks) {
        const BlockRuns r = block_runs(end, n, i0, i1, window, sinks);
        w_tile = r.w_tile;
        sink_end = r.sink_end;
        sink_tiles = (r.sink_end + kTileT - 1) / kTileT;
        tiles = sink_tiles + (r.lim - r.w_tile + kTileT - 1) / kTileT;
    }
    __host__ __device__ int token(int tile) const {
        return tile < sink_tiles ? tile * kTileT : w_tile + (tile - sink_tiles) * kTileT;
    }
};

template <int QT, int PP, int VP, bool RB>
__global__ void __launch_bounds__(Cfg<QT>::THREADS, 1)
    prefill_bf16_kernel(const __grid_constant__ Maps maps, const Bf16Args a) {
    using C = Cfg<QT>;
    constexpr int NS = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar_full[NS], bar_empty[NS], bar_sfull[2], bar_pfull[2], bar_odone[QT];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ uint8_t s_bad[kTileT];

    const uint32_t raw_base = smem_u32(smem_raw);
    uint8_t *sm = smem_raw + (((raw_base + 1023u) & ~1023u) - raw_base);   // Q row tiles, then the stages
    const uint32_t sbase = smem_u32(sm);
    uint8_t *stages = sm + QT * kStageBytes;
    const uint32_t sstage = sbase + QT * kStageBytes;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int split = blockIdx.x, h = a.h0 + blockIdx.y, z = blockIdx.z / a.nqb * a.heads + blockIdx.y;
    const int b = blockIdx.z / a.nqb, qb = a.nqb - 1 - blockIdx.z % a.nqb;   // the longest row blocks first
    const int r0 = qb * QT * kTileR;
    const int nr = min(QT * kTileR, a.n * a.G - r0);
    const int Tb = a.seqT.v[b] + a.n_tail;   // tokens of the sequence
    const Runs runs(Tb, a.n, r0 / a.G, (r0 + nr - 1) / a.G, a.window, a.sinks);
    // this split's tiles
    const int j0 = (int)((long long)split * runs.tiles / a.S), j1 = (int)((long long)(split + 1) * runs.tiles / a.S);
    const int nt = j1 - j0;
    // stages of tile j of the split: K in KP parts, V in VP
    constexpr int KP = RB ? 2 : 1;
    // S buffer of row tile q's token tile j, and the parity of its phase then
    auto sbuf = [](int q, int j) { return QT == 2 ? q : j & 1; };
    auto sphase = [](int j) { return QT == 2 ? j & 1 : (j >> 1) & 1; };
    auto kstage = [](int j) { return (KP + VP) * j; };
    auto vstage = [](int j) { return (KP + VP) * j + KP; };

    if (tid == 0) {
        for (int i = 0; i < NS; i++) {
            mbar_init(&bar_full[i], 1);
            mbar_init(&bar_empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&bar_sfull[i], 1);
            mbar_init(&bar_pfull[i], 4);   // a lane of each of its softmax warps
        }
        for (int i = 0; i < QT; i++) mbar_init(&bar_odone[i], 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4 * QT + 1) {
        tc::alloc(&s_tmem, C::COLS);
        tc::relinquish();
    }
    // Q rows, 16-byte chunks swizzled as TMA does; rows past nr are zero
    for (int i = tid; i < QT * kTileR * 16; i += C::THREADS) {
        const int row = i >> 4, c = i & 15;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < nr) {
            const int rg = r0 + row, t = rg / a.G, gq = rg % a.G;
            v = __ldg(reinterpret_cast<const uint4 *>(a.q + (((size_t)b * a.n + t) * a.Hq + h * a.G + gq) * kHeadDim) + c);
        }
        *reinterpret_cast<uint4 *>(sm + (row / kTileR) * kStageBytes + (c >> 3) * kBlkBytes +
                                   tc::sw_chunk(row % kTileR, c & 7)) = v;
    }
    tc::fence_async_smem();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s_tmem;
    // RB: the rebuilding launch before this one may still be running until here
    // (q and the tail were written before that one began)
    if (RB) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    volatile int *abort_flag = &s_abort;
    auto wait = [&](uint64_t *bar, int parity, int code) {
        if (mbar_wait(bar, (uint32_t)parity, abort_flag)) return true;
        *abort_flag = 1;
        atomicExch(a.err, code);
        return false;
    };

    if (warp == 4 * QT) {
        // ------------------------------------------------------- TMA
        if (lane == 0) {
            const RebuiltRows rb = RB ? rebuilt_rows(Tb, a.n, a.window, a.sinks) : RebuiltRows{0, 0};
            int it = 0;
            bool ok = true;
            // rows from y on of (sequence, head) z into the next stage
            auto load = [&](const CUtensorMap *map, int y) {
                const int s = it % NS;
                if (ok && it >= NS) ok = wait(&bar_empty[s], (it / NS - 1) & 1, 31);
                if (!ok) return;
                const uint32_t dst = sstage + s * kStageBytes;
                expect_tx(&bar_full[s], kStageBytes);
                tma_3d(dst, map, 0, y, z, &bar_full[s]);
                tma_3d(dst + kBlkBytes, map, 64, y, z, &bar_full[s]);
                it++;
            };
            for (int j = 0; j < nt && ok; j++) {
                const int t = runs.token(j0 + j);
                const int y = RB && j0 + j >= runs.sink_tiles ? rb.sink_pad + t - rb.w_base : t;
                load(&maps.k, y);
                if (KP > 1) load(&maps.k_lo, y);
                load(&maps.v, y);
                if (VP > 1) load(&maps.v_lo, y);
            }
            // every issued load must have landed before the CTA exits
            for (int i = max(0, it - NS); i < it; i++) mbar_wait<256>(&bar_full[i % NS], (i / NS) & 1, abort_flag);
        }
        __syncwarp();
    } else if (warp == 4 * QT + 1) {
        // ------------------------------------------------------- MMA
        if (lane == 0) {
            constexpr uint32_t idS = tc::idesc_bf16(kTileR, kTileT, false);    // K: K-major
            constexpr uint32_t idO = tc::idesc_bf16(kTileR, kHeadDim, true);   // V: MN-major
            auto logits = [&](int q, int j) {
                const uint64_t da = tc::desc_k(sbase + q * kStageBytes);
#pragma unroll
                for (int p = 0; p < KP; p++) {
                    const int s = (kstage(j) + p) % NS;
                    const uint64_t db = tc::desc_k(sstage + s * kStageBytes);
#pragma unroll
                    for (int kk = 0; kk < 8; kk++) {
                        const uint64_t o = (uint64_t)(((kk >> 2) * kBlkBytes + (kk & 3) * 32) >> 4);
                        tc::mma_bf16(tmem + sbuf(q, j) * 128, da + o, db + o, idS, p > 0 || kk > 0);
                    }
                    if (q == QT - 1) tc::commit(&bar_empty[s]);
                }
                tc::commit(&bar_sfull[sbuf(q, j)]);
            };
            auto values = [&](int q, int j) {
                // P's parts against V, then its high part against V's low one
                constexpr int terms = PP + VP - 1;
#pragma unroll
                for (int p = 0; p < terms; p++) {
                    const int s = (vstage(j) + (p == PP ? 1 : 0)) % NS;
                    const uint64_t dv = tc::desc_mn(sstage + s * kStageBytes, kBlkBytes);
                    const uint32_t pa = tmem + sbuf(q, j) * 128 + (p == 1 && PP > 1 ? 64 : 0);
#pragma unroll
                    for (int kk = 0; kk < 8; kk++)
                        mma_ts(tmem + 256 + q * 128, pa + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), idO,
                               j > 0 || p > 0 || kk > 0);
                    if (q == QT - 1 && p >= PP - 1) tc::commit(&bar_empty[s]);
                }
                tc::commit(&bar_odone[q]);
            };
            auto loaded = [&](int i, int code) { return wait(&bar_full[i % NS], (i / NS) & 1, code); };
            auto k_loaded = [&](int j) { return loaded(kstage(j), 32) && (KP == 1 || loaded(kstage(j) + 1, 33)); };
            auto v_loaded = [&](int j) { return loaded(vstage(j), 34) && (VP == 1 || loaded(vstage(j) + 1, 35)); };
            // logits run AHEAD tiles before values: with QT = 1 into the other S buffer
            constexpr int AHEAD = QT == 2 ? 1 : 2;
            bool ok = true;
            for (int j = 0; j < min(AHEAD, nt) && ok; j++) {
                ok = k_loaded(j);
                if (!ok) break;
                tc::fence_after();
                for (int q = 0; q < QT; q++) logits(q, j);
            }
            for (int j = 0; j < nt && ok; j++) {
                ok = v_loaded(j);
                for (int q = 0; q < QT && ok; q++) {
                    ok = wait(&bar_pfull[sbuf(q, j)], sphase(j), 36);
                    if (!ok) break;
                    tc::fence_after();
                    values(q, j);
                    if (j + AHEAD < nt) {
                        if (q == 0) ok = k_loaded(j + AHEAD);
                        if (!ok) break;
                        logits(q, j + AHEAD);
                    }
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- softmax
        const int q = warp >> 2;                       // row tile
        const int row = q * kTileR + (warp & 3) * 32 + lane;
        const bool live = q * kTileR + (warp & 3) * 32 < nr;   // warp-uniform: some row of the warp exists
        const int pos = Tb - a.n + (r0 + row) / a.G;   // the row's position
        const int lim = pos + 1;
        const int lo = (int)max(0ll, (long long)pos + 1 - a.window);
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16), tO = lanes + 256 + q * 128;
        const bool careful = __ldcg(a.nonfinite) != 0;
        const float scale_log2 = a.scale_log2;
        float m_used = -CUDART_INF_F, l = 0.f;
        for (int j = 0; j < nt; j++) {
            const int tb = runs.token(j0 + j);
            // a sinks' tile may reach into the window's: its part ends before that
            const int end = j0 + j < runs.sink_tiles ? min(lim, runs.sink_end) : lim;
            const uint32_t tS = lanes + sbuf(q, j) * 128;
            wait(&bar_sfull[sbuf(q, j)], sphase(j), 38);
            tc::fence_after();
            if (careful) {
                // V rows that are not finite become zeros with a flag (thread t: token t);
                // after S, so that the stage's phase before V's is known to be over
                asm volatile("bar.sync 1, %0;" ::"n"(128 * QT) : "memory");
                if (q == 0) {
                    const int s = vstage(j) % NS, t = tid;
                    wait(&bar_full[s], (vstage(j) / NS) & 1, 37);
                    const int s_lo = (vstage(j) + 1) % NS;
                    constexpr bool has_lo = VP > 1;
                    if (has_lo) wait(&bar_full[s_lo], ((vstage(j) + 1) / NS) & 1, 37);
                    uint32_t bad = 0;
                    for (int c = 0; c < 16; c++) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(stages + s * kStageBytes + (c >> 3) * kBlkBytes +
                                                                         t * 128 + (c & 7) * 16);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; i++)   // exponents all ones
                            bad |= ((w[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                    }
                    if (bad)
                        for (int c = 0; c < (has_lo ? 32 : 16); c++)
                            *reinterpret_cast<uint4 *>(stages + (c < 16 ? s : s_lo) * kStageBytes + ((c >> 3) & 1) * kBlkBytes +
                                                       t * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    s_bad[t] = bad ? 1 : 0;
                    tc::fence_async_smem();
                }
                asm volatile("bar.sync 1, %0;" ::"n"(128 * QT) : "memory");
            }
            if (live) {
                uint32_t s[128];
#pragma unroll
                for (int c = 0; c < 4; c++) ld32(tS + 32 * c, s + 32 * c);
                wait_ld32(s);
#pragma unroll
                for (int c = 1; c < 4; c++) settle32(s + 32 * c);
                if (__any_sync(0xffffffffu, tb + kTileT > end || (tb < lo && tb + kTileT > a.sinks))) {   // an edge lies in the tile
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        const int p = tb + 32 * c;
                        const uint32_t vis = range_bits(0, end - p) & (range_bits(lo - p, 32) | range_bits(0, a.sinks - p));
                        if (__all_sync(0xffffffffu, vis == 0xFFFFFFFFu)) continue;   // uniform
#pragma unroll
                        for (int k = 0; k < 32; k++)
                            if (!((vis >> k) & 1u)) s[32 * c + k] = 0xFF800000u;   // -inf
                    }
                }
                if (careful) {   // a visible token whose V is not finite
#pragma unroll
                    for (int k = 0; k < 128; k++)
                        if (s_bad[k] && s[k] != 0xFF800000u) s[k] = 0x7FC00000u;   // NaN
                }
                float m8[8];   // independent chains: one would be 127 dependent steps
#pragma unroll
                for (int k = 0; k < 8; k++) m8[k] = __uint_as_float(s[k]);
#pragma unroll
                for (int k = 8; k < 128; k += 8)
#pragma unroll
                    for (int i = 0; i < 8; i++) m8[i] = fmaxf(m8[i], __uint_as_float(s[k + i]));
                float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
                mx *= scale_log2;
                const bool raise = mx > m_used + kRaiseLog2;   // false while nothing is seen
                const bool rescale = raise && m_used != -CUDART_INF_F;
                const float f = rescale ? exp2f(m_used - mx) : 1.f;
                if (raise) m_used = mx;
                if (__any_sync(0xffffffffu, rescale)) {
                    // QT = 1: the values of tile j - 1 may still be running (those of j - 2 are
                    // not: S of this tile came after them)
                    if (QT == 1 && j > 0) {
                        wait(&bar_odone[q], (j - 1) & 1, 40);
                        tc::fence_after();
                    }
#pragma unroll 1
                    for (int c = 0; c < 4; c++) {
                        uint32_t v[32];
                        ld32(tO + 32 * c, v);
                        wait_ld32(v);
#pragma unroll
                        for (int k = 0; k < 32; k++) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
                        st32(tO + 32 * c, v);
                    }
                }
                l *= f;
                const float off = m_used == -CUDART_INF_F ? 0.f : -m_used;
                const F2 sc2 = pack2(scale_log2, scale_log2), off2 = pack2(off, off), neg1 = pack2(-1.f, -1.f);
                F2 sum[4];
#pragma unroll
                for (int k = 0; k < 4; k++) sum[k] = pack2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    uint32_t hi[32], low[PP > 1 ? 32 : 1];
#pragma unroll
                    for (int k = 0; k < 32; k++) {
                        const int u = 64 * c + 2 * k;
                        float p0, p1;
                        unpack2(fma2(pack2(__uint_as_float(s[u]), __uint_as_float(s[u + 1])), sc2, off2), p0, p1);
                        p0 = ex2f(p0);
                        p1 = ex2f(p1);
                        sum[k & 3] = add2(sum[k & 3], pack2(p0, p1));
                        const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
                        if (RB && VP == 1) {   // BF16 output: the high part cut off, what is left rounded (2^-16)
                            hi[k] = __byte_perm(b0, b1, 0x7632);
                            float r0, r1;
                            unpack2(fma2(pack2(__uint_as_float(b0 & 0xFFFF0000u), __uint_as_float(b1 & 0xFFFF0000u)), neg1,
                                         pack2(p0, p1)), r0, r1);
                            low[k] = pack_bf16(r0, r1);
                        } else {
                            hi[k] = pack_bf16(p0, p1);
                            if (PP > 1)
                                low[k] = pack_bf16(p0 - __uint_as_float(hi[k] << 16), p1 - __uint_as_float(hi[k] & 0xFFFF0000u));
                        }
                    }
                    __syncwarp();
                    st32(tS + 32 * c, hi);
                    if (PP > 1) st32(tS + 64 + 32 * c, low);
                }
                float l0, l1;
                unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), l0, l1);
                l += l0 + l1;
                tc::wait_st();
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_pfull[sbuf(q, j)]);
        }
        // ------------------------------------------------------- output
        if (nt > 0) {
            // (QT = 1: the last S says that the values of tile nt - 3 are complete, so the phase
            // before the last is waited for first)
            if (QT == 1 && nt > 1) wait(&bar_odone[q], nt & 1, 39);
            wait(&bar_odone[q], (nt - 1) & 1, 39);
            tc::fence_after();
        }
        if (live) {
            const int rg = r0 + row, t = rg / a.G, gq = rg % a.G;
            const size_t prow = ((size_t)b * a.n + t) * a.Hq + h * a.G + gq;
            float *part = a.partials + (prow * a.S + split) * kPartialStride;
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
            for (int c = 0; c < 4; c++) {
                uint32_t v[32];
                if (nt > 0) {
                    ld32(tO + 32 * c, v);
                    wait_ld32(v);
                }
                if (row < nr) {
                    if (nt == 0 || l == 0.f) {
#pragma unroll
                        for (int k = 0; k < 32; k++) v[k] = 0u;
                    }
                    if (a.S > 1) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4 *>(part + 32 * c + k) =
                                make_float4(__uint_as_float(v[k]), __uint_as_float(v[k + 1]), __uint_as_float(v[k + 2]),
                                            __uint_as_float(v[k + 3]));
                    } else if (a.out16) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                w[i] = pack_bf16(__uint_as_float(v[k + 2 * i]) * inv, __uint_as_float(v[k + 2 * i + 1]) * inv);
                            *reinterpret_cast<uint4 *>(a.out16 + prow * kHeadDim + 32 * c + k) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4 *>(a.out + prow * kHeadDim + 32 * c + k) =
                                make_float4(__uint_as_float(v[k]) * inv, __uint_as_float(v[k + 1]) * inv,
                                            __uint_as_float(v[k + 2]) * inv, __uint_as_float(v[k + 3]) * inv);
                    }
                }
                __syncwarp();   // converged for the next load
            }
            if (a.S > 1 && row < nr) {
                part[kHeadDim] = l == 0.f ? -CUDART_INF_F : m_used;
                part[kHeadDim + 1] = l;
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 4 * QT + 1) {
        tc::fence_after();
        tc::dealloc(tmem, C::COLS);
    }
}

// Merges the split partials of the output rows: a warp per row.  A launch of its
// own -- the last CTA of a row block merging its 128 rows, as the other kernels
// do for few rows, took up to 40 us.
__global__ void __launch_bounds__(128) merge_rows_kernel(const Bf16Args a, long long rows) {
    const int lane = threadIdx.x & 31;
    const long long prow = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (prow >= rows) return;   // uniform per warp
    const float *part = a.partials + (size_t)prow * a.S * kPartialStride;
    float M = -CUDART_INF_F, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < a.S; s0 += kMerge) {   // a batch's loads are in flight together
        float m[kMerge], ls[kMerge];
        float4 v[kMerge];
#pragma unroll
        for (int u = 0; u < kMerge; u++) {
            const float *p = part + (size_t)min(s0 + u, a.S - 1) * kPartialStride;
            m[u] = __ldcg(p + kHeadDim);
            ls[u] = __ldcg(p + kHeadDim + 1);
            v[u] = __ldcg(reinterpret_cast<const float4 *>(p) + lane);
        }
#pragma unroll
        for (int u = 0; u < kMerge; u++) {
            if (s0 + u >= a.S || (m[u] == -CUDART_INF_F && ls[u] == 0.f)) continue;   // uniform: no key in this split
            const float Mn = fmaxf(M, m[u]);
            const float c0 = M == -CUDART_INF_F ? 0.f : exp2f(M - Mn), c = m[u] == -CUDART_INF_F ? 1.f : exp2f(m[u] - Mn);
            l = fmaf(ls[u], c, l * c0);
            o[0] = fmaf(v[u].x, c, o[0] * c0);
            o[1] = fmaf(v[u].y, c, o[1] * c0);
            o[2] = fmaf(v[u].z, c, o[2] * c0);
            o[3] = fmaf(v[u].w, c, o[3] * c0);
            M = Mn;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (a.out16)
        *reinterpret_cast<uint2 *>(a.out16 + prow * kHeadDim + 4 * lane) =
            make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
    else
        *reinterpret_cast<float4 *>(a.out + prow * kHeadDim + 4 * lane) =
            make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
}

// cuTensorMapEncodeTiled through the runtime (the library links no libcuda).
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// [heads][rows][128] BF16 numbers (a BF16 cache's K or V with rows = Tp, or a
// part of the rebuilt rows): boxes of 128 rows x 64 elements, 128-byte swizzled;
// rows past the last read as zeros.
bool make_map(CUtensorMap *map, const void *base, long long rows, long long heads) {
    const EncodeFn fn = encode_fn();
    const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)rows, (cuuint64_t)heads};
    const cuuint64_t strides[2] = {kHeadDim * 2, (cuuint64_t)rows * kHeadDim * 2};
    const cuuint32_t box[3] = {64, kTileT, 1}, step[3] = {1, 1, 1};
    return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base),
                    dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch that may begin while the one before it on the stream still runs.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*f)(P...), dim3 grid, int threads, int smem, bool overlap, cudaStream_t st, A... args) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = overlap ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&lc, f, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int QT, int PP, int VP, bool RB>
cudaError_t launch_t(const Maps &m, const Bf16Args &a, cudaStream_t st) {
    static bool done[kMaxDevices];
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(prefill_bf16_kernel<QT, PP, VP, RB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Cfg<QT>::SMEM);
    });
    if (e != cudaSuccess) return e;
    return launch_overlapped(prefill_bf16_kernel<QT, PP, VP, RB>, dim3(a.S, a.heads, a.B * a.nqb), Cfg<QT>::THREADS,
                             Cfg<QT>::SMEM, RB, st, m, a);
}
cudaError_t launch_plain(int qt, const Maps &m, const Bf16Args &a, cudaStream_t st) {
    if (qt == 1) return a.out16 ? launch_t<1, 1, 1, false>(m, a, st) : launch_t<1, 2, 1, false>(m, a, st);
    return a.out16 ? launch_t<2, 1, 1, false>(m, a, st) : launch_t<2, 2, 1, false>(m, a, st);
}
cudaError_t launch_rebuilt(int qt, const Maps &m, const Bf16Args &a, cudaStream_t st) {
    if (qt == 1) return a.out16 ? launch_t<1, 2, 1, true>(m, a, st) : launch_t<1, 2, 2, true>(m, a, st);
    return a.out16 ? launch_t<2, 2, 1, true>(m, a, st) : launch_t<2, 2, 2, true>(m, a, st);
}

// How a call is cut: QT row tiles per CTA and S splits.  The time of the launch
// is estimated in the time of one token tile of one row tile (about 1.1 us): a
// CTA takes its tiles (two row tiles at once cost 1.7: 3700 against 2160 cycles)
// and a fixed part of three (set-up, output).  If the CTAs do not fit the SMs at
// once, it is their total over the SMs and what the uneven end leaves idle:
// little where they differ in length, as the longest start first, and up to the
// last, partly filled round where they do not.  Splits add a launch (four) and
// their partials' way through memory (3.3 MB in that time): for a causal chunk
// of 4096 tokens of 8 heads, 86 us with two splits and 51 with one.
struct Cut {
    int qt, S;
};
Cut choose_cut(const PrefillArgs &a, int sms) {
    Cut best = {1, 1};
    double best_cost = -1;
    const int nq = a.n * a.G;
    for (int qt = 1; qt <= (nq > kTileR ? 2 : 1); qt++) {
        const int rows = kTileR * qt, nqb = (nq + rows - 1) / rows;
        long total = 0;   // tiles of all row blocks of a kv head
        int most = 1, least = 1 << 30;
        for (int b = 0; b < a.B; b++)
            for (int r0 = 0; r0 < nq; r0 += rows) {
                const int t = Runs(a.seqT.v[b] + a.n_tail, a.n, r0 / a.G, (std::min(r0 + rows, nq) - 1) / a.G, a.window, a.sinks).tiles;
                total += t;
                most = std::max(most, t);
                least = std::min(least, t);
            }
        const double tile = qt == 2 ? 1.7 : 1.0, units = (double)a.B * a.H * nqb, same = (double)least / most;
        for (int S = 1; S <= std::min(most, kMaxSplits); S++) {
            const double fixed = 3, ctas = units * S;
            const double longest = (most + S - 1) / S * tile + fixed;
            const double mean = (double)total * a.H * tile / ctas + fixed;
            double cost = longest;
            if (ctas > sms) {
                const double rounds = ctas / sms;
                cost = std::max(cost, rounds * mean + (same * (std::ceil(rounds) - rounds) + (1 - same) * 0.25) * mean);
            }
            if (S > 1) cost += 4 + (double)a.B * nq * a.H * S * (2 * kPartialStride * sizeof(float)) / 3.3e6;
            if (best_cost < 0 || cost < best_cost) {
                best_cost = cost;
                best = Cut{qt, S};
            }
        }
    }
    return best;
}

}  // namespace

void prefill_bf16_plan(PrefillArgs *a, int sms) {
    const Cut cut = choose_cut(*a, sms);
    a->row_tiles = cut.qt;
    a->S = cut.S;
    a->nqb = (a->n * a->G + kTileR * cut.qt - 1) / (kTileR * cut.qt);
}

static Bf16Args bf16_args(const PrefillArgs &p, const int *nonfinite) {
    Bf16Args a;
    a.q = p.q;
    a.partials = p.partials;
    a.out = p.out;
    a.out16 = p.out16;
    a.err = p.err;
    a.nonfinite = nonfinite;
    a.seqT = p.seqT;
    a.B = p.B;
    a.H = p.H;
    a.Hq = p.Hq;
    a.G = p.G;
    a.n = p.n;
    a.n_tail = p.n_tail;
    a.S = p.S;
    a.nqb = p.nqb;
    a.window = p.window;
    a.sinks = p.sinks;
    a.scale_log2 = p.scale_log2;
    a.h0 = 0;
    a.heads = p.H;
    return a;
}

cudaError_t launch_prefill_bf16(const PrefillArgs &p, const uint16_t *k, const uint16_t *v, const int *nonfinite,
                                cudaStream_t st) {
    Maps m;
    std::memset(&m, 0, sizeof(m));
    const long long heads = (long long)p.B * p.H;
    if (!make_map(&m.k, k, p.Tp, heads) || !make_map(&m.v, v, p.Tp, heads)) return cudaErrorInvalidValue;
    return launch_plain(p.row_tiles, m, bf16_args(p, nonfinite), st);
}

cudaError_t launch_prefill_rebuilt(const PrefillArgs &p, const ReadArgs &r, cudaStream_t st) {
    Maps m;
    std::memset(&m, 0, sizeof(m));
    const long long heads = (long long)p.B * r.H;
    if (!make_map(&m.k, r.out[0], r.pair_stride, heads) || !make_map(&m.v, r.out[1], r.pair_stride, heads) ||
        !make_map(&m.k_lo, r.out_lo[0], r.pair_stride, heads) ||
        (r.out_lo[1] && !make_map(&m.v_lo, r.out_lo[1], r.pair_stride, heads)))
        return cudaErrorInvalidValue;
    Bf16Args a = bf16_args(p, r.nonfinite);
    a.h0 = r.h0;
    a.heads = r.H;
    return launch_rebuilt(p.row_tiles, m, a, st);
}

cudaError_t launch_merge_rows(const PrefillArgs &p, cudaStream_t st) {
    const long long rows = (long long)p.B * p.n * p.Hq;
    if ((rows + 3) / 4 > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    return launch_overlapped(merge_rows_kernel, dim3((unsigned)((rows + 3) / 4)), 128, 0, true, st, bf16_args(p, nullptr), rows);
}

}  // namespace rq
