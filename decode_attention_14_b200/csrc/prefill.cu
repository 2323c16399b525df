// prefill.cu -- multi-token causal attention over the compressed cache
// (rq_prefill_attn): the instantiations of prefill.cuh without a window, the
// combine kernel for caches that hold nothing committed, and the split plans.
#include "prefill.cuh"

namespace rq {
namespace {

// One CTA per (q head, query token, sequence): the row's split partials,
// then the tail tokens it may see, 128 at a time: their logits (a warp per
// token, 4 elements per lane), the chunk's maximum, then o += sum 2^(z - M) v
// with thread tid owning element tid.
__global__ void __launch_bounds__(128) prefill_combine_kernel(const PrefillArgs a) {
    constexpr int kChunk = 128;
    __shared__ float s_z[kChunk];
    __shared__ float s_red[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hq = blockIdx.x, i = blockIdx.y, b = blockIdx.z;
    const int h = hq / a.G;
    const size_t row = ((size_t)b * a.n + i) * a.Hq + hq;
    // of [committed, tail] the row sees T_b + n_tail - n + 1 + i tokens: all
    // committed ones when the new tokens are in the tail
    const int nt = (a.tail_k && !a.tail_in_kernel) ? max(0, a.n_tail - a.n + 1 + i) : 0;
    const size_t tstride = (size_t)a.H * kHeadDim;
    const uint16_t *tk = a.tail_k ? a.tail_k + ((size_t)b * a.tail_cap * a.H + h) * kHeadDim : nullptr;
    const uint16_t *tv = a.tail_v ? a.tail_v + ((size_t)b * a.tail_cap * a.H + h) * kHeadDim : nullptr;
    float q4[4] = {0.f, 0.f, 0.f, 0.f};
    if (nt > 0) {
        const uint2 qr = *reinterpret_cast<const uint2 *>(a.q + row * kHeadDim + 4 * lane);
        q4[0] = bf16_to_f32(qr.x & 0xFFFFu) * a.scale_log2;
        q4[1] = bf16_to_f32(qr.x >> 16) * a.scale_log2;
        q4[2] = bf16_to_f32(qr.y & 0xFFFFu) * a.scale_log2;
        q4[3] = bf16_to_f32(qr.y >> 16) * a.scale_log2;
    }
    float M, l, o;
    merge_partials(a.partials + row * a.S * kPartialStride, a.S, tid, M, l, o);
    for (int c0 = 0; c0 < nt; c0 += kChunk) {
        const int cn = min(kChunk, nt - c0);
        // logits of the chunk (L2 loads: the tail rows may just have been written)
#pragma unroll 4
        for (int jj = warp; jj < cn; jj += 4) {
            const uint2 kr = __ldcg(reinterpret_cast<const uint2 *>(tk + (size_t)(c0 + jj) * tstride + 4 * lane));
            float z = q4[0] * bf16_to_f32(kr.x & 0xFFFFu);
            z = fmaf(q4[1], bf16_to_f32(kr.x >> 16), z);
            z = fmaf(q4[2], bf16_to_f32(kr.y & 0xFFFFu), z);
            z = fmaf(q4[3], bf16_to_f32(kr.y >> 16), z);
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) z += __shfl_xor_sync(0xffffffffu, z, m);
            if (lane == 0) s_z[jj] = z;
        }
        __syncthreads();
        float mc = tid < cn ? s_z[tid] : -CUDART_INF_F;
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, m));
        if (lane == 0) s_red[warp] = mc;
        __syncthreads();
        const float Mn = fmaxf(M, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
        const float c = exp2f(M - Mn);   // 0 while M = -inf
        l *= c;
        o *= c;
#pragma unroll 8
        for (int j = 0; j < cn; j++) {
            const float w = exp2f(s_z[j] - Mn);
            l += w;
            o = fmaf(w, bf16_to_f32(__ldcg(tv + (size_t)(c0 + j) * tstride + tid)), o);
        }
        M = Mn;
        __syncthreads();   // s_z and s_red are rewritten by the next chunk
    }
    a.out[row * kHeadDim + tid] = (l > 0.f) ? o / l : 0.f;
}

}  // namespace

// Row blocks of 64 query rows per kv head; splits: the count with the least
// wave-quantised work (waves x 64-token steps of the largest split, plus a
// fixed cost of RQ_PREFILL_STEP_OVERHEAD steps per CTA), one CTA per SM (the tiles take 193 KB of shared memory
// and the accumulators all 512 tensor-memory columns).
#ifndef RQ_PREFILL_STEP_OVERHEAD
#define RQ_PREFILL_STEP_OVERHEAD 3
#endif
static int splits_for(int nt, long units, int sms) {
    const long slots = (long)std::max(1, sms);
    long best = -1;
    int pick = 1;
    for (int S = 1; S <= std::min(nt, kMaxSplits); S++) {
        const long waves = (S * units + slots - 1) / slots;
        const long cost = waves * ((nt + S - 1) / S + RQ_PREFILL_STEP_OVERHEAD);
        if (best < 0 || cost < best) {
            best = cost;
            pick = S;
        }
    }
    return pick;
}

void prefill_plan(PrefillArgs *a, int T, int ba, int br, int sms) {
    (void)ba;
    (void)br;
    const int nq = a->n * a->G;
    a->nqb = (nq + kRows - 1) / kRows;
    a->S = 0;
    a->tail_in_kernel = 0;
    if (T <= 0) return;   // nothing committed: the combine kernel takes the tail
    a->tail_in_kernel = 1;
    a->S = splits_for((T + kTokTile - 1) / kTokTile, (long)a->B * a->H * a->nqb, sms);
}

void prefill_window_plan(PrefillArgs *a, int sms) {
    const int nq = a->n * a->G;
    a->nqb = (nq + kRows - 1) / kRows;
    a->tail_in_kernel = 1;
    // the most tokens a row block reads of a sequence: its rows' windows, the
    // sinks, a tile's padding on each run
    int nt = 1;
    for (int b = 0; b < a->B; b++) {
        const BlockRuns last = block_runs(a->seqT.v[b], a->n_tail, a->n, (nq - 1) / kRows * kRows / a->G, a->n - 1, a->window,
                                          a->sinks);
        const BlockRuns first = block_runs(a->seqT.v[b], a->n_tail, a->n, 0, std::min(a->n, (kRows - 1) / a->G + 1) - 1,
                                           a->window, a->sinks);
        nt = std::max(nt, (std::max(first.total(), last.total()) + kTokTile - 1) / kTokTile);
    }
    a->S = splits_for(nt, (long)a->B * a->H * a->nqb, sms);
}

cudaError_t launch_prefill(const PrefillArgs &a, int ba, int br, cudaStream_t st) {
    if (!((ba == 4 && br == 2) || (ba == 2 && br == 2) || (ba == 4 && br == 4))) return cudaErrorInvalidValue;
    if (a.g != 16 && a.g != 32) return cudaErrorInvalidValue;
    if (a.window > 0) return launch_prefill_window(a, ba, br, st);
    cudaError_t e = a.g == 16 ? launch_group<false, 16>(a, ba, br, st) : launch_group<false, 32>(a, ba, br, st);
    if (e != cudaSuccess) return e;
    if (a.S == 0) prefill_combine_kernel<<<dim3(a.Hq, a.n, a.B), 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace rq
