// prefill.h -- launch interface of the multi-token (chunked-prefill) attention
// over the compressed cache.  Not part of the public ABI.
#pragma once

#include "rq_internal.h"

namespace rq {

constexpr int kPrefillTile = 32;   // committed tokens per step of a CTA

// Causal attention of the n most recent tokens of every sequence: query row
// (i, hq) of sequence b (i < n) sees the first T_b + n_tail - n + 1 + i tokens
// of [committed tokens of the group, then the loop's tail tokens].
struct PrefillArgs {
    // anchor streams (kv 0 = K, 1 = V); residual streams null for an anchor loop
    const uint8_t *a_codes[2], *a_meta[2];
    const uint8_t *r_codes[2], *r_meta[2];
    const uint16_t *r_coef[2];
    const uint16_t *q;                 // [B][n][Hq][d] bf16
    const uint16_t *tail_k, *tail_v;   // [B][tail_cap][H][d] bf16, or null
    float *partials;                   // [B][n][Hq][S][kPartialStride]
    float *out;                        // [B][n][Hq][d] fp32
    SeqLens seqT;                      // committed tokens of each sequence
    Pages pg;                          // token -> record row (contiguous: row bh * Tp + t)
    int B, H, Hq, G, n, n_tail, tail_cap, Tp, S;
    int nqb;                           // blocks of 64 query rows per kv head
    int g;                             // quantization group size
    float scale_log2;                  // softmax_scale * log2(e)
    int rotate;
    uint32_t sigma[4];
    int *err;                          // device error word (bounded waits that gave up)
    int *counters;                     // [B][H][nqb] split arrivals (zero between calls): the last
                                       // split of a row block merges the partials; null: the
                                       // combine kernel merges them
    int tail_in_kernel;                // the attention kernel (last split) takes the tail tokens
    int window, sinks;                 // windowed calls: the query at position p sees (p - window, p] and [0, sinks)
    uint16_t *out16;                   // the output in BF16 instead of `out`, or null
    int row_tiles;                     // of 128 rows per CTA, 1 or 2 (windowed calls)
};

// What the rows of query tokens [i0, i1] (of the n last) of a windowed call see
// of a sequence of `end` tokens: positions [0, sink_end) and [w_tile, lim) (the
// first row's window begins at w0, in the 64 positions from w_tile on).
struct BlockRuns {
    int sink_end, w_tile, w0, lim;
};
__host__ __device__ inline BlockRuns block_runs(int end, int n, int i0, int i1, int window, int sinks) {
    BlockRuns r;
    const long long first = (long long)end - n + i0 + 1 - window;   // of row i0's window
    r.lim = end - n + i1 + 1;
    r.w0 = first < 0 ? 0 : (int)first;
    r.w_tile = r.w0 / kTokTile * kTokTile;
    r.sink_end = sinks < r.w_tile ? sinks : r.w_tile;
    return r;
}

// Sets a->nqb and the split count a->S over the committed tokens (T
// = the longest sequence); a->B, H, G and n must be set.
void prefill_plan(PrefillArgs *a, int T, int ba, int br, int sms);
cudaError_t launch_prefill(const PrefillArgs &a, int ba, int br, cudaStream_t st);

// Windowed attention of several new tokens (prefill_bf16.cu): over a BF16 cache,
// k, v [B * H][Tp][d]; or over the rows that launch_rebuild wrote as `r` says,
// for the kv heads [r.h0, r.h0 + r.H).  a->row_tiles, a->nqb and
// a->S are the plan's; record fields are unused.  With a->S > 1 launch_merge_rows follows.
struct ReadArgs;
void prefill_bf16_plan(PrefillArgs *a, int sms);
cudaError_t launch_prefill_bf16(const PrefillArgs &a, const uint16_t *k, const uint16_t *v, const int *nonfinite,
                                cudaStream_t st);
cudaError_t launch_prefill_rebuilt(const PrefillArgs &a, const ReadArgs &r, cudaStream_t st);
cudaError_t launch_merge_rows(const PrefillArgs &a, cudaStream_t st);

}  // namespace rq
