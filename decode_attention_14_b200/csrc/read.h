// read.h -- launch interface of reading the cache back (rq_cache_read).  Not
// part of the public ABI.
#pragma once

#include "rq_internal.h"

namespace rq {

// Tokens [t0, t0 + n) of [committed tokens, tail tokens] of every sequence as
// K and V rows; rows at and past a sequence's end are not written.
struct ReadArgs {
    // anchor streams (kv 0 = K, 1 = V), and the residual streams of the first
    // of the nr records the loop's reconstruction reads after it (record k of
    // the chain lies k * resid_stride bytes further on)
    const uint8_t *a_codes[2], *a_meta[2];
    const uint8_t *r_codes[2], *r_meta[2], *r_coef[2];
    size_t resid_stride;
    int nr;
    const uint16_t *bf[2];             // BF16 format: [B][H][Tp][d] (the compressed streams are null then)
    const uint16_t *tail[2];           // [B][tail_cap][H][d] BF16, or null
    void *out[2];                      // element (b, i, h, e) at b * sb + i * st + h * sh + e
    long long sb, st, sh;              // strides in elements
    int out_type;                      // rq_out_type
    SeqLens seqT;                      // committed tokens of each sequence
    Pages pg;
    int B, H, t0, n, n_tail, tail_cap, Tp;
    int sms;                           // of the device
    int tiles;                         // 16-token tiles per warp (set by the launches)
    int g;
    int rotate;
    uint32_t sigma[4];
    // launch_rebuild: rows as pairs of BF16 numbers, the high ones in `out`
    // [B * H][pair_stride][d], the low ones in `out_lo` (null: left out); pair_rows rows (a multiple of 16) of every sequence are written,
    // zeros past its rebuilt ones; n, n_tail, window and sinks are the attention
    // call's.  *nonfinite is set to 1 when a V value is not finite.  The kv heads
    // are [h0, h0 + H) of H_all.
    uint16_t *out_lo[2];
    int h0, H_all;
    long long pair_stride;
    int pair_rows;
    int window, sinks;
    int *nonfinite;
};

// The positions that n new tokens of a windowed call see between them, of a
// sequence of `end` tokens: the sinks (rows 0 .. sink_pad - 1 of the workspace,
// whole tiles of 16), then positions w_base .. end - 1.
struct RebuiltRows {
    int sink_pad, w_base;
    // rows of the positions below p
    __host__ __device__ int rows(int p) const { return p <= sink_pad ? p : sink_pad + (p > w_base ? p - w_base : 0); }
    __host__ __device__ int position(int row) const { return row < sink_pad ? row : row - sink_pad + w_base; }
};
__host__ __device__ inline RebuiltRows rebuilt_rows(int end, int n, int window, int sinks) {
    const long long first = (long long)end - n + 1 - window;   // of the first row's window
    const int base = first <= 0 ? 0 : (int)(first / kTokTile * kTokTile);
    if (sinks > base) return RebuiltRows{0, 0};   // no gap between them
    return RebuiltRows{(sinks + 15) / 16 * 16, base};
}

cudaError_t launch_rebuild(const ReadArgs &a, int ba, int br, cudaStream_t st);
cudaError_t launch_read(const ReadArgs &a, int ba, int br, cudaStream_t st);

}  // namespace rq
