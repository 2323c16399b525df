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
    int tiles;                         // 16-token tiles per warp (set by launch_read)
    int g;
    int rotate;
    uint32_t sigma[4];
};

cudaError_t launch_read(const ReadArgs &a, int ba, int br, cudaStream_t st);

}  // namespace rq
