// read.cuh -- reading the cache back: tokens of one (layer, loop) rebuilt from
// their records as K and V rows (the inverse of append.cu; ai4snews summary,
// paragraph 3: the shared-anchor reconstruction k = s a + R^T y, two reads).
//
// Mathematics.  x = sc code + mn per quantization group (the anchor), then per
// residual record x <- s x + R^T y, y = sc_r code_r + mn_r, with
//   R^T y = diag(sigma) H_128 y / sqrt(128),   H_128 = H_8 (x) H_16
// (Sylvester order).  A 16-element segment g of y has one scale and one
// minimum, and H_16 maps a constant to 16 times that constant in element 0:
//   H_16 y_g = sc_g (H_16 c_g) + 16 mn_g e_0.
// H_16 c_g are small integers: one tensor-core step (mma.sync m16n8k16, BF16
// codes, +-1 matrix, fp32 accumulators) gives it exactly for 16 records and 8
// elements.  H_8 over the segments then adds registers of one thread.
//
// Layout.  A warp takes 16 consecutive tokens at a time of one (K|V, sequence,
// kv head).  The columns of the +-1 matrix are permuted so that lane 4 r + q
// ends with elements 16 g + 4 q .. 16 g + 4 q + 3 of records r and r + 8 for
// every segment g: H_8 needs no exchange between lanes, and the four lanes of a
// record write whole 32-byte sectors.  The codes enter the tensor core as
// 128 + c (bits of a code beside 0x4300 are that BF16 number; 2-bit codes of
// odd elements as 128 + 4 c against +-1/4, which saves a shift); the biases come
// out in elements 0 and 1 and are taken off by the accumulators' initial
// values.  The rows (K dimension) are permuted so that two codes of a word 16
// bits apart are one operand register.
//
// Data movement.  Tiles of 16 tokens are aligned in the sequence, so the 16
// records of a tile lie behind one another (a block holds 128 or 256 tokens, a
// contiguous sequence is padded to 64).  Each warp runs through its records (of
// each tile the residual records, last of the chain first, then the anchor)
// with a ring of kSlots slots in shared memory, filled ahead by 16-byte
// asynchronous copies; rows are padded by 16 bytes so that no read of eight
// records conflicts.
//
// What bounds it: instructions, and latency that 16 warps an SM do not hide.  A
// tile of 16 records with one residual takes about 1100 warp instructions, and an
// issue slot is used in 66% of the cycles: 4 x 16 heads x 8192 tokens (residual, BF16 out, 405 MB read and
// written) 98.8 us = 4.1 TB/s, 63% of a plain copy; an anchor group alone to
// fp32, 13 000 paged tokens x 8 heads (123 MB), 21.1 us = 5.8 TB/s, 89%.
//
// fp32 throughout (the codes, FP8 scales and minima are exact in it; two
// elements per instruction), rounded once to the output's type.
//
// kOutPair (rebuild.cu) writes the rows that a chunk of new tokens attends to,
// the tail's among them, into a workspace for the tensor-core attention of
// prefill_bf16.cu: a value as the BF16 number next to it and a second one for
// what that leaves (2^-18 of the value is lost; V for BF16 output: the first
// alone, 2^-9); sequence by sequence the rows that rebuilt_rows() names.
#pragma once

#include "common.cuh"
#include "read.h"
#include "sync.cuh"

namespace rq {
namespace {

constexpr float kRsqrtD = 0.088388347648318440f;   // 1 / sqrt(128)
constexpr int kWarps = 4;                          // warps per CTA
constexpr int kCtas = 4;                           // CTAs per SM
static_assert(32 * kWarps == kHeadDim, "a thread per sign");
constexpr int kRecs = 16;                          // records of a tile
constexpr int kTiles = 4;                          // tiles per warp of a large call
constexpr int kSlots = 4;                          // ring slots per warp: kSlots - 1 steps in flight

// d = a b + c on the tensor cores: a 16 x 16, b 16 x 8, BF16, fp32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2],
                                         const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(c[0]), "f"(c[1]), "f"(c[2]),
          "f"(c[3]));
}

// Tiles per warp of a launch of `tiles` in all: those of one warp share its
// set-up and overlap, as long as four rounds of the 16 warps an SM holds remain
// to even out the end: at 8k b4 (residual) 99 / 104 / 119 us with 4 / 2 / 1, at
// 15 000 tiles 24.4 / 21.1 / 21.2 us.
inline int warp_tiles(long long tiles, int sms) {
    int per = kTiles;
    while (per > 1 && tiles < (long long)sms * 16 * 4 * per) per /= 2;
    return per;
}

constexpr int kOutPair = 2;   // beside the rq_out_type values

template <int OUT>
__device__ __forceinline__ void store4(void *out, long long at, const float x[4]) {
    if (OUT == RQ_OUT_BF16) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + at) = make_float4(x[0], x[1], x[2], x[3]);
    }
}

// One row of BF16 values (a tail token, or a token of a BF16 cache) by a warp.
template <int OUT>
__device__ __forceinline__ void copy_row(void *out, long long at, const uint16_t *row, int lane) {
    const uint2 w = *reinterpret_cast<const uint2 *>(row + 4 * lane);
    const float x[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                        __uint_as_float(w.y & 0xFFFF0000u)};
    store4<OUT>(out, at + 4 * lane, x);
}

// What a warp reads: tiles [tile0, tile0 + tiles) of 16 tokens of one
// (kv, b, h), of those that hold the call's tokens.
struct Span {
    int kv, b, h, tile0, tiles;
};
__host__ __device__ inline int tiles_of(int t0, int n) { return (t0 + n - 1) / kRecs - t0 / kRecs + 1; }
__device__ __forceinline__ bool span_of(const ReadArgs &a, Span &s) {
    const int nt = tiles_of(a.t0, a.n), per = a.tiles * kWarps, chunks = (nt + per - 1) / per;
    unsigned u = blockIdx.x / (unsigned)chunks;
    const int first = ((blockIdx.x - u * chunks) * kWarps + (threadIdx.x >> 5)) * a.tiles;
    s.tile0 = a.t0 / kRecs + first;
    s.tiles = min(a.tiles, nt - first);
    s.h = (int)(u % a.H);
    u /= a.H;
    s.b = (int)(u % a.B);
    s.kv = (int)(u / a.B);
    return s.tiles > 0;   // uniform per warp
}
// The same for kOutPair: tile0 counts the 16-row tiles of the sequence's
// rebuilt rows.
__device__ __forceinline__ bool pair_span_of(const ReadArgs &a, Span &s) {
    const int nt = a.pair_rows / kRecs, per = a.tiles * kWarps, chunks = (nt + per - 1) / per;
    unsigned u = blockIdx.x / (unsigned)chunks;
    s.tile0 = ((blockIdx.x - u * chunks) * kWarps + (threadIdx.x >> 5)) * a.tiles;
    s.tiles = min(a.tiles, nt - s.tile0);
    s.h = (int)(u % a.H);
    u /= a.H;
    s.b = (int)(u % a.B);
    s.kv = (int)(u / a.B);
    return s.tiles > 0;
}
// Where token t (t0 <= t < t0 + n) of the span's sequence goes.
__device__ __forceinline__ long long row_at(const ReadArgs &a, const Span &s, int t) {
    return s.b * a.sb + (t - a.t0) * a.st + s.h * a.sh;
}

__device__ __forceinline__ void async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void async8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A ring slot: codes of 16 records (rows padded by 16 bytes), then their meta.
template <int BA, int BR>
struct Slot {
    static constexpr int pitch(int bits) { return 16 * bits + 16; }
    static constexpr int META = kRecs * pitch(BA > BR ? BA : BR);
    static constexpr int BYTES = META + kRecs * 16;
};

// Codes and meta of the 16 records from row rec on into a slot.
template <int BITS, int GS>
__device__ __forceinline__ void fetch(uint32_t slot, int meta_off, const uint8_t *codes, const uint8_t *meta,
                                      size_t rec, int lane) {
    constexpr int MR = 2 * (kHeadDim / GS);
    const uint8_t *src = codes + rec * (16 * BITS) + lane * 16;
#pragma unroll
    for (int i = 0; i < BITS / 2; i++) {   // 32 chunks a round, BITS chunks a record
        const int ch = i * 32 + lane;
        async16(slot + (ch / BITS) * (16 * BITS + 16) + (ch % BITS) * 16, src + i * 512);
    }
    if (lane < kRecs) {
        if (MR == 16) async16(slot + meta_off + lane * 16, meta + rec * MR + lane * 16);
        else async8(slot + meta_off + lane * 16, meta + rec * MR + lane * 8);
    }
}

// (scale, minimum) of segment sg of a record's meta bytes.
template <int GS>
__device__ __forceinline__ float2 seg_meta(const uint4 &m, int sg) {
    const int grp = sg * 16 / GS;
    const uint32_t w = (grp >> 1) == 0 ? m.x : (grp >> 1) == 1 ? m.y : (grp >> 1) == 2 ? m.z : m.w;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((w >> (16 * (grp & 1))) & 0xFFFFu), __NV_E4M3);
    return __half22float2(__half2(h));
}

// The lane's four values sc c + mn of segment sg of a record (elements
// 16 sg + 4 q ..).  A code's bits at position p of the low mantissa beside the
// exponent of 2^(23 - p) are the float 2^(23 - p) + c, exactly.
template <int BITS>
__device__ __forceinline__ void expand4(const uint8_t *row, int sg, int q, float2 sm, F2 (&x)[2]) {
    const uint32_t w = BITS == 4 ? (uint32_t)reinterpret_cast<const uint16_t *>(row)[4 * sg + q] : (uint32_t)row[4 * sg + q];
    float f[4], e[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const uint32_t ex = (uint32_t)(127 + 23 - k * BITS) << 23;
        f[k] = __uint_as_float((w & ((uint32_t)((1 << BITS) - 1) << (k * BITS))) | ex);
        e[k] = -__uint_as_float(ex);
    }
    const F2 sc = pack2(sm.x, sm.x), mn = pack2(sm.y, sm.y);
    x[0] = fma2(sc, add2(pack2(f[0], f[1]), pack2(e[0], e[1])), mn);
    x[1] = fma2(sc, add2(pack2(f[2], f[3]), pack2(e[2], e[3])), mn);
}

// kOutPair: row i of the span's sequence in the workspace.
__device__ __forceinline__ long long pair_at(const ReadArgs &a, const Span &s, int i) {
    return (((long long)s.b * a.H + s.h) * a.pair_stride + i) * kHeadDim;
}
// Writes four values; nonzero if one of them is a V that is not finite.
__device__ __forceinline__ uint32_t store_pair(const ReadArgs &a, int kv, long long at, const float (&x)[4]) {
    const __nv_bfloat162 h0 = __floats2bfloat162_rn(x[0], x[1]), h1 = __floats2bfloat162_rn(x[2], x[3]);
    const uint2 hi = make_uint2(*reinterpret_cast<const uint32_t *>(&h0), *reinterpret_cast<const uint32_t *>(&h1));
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out[kv]) + at) = hi;
    // exponents all ones
    const uint32_t bad = (((hi.x & 0x7F807F80u) + 0x00800080u) | ((hi.y & 0x7F807F80u) + 0x00800080u)) & 0x80008000u;
    if (a.out_lo[kv]) {   // uniform
        const __nv_bfloat162 l0 =
            __floats2bfloat162_rn(x[0] - __uint_as_float(hi.x << 16), x[1] - __uint_as_float(hi.x & 0xFFFF0000u));
        const __nv_bfloat162 l1 =
            __floats2bfloat162_rn(x[2] - __uint_as_float(hi.y << 16), x[3] - __uint_as_float(hi.y & 0xFFFF0000u));
        // (beside an infinity nothing: it would be an infinity less itself)
        *reinterpret_cast<uint2 *>(a.out_lo[kv] + at) =
            bad ? make_uint2(0u, 0u) : make_uint2(*reinterpret_cast<const uint32_t *>(&l0), *reinterpret_cast<const uint32_t *>(&l1));
    }
    return kv == 0 ? 0u : bad;
}
// The span's rows beside those with records: the tail's tokens, and zero rows
// past the sequence's end (a reader's tile of 128 rows ends there).
__device__ __forceinline__ void pair_rest(const ReadArgs &a, const Span &s, const RebuiltRows &rb, int T, int lane) {
    constexpr int kFly = 8;   // rows in flight
    const int end = min((s.tile0 + s.tiles) * kRecs, a.pair_rows);
    const uint16_t *base =
        a.n_tail > 0 ? a.tail[s.kv] + ((size_t)s.b * a.tail_cap * a.H_all + a.h0 + s.h) * kHeadDim + 4 * lane : nullptr;
    uint32_t bad = 0;
    for (int i0 = max(s.tile0 * kRecs, rb.rows(T)); i0 < end; i0 += kFly) {
        uint2 w[kFly];
#pragma unroll
        for (int u = 0; u < kFly; u++) {
            const int j = rb.position(i0 + u) - T;
            w[u] = j < a.n_tail && i0 + u < end
                       ? __ldcg(reinterpret_cast<const uint2 *>(base + (size_t)j * a.H_all * kHeadDim))
                       : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < kFly; u++) {
            const float x[4] = {__uint_as_float(w[u].x << 16), __uint_as_float(w[u].x & 0xFFFF0000u),
                                __uint_as_float(w[u].y << 16), __uint_as_float(w[u].y & 0xFFFF0000u)};
            if (i0 + u < end) bad |= store_pair(a, s.kv, pair_at(a, s, i0 + u) + 4 * lane, x);
        }
    }
    if (s.kv == 1 && bad) *a.nonfinite = 1;
}

// NR: residual records read, 0 or 1 (the shared reference), or 2 for any
// number (a.nr, the chained reference).
template <int BA, int BR, int GS, int NR, bool ROT, int OUT>
__global__ void __launch_bounds__(32 * kWarps, NR == 2 ? 3 : kCtas) read_rq_kernel(const ReadArgs a) {
    using S = Slot<BA, BR>;
    const int nr = NR < 2 ? NR : a.nr;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float s_sign[kHeadDim];   // sigma / sqrt(d)
    const int lane = threadIdx.x & 31, q = lane & 3;
    if (ROT) {
        s_sign[threadIdx.x] = sigma_neg(a.sigma, threadIdx.x) ? -kRsqrtD : kRsqrtD;
        __syncthreads();
    }
    Span sp;
    if (!(OUT == kOutPair ? pair_span_of(a, sp) : span_of(a, sp))) return;
    const int T = a.seqT.v[sp.b];
    // the span's tokens: [lo, hi) of the call, of them [lo, mid) committed
    int lo, mid;
    RebuiltRows rb = {0, 0};
    if (OUT == kOutPair) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the attention may set itself up meanwhile
        rb = rebuilt_rows(T + a.n_tail, a.n, a.window, a.sinks);
        pair_rest(a, sp, rb, T, lane);
        lo = 0;
        mid = T;
    } else {
        lo = max(a.t0, sp.tile0 * kRecs);
        const int hi = min(min(a.t0 + a.n, (sp.tile0 + sp.tiles) * kRecs), T + a.n_tail);
        mid = min(hi, T);
        // tail tokens, a row at a time
        for (int t = max(lo, mid); t < hi; t++) {
            const uint16_t *row = a.tail[sp.kv] + (((size_t)sp.b * a.tail_cap + (t - T)) * a.H + sp.h) * kHeadDim;
            copy_row<OUT>(a.out[sp.kv], row_at(a, sp, t), row, lane);
        }
        if (mid <= lo) return;
    }
    // first token of tile i of the span
    auto tile_tok = [&](int i) { return OUT == kOutPair ? rb.position((sp.tile0 + i) * kRecs) : (sp.tile0 + i) * kRecs; };

    uint8_t *ring = smem + (threadIdx.x >> 5) * (kSlots * S::BYTES);
    const uint32_t ring_s = smem_u32(ring);
    const int tiles = OUT == kOutPair ? min(sp.tiles, (rb.rows(T) + kRecs - 1) / kRecs - sp.tile0)
                                      : (mid - 1) / kRecs - sp.tile0 + 1;
    const int nstep = tiles * (nr + 1);
    // the step being fetched: tile ft, record fk of the chain (-1: the anchor),
    // slot fs; its first row and, for residual records, the coefficients (lane
    // r keeps record r's until the step is consumed)
    int ft = 0, fk = nr - 1, fs = 0, fstep = 0;
    size_t frec = 0;
    uint32_t coef[kSlots];
    auto fetch_next = [&](uint32_t &cf) {
        if (fstep < nstep) {
            if (fk == nr - 1)   // a new tile
                frec = OUT == kOutPair ? rec_row(a.pg, a.H_all, sp.b, a.h0 + sp.h, tile_tok(ft))
                                       : rec_row(a.pg, a.H, sp.b, sp.h, tile_tok(ft));
            const uint32_t slot = ring_s + fs * S::BYTES;
            if (fk >= 0) {
                const size_t o = fk * a.resid_stride;
                fetch<BR, GS>(slot, S::META, a.r_codes[sp.kv] + o, a.r_meta[sp.kv] + o, frec, lane);
                cf = __ldg(reinterpret_cast<const uint16_t *>(a.r_coef[sp.kv] + o) + frec + (lane & 15));
                fk--;
            } else {
                fetch<BA, GS>(slot, S::META, a.a_codes[sp.kv], a.a_meta[sp.kv], frec, lane);
                fk = nr - 1;
                ft++;
            }
            fstep++;
            fs = fs + 1 == kSlots ? 0 : fs + 1;
        }
        async_commit();
    };
    // coefficients rotate through registers with the slots: coef[0] is the
    // step's being consumed
#pragma unroll
    for (int i = 0; i < kSlots - 1; i++) {
        coef[i] = 0;
        fetch_next(coef[i]);
    }

    // +-1 operand: column lane / 4 of output half nt is element
    // 4 (col / 2) + 2 nt + col % 2; row slots 2 q, 2 q + 1, 2 q + 8, 2 q + 9
    // are elements 2 q, 2 q + 8, 2 q + 1, 2 q + 9
    uint32_t hm[2][2];
    float init[2][4];
    if (ROT) {
        const int col = lane >> 2;
#pragma unroll
        for (int nt = 0; nt < 2; nt++) {
            const int e = 4 * (col >> 1) + 2 * nt + (col & 1);
#pragma unroll
            for (int s = 0; s < 2; s++) {
                const uint32_t one = BR == 2 && s == 1 ? 0x3E80u : 0x3F80u;   // 1/4 or 1
                const uint32_t x = (__popc((2 * q + s) & e) & 1) ? one | 0x8000u : one;
                const uint32_t y = (__popc((2 * q + s + 8) & e) & 1) ? one | 0x8000u : one;
                hm[nt][s] = x | (y << 16);
            }
        }
        // biases: 8 rows of 128 and 8 of 128 / 4 (or 128), summed in element
        // 0 and, even rows against odd, in element 1
        const float odd = BR == 2 ? 32.f : 128.f;
#pragma unroll
        for (int k = 0; k < 4; k++) {
            init[0][k] = q == 0 ? ((k & 1) ? -8.f * (128.f - odd) : -8.f * (128.f + odd)) : 0.f;
            init[1][k] = 0.f;
        }
    }
    const float e0 = q == 0 ? 16.f : 0.f;   // the lanes that hold element 0 of every segment
    const F2 neg1 = pack2(-1.f, -1.f);

    // z = sum_k c_k y_k over the residual records, c_k the product of the
    // coefficients of the records after k (1 for the last): the chain
    // x <- s_k x + R^T y_k unrolled, so that the anchor gets the product of
    // all of them and R^T is applied once.  Under ROT z holds H_16 z_g.
    int cs = 0;   // slot consumed
    uint32_t bad = 0;   // kOutPair: a value is not finite
#pragma unroll 1
    for (int tile = 0; tile < tiles; tile++) {
        F2 z[2][8][2];
        float c[2] = {1.f, 1.f};
        if (nr > 0) {
#pragma unroll 1
            for (int k = nr - 1; k >= 0; k--) {
                async_wait<kSlots - 2>();
                __syncwarp();
                const uint8_t *st = ring + cs * S::BYTES;
                uint4 m[2];
                const uint8_t *cp[2];
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    const int r = (lane >> 2) + 8 * u;
                    m[u] = *reinterpret_cast<const uint4 *>(st + S::META + 16 * r);
                    cp[u] = st + r * S::pitch(BR);
                }
                const bool first = NR < 2 || k == nr - 1;
#pragma unroll
                for (int sg = 0; sg < 8; sg++) {
                    F2 y[2][2];
                    if (ROT) {
                        uint32_t av[4];
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            if (BR == 2) {   // element k at bits 2 k of the segment's word
                                const uint32_t v = reinterpret_cast<const uint32_t *>(cp[u])[sg] >> (4 * q);
                                av[u] = (v & 0x00030003u) | 0x43004300u;              // elements 2q, 2q + 8
                                av[2 + u] = (v & 0x000C000Cu) | 0x43004300u;          // 2q + 1, 2q + 9, times 4
                            } else {         // elements 0-7 and 8-15 in two words: byte q of each, into bytes 0, 2
                                const uint2 w = reinterpret_cast<const uint2 *>(cp[u])[sg];
                                const uint32_t v = __byte_perm(w.x, w.y, (uint32_t)(q | ((4 + q) << 8)));
                                av[u] = (v & 0x000F000Fu) | 0x43004300u;
                                av[2 + u] = ((v >> 4) & 0x000F000Fu) | 0x43004300u;
                            }
                        }
                        float d0[4], d1[4];
                        mma16816(d0, av, hm[0], init[0]);
                        mma16816(d1, av, hm[1], init[1]);
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            const float2 sm = seg_meta<GS>(m[u], sg);
                            const F2 sc = pack2(sm.x, sm.x);
                            y[u][0] = fma2(sc, pack2(d0[2 * u], d0[2 * u + 1]), pack2(e0 * sm.y, 0.f));
                            y[u][1] = mul2(sc, pack2(d1[2 * u], d1[2 * u + 1]));
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < 2; u++) expand4<BR>(cp[u], sg, q, seg_meta<GS>(m[u], sg), y[u]);
                    }
#pragma unroll
                    for (int u = 0; u < 2; u++)
#pragma unroll
                        for (int e = 0; e < 2; e++)
                            z[u][sg][e] = first ? y[u][e] : fma2(pack2(c[u], c[u]), y[u][e], z[u][sg][e]);
                }
#pragma unroll
                for (int u = 0; u < 2; u++)
                    c[u] *= bf16_to_f32((uint16_t)__shfl_sync(0xffffffffu, coef[0], (lane >> 2) + 8 * u));
                __syncwarp();
#pragma unroll
                for (int i = 0; i + 1 < kSlots - 1; i++) coef[i] = coef[i + 1];
                fetch_next(coef[kSlots - 2]);
                cs = cs + 1 == kSlots ? 0 : cs + 1;
            }
            if (ROT) {   // H_8 over the segments
#pragma unroll
                for (int g = 1; g < 8; g <<= 1)
#pragma unroll
                    for (int sg = 0; sg < 8; sg++)
                        if ((sg & g) == 0) {
#pragma unroll
                            for (int u = 0; u < 2; u++)
#pragma unroll
                                for (int e = 0; e < 2; e++) {
                                    const F2 p = z[u][sg][e], r = z[u][sg + g][e];
                                    z[u][sg][e] = add2(p, r);
                                    z[u][sg + g][e] = fma2(r, neg1, p);
                                }
                        }
            }
        }
        // x = c a + diag(sigma) z / sqrt(d)
        async_wait<kSlots - 2>();
        __syncwarp();
        const uint8_t *st = ring + cs * S::BYTES;
        uint4 m[2];
        long long at[2];
        bool in[2];
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const int r = (lane >> 2) + 8 * u, t = tile_tok(tile) + r;
            m[u] = *reinterpret_cast<const uint4 *>(st + S::META + 16 * r);
            at[u] = (OUT == kOutPair ? pair_at(a, sp, (sp.tile0 + tile) * kRecs + r) : row_at(a, sp, t)) + 4 * q;
            in[u] = t >= lo && t < mid;
        }
#pragma unroll
        for (int sg = 0; sg < 8; sg++) {
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (ROT) f = *reinterpret_cast<const float4 *>(s_sign + 16 * sg + 4 * q);
#pragma unroll
            for (int u = 0; u < 2; u++) {
                F2 x[2];
                expand4<BA>(st + ((lane >> 2) + 8 * u) * S::pitch(BA), sg, q, seg_meta<GS>(m[u], sg), x);
                if (nr > 0) {
                    const F2 cc = pack2(c[u], c[u]);
                    x[0] = fma2(cc, x[0], ROT ? mul2(z[u][sg][0], pack2(f.x, f.y)) : z[u][sg][0]);
                    x[1] = fma2(cc, x[1], ROT ? mul2(z[u][sg][1], pack2(f.z, f.w)) : z[u][sg][1]);
                }
                float o[4];
                unpack2(x[0], o[0], o[1]);
                unpack2(x[1], o[2], o[3]);
                if (OUT == kOutPair) {
                    if (in[u]) bad |= store_pair(a, sp.kv, at[u] + 16 * sg, o);
                } else if (in[u]) {
                    store4<OUT>(a.out[sp.kv], at[u] + 16 * sg, o);
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i + 1 < kSlots - 1; i++) coef[i] = coef[i + 1];
        fetch_next(coef[kSlots - 2]);
        cs = cs + 1 == kSlots ? 0 : cs + 1;
    }
    async_wait<0>();
    if (OUT == kOutPair && sp.kv == 1 && bad) *a.nonfinite = 1;
}

template <int BA, int BR, int GS, int NR, bool ROT, int OUT>
cudaError_t launch_t(const ReadArgs &a, unsigned blocks, cudaStream_t st) {
    constexpr int smem = kWarps * kSlots * Slot<BA, BR>::BYTES;
    static_assert(smem <= 48 * 1024, "no opt-in needed");
    read_rq_kernel<BA, BR, GS, NR, ROT, OUT><<<blocks, 32 * kWarps, smem, st>>>(a);
    return cudaGetLastError();
}
}  // namespace
}  // namespace rq
