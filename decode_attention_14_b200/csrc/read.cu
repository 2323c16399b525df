// read.cu -- reading the cache back: tokens of one (layer, loop) rebuilt from
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
// Layout.  A warp takes 16 consecutive tokens of one (K|V, sequence, kv head).
// The columns of the +-1 matrix are permuted so that lane 4 r + q ends with
// elements 16 g + 4 q .. 16 g + 4 q + 3 of records r and r + 8 for every
// segment g: H_8 needs no exchange between lanes, and the four lanes of a
// record write whole 32-byte sectors.  The codes enter the tensor core as
// 128 + c (bits of a code beside 0x4300 are that BF16 number); the bias comes
// out as 16 * 128 in element 0 and is taken off by the accumulators' initial
// value.  The rows (K dimension) are permuted so that two codes of a word 16
// bits apart are one operand register.
//
// fp32 throughout (the codes, FP8 scales and minima are exact in it), rounded
// once to the output's type.
#include "common.cuh"
#include "read.h"

namespace rq {
namespace {

constexpr float kRsqrtD = 0.088388347648318440f;   // 1 / sqrt(128)
constexpr int kWarps = 4;                          // warps per CTA
#ifndef RQ_READ_CTAS
#define RQ_READ_CTAS 4
#endif
constexpr int kRecs = 16;                          // records per warp

// d = a b + c on the tensor cores: a 16 x 16, b 16 x 8, BF16, fp32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2],
                                         const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(c[0]), "f"(c[1]), "f"(c[2]),
          "f"(c[3]));
}

// (scale, minimum) of segment sg of a record's meta bytes.
template <int GS>
__device__ __forceinline__ float2 seg_meta(const uint32_t (&m)[GS == 16 ? 4 : 2], int sg) {
    const int grp = sg * 16 / GS;
    const uint32_t pr = (m[grp >> 1] >> (16 * (grp & 1))) & 0xFFFFu;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pr, __NV_E4M3);
    return __half22float2(__half2(h));
}
template <int GS>
__device__ __forceinline__ void load_meta(const uint8_t *p, uint32_t (&m)[GS == 16 ? 4 : 2]) {
    if (GS == 16) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
        m[0] = v.x;
        m[1] = v.y;
        m[GS == 16 ? 2 : 0] = v.z;
        m[GS == 16 ? 3 : 0] = v.w;
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        m[0] = v.x;
        m[1] = v.y;
    }
}

// The lane's four codes of segment sg (elements 16 sg + 4 q ..), packed.
template <int BITS>
__device__ __forceinline__ uint32_t lane_codes(const uint8_t *codes, int sg, int q) {
    return BITS == 4 ? (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(codes) + 4 * sg + q)
                     : (uint32_t)__ldg(codes + 4 * sg + q);
}
// sc code + mn of those four: 128 + c as a float is the code's bits beside
// 0x43000000, and sc (128 + c) + (mn - 128 sc) is one rounding away from it.
template <int BITS>
__device__ __forceinline__ void expand4(uint32_t w, float2 sm, float x[4]) {
    const float off = fmaf(-128.f, sm.x, sm.y);
#pragma unroll
    for (int k = 0; k < 4; k++) {
        constexpr uint32_t mask = (uint32_t)((1 << BITS) - 1) << 16;
        const int sh = 16 - k * BITS;
        const uint32_t c = (sh >= 0 ? w << sh : w >> -sh) & mask;
        x[k] = fmaf(sm.x, __uint_as_float(c | 0x43000000u), off);
    }
}

template <int OUT>
__device__ __forceinline__ void store4(void *out, size_t at, const float x[4]) {
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
__device__ __forceinline__ void copy_row(void *out, size_t at, const uint16_t *row, int lane) {
    const uint2 w = *reinterpret_cast<const uint2 *>(row + 4 * lane);
    const float x[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                        __uint_as_float(w.y & 0xFFFF0000u)};
    store4<OUT>(out, at + 4 * lane, x);
}

// The tile of 16 tokens of this warp: (kv, b, h) and the first token's index.
struct Tile {
    int kv, b, h, i0;
};
__device__ __forceinline__ bool tile_of(const ReadArgs &a, Tile &t) {
    const long long wid = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int per = (a.n + kRecs - 1) / kRecs;
    if (wid >= 2LL * a.B * a.H * per) return false;   // uniform per warp
    long long r = wid;
    t.i0 = (int)(r % per) * kRecs;
    r /= per;
    t.h = (int)(r % a.H);
    r /= a.H;
    t.b = (int)(r % a.B);
    t.kv = (int)(r / a.B);
    return true;
}
__device__ __forceinline__ size_t row_at(const ReadArgs &a, const Tile &t, int i) {
    return (size_t)(t.b * a.sb + i * a.st + t.h * a.sh);
}

template <int BA, int BR, int GS, bool ROT, int OUT>
__global__ void __launch_bounds__(32 * kWarps, RQ_READ_CTAS) read_rq_kernel(const ReadArgs a) {
    const int lane = threadIdx.x & 31, q = lane & 3;
    Tile tl;
    if (!tile_of(a, tl)) return;
    const int T = a.seqT.v[tl.b];
    const int cnt = min(kRecs, a.n - tl.i0);       // tokens of the tile
    const int t0 = a.t0 + tl.i0;
    const int nc = min(cnt, T - t0);               // of them committed
    // tail tokens, a row at a time
    for (int i = max(0, nc); i < cnt && t0 + i < T + a.n_tail; i++) {
        const uint16_t *row = a.tail[tl.kv] + (((size_t)tl.b * a.tail_cap + (t0 + i - T)) * a.H + tl.h) * kHeadDim;
        copy_row<OUT>(a.out[tl.kv], row_at(a, tl, tl.i0 + i), row, lane);
    }
    if (nc <= 0) return;

    constexpr int MR = 2 * (kHeadDim / GS), NM = GS == 16 ? 4 : 2;
    // the lane's two records; a row past the committed ones repeats the last
    const int row[2] = {lane >> 2, (lane >> 2) + 8};
    size_t rec[2];
#pragma unroll
    for (int u = 0; u < 2; u++) rec[u] = rec_row(a.pg, a.H, tl.b, tl.h, t0 + min(row[u], nc - 1));

    // z = sum_k c_k y_k over the residual records, c_k the product of the
    // coefficients of the records after k (1 for the last): the chain
    // x <- s_k x + R^T y_k unrolled, so that the anchor gets the product of
    // all of them and R^T is applied once.  Under ROT z holds H_16 z_g.
    float z[2][8][4], c[2] = {1.f, 1.f};
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
        for (int sg = 0; sg < 8; sg++)
#pragma unroll
            for (int e = 0; e < 4; e++) z[u][sg][e] = 0.f;
    if (a.nr > 0) {
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
                    const uint32_t lo = (__popc((2 * q + s) & e) & 1) ? 0xBF80u : 0x3F80u;
                    const uint32_t hi = (__popc((2 * q + s + 8) & e) & 1) ? 0xBF80u : 0x3F80u;
                    hm[nt][s] = lo | (hi << 16);
                }
#pragma unroll
                for (int k = 0; k < 4; k++) init[nt][k] = (nt == 0 && q == 0 && (k & 1) == 0) ? -2048.f : 0.f;
            }
        }
        const float e0 = q == 0 ? 16.f : 0.f;   // the lanes that hold element 0 of every segment
#pragma unroll 1
        for (int k = a.nr - 1; k >= 0; k--) {
            const size_t o = k * a.resid_stride;
            uint32_t m[2][NM];
#pragma unroll
            for (int u = 0; u < 2; u++) load_meta<GS>(a.r_meta[tl.kv] + o + rec[u] * MR, m[u]);
            const uint8_t *cp[2] = {a.r_codes[tl.kv] + o + rec[0] * (16 * BR), a.r_codes[tl.kv] + o + rec[1] * (16 * BR)};
            uint16_t sb[2];
#pragma unroll
            for (int u = 0; u < 2; u++) sb[u] = __ldg(reinterpret_cast<const uint16_t *>(a.r_coef[tl.kv] + o) + rec[u]);
#pragma unroll
            for (int sg = 0; sg < 8; sg++) {
                float y[2][4];
                if (ROT) {
                    uint32_t av[4];
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        if (BR == 2) {   // element k at bits 2 k of the segment's word
                            const uint32_t v = __ldg(reinterpret_cast<const uint32_t *>(cp[u]) + sg) >> (4 * q);
                            av[u] = (v & 0x00030003u) | 0x43004300u;              // elements 2q, 2q + 8
                            av[2 + u] = ((v >> 2) & 0x00030003u) | 0x43004300u;   // 2q + 1, 2q + 9
                        } else {         // elements 0-7 and 8-15 in two words: byte q of each
                            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(cp[u]) + sg);
                            const uint32_t v = __byte_perm(w.x, w.y, (uint32_t)(q | ((4 + q) << 8)));   // into bytes 0, 2
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
                        y[u][0] = fmaf(sm.x, d0[2 * u], e0 * sm.y);
                        y[u][1] = sm.x * d0[2 * u + 1];
                        y[u][2] = sm.x * d1[2 * u];
                        y[u][3] = sm.x * d1[2 * u + 1];
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < 2; u++) expand4<BR>(lane_codes<BR>(cp[u], sg, q), seg_meta<GS>(m[u], sg), y[u]);
                }
#pragma unroll
                for (int u = 0; u < 2; u++)
#pragma unroll
                    for (int e = 0; e < 4; e++) z[u][sg][e] = fmaf(c[u], y[u][e], z[u][sg][e]);
            }
#pragma unroll
            for (int u = 0; u < 2; u++) c[u] *= bf16_to_f32(sb[u]);
        }
        if (ROT) {   // H_8 over the segments
#pragma unroll
            for (int w = 1; w < 8; w <<= 1)
#pragma unroll
                for (int sg = 0; sg < 8; sg++)
                    if ((sg & w) == 0) {
#pragma unroll
                        for (int u = 0; u < 2; u++)
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const float p = z[u][sg][e], r = z[u][sg + w][e];
                                z[u][sg][e] = p + r;
                                z[u][sg + w][e] = p - r;
                            }
                    }
        }
    }
    // x = c a + diag(sigma) z / sqrt(d)
#pragma unroll
    for (int u = 0; u < 2; u++) {
        uint32_t m[NM];
        load_meta<GS>(a.a_meta[tl.kv] + rec[u] * MR, m);
        const uint8_t *codes = a.a_codes[tl.kv] + rec[u] * (16 * BA);
        const size_t at = row_at(a, tl, tl.i0 + row[u]) + 4 * q;
#pragma unroll
        for (int sg = 0; sg < 8; sg++) {
            float x[4];
            expand4<BA>(lane_codes<BA>(codes, sg, q), seg_meta<GS>(m, sg), x);
            const uint32_t sig = a.sigma[sg >> 1] >> (16 * (sg & 1) + 4 * q);   // signs of the lane's four elements
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float f = ROT ? __uint_as_float(__float_as_uint(kRsqrtD) | ((sig << (31 - e)) & 0x80000000u)) : 1.f;
                x[e] = fmaf(c[u], x[e], ROT ? z[u][sg][e] * f : z[u][sg][e]);
            }
            if (row[u] < nc) store4<OUT>(a.out[tl.kv], at + 16 * sg, x);
        }
    }
}

template <int OUT>
__global__ void __launch_bounds__(32 * kWarps) read_bf16_kernel(const ReadArgs a) {
    Tile tl;
    if (!tile_of(a, tl)) return;
    const int lane = threadIdx.x & 31, T = a.seqT.v[tl.b], cnt = min(kRecs, a.n - tl.i0), t0 = a.t0 + tl.i0;
    const uint16_t *base = a.bf[tl.kv] + (((size_t)tl.b * a.H + tl.h) * a.Tp + t0) * kHeadDim;
#pragma unroll 4
    for (int i = 0; i < cnt && t0 + i < T; i++)
        copy_row<OUT>(a.out[tl.kv], row_at(a, tl, tl.i0 + i), base + (size_t)i * kHeadDim, lane);
}

template <int BA, int BR, int GS, bool ROT>
void launch_out(const ReadArgs &a, unsigned blocks, cudaStream_t st) {
    if (a.out_type == RQ_OUT_BF16)
        read_rq_kernel<BA, BR, GS, ROT, RQ_OUT_BF16><<<blocks, 32 * kWarps, 0, st>>>(a);
    else
        read_rq_kernel<BA, BR, GS, ROT, RQ_OUT_FP32><<<blocks, 32 * kWarps, 0, st>>>(a);
}
template <int BA, int BR>
void launch_bits(const ReadArgs &a, unsigned blocks, cudaStream_t st) {
    const bool rot = a.rotate != 0;
    if (a.g == 16) rot ? launch_out<BA, BR, 16, true>(a, blocks, st) : launch_out<BA, BR, 16, false>(a, blocks, st);
    else rot ? launch_out<BA, BR, 32, true>(a, blocks, st) : launch_out<BA, BR, 32, false>(a, blocks, st);
}

}  // namespace

cudaError_t launch_read(const ReadArgs &a, int ba, int br, cudaStream_t st) {
    const long long warps = 2LL * a.B * a.H * ((a.n + kRecs - 1) / kRecs);
    const long long blocks = (warps + kWarps - 1) / kWarps;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const unsigned nb = (unsigned)blocks;
    if (a.bf[0])
        a.out_type == RQ_OUT_BF16 ? read_bf16_kernel<RQ_OUT_BF16><<<nb, 32 * kWarps, 0, st>>>(a)
                                  : read_bf16_kernel<RQ_OUT_FP32><<<nb, 32 * kWarps, 0, st>>>(a);
    else if (ba == 4)
        br == 2 ? launch_bits<4, 2>(a, nb, st) : launch_bits<4, 4>(a, nb, st);
    else
        br == 2 ? launch_bits<2, 2>(a, nb, st) : launch_bits<2, 4>(a, nb, st);
    return cudaGetLastError();
}

}  // namespace rq
