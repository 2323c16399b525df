// read.cu -- reading the cache back: tokens of one (layer, loop) rebuilt from
// their records as K and V rows (the inverse of append.cu; ai4snews summary,
// paragraph 3: the shared-anchor reconstruction k = s a + R^T y, two reads).
//
// One warp rebuilds one record of one (K|V, sequence, token, kv head): lane l
// holds the four head_dim elements 4l..4l+3.
//   x = sc code + mn per quantization group (the anchor), then per residual
//   record x <- s x + R^T (sc_r code_r + mn_r),  R^T y = diag(sigma) H y / sqrt(d)
// in fp32 (the codes, FP8 scales and minima are exact in it), rounded once to
// the output's type.
#include "common.cuh"
#include "read.h"

namespace rq {
namespace {

constexpr float kRsqrtD = 0.088388347648318440f;   // 1 / sqrt(128)

// The four values of this lane: codes 4 lane .. 4 lane + 3 and their group's
// scale and minimum.
__device__ __forceinline__ void record4(const uint8_t *codes, const uint8_t *meta, int bits, int g, int lane,
                                        float x[4]) {
    const uint32_t w = bits == 4 ? __ldg(reinterpret_cast<const uint16_t *>(codes) + lane) : __ldg(codes + lane);
    const uint32_t m = __ldg(reinterpret_cast<const uint16_t *>(meta) + (4 * lane) / g);
    const float sc = e4m3_to_f32(m & 0xFFu), mn = e4m3_to_f32(m >> 8);
#pragma unroll
    for (int k = 0; k < 4; k++) x[k] = fmaf(sc, (float)((w >> (k * bits)) & ((1u << bits) - 1u)), mn);
}

__device__ __forceinline__ void store4(const ReadArgs &a, int kv, size_t at, const float x[4]) {
    if (a.out_type == RQ_OUT_BF16) {
        uint2 v;
        v.x = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x[0])) |
              (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x[1])) << 16;
        v.y = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x[2])) |
              (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x[3])) << 16;
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out[kv]) + at) = v;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out[kv]) + at) = make_float4(x[0], x[1], x[2], x[3]);
    }
}

__global__ void __launch_bounds__(128) read_kernel(const ReadArgs a, int ba, int br) {
    const int lane = threadIdx.x & 31;
    const long long wid = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (wid >= 2LL * a.B * a.n * a.H) return;   // uniform per warp
    long long r = wid;
    const int h = (int)(r % a.H);
    r /= a.H;
    const int i = (int)(r % a.n);
    r /= a.n;
    const int b = (int)(r % a.B);
    const int kv = (int)(r / a.B);
    const int t = a.t0 + i, T = a.seqT.v[b];
    if (t >= T + a.n_tail) return;
    const size_t at = (size_t)(b * a.sb + i * a.st + h * a.sh) + 4 * lane;
    float x[4];
    if (t >= T || a.bf[0]) {
        const uint16_t *row = t >= T ? a.tail[kv] + (((size_t)b * a.tail_cap + (t - T)) * a.H + h) * kHeadDim
                                     : a.bf[kv] + (((size_t)b * a.H + h) * a.Tp + t) * kHeadDim;
        const uint2 w = *reinterpret_cast<const uint2 *>(row + 4 * lane);
        x[0] = bf16_to_f32((uint16_t)(w.x & 0xFFFFu));
        x[1] = bf16_to_f32((uint16_t)(w.x >> 16));
        x[2] = bf16_to_f32((uint16_t)(w.y & 0xFFFFu));
        x[3] = bf16_to_f32((uint16_t)(w.y >> 16));
        store4(a, kv, at, x);
        return;
    }
    const size_t rec = rec_row(a.pg, a.H, b, h, t);
    const int meta_rec = 2 * (kHeadDim / a.g);
    record4(a.a_codes[kv] + rec * (16 * ba), a.a_meta[kv] + rec * meta_rec, ba, a.g, lane, x);
    for (int k = 0; k < a.nr; k++) {
        float y[4];
        const size_t o = k * a.resid_stride;
        record4(a.r_codes[kv] + o + rec * (16 * br), a.r_meta[kv] + o + rec * meta_rec, br, a.g, lane, y);
        const float s = bf16_to_f32(__ldg(reinterpret_cast<const uint16_t *>(a.r_coef[kv] + o) + rec));
        if (a.rotate) {
            wht128_warp<float>(y, lane);
#pragma unroll
            for (int e = 0; e < 4; e++) y[e] *= sigma_neg(a.sigma, 4 * lane + e) ? -kRsqrtD : kRsqrtD;
        }
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = fmaf(s, x[e], y[e]);
    }
    store4(a, kv, at, x);
}

}  // namespace

cudaError_t launch_read(const ReadArgs &a, int ba, int br, cudaStream_t st) {
    const long long warps = 2LL * a.B * a.n * a.H;
    const long long blocks = (warps + 3) / 4;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    read_kernel<<<(unsigned)blocks, 128, 0, st>>>(a, ba, br);
    return cudaGetLastError();
}

}  // namespace rq
