// read.cu -- rq_cache_read: the instantiations of read.cuh that write rows in
// the caller's layout, and the plain copy of a BF16 cache's rows.
#include "read.cuh"

namespace rq {
namespace {

template <int OUT>
__global__ void __launch_bounds__(32 * kWarps) read_bf16_kernel(const ReadArgs a) {
    Span sp;
    if (!span_of(a, sp)) return;
    const int lane = threadIdx.x & 31;
    const int lo = max(a.t0, sp.tile0 * kRecs);
    const int hi = min(min(a.t0 + a.n, (sp.tile0 + sp.tiles) * kRecs), a.seqT.v[sp.b]);
    const uint16_t *base = a.bf[sp.kv] + ((size_t)sp.b * a.H + sp.h) * a.Tp * kHeadDim;
#pragma unroll 4
    for (int t = lo; t < hi; t++)
        copy_row<OUT>(a.out[sp.kv], row_at(a, sp, t), base + (size_t)t * kHeadDim, lane);
}

template <int BA, int BR, int GS, int NR, bool ROT>
cudaError_t launch_out(const ReadArgs &a, unsigned blocks, cudaStream_t st) {
    return a.out_type == RQ_OUT_BF16 ? launch_t<BA, BR, GS, NR, ROT, RQ_OUT_BF16>(a, blocks, st)
                                     : launch_t<BA, BR, GS, NR, ROT, RQ_OUT_FP32>(a, blocks, st);
}
template <int BA, int BR, int GS>
cudaError_t launch_chain(const ReadArgs &a, unsigned blocks, cudaStream_t st) {
    if (a.nr == 0) return launch_out<BA, 2, GS, 0, false>(a, blocks, st);
    if (a.nr == 1)
        return a.rotate ? launch_out<BA, BR, GS, 1, true>(a, blocks, st) : launch_out<BA, BR, GS, 1, false>(a, blocks, st);
    return a.rotate ? launch_out<BA, BR, GS, 2, true>(a, blocks, st) : launch_out<BA, BR, GS, 2, false>(a, blocks, st);
}
template <int BA, int BR>
cudaError_t launch_bits(const ReadArgs &a, unsigned blocks, cudaStream_t st) {
    return a.g == 16 ? launch_chain<BA, BR, 16>(a, blocks, st) : launch_chain<BA, BR, 32>(a, blocks, st);
}

}  // namespace

cudaError_t launch_read(const ReadArgs &args, int ba, int br, cudaStream_t st) {
    ReadArgs a = args;
    const long long units = 2LL * a.B * a.H, nt = tiles_of(a.t0, a.n);
    a.tiles = warp_tiles(units * nt, a.sms);
    const int per = a.tiles * kWarps;
    const long long blocks = units * ((nt + per - 1) / per);
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const unsigned nb = (unsigned)blocks;
    if (a.bf[0]) {
        a.out_type == RQ_OUT_BF16 ? read_bf16_kernel<RQ_OUT_BF16><<<nb, 32 * kWarps, 0, st>>>(a)
                                  : read_bf16_kernel<RQ_OUT_FP32><<<nb, 32 * kWarps, 0, st>>>(a);
        return cudaGetLastError();
    }
    if (ba == 4) return br == 2 ? launch_bits<4, 2>(a, nb, st) : launch_bits<4, 4>(a, nb, st);
    return br == 2 ? launch_bits<2, 2>(a, nb, st) : launch_bits<2, 4>(a, nb, st);
}

}  // namespace rq
