// rebuild.cu -- the rows that a chunk of new tokens attends to, rebuilt from the
// compressed cache as BF16 pairs in a workspace (the first launch of
// rq_prefill_attn_window): the kOutPair instantiations of read.cuh.  The chunk's
// rows share this work, which a fused kernel would repeat for every block of 64
// of them (500 / 2048 tokens 147 / 250 us fused, 48 / 70 us with the workspace).
// Bound as a plain read is: 2048 tokens of 16 heads after the 1024 of their window
// (residual, tail), 18.7 us, issue slots used in 62% of the cycles.
#include "read.cuh"

namespace rq {
namespace {

template <int BA, int BR, int GS>
cudaError_t launch_group(const ReadArgs &a, unsigned blocks, cudaStream_t st) {
    if (a.nr == 0) return launch_t<BA, 2, GS, 0, false, kOutPair>(a, blocks, st);
    return a.rotate ? launch_t<BA, BR, GS, 1, true, kOutPair>(a, blocks, st)
                    : launch_t<BA, BR, GS, 1, false, kOutPair>(a, blocks, st);
}
template <int BA, int BR>
cudaError_t launch_bits(const ReadArgs &a, unsigned blocks, cudaStream_t st) {
    return a.g == 16 ? launch_group<BA, BR, 16>(a, blocks, st) : launch_group<BA, BR, 32>(a, blocks, st);
}

}  // namespace

cudaError_t launch_rebuild(const ReadArgs &args, int ba, int br, cudaStream_t st) {
    ReadArgs a = args;
    const long long units = 2LL * a.B * a.H, nt = a.pair_rows / kRecs;
    a.tiles = warp_tiles(units * nt, a.sms);
    const int per = a.tiles * kWarps;
    const long long blocks = units * ((nt + per - 1) / per);
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const unsigned nb = (unsigned)blocks;
    if (ba == 4) return br == 2 ? launch_bits<4, 2>(a, nb, st) : launch_bits<4, 4>(a, nb, st);
    return launch_bits<2, 2>(a, nb, st);
}

}  // namespace rq
