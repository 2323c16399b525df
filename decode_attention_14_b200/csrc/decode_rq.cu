// decode_rq.cu -- decode attention over the compressed cache, all tokens
// (rq_decode_attn): the instantiations of decode_rq.cuh without a window.
#include "decode_rq.cuh"

#ifdef RQ_FAULT_INJECT
extern "C" int rq_test_arm_fault(void) {
    const int one = 1;
    return cudaMemcpyToSymbol(g_rq_fault_once, &one, sizeof(int)) == cudaSuccess ? 0 : -6;
}
#endif

namespace rq {
namespace {

struct OccF {
    int chunk;
    template <int GK, int BA, int BR, int GS, int NR>
    int go() const { return occupancy_t<GK, BA, BR, GS, NR, false, false>(chunk); }   // same resources paged or not
};

}  // namespace

bool decode_rq_supported(int ba, int br, int nr) {
    return nr >= 0 && nr <= kMaxChain && (nr <= 1 || (ba == 4 && br == 2));
}

cudaError_t launch_decode_rq(const DecodeArgs &a, int ba, int br, cudaStream_t st) {
    // G = 2, 4, 8 run as pairs of query heads per CTA
    if (!decode_rq_supported(ba, br, a.nr)) return cudaErrorInvalidValue;
    return dispatch(a.G, a.g, ba, br, a.nr, LaunchF<false>{&a, st});
}

int decode_rq_occupancy(int G, int ba, int br, int nr, int g, int chunk) {
    if (!decode_rq_supported(ba, br, nr)) return 1;
    return dispatch(G, g, ba, br, nr, OccF{chunk});
}

}  // namespace rq
