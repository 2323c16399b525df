// decode_window.cu -- single-token attention with a sliding window and sinks
// over the compressed cache (rq_decode_attn_window): the windowed
// instantiations of decode_rq.cuh, in a file of their own so that the two sets
// compile side by side.  Bound as without a window by instructions (issue slots
// used in 61% of the cycles) and by waiting in the rest: 4 x 16 heads, one residual, window 4096 + 4 sinks (68 MB)
// 24.0 us (the records in L2; 29.6 us from DRAM); two paged sequences at an
// anchor loop, 8 kv heads of 4 heads, window 32768 (84 MB) 68.4 us, two CTAs per
// kv head and split, each for two of its heads; a window of 256 is a launch's
// latency, 7.9 us.
#include "decode_rq.cuh"

namespace rq {

cudaError_t launch_decode_rq_window(const DecodeArgs &a, int ba, int br, cudaStream_t st) {
    if (!decode_rq_supported(ba, br, a.nr)) return cudaErrorInvalidValue;
    return dispatch(a.G, a.g, ba, br, a.nr, LaunchF<true>{&a, st});
}

}  // namespace rq
