// decode_window.cu -- single-token attention with a sliding window and sinks
// over the compressed cache (rq_decode_attn_window): the windowed
// instantiations of decode_rq.cuh, in a file of their own so that the two sets
// compile side by side.
#include "decode_rq.cuh"

namespace rq {

cudaError_t launch_decode_rq_window(const DecodeArgs &a, int ba, int br, cudaStream_t st) {
    if (!decode_rq_supported(ba, br, a.nr)) return cudaErrorInvalidValue;
    return dispatch(a.G, a.g, ba, br, a.nr, LaunchF<true>{&a, st});
}

}  // namespace rq
