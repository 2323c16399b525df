// prefill_window.cu -- attention of several new tokens with a sliding window and
// sinks over the compressed cache (rq_prefill_attn_window): the windowed
// instantiations of prefill.cuh, in a file of their own so that the two sets
// compile side by side.
#include "prefill.cuh"

namespace rq {

cudaError_t launch_prefill_window(const PrefillArgs &a, int ba, int br, cudaStream_t st) {
    return a.g == 16 ? launch_group<true, 16>(a, ba, br, st) : launch_group<true, 32>(a, ba, br, st);
}

}  // namespace rq
