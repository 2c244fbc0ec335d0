// fa_sink.cu -- the kernel variants for causal windows with sinks and shared
// key heads, whole-tile and balanced schedules; see fa_launch.cuh.
#include "fa_launch.cuh"

namespace fa_launch {

fa_status launch_sink(int D, bool bf16, bool split, const CUtensorMap &q, const CUtensorMap &k,
                      const CUtensorMap &v, const fa::SinkParams &p, int grid, cudaStream_t s, int dev)
{
    return split ? launch_mask<fa::kMaskSink, true>(D, bf16, q, k, v, p, grid, s, dev)
                 : launch_mask<fa::kMaskSink, false>(D, bf16, q, k, v, p, grid, s, dev);
}

unsigned int *status_word_sink()
{
    return fa::status_word_address();
}

}  // namespace fa_launch
