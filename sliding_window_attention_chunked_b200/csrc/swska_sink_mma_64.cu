// swska_sink_mma_64.cu -- the kernels of swska_sink_mma.cuh for key head dim 64.
#include "swska_sink_mma.cuh"

namespace rod {

template <>
cudaError_t sink_mma_launch<64>(const SinkArgs& a, bool backward, cudaStream_t s) {
    return pick_dv<64>(a, backward, s);
}

}  // namespace rod
