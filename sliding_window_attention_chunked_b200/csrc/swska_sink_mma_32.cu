// swska_sink_mma_32.cu -- the kernels of swska_sink_mma.cuh for key head dim 32.
#include "swska_sink_mma.cuh"

namespace rod {

template <>
cudaError_t sink_mma_launch<32>(const SinkArgs& a, bool backward, cudaStream_t s) {
    return pick_dv<32>(a, backward, s);
}

}  // namespace rod
