// swska_sink_mma_128.cu -- the kernels of swska_sink_mma.cuh for key head dim 128.
#include "swska_sink_mma.cuh"

namespace rod {

template <>
cudaError_t sink_mma_launch<128>(const SinkArgs& a, bool backward, cudaStream_t s) {
    return pick_dv<128>(a, backward, s);
}

}  // namespace rod
