// swska_sink_simt_16.cu -- the kernels of swska_sink_simt.cuh for key head dim 16.
#include "swska_sink_simt.cuh"

namespace rod {

template <>
cudaError_t sink_simt_launch<16>(const SinkArgs& a, bool backward, cudaStream_t s) {
    return pick_dv<16>(a, backward, s);
}

}  // namespace rod
