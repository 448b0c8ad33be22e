// swska_sink.cu -- routes of SW-SKA with first tokens that stay visible (forward and backward).
#include "sink_parts.cuh"

namespace rod {

template <int DK> cudaError_t sink_simt_launch(const SinkArgs& a, bool backward, cudaStream_t s);
template <> cudaError_t sink_simt_launch<16>(const SinkArgs&, bool, cudaStream_t);
template <> cudaError_t sink_simt_launch<32>(const SinkArgs&, bool, cudaStream_t);
template <> cudaError_t sink_simt_launch<64>(const SinkArgs&, bool, cudaStream_t);
template <> cudaError_t sink_simt_launch<128>(const SinkArgs&, bool, cudaStream_t);
template <int DK> cudaError_t sink_mma_launch(const SinkArgs& a, bool backward, cudaStream_t s);
template <> cudaError_t sink_mma_launch<16>(const SinkArgs&, bool, cudaStream_t);
template <> cudaError_t sink_mma_launch<32>(const SinkArgs&, bool, cudaStream_t);
template <> cudaError_t sink_mma_launch<64>(const SinkArgs&, bool, cudaStream_t);
template <> cudaError_t sink_mma_launch<128>(const SinkArgs&, bool, cudaStream_t);

namespace {

cudaError_t by_dim(const SinkArgs& a, bool bf16, bool backward, cudaStream_t s) {
    switch (a.d_k) {
        case 16: return bf16 ? sink_mma_launch<16>(a, backward, s) : sink_simt_launch<16>(a, backward, s);
        case 32: return bf16 ? sink_mma_launch<32>(a, backward, s) : sink_simt_launch<32>(a, backward, s);
        case 64: return bf16 ? sink_mma_launch<64>(a, backward, s) : sink_simt_launch<64>(a, backward, s);
        case 128: return bf16 ? sink_mma_launch<128>(a, backward, s) : sink_simt_launch<128>(a, backward, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

// bf16 with 128-wide heads and at least one full tile runs on tcgen05, other bf16 on warp-level matrix
// instructions, fp32 on CUDA cores
cudaError_t swska_sink_prefill_launch(const SinkArgs& a, bool bf16, cudaStream_t s) {
    if (bf16 && swska_prefill_tc_supported(a.H, a.T, a.d_k, a.d_v))
        return swska_prefill_tc_stats_launch(a.q, a.k, a.v, a.out, nullptr, a.lse_out, nullptr, a.T, a.B, a.H, a.T, a.W,
                                             a.scale, s, 0.6931471805599453f, a.S);
    return by_dim(a, bf16, false, s);
}
cudaError_t swska_sink_backward_launch(const SinkArgs& a, bool bf16, cudaStream_t s) {
    if (bf16 && swska_backward_tc_supported(a.H, a.T, a.d_k, a.d_v)) return swska_sink_backward_tc_launch(a, s);
    return by_dim(a, bf16, true, s);
}
size_t swska_sink_backward_workspace_size(int B, int H, int T, int dk, int dv, int W, int S) {
    SinkArgs a{};
    a.B = B, a.H = H, a.T = T, a.d_k = dk, a.d_v = dv, a.W = W, a.S = S;
    // enough for either route (their key and query tiles), with at most H head groups
    const size_t x = sink_parts_floats(sink_parts_plan(a, 32, 64, H)), y = sink_parts_floats(sink_parts_plan(a, 64, 64, H)),
                 z = sink_parts_floats(sink_parts_plan(a, 128, 128, H)), w = x > y ? x : y;
    return (w > z ? w : z) * sizeof(float);
}

}  // namespace rod
