// sink_parts.cu -- host side and reduction launch of sink_parts.cuh.
#include "sink_parts.cuh"

#include "simt_tile.cuh"

namespace rod {
namespace {

// Memory bound: reads every part once, writes dk (and the S rows of dv) once.
__global__ void __launch_bounds__(256)
sink_reduce_kernel(const SinkParts p, void* __restrict__ dk, void* __restrict__ dv, bool bf16, float scale) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the launch that made the parts
    const int64_t n_dk = (int64_t)p.B * p.T * p.dk / 4;
    const int64_t n_dv = p.nseg > 0 ? (int64_t)p.B * p.H * p.R * p.dv / 4 : 0;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n_dk + n_dv;
         i += (int64_t)gridDim.x * blockDim.x) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float* x) {
            const float4 t = __ldcg(reinterpret_cast<const float4*>(x));
            s.x += t.x;
            s.y += t.y;
            s.z += t.z;
            s.w += t.w;
        };
        if (i < n_dk) {
            const int64_t row = (4 * i) >> (__ffs(p.dk) - 1);  // dk is a power of two
            const int b = (int)(row >> 32 == 0 ? (uint32_t)row / (uint32_t)p.T : row / p.T);
            const int c = (int)(4 * i & (p.dk - 1)), key = (int)(row - (int64_t)b * p.T);
#pragma unroll 8
            for (int g = 0; g < p.G; ++g) add(p.dk_part + (int64_t)g * n_dk * 4 + 4 * i);
            if (p.nseg > 0 && key < p.R)
                for (int sl = 1; sl <= p.nseg; ++sl)
                    for (int g = 0; g < p.G; ++g) add(p.dk_at(sl, g, b, key) + c);
            simt::store4_as(dk, bf16, 4 * i, make_float4(s.x * scale, s.y * scale, s.z * scale, s.w * scale));
        } else {
            const int64_t e = 4 * (i - n_dk), row = e / p.dv;
            const int c = (int)(e - row * p.dv), key = (int)(row % p.R);
            const int64_t bh = row / p.R;
            for (int sl = 0; sl <= p.nseg; ++sl) add(p.dv_at(sl, bh, key) + c);
            simt::store4_as(dv, bf16, (bh * p.T + key) * p.dv + c, s);
        }
    }
}

int64_t tpad(int T) { return ((int64_t)T + 127) / 128 * 128; }

}  // namespace

SinkParts sink_parts_plan(const SinkArgs& a, int ks, int qs, int G) {
    SinkParts p;
    p.ks = ks;
    p.qs = qs;
    p.nk = (a.T + ks - 1) / ks;
    p.nq = (a.T + qs - 1) / qs;
    p.G = G;
    p.B = a.B;
    p.H = a.H;
    p.T = a.T;
    p.W = a.W;
    p.dk = a.d_k;
    p.dv = a.d_v;
    p.R = a.S < a.T ? a.S : a.T;
    const int near = SinkParts::near_hi(0, ks, qs, p.nq, a.W) + 1, far = p.nq - near;  // the first tile has the most
    if (p.R > 0 && far > 0) {
        p.n_tiles = (p.R + ks - 1) / ks;
        // a segment is no longer than a window, 4 to 8 tiles (short ones fill the end of the launch; each
        // costs S rows of memory traffic), and there are at most 64 of them
        p.seg_len = near > 4 ? (near < 8 ? near : 8) : 4;
        if (p.seg_len * 64 < far) p.seg_len = (far + 63) / 64;
        p.nseg = (far + p.seg_len - 1) / p.seg_len;
    }
    return p;
}

size_t sink_parts_floats(const SinkParts& p) {
    const size_t bh = (size_t)p.B * p.H;
    size_t n = 2 * bh * (size_t)tpad(p.T) + (size_t)p.G * p.B * p.T * p.dk;
    if (p.nseg > 0) n += (size_t)(1 + p.nseg) * bh * p.R * p.dv + (size_t)p.nseg * p.G * p.B * p.R * p.dk;
    return n;
}

float* sink_parts_bind(SinkParts& p, const SinkArgs& a) {
    float* ws = static_cast<float*>(a.workspace);
    p.dk_part = ws + 2 * (size_t)p.B * p.H * tpad(p.T);
    p.dv_far = p.dk_part + (size_t)p.G * p.B * p.T * p.dk;
    p.dk_far = p.dv_far + (p.nseg > 0 ? (size_t)(1 + p.nseg) * p.B * p.H * p.R * p.dv : 0);
    return ws;
}

cudaError_t sink_parts_reduce(const SinkParts& p, const SinkArgs& a, bool bf16, cudaStream_t s) {
    const int64_t n = (int64_t)p.B * p.T * p.dk / 4 + (p.nseg > 0 ? (int64_t)p.B * p.H * p.R * p.dv / 4 : 0);
    const int64_t want = (n + 255) / 256, cap = 8 * (int64_t)device_sm_count();
    const cudaError_t e = launch_overlapped(sink_reduce_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(256), 0, s, p, a.dk,
                                            a.dv, bf16, a.grad_scale);
    note_launches(1);
    return e;
}

}  // namespace rod
