// sink_parts.cuh -- how the backward kernels of SW-SKA with first tokens that stay visible divide the
// key side, and the launch that adds the parts.
//
// A key tile is seen by its near queries (its own tile to the end of its window). A tile that
// holds some of the first S keys is also seen by every later, far query: those are dealt out in
// segments of about a window's length, so that no CTA works much longer than the others. Slot 0
// holds a tile's near sums, slot 1 + g those of segment g; only the S rows are kept, in fp32.
// The sums are added slot by slot and head group by head group, in that order, by one thread per
// element: the result does not depend on which CTA finished first.
#pragma once

#include "kernels.h"

namespace rod {

struct SinkWork {
    int tile, slot, q_lo, q_hi;  // key tile, slot, query tiles [q_lo, q_hi]
};

struct SinkParts {
    int ks = 0, qs = 0, nk = 0, nq = 0;        // rows of a key tile and of a query tile, and their numbers
    int n_tiles = 0, nseg = 0, seg_len = 0;    // key tiles with far queries, segments each, query tiles per segment
    int G = 0, B = 0, H = 0, T = 0, W = 0, R = 0, dk = 0, dv = 0;  // head groups of dk; R = min(S, T) rows
    float* dk_part = nullptr;  // [G][B][T][dk]       near sums of every key
    float* dv_far = nullptr;   // [1 + nseg][B H][R][dv]
    float* dk_far = nullptr;   // [nseg][G][B][R][dk]

    // the last query tile that sees a key tile through the window
    __host__ __device__ static int near_hi(int tile, int ks, int qs, int nq, int W) {
        const int64_t last = ((int64_t)tile * ks + ks - 1 + W - 1) / qs;
        return last < nq - 1 ? (int)last : nq - 1;
    }
    __host__ __device__ int ctas() const { return nk + n_tiles * nseg; }
    __device__ __forceinline__ SinkWork work(int x) const {
        SinkWork w;
        if (x < nk) {
            w.tile = x;
            w.slot = 0;
            w.q_lo = x * ks / qs;
            w.q_hi = near_hi(x, ks, qs, nq, W);
        } else {
            w.tile = (x - nk) / nseg;
            const int g = (x - nk) % nseg;
            w.slot = 1 + g;
            w.q_lo = near_hi(w.tile, ks, qs, nq, W) + 1 + g * seg_len;
            w.q_hi = w.q_lo + seg_len - 1 < nq - 1 ? w.q_lo + seg_len - 1 : nq - 1;
        }
        return w;
    }
    __device__ __forceinline__ float* dv_at(int slot, int64_t bh, int key) const {
        return dv_far + (((int64_t)slot * B * H + bh) * R + key) * dv;
    }
    __device__ __forceinline__ float* dk_at(int slot, int g, int b, int key) const {
        return dk_far + ((((int64_t)(slot - 1) * G + g) * B + b) * R + key) * dk;
    }
};

// the split for key tiles of ks rows, query tiles of qs and G head groups (pointers not set)
SinkParts sink_parts_plan(const SinkArgs& a, int ks, int qs, int G);
// floats of workspace: row statistics (two arrays of T rounded up to 128 rows), then the parts
size_t sink_parts_floats(const SinkParts& p);
// sets the pointers inside a.workspace; returns the statistics array (2 B H Tpad floats)
float* sink_parts_bind(SinkParts& p, const SinkArgs& a);
// dk = scale * (all parts), and dv of the first S keys where they have parts
cudaError_t sink_parts_reduce(const SinkParts& p, const SinkArgs& a, bool bf16, cudaStream_t s);

}  // namespace rod
