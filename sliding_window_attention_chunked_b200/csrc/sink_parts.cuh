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

// The order in which one CTA per SM takes (tile, head) pairs: up to 16 heads side by side, then the next tile
// of each, so that the long tiles of all these heads start first and the short ones (a sequence's ends) fill
// the last round; 148 CTAs are then some nine neighbouring tiles of each head, which share what they read
// through L2. Head by head instead, the last head's long tiles end alone: 201 key tiles' time in place of 188
// by count at T 8192, W 4096, H 16; 967 us a step and 940 so, alternated (the power cap takes the rest back).
struct SinkOrder {
    int rank, head;  // the tile's place in its head's order; the head (of all sequences)
    static __device__ __forceinline__ SinkOrder of(int x, int tiles, int heads) {
        const int g = x / (16 * tiles), r = x - g * 16 * tiles, n = heads - 16 * g < 16 ? heads - 16 * g : 16;
        return {r / n, 16 * g + r % n};
    }
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
    // the CTA of place `rank` when the segments come first, which are no longer than the longest tiles
    __device__ __forceinline__ int far_first(int rank) const {
        const int far = n_tiles * nseg;
        return rank < far ? nk + rank : rank - far;
    }
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
// dk = grad_scale * (all parts), and dv of the first S keys where they have parts
cudaError_t sink_parts_reduce(const SinkParts& p, const SinkArgs& a, bool bf16, cudaStream_t s);

}  // namespace rod
