// extend.cuh -- work division of the paged SW-SKA attention of new tokens (swska_extend*.cu).
//
// A query tile is up to `rows` new tokens of one sequence; it visits the key tiles (tile keys at
// positions that are multiples of `tile`) of the first S tokens that lie before its window, then
// those of the window. The CTAs of a head group share this work evenly whatever the lengths are: all
// key tiles of all query tiles stand in one line, which is cut into `cols` chunks of equal length, one
// per CTA. A query tile that a cut goes through is split: each CTA leaves its rows' maxima, sums
// and unnormalised outputs in fp32, and the one that finishes last (a counter per tile and head)
// adds them in the order of the keys, so the result does not depend on timing. A CTA has at most two
// such parts (of its first and its last query tile), which bounds the workspace by the GPU, not
// by the batch. The division depends on the lengths, which live on the device, so the launch that
// writes the new tokens to the cache also makes the list of units (query tile x chunk).
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace rod {

struct ExtendUnit {  // 48 bytes: all that a CTA needs besides the table, so that it waits for one load
    int n, q0;          // sequence, its first query of the tile
    int kt0, kt1;       // this unit's range in the tile's list of key tiles (may be empty)
    int part, first;    // this unit's part and the tile's first, -1: the tile is not split
    int c0, nsplit;     // chunk of the first part, parts: the others have numbers 2 (c0 + 1), 2 (c0 + 2), ...
    int row0, len, ctx; // of the sequence (ExtendSeq)
    int counter;
    __device__ __forceinline__ int part_of(int s) const { return s == 0 ? first : 2 * (c0 + s); }
};

struct ExtendRoute {
    int rows = 0, tile = 0;  // queries per tile (0: route not used), keys per key tile
    int groups = 1;          // head groups
    int cols = 1;            // CTAs per head group
    int min_chunk = 1;       // key tiles that a CTA takes at least
    int rows_div = 0;        // > 0: a CTA takes at least sqrt(key tiles x rows of the largest query tile / rows_div)
    int split_cost = 0;      // what the parts of a cut query tile cost, in key tiles
    int part_rows = 0;       // rows kept of a part
    int cap_items = 0;
    ExtendUnit* units = nullptr;  // [cap_items + cols]: unit of query tile i in chunk c at i + c
    int* range = nullptr;         // [cols][2]: first and last query tile of each chunk (first > last: none)
    int* count = nullptr;         // [cols][H]
    float* part_o = nullptr;      // [2 cols][H][part_rows][dv]
    float2* part_ml = nullptr;    // [2 cols][H][part_rows]: maximum (base 2) and sum
    __device__ __forceinline__ int64_t part_at(int part, int H, int h, int row) const {
        return ((int64_t)part * H + h) * part_rows + row;
    }
};
__device__ __forceinline__ ExtendUnit load_unit(const ExtendUnit* p) {
    const int4* x = reinterpret_cast<const int4*>(p);
    const int4 a = __ldcg(x), b = __ldcg(x + 1), c = __ldcg(x + 2);
    return ExtendUnit{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
}
// the units of a CTA: x in [lo, hi]
struct ExtendRange {
    int lo, hi;
};
__device__ __forceinline__ ExtendRange load_range(const ExtendRoute& r, int col) {
    const int2 t = __ldcg(reinterpret_cast<const int2*>(r.range) + col);
    return ExtendRange{t.x + col, t.y + col};
}

struct ExtendPlan {
    ExtendRoute r[2];  // [0] sequences of at most short_len new tokens, [1] the others
    int short_len = 0;
};

// one sequence of the batch; all arguments come from the device, so everything is bounded here
struct ExtendSeq {
    int row0, len;  // rows of q, k_new, v_new, o
    int ctx;        // position of the first new token
    bool bad;       // a position outside [0, 2^31 - len): outputs NaN
};
__device__ __forceinline__ ExtendSeq extend_seq(const ExtendArgs& a, int n) {
    ExtendSeq s;
    int lo = a.cu[n], hi = a.cu[n + 1];
    lo = lo < 0 ? 0 : (lo > a.M ? a.M : lo);
    hi = hi < lo ? lo : (hi > a.M ? a.M : hi);
    s.row0 = lo;
    s.len = hi - lo < a.max_len ? hi - lo : a.max_len;
    const int64_t c = a.ctx[n];
    s.bad = c < 0 || c > (int64_t)0x7fffffff - s.len;
    s.ctx = s.bad ? 0 : (int)c;
    return s;
}

// key tiles of the query tile [q0, q0 + rows) of a sequence
struct ExtendKeys {
    int n_sink, lo, n;  // tiles of the first S keys, first tile of the window, tiles in all
    __device__ __forceinline__ int at(int i) const { return i < n_sink ? i : lo + i - n_sink; }
};
__device__ __forceinline__ ExtendKeys extend_keys(const ExtendSeq& s, int q0, int rows, int tile, int W, int S) {
    ExtendKeys k;
    const int p0 = s.ctx + q0, last = q0 + rows < s.len ? q0 + rows : s.len;
    const int p1 = s.ctx + last - 1;
    const int64_t lo = (int64_t)p0 - W + 1;
    const int tl = __ffs(tile) - 1;  // a power of two
    k.lo = (int)(lo > 0 ? lo : 0) >> tl;
    const int ns = (S + tile - 1) >> tl;
    k.n_sink = ns < k.lo ? ns : k.lo;
    k.n = k.n_sink + (p1 >> tl) - k.lo + 1;
    return k;
}

// The physical page of a logical page, or -1 where the table has none inside the pool.
__device__ __forceinline__ int extend_page(const ExtendArgs& a, int n, int page) {
    if (page < 0 || page >= a.max_pages) return -1;
    const int e = a.table[(int64_t)n * a.max_pages + page];
    return (unsigned)e < (unsigned)a.P ? e : -1;
}

// host: routes and workspace
ExtendPlan extend_plan(int M, int N, int H, int dk, int dv, int max_len, bool bf16);
size_t extend_bind(ExtendPlan& p, int H, int dv, void* workspace);  // returns the bytes

// The launch before wrote the units and the cache: a kernel launched to overlap its tail waits here.
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// kernels; each launcher runs one route of the plan
cudaError_t swska_extend_simt_launch(const ExtendArgs& a, const ExtendRoute& r, bool bf16, cudaStream_t s);
cudaError_t swska_extend_few_launch(const ExtendArgs& a, const ExtendRoute& r, cudaStream_t s);
unsigned swska_extend_few_take_timeout_flag();
cudaError_t swska_extend_tc_launch(const ExtendArgs& a, const ExtendRoute& r, cudaStream_t s);
unsigned swska_extend_tc_take_timeout_flag();
constexpr int kChunkRows = 128;  // bf16, 128-wide heads: longer sequences, in tiles of so many queries
constexpr int kChunkTile = 128;  // and keys
constexpr int kFewRows = 16;   // bf16, 128-wide heads: sequences of at most this many new tokens
constexpr int kFewTile = 32;   // keys per tile there
constexpr int kFewHeads = 8;   // heads per CTA there

}  // namespace rod
