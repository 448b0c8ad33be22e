// swska_extend.cu -- SW-SKA attention of a ragged batch of new tokens over a paged cache: routes,
// workspace, and the launch that writes the new tokens to their slots and divides the work.
//
// SALA blog §3.3: chunked prefill over a paged KV cache; CodeFuse Rodimus* article, SKA paragraph:
// one K, per-head V. The write is a copy of M (dk + H dv) elements (bound by HBM at large M, by
// launch latency at a decode step), so the division of the work, one CTA's, hides behind it.
#include "extend.cuh"

#include <math.h>

namespace rod {
namespace {

constexpr int NT = 256;
constexpr int NW = NT / 32;

__device__ __forceinline__ int block_incl(int x, int* sums, int* total) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const int t = sums[w];
        if (w < warp) before += t;
        all += t;
    }
    *total = all;
    return x + before;
}

// query tiles and, at most, key tiles per query tile of a sequence on route i (0 tiles: not on it)
struct SeqWork {
    int items, tiles;
};
__device__ __forceinline__ SeqWork seq_work(const ExtendArgs& a, const ExtendPlan& p, int i, const ExtendSeq& s) {
    const ExtendRoute& r = p.r[i];
    SeqWork w{0, 0};
    if (s.len == 0 || s.bad || r.rows == 0) return w;
    const bool is_short = p.r[0].rows != 0 && (s.len <= p.short_len || p.r[1].rows == 0);
    if (is_short != (i == 0)) return w;
    w.items = (s.len + r.rows - 1) / r.rows;
    // the widest query tile: a window and the tile's rows, at any alignment, and the first tokens
    const int rows = s.len < r.rows ? s.len : r.rows;
    const int64_t span = (int64_t)(a.W < s.ctx + s.len ? a.W : s.ctx + s.len) + rows;
    const int most = (int)((span + r.tile - 1) / r.tile) + 1 + (a.S + r.tile - 1) / r.tile;
    const int all = (s.ctx + s.len - 1) / r.tile + 1;
    w.tiles = most < all ? most : all;
    return w;
}

__global__ void __launch_bounds__(NT) extend_prepare_kernel(const ExtendArgs a, const ExtendPlan p) {
    // the attention kernel may set itself up meanwhile; it waits for this launch's end before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x > 0) {
        // ---- new keys and values to their slots, 16 bytes a thread
        if (a.k_new == nullptr) return;
        const int ck = a.d_k * a.es / 16, cv = a.d_v * a.es / 16, per = ck + a.H * cv;
        const int64_t n = (int64_t)a.M * per;
        const int64_t slots = (int64_t)a.P * a.page;
        for (int64_t i = (int64_t)(blockIdx.x - 1) * NT + threadIdx.x; i < n; i += (int64_t)(gridDim.x - 1) * NT) {
            const int row = (int)(i / per), c = (int)(i - (int64_t)row * per);
            const int64_t slot = a.slot[row];
            if (slot < 0 || slot >= slots) continue;
            const int64_t pg = slot / a.page;
            const int off = (int)(slot - pg * a.page);
            if (c < ck) {
                static_cast<uint4*>(a.k_pool)[slot * ck + c] = static_cast<const uint4*>(a.k_new)[(int64_t)row * ck + c];
            } else {
                const int h = (c - ck) / cv, cc = (c - ck) % cv;
                static_cast<uint4*>(a.v_pool)[((pg * a.H + h) * a.page + off) * cv + cc] =
                    static_cast<const uint4*>(a.v_new)[((int64_t)row * a.H + h) * cv + cc];
            }
        }
        return;
    }
    // ---- rows of sequences at impossible positions
    for (int base = 0; base < a.N; base += NT) {
        const int n = base + (int)threadIdx.x;
        if (!__syncthreads_or(n < a.N && extend_seq(a, n).bad)) continue;
        for (int m = base; m < base + NT && m < a.N; ++m) {
            const ExtendSeq s = extend_seq(a, m);
            if (!s.bad) continue;
            const int64_t lo = (int64_t)s.row0 * a.H * a.d_v, n_o = (int64_t)s.len * a.H * a.d_v;
            for (int64_t i = threadIdx.x; i < n_o; i += NT) {
                if (a.es == 2) static_cast<unsigned short*>(a.o)[lo + i] = 0x7fff;
                else static_cast<unsigned*>(a.o)[lo + i] = 0x7fffffffu;
            }
        }
    }
    // ---- the units of each route
    __shared__ int s_sums[NW];
    __shared__ int s_at[NT + 1];     // first unit of each sequence of the chunk
    __shared__ int s_items[NT + 1];  // first query tile
    __shared__ int s_ns[NT];
    for (int i = 0; i < 2; ++i) {
        const ExtendRoute& r = p.r[i];
        if (r.rows == 0) continue;
        long long tiles = 0;
        int items = 0;
        for (int n = threadIdx.x; n < a.N; n += NT) {
            const SeqWork w = seq_work(a, p, i, extend_seq(a, n));
            items += w.items;
            tiles += (long long)w.items * w.tiles;
        }
        int n_items, lo, hi;
        block_incl(items, s_sums, &n_items);
        // the sum of up to 2^47 in two halves
        block_incl((int)(tiles & 0xffff), s_sums, &lo);
        block_incl((int)(tiles >> 16), s_sums, &hi);
        const long long n_tiles = ((long long)hi << 16) + lo;
        // key tiles per unit: enough units for the GPU, and no split when the query tiles do
        long long C = 1ll << 40;
        if ((long long)n_items * r.groups < r.target) {
            C = (n_tiles * r.groups + r.target - 1) / r.target;
            const long long even = (n_tiles * r.groups + r.share - 1) / r.share;
            const long long least = even < r.min_tiles ? even : r.min_tiles;
            if (C < least) C = least;
            if (C < 1) C = 1;
            for (int x = threadIdx.x; x < n_items * a.H; x += NT) r.count[x] = 0;
        }
        int units = 0, item0 = 0;
        for (int base = 0; base < a.N; base += NT) {
            const int n = base + (int)threadIdx.x;
            SeqWork w{0, 0};
            if (n < a.N) w = seq_work(a, p, i, extend_seq(a, n));
            const int ns = w.items > 0 ? (int)((w.tiles + C - 1) / C) : 1;
            int tot_u, tot_i;
            const int at = block_incl(w.items * ns, s_sums, &tot_u);
            const int it = block_incl(w.items, s_sums, &tot_i);
            s_at[threadIdx.x] = at - w.items * ns;
            s_items[threadIdx.x] = item0 + it - w.items;
            s_ns[threadIdx.x] = ns;
            if (threadIdx.x == NT - 1) s_at[NT] = at;
            __syncthreads();
            for (int u = threadIdx.x; u < tot_u; u += NT) {
                int l = 0, h = NT - 1;  // the last sequence that starts at or before u
                while (l < h) {
                    const int m = (l + h + 1) >> 1;
                    if (s_at[m] <= u) l = m;
                    else h = m - 1;
                }
                const int nsp = s_ns[l], local = u - s_at[l];
                ExtendUnit e;
                e.n = base + l;
                e.q0 = local / nsp * r.rows;
                e.split = local % nsp;
                e.nsplit = nsp;
                e.item = s_items[l] + local / nsp;
                const int at_u = units + u;
                e.part = nsp > 1 ? at_u - e.split : -1;
                const ExtendSeq sq = extend_seq(a, e.n);
                e.row0 = sq.row0;
                e.len = sq.len;
                e.ctx = sq.ctx;
                const ExtendKeys k = extend_keys(sq, e.q0, r.rows, r.tile, a.W, a.S);
                e.kt0 = (int)((long long)e.split * k.n / nsp);
                e.kt1 = (int)((long long)(e.split + 1) * k.n / nsp);
                if (at_u < r.cap_units) {
                    int4* to = reinterpret_cast<int4*>(r.units + at_u);
                    to[0] = make_int4(e.n, e.q0, e.kt0, e.kt1);
                    to[1] = make_int4(e.part, e.nsplit, e.split, e.item);
                    to[2] = make_int4(e.row0, e.len, e.ctx, 0);
                }
            }
            units += tot_u;
            item0 += tot_i;
            __syncthreads();
        }
        if (threadIdx.x == 0) *r.n_units = units < r.cap_units ? units : r.cap_units;
    }
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

ExtendPlan extend_plan(int M, int N, int H, int dk, int dv, int max_len, bool bf16) {
    ExtendPlan p;
    if (max_len > M) max_len = M;
    auto route = [&](int i, int rows, int part_rows, int tile, int groups, int target, int share, int min_tiles,
                     int64_t items) {
        ExtendRoute& r = p.r[i];
        r.rows = rows;
        r.tile = tile;
        r.groups = groups;
        r.part_rows = part_rows;
        r.target = target;
        r.share = share;
        r.min_tiles = min_tiles;
        r.cap_items = (int)items;
        // split units: at most one per query tile and target / groups more (sum of ceil(t / C))
        const int split = 2 * (target / groups + 1);
        r.cap_units = items > split ? (int)items : split;
        r.cap_parts = split;
    };
    const int sms = device_sm_count();
    if (bf16 && dk == 128 && dv == 128 && max_len <= kFewRows) {
        // One CTA per SM. Units of equal length come in whole rounds, so a few rounds waste part of the
        // last one; more, shorter units waste less and add parts of at most max_len rows per head.
        const int few = max_len < kFewRows ? max_len : kFewRows;
        route(0, kFewRows, few, kFewTile, (H + kFewHeads - 1) / kFewHeads, few <= 4 ? 8 * sms : 2 * sms, sms, 8, N);
        return p;
    }
    // CUDA cores: 16 queries a tile while every sequence has few, else 64
    const int rows = max_len <= 16 ? 16 : 64;
    int64_t items = (int64_t)M / rows + N;
    if (items > M) items = M;
    route(0, rows, rows, 64, H, 4 * sms, sms, 1, items);
    return p;
}

size_t extend_bind(ExtendPlan& p, int H, int dv, void* workspace) {
    char* w = static_cast<char*>(workspace);
    size_t at = 256;
    for (int i = 0; i < 2; ++i) {
        ExtendRoute& r = p.r[i];
        if (r.rows == 0) continue;
        r.n_units = reinterpret_cast<int*>(w) + i;
        auto take = [&](size_t bytes) {
            char* q = w + at;
            at += up(bytes);
            return q;
        };
        r.units = reinterpret_cast<ExtendUnit*>(take((size_t)r.cap_units * sizeof(ExtendUnit)));
        // counters exist for split tiles only, and those are fewer than target / groups
        r.count = reinterpret_cast<int*>(take((size_t)r.cap_parts * H * sizeof(int)));
        r.part_ml = reinterpret_cast<float2*>(take((size_t)r.cap_parts * H * r.part_rows * sizeof(float2)));
        r.part_o = reinterpret_cast<float*>(take((size_t)r.cap_parts * H * r.part_rows * dv * sizeof(float)));
    }
    return at;
}

size_t swska_extend_workspace_size(int M, int N, int H, int dk, int dv, int max_len, bool bf16) {
    ExtendPlan p = extend_plan(M, N, H, dk, dv, max_len, bf16);
    return extend_bind(p, H, dv, nullptr);
}

cudaError_t swska_extend_launch(const ExtendArgs& a, bool bf16, cudaStream_t s) {
    ExtendPlan p = extend_plan(a.M, a.N, a.H, a.d_k, a.d_v, a.max_len, bf16);
    extend_bind(p, a.H, a.d_v, a.workspace);
    const int64_t chunks = a.k_new ? (int64_t)a.M * (a.d_k + a.H * a.d_v) * a.es / 16 : 0;
    const int64_t want = (chunks + NT - 1) / NT, cap = 8 * (int64_t)device_sm_count();
    extend_prepare_kernel<<<1 + (unsigned)(want < cap ? want : cap), NT, 0, s>>>(a, p);
    note_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (p.r[0].tile == kFewTile) return swska_extend_few_launch(a, p.r[0], s);
    return swska_extend_simt_launch(a, p.r[0], bf16, s);
}

unsigned swska_extend_take_timeout_flag() { return swska_extend_few_take_timeout_flag(); }

}  // namespace rod
