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

// inclusive scan of a pair over the block, with the block's sums
struct Pair {
    int items;
    long long v;
};
__device__ __forceinline__ Pair block_incl(Pair x, Pair* sums, Pair* total) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x.items, d);
        const long long z = __shfl_up_sync(0xffffffffu, x.v, d);
        if (lane >= d) {
            x.items += y;
            x.v += z;
        }
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    Pair all{0, 0};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const Pair t = sums[w];
        if (w < warp) {
            x.items += t.items;
            x.v += t.v;
        }
        all.items += t.items;
        all.v += t.v;
    }
    *total = all;
    return x;
}

// query tiles and, at most, key tiles per query tile of a sequence on route i (0 tiles: not on it);
// rows and tile are powers of two
struct SeqWork {
    int items, tiles;
};
__device__ __forceinline__ SeqWork seq_work(const ExtendArgs& a, const ExtendPlan& p, int i, const ExtendSeq& s) {
    const ExtendRoute& r = p.r[i];
    SeqWork w{0, 0};
    if (s.len == 0 || s.bad) return w;
    const bool is_short = p.r[0].rows != 0 && (s.len <= p.short_len || p.r[1].rows == 0);
    if (is_short != (i == 0)) return w;
    const int rl = __ffs(r.rows) - 1, tl = __ffs(r.tile) - 1;
    w.items = (s.len + r.rows - 1) >> rl;
    // the widest query tile: a window and the tile's rows, at any alignment, and the first tokens
    const int rows = s.len < r.rows ? s.len : r.rows;
    const int64_t span = (int64_t)(a.W < s.ctx + s.len ? a.W : s.ctx + s.len) + rows;
    const int most = (int)((span + r.tile - 1) >> tl) + 1 + ((a.S + r.tile - 1) >> tl);
    const int all = ((s.ctx + s.len - 1) >> tl) + 1;
    w.tiles = most < all ? most : all;
    return w;
}

__global__ void __launch_bounds__(NT) extend_prepare_kernel(const ExtendArgs a, const ExtendPlan p) {
    // the attention kernel may set itself up meanwhile; it waits for this launch's end before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x >= 2) {
        // ---- new keys and values to their slots, a warp per token
        const int ck = a.d_k * a.es / 16, cv = a.d_v * a.es / 16, vl = __ffs(cv) - 1, per = ck + a.H * cv;  // 16-byte pieces
        const int64_t slots = (int64_t)a.P * a.page;
        const int lane = threadIdx.x % 32;
        for (int row = (int)(blockIdx.x - 2) * NW + (int)threadIdx.x / 32; row < a.M; row += (int)(gridDim.x - 2) * NW) {
            const int64_t slot = a.slot[row];
            if (slot < 0 || slot >= slots) continue;
            const int pg = (int)slot / a.page, off = (int)slot - pg * a.page;
            const uint4* kn = static_cast<const uint4*>(a.k_new) + (int64_t)row * ck;
            const uint4* vn = static_cast<const uint4*>(a.v_new) + (int64_t)row * a.H * cv;
            uint4* kp = static_cast<uint4*>(a.k_pool) + slot * ck;
            uint4* vp = static_cast<uint4*>(a.v_pool) + ((int64_t)pg * a.H * a.page + off) * cv;
#pragma unroll 4
            for (int c = lane; c < per; c += 32) {
                if (c < ck) kp[c] = kn[c];
                else vp[(int64_t)((c - ck) >> vl) * a.page * cv + ((c - ck) & (cv - 1))] = vn[c - ck];
            }
        }
        return;
    }
    if (blockIdx.x == 1 && p.r[1].rows == 0) return;
    __shared__ ExtendSeq s_seq[NT];  // the block of sequences at hand
    __shared__ Pair s_sums[NW];
    __shared__ int s_at[NT];         // first unit of each
    __shared__ int s_item[NT];       // first query tile
    __shared__ unsigned s_v[NT];     // first key tile in the line
    __shared__ unsigned s_most, s_rows;  // the largest query tile: key tiles, and key tiles x rows
    __shared__ unsigned s_tiles[NT]; // key tiles in the line of each of its query tiles
    // ---- rows of sequences at impossible positions (block 0); s_seq for both
    for (int base = 0; base < a.N; base += NT) {
        const int n = base + (int)threadIdx.x;
        ExtendSeq mine{0, 0, 0, false};
        if (n < a.N) mine = extend_seq(a, n);
        s_seq[threadIdx.x] = mine;
        if (!__syncthreads_or(mine.bad) || blockIdx.x > 0) continue;
        for (int m = 0; m < NT; ++m) {
            const ExtendSeq s = s_seq[m];
            if (!s.bad) continue;
            const int64_t lo = (int64_t)s.row0 * a.H * a.d_v, n_o = (int64_t)s.len * a.H * a.d_v;
            for (int64_t i = threadIdx.x; i < n_o; i += NT) {
                if (a.es == 2) static_cast<unsigned short*>(a.o)[lo + i] = 0x7fff;
                else static_cast<unsigned*>(a.o)[lo + i] = 0x7fffffffu;
            }
        }
        __syncthreads();
    }
    // ---- the units of route blockIdx.x; s_seq has every sequence if they are one block
    const bool one_block = a.N <= NT;
    {
        const int i = blockIdx.x;
        const ExtendRoute& r = p.r[i];
        for (int x = threadIdx.x; x < r.cols * a.H; x += NT) r.count[x] = 0;
        // this thread's sequence of a block: its query tiles and what each takes of the line
        auto work_at = [&](int base, int shift, unsigned* t) {
            const int n = base + (int)threadIdx.x;
            SeqWork w{0, 0};
            if (n < a.N) {
                if (!one_block) s_seq[threadIdx.x] = extend_seq(a, n);
                w = seq_work(a, p, i, s_seq[threadIdx.x]);
            }
            *t = w.items ? (unsigned)(w.tiles >> shift) + (shift > 0) : 0u;
            return w;
        };
        // the line of all key tiles; lengths are halved until it fits 31 bits (a split is proportional)
        int shift = 0;
        unsigned t = 0;
        SeqWork w{0, 0};
        Pair at{0, 0}, tot{0, 0}, all;
        for (;; ++shift) {
            all = Pair{0, 0};
            for (int base = 0; base < a.N; base += NT) {
                w = work_at(base, shift, &t);
                at = block_incl(Pair{w.items, (long long)w.items * t}, s_sums, &tot);
                all.items += tot.items;
                all.v += tot.v;
            }
            if (all.v < 0x7fffffff) break;
        }
        // No query tile for this route: nothing to divide. Rows of two sequences at once (cu_seqlens that falls) could
        // make more query tiles than there is room for: then nothing is computed
        if (all.items == 0 || all.items > r.cap_items) {
            for (int c = threadIdx.x; c < r.cols; c += NT) reinterpret_cast<int2*>(r.range)[c] = make_int2(1, 0);
            return;
        }
        // Even chunks cost r.split_cost key tiles more (parts to write and add). Whole query tiles, dealt
        // out with the longest one's room for each, are taken where that is less.
        if (threadIdx.x == 0) s_most = s_rows = 0;
        __syncthreads();
        for (int base = 0; base < a.N; base += NT) {
            if (!one_block) work_at(base, shift, &t);
            const int len = t > 0 ? s_seq[threadIdx.x].len : 0;
            const unsigned most = __reduce_max_sync(0xffffffffu, t);
            const unsigned rows = __reduce_max_sync(0xffffffffu, t * (unsigned)(len < r.rows ? len : r.rows));
            if (threadIdx.x % 32 == 0 && most > 0) {
                atomicMax(&s_most, most);
                atomicMax(&s_rows, rows);
            }
        }
        __syncthreads();
        const unsigned t_max = s_most;
        unsigned V = (unsigned)all.v;
        const unsigned even = (V + r.cols - 1) / r.cols, rounds = ((unsigned)all.items + r.cols - 1) / r.cols;
        unsigned Q = even > (unsigned)r.min_chunk ? even : r.min_chunk;
        // Small batches: a part's rows are read back by the one that adds them, so n chunks of a tile of x key
        // tiles take a CTA x / n tiles' time and then n parts' rows; n = sqrt(x / rows) is least for the two. (Chunks of
        // at least two key tiles and so: one sequence of 16 tokens with W 4096 80.1 and 37.1 us, of 8 46.9 and 27.8, of
        // 2 21.4 and 18.3; of 16 with W 500 22.9 and 18.9. Half and twice the divisor: within 10% of that.)
        if (r.rows_div > 0) {
            const unsigned q = (unsigned)ceilf(sqrtf((float)s_rows / (float)r.rows_div));
            Q = q > Q ? q : Q;
        }
        const bool whole = (unsigned long long)rounds * t_max <= (unsigned long long)Q + r.split_cost;
        if (whole) {
            Q = rounds * t_max;
            V = (unsigned)all.items * t_max;
        }
        unsigned v_done = 0;
        int i_done = 0;
        for (int base = 0; base < a.N; base += NT) {
            if (!one_block) {
                w = work_at(base, shift, &t);
                at = block_incl(Pair{w.items, (long long)w.items * t}, s_sums, &tot);
            }
            if (whole) {
                t = w.items ? t_max : 0;
                at.v = (long long)at.items * t_max;
                tot.v = (long long)tot.items * t_max;
            }
            const int it = i_done + at.items - w.items;
            const unsigned v0 = v_done + (unsigned)at.v - w.items * t;
            s_item[threadIdx.x] = it;
            s_v[threadIdx.x] = v0;
            s_at[threadIdx.x] = it + (int)(v0 / Q);
            s_tiles[threadIdx.x] = t;
            __syncthreads();
            const int last = min(NT, a.N - base) - 1;
            // the sequence of the block at a place of an array of firsts (ties: the last, which has items)
            auto find = [&](auto* first, auto x) {
                int l = 0, h = last;
                while (l < h) {
                    const int m = (l + h + 1) >> 1;
                    if (first[m] <= x) l = m;
                    else h = m - 1;
                }
                return l;
            };
            const unsigned vb = v_done, ve = v_done + (unsigned)tot.v;
            for (int c = threadIdx.x; c < r.cols; c += NT) {
                const unsigned long long b64 = (unsigned long long)c * Q;
                if (b64 >= V) {
                    if (base == 0) reinterpret_cast<int2*>(r.range)[c] = make_int2(1, 0);
                    continue;
                }
                const unsigned b = (unsigned)b64, e = (V - b > Q ? b + Q : V) - 1;
                if (b >= vb && b < ve) {
                    const int l = find(s_v, b);
                    r.range[2 * c] = s_item[l] + (int)((b - s_v[l]) / s_tiles[l]);
                }
                if (e >= vb && e < ve) {
                    const int l = find(s_v, e);
                    r.range[2 * c + 1] = s_item[l] + (int)((e - s_v[l]) / s_tiles[l]);
                }
            }
            const int id_end = tot.items > 0 ? i_done + tot.items - 1 + (int)((ve - 1) / Q) : -1;
            for (int id = s_at[0] + (int)threadIdx.x; id <= id_end; id += NT) {
                const int l = find(s_at, id);
                const ExtendSeq sq = s_seq[l];
                const unsigned t2 = s_tiles[l], vs = s_v[l];
                if (t2 == 0) continue;
                int lo = 0, hi = ((sq.len + r.rows - 1) >> (__ffs(r.rows) - 1)) - 1;
                while (lo < hi) {  // the query tile: the last whose first unit is at or before id
                    const int m = (lo + hi + 1) >> 1;
                    if (s_item[l] + m + (int)((vs + m * t2) / Q) <= id) lo = m;
                    else hi = m - 1;
                }
                const unsigned b = vs + lo * t2, e = b + t2 - 1, c = (unsigned)(id - s_item[l] - lo);
                const unsigned c0 = b / Q, c1 = e / Q;
                if (c < c0 || c > c1) continue;  // a cut between two tiles: no unit there
                const ExtendKeys k = extend_keys(sq, lo * r.rows, r.rows, r.tile, a.W, a.S);
                const unsigned x0 = c * Q > b ? c * Q - b : 0, x1 = t2 < (c + 1) * Q - b ? t2 : (c + 1) * Q - b;
                const int kt0 = (int)((unsigned long long)x0 * k.n / t2), kt1 = (int)((unsigned long long)x1 * k.n / t2);
                // parts of chunk x: 2 x for its first query tile, 2 x + 1 for a later one (its last)
                const int first = 2 * (int)c0 + (c0 * Q == b ? 0 : 1);
                const bool split = c0 != c1;
                int4* to = reinterpret_cast<int4*>(r.units + id);
                to[0] = make_int4(base + l, lo * r.rows, kt0, kt1);
                to[1] = make_int4(split ? (c == c0 ? first : 2 * (int)c) : -1, split ? first : -1, (int)c0, (int)(c1 - c0 + 1));
                to[2] = make_int4(sq.row0, sq.len, sq.ctx, (int)c1);
            }
            v_done += (unsigned)tot.v;
            i_done += tot.items;
            __syncthreads();
        }
    }
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

ExtendPlan extend_plan(int M, int N, int H, int dk, int dv, int max_len, bool bf16) {
    ExtendPlan p;
    if (max_len > M) max_len = M;
    // ctas: about what the GPU holds at once (on CUDA cores with d 128 half of them fit: two rounds)
    auto route = [&](int i, int rows, int part_rows, int tile, int groups, int ctas, int min_chunk, int rows_div, int split_cost,
                     int64_t items) {
        ExtendRoute& r = p.r[i];
        r.rows = rows;
        r.part_rows = part_rows;
        r.tile = tile;
        r.groups = groups;
        r.cols = ctas / groups > 1 ? ctas / groups : 1;
        r.min_chunk = min_chunk;
        r.rows_div = rows_div;
        r.split_cost = split_cost;
        r.cap_items = (int)(items < M ? items : M);
    };
    const int sms = device_sm_count();
    if (bf16 && dk == 128 && dv == 128) {
        const int few = max_len < kFewRows ? max_len : kFewRows;
        // Up to four heads a CTA, two CTAs an SM, or up to eight and one: eight fetch a key tile once for
        // all, four put twice the CTAs to work on small batches and leave each less to add up. H 16, W 4096:
        // 17.5 us for 2 sequences with eight, 16.9 with four; 59.5 both for 16; 177 and 183 for 64, 335 and
        // 346 for 128 (short runs)
        const int heads = (int64_t)N * ((H + kFewHeads - 1) / kFewHeads) >= 48 ? kFewHeads : kFewHeads / 2;
        const int groups = (H + heads - 1) / heads, hpg = (H + groups - 1) / groups;
        route(0, kFewRows, few, kFewTile, groups, (hpg <= kFewHeads / 2 ? 2 : 1) * sms, 2, 16, 6, N);
        p.short_len = kFewRows;
        // A cut in a tile's keys costs the parts' way through memory, 128 rows of 128 columns of 32 bits a head
        // each, so whole query tiles are dealt out unless even chunks save more than twelve key tiles a CTA.
        // With three and with twelve: 33 sequences of mixed lengths 66.8 and 52.4 us, one of 512 tokens with
        // W 1000 44.8 and 37.8, twelve of 250 with H 5 47.5 and 40.0; one chunk with W 4096 is cut either way
        if (max_len > kFewRows)
            route(1, kChunkRows, kChunkRows, kChunkTile, (H + 1) / 2, sms, 4, 0, 12, (int64_t)M / kChunkRows + N);
        return p;
    }
    // CUDA cores: 16 queries a tile while every sequence has few, else 64
    const int rows = max_len <= 16 ? 16 : 64;
    route(0, rows, rows, 64, H, (rows == 16 ? 4 : 2) * sms, 1, 0, 1, (int64_t)M / rows + N);
    return p;
}

size_t extend_bind(ExtendPlan& p, int H, int dv, void* workspace) {
    char* w = static_cast<char*>(workspace);
    size_t at = 0;
    for (int i = 0; i < 2; ++i) {
        ExtendRoute& r = p.r[i];
        if (r.rows == 0) continue;
        auto take = [&](size_t bytes) {
            char* q = w + at;
            at += up(bytes);
            return q;
        };
        const size_t parts = (size_t)2 * r.cols * H * r.part_rows;
        r.units = reinterpret_cast<ExtendUnit*>(take((size_t)(r.cap_items + r.cols) * sizeof(ExtendUnit)));
        r.range = reinterpret_cast<int*>(take((size_t)r.cols * 2 * sizeof(int)));
        r.count = reinterpret_cast<int*>(take((size_t)r.cols * H * sizeof(int)));
        r.part_ml = reinterpret_cast<float2*>(take(parts * sizeof(float2)));
        r.part_o = reinterpret_cast<float*>(take(parts * dv * sizeof(float)));
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
    const int want = a.k_new ? (a.M + NW - 1) / NW : 0, cap = 8 * device_sm_count();
    extend_prepare_kernel<<<2 + (unsigned)(want < cap ? want : cap), NT, 0, s>>>(a, p);
    note_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (p.r[0].tile == kFewTile) {
        e = swska_extend_few_launch(a, p.r[0], s);
        return e == cudaSuccess && p.r[1].rows ? swska_extend_tc_launch(a, p.r[1], s) : e;
    }
    return swska_extend_simt_launch(a, p.r[0], bf16, s);
}

unsigned swska_extend_take_timeout_flag() {
    return swska_extend_few_take_timeout_flag() | swska_extend_tc_take_timeout_flag();
}

}  // namespace rod
