// swska_page_tables.cu -- block tables, free list and slot map of a paged SW-SKA cache, built on
// the GPU from each sequence's cached and new lengths.
//
// A page holds page_size tokens; entry i of a sequence's row of the block table is the physical
// page of its positions i * page_size .. (i + 1) * page_size - 1, or -1 (SALA blog §3.3: a paged KV
// cache split into small blocks that are allocated on demand and evicted by window). With c
// cached and m new tokens, window W and S first tokens that stay visible, the next query sits at
// position c and sees no key below lo = c - W + 1 except the first S, so
//   pages back  : held entries in [max(first, ceil(S / page)), lo / page)   (a finished
//                 sequence, m < 0: every held entry of its row)
//   pages wanted: entries in [ceil(c / page), ceil((c + m) / page)) that hold none yet
// The free list is a stack. Pages given back are pushed in (sequence, position) order, then the
// j-th page wanted pops the j-th entry from the top, so the result is one fixed function of the
// inputs: the ranks come from prefix sums over the sequences, not from atomics.
//
// What bounds it is latency: a decode step of 256 sequences touches about 10 KB. One launch of
// one thread-block cluster does it all: a warp per sequence counts, the CTAs exchange their sums
// through distributed shared memory, and cluster barriers stand where a page pushed by one CTA
// may be popped by another. Two launches (counts, then writes) would each cost about what the
// whole kernel does. The slot map is written by all CTAs together, four tokens to a thread, so
// that one long sequence is not one CTA's work.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace rod {
namespace {

constexpr int NT = 1024;
constexpr int NW = NT / 32;
constexpr int kClusterMax = 16;  // opt-in: 8 is the portable size

struct Sums {
    long long rel, need, tok;
};

__device__ __forceinline__ long long warp_incl(long long x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    return x;
}

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

struct TableArgs {
    const int64_t* ctx;
    const int32_t* n_new;
    int32_t* table;
    int32_t* first;
    int32_t* free_list;
    int32_t* free_count;
    int32_t* cu;
    int32_t* slot;
    int N, max_pages, P, page, W, S, M;
};

// what one sequence gives back and wants, as logical pages. Positions are clamped to 2^31, past any
// row of the table (max_pages * page is below), so that the divisions are 32-bit ones.
struct Range {
    int rel_lo, rel_hi;    // pages that may go back
    int want_lo, want_hi;  // pages of the new tokens
    int first;             // new value of first
    int tokens;            // wanted; -1: the row has no room for them, -2: finished (walked by the whole CTA)
};
__device__ __forceinline__ Range range_of(const TableArgs& a, int64_t c, int m, int f) {
    Range r{0, 0, 0, 0, f, 0};
    if (c < 0 || m == 0) return r;
    if (m < 0) {
        r.rel_hi = a.max_pages;
        r.first = 0;
        return r;
    }
    const unsigned page = (unsigned)a.page, cap = 1u << 31;
    c = c < (1ll << 32) ? c : (1ll << 32);
    auto clamp = [&](int64_t x) { return x < 0 ? 0u : (x < (int64_t)cap ? (unsigned)x : cap); };
    const unsigned whole = (unsigned)a.S / page + ((unsigned)a.S % page != 0);  // S + page may pass 2^31
    const int sp = (int)(whole < (unsigned)a.max_pages ? whole : (unsigned)a.max_pages);
    const unsigned used = clamp(c) / page + (clamp(c) % page != 0);
    const unsigned end = clamp(c + m) / page + (clamp(c + m) % page != 0);
    unsigned low = clamp(c - a.W + 1) / page;
    low = low > (unsigned)sp ? low : (unsigned)sp;
    low = low < used ? low : used;
    low = low < (unsigned)a.max_pages ? low : (unsigned)a.max_pages;
    r.rel_lo = f > sp ? f : sp;
    r.rel_hi = (int)low;
    r.first = f > (int)low ? f : (int)low;
    const bool fits = end <= (unsigned)a.max_pages;
    r.want_lo = fits ? (int)used : 0;
    r.want_hi = fits ? (int)end : 0;
    r.tokens = fits ? m : -1;
    return r;
}

// entries of a row in [lo, hi) through the warp, UN x 32 at a time so that their loads overlap; take(p,
// e) gets each lane's entry (-1 outside the range)
template <int UN, typename F>
__device__ __forceinline__ void walk(const int32_t* row, int lo, int hi, int lane, F take) {
    for (int p0 = lo; p0 < hi; p0 += 32 * UN) {
        int32_t e[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int p = p0 + 32 * i + lane;
            e[i] = p < hi ? __ldcg(row + p) : -1;
        }
#pragma unroll
        for (int i = 0; i < UN; ++i)
            if (p0 + 32 * i < hi) take(p0 + 32 * i + lane, e[i]);
    }
}

__global__ void __launch_bounds__(NT, 1) page_tables_kernel(const TableArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per = (a.N + CL - 1) / CL;                       // sequences per CTA
    const int n0 = min(a.N, rank * per), n1 = min(a.N, n0 + per);

    extern __shared__ int32_t sh[];
    // own sequences: their ranges, pages back and wanted, and the ranks where these start; then all
    // sequences' cu and positions
    Range* s_range = reinterpret_cast<Range*>(sh);
    int32_t* s_rel = sh + 6 * per;
    int32_t* s_need = s_rel + per;
    int32_t* s_relat = s_need + per;
    int32_t* s_takeat = s_relat + per;  // -1: not served
    int32_t* s_cu = s_takeat + per;     // [N + 1]
    int32_t* s_ctx = s_cu + a.N + 1;    // [N]
    __shared__ Sums s_tot;              // this CTA's sums of the first exchange
    __shared__ long long s_tot2[2];     // pages taken and tokens served, of the second
    __shared__ int s_done[NT];          // finished sequences of this CTA, while they fit
    __shared__ int s_ndone;
    __shared__ int s_held[4][NW];

    int count0 = *a.free_count;
    count0 = count0 < 0 ? 0 : (count0 > a.P ? a.P : count0);
    const unsigned P = (unsigned)a.P;
    const int mine = n1 - n0;

    if (threadIdx.x == 0) s_ndone = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < mine; i += NT) {
        const int m = a.n_new[n0 + i];
        s_range[i] = range_of(a, a.ctx[n0 + i], m, a.first[n0 + i]);
        s_rel[i] = s_need[i] = 0;
        // a finished row is walked to its end: by all warps together (past NT of them, by one)
        if (s_range[i].rel_hi == a.max_pages && m < 0) {
            const int d = atomicAdd(&s_ndone, 1);
            if (d < NT) {
                s_done[d] = i;
                s_range[i].tokens = -2;
            }
        }
    }
    // positions of the slot map: a served one is below 2^31
    for (int n = threadIdx.x; n < a.N; n += NT) s_ctx[n] = (int32_t)a.ctx[n];
    __syncthreads();
    const int n_done = min(s_ndone, NT);
    // ---- counts: a warp per sequence
    for (int i = warp; i < mine; i += NW) {
        const Range r = s_range[i];
        if (r.tokens == -2) continue;
        const int32_t* row = a.table + (int64_t)(n0 + i) * a.max_pages;
        int rel = 0, need = 0;
        walk<4>(row, r.rel_lo, r.rel_hi, lane, [&](int, int32_t e) { rel += (unsigned)e < P; });
        walk<4>(row, r.want_lo, r.want_hi, lane, [&](int p, int32_t e) { need += p < r.want_hi && (unsigned)e >= P; });
        rel = __reduce_add_sync(0xffffffffu, rel);
        need = __reduce_add_sync(0xffffffffu, need);
        if (lane == 0) {
            s_rel[i] = rel;
            s_need[i] = need;
        }
    }
    for (int d = 0; d < n_done; ++d) {
        const int32_t* row = a.table + (int64_t)(n0 + s_done[d]) * a.max_pages;
        int rel = 0;
#pragma unroll 4
        for (int p = threadIdx.x; p < a.max_pages; p += NT) rel += (unsigned)__ldcg(row + p) < P;
        rel = __reduce_add_sync(0xffffffffu, rel);
        if (lane == 0 && rel > 0) atomicAdd(&s_rel[s_done[d]], rel);
    }
    __syncthreads();
    // ---- this CTA's sums (tokens wanted count whether or not they fit)
    if (warp == 0) {
        Sums t{0, 0, 0};
        for (int i = lane; i < mine; i += 32) {
            const int tokens = s_range[i].tokens;
            t.rel += s_rel[i];
            t.need += s_need[i];
            t.tok += tokens == 0 || tokens == -2 ? 0 : a.n_new[n0 + i];
        }
        t.rel = warp_sum(t.rel);
        t.need = warp_sum(t.need);
        t.tok = warp_sum(t.tok);
        if (lane == 0) s_tot = t;
    }
    cluster.sync();
    Sums before{0, 0, 0};
    long long R = 0;
    for (int c = 0; c < CL; ++c) {
        const Sums t = *cluster.map_shared_rank(&s_tot, c);
        if (c < rank) {
            before.rel += t.rel;
            before.need += t.need;
            before.tok += t.tok;
        }
        R += t.rel;
    }
    const long long avail = (long long)count0 + R;

    // ---- which sequences are served, and the ranks inside this CTA
    if (warp == 0) {
        long long run_rel = 0, run_need = before.need, run_tok = before.tok, run_take = 0, run_served = 0;
        for (int base = 0; base < mine; base += 32) {
            const int i = base + lane;
            const bool in = i < mine;
            const int tokens = in ? s_range[i].tokens : 0;
            const int m = tokens == 0 || tokens == -2 ? 0 : a.n_new[n0 + i];
            const int rel = in ? s_rel[i] : 0, need = in ? s_need[i] : 0;
            const long long at_rel = run_rel + warp_incl(rel, lane), at_need = run_need + warp_incl(need, lane),
                            at_tok = run_tok + warp_incl(m, lane);
            const bool ok = tokens > 0 && at_tok <= a.M && (need == 0 || at_need <= avail);
            const long long at_take = run_take + warp_incl(ok ? need : 0, lane);
            const long long at_served = run_served + warp_incl(ok ? m : 0, lane);
            if (in) {
                s_relat[i] = (int)(at_rel - rel);
                s_takeat[i] = ok ? (int)(at_take - need) : -1;
                s_cu[n0 + i + 1] = (int)at_served;  // relative to this CTA until the second exchange
            }
            run_rel = __shfl_sync(0xffffffffu, at_rel, 31);
            run_need = __shfl_sync(0xffffffffu, at_need, 31);
            run_tok = __shfl_sync(0xffffffffu, at_tok, 31);
            run_take = __shfl_sync(0xffffffffu, at_take, 31);
            run_served = __shfl_sync(0xffffffffu, at_served, 31);
        }
        if (lane == 0) {
            s_tot2[0] = run_take;
            s_tot2[1] = run_served;
        }
    }
    __syncthreads();
    // ---- pages back: onto the stack
    for (int i = warp; i < mine; i += NW) {
        const Range r = s_range[i];
        if (r.tokens == -2) continue;
        int32_t* row = a.table + (int64_t)(n0 + i) * a.max_pages;
        long long at = count0 + before.rel + s_relat[i];
        walk<4>(row, r.rel_lo, r.rel_hi, lane, [&](int p, int32_t e) {
            const bool held = (unsigned)e < P;
            const unsigned who = __ballot_sync(0xffffffffu, held);
            const long long to = at + __popc(who & ((1u << lane) - 1u));
            if (held && to < a.P) a.free_list[to] = e;
            if (e != -1) row[p] = -1;
            at += __popc(who);
        });
    }
    for (int d = 0; d < n_done; ++d) {
        int32_t* row = a.table + (int64_t)(n0 + s_done[d]) * a.max_pages;
        long long at = count0 + before.rel + s_relat[s_done[d]];
        for (int p0 = 0; p0 < a.max_pages; p0 += 4 * NT) {
            int32_t e[4];
            unsigned who[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int p = p0 + k * NT + (int)threadIdx.x;
                e[k] = p < a.max_pages ? __ldcg(row + p) : -1;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                who[k] = __ballot_sync(0xffffffffu, (unsigned)e[k] < P);
                if (lane == 0) s_held[k][warp] = __popc(who[k]);
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = s_held[k][lane];
                const int all = __reduce_add_sync(0xffffffffu, c);
                if (all > 0) {
                    const long long to = at + __reduce_add_sync(0xffffffffu, lane < warp ? c : 0) + __popc(who[k] & ((1u << lane) - 1u));
                    if ((unsigned)e[k] < P && to < a.P) a.free_list[to] = e[k];
                }
                if (e[k] != -1) row[p0 + k * NT + (int)threadIdx.x] = -1;
                at += all;
            }
            __syncthreads();
        }
    }
    for (int i = threadIdx.x; i < mine; i += NT) a.first[n0 + i] = s_range[i].first;
    // stack entries written by the other CTAs are visible after this barrier
    cluster.sync();
    long long take0 = 0, served0 = 0, A = 0, total = 0;
    for (int c = 0; c < CL; ++c) {
        const long long* t = cluster.map_shared_rank(s_tot2, c);
        if (c < rank) {
            take0 += t[0];
            served0 += t[1];
        }
        A += t[0];
        total += t[1];
    }
    const long long top = avail < a.P ? avail : a.P;
    // ---- pages wanted: off the stack
    for (int i = warp; i < mine; i += NW) {
        const int takeat = s_takeat[i];
        if (takeat < 0 || s_need[i] == 0) continue;  // the whole warp
        const Range r = s_range[i];
        int32_t* row = a.table + (int64_t)(n0 + i) * a.max_pages;
        long long j = take0 + takeat;
        walk<4>(row, r.want_lo, r.want_hi, lane, [&](int p, int32_t e) {
            const bool lack = p < r.want_hi && (unsigned)e >= P;
            const unsigned who = __ballot_sync(0xffffffffu, lack);
            const long long from = top - 1 - (j + __popc(who & ((1u << lane) - 1u)));
            if (lack) row[p] = from >= 0 ? __ldcg(a.free_list + from) : -1;
            j += __popc(who);
        });
    }
    for (int i = threadIdx.x; i < mine; i += NT) a.cu[n0 + i + 1] = (int)(served0 + s_cu[n0 + i + 1]);
    if (rank == 0 && threadIdx.x == 0) {
        a.cu[0] = 0;
        *a.free_count = (int)(top - A > 0 ? top - A : 0);
    }
    // tables and cu are complete for every CTA after this barrier
    cluster.sync();
    for (int n = threadIdx.x; n <= a.N; n += NT) s_cu[n] = __ldcg(a.cu + n);
    __syncthreads();
    // ---- slot map: four tokens to a thread
    const int64_t quads = ((int64_t)a.M + 3) / 4;
    for (int64_t qd = (int64_t)rank * NT + threadIdx.x; qd < quads; qd += (int64_t)CL * NT) {
        const int i0 = (int)(4 * qd);
        int32_t out[4] = {-1, -1, -1, -1};
        if (i0 < total) {
            int lo = 0, hi = a.N - 1;  // the last n with cu[n] <= i0
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_cu[mid] <= i0) lo = mid;
                else hi = mid - 1;
            }
            // one division per four tokens: the others step through the pages
            int n = lo, left = s_cu[n + 1] - i0, p = 0, off = 0;
            int32_t e = -1;
            bool go = true;  // (n, p) is new: its table entry is not loaded yet
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (i0 + u >= total) break;
                if (u == 0 || left == 0) {
                    while (s_cu[n + 1] <= i0 + u) ++n;  // past sequences without tokens too
                    const unsigned pos = (unsigned)s_ctx[n] + (unsigned)(i0 + u - s_cu[n]);
                    p = (int)(pos / (unsigned)a.page);
                    off = (int)(pos - (unsigned)p * (unsigned)a.page);
                    left = s_cu[n + 1] - (i0 + u);
                    go = true;
                } else if (off == a.page) {
                    ++p;
                    off = 0;
                    go = true;
                }
                if (go) e = __ldcg(a.table + (int64_t)n * a.max_pages + p);
                go = false;
                if ((unsigned)e < P) out[u] = e * a.page + off;
                ++off;
                --left;
            }
        }
        if (a.M - i0 >= 4) {  // i0 + 4 may pass 2^31
            *reinterpret_cast<int4*>(a.slot + i0) = make_int4(out[0], out[1], out[2], out[3]);
        } else {
            for (int u = 0; i0 + u < a.M; ++u) a.slot[i0 + u] = out[u];
        }
    }
}

}  // namespace

cudaError_t swska_page_tables_launch(const int64_t* ctx, const int32_t* n_new, int32_t* table, int32_t* first,
                                     int32_t* free_list, int32_t* free_count, int32_t* cu, int32_t* slot, int N,
                                     int max_pages, int P, int page, int W, int S, int M, cudaStream_t stream) {
    const TableArgs a{ctx, n_new, table, first, free_list, free_count, cu, slot, N, max_pages, P, page, W, S, M};
    // A CTA has a warp for each of 32 sequences and writes 4096 slots in one sweep. Clusters of 1, 8 and
    // 16: the smallest that does all in one go, else 16 (256 decode sequences: 19.6 us with 8 CTAs, 22.3
    // with 16, whose barriers take longer; 512 sequences with 180,000 new tokens: 39 and 33 us)
    const int CL = N <= NW && M <= 4 * NT ? 1 : (N <= 8 * NW && M <= 8 * 4 * NT ? 8 : kClusterMax);
    const int per = (N + CL - 1) / CL;
    const size_t smem = ((size_t)10 * per + 2 * (size_t)N + 1) * sizeof(int32_t);
    static std::atomic<uint64_t> smem_set{0};
    constexpr int kMost = (10 * (kMaxTableSeqs / kClusterMax) + 2 * kMaxTableSeqs + 1) * (int)sizeof(int32_t);  // CL = 16 there
    static_assert(kMost <= 220 * 1024, "shared memory");
    cudaError_t e = allow_smem(smem_set, (const void*)page_tables_kernel, kMost);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> cluster_set{0};
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if (dev >= 64 || !(cluster_set.load(std::memory_order_relaxed) >> dev & 1)) {
        if ((e = cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
        if (dev < 64) cluster_set.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CL);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)CL;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, page_tables_kernel, a);
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rod
