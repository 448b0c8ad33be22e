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
constexpr int kClusterMax = 8;

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

// Inclusive scan of one value per thread over the block; every thread also gets the block's sum.
__device__ long long block_incl(long long x, long long* warp_sums, long long* total) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    x = warp_incl(x, lane);
    __syncthreads();  // the previous use of warp_sums is over
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const long long w = warp_incl(lane < NW ? warp_sums[lane] : 0, lane);
        if (lane < NW) warp_sums[lane] = w;
    }
    __syncthreads();
    if (warp > 0) x += warp_sums[warp - 1];
    *total = warp_sums[NW - 1];
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

// what one sequence gives back and wants; pages are counted by the warp that owns the sequence
struct Range {
    int rel_lo, rel_hi;  // logical pages that may go back
    int want_lo, want_hi;
    bool active, done, fits;
    int low;
};
__device__ __forceinline__ Range range_of(const TableArgs& a, int n) {
    Range r;
    const int64_t c = a.ctx[n];
    const int m = a.n_new[n];
    const int sp = (a.S + a.page - 1) / a.page;
    r.active = m > 0 && c >= 0;
    r.done = m < 0 && c >= 0;
    const int64_t used = (c + a.page - 1) / a.page, end = (c + (m > 0 ? m : 0) + a.page - 1) / a.page;
    int64_t low = (c - a.W + 1 > 0 ? c - a.W + 1 : 0) / a.page;
    low = low > sp ? low : sp;
    low = low < used ? low : used;
    low = low < a.max_pages ? low : a.max_pages;
    const int f = a.first[n];
    r.low = (int)low;
    r.rel_lo = r.done ? 0 : (f > sp ? f : sp);
    r.rel_hi = r.done ? a.max_pages : (r.active ? (int)low : 0);
    r.fits = r.active && end <= a.max_pages;
    r.want_lo = r.fits ? (int)used : 0;
    r.want_hi = r.fits ? (int)end : 0;
    return r;
}

__global__ void __launch_bounds__(NT, 1) page_tables_kernel(const TableArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per = (a.N + CL - 1) / CL;                       // sequences per CTA
    const int n0 = min(a.N, rank * per), n1 = min(a.N, n0 + per);

    extern __shared__ int32_t sh[];
    // own sequences: pages back, pages wanted, and the ranks where they start; all sequences: cu
    int32_t* s_rel = sh;
    int32_t* s_need = s_rel + per;
    int32_t* s_relat = s_need + per;
    int32_t* s_takeat = s_relat + per;  // -1: not served
    int32_t* s_cu = s_takeat + per;     // [N + 1]
    __shared__ long long warp_sums[NW];
    __shared__ Sums s_tot;              // this CTA's sums of the first exchange
    __shared__ long long s_tot2[2];     // pages taken and tokens served, of the second

    int count0 = *a.free_count;
    count0 = count0 < 0 ? 0 : (count0 > a.P ? a.P : count0);
    const unsigned P = (unsigned)a.P;

    // ---- counts: a warp per sequence
    for (int n = n0 + warp; n < n1; n += NW) {
        const Range r = range_of(a, n);
        const int32_t* row = a.table + (int64_t)n * a.max_pages;
        int rel = 0, need = 0;
        for (int p = r.rel_lo + lane; p < r.rel_hi; p += 32) rel += (unsigned)row[p] < P;
        for (int p = r.want_lo + lane; p < r.want_hi; p += 32) need += (unsigned)row[p] >= P;
        rel = __reduce_add_sync(0xffffffffu, rel);
        need = __reduce_add_sync(0xffffffffu, need);
        if (lane == 0) {
            s_rel[n - n0] = rel;
            s_need[n - n0] = need;
        }
    }
    __syncthreads();
    // ---- this CTA's sums
    {
        Sums t{0, 0, 0};
        for (int i = threadIdx.x; i < n1 - n0; i += NT) {
            const int m = a.n_new[n0 + i];
            t.rel += s_rel[i];
            t.need += s_need[i];
            t.tok += (m > 0 && a.ctx[n0 + i] >= 0) ? m : 0;
        }
        long long all;
        block_incl(t.rel, warp_sums, &all);
        if (threadIdx.x == 0) s_tot.rel = all;
        block_incl(t.need, warp_sums, &all);
        if (threadIdx.x == 0) s_tot.need = all;
        block_incl(t.tok, warp_sums, &all);
        if (threadIdx.x == 0) s_tot.tok = all;
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
    long long run_rel = 0, run_need = 0, run_tok = 0, run_take = 0, run_served = 0;
    for (int base = 0; base < n1 - n0; base += NT) {
        const int i = base + (int)threadIdx.x;
        const bool in = i < n1 - n0;
        const int n = n0 + i;
        const int m = in ? a.n_new[n] : 0;
        const bool active = in && m > 0 && a.ctx[n] >= 0;
        const int rel = in ? s_rel[i] : 0, need = in ? s_need[i] : 0;
        long long tot_rel, tot_need, tot_tok, tot_take, tot_served;
        const long long at_rel = block_incl(rel, warp_sums, &tot_rel);
        const long long at_need = block_incl(need, warp_sums, &tot_need);
        const long long at_tok = block_incl(active ? m : 0, warp_sums, &tot_tok);
        bool ok = false;
        if (active)
            ok = range_of(a, n).fits && before.tok + run_tok + at_tok <= a.M &&
                 (need == 0 || before.need + run_need + at_need <= avail);
        const long long at_take = block_incl(ok ? need : 0, warp_sums, &tot_take);
        const long long at_served = block_incl(ok ? m : 0, warp_sums, &tot_served);
        if (in) {
            s_relat[i] = (int)(run_rel + at_rel - rel);
            s_takeat[i] = ok ? (int)(run_take + at_take - need) : -1;
            s_cu[n + 1] = (int)(run_served + at_served);  // relative to this CTA until the second exchange
        }
        run_rel += tot_rel;
        run_need += tot_need;
        run_tok += tot_tok;
        run_take += tot_take;
        run_served += tot_served;
    }
    if (threadIdx.x == 0) {
        s_tot2[0] = run_take;
        s_tot2[1] = run_served;
    }
    __syncthreads();
    // ---- pages back: onto the stack
    for (int n = n0 + warp; n < n1; n += NW) {
        const Range r = range_of(a, n);
        int32_t* row = a.table + (int64_t)n * a.max_pages;
        long long at = count0 + before.rel + s_relat[n - n0];
        __syncwarp();
        for (int p0 = r.rel_lo; p0 < r.rel_hi; p0 += 32) {
            const int p = p0 + lane;
            const int32_t e = p < r.rel_hi ? row[p] : -1;
            const bool held = (unsigned)e < P;
            const unsigned who = __ballot_sync(0xffffffffu, held);
            const long long to = at + __popc(who & ((1u << lane) - 1u));
            if (held && to < a.P) a.free_list[to] = e;
            if (p < r.rel_hi) row[p] = -1;
            at += __popc(who);
        }
        if (lane == 0) {
            if (r.done) a.first[n] = 0;
            else if (r.active && a.first[n] < r.low) a.first[n] = r.low;
        }
    }
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
    for (int n = n0 + warp; n < n1; n += NW) {
        const int takeat = s_takeat[n - n0];
        if (takeat < 0) continue;  // the whole warp
        const Range r = range_of(a, n);
        int32_t* row = a.table + (int64_t)n * a.max_pages;
        long long j = take0 + takeat;
        for (int p0 = r.want_lo; p0 < r.want_hi; p0 += 32) {
            const int p = p0 + lane;
            const bool lack = p < r.want_hi && (unsigned)row[p] >= P;
            const unsigned who = __ballot_sync(0xffffffffu, lack);
            const long long from = top - 1 - (j + __popc(who & ((1u << lane) - 1u)));
            if (lack) row[p] = from >= 0 ? __ldcg(a.free_list + from) : -1;
            j += __popc(who);
        }
    }
    for (int i = threadIdx.x; i < n1 - n0; i += NT) a.cu[n0 + i + 1] = (int)(served0 + s_cu[n0 + i + 1]);
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
            int n = lo, seen_n = -1, seen_p = -1;
            int32_t e = -1;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u;
                if (i >= total) break;
                while (s_cu[n + 1] <= i) ++n;  // past sequences without tokens too
                const unsigned pos = (unsigned)(a.ctx[n] + (i - s_cu[n]));
                const int p = (int)(pos / (unsigned)a.page);
                if (n != seen_n || p != seen_p) {
                    e = __ldcg(a.table + (int64_t)n * a.max_pages + p);
                    seen_n = n;
                    seen_p = p;
                }
                if ((unsigned)e < P) out[u] = e * a.page + (int)(pos - (unsigned)p * (unsigned)a.page);
            }
        }
        if (i0 + 4 <= a.M) {
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
    // one CTA has a warp for each of 32 sequences and writes 4096 slots in one sweep; more work
    // than that takes the largest portable cluster
    const int CL = N <= NW && M <= 4 * NT ? 1 : kClusterMax;
    const int per = (N + CL - 1) / CL;
    const size_t smem = ((size_t)4 * per + N + 1) * sizeof(int32_t);
    cudaError_t e = cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
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
