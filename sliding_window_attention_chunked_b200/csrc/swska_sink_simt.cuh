// swska_sink_simt.cuh -- SW-SKA with first tokens that stay visible, forward and backward in fp32 on
// CUDA cores (every product an fp32 FMA).
//
// Query t sees the keys j <= t with j > t - W or j < S:
//   p_tj = softmax_j(scale q_t . k_j),  o_t = sum_j p_tj v_j,  lse_t = log sum_j exp(scale q_t . k_j)
//   D_t = dO_t . o_t,  dS_tj = p_tj (dO_t . v_j - D_t)
//   dq_t = scale sum_j dS_tj k_j,  dv_j = sum_t p_tj dO_t,  dk_j = scale sum_h sum_t dS_tj q_t
// One CTA per 32 queries of a head (forward, dq) or per 32 keys of a head (dk, dv), with the tiles of
// simt_tile.cuh; it visits the tiles that its rows can see and masks inside them. What a tile costs is
// mostly waiting (loads, then products of a few warps), so up to four groups of 128 threads share a
// CTA's tiles in turn, each with its own buffers and sums, which are added at the end in the order of
// the groups (fp32, T 1000, 4 heads, d_k 64, d_v 128, window 256: one group of 256 threads and 64 rows a
// CTA takes 215 us a step). The
// kernels are bound by FMA issue: a 64 x 64 tile of head dim 128 is 1 M FMAs per product against 64 KB
// of tile loads that stay in L2.
//
// A key tile among the first S is seen by every later query, up to T / W times the work of another
// tile. Its queries past the window are dealt out in segments to further CTAs, each with its own
// partial sums for the S rows; the last launch adds the parts in a fixed order, so the result does
// not depend on timing. The same launch adds the heads' parts of the shared dk.
#pragma once

#include <math.h>

#include "kernels.h"
#include "simt_tile.cuh"
#include "sink_parts.cuh"

namespace rod {
namespace {

using namespace simt;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ROWS rows of D floats that follow one another into rows of D + 4, by asynchronous 16-byte copies that are all
// in flight at once; rows from n on are zeros. A commit ends a set of them
template <int D, int ROWS, int NTH>
__device__ __forceinline__ void copy_tile(float* s, const float* from, int n, int tid = threadIdx.x) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(s);
    if (ROWS * (D / 4) < NTH && tid >= ROWS * (D / 4)) return;
#pragma unroll
    for (int e = 0; e < (ROWS * (D / 4) + NTH - 1) / NTH; ++e) {
        const int i = tid + e * NTH, r = i / (D / 4);
        if (ROWS * (D / 4) % NTH != 0 && i >= ROWS * (D / 4)) break;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + 16 * (i + r)), "l"(r < n ? from + 4 * i : from),
                     "r"(r < n ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void copies_sent() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LATER> __device__ __forceinline__ void copies_here() { asm volatile("cp.async.wait_group %0;" ::"n"(LATER) : "memory"); }

constexpr int BQ = 32;
constexpr int NTH = 4 * BQ;  // threads of a group
// groups that fit: `own` floats for all, `each` per group, 227 KB in all
constexpr int groups_for(int own, int each) {
    const int n = (56 * 1024 - own) / each;
    return n < 4 ? n : 4;
}
// forward: Q | per group K, V, P
template <int DK, int DV> struct Fwd {
    static constexpr int own = BQ * ld<DK>(), each = BK * (ld<DK>() + ld<DV>()) + BQ * LDP;
    static constexpr int NG = groups_for(own, each), smem = (own + NG * each) * 4;
};
// dq: Q, dO | per group K, V, dS
template <int DK, int DV> struct Dq {
    static constexpr int own = BQ * (ld<DK>() + ld<DV>()), each = BK * (ld<DK>() + ld<DV>()) + BQ * LDP;
    static constexpr int NG = groups_for(own, each), smem = (own + NG * each) * 4;
};
// dk, dv: K, V | per group Q, dO, P, log-sum-exp, D, e
template <int DK, int DV> struct Dkv {
    static constexpr int own = BQ * (ld<DK>() + ld<DV>()), each = BK * (ld<DK>() + ld<DV>()) + BQ * LDP + 3 * BK;
    static constexpr int NG = groups_for(own, each), smem = (own + NG * each) * 4;
    static_assert(2 * BK == NTH, "a thread of the group per log-sum-exp and D of a tile");
};

// a group's sums (rows 4 ty + i, N columns a thread) to and from its buffers
template <int N>
__device__ __forceinline__ void put_sums(float* w, int tid, const float acc[4][N]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < N; ++c) w[(i * N + c) * NTH + tid] = acc[i][c];
}
template <int N>
__device__ __forceinline__ void add_sums(const float* w, int tid, float acc[4][N]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < N; ++c) acc[i][c] += w[(i * N + c) * NTH + tid];
}

// key tiles of a query tile: those of the first S keys that lie before the window's, then the window's
struct KeyTiles {
    int n_sink, lo, n;
    __device__ __forceinline__ int at(int i) const { return i < n_sink ? i : lo + i - n_sink; }
};
__device__ __forceinline__ KeyTiles key_tiles(int t0, int t1, int W, int S) {
    KeyTiles k;
    k.lo = (t0 - W + 1 > 0 ? t0 - W + 1 : 0) / BK;
    const int ns = (S + BK - 1) / BK;
    k.n_sink = ns < k.lo ? ns : k.lo;
    k.n = k.n_sink + t1 / BK - k.lo + 1;
    return k;
}

template <int DK, int DV>
__global__ void __launch_bounds__(NTH * Fwd<DK, DV>::NG)
sink_fwd_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                float* __restrict__ o, float* __restrict__ lse, int H, int T, int W, int S, float scale_log2,
                int qtiles) {
    constexpr int NG = Fwd<DK, DV>::NG, N = DV / 16;
    extern __shared__ __align__(16) float sm[];
    const int g = threadIdx.x / NTH, tid = threadIdx.x % NTH;
    float* sQ = sm;
    float* mine = sm + Fwd<DK, DV>::own + g * Fwd<DK, DV>::each;
    float* sK = mine;
    float* sV = sK + BK * ld<DK>();
    float* sP = sV + BK * ld<DV>();
    const int64_t bh = blockIdx.x / qtiles, b = bh / H;
    const int t0 = (qtiles - 1 - (int)(blockIdx.x % qtiles)) * BQ;
    const int tx = tid % 16, ty = tid / 16;
    const int t1 = (t0 + BQ < T ? t0 + BQ : T) - 1;
    const KeyTiles kt = key_tiles(t0, t1, W, S);
    auto send_k = [&](int it) {
        const int key0 = it < kt.n ? kt.at(it) * BK : T;
        if (key0 < T) copy_tile<DK, BK, NTH>(sK, k + (b * (int64_t)T + key0) * (int64_t)DK, T - key0, tid);
        copies_sent();
    };
    auto send_v = [&](int it) {
        const int key0 = it < kt.n ? kt.at(it) * BK : T;
        if (key0 < T) copy_tile<DV, BK, NTH>(sV, v + (bh * T + key0) * (int64_t)DV, T - key0, tid);
        copies_sent();
    };
    copy_tile<DK, BQ, NTH * NG>(sQ, q + (bh * T + t0) * (int64_t)DK, T - t0);
    send_k(g);
    send_v(g);
    copies_here<1>();
    __syncthreads();
    float m[4], l[4], acc[4][N];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < N; ++c) acc[i][c] = 0.f;
    }
    for (int it = g; it < kt.n; it += NG) {
        const int key0 = kt.at(it) * BK;
        copies_here<1>();
        group_sync<NTH>(g);
        float s[4][4];
        tile_dot<DK>(sQ, sK, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[i][j] = ska_visible(t0 + 4 * ty + i, key0 + tx + 16 * j, W, S) ? s[i][j] * scale_log2 : -INFINITY;
        softmax_step<N>(s, m, l, acc);
        put_tile(sP, ty, tx, s);
        copies_here<0>();
        group_sync<NTH>(g);
        send_k(it + NG);
        tile_mul<DV>(sP, sV, ty, tx, acc);
        group_sync<NTH>(g);
        send_v(it + NG);
    }
    if (NG > 1) {
        __syncthreads();
        if (g > 0) {
            put_sums<N>(mine, tid, acc);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mine[(4 * N + i) * NTH + tid] = m[i];
                mine[(4 * N + 4 + i) * NTH + tid] = l[i];
            }
        }
        __syncthreads();
        if (g > 0) return;
        for (int x = 1; x < NG; ++x) {
            const float* w = mine + x * Fwd<DK, DV>::each;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float mx = w[(4 * N + i) * NTH + tid], lx = w[(4 * N + 4 + i) * NTH + tid];
                const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
                const float a0 = exp2f(m[i] - base), a1 = exp2f(mx - base);
                m[i] = mn;
                l[i] = fmaf(l[i], a0, lx * a1);
#pragma unroll
                for (int c = 0; c < N; ++c) acc[i][c] = fmaf(acc[i][c], a0, w[(i * N + c) * NTH + tid] * a1);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + 4 * ty + i;
        if (t >= T) continue;
        const float inv = 1.f / l[i];
#pragma unroll
        for (int c = 0; c < N; ++c)
            o[(bh * T + t) * (int64_t)DV + Cols<DV>::at(tx, c)] = acc[i][c] * inv;
        if (tx == 0) lse[bh * T + t] = (m[i] + log2f(l[i])) * kLn2;
    }
}

template <int DK, int DV>
__global__ void __launch_bounds__(NTH * Dq<DK, DV>::NG)
sink_dq_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
               const float* __restrict__ o, const float* __restrict__ lse, const float* __restrict__ dO,
               float* __restrict__ dq, float* __restrict__ dbuf, float* __restrict__ ebuf, int H, int T, int W, int S, float scale,
               int qtiles) {
    constexpr int NG = Dq<DK, DV>::NG;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the key side may set itself up
    extern __shared__ __align__(16) float sm[];
    const int g0 = threadIdx.x / NTH, tid = threadIdx.x % NTH;
    float* sQ = sm;
    float* sG = sQ + BQ * ld<DK>();
    float* mine = sm + Dq<DK, DV>::own + g0 * Dq<DK, DV>::each;
    float* sK = mine;
    float* sV = sK + BK * ld<DK>();
    float* sP = sV + BK * ld<DV>();
    const int64_t bh = blockIdx.x / qtiles, b = bh / H;
    const int t0 = (qtiles - 1 - (int)(blockIdx.x % qtiles)) * BQ;
    const int tx = tid % 16, ty = tid / 16;
    const int t1 = (t0 + BQ < T ? t0 + BQ : T) - 1;
    const float scale_log2 = scale * kLog2e;
    const KeyTiles kt = key_tiles(t0, t1, W, S);
    auto send_k = [&](int it) {
        const int key0 = it < kt.n ? kt.at(it) * BK : T;
        if (key0 < T) copy_tile<DK, BK, NTH>(sK, k + (b * (int64_t)T + key0) * (int64_t)DK, T - key0, tid);
        copies_sent();
    };
    auto send_v = [&](int it) {
        const int key0 = it < kt.n ? kt.at(it) * BK : T;
        if (key0 < T) copy_tile<DV, BK, NTH>(sV, v + (bh * T + key0) * (int64_t)DV, T - key0, tid);
        copies_sent();
    };
    // D = dO . o of a row, summed by one thread in tile_dot's order: where a row gives one key all of its
    // attention, o is that key's v and dP - D is exactly 0, not the difference of two roundings (shared out over
    // 16 threads a row, dq and dk of rows that see one key were 1e-7 |dO| |v| of noise). The rows of o wait in the dS
    // tiles, 64 columns to a group's.
    // Where all keys of the CTA's rows lie in one tile, what D is off by, e = sum_j p_j (dP_j - D), is taken out too (sum_j dS_j = 0):
    // dS = p ((dP - D) - e), whose terms are small where attention is peaked (dq of two tokens, the first drawing attention, was
    // off by up to 1e-3 of its norm). With more tiles dq would need a second sweep, for rows that such peaks are few of.
    static_assert(DV <= BK || NG >= 2, "room for the rows of o");
    float* sO = sm + Dq<DK, DV>::own + BK * (ld<DK>() + ld<DV>());
    auto o_at = [&](int r, int c) { return sO + (c / BK) * Dq<DK, DV>::each + r * LDP + c % BK; };
    for (int i = threadIdx.x; i < BQ * (DV / 4); i += NTH * NG) {
        const int r = i / (DV / 4), c = 4 * (i % (DV / 4)), t = t0 + r < T ? t0 + r : t0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(o_at(r, c))),
                     "l"(o + (bh * T + t) * (int64_t)DV + c), "r"(t0 + r < T ? 16 : 0)
                     : "memory");
    }
    copy_tile<DV, BQ, NTH * NG>(sG, dO + (bh * T + t0) * (int64_t)DV, T - t0);
    copy_tile<DK, BQ, NTH * NG>(sQ, q + (bh * T + t0) * (int64_t)DK, T - t0);
    send_v(g0);
    send_k(g0);
    copies_here<1>();
    __syncthreads();
    if (threadIdx.x < BQ) {
        const int r = threadIdx.x;
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int d = 0; d < DV; d += 4) {
            const float4 x = *reinterpret_cast<const float4*>(sG + r * ld<DV>() + d), y = *reinterpret_cast<const float4*>(o_at(r, d));
            sum = fx::f2fma(make_float2(x.x, x.y), make_float2(y.x, y.y), sum);
            sum = fx::f2fma(make_float2(x.z, x.w), make_float2(y.z, y.w), sum);
        }
        sO[r * LDP + BK] = sum.x + sum.y;  // in the row's pad
        if (t0 + r < T) dbuf[bh * T + t0 + r] = sum.x + sum.y;
    }
    __syncthreads();
    float L2[4], D[4], e[4] = {0.f, 0.f, 0.f, 0.f}, acc[4][DK / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i, t = t0 + r;
        D[i] = sO[r * LDP + BK];
        L2[i] = t < T ? lse[bh * T + t] * kLog2e : INFINITY;  // rows past the end: p = 0
#pragma unroll
        for (int c = 0; c < DK / 16; ++c) acc[i][c] = 0.f;
    }
    for (int it = g0; it < kt.n; it += NG) {
        const int key0 = kt.at(it) * BK;
        copies_here<1>();
        group_sync<NTH>(g0);
        float s[4][4], g[4][4];
        tile_dot<DV>(sG, sV, ty, tx, g);
        copies_here<0>();
        group_sync<NTH>(g0);
        send_v(it + NG);
        tile_dot<DK>(sQ, sK, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool see = ska_visible(t0 + 4 * ty + i, key0 + tx + 16 * j, W, S);
                g[i][j] -= D[i];
                s[i][j] = see ? exp2f(fmaf(s[i][j], scale_log2, -L2[i])) : 0.f;
            }
        if (kt.n == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) e[i] = fmaf(s[i][j], g[i][j], e[i]);
                e[i] = row_sum(e[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] *= g[i][j] - e[i];
        put_tile(sP, ty, tx, s);
        group_sync<NTH>(g0);
        tile_mul<DK>(sP, sK, ty, tx, acc);
        group_sync<NTH>(g0);
        send_k(it + NG);
    }
    if (NG > 1) {
        __syncthreads();
        if (g0 > 0) {
            put_sums<DK / 16>(mine, tid, acc);
        }
        __syncthreads();
        if (g0 > 0) return;
        for (int x = 1; x < NG; ++x) {
            const float* w = mine + x * Dq<DK, DV>::each;
            add_sums<DK / 16>(w, tid, acc);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + 4 * ty + i;
        if (t >= T) continue;
        if (tx == 0) ebuf[bh * T + t] = e[i];
#pragma unroll
        for (int c = 0; c < DK / 16; ++c)
            dq[(bh * T + t) * (int64_t)DK + Cols<DK>::at(tx, c)] = acc[i][c] * scale;
    }
}

// blockIdx.x: for each sequence and head, its key tiles, then (tile s, segment g) of the first tokens' far queries
template <int DK, int DV>
__global__ void __launch_bounds__(NTH * Dkv<DK, DV>::NG)
sink_dkv_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                const float* __restrict__ lse, const float* dbuf, const float* ebuf, const float* __restrict__ dO,
                float* __restrict__ dv, SinkParts parts, int B, int H, int T, int W, int S, float scale) {
    constexpr int NG = Dkv<DK, DV>::NG;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the launch that adds the parts waits for the end
    extern __shared__ __align__(16) float sm[];
    const int g0 = threadIdx.x / NTH, tid = threadIdx.x % NTH;
    float* sK = sm;
    float* sV = sK + BQ * ld<DK>();
    float* mine = sm + Dkv<DK, DV>::own + g0 * Dkv<DK, DV>::each;
    float* sQ = mine;
    float* sG = sQ + BK * ld<DK>();
    float* sP = sG + BK * ld<DV>();
    float* sL = sP + BQ * LDP;
    float* sD = sL + BK;
    float* sE = sD + BK;
    const int tiles = parts.ctas();
    const int64_t bh = blockIdx.x / tiles;
    const int b = (int)bh / H, h = (int)bh - b * H;
    const int tx = tid % 16, ty = tid / 16;
    const SinkWork w = parts.work((int)blockIdx.x - (int)bh * tiles);
    const int key0 = w.tile * BQ;
    auto send_g = [&](int qt) {
        const int t0 = qt * BK;
        if (qt <= w.q_hi) copy_tile<DV, BK, NTH>(sG, dO + (bh * T + t0) * (int64_t)DV, T - t0, tid);
        copies_sent();
    };
    auto send_q = [&](int qt) {
        const int t0 = qt * BK;
        if (qt <= w.q_hi) {
            copy_tile<DK, BK, NTH>(sQ, q + (bh * T + t0) * (int64_t)DK, T - t0, tid);
            const int x = tid % BK;  // half of the threads: log-sum-exp, the others: D (2 BK = NTH)
            const float* from = (tid < BK ? lse : dbuf) + (t0 + x < T ? bh * T + t0 + x : 0);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared((tid < BK ? sL : sD) + x)),
                         "l"(from), "r"(t0 + x < T ? 4 : 0)
                         : "memory");
            if (tid < BK)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(sE + x)),
                             "l"(ebuf + (t0 + x < T ? bh * T + t0 + x : 0)), "r"(t0 + x < T ? 4 : 0)
                             : "memory");
        }
        copies_sent();
    };
    copy_tile<DV, BQ, NTH * NG>(sV, v + (bh * T + key0) * (int64_t)DV, T - key0);
    copy_tile<DK, BQ, NTH * NG>(sK, k + (b * (int64_t)T + key0) * (int64_t)DK, T - key0);
    send_g(w.q_lo + g0);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the query side's D
    send_q(w.q_lo + g0);
    copies_here<1>();
    __syncthreads();
    const float scale_log2 = scale * kLog2e;
    float ak[4][DK / 16], av[4][DV / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int c = 0; c < DK / 16; ++c) ak[i][c] = 0.f;
#pragma unroll
        for (int c = 0; c < DV / 16; ++c) av[i][c] = 0.f;
    }
    for (int qt = w.q_lo + g0; qt <= w.q_hi; qt += NG) {
        const int t0 = qt * BK;
        copies_here<1>();
        group_sync<NTH>(g0);
        float s[4][4], g[4][4];  // rows: keys, columns: queries
        tile_dot<DV>(sV, sG, ty, tx, g);
        copies_here<0>();
        group_sync<NTH>(g0);
        tile_dot<DK>(sK, sQ, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = tx + 16 * j;
                const bool see = t0 + c < T && ska_visible(t0 + c, key0 + 4 * ty + i, W, S);
                s[i][j] = see ? exp2f(fmaf(s[i][j], scale_log2, -kLog2e * sL[c])) : 0.f;
                g[i][j] = s[i][j] * ((g[i][j] - sD[c]) - sE[c]);
            }
        put_tile(sP, ty, tx, s);
        group_sync<NTH>(g0);
        tile_mul<DV>(sP, sG, ty, tx, av);
        group_sync<NTH>(g0);
        send_g(qt + NG);
        put_tile(sP, ty, tx, g);
        group_sync<NTH>(g0);
        tile_mul<DK>(sP, sQ, ty, tx, ak);
        group_sync<NTH>(g0);
        send_q(qt + NG);
    }
    if (NG > 1) {
        __syncthreads();
        if (g0 > 0) {
            put_sums<DK / 16>(mine, tid, ak);
            put_sums<DV / 16>(mine + 4 * (DK / 16) * NTH, tid, av);
        }
        __syncthreads();
        if (g0 > 0) return;
        for (int x = 1; x < NG; ++x) {
            add_sums<DK / 16>(mine + x * Dkv<DK, DV>::each, tid, ak);
            add_sums<DV / 16>(mine + x * Dkv<DK, DV>::each + 4 * (DK / 16) * NTH, tid, av);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int key = key0 + 4 * ty + i;
        if (key >= T) continue;
        const bool part = parts.nseg > 0 && key < S;
#pragma unroll
        for (int c = 0; c < DV / 16; ++c) {
            const int col = Cols<DV>::at(tx, c);
            if (part) parts.dv_at(w.slot, bh, key)[col] = av[i][c];
            else if (w.slot == 0) dv[(bh * T + key) * (int64_t)DV + col] = av[i][c];
        }
#pragma unroll
        for (int c = 0; c < DK / 16; ++c) {
            const int col = Cols<DK>::at(tx, c);
            if (w.slot == 0) parts.dk_part[(((int64_t)h * B + b) * T + key) * DK + col] = ak[i][c];
            else if (part) parts.dk_at(w.slot, h, b, key)[col] = ak[i][c];
        }
    }
}

const float* f32(const void* p) { return static_cast<const float*>(p); }

template <int DK, int DV>
cudaError_t fwd_t(const SinkArgs& a, cudaStream_t s) {
    using F = Fwd<DK, DV>;
    const int qtiles = (a.T + BQ - 1) / BQ;
    const int64_t grid = (int64_t)qtiles * a.B * a.H;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_smem(smem_set, (const void*)sink_fwd_kernel<DK, DV>, F::smem);
    if (e != cudaSuccess) return e;
    sink_fwd_kernel<DK, DV><<<(unsigned)grid, NTH * F::NG, F::smem, s>>>(
        f32(a.q), f32(a.k), f32(a.v), static_cast<float*>(a.out), a.lse_out, a.H, a.T, a.W, a.S, a.scale * kLog2e, qtiles);
    note_launches(1);
    return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t bwd_t(const SinkArgs& a, cudaStream_t s) {
    using Q = Dq<DK, DV>;
    using K = Dkv<DK, DV>;
    const int qtiles = (a.T + BQ - 1) / BQ;
    SinkParts parts = sink_parts_plan(a, BQ, BK, a.H);
    float* dbuf = sink_parts_bind(parts, a);
    float* ebuf = dbuf + (size_t)a.B * a.H * a.T;  // the second array of row statistics
    const int64_t grid = (int64_t)qtiles * a.B * a.H, key_grid = (int64_t)parts.ctas() * a.B * a.H;
    if (grid > 0x7fffffffLL || key_grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaError_t e;
    static std::atomic<uint64_t> q_set{0}, k_set{0};
    if ((e = allow_smem(q_set, (const void*)sink_dq_kernel<DK, DV>, Q::smem)) != cudaSuccess) return e;
    if ((e = allow_smem(k_set, (const void*)sink_dkv_kernel<DK, DV>, K::smem)) != cudaSuccess) return e;
    sink_dq_kernel<DK, DV><<<(unsigned)grid, NTH * Q::NG, Q::smem, s>>>(
        f32(a.q), f32(a.k), f32(a.v), f32(a.o), a.lse, f32(a.dO), static_cast<float*>(a.dq), dbuf, ebuf, a.H, a.T, a.W, a.S, a.scale, qtiles);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_overlapped(sink_dkv_kernel<DK, DV>, dim3((unsigned)key_grid), dim3(NTH * K::NG),
                          K::smem, s, f32(a.q), f32(a.k), f32(a.v), a.lse, static_cast<const float*>(dbuf),
                          static_cast<const float*>(ebuf), f32(a.dO),
                          static_cast<float*>(a.dv), parts, a.B, a.H, a.T, a.W, a.S, a.scale);
    note_launches(2);
    if (e != cudaSuccess) return e;
    return sink_parts_reduce(parts, a, false, s);
}

template <int DK>
cudaError_t pick_dv(const SinkArgs& a, bool backward, cudaStream_t s) {
    switch (a.d_v) {
        case 16: return backward ? bwd_t<DK, 16>(a, s) : fwd_t<DK, 16>(a, s);
        case 32: return backward ? bwd_t<DK, 32>(a, s) : fwd_t<DK, 32>(a, s);
        case 64: return backward ? bwd_t<DK, 64>(a, s) : fwd_t<DK, 64>(a, s);
        case 128: return backward ? bwd_t<DK, 128>(a, s) : fwd_t<DK, 128>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

// forward or backward for one key head dim (an instance each in swska_sink_simt_<dk>.cu, which
// compile side by side)
template <int DK>
cudaError_t sink_simt_launch(const SinkArgs& a, bool backward, cudaStream_t s);

}  // namespace rod
