// swska_sink_mma.cuh -- SW-SKA with first tokens that stay visible, forward and backward in bf16 for the
// shapes outside the tcgen05 kernels (head dims of 16, 32, 64, sequences below 128): warp-level
// m16n8k16 products, fp32 accumulators.
//
// The formulas are those of swska_sink_simt.cuh. A CTA of four warps owns 64 queries of a head (forward,
// dq) or 64 keys of a head (dk, dv), 16 rows a warp, and visits tiles of 64 rows of the other side,
// which arrive by 16-byte asynchronous copies into one of two stages while the other is used. Rows
// in shared memory are padded by 16 bytes, so that the eight rows of a fragment load fall into
// different banks for every head dim. The kernels are bound by the latency of a tile's chain (copy, score
// product, exponentials, second product): several CTAs an SM overlap theirs. A tcgen05 tile of 128 x 128
// would leave most of itself empty at these sizes.
// Probabilities and dS go to the second products in bf16 (relative 2^-9 each, as the inputs). dS = p (dP -
// D) is a small difference where a row's attention is peaked, and D from the rounded o is off by about
// 2^-9 of it. So, as in swska_backward_tc.cu, dq sums e = sum p (dP - D) of its rows in fp32 on the
// way, visits the first tile (where attention with first tokens peaks) last, with D + e, and sweeps
// again where some p of another tile is above 1/2; the key side gets D + e. The first tokens' keys share the direction
// that draws the queries, and sum_j dS_j = 0 makes it cancel in dq, which the roundings of their dS do not: their tiles are
// multiplied by dS in two bf16 parts (dq was off by 2.8e-3 of its norm in place of 1.7e-3 at d 64, by 3.7e-3 at d 32).
#pragma once

#include <math.h>

#include "mma16.cuh"
#include "sink_parts.cuh"
#include "tc.cuh"

namespace rod {
namespace {

using mma::bits_from;
using mma::bits_to;
using mma::ldsm4;
using mma::ldsm4t;
using mma::mma16816;

constexpr int R = 64;          // rows of a CTA, and of the tiles it visits
constexpr int NTH = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
using bf16_t = __nv_bfloat16;

template <int D> constexpr int pitch() { return 2 * D + 16; }       // bytes of a padded row
template <int D> constexpr int tile_bytes() { return R * pitch<D>(); }

// rows row0 .. row0 + 63 of a [T][D] matrix, zeros past T
template <int D>
__device__ __forceinline__ void copy_tile(uint32_t dst, const bf16_t* m, int row0, int T) {
#pragma unroll
    for (int i = threadIdx.x; i < R * (D / 8); i += NTH) {
        const int r = i / (D / 8), c = i % (D / 8), row = row0 + r;
        const bf16_t* src = m + (int64_t)(row < T ? row : 0) * D + 8 * c;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + r * pitch<D>() + 16 * c), "l"(src),
                     "r"(row < T ? 16 : 0) : "memory");
    }
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the most recent group of copies have landed
__device__ __forceinline__ void wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// fragment addresses in a padded tile: A (16 rows), B from [n][k] rows (two 8-column tiles), B from
// [k][n] rows (transposed load, two 8-column tiles)
template <int D> __device__ __forceinline__ uint32_t a_at(uint32_t t, int row, int k, int lane) {
    return t + (row + (lane & 15)) * pitch<D>() + 32 * k + 16 * (lane >> 4);
}
template <int D> __device__ __forceinline__ uint32_t b_at(uint32_t t, int n, int k, int lane) {
    return t + (8 * n + (lane & 7) + ((lane >> 4) << 3)) * pitch<D>() + 32 * k + 16 * (lane >> 3 & 1);
}
template <int D> __device__ __forceinline__ uint32_t bt_at(uint32_t t, int n, int k, int lane) {
    return t + (16 * k + (lane & 15)) * pitch<D>() + 16 * (n + (lane >> 4));
}

// x[n] (16 x 64) = A (16 rows, fragments a) times the rows of tile t transposed
template <int D>
__device__ __forceinline__ void dot_tile(uint32_t t, const uint32_t (*a)[4], float (*x)[4], int lane) {
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
            uint32_t b[4];
            ldsm4(b_at<D>(t, n, k, lane), b);
            mma16816(x[n], a[k], b);
            mma16816(x[n + 1], a[k], b + 2);
        }
}
// the same with the fragments of A taken from rows of a tile on the way (registers are short)
template <int D>
__device__ __forceinline__ void dot_tiles(uint32_t t, uint32_t ta, int row, float (*x)[4], int lane) {
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        uint32_t a[4];
        ldsm4(a_at<D>(ta, row, k, lane), a);
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
            uint32_t b[4];
            ldsm4(b_at<D>(t, n, k, lane), b);
            mma16816(x[n], a, b);
            mma16816(x[n + 1], a, b + 2);
        }
    }
}
// acc (16 x D) += w (16 x 64, rounded to bf16) times tile t
template <int D>
__device__ __forceinline__ void mul_tile(uint32_t t, const float (*w)[4], float (*acc)[4], int lane) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t a[4];
        mma::to_a(w[2 * k], w[2 * k + 1], a);
#pragma unroll
        for (int n = 0; n < D / 8; n += 2) {
            uint32_t b[4];
            ldsm4t(bt_at<D>(t, n, k, lane), b);
            mma16816(acc[n], a, b);
            mma16816(acc[n + 1], a, b + 2);
        }
    }
}

struct KeyTiles {  // those of the first S keys that lie before the window's, then the window's
    int n_sink, lo, n;
    __device__ __forceinline__ int key0(int i) const { return (i < n_sink ? i : lo + i - n_sink) * R; }
};
__device__ __forceinline__ KeyTiles key_tiles(int t0, int T, int W, int S) {
    KeyTiles k;
    const int t1 = (t0 + R < T ? t0 + R : T) - 1;
    k.lo = (t0 - W + 1 > 0 ? t0 - W + 1 : 0) / R;
    k.n_sink = min((S + R - 1) / R, k.lo);
    k.n = k.n_sink + t1 / R - k.lo + 1;
    return k;
}
// scores of keys that a row does not see become -inf; rows t and t + 8
__device__ __forceinline__ void mask_keys(float (*s)[4], int t, int t0, int key0, int W, int S, int c2) {
    if (key0 + R - 1 <= t0 && (key0 > t0 + R - 1 - W || key0 + R <= S)) return;  // every row sees every key
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int p = t + 8 * e - key0;
        uint32_t v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            v[h] = bits_to(p - 32 * h) & (bits_from((int64_t)p - W + 1 - 32 * h) | bits_to(S - 1 - key0 - 32 * h));
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const uint32_t b = v[n / 4] >> (8 * (n % 4) + c2);
            if (!(b & 1u)) s[n][2 * e] = -INFINITY;
            if (!(b & 2u)) s[n][2 * e + 1] = -INFINITY;
        }
    }
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
template <int N>
__device__ __forceinline__ void store_rows(bf16_t* m, int t, int T, int D, const float (*acc)[4], const float f[2], int c2) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (t + 8 * e < T) {
            uint32_t* p = reinterpret_cast<uint32_t*>(m + (int64_t)(t + 8 * e) * D + c2);
#pragma unroll
            for (int n = 0; n < N; ++n) p[4 * n] = pack_bf16x2(acc[n][2 * e] * f[e], acc[n][2 * e + 1] * f[e]);
        }
}

// ---- forward ------------------------------------------------------------------------------------
template <int DK, int DV> constexpr int fwd_smem() { return tile_bytes<DK>() + 2 * (tile_bytes<DK>() + tile_bytes<DV>()); }

template <int DK, int DV>
__global__ void __launch_bounds__(NTH)
sink_mma_fwd_kernel(const bf16_t* __restrict__ q, const bf16_t* __restrict__ k, const bf16_t* __restrict__ v,
                    bf16_t* __restrict__ o, float* __restrict__ lse, int H, int T, int W, int S, float scale_log2, int qtiles) {
    extern __shared__ __align__(16) unsigned char sm[];
    const uint32_t sQ = smem_u32(sm), stage = sQ + tile_bytes<DK>();
    constexpr int STAGE = tile_bytes<DK>() + tile_bytes<DV>();
    const int64_t bh = blockIdx.x / qtiles, b = bh / H;
    const int t0 = (qtiles - 1 - (int)(blockIdx.x % qtiles)) * R;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c2 = 2 * (lane % 4);
    const int t = t0 + 16 * warp + lane / 4;  // this thread's rows: t, t + 8
    const bf16_t *kb = k + b * T * DK, *vb = v + bh * T * DV;
    const KeyTiles kt = key_tiles(t0, T, W, S);
    copy_tile<DK>(sQ, q + bh * T * DK, t0, T);
    auto fetch = [&](int i) {
        if (i < kt.n) {
            copy_tile<DK>(stage + (i & 1) * STAGE, kb, kt.key0(i), T);
            copy_tile<DV>(stage + (i & 1) * STAGE + tile_bytes<DK>(), vb, kt.key0(i), T);
        }
        copies_done();
    };
    fetch(0);
    fetch(1);
    uint32_t qa[DK / 16][4];
    float acc[DV / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < DV / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    for (int i = 0; i < kt.n; ++i) {
        wait_but_one();
        __syncthreads();
        if (i == 0) {
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) ldsm4(a_at<DK>(sQ, 16 * warp, kk, lane), qa[kk]);
        }
        const uint32_t sK = stage + (i & 1) * STAGE, sV = sK + tile_bytes<DK>();
        float s[8][4];
        dot_tile<DK>(sK, qa, s, lane);
        mask_keys(s, t, t0, kt.key0(i), W, S, c2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s[0][2 * e], s[0][2 * e + 1]);
#pragma unroll
            for (int n = 1; n < 8; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * e], s[n][2 * e + 1]));
            mx = quad_max(mx) * scale_log2;
            const float mn = fmaxf(m[e], mx), base = mn == -INFINITY ? 0.f : mn;
            const float alpha = tc::ex2(m[e] - base);
            m[e] = mn;
            l[e] *= alpha;
#pragma unroll
            for (int n = 0; n < DV / 8; ++n) {
                acc[n][2 * e] *= alpha;
                acc[n][2 * e + 1] *= alpha;
            }
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                s[n][2 * e] = tc::ex2(fmaf(s[n][2 * e], scale_log2, -base));
                s[n][2 * e + 1] = tc::ex2(fmaf(s[n][2 * e + 1], scale_log2, -base));
                l[e] += s[n][2 * e] + s[n][2 * e + 1];
            }
        }
        mul_tile<DV>(sV, s, acc, lane);
        __syncthreads();  // the stage is free
        fetch(i + 2);
    }
    float inv[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] = quad_sum(l[e]);
        inv[e] = 1.f / l[e];
        if (lane % 4 == 0 && t + 8 * e < T) lse[bh * T + t + 8 * e] = (m[e] + log2f(l[e])) * kLn2;
    }
    store_rows<DV / 8>(o + bh * T * DV, t, T, DV, acc, inv, c2);
}

// ---- dq, and D for the key side -------------------------------------------------------------------
template <int DK, int DV> constexpr int dq_smem() { return 3 * (tile_bytes<DK>() + tile_bytes<DV>()); }

template <int DK, int DV>
__global__ void __launch_bounds__(NTH, DK + DV <= 128 ? 3 : 1)
sink_mma_dq_kernel(const bf16_t* __restrict__ q, const bf16_t* __restrict__ k, const bf16_t* __restrict__ v,
                   const bf16_t* __restrict__ o, const float* __restrict__ lse, const bf16_t* __restrict__ dO,
                   bf16_t* __restrict__ dq, float* __restrict__ dbuf, int H, int T, int W, int S, float scale,
                   float grad_scale, int qtiles) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the key side may set itself up
    extern __shared__ __align__(16) unsigned char sm[];
    constexpr int STAGE = tile_bytes<DK>() + tile_bytes<DV>();
    const uint32_t sQ = smem_u32(sm), sG = sQ + tile_bytes<DK>(), stage = sQ + STAGE;
    const int64_t bh = blockIdx.x / qtiles, b = bh / H;
    const int t0 = (qtiles - 1 - (int)(blockIdx.x % qtiles)) * R;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c2 = 2 * (lane % 4);
    const int t = t0 + 16 * warp + lane / 4;
    const float scale_log2 = scale * kLog2e;
    const bf16_t *kb = k + b * T * DK, *vb = v + bh * T * DV;
    const KeyTiles kt = key_tiles(t0, T, W, S);
    copy_tile<DK>(sQ, q + bh * T * DK, t0, T);
    copy_tile<DV>(sG, dO + bh * T * DV, t0, T);
    auto key0_of = [&](int i) { return kt.key0(i + 1 < kt.n ? i + 1 : 0); };  // the first tile last
    auto fetch = [&](int i) {
        if (i < kt.n) {
            copy_tile<DK>(stage + (i & 1) * STAGE, kb, key0_of(i), T);
            copy_tile<DV>(stage + (i & 1) * STAGE + tile_bytes<DK>(), vb, key0_of(i), T);
        }
        copies_done();
    };
    fetch(0);
    fetch(1);
    float L2[2], D[2], e2[2] = {0.f, 0.f}, p_max = 0.f, acc[DK / 8][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int row = t + 8 * e;
        float d = 0.f;
        if (row < T) {
            const int64_t at = (bh * T + row) * DV + (DV / 4) * (lane % 4);  // a quarter of the row
            if constexpr (DV >= 32) {
#pragma unroll
                for (int c = 0; c < DV / 4; c += 8) {
                    float x[8], y[8];
                    load8(o + at + c, x);
                    load8(dO + at + c, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) d = fmaf(x[i], y[i], d);
                }
            } else {
                const float4 x = load4(o + at), y = load4(dO + at);
                d = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, x.w * y.w)));
            }
        }
        D[e] = quad_sum(d);
        L2[e] = row < T ? lse[bh * T + row] * kLog2e : INFINITY;  // past the end: p = 0
    }
    for (int sweep = 0; sweep < 2; ++sweep) {
#pragma unroll
        for (int n = 0; n < DK / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
        for (int i = 0; i < kt.n; ++i) {
            wait_but_one();
            __syncthreads();
            const uint32_t sK = stage + (i & 1) * STAGE, sV = sK + tile_bytes<DK>();
            float s[8][4], g[8][4];
            dot_tiles<DK>(sK, sQ, 16 * warp, s, lane);
            mask_keys(s, t, t0, key0_of(i), W, S, c2);
            dot_tiles<DV>(sV, sG, 16 * warp, g, lane);
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = tc::ex2(fmaf(s[n][e], scale_log2, -L2[e / 2]));
                    if (sweep == 0) e2[e / 2] = fmaf(s[n][e], g[n][e] - D[e / 2], e2[e / 2]);
                }
            if (sweep == 0) {
                if (i + 1 < kt.n) {
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) p_max = fmaxf(p_max, s[n][e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        D[e] += quad_sum(e2[e]);
                        if (lane % 4 == 0 && t + 8 * e < T) dbuf[bh * T + t + 8 * e] = D[e];
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] *= g[n][e] - D[e / 2];
            mul_tile<DK>(sK, s, acc, lane);
            if (key0_of(i) < S) {  // and what the rounding left of the first tokens' dS
#pragma unroll
                for (int n = 0; n < 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] -= __bfloat162float(__float2bfloat16_rn(s[n][e]));
                mul_tile<DK>(sK, s, acc, lane);
            }
            __syncthreads();
            fetch(i + 2);
        }
        if (sweep > 0 || !__syncthreads_or(p_max > 0.5f)) break;
        fetch(0);
        fetch(1);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    const float f[2] = {grad_scale, grad_scale};
    store_rows<DK / 8>(dq + bh * T * DK, t, T, DK, acc, f, c2);
}

// ---- dk (one part per head), dv ----------------------------------------------------------------------
template <int DK, int DV> constexpr int dkv_smem() { return 3 * (tile_bytes<DK>() + tile_bytes<DV>()) + 2 * 2 * R * 4; }

// blockIdx.x: for each sequence and head, its key tiles, then (tile s, segment g) of the first tokens' far queries
template <int DK, int DV>
__global__ void __launch_bounds__(NTH, DK + DV <= 128 ? 3 : 1)
sink_mma_dkv_kernel(const bf16_t* __restrict__ q, const bf16_t* __restrict__ k, const bf16_t* __restrict__ v,
                    const float* __restrict__ lse, const float* dbuf, const bf16_t* __restrict__ dO,
                    bf16_t* __restrict__ dv, SinkParts parts, int B, int H, int T, int W, int S, float scale) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the launch that adds the parts waits for the end
    extern __shared__ __align__(16) unsigned char sm[];
    constexpr int STAGE = tile_bytes<DK>() + tile_bytes<DV>();
    const uint32_t sK = smem_u32(sm), sV = sK + tile_bytes<DK>(), stage = sK + STAGE;
    float* stats = reinterpret_cast<float*>(sm + 3 * STAGE);  // per stage: 64 log-sum-exps, 64 D
    const int tiles = parts.ctas();
    const int64_t bh = blockIdx.x / tiles;
    const int b = (int)bh / H, h = (int)bh - b * H;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c2 = 2 * (lane % 4);
    const SinkWork w = parts.work((int)blockIdx.x - (int)bh * tiles);
    const int key0 = w.tile * R, key = key0 + 16 * warp + lane / 4;  // this thread's rows: key, key + 8
    const float scale_log2 = scale * kLog2e;
    const bf16_t *qb = q + bh * T * DK, *gb = dO + bh * T * DV;
    copy_tile<DK>(sK, k + (int64_t)b * T * DK, key0, T);
    copy_tile<DV>(sV, v + bh * T * DV, key0, T);
    auto fetch = [&](int qt) {
        if (qt <= w.q_hi) {
            const int s = (qt - w.q_lo) & 1, r = threadIdx.x % R, row = qt * R + r;
            copy_tile<DK>(stage + s * STAGE, qb, qt * R, T);
            copy_tile<DV>(stage + s * STAGE + tile_bytes<DK>(), gb, qt * R, T);
            if (threadIdx.x < R) stats[2 * R * s + r] = row < T ? lse[bh * T + row] * kLog2e : INFINITY;
            else stats[2 * R * s + R + r] = row < T ? __ldcg(dbuf + bh * T + row) : 0.f;
        }
        copies_done();
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the query side's D
    fetch(w.q_lo);
    fetch(w.q_lo + 1);
    float ak[DK / 8][4], av[DV / 8][4];
#pragma unroll
    for (int n = 0; n < DK / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) ak[n][e] = 0.f;
#pragma unroll
    for (int n = 0; n < DV / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) av[n][e] = 0.f;
    for (int qt = w.q_lo; qt <= w.q_hi; ++qt) {
        wait_but_one();
        __syncthreads();
        const int st = (qt - w.q_lo) & 1, t0 = qt * R;
        const uint32_t sQ = stage + st * STAGE, sG = sQ + tile_bytes<DK>();
        const float *sL = stats + 2 * R * st, *sD = sL + R;
        float s[8][4], g[8][4];  // rows: keys, columns: queries
        dot_tiles<DK>(sQ, sK, 16 * warp, s, lane);
        dot_tiles<DV>(sG, sV, 16 * warp, g, lane);
        const bool whole = t0 >= key0 + R - 1 && (t0 + R - 1 < key0 + W || key0 + R <= S);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 L = *reinterpret_cast<const float2*>(sL + 8 * n + c2), Dn = *reinterpret_cast<const float2*>(sD + 8 * n + c2);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float p = tc::ex2(fmaf(s[n][e], scale_log2, -(e & 1 ? L.y : L.x)));
                if (!whole) {
                    const int tq = t0 + 8 * n + c2 + (e & 1), kq = key + 8 * (e / 2);
                    if (kq > tq || (kq <= tq - W && kq >= S)) p = 0.f;
                }
                s[n][e] = p;
                g[n][e] = p * (g[n][e] - (e & 1 ? Dn.y : Dn.x));
            }
        }
        mul_tile<DV>(sG, s, av, lane);
        mul_tile<DK>(sQ, g, ak, lane);
        __syncthreads();
        fetch(qt + 2);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // also where no query tile was visited
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int kr = key + 8 * e;
        if (kr >= T) continue;
        const bool part = parts.nseg > 0 && kr < S;
        if (part) {
            float* p = parts.dv_at(w.slot, bh, kr) + c2;
#pragma unroll
            for (int n = 0; n < DV / 8; ++n) *reinterpret_cast<float2*>(p + 8 * n) = make_float2(av[n][2 * e], av[n][2 * e + 1]);
        } else if (w.slot == 0) {
            uint32_t* p = reinterpret_cast<uint32_t*>(dv + (bh * T + kr) * (int64_t)DV + c2);
#pragma unroll
            for (int n = 0; n < DV / 8; ++n) p[4 * n] = pack_bf16x2(av[n][2 * e], av[n][2 * e + 1]);
        }
        if (w.slot == 0 || part) {
            float* p = (w.slot == 0 ? parts.dk_part + (((int64_t)h * B + b) * T + kr) * DK : parts.dk_at(w.slot, h, b, kr)) + c2;
#pragma unroll
            for (int n = 0; n < DK / 8; ++n) *reinterpret_cast<float2*>(p + 8 * n) = make_float2(ak[n][2 * e], ak[n][2 * e + 1]);
        }
    }
}

template <int DK, int DV>
cudaError_t fwd_t(const SinkArgs& a, cudaStream_t s) {
    constexpr int smem = fwd_smem<DK, DV>();
    const int qtiles = (a.T + R - 1) / R;
    const int64_t grid = (int64_t)qtiles * a.B * a.H;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_smem(smem_set, (const void*)sink_mma_fwd_kernel<DK, DV>, smem);
    if (e != cudaSuccess) return e;
    sink_mma_fwd_kernel<DK, DV><<<(unsigned)grid, NTH, smem, s>>>(
        static_cast<const bf16_t*>(a.q), static_cast<const bf16_t*>(a.k), static_cast<const bf16_t*>(a.v),
        static_cast<bf16_t*>(a.out), a.lse_out, a.H, a.T, a.W, a.S, a.scale * kLog2e, qtiles);
    note_launches(1);
    return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t bwd_t(const SinkArgs& a, cudaStream_t s) {
    constexpr int q_smem = dq_smem<DK, DV>(), kv_smem = dkv_smem<DK, DV>();
    const int qtiles = (a.T + R - 1) / R;
    SinkParts parts = sink_parts_plan(a, R, R, a.H);
    float* dbuf = sink_parts_bind(parts, a);
    const int64_t grid = (int64_t)qtiles * a.B * a.H, key_grid = (int64_t)parts.ctas() * a.B * a.H;
    if (grid > 0x7fffffffLL || key_grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaError_t e;
    static std::atomic<uint64_t> q_set{0}, k_set{0};
    if ((e = allow_smem(q_set, (const void*)sink_mma_dq_kernel<DK, DV>, q_smem)) != cudaSuccess) return e;
    if ((e = allow_smem(k_set, (const void*)sink_mma_dkv_kernel<DK, DV>, kv_smem)) != cudaSuccess) return e;
    const bf16_t *q = static_cast<const bf16_t*>(a.q), *k = static_cast<const bf16_t*>(a.k), *v = static_cast<const bf16_t*>(a.v),
                 *dO = static_cast<const bf16_t*>(a.dO);
    sink_mma_dq_kernel<DK, DV><<<(unsigned)grid, NTH, q_smem, s>>>(q, k, v, static_cast<const bf16_t*>(a.o), a.lse, dO, static_cast<bf16_t*>(a.dq), dbuf, a.H, a.T,
                                                                  a.W, a.S, a.scale, a.grad_scale, qtiles);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_overlapped(sink_mma_dkv_kernel<DK, DV>, dim3((unsigned)key_grid), dim3(NTH), kv_smem,
                          s, q, k, v, a.lse, static_cast<const float*>(dbuf), dO, static_cast<bf16_t*>(a.dv), parts, a.B, a.H, a.T,
                          a.W, a.S, a.scale);
    note_launches(2);
    if (e != cudaSuccess) return e;
    return sink_parts_reduce(parts, a, true, s);
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

// forward or backward for one key head dim (an instance each in swska_sink_mma_<dk>.cu, which compile
// side by side)
template <int DK>
cudaError_t sink_mma_launch(const SinkArgs& a, bool backward, cudaStream_t s);

}  // namespace rod
