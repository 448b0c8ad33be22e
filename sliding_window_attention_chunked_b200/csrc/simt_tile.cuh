// simt_tile.cuh -- fp32 tile products on CUDA cores for the SW-SKA kernels with first tokens that
// stay visible (fp32 inputs, and bf16 with head dims that the tensor-core kernels do not take).
//
// A CTA of 4 BQ threads owns BQ query rows (or BQ keys) and visits tiles of 64 rows of the other
// side. Thread (ty, tx) = (tid / 16, tid % 16) holds a 4 x 4 piece of a BQ x 64 score tile, rows
// 4 ty + i and columns tx + 16 j, and of a BQ x D product rows 4 ty + i and D / 16 columns. Tiles
// sit in shared memory as fp32 rows of D + 4 floats: the pad moves neighbouring rows by four
// banks, so that the 16-byte loads of eight neighbouring rows touch every bank once. A 4-wide step
// of a score product is then 8 16-byte loads for 64 FMAs, which go out two to an instruction
// (fma.rn.f32x2): along d in a score product (even and odd terms summed apart), along the columns in
// a product of probabilities. That leaves the issue slots that the loads need.
#pragma once

#include "common.cuh"
#include "exp2x2.cuh"

namespace rod {
namespace simt {

constexpr int BK = 64;        // rows of the tiles that are visited
constexpr int LDP = BK + 4;   // row of a probability tile

template <int D> __host__ __device__ constexpr int ld() { return D + 4; }

__device__ __forceinline__ float4 load4_as(const void* p, bool bf16, int64_t i) {
    return bf16 ? load4(static_cast<const __nv_bfloat16*>(p) + i) : load4(static_cast<const float*>(p) + i);
}
__device__ __forceinline__ void store4_as(void* p, bool bf16, int64_t i, float4 f) {
    if (bf16) store4(static_cast<__nv_bfloat16*>(p) + i, f);
    else store4(static_cast<float*>(p) + i, f);
}
__device__ __forceinline__ void store1_as(void* p, bool bf16, int64_t i, float f) {
    if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f);
    else static_cast<float*>(p)[i] = f;
}

// ROWS rows of D elements into fp32 rows of D + 4; at(r) gives the element offset of row r, or -1
// for a row of zeros
template <int D, int ROWS, int NTH, typename At>
__device__ __forceinline__ void load_tile(float* s, const void* base, bool bf16, At at, int tid = threadIdx.x) {
    for (int i = tid; i < ROWS * (D / 4); i += NTH) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4));
        const int64_t off = at(r);
        const float4 x = off >= 0 ? load4_as(base, bf16, off + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(s + r * ld<D>() + c) = x;
    }
}

// acc[i][j] = a_row(4 ty + i) . b_row(tx + 16 j)
template <int D>
__device__ __forceinline__ void tile_dot(const float* a, const float* b, int ty, int tx, float acc[4][4]) {
    float2 sum[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int d = 0; d < D; d += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (4 * ty + i) * ld<D>() + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * ld<D>() + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum[i][j] = fx::f2fma(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), sum[i][j]);
                sum[i][j] = fx::f2fma(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), sum[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = sum[i][j].x + sum[i][j].y;
}

// columns of a BQ x D accumulator held by thread column tx: groups of VW neighbours
template <int D> struct Cols {
    static constexpr int VW = D >= 64 ? 4 : D / 16;
    static constexpr int NG = D / (16 * VW);
    static constexpr int N = D / 16;
    static __device__ __forceinline__ int at(int tx, int c) { return 16 * VW * (c / VW) + VW * tx + c % VW; }
};

// acc[i][c] += sum over 64 k of w[4 ty + i][k] x[k][column c]; w has rows of LDP, x rows of D + 4
template <int D>
__device__ __forceinline__ void tile_mul(const float* w, const float* x, int ty, int tx, float acc[4][D / 16]) {
    using C = Cols<D>;
#pragma unroll 2
    for (int k = 0; k < BK; k += 4) {
        float p[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 t = *reinterpret_cast<const float4*>(w + (4 * ty + i) * LDP + k);
            p[i][0] = t.x; p[i][1] = t.y; p[i][2] = t.z; p[i][3] = t.w;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float v[C::N];
            const float* row = x + (k + u) * ld<D>();
#pragma unroll
            for (int g = 0; g < C::NG; ++g) {
                const float* s = row + 16 * C::VW * g + C::VW * tx;
                if constexpr (C::VW == 4) {
                    const float4 t = *reinterpret_cast<const float4*>(s);
                    v[4 * g] = t.x; v[4 * g + 1] = t.y; v[4 * g + 2] = t.z; v[4 * g + 3] = t.w;
                } else if constexpr (C::VW == 2) {
                    const float2 t = *reinterpret_cast<const float2*>(s);
                    v[2 * g] = t.x; v[2 * g + 1] = t.y;
                } else {
                    v[g] = s[0];
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (C::N == 1) {
                    acc[i][0] = fmaf(p[i][u], v[0], acc[i][0]);
                } else {
#pragma unroll
                    for (int c = 0; c < C::N; c += 2) {
                        const float2 t = fx::f2fma(make_float2(p[i][u], p[i][u]), make_float2(v[c], v[c + 1]),
                                                   make_float2(acc[i][c], acc[i][c + 1]));
                        acc[i][c] = t.x;
                        acc[i][c + 1] = t.y;
                    }
                }
            }
        }
    }
}

// the NTH threads of group g of a CTA meet (barrier 0 is the CTA's)
template <int NTH> __device__ __forceinline__ void group_sync(int g) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "n"(NTH) : "memory");
}

// sum / maximum over the 16 threads of a row group (lanes that differ in tx)
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}

// One online-softmax step: scores (already in base-2 units, -inf where masked) become
// probabilities relative to the running maximum, which each row's 16 threads share; O and the
// running sum are rescaled when the maximum moves. A row with no visible key so far keeps
// m = -inf, l = 0 and probabilities of 0.
template <int N>
__device__ __forceinline__ void softmax_step(float s[4][4], float m[4], float l[4], float o[4][N]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float mt = row_max(fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3])));
        const float mn = fmaxf(m[i], mt);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float alpha = exp2f(m[i] - base);  // 0 when m = -inf
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[i][j] = exp2f(s[i][j] - base);  // 0 when masked
            sum += s[i][j];
        }
        l[i] = fmaf(l[i], alpha, row_sum(sum));
        m[i] = mn;
#pragma unroll
        for (int c = 0; c < N; ++c) o[i][c] *= alpha;
    }
}

__device__ __forceinline__ void put_tile(float* w, int ty, int tx, const float s[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) w[(4 * ty + i) * LDP + tx + 16 * j] = s[i][j];
}

}  // namespace simt

// A query at position p sees key j: causal, and inside the window of W or among the first S.
__device__ __forceinline__ bool ska_visible(int64_t p, int64_t j, int W, int S) {
    return j <= p && (j > p - W || j < S);
}

}  // namespace rod
