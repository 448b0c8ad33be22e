// swska_extend_simt.cu -- SW-SKA attention of new tokens over a paged cache on CUDA cores (every
// product an fp32 FMA): fp32 caches, and bf16 shapes outside the tensor-core kernels.
//
//   o[i,h] = sum_j softmax_j(scale q[i,h] . k[j]) v[h,j],  j <= p, j > p - W or j < S
// where the token i of a sequence sits at position p = ctx + i and key j in page j / page of the
// sequence's row of the block table. One CTA takes a unit (16 or 64 queries, some key tiles of 64)
// of one head with the tiles of simt_tile.cuh; keys that no query of the tile sees, and keys of
// pages that the table does not have, are loaded as zeros (the memory there may hold anything)
// and masked. A row that sees no key gives zeros.
#include <math.h>

#include "extend.cuh"
#include "simt_tile.cuh"

namespace rod {
namespace {

using namespace simt;

template <int DK, int DV, int BQ>
constexpr int smem_bytes() {
    return (BQ * ld<DK>() + BK * ld<DK>() + BK * ld<DV>() + BQ * LDP) * 4 + BK * 4 + 16;
}

template <int DK, int DV, int BQ>
__global__ void __launch_bounds__(4 * BQ)
extend_simt_kernel(const ExtendArgs a, const ExtendRoute r, bool bf16, float scale_log2) {
    constexpr int NTH = 4 * BQ;
    extern __shared__ __align__(16) float sm[];
    float* sQ = sm;
    float* sK = sQ + BQ * ld<DK>();
    float* sV = sK + BK * ld<DK>();
    float* sP = sV + BK * ld<DV>();
    int* sAt = reinterpret_cast<int*>(sP + BQ * LDP);  // slot of each key of the tile, -1: none
    int* sLast = sAt + BK;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int h = blockIdx.x % a.H;
    const ExtendRange range = load_range(r, blockIdx.x / a.H);
    for (int x = range.lo; x <= range.hi; ++x) {
        const ExtendUnit u = load_unit(r.units + x);
        const ExtendSeq sq{u.row0, u.len, u.ctx, false};
        const int rows = sq.len - u.q0 < BQ ? sq.len - u.q0 : BQ;
        const int p0 = sq.ctx + u.q0, p1 = p0 + rows - 1;
        const ExtendKeys kt = extend_keys(sq, u.q0, BQ, BK, a.W, a.S);
        const int64_t row0 = sq.row0 + u.q0;
        __syncthreads();
        load_tile<DK, BQ, NTH>(sQ, a.q, bf16, [&](int i) { return i < rows ? ((row0 + i) * a.H + h) * (int64_t)DK : -1; });
        float m[4], l[4], acc[4][DV / 16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < DV / 16; ++c) acc[i][c] = 0.f;
        }
        for (int it = u.kt0; it < u.kt1; ++it) {
            const int key0 = kt.at(it) * BK;
            __syncthreads();
            for (int i = threadIdx.x; i < BK; i += NTH) {
                const int j = key0 + i;
                // some query of the tile sees it: not past the last, in the first one's window or among the first S
                const bool seen = j <= p1 && ((int64_t)j > (int64_t)p0 - a.W || j < a.S);
                const int pg = seen ? extend_page(a, u.n, j / a.page) : -1;
                sAt[i] = pg >= 0 ? pg * a.page + j % a.page : -1;
            }
            __syncthreads();
            load_tile<DK, BK, NTH>(sK, a.k_pool, bf16, [&](int i) { return sAt[i] >= 0 ? (int64_t)sAt[i] * DK : -1; });
            load_tile<DV, BK, NTH>(sV, a.v_pool, bf16, [&](int i) {
                const int s = sAt[i], pg = s / a.page;
                return s >= 0 ? (((int64_t)pg * a.H + h) * a.page + (s - pg * a.page)) * DV : -1;
            });
            __syncthreads();
            float s[4][4];
            tile_dot<DK>(sQ, sK, ty, tx, s);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = tx + 16 * j;
                    const bool see = sAt[c] >= 0 && ska_visible(p0 + 4 * ty + i, key0 + c, a.W, a.S);
                    s[i][j] = see ? s[i][j] * scale_log2 : -INFINITY;
                }
            softmax_step<DV / 16>(s, m, l, acc);
            put_tile(sP, ty, tx, s);
            __syncthreads();
            tile_mul<DV>(sP, sV, ty, tx, acc);
        }
        if (u.part < 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (4 * ty + i >= rows) continue;
                const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);
#pragma unroll
                for (int c = 0; c < DV / 16; ++c)
                    store1_as(a.o, bf16, ((row0 + 4 * ty + i) * a.H + h) * (int64_t)DV + Cols<DV>::at(tx, c), acc[i][c] * inv);
            }
            continue;
        }
        // this unit's part, then the last unit of the tile adds them in order
        const int64_t mine = r.part_at(u.part, a.H, h, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * ty + i;
            if (row >= rows) continue;
            if (tx == 0) r.part_ml[mine + row] = make_float2(m[i], l[i]);
#pragma unroll
            for (int c = 0; c < DV / 16; ++c) r.part_o[(mine + row) * DV + Cols<DV>::at(tx, c)] = acc[i][c];
        }
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) *sLast = atomicAdd(r.count + (int64_t)u.counter * a.H + h, 1) == u.nsplit - 1;
        __syncthreads();
        if (!*sLast) continue;
        __threadfence();
        for (int i = threadIdx.x; i < rows * DV; i += NTH) {
            const int row = i / DV, c = i % DV;
            float M = -INFINITY, L = 0.f, O = 0.f;
            for (int s = 0; s < u.nsplit; ++s)
                M = fmaxf(M, __ldcg(&r.part_ml[r.part_at(u.part_of(s), a.H, h, row)].x));
            const float base = M == -INFINITY ? 0.f : M;
            for (int s = 0; s < u.nsplit; ++s) {
                const int64_t at = r.part_at(u.part_of(s), a.H, h, row);
                const float2 ml = __ldcg(&r.part_ml[at]);
                const float w = exp2f(ml.x - base);
                L = fmaf(ml.y, w, L);
                O = fmaf(__ldcg(&r.part_o[at * DV + c]), w, O);
            }
            store1_as(a.o, bf16, ((row0 + row) * a.H + h) * (int64_t)DV + c, L == 0.f ? 0.f : O / L);
        }
    }
}

template <int DK, int DV, int BQ>
cudaError_t launch_t(const ExtendArgs& a, const ExtendRoute& r, bool bf16, cudaStream_t s) {
    constexpr int smem = smem_bytes<DK, DV, BQ>();
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_smem(smem_set, (const void*)extend_simt_kernel<DK, DV, BQ>, smem);
    if (e != cudaSuccess) return e;
    extend_simt_kernel<DK, DV, BQ><<<(unsigned)(r.cols * r.groups), 4 * BQ, smem, s>>>(
        a, r, bf16, a.scale * 1.4426950408889634f);
    note_launches(1);
    return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t pick_rows(const ExtendArgs& a, const ExtendRoute& r, bool bf16, cudaStream_t s) {
    return r.rows == 16 ? launch_t<DK, DV, 16>(a, r, bf16, s) : launch_t<DK, DV, 64>(a, r, bf16, s);
}

template <int DK>
cudaError_t pick_dv(const ExtendArgs& a, const ExtendRoute& r, bool bf16, cudaStream_t s) {
    switch (a.d_v) {
        case 16: return pick_rows<DK, 16>(a, r, bf16, s);
        case 32: return pick_rows<DK, 32>(a, r, bf16, s);
        case 64: return pick_rows<DK, 64>(a, r, bf16, s);
        case 128: return pick_rows<DK, 128>(a, r, bf16, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t swska_extend_simt_launch(const ExtendArgs& a, const ExtendRoute& r, bool bf16, cudaStream_t s) {
    switch (a.d_k) {
        case 16: return pick_dv<16>(a, r, bf16, s);
        case 32: return pick_dv<32>(a, r, bf16, s);
        case 64: return pick_dv<64>(a, r, bf16, s);
        case 128: return pick_dv<128>(a, r, bf16, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace rod
