// swska_extend_few.cu -- SW-SKA attention of a few new tokens (at most 16 per sequence: decode steps,
// speculative tokens) over a paged cache, bf16, 128-wide heads.
//
//   o[i,h] = sum_j softmax_j(scale q[i,h] . k[j]) v[h,j],  j <= p, j > p - W or j < S,  p = ctx + i
// Few queries against a window of keys: every value row is used for at most 16 dot products, so the
// kernel is bound by reading the cache (values: H times the keys) from HBM. A CTA takes units (one
// sequence, some key tiles of 32) of up to eight heads, so that the shared key tile is fetched once
// for them: one warp per head, which multiplies with m16n8k16 instructions (16 query rows; a
// tcgen05 tile of 128 rows would be seven eighths padding), and two warps that feed a ring of
// stages by TMA. With eight heads a stage (a key tile and eight value tiles) is 72 KB and an SM holds
// three; with up to four, two CTAs an SM hold two stages of 40 KB each. Both are more than the bytes in
// flight that HBM's rate times its latency asks of an SM (128 sequences, H 16, W 4096: 330 us and
// 7.0 TB/s in a short run, 352 to 386 us over seconds of passes). The pages' rows land in shared
// memory with the 128-byte swizzle, which keeps the fragment loads free of bank conflicts; a page of
// any multiple of 8 tokens is a row of boxes of 8, 16 or 32 rows. A warp issues a copy every 100
// clocks or so, and a tile has to come every 3100 at HBM's rate, so a box takes the rows of all of
// the CTA's heads, and two warps share them (one for the first 64 columns, one for the last): 4 copies a
// tile for pages of 32 k tokens, 16 for pages of 8 (18 and 72 head by head).
// Softmax: running maximum and sum in fp32, base 2; the output is rescaled only when a row's maximum
// moves. Probabilities go to the second product in bf16 (relative 2^-9 each, like the cached values).
#include <cuda.h>
#include <math.h>

#include <type_traits>

#include "extend.cuh"
#include "mma16.cuh"
#include "tc.cuh"

namespace rod {
namespace {

using mma::bits_from;
using mma::bits_to;
using mma::ldsm4;
using mma::ldsm4t;
using mma::mma16816;

__device__ unsigned int g_extend_few_timeout = 0;

constexpr int HD = 128;
constexpr int KT = kFewTile;               // keys per tile
constexpr int HALF = KT * 128;             // bytes: KT rows x 64 columns
constexpr int TILE = 2 * HALF;             // 8 KB: a key tile or one head's value tile
constexpr int NTH = 32 * (kFewHeads + 2);  // and two producer warps
constexpr int MAXST = 12;
constexpr int kMaxParts = 10;              // parts of a query tile, in units of 32 (see cols below)
// The ring for one CTA an SM (up to eight heads) or two (up to four): barriers and masks come first
constexpr int OFF_MASK = 2 * MAXST * 8;
constexpr int OFF_MISC = OFF_MASK + MAXST * 4;
constexpr int OFF_RING = 1024;
static_assert(OFF_MISC + 16 <= OFF_RING, "barriers");
constexpr int ring_for(int ctas) { return ctas == 1 ? 216 * 1024 : 104 * 1024; }
constexpr int smem_for(int ctas) { return OFF_RING + ring_for(ctas) + 1024; }
static_assert(smem_for(1) <= 232448 && 2 * (smem_for(2) + 1024) <= 233472, "shared memory");

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    for (uint32_t i = 1;; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((i & 255u) == 0) {
            if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
            if (i >= kWaitLimit) {
                *abort_flag = 1;
                atomicExch(&g_extend_few_timeout, 1u);
                return false;
            }
        }
    }
}

// 16-byte chunk c (of 16) of row r of the key tile: two halves of 64 columns, swizzled
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return (uint32_t)((c >> 3) * HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// Value tiles: [half][box of rows][head][row of the box], so that one box holds every head's rows.
// Start of the eight rows 8 rg .. 8 rg + 7 of a head in half 0; half 1 is hpg halves further.
__device__ __forceinline__ uint32_t rows_at(int rg, int head, int hpg, int box) {
    const int per = box / 8;
    return (uint32_t)(((rg / per * hpg + head) * per + rg % per) * 1024);
}

// Adds the parts of rows r0 .. r0 + R - 1 of a head (one warp). For the weights a lane is a (part, row) pair, 32 / R
// parts at a time; for the sums it is four columns, with 16 loads in flight and the parts in their order. (The loads of
// two parts in flight instead: 51.5 us in place of 21.4 for 2 tokens with W 4096, H 16 in 65 parts a head.)
template <int R>
__device__ __forceinline__ void add_rows(const ExtendRoute& r, int nsplit, int at0, int at1, int step, int r0, int rows,
                                         int lane, __nv_bfloat16* out, int out_step) {
    constexpr int P = 32 / R;
    auto part0 = [&](int s) { return s == 0 ? at0 : at1 + s * step; };  // the part's row 0
    const int e = lane / R, i = lane % R;
    const bool in = r0 + i < rows;
    float M = -INFINITY, L = 0.f;
#pragma unroll 4
    for (int s0 = 0; s0 < nsplit; s0 += P) {
        const float2 ml = in && s0 + e < nsplit ? __ldcg(r.part_ml + part0(s0 + e) + r0 + i) : make_float2(-INFINITY, 0.f);
        const float mn = fmaxf(M, ml.x), base = mn == -INFINITY ? 0.f : mn;
        L = fmaf(ml.y, tc::ex2(ml.x - base), L * tc::ex2(M - base));
        M = mn;
    }
#pragma unroll
    for (int d = R; d < 32; d <<= 1) {  // the same sum on both sides of the exchange
        const float m2 = __shfl_xor_sync(0xffffffffu, M, d), l2 = __shfl_xor_sync(0xffffffffu, L, d);
        const float mn = fmaxf(M, m2), base = mn == -INFINITY ? 0.f : mn;
        L = __fadd_rn(__fmul_rn(L, tc::ex2(M - base)), __fmul_rn(l2, tc::ex2(m2 - base)));
        M = mn;
    }
    const float base = M == -INFINITY ? 0.f : M, inv = L == 0.f ? 0.f : 1.f / L;
    float4 O[R];
#pragma unroll
    for (int n = 0; n < R; ++n) O[n] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < nsplit; s0 += P) {
        const float w = in && s0 + e < nsplit ? tc::ex2(__ldcg(&r.part_ml[part0(s0 + e) + r0 + i].x) - base) * inv : 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float4 x[P / 2][R];
#pragma unroll
            for (int c = 0; c < P / 2; ++c) {
                const int s = s0 + half * (P / 2) + c;
                const float4* from = reinterpret_cast<const float4*>(r.part_o + (int64_t)(part0(s < nsplit ? s : 0) + r0) * HD) + lane;
#pragma unroll
                for (int n = 0; n < R; ++n)
                    x[c][n] = s < nsplit && r0 + n < rows ? __ldcg(from + n * (HD / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int c = 0; c < P / 2; ++c)
#pragma unroll
                for (int n = 0; n < R; ++n) {
                    const float wi = __shfl_sync(0xffffffffu, w, (half * (P / 2) + c) * R + n);
                    O[n].x = fmaf(x[c][n].x, wi, O[n].x);
                    O[n].y = fmaf(x[c][n].y, wi, O[n].y);
                    O[n].z = fmaf(x[c][n].z, wi, O[n].z);
                    O[n].w = fmaf(x[c][n].w, wi, O[n].w);
                }
        }
    }
#pragma unroll
    for (int n = 0; n < R; ++n)
        if (r0 + n < rows) store4(out + (r0 + n) * out_step + 4 * lane, O[n]);
}

__global__ void __launch_bounds__(NTH, 1)
extend_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const ExtendArgs a, const ExtendRoute r, int hpg, int n_stages, int box, float scale_log2) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);
    uint64_t* empty = full + MAXST;
    volatile uint32_t* mask = reinterpret_cast<volatile uint32_t*>(smem + OFF_MASK);  // keys whose page exists
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC);
    unsigned char* ring = smem + OFF_RING;
    const int stage_bytes = TILE * (1 + hpg);

    // a CTA keeps to one head group: blockIdx.x = group + groups * column
    const int grp = blockIdx.x % r.groups;
    const int h0 = grp * hpg, nh = min(hpg, a.H - h0);
    if (threadIdx.x == 32 * hpg) {
        tc::tma_prefetch_desc(&tm_k);
        tc::tma_prefetch_desc(&tm_v);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < n_stages; ++s) {
            mbar_init(&full[s], 2);
            mbar_init(&empty[s], (uint32_t)nh);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    wait_for_launch_before();
    // the chunks' kernel (swska_extend_tc.cu) may take over SMs as they fall free
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const ExtendRange range = load_range(r, blockIdx.x / r.groups);

    if (warp >= hpg) {
        // ------------------------------- producers: one per half -------------------------------
        const int half = warp - hpg;
        const int nbox = KT / box, ops = 2 * nbox;  // (keys, values) x boxes: at most 8
        int t = 0;  // tiles fed so far
        bool ok = true;
        for (int x = range.lo; x <= range.hi && ok; ++x) {
            const ExtendUnit u = load_unit(r.units + x);
            const ExtendSeq sq{u.row0, u.len, u.ctx, false};
            const ExtendKeys kt = extend_keys(sq, u.q0, kFewRows, KT, a.W, a.S);
            // lanes 0 .. nbox - 1 hold the page of the tile's box, one tile ahead
            auto page_of = [&](int i) {
                return i < u.kt1 && lane < nbox ? extend_page(a, u.n, (kt.at(i) * KT + lane * box) / a.page) : -1;
            };
            int pg_next = page_of(u.kt0);
            for (int i = u.kt0; i < u.kt1; ++i, ++t) {
                const int pg = pg_next, key0 = kt.at(i) * KT;
                pg_next = page_of(i + 1);
                const int s = t % n_stages, use = t / n_stages;
                if (use > 0 && !wait_warp(&empty[s], (uint32_t)((use - 1) & 1), abort_flag)) { ok = false; break; }
                unsigned have = 0;
                for (int b = 0; b < nbox; ++b)
                    if (__shfl_sync(0xffffffffu, pg, b) >= 0) have |= (box == 32 ? 0xffffffffu : ((1u << box) - 1u) << (b * box));
                if (lane == 0) {
                    if (half == 0) mask[s] = have;
                    mbar_arrive_expect_tx(&full[s], (uint32_t)stage_bytes / 2);
                }
                __syncwarp();
                const int b = lane % nbox;
                const int p = __shfl_sync(0xffffffffu, pg, b);
                if (lane < ops) {
                    unsigned char* dst = ring + s * stage_bytes;
                    const int y = (key0 + b * box) % a.page;
                    // a page that the table does not have: a coordinate past the end, which fills zeros
                    if (lane < nbox)
                        tc::tma_load_3d(dst + half * HALF + b * box * 128, &tm_k, half * 64, y, p >= 0 ? p : a.P, &full[s]);
                    else
                        tc::tma_load_3d(dst + TILE + (half * nbox + b) * hpg * box * 128, &tm_v, half * 64, y,
                                        p >= 0 ? p * a.H + h0 : a.P * a.H, &full[s]);
                }
            }
        }
        // every copy started here has landed before the CTA can leave
        for (int i = t > n_stages ? t - n_stages : 0; i < t; ++i)
            mbar_wait_bounded(&full[i % n_stages], (uint32_t)((i / n_stages) & 1), kWaitLimit);
        return;
    }
    if (warp >= nh) return;  // the last group may have fewer heads
    // ------------------------------- one warp per head -------------------------------
    const int h = h0 + warp;
    const int g = lane / 4, c2 = 2 * (lane % 4);  // this thread's rows g, g + 8 and its column pair
    const int mat = lane / 8, mr = lane % 8;      // this lane's row address in a 4-matrix load
    // of the values: rows 16 k + 8 (mat & 1) + mr for k = 0, 1
    const uint32_t vrow[2] = {rows_at(mat & 1, warp, hpg, box) + mr * 128, rows_at(2 + (mat & 1), warp, hpg, box) + mr * 128};
    int t = 0;
    for (int x = range.lo; x <= range.hi; ++x) {
        const ExtendUnit u = load_unit(r.units + x);
        const ExtendSeq sq{u.row0, u.len, u.ctx, false};
        const ExtendKeys kt = extend_keys(sq, u.q0, kFewRows, KT, a.W, a.S);
        const int rows = min(u.len - u.q0, kFewRows), p0 = u.ctx + u.q0, p1 = p0 + rows - 1;
        const int64_t row0 = u.row0 + u.q0;
        uint32_t qa[8][4];
        {
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
            const uint32_t* q0p = reinterpret_cast<const uint32_t*>(q + ((row0 + g) * a.H + h) * HD + c2);
            const uint32_t* q1p = reinterpret_cast<const uint32_t*>(q + ((row0 + g + 8) * a.H + h) * HD + c2);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                qa[k][0] = g < rows ? q0p[8 * k] : 0u;
                qa[k][1] = g + 8 < rows ? q1p[8 * k] : 0u;
                qa[k][2] = g < rows ? q0p[8 * k + 4] : 0u;
                qa[k][3] = g + 8 < rows ? q1p[8 * k + 4] : 0u;
            }
        }
        float o[16][4];
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        for (int i = u.kt0; i < u.kt1; ++i, ++t) {
            const int st = t % n_stages, key0 = kt.at(i) * KT;
            if (!wait_warp(&full[st], (uint32_t)((t / n_stages) & 1), abort_flag)) return;
            const uint32_t kb = smem_u32(ring + st * stage_bytes), vb = kb + TILE;
            float s[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int n = 0; n < 4; n += 2) {
                    uint32_t b[4];
                    ldsm4(kb + chunk_at((n + (mat >> 1)) * 8 + mr, 2 * k + (mat & 1)), b);
                    mma16816(s[n], qa[k], b);
                    mma16816(s[n + 1], qa[k], b + 2);
                }
            const uint32_t have = mask[st];
            const bool whole = have == 0xffffffffu && key0 + KT - 1 <= p0 &&
                               ((int64_t)key0 > (int64_t)p1 - a.W || key0 + KT <= a.S);
            bool zeroed = false;
            if (!whole) {
                // keys that no query sees: the rows behind them may hold anything, so clear this head's
                const int j = key0 + lane;
                const bool seen = (have >> lane & 1u) && j <= p1 && ((int64_t)j > (int64_t)p0 - a.W || j < a.S);
                zeroed = !__all_sync(0xffffffffu, seen);
                if (!seen) {  // lane = key; neighbouring lanes start at neighbouring chunks: no bank conflicts
                    unsigned char* v = ring + st * stage_bytes + TILE + rows_at(lane / 8, warp, hpg, box) + (lane & 7) * 128;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        *reinterpret_cast<uint4*>(v + ((c + lane) & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4*>(v + hpg * HALF + ((c + lane) & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                __syncwarp();
                // bit per key: seen by row g (v[0]) and by row g + 8 (v[1])
                uint32_t v[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int p = p0 + g + 8 * e;
                    v[e] = have & bits_to(p - key0) & (bits_from((int64_t)p - a.W + 1 - key0) | bits_to(a.S - 1 - key0));
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int c = 8 * n + c2;
                    if (!(v[0] >> c & 1u)) s[n][0] = -INFINITY;
                    if (!(v[0] >> c & 2u)) s[n][1] = -INFINITY;
                    if (!(v[1] >> c & 1u)) s[n][2] = -INFINITY;
                    if (!(v[1] >> c & 2u)) s[n][3] = -INFINITY;
                }
            }
            // row maxima over the four threads of a row
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                mx[0] = fmaxf(mx[0], fmaxf(s[n][0], s[n][1]));
                mx[1] = fmaxf(mx[1], fmaxf(s[n][2], s[n][3]));
            }
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], d));
                mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], d));
            }
            const float t0 = mx[0] * scale_log2, t1 = mx[1] * scale_log2;
            if (__any_sync(0xffffffffu, t0 > m[0] || t1 > m[1])) {
                const float n0 = fmaxf(m[0], t0), n1 = fmaxf(m[1], t1);
                const float a0 = n0 == -INFINITY ? 1.f : tc::ex2(m[0] - n0), a1 = n1 == -INFINITY ? 1.f : tc::ex2(m[1] - n1);
                m[0] = n0;
                m[1] = n1;
                l[0] *= a0;
                l[1] *= a1;
#pragma unroll
                for (int i2 = 0; i2 < 16; ++i2) {
                    o[i2][0] *= a0;
                    o[i2][1] *= a0;
                    o[i2][2] *= a1;
                    o[i2][3] *= a1;
                }
            }
            const float b0 = m[0] == -INFINITY ? 0.f : m[0], b1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                s[n][0] = tc::ex2(fmaf(s[n][0], scale_log2, -b0));
                s[n][1] = tc::ex2(fmaf(s[n][1], scale_log2, -b0));
                s[n][2] = tc::ex2(fmaf(s[n][2], scale_log2, -b1));
                s[n][3] = tc::ex2(fmaf(s[n][3], scale_log2, -b1));
                l[0] += s[n][0] + s[n][1];
                l[1] += s[n][2] + s[n][3];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t pa[4];
                pa[0] = pack_bf16x2(s[2 * k][0], s[2 * k][1]);
                pa[1] = pack_bf16x2(s[2 * k][2], s[2 * k][3]);
                pa[2] = pack_bf16x2(s[2 * k + 1][0], s[2 * k + 1][1]);
                pa[3] = pack_bf16x2(s[2 * k + 1][2], s[2 * k + 1][3]);
#pragma unroll
                for (int c = 0; c < 16; c += 2) {
                    uint32_t b[4];
                    const int ch = c + (mat >> 1);
                    ldsm4t(vb + vrow[k] + (uint32_t)((ch >> 3) * hpg * HALF + (((ch & 7) ^ mr) << 4)), b);
                    mma16816(o[c], pa, b);
                    mma16816(o[c + 1], pa, b + 2);
                }
            }
            if (zeroed) tc::fence_proxy_async();  // before the next copy into this stage
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
            l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
        }
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o);
        if (u.part < 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = g + 8 * e;
                if (row >= rows) continue;
                const float inv = l[e] == 0.f ? 0.f : 1.f / l[e];
                __nv_bfloat16* op = out + ((row0 + row) * a.H + h) * HD + c2;
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    *reinterpret_cast<uint32_t*>(op + 8 * c) = pack_bf16x2(o[c][2 * e] * inv, o[c][2 * e + 1] * inv);
            }
            continue;
        }
        // this unit's part; the warp that comes last for the head adds the parts in the order of the keys
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = g + 8 * e;
            if (row >= rows) continue;
            const int64_t at = r.part_at(u.part, a.H, h, row);
            if (lane % 4 == 0) r.part_ml[at] = make_float2(m[e], l[e]);
#pragma unroll
            for (int c = 0; c < 16; ++c)
                *reinterpret_cast<float2*>(r.part_o + at * HD + 8 * c + c2) = make_float2(o[c][2 * e], o[c][2 * e + 1]);
        }
        __threadfence();
        __syncwarp();
        int last = 0;
        if (lane == 0) last = atomicAdd(r.count + (int64_t)u.counter * a.H + h, 1) == u.nsplit - 1;
        if (!__shfl_sync(0xffffffffu, last, 0)) continue;
        __threadfence();
        // parts 1, 2, ... lie two part numbers apart
        const int64_t step = 2 * (int64_t)a.H * r.part_rows;
        if (rows > 1) {
            // part rows are fewer than 2 x 32 kMaxParts CTAs x 64 heads x 16 rows: 32 bits
            const int at0 = (int)r.part_at(u.first, a.H, h, 0), at1 = (int)r.part_at(2 * u.c0, a.H, h, 0);
            auto add = [&](auto n, int r0) {
                add_rows<decltype(n)::value>(r, u.nsplit, at0, at1, (int)step, r0, rows, lane, out + (row0 * a.H + h) * HD, a.H * HD);
            };
            if (rows <= 2) {
                add(std::integral_constant<int, 2>(), 0);
            } else if (rows <= 4) {
                add(std::integral_constant<int, 4>(), 0);
            } else {
                for (int r0 = 0; r0 < rows; r0 += 8) add(std::integral_constant<int, 8>(), r0);
            }
        } else {
            const int row = 0;
            const int64_t at0 = r.part_at(u.first, a.H, h, row), at1 = r.part_at(2 * u.c0, a.H, h, row);
            const float4* x0 = reinterpret_cast<const float4*>(r.part_o + at0 * HD) + lane;
            const float4* x1 = reinterpret_cast<const float4*>(r.part_o + at1 * HD) + lane;
            // lane = part for the weights (as many as CTAs per head group, at most), lane = four columns for the sum
            float M = -INFINITY, L = 0.f, mv[kMaxParts], w[kMaxParts];
#pragma unroll
            for (int i = 0; i < kMaxParts; ++i) {
                const int s = lane + 32 * i;
                const float2 ml = s < u.nsplit ? __ldcg(r.part_ml + (s == 0 ? at0 : at1 + s * step)) : make_float2(-INFINITY, 0.f);
                mv[i] = ml.x;
                w[i] = ml.y;
                M = fmaxf(M, ml.x);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
            const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int i = 0; i < kMaxParts; ++i) {
                mv[i] = tc::ex2(mv[i] - base);
                L = fmaf(w[i], mv[i], L);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
            const float inv = L == 0.f ? 0.f : 1.f / L;
            float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kMaxParts; ++i) {
                for (int s0 = 32 * i; s0 < min(32 * i + 32, u.nsplit); s0 += 16) {
                    float4 x4[16];  // loads in flight together
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        x4[e] = s0 + e < u.nsplit ? __ldcg(s0 + e == 0 ? x0 : x1 + (s0 + e) * (int)step * (HD / 4))
                                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float ws = __shfl_sync(0xffffffffu, mv[i], (s0 + e) & 31);
                        O.x = fmaf(x4[e].x, ws, O.x);
                        O.y = fmaf(x4[e].y, ws, O.y);
                        O.z = fmaf(x4[e].z, ws, O.z);
                        O.w = fmaf(x4[e].w, ws, O.w);
                    }
                }
            }
            store4(out + ((row0 + row) * a.H + h) * HD + 4 * lane, make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
        }
    }
}

}  // namespace

cudaError_t swska_extend_few_launch(const ExtendArgs& a, const ExtendRoute& r, cudaStream_t s) {
    if (r.cols > 32 * kMaxParts) return cudaErrorInvalidConfiguration;
    const int hpg = (a.H + r.groups - 1) / r.groups;
    int box = KT;
    while (a.page % box != 0) box /= 2;
    CUtensorMap mk, mv;
    cudaError_t e;
    if ((e = make_tmap_bf16_3d(&mk, a.k_pool, HD, (uint64_t)a.page, (uint64_t)a.P, 64, (uint32_t)box)) != cudaSuccess) return e;
    if ((e = make_tmap_bf16_3d_strided(&mv, a.v_pool, HD, (uint64_t)a.page, (uint64_t)a.P * a.H, HD * 2, (uint64_t)a.page * HD * 2,
                                       64, (uint32_t)box, (uint32_t)hpg)) != cudaSuccess)
        return e;
    const int ctas = hpg <= kFewHeads / 2 ? 2 : 1;
    int stages = ring_for(ctas) / (TILE * (1 + hpg));
    if (stages > MAXST) stages = MAXST;
    static std::atomic<uint64_t> smem_set{0};
    if ((e = allow_smem(smem_set, (const void*)extend_few_kernel, smem_for(1))) != cudaSuccess) return e;
    e = launch_overlapped(extend_few_kernel, dim3((unsigned)(r.cols * r.groups)), dim3(32 * (hpg + 2)), (size_t)smem_for(ctas), s, mk, mv,
                          a, r, hpg, stages, box, a.scale * 1.4426950408889634f);
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

unsigned swska_extend_few_take_timeout_flag() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_extend_few_timeout, sizeof(v)) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_extend_few_timeout, &zero, sizeof(zero));
    return v;
}

}  // namespace rod
