// swska_extend_tc.cu -- SW-SKA attention of chunks of new tokens (more than 16 per sequence) over a
// paged cache on the 5th-generation tensor cores, bf16 in / fp32 accumulate, 128-wide heads.
//
//   o[i,h] = sum_j softmax_j(scale q[i,h] . k[j]) v[h,j],  j <= p, j > p - W or j < S,  p = ctx + i
// A unit is a 128-query tile of one sequence and some of its key tiles of 128 keys, for a PAIR of
// heads: the shared key tile feeds both heads' score products. Bound by the tensor cores and the
// exponentials from about 100 queries up, by HBM below. The division of the warps, of tensor memory
// and the order of the products are those of the contiguous prefill (swska_prefill_tc.cu):
//   warps 0-3 / 4-7  softmax of head 0 / 1 (thread = query row = TMEM lane)
//   warp 8, 10, 11   TMA: Q of the unit and K_j; V0_j; V1_j, through a ring of four 32 KB slots
//   warp 9           TMEM allocation and MMA issue
//   TMEM: S0 | O0 | S1 | O1;  S0(0) S1(0) | PV0(j) S0(j+1) PV1(j) S1(j+1) | ...
// What the pages add: a tile of 128 keys arrives as boxes of as many rows as divide both the page
// and 128, each lane of a producer warp issuing its own (page 8: 32 boxes, one per lane; a warp issues
// one in about 100 clocks, hence three such warps), with the next tile's pages looked up while this
// one's copies run. A page that the table does not have is
// fetched as zeros and masked. Rows of a tile that no query sees may hold anything, NaN included, and
// 0 x NaN would reach the output, so the softmax warps clear those value rows before they hand over P
// (the keys need no clearing: their scores are replaced).
// Every wait is bounded; a timeout makes all roles stop, drain and raise a flag.
#include <cuda.h>
#include <math.h>

#include "extend.cuh"
#include "mma16.cuh"
#include "tc.cuh"

namespace rod {
namespace {

using mma::bits_from;
using mma::bits_to;

__device__ unsigned int g_extend_tc_timeout = 0;

constexpr int BM = kChunkRows;             // queries per tile
constexpr int BN = kChunkTile;             // keys per tile
constexpr int HD = 128;
constexpr int NSLOT = 4;
constexpr int TILE_BYTES = BM * HD * 2;
constexpr int HALF_BYTES = TILE_BYTES / 2;
constexpr int NTHREADS = 384;
// register split as in swska_prefill_tc.cu: 2 x 216 + 72 = 3 x 168
constexpr int kSoftmaxRegs = 216;
constexpr int kControlRegs = 72;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

constexpr int OFF_Q = 0;
constexpr int OFF_RING = 2 * TILE_BYTES;
constexpr int OFF_BAR = OFF_RING + NSLOT * TILE_BYTES;
// full, empty, qfull, qempty, sfull[2], pfull[2], phalf[2], odone[2], meet[2], drain, known[4]
constexpr int NBAR = 2 * NSLOT + 17;
constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
constexpr int OFF_HAVE = OFF_MISC + 24;    // per key tile (mod 4): 8-row groups whose page exists
constexpr int SMEM_BYTES = OFF_HAVE + 16 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory");

// every lane of the warp probes and all leave with the same result, so that a warp stays together
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    for (uint32_t i = 1;; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((i & 255u) == 0) {
            if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
            if (i >= kWaitLimit) {
                *abort_flag = 1;
                atomicExch(&g_extend_tc_timeout, 1u);
                return false;
            }
        }
    }
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mov.b64 rc, {%6, %7};\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__global__ void __launch_bounds__(NTHREADS, 1)
extend_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const ExtendArgs a, const ExtendRoute r, int box,
                 float scale_log2) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* full = bars;
    uint64_t* empty = bars + NSLOT;
    uint64_t* qfull = bars + 2 * NSLOT;
    uint64_t* qempty = qfull + 1;
    uint64_t* sfull = qempty + 1;
    uint64_t* pfull = sfull + 2;
    uint64_t* phalf = pfull + 2;
    uint64_t* odone = phalf + 2;
    uint64_t* meet = odone + 2;  // the softmax threads of a head, around the counter of a split tile
    uint64_t* drain = meet + 2;
    uint64_t* known = drain + 1;  // [4]: `have` of a key tile is written
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
    volatile int* came_last = reinterpret_cast<volatile int*>(smem + OFF_MISC + 8);  // [2]
    volatile uint32_t* have = reinterpret_cast<volatile uint32_t*>(smem + OFF_HAVE);

    if (threadIdx.x == 256) {
        tc::tma_prefetch_desc(&tm_q);
        tc::tma_prefetch_desc(&tm_k);
        tc::tma_prefetch_desc(&tm_v);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < NSLOT; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        for (int h = 0; h < 2; ++h) {
            mbar_init(&sfull[h], 1);
            mbar_init(&pfull[h], 128);
            mbar_init(&phalf[h], 128);
            mbar_init(&odone[h], 1);
            mbar_init(&meet[h], 128);
        }
        mbar_init(drain, 1);
        for (int i = 0; i < 4; ++i) mbar_init(&known[i], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tc::tmem_alloc(tmem_holder, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_holder;
    // This launch comes after the one for few tokens (swska_extend_few.cu), which lets it start once
    // all of its CTAs have seen the end of the launch that wrote the units and the cache: the two share
    // the GPU, and only the end of this one waits for the other.
    // neighbouring CTAs take the head pairs of one chunk: they share its keys in L2
    const int hp = blockIdx.x % r.groups;
    const int head[2] = {2 * hp, min(2 * hp + 1, a.H - 1)};  // an odd H's last pair has one head twice
    const ExtendRange range = load_range(r, blockIdx.x / r.groups);

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == 8 || warp >= 10) {
        // ------------------------------- TMA producers (all lanes): keys, values of head 0, of head 1
        const int which = warp == 8 ? 0 : warp - 9;
        const int nbox = BN / box;  // boxes of a tile's half: 1 .. 16
        int nq = 0, tiles = 0;      // ring position of this warp's load of tile t: 3 t + which
        bool ok = true;
        for (int x = range.lo; x <= range.hi && ok; ++x) {
            const ExtendUnit u = load_unit(r.units + x);
            if (u.kt0 == u.kt1) continue;
            const ExtendSeq sq{u.row0, u.len, u.ctx, false};
            const ExtendKeys kt = extend_keys(sq, u.q0, BM, BN, a.W, a.S);
            auto page_of = [&](int i) {
                return i < u.kt1 && lane < nbox ? extend_page(a, u.n, (kt.at(i) * BN + lane * box) / a.page) : -1;
            };
            int pg_next = page_of(u.kt0);
            if (which == 0) {
                if (nq > 0 && !wait_bar_warp(qempty, (uint32_t)((nq - 1) & 1), abort_flag)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(qfull, 2 * TILE_BYTES);
                    for (int h = 0; h < 2; ++h)
                        for (int half = 0; half < 2; ++half)
                            tc::tma_load_3d(smem + OFF_Q + h * TILE_BYTES + half * HALF_BYTES, &tm_q, half * 64,
                                            u.row0 + u.q0, head[h], qfull);
                }
                ++nq;
            }
            for (int i = u.kt0; i < u.kt1; ++i, ++tiles) {
                const int pg = pg_next, key0 = kt.at(i) * BN;
                pg_next = page_of(i + 1);
                uint32_t there = 0;  // bit per 8 rows
                if (which == 0) {
                    for (int b = 0; b < nbox; ++b)
                        if (__shfl_sync(0xffffffffu, pg, b) >= 0) there |= ((1u << (box / 8)) - 1u) << (b * (box / 8));
                }
                const int L = 3 * tiles + which, slot = L % NSLOT, use = L / NSLOT;
                if (use > 0 && !wait_bar_warp(&empty[slot], (uint32_t)((use - 1) & 1), abort_flag)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    if (which == 0) {
                        have[tiles & 3] = there;
                        mbar_arrive(&known[tiles & 3]);
                    }
                    mbar_arrive_expect_tx(&full[slot], TILE_BYTES);
                }
                __syncwarp();
                // lane = (half, box)
                const int b = lane % 16, half = lane / 16;
                const int p = __shfl_sync(0xffffffffu, pg, b);
                if (b < nbox) {
                    unsigned char* dst = smem + OFF_RING + slot * TILE_BYTES + half * HALF_BYTES + b * box * 128;
                    const int y = (key0 + b * box) % a.page;
                    if (which == 0) tc::tma_load_3d(dst, &tm_k, half * 64, y, p >= 0 ? p : a.P, &full[slot]);
                    else tc::tma_load_3d(dst, &tm_v, half * 64, y, p >= 0 ? p * a.H + head[which - 1] : a.P * a.H, &full[slot]);
                }
            }
        }
        // every copy that this warp started has landed before the CTA can leave: those whose slot no later
        // load takes (the others were used by products that have completed)
        if (nq > 0) mbar_wait_bounded(qfull, (uint32_t)((nq - 1) & 1), kWaitLimit);
        for (int t = tiles > 2 ? tiles - 2 : 0; t < tiles; ++t) {
            const int L = 3 * t + which;
            if (L + NSLOT >= 3 * tiles) mbar_wait_bounded(&full[L % NSLOT], (uint32_t)((L / NSLOT) & 1), kWaitLimit);
        }
    } else if (warp == 9) {
        // ------------------------------- MMA issue (whole warp) -------------------------------
        const uint32_t idesc_s = tc::idesc_bf16_f32(BM, BN, 0, 0);
        const uint32_t idesc_o = tc::idesc_bf16_f32(BM, HD, 0, 1);
        const uint32_t q_base = smem_u32(smem + OFF_Q);
        auto ring = [&](int L) { return smem_u32(smem + OFF_RING + (L % NSLOT) * TILE_BYTES); };
        auto acquire = [&](int L) {
            const bool ok = wait_bar_warp(&full[L % NSLOT], (uint32_t)((L / NSLOT) & 1), abort_flag);
            tc::fence_after_sync();
            return ok;
        };
        auto handoff = [&](uint64_t* bar, int j) {
            const bool ok = wait_bar_warp(bar, (uint32_t)(j & 1), abort_flag);
            tc::fence_after_sync();
            return ok;
        };
        const uint64_t dq0 = tc::sdesc_sw128(q_base, 16, 1024);
        const uint64_t dq1 = tc::sdesc_sw128(q_base + TILE_BYTES, 16, 1024);
        const uint32_t dk_hi = tc::desc_hi(tc::sdesc_sw128(q_base, 16, 1024));
        const uint32_t dv_hi = tc::desc_hi(tc::sdesc_sw128(q_base, HALF_BYTES, 1024));
        auto issue_s = [&](int h, int L) {
            const uint32_t a_lo = tc::desc_lo(h ? dq1 : dq0), a_hi = tc::desc_hi(h ? dq1 : dq0);
            const uint32_t b_lo = tc::desc_lo(tc::sdesc_sw128(ring(L), 16, 1024));
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                const uint32_t koff = (uint32_t)(((k / 4) * HALF_BYTES + (k % 4) * 32) >> 4);
                tc::mma_ss_lh_warp(tmem + 256u * h, a_lo + koff, a_hi, b_lo + koff, dk_hi, idesc_s, k > 0);
            }
        };
        auto issue_pv = [&](int h, int L, bool acc, int half) {
            const uint32_t b_lo = tc::desc_lo(tc::sdesc_sw128(ring(L), HALF_BYTES, 1024));
#pragma unroll
            for (int k = 4 * half; k < 4 * half + 4; ++k)
                tc::mma_ts_lh_warp(tmem + 256u * h + 128u, tmem + 256u * h + 8u * k,
                                   b_lo + (uint32_t)((2048 * k) >> 4), dv_hi, idesc_o, (acc || k > 0) ? 1u : 0u);
        };
        // ring position, tile count and unit count run on across units (the phases of the barriers)
        int Lb = 0, tb = 0, units = 0;
        bool ok = true;
        for (int x = range.lo; x <= range.hi && ok; ++x) {
            const ExtendUnit u = load_unit(r.units + x);
            const int n_it = u.kt1 - u.kt0;
            if (n_it == 0) continue;
            if (!handoff(qfull, units) || !acquire(Lb)) break;
            issue_s(0, Lb);
            tc::mma_commit_warp(&sfull[0]);
            issue_s(1, Lb);
            tc::mma_commit_warp(&sfull[1]);
            tc::mma_commit_warp(&empty[Lb % NSLOT]);
            if (n_it == 1) tc::mma_commit_warp(qempty);
            for (int j = 0; j < n_it; ++j) {
                const bool more = j + 1 < n_it;
                const int Lj = Lb + 3 * j, tj = tb + j;
                if (!acquire(Lj + 1) || !handoff(&phalf[0], tj)) { ok = false; break; }
                issue_pv(0, Lj + 1, j > 0, 0);
                if (!handoff(&pfull[0], tj)) { ok = false; break; }
                const bool k_ready =
                    more && __all_sync(0xffffffffu, mbar_test_wait(&full[(Lj + 3) % NSLOT],
                                                                   (uint32_t)(((Lj + 3) / NSLOT) & 1)));
                tc::fence_after_sync();
                issue_pv(0, Lj + 1, j > 0, 1);
                tc::mma_commit_warp(&empty[(Lj + 1) % NSLOT]);
                if (more) {
                    if (!k_ready && !acquire(Lj + 3)) { ok = false; break; }
                    issue_s(0, Lj + 3);
                    tc::mma_commit_warp(&sfull[0]);
                } else {
                    tc::mma_commit_warp(&odone[0]);
                }
                if (!acquire(Lj + 2) || !handoff(&phalf[1], tj)) { ok = false; break; }
                issue_pv(1, Lj + 2, j > 0, 0);
                if (!handoff(&pfull[1], tj)) { ok = false; break; }
                issue_pv(1, Lj + 2, j > 0, 1);
                tc::mma_commit_warp(&empty[(Lj + 2) % NSLOT]);
                if (more) {
                    issue_s(1, Lj + 3);
                    tc::mma_commit_warp(&sfull[1]);
                    tc::mma_commit_warp(&empty[(Lj + 3) % NSLOT]);
                    if (j + 2 == n_it) tc::mma_commit_warp(qempty);
                } else {
                    tc::mma_commit_warp(&odone[1]);
                }
            }
            Lb += 3 * n_it;
            tb += n_it;
            ++units;
        }
        tc::mma_commit_warp(drain);
        mbar_wait_bounded(drain, 0, kWaitLimit);
    } else if (warp < 8) {
        // ------------------------------- softmax warpgroups -------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int h = warp / 4;
        const int row = threadIdx.x % 128;
        const uint32_t lane_base = (uint32_t)(32 * (warp % 4)) << 16;
        const uint32_t tS = tmem + 256u * h + lane_base;
        const uint32_t tO = tS + 128u;
        const bool mine = 2 * hp + h < a.H;  // else the pair's head twice: nothing is stored
        int Lb = 0, tb = 0, units = 0, meets = 0;
        bool ok = true;
        for (int x = range.lo; x <= range.hi && ok; ++x) {
            const ExtendUnit u = load_unit(r.units + x);
            const int n_it = u.kt1 - u.kt0;
            const ExtendSeq sq{u.row0, u.len, u.ctx, false};
            const ExtendKeys kt = extend_keys(sq, u.q0, BM, BN, a.W, a.S);
            const int rows = min(u.len - u.q0, BM), p0 = u.ctx + u.q0, p1 = p0 + rows - 1;
            const int p = p0 + row;
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = 0; j < n_it; ++j) {
                if (!wait_bar_warp(&sfull[h], (uint32_t)((tb + j) & 1), abort_flag)) { ok = false; break; }
                tc::fence_after_sync();
                uint32_t s[BN];
                tc::tmem_ld32(tS + 0, s);
                tc::tmem_ld32(tS + 32, s + 32);
                tc::tmem_ld32(tS + 64, s + 64);
                tc::tmem_ld32(tS + 96, s + 96);
                // written when the tile's keys were asked for, and not again before this head is done with it
                if (!wait_bar_warp(&known[(tb + j) & 3], (uint32_t)(((tb + j) >> 2) & 1), abort_flag)) { ok = false; break; }
                tc::tmem_wait_ld();
                const int key0 = kt.at(u.kt0 + j) * BN;
                const uint32_t there = have[(tb + j) & 3];
                const bool all_there = there == 0xffffu;
                const bool in_reach = key0 > p1 - a.W || key0 + (BN - 1) < a.S;  // every key, for every row
                if (!all_there || !in_reach || key0 + (BN - 1) > p0) {
                    // bit per key: 32 keys a word, four page bits of eight keys each
                    const int64_t lo = (int64_t)p - key0 - a.W + 1;
                    const int hi = p - key0, first = a.S - 1 - key0;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t pages = (((there >> (4 * w) & 15u) * 0x00204081u) & 0x01010101u) * 255u;
                        const uint32_t v = pages & bits_to(hi - 32 * w) & (bits_from(lo - 32 * w) | bits_to(first - 32 * w));
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!(v >> c & 1u)) s[32 * w + c] = 0xff800000u;
                    }
                    // this thread's value row, if no query of the tile sees it: the slot is held until P is handed
                    // over, so the phase of its barrier cannot run ahead
                    const int key = key0 + row;
                    const bool seen = (there >> (row / 8) & 1u) && key <= p1 && (key > p0 - a.W || key < a.S);
                    const int Lv = Lb + 3 * j + 1 + h;
                    if (!__all_sync(0xffffffffu, seen) &&
                        !wait_bar_warp(&full[Lv % NSLOT], (uint32_t)((Lv / NSLOT) & 1), abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (!seen) {
                        unsigned char* vr = smem + OFF_RING + (Lv % NSLOT) * TILE_BYTES + row * 128;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            // neighbouring threads start at neighbouring chunks: no bank conflicts
                            const int o16 = 16 * ((c + row) & 7);
                            *reinterpret_cast<uint4*>(vr + o16) = make_uint4(0u, 0u, 0u, 0u);
                            *reinterpret_cast<uint4*>(vr + HALF_BYTES + o16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        tc::fence_proxy_async();
                    }
                    __syncwarp();
                }
                float m8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float m = __uint_as_float(s[i]);
#pragma unroll
                    for (int k = 1; k < 15; k += 2)
                        m = fmax3(m, __uint_as_float(s[8 * k + i]), __uint_as_float(s[8 * k + 8 + i]));
                    m8[i] = fmaxf(m, __uint_as_float(s[120 + i]));
                }
                const float mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
                const float m_tile = mx * scale_log2;
                const bool need = m_tile > m_run + kRescaleThreshold;
                const float alpha = need ? tc::ex2(m_run - m_tile) : 1.f;
                l_run *= alpha;
                if (need) m_run = m_tile;
                const float m_use = m_run == -INFINITY ? 0.f : m_run;
                if (j > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll
                    for (int cb = 0; cb < HD; cb += 32) {
                        uint32_t t[32];
                        tc::tmem_ld32(tO + cb, t);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) t[i] = __float_as_uint(__uint_as_float(t[i]) * alpha);
                        tc::tmem_st32(tO + cb, t);
                    }
                }
                const float2 sc2 = make_float2(scale_log2, scale_log2), nm2 = make_float2(-m_use, -m_use);
                float2 l4[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int c = 64 * half + 2 * i;
                        const float2 e = ffma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, nm2);
                        const float2 pr = make_float2(tc::ex2(e.x), tc::ex2(e.y));
                        l4[i & 3] = fadd2(l4[i & 3], pr);
                        pk[i] = pack_bf16x2(pr.x, pr.y);
                    }
                    tc::tmem_st32(tS + 32u * half, pk);
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    mbar_arrive(half == 0 ? &phalf[h] : &pfull[h]);
                }
                const float2 x2 = fadd2(l4[0], l4[1]), y2 = fadd2(l4[2], l4[3]), t2 = fadd2(x2, y2);
                l_run += t2.x + t2.y;
            }
            // the rows: output, or this unit's part of it
            if (!ok || (n_it > 0 && !wait_bar_warp(&odone[h], (uint32_t)(units & 1), abort_flag))) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            const bool live = row < rows && mine;
            const int hd = head[h];
            __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.o) + ((int64_t)(u.row0 + u.q0 + row) * a.H + hd) * HD;
            const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
            // this row's four columns of group c in a part
            auto part_col = [&](int part, int hdx, int c) {
                return r.part_o + r.part_at(part, a.H, hdx, 0) * HD + ((int64_t)c * BM + row) * 4;
            };
            const int64_t at = u.part >= 0 ? r.part_at(u.part, a.H, hd, row) : 0;
            if (n_it > 0) {
#pragma unroll
                for (int cb = 0; cb < HD; cb += 32) {
                    uint32_t t[32];
                    tc::tmem_ld32(tO + cb, t);
                    tc::tmem_wait_ld();
                    if (live && u.part < 0) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint4 w;
                            w.x = pack_bf16x2(__uint_as_float(t[i + 0]) * inv, __uint_as_float(t[i + 1]) * inv);
                            w.y = pack_bf16x2(__uint_as_float(t[i + 2]) * inv, __uint_as_float(t[i + 3]) * inv);
                            w.z = pack_bf16x2(__uint_as_float(t[i + 4]) * inv, __uint_as_float(t[i + 5]) * inv);
                            w.w = pack_bf16x2(__uint_as_float(t[i + 6]) * inv, __uint_as_float(t[i + 7]) * inv);
                            *reinterpret_cast<uint4*>(orow + cb + i) = w;
                        }
                    } else if (live) {
                        // a part's rows are stored column group by column group: neighbouring threads write
                        // neighbouring 16 bytes
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<uint4*>(part_col(u.part, hd, (cb + i) / 4)) = make_uint4(t[i], t[i + 1], t[i + 2], t[i + 3]);
                    }
                }
                Lb += 3 * n_it;
                tb += n_it;
                ++units;
            }
            if (u.part < 0) continue;
            if (live) r.part_ml[at] = make_float2(m_run, l_run);
            // the head's threads meet, one counts, and if the part was the last of the tile they add all
            // (the second meeting also keeps the next unit's rows behind this one's)
            __threadfence();
            mbar_arrive(&meet[h]);
            if (!wait_bar_warp(&meet[h], (uint32_t)(meets++ & 1), abort_flag)) { ok = false; break; }
            if (row == 0) {
                came_last[h] = mine && atomicAdd(r.count + (int64_t)u.counter * a.H + hd, 1) == u.nsplit - 1;
                __threadfence();
            }
            mbar_arrive(&meet[h]);
            if (!wait_bar_warp(&meet[h], (uint32_t)(meets++ & 1), abort_flag)) { ok = false; break; }
            if (!came_last[h]) continue;
            __threadfence();
            // every thread adds its row: the maximum and sum first, then 32 columns at a time with the loads of
            // four parts in flight. One chunk of 64 tokens, H 16, W 4096: 42.2 us with two parts, 43.1 with 16
            // columns of eight, 38.2 so; one of 512 tokens 61.0, 59.3 and 57.9
            if (row >= rows) continue;
            float M = -INFINITY, Lsum = 0.f;
#pragma unroll 4
            for (int s = 0; s < u.nsplit; ++s) {
                const float2 ml = __ldcg(&r.part_ml[r.part_at(u.part_of(s), a.H, hd, row)]);
                const float mn = fmaxf(M, ml.x), base = mn == -INFINITY ? 0.f : mn;
                Lsum = fmaf(ml.y, tc::ex2(ml.x - base), Lsum * tc::ex2(M - base));
                M = mn;
            }
            const float base = M == -INFINITY ? 0.f : M, iv = Lsum == 0.f ? 0.f : 1.f / Lsum;
            for (int cb = 0; cb < HD; cb += 32) {
                float4 O[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) O[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int s0 = 0; s0 < u.nsplit; s0 += 4) {
                    float4 x4[4][8];
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int part = u.part_of(s0 + e < u.nsplit ? s0 + e : 0);
                        const float m = s0 + e < u.nsplit ? __ldcg(&r.part_ml[r.part_at(part, a.H, hd, row)].x) : -INFINITY;
                        const float4* x = reinterpret_cast<const float4*>(part_col(part, hd, cb / 4));
                        w[e] = tc::ex2(m - base) * iv;
                        // nothing seen there (an empty part holds no output): zeros
#pragma unroll
                        for (int i = 0; i < 8; ++i) x4[e][i] = m != -INFINITY ? __ldcg(x + i * BM) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            O[i].x = fmaf(x4[e][i].x, w[e], O[i].x);
                            O[i].y = fmaf(x4[e][i].y, w[e], O[i].y);
                            O[i].z = fmaf(x4[e][i].z, w[e], O[i].z);
                            O[i].w = fmaf(x4[e][i].w, w[e], O[i].w);
                        }
                }
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    uint4 wv;
                    wv.x = pack_bf16x2(O[i].x, O[i].y);
                    wv.y = pack_bf16x2(O[i].z, O[i].w);
                    wv.z = pack_bf16x2(O[i + 1].x, O[i + 1].y);
                    wv.w = pack_bf16x2(O[i + 1].z, O[i + 1].w);
                    *reinterpret_cast<uint4*>(orow + cb + 4 * i) = wv;
                }
            }
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 9) tc::tmem_dealloc(tmem, 512);
    wait_for_launch_before();
}

}  // namespace

cudaError_t swska_extend_tc_launch(const ExtendArgs& a, const ExtendRoute& r, cudaStream_t s) {
    int box = BN;
    while (a.page % box != 0) box /= 2;
    CUtensorMap mq, mk, mv;
    cudaError_t e;
    // q [M][H][128] read as H matrices of M rows
    if ((e = make_tmap_bf16_3d_strided(&mq, a.q, HD, (uint64_t)a.M, (uint64_t)a.H, (uint64_t)a.H * HD * 2, HD * 2, 64, BM)) !=
        cudaSuccess)
        return e;
    if ((e = make_tmap_bf16_3d(&mk, a.k_pool, HD, (uint64_t)a.page, (uint64_t)a.P, 64, (uint32_t)box)) != cudaSuccess) return e;
    if ((e = make_tmap_bf16_3d(&mv, a.v_pool, HD, (uint64_t)a.page, (uint64_t)a.P * a.H, 64, (uint32_t)box)) != cudaSuccess)
        return e;
    static std::atomic<uint64_t> smem_set{0};
    if ((e = allow_smem(smem_set, (const void*)extend_tc_kernel, SMEM_BYTES)) != cudaSuccess) return e;
    e = launch_overlapped(extend_tc_kernel, dim3((unsigned)(r.cols * r.groups)), dim3(NTHREADS), (size_t)SMEM_BYTES, s, mq, mk, mv, a, r,
                          box, a.scale * 1.4426950408889634f);
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

unsigned swska_extend_tc_take_timeout_flag() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_extend_tc_timeout, sizeof(v)) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_extend_tc_timeout, &zero, sizeof(zero));
    return v;
}

}  // namespace rod
