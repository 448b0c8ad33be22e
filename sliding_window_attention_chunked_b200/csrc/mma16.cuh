// mma16.cuh -- warp-level m16n8k16 bf16 products and the fragment loads that feed them.
//
// A fragment of A (16 rows x 16) is four registers: rows g and g + 8 (g = lane / 4), columns c and
// c + 1, c + 8 and c + 9 (c = 2 (lane mod 4)); of B (16 x 8 columns) two, with the columns in g and
// the rows in c; the sum has rows g (elements 0, 1) and g + 8 (2, 3), columns c, c + 1. So the sums of
// two neighbouring 8-column tiles, rounded to bf16 in pairs, are an A fragment of the next product.
#pragma once

#include "common.cuh"

namespace rod {
namespace mma {

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, const uint32_t* b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// A fragment from two neighbouring 8-column sums
__device__ __forceinline__ void to_a(const float* lo, const float* hi, uint32_t* a) {
    a[0] = pack_bf16x2(lo[0], lo[1]);
    a[1] = pack_bf16x2(lo[2], lo[3]);
    a[2] = pack_bf16x2(hi[0], hi[1]);
    a[3] = pack_bf16x2(hi[2], hi[3]);
}
// bits 0 .. x and bits x .. 31 of a word, for any x
__device__ __forceinline__ uint32_t bits_to(int x) { return x < 0 ? 0u : (x >= 31 ? 0xffffffffu : (2u << x) - 1u); }
__device__ __forceinline__ uint32_t bits_from(int64_t x) { return x <= 0 ? 0xffffffffu : (x > 31 ? 0u : 0xffffffffu << x); }

}  // namespace mma
}  // namespace rod
