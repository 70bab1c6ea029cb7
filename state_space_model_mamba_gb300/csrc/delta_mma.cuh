// delta_mma.cuh -- warp-level building blocks of the chunked delta-rule
// kernels: asynchronous 16-byte copies, 8x8 matrix loads and stores of swizzled
// shared-memory tiles, and the register-fed matrix instructions.
//
// Tiles are rows of bf16 in 128- or 256-byte lines; the 16-byte piece c of row
// r is kept at c ^ (r & 7), so that the eight rows of one 8x8 matrix fall on
// different banks.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "tc_ptx.cuh"

namespace ssd {
namespace delta {

using tc::smem_u32;

// ---- copies
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// byte offset of 16-byte piece c of row r, rows of LINE bytes
template <int LINE>
__device__ __forceinline__ uint32_t swz(int r, int c) {
    return (uint32_t)(r * LINE + ((c ^ (r & 7)) << 4));
}
// 16x16 blocks of bf16, rows of 32 bytes: the two pieces of rows 4-7 are exchanged
__device__ __forceinline__ uint32_t blk_swz(int r, int c) { return (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4)); }
// index of block (i, j), j <= i, of a lower triangle of 16x16 blocks
__device__ __forceinline__ constexpr int blk_at(int i, int j) { return i * (i + 1) / 2 + j; }

// ---- 8x8 matrices
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

// ---- matrix instructions, fp32 accumulators in the registers of one warp:
// element (row l / 4, columns 2 (l % 4), +1) and the same of row + 8.
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---- an fp32 pair as two bf16 pairs, x = hi + lo up to 2^-17 of x.  The products of an
// exact bf16 operand with both keep fp32 outputs (states, gate gradients) at fp32-like
// error, where one bf16 alone would leave 2^-9.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = tc::pack_bf2(x, y);
    lo = tc::pack_bf2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
}
// A operand (16 rows x 16 columns) from two neighbouring accumulator tiles
__device__ __forceinline__ void split_frag(const float (&t0)[4], const float (&t1)[4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(t0[0], t0[1], hi[0], lo[0]);
    split2(t0[2], t0[3], hi[1], lo[1]);
    split2(t1[0], t1[1], hi[2], lo[2]);
    split2(t1[2], t1[3], hi[3], lo[3]);
}
// the same with the columns scaled: s0 for t0's pair, s1 for t1's
__device__ __forceinline__ void split_frag(const float (&t0)[4], const float (&t1)[4], float2 s0, float2 s1,
                                           uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(t0[0] * s0.x, t0[1] * s0.y, hi[0], lo[0]);
    split2(t0[2] * s0.x, t0[3] * s0.y, hi[1], lo[1]);
    split2(t1[0] * s1.x, t1[1] * s1.y, hi[2], lo[2]);
    split2(t1[2] * s1.x, t1[3] * s1.y, hi[3], lo[3]);
}

}  // namespace delta
}  // namespace ssd
