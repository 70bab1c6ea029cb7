// delta_mma.cuh -- building blocks of the chunked delta-rule kernels beside
// tc_ptx.cuh: copies addressed in shared memory, the unswizzled operand, and fp32
// values as two bf16 parts.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "tc_ptx.cuh"

namespace ssd {
namespace delta {

using tc::smem_u32;

// ---- copies
__device__ __forceinline__ void tma_tile(uint32_t dst, const void *map, uint64_t *bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// shared to global; the issuing thread's group of stores is waited for with bulk_wait_*
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
// the loads into the L2 cache only, ahead of their use
__device__ __forceinline__ void prefetch_tile(const void *map, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(map), "r"(c0), "r"(c1),
                 "r"(c2), "r"(c3)
                 : "memory");
}
__device__ __forceinline__ void prefetch_bulk(const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// ---- descriptors of operands kept without swizzle (8x8 matrices of 128 contiguous bytes): lbo is the distance of
// neighbouring matrices along K, sbo along M
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t base, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((base & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | (uint64_t)1 << 46;
}
// a descriptor moved by `bytes`
__device__ __forceinline__ uint64_t sdesc_add(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// ---- two or three sets of 16 accumulator columns of this warp's 32 lanes, one wait
__device__ __forceinline__ void tmem_ld16x2(uint32_t t0, uint32_t t1, float *v0, float *v1) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t0), "r"(t1)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v0[i] = __uint_as_float(r[0 + i]), v1[i] = __uint_as_float(r[16 + i]);
}
__device__ __forceinline__ void tmem_ld16x3(uint32_t t0, uint32_t t1, uint32_t t2, float *v0, float *v1, float *v2) {
    uint32_t r[48];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%48];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%49];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47}, [%50];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47])
        : "r"(t0), "r"(t1), "r"(t2)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v0[i] = __uint_as_float(r[0 + i]), v1[i] = __uint_as_float(r[16 + i]), v2[i] = __uint_as_float(r[32 + i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
        "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
        "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
        "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// off by 2^-22 of the result, a thirtieth of what operands in two parts are off by
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- an fp32 pair as two bf16 pairs, x = hi + lo up to 2^-16 of x (2^-18 on average).  The products of an
// exact bf16 operand with both keep fp32 outputs (states, gate gradients) at fp32-like
// error, where one bf16 alone would leave 2^-8.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = tc::pack_bf2(x, y);
    const float2 r = tc::ffma2(tc::bf2_to_f2(hi), make_float2(-1.f, -1.f), make_float2(x, y));
    lo = tc::pack_bf2(r.x, r.y);
}

// and what the two parts leave: x = hi + lo + rest up to 2^-25 of x
__device__ __forceinline__ void split3(float x, float y, uint32_t &hi, uint32_t &lo, uint32_t &rest) {
    const float2 minus = make_float2(-1.f, -1.f);
    hi = tc::pack_bf2(x, y);
    const float2 r = tc::ffma2(tc::bf2_to_f2(hi), minus, make_float2(x, y));
    lo = tc::pack_bf2(r.x, r.y);
    const float2 e = tc::ffma2(tc::bf2_to_f2(lo), minus, r);
    rest = tc::pack_bf2(e.x, e.y);
}

// 8 values as one 16-byte piece of row `row` of a hi and of a lo tile (SW128)
__device__ __forceinline__ void store_parts8(uint32_t hi_tile, uint32_t lo_tile, int row, int piece, const float2 *x) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(x[e].x, x[e].y, h[e], l[e]);
    tc::st_shared_v4(hi_tile + tc::sw128_chunk(row, piece), h[0], h[1], h[2], h[3]);
    tc::st_shared_v4(lo_tile + tc::sw128_chunk(row, piece), l[0], l[1], l[2], l[3]);
}
// in three parts
__device__ __forceinline__ void store_parts8(uint32_t hi_tile, uint32_t lo_tile, uint32_t rest_tile, int row, int piece, const float2 *x) {
    uint32_t h[4], l[4], r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split3(x[e].x, x[e].y, h[e], l[e], r[e]);
    const uint32_t at = tc::sw128_chunk(row, piece);
    tc::st_shared_v4(hi_tile + at, h[0], h[1], h[2], h[3]);
    tc::st_shared_v4(lo_tile + at, l[0], l[1], l[2], l[3]);
    tc::st_shared_v4(rest_tile + at, r[0], r[1], r[2], r[3]);
}
// the same to global memory, the lo tile `lo_off` bytes behind the hi one
__device__ __forceinline__ void store_parts8(char *tile, int lo_off, int row, int piece, const float2 *x) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(x[e].x, x[e].y, h[e], l[e]);
    char *dst = tile + tc::sw128_chunk(row, piece);
    *(uint4 *)dst = make_uint4(h[0], h[1], h[2], h[3]);
    *(uint4 *)(dst + lo_off) = make_uint4(l[0], l[1], l[2], l[3]);
}
// the sum of hi and lo parts
__device__ __forceinline__ void join8(const uint4 hi, const uint4 lo, float2 *x) {
    const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = tc::ffma2(tc::bf2_to_f2(l[e]), make_float2(1.f, 1.f), tc::bf2_to_f2(h[e]));
}
// sum of products with 8 bf16 values
__device__ __forceinline__ float dot8(const uint4 w, const float2 *x, float acc) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    float2 a = make_float2(acc, 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) a = tc::ffma2(tc::bf2_to_f2(v[e]), x[e], a);
    return a.x + a.y;
}
__device__ __forceinline__ uint4 pack8(const float2 *x) {
    return make_uint4(tc::pack_bf2(x[0].x, x[0].y), tc::pack_bf2(x[1].x, x[1].y), tc::pack_bf2(x[2].x, x[2].y),
                      tc::pack_bf2(x[3].x, x[3].y));
}

}  // namespace delta
}  // namespace ssd
