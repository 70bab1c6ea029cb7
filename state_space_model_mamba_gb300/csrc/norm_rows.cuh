// norm_rows.cuh -- what the norm kernels share (norm.cu, norm_group.cu): rows in vectors of
// a thread, and sums over the threads of a row.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "norm.h"
#include "ssd_internal.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace norm_rows {

using tc::ffma2;
using tc::fmul2;

// sums of pairs
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// ---- VEC consecutive elements of a row, in 32-bit words as they are stored (VEC sizeof(T) bytes, at most 16 a load)
template <typename T, int VEC>
struct Vec {
    static constexpr int BYTES = VEC * (int)sizeof(T), WORDS = (BYTES + 3) / 4;
    uint32_t w[WORDS];
    // ONCE: evicted from the caches first, as a row that is read once may be
    template <typename W, bool ONCE>
    static __device__ __forceinline__ W ld(const W *p) {
        if constexpr (ONCE)
            return __ldcs(p);
        else
            return __ldg(p);
    }
    template <bool ONCE = false>
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (BYTES == 32) {
            const uint4 a = ld<uint4, ONCE>((const uint4 *)p), b = ld<uint4, ONCE>((const uint4 *)p + 1);
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        } else if constexpr (BYTES == 16) {
            const uint4 a = ld<uint4, ONCE>((const uint4 *)p);
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        } else if constexpr (BYTES == 8) {
            const uint2 a = ld<uint2, ONCE>((const uint2 *)p);
            w[0] = a.x, w[1] = a.y;
        } else if constexpr (BYTES == 4) {
            w[0] = ld<uint32_t, ONCE>((const uint32_t *)p);
        } else {
            w[0] = ld<unsigned short, ONCE>((const unsigned short *)p);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
    }
    // elements 2 i and 2 i + 1 (VEC = 1: the element and 0)
    [[maybe_unused]] static constexpr int PAIRS = (VEC + 1) / 2;
    __device__ __forceinline__ float2 get(int i) const {
        if constexpr (sizeof(T) == 4)
            return make_float2(__uint_as_float(w[2 * i]), VEC > 1 ? __uint_as_float(w[2 * i + (VEC > 1)]) : 0.f);
        else
            return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    __device__ __forceinline__ void set(int i, float2 f) {
        if constexpr (sizeof(T) == 4) {
            w[2 * i] = __float_as_uint(f.x);
            if (VEC > 1) w[2 * i + (VEC > 1)] = __float_as_uint(f.y);
        } else {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
            w[i] = *(const uint32_t *)&v;
        }
    }
    // what added leaves every value as it is
    __device__ __forceinline__ void minus_zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
    }
    // the sum rounded to T (in bf16 the same as the fp32 sum rounded: 24 bits are more than twice 8 and two)
    __device__ __forceinline__ void add(const Vec &o) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (sizeof(T) == 4)
                w[i] = __float_as_uint(__uint_as_float(w[i]) + __uint_as_float(o.w[i]));
            else {
                const __nv_bfloat162 v = __hadd2(*(const __nv_bfloat162 *)&w[i], *(const __nv_bfloat162 *)&o.w[i]);
                w[i] = *(const uint32_t *)&v;
            }
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (BYTES == 32) {
            ((uint4 *)p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            ((uint4 *)p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else if constexpr (BYTES == 16) {
            *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
        } else if constexpr (BYTES == 8) {
            *(uint2 *)p = make_uint2(w[0], w[1]);
        } else if constexpr (BYTES == 4) {
            *(uint32_t *)p = w[0];
        } else {
            *(unsigned short *)p = (unsigned short)w[0];
        }
    }
};

struct Sum {
    static __device__ __forceinline__ float op(float a, float b) { return a + b; }
};
// Reduction of K values over the TPR threads of a row; every thread gets the results.  `buf` holds K floats
// per warp, twice: `turn` alternates between reductions, so that one barrier each is enough.
template <typename Op, int TPR, int K>
__device__ __forceinline__ void row_reduce(float (&x)[K], float (*buf)[32][K], int &turn) {
#pragma unroll
    for (int o = TPR < 32 ? TPR / 2 : 16; o; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] = Op::op(x[k], __shfl_xor_sync(0xffffffffu, x[k], o));
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x / 32, w0 = warp / (TPR / 32) * (TPR / 32);
        float(*b)[K] = buf[turn];
        turn ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) b[warp][k] = x[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] = b[w0][k];
#pragma unroll
        for (int i = 1; i < TPR / 32; ++i)
#pragma unroll
            for (int k = 0; k < K; ++k) x[k] = Op::op(x[k], b[w0 + i][k]);
    }
}

}  // namespace norm_rows
}  // namespace ssd
