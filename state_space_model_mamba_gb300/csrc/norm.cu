// norm.cu -- the block's entry norm (include/norm.h): residual addition and
// root-mean-square norm in one pass over the row, the output in the stream's
// type or in e4m3 with scales, and the backward.
//
// All three are streams bound by HBM: a row is read once into registers, its
// sum of squares reduced over the block, and the outputs written from the
// registers.  A row is held by TPR threads with NV vectors of VEC columns
// each, vector j of thread t at columns (j TPR + t) VEC, so that every load of
// a warp is contiguous (512 bytes at VEC = 8 in bf16).  VEC is 8 where D is a
// multiple of 8, else 2 or 1: rows then start on the vector's alignment.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdio.h>

#include "norm.h"
#include "ssd_internal.cuh"

namespace ssd {
namespace {

constexpr float kE4m3Max = 448.f;

// ---- VEC consecutive elements of a row as floats (aligned to the vector's size, or to 16 bytes)
template <typename T, int VEC>
struct Vec;
template <>
struct Vec<bf16, 8> {
    static __device__ __forceinline__ void ld(const bf16 *p, float *f) {
        const uint4 u = __ldg((const uint4 *)p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ void st(bf16 *p, const float *f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *(const uint32_t *)&v;
        }
        *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec<float, 8> {
    static __device__ __forceinline__ void ld(const float *p, float *f) {
        const float4 a = __ldg((const float4 *)p), b = __ldg((const float4 *)p + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    static __device__ __forceinline__ void st(float *p, const float *f) {
        ((float4 *)p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        ((float4 *)p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};
template <>
struct Vec<bf16, 2> {
    static __device__ __forceinline__ void ld(const bf16 *p, float *f) {
        const uint32_t u = __ldg((const uint32_t *)p);
        f[0] = __uint_as_float(u << 16);
        f[1] = __uint_as_float(u & 0xFFFF0000u);
    }
    static __device__ __forceinline__ void st(bf16 *p, const float *f) {
        *(__nv_bfloat162 *)p = __floats2bfloat162_rn(f[0], f[1]);
    }
};
template <>
struct Vec<float, 2> {
    static __device__ __forceinline__ void ld(const float *p, float *f) {
        const float2 a = __ldg((const float2 *)p);
        f[0] = a.x, f[1] = a.y;
    }
    static __device__ __forceinline__ void st(float *p, const float *f) { *(float2 *)p = make_float2(f[0], f[1]); }
};
template <typename T>
struct Vec<T, 1> {
    static __device__ __forceinline__ void ld(const T *p, float *f) { f[0] = (float)*p; }
    static __device__ __forceinline__ void st(T *p, const float *f) { *p = (T)f[0]; }
};

// e4m3 bytes of VEC floats
template <int VEC>
__device__ __forceinline__ void st_e4m3(uint8_t *p, const float *f) {
    if constexpr (VEC == 1) {
        *p = __nv_cvt_float_to_fp8(f[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint16_t h[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            h[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        if constexpr (VEC == 2)
            *(uint16_t *)p = h[0];
        else
            *(uint2 *)p = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
    }
}

// a maximum that keeps NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
struct Sum {
    static __device__ __forceinline__ float op(float a, float b) { return a + b; }
};
struct Max {
    static __device__ __forceinline__ float op(float a, float b) { return max_nan(a, b); }
};
// Reduction over the TPR threads of a row; every thread gets the result.  `buf` has a float per warp.
template <typename Op, int TPR>
__device__ __forceinline__ float row_reduce(float x, float *buf) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = Op::op(x, __shfl_xor_sync(0xffffffffu, x, o));
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x / 32, w0 = warp / (TPR / 32) * (TPR / 32);
        __syncthreads();  // buf may still be read from the reduction before
        if ((threadIdx.x & 31) == 0) buf[warp] = x;
        __syncthreads();
        x = buf[w0];
#pragma unroll
        for (int i = 1; i < TPR / 32; ++i) x = Op::op(x, buf[w0 + i]);
    }
    return x;
}

struct NormArgs {
    const void *x, *residual;
    const float *weight;
    float eps;
    void *y;             // T, or e4m3 bytes
    float *scales;       // null: y in T
    void *stream;        // may be null
    long long rows;
    int D, group;        // group 0: a scale per row
};

// ------------------------------------------------------------------ forward
template <typename T, int VEC, int TPR, int NV, bool FP8>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) add_rms_kernel(NormArgs a) {
    __shared__ float buf[32];
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
    const long long row = blockIdx.x * (long long)RPB + threadIdx.x / TPR;
    const int t = threadIdx.x % TPR;
    const bool live = row < a.rows;
    const long long at = row * a.D;
    float f[NV][VEC];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + t) * VEC;
        if (live && c < a.D) {
            Vec<T, VEC>::ld((const T *)a.x + at + c, f[j]);
            if (a.residual) {
                float r[VEC];
                Vec<T, VEC>::ld((const T *)a.residual + at + c, r);
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[j][i] = (float)(T)(f[j][i] + r[i]);  // the stream as it is stored
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[j][i] = 0.f;
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + t) * VEC;
        if (a.stream && live && c < a.D) Vec<T, VEC>::st((T *)a.stream + at + c, f[j]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) ss += f[j][i] * f[j][i];
    }
    ss = row_reduce<Sum, TPR>(ss, buf);
    const float rstd = rsqrtf(ss / (float)a.D + a.eps);
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + t) * VEC;
        if (c < a.D) {
            float w[VEC];
            Vec<float, VEC>::ld(a.weight + c, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                f[j][i] = f[j][i] * rstd * w[i];
                if (FP8) amax = max_nan(amax, fabsf(f[j][i]));
            }
            if (!FP8 && live) Vec<T, VEC>::st((T *)a.y + at + c, f[j]);
        }
        if constexpr (FP8 && VEC == 8) {
            if (a.group) {  // group / 8 neighbouring lanes hold a group's columns of vector j
                float m = amax;
                for (int o = a.group / 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                amax = 0.f;
                const float s = m / kE4m3Max;
                if (live && c < a.D) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) f[j][i] = m == 0.f ? 0.f : f[j][i] / s;
                    st_e4m3<VEC>((uint8_t *)a.y + at + c, f[j]);
                    if (c % a.group == 0) a.scales[row * (a.D / a.group) + c / a.group] = s;
                }
            }
        }
    }
    if constexpr (FP8) {
        if (a.group) return;
        const float m = row_reduce<Max, TPR>(amax, buf), s = m / kE4m3Max;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            if (live && c < a.D) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[j][i] = m == 0.f ? 0.f : f[j][i] / s;
                st_e4m3<VEC>((uint8_t *)a.y + at + c, f[j]);
            }
        }
        if (live && t == 0) a.scales[row] = s;
    }
}

// ------------------------------------------------------------------ backward
// Blocks walk rows blockIdx.x, + gridDim.x, ...; a thread's columns are the
// same in every row, so its share of dweight stays in registers and leaves as
// one partial row per block, which a second kernel adds in the blocks' order.
template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(TPR) rms_bwd_kernel(const T *dy, const T *h, const float *weight, float eps,
                                                      const T *d_stream, T *dx, float *part, long long rows, int D) {
    __shared__ float buf[2][32];
    const int t = threadIdx.x;
    float w[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + t) * VEC;
        if (c < D) Vec<float, VEC>::ld(weight + c, w[j]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            dw[j][i] = 0.f;
            if (c >= D) w[j][i] = 0.f;
        }
    }
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        const long long at = row * D;
        float hv[NV][VEC], dv[NV][VEC], sv[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) hv[j][i] = dv[j][i] = sv[j][i] = 0.f;
            if (c < D) {
                Vec<T, VEC>::ld(h + at + c, hv[j]);
                Vec<T, VEC>::ld(dy + at + c, dv[j]);
                if (d_stream) Vec<T, VEC>::ld(d_stream + at + c, sv[j]);
            }
        }
        float ss = 0.f, th = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                ss += hv[j][i] * hv[j][i];
                th += dv[j][i] * w[j][i] * hv[j][i];
            }
        ss = row_reduce<Sum, TPR>(ss, buf[0]);
        th = row_reduce<Sum, TPR>(th, buf[1]);
        const float rstd = rsqrtf(ss / (float)D + eps);
        const float coef = rstd * rstd * (th / (float)D);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            if (c < D) {
                float out[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    out[i] = sv[j][i] + rstd * (dv[j][i] * w[j][i] - hv[j][i] * coef);
                    dw[j][i] += dv[j][i] * hv[j][i] * rstd;
                }
                Vec<T, VEC>::st(dx + at + c, out);
            }
        }
    }
    if (part) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            if (c < D) Vec<float, VEC>::st(part + (long long)blockIdx.x * D + c, dw[j]);
        }
    }
}

// dweight[c] = the sum over the blocks' partial rows: 32 columns a block, 8 rows of threads, fixed order.
__global__ void __launch_bounds__(256) rms_dweight_reduce(const float *part, float *dweight, int blocks, int D) {
    __shared__ float red[8][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
    float a = 0.f;
    if (c < D)
        for (int i = r; i < blocks; i += 8) a += part[(long long)i * D + c];
    red[r][threadIdx.x & 31] = a;
    __syncthreads();
    if (r == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) a += red[i][threadIdx.x];
        dweight[c] = a;
    }
}

// ------------------------------------------------------------------ host side
constexpr long long kMaxD = 16384;
constexpr int kBwdBlocks = 608;  // four per SM

ssd_status norm_fail(ssd_status st, const char *msg) {
    record_error(msg);
    return st;
}
bool al16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
ssd_status check(ssd_dtype dtype, const void *const *req, int nreq, const void *const *opt, int nopt, int64_t rows,
                 int64_t D) {
    if (dtype != SSD_F32 && dtype != SSD_BF16) return norm_fail(SSD_ERR_INVALID_ARG, "unknown dtype");
    if (rows < 1 || D < 1) return norm_fail(SSD_ERR_INVALID_ARG, "every dimension must be >= 1");
    if (D > kMaxD) return norm_fail(SSD_ERR_UNSUPPORTED, "more than 16384 columns");
    if (rows > (1LL << 31) - 1) return norm_fail(SSD_ERR_UNSUPPORTED, "problem too large");
    for (int i = 0; i < nreq; ++i)
        if (!req[i] || !al16(req[i])) return norm_fail(SSD_ERR_INVALID_ARG, "a required pointer is NULL or not 16-byte aligned");
    for (int i = 0; i < nopt; ++i)
        if (!al16(opt[i])) return norm_fail(SSD_ERR_INVALID_ARG, "a pointer is not 16-byte aligned");
    return SSD_OK;
}
ssd_status norm_cuda(cudaError_t e) {
    if (e == cudaSuccess) return SSD_OK;
    char msg[256];
    snprintf(msg, sizeof(msg), "launch failed: %s", cudaGetErrorString(e));
    return norm_fail(SSD_ERR_CUDA, msg);
}
int vec_of(int64_t D) { return D % 8 == 0 ? 8 : (D % 2 == 0 ? 2 : 1); }

// Calls f<VEC, TPR, NV> with a row's threads: the fewest of 32 .. 1024 that hold D columns in two vectors of
// 8 (four where that passes 1024 threads), or in up to 16 of the narrow vectors.
#define NORM_BY_D(F)                                                         \
    do {                                                                     \
        const int vec_ = vec_of(D);                                          \
        const int64_t n_ = D / vec_;                                         \
        if (vec_ == 8) {                                                     \
            if (n_ <= 32) F(8, 32, 1);                                       \
            else if (n_ <= 64) F(8, 32, 2);                                  \
            else if (n_ <= 128) F(8, 64, 2);                                 \
            else if (n_ <= 256) F(8, 128, 2);                                \
            else if (n_ <= 320) F(8, 160, 2);                                \
            else if (n_ <= 512) F(8, 256, 2);                                \
            else if (n_ <= 1024) F(8, 512, 2);                               \
            else F(8, 1024, 2);                                              \
        } else if (vec_ == 2) {                                              \
            if (n_ <= 512) F(2, 128, 4);                                     \
            else if (n_ <= 2048) F(2, 256, 8);                               \
            else F(2, 1024, 8);                                              \
        } else {                                                             \
            if (n_ <= 512) F(1, 128, 4);                                     \
            else if (n_ <= 4096) F(1, 512, 8);                               \
            else F(1, 1024, 16);                                             \
        }                                                                    \
    } while (0)

template <typename T, bool FP8>
cudaError_t forward(const NormArgs &a, cudaStream_t s) {
    const int64_t D = a.D;
#define F(V, TPR, NV)                                                                       \
    do {                                                                                    \
        constexpr int rpb = TPR < 128 ? 128 / TPR : 1;                                      \
        add_rms_kernel<T, V, TPR, NV, FP8>                                                  \
            <<<(unsigned)((a.rows + rpb - 1) / rpb), TPR * rpb, 0, s>>>(a);                 \
    } while (0)
    NORM_BY_D(F);
#undef F
    return cudaGetLastError();
}
int bwd_blocks(int64_t rows) { return (int)(rows < kBwdBlocks ? rows : kBwdBlocks); }
template <typename T>
cudaError_t backward(const void *dy, const void *h, const float *weight, float eps, const void *ds, void *dx, float *dw,
                     int64_t rows, int64_t D, float *part, cudaStream_t s) {
    const int blocks = bwd_blocks(rows);
#define F(V, TPR, NV)                                                                                     \
    rms_bwd_kernel<T, V, TPR, NV><<<blocks, TPR, 0, s>>>((const T *)dy, (const T *)h, weight, eps,        \
                                                         (const T *)ds, (T *)dx, dw ? part : nullptr, rows, (int)D)
    NORM_BY_D(F);
#undef F
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !dw) return e;
    rms_dweight_reduce<<<(unsigned)((D + 31) / 32), 256, 0, s>>>(part, dw, blocks, (int)D);
    return cudaGetLastError();
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status norm_add_rms(ssd_dtype dtype, const void *x, const void *residual, const float *weight, float eps,
                        void *y, void *stream_out, int64_t rows, int64_t D, void *stream_) {
    record_error("");
    const void *req[] = {x, weight, y}, *opt[] = {residual, stream_out};
    ssd_status st = check(dtype, req, 3, opt, 2, rows, D);
    if (st != SSD_OK) return st;
    if (residual && !stream_out) return norm_fail(SSD_ERR_INVALID_ARG, "stream_out is NULL with a residual");
    const NormArgs a{x, residual, weight, eps, y, nullptr, stream_out, rows, (int)D, 0};
    return norm_cuda(dtype == SSD_BF16 ? forward<bf16, false>(a, (cudaStream_t)stream_)
                                       : forward<float, false>(a, (cudaStream_t)stream_));
}

ssd_status norm_add_rms_fp8(ssd_dtype dtype, const void *x, const void *residual, const float *weight, float eps,
                            void *y8, float *scales, void *stream_out, int64_t rows, int64_t D, int64_t group,
                            void *stream_) {
    record_error("");
    const void *req[] = {x, weight, y8, scales}, *opt[] = {residual, stream_out};
    ssd_status st = check(dtype, req, 4, opt, 2, rows, D);
    if (st != SSD_OK) return st;
    if (residual && !stream_out) return norm_fail(SSD_ERR_INVALID_ARG, "stream_out is NULL with a residual");
    if (!(group == 0 || ((group == 32 || group == 64 || group == 128) && D % group == 0)))
        return norm_fail(SSD_ERR_UNSUPPORTED, "group must be 0, 32, 64 or 128 and divide the columns");
    const NormArgs a{x, residual, weight, eps, y8, scales, stream_out, rows, (int)D, (int)group};
    return norm_cuda(dtype == SSD_BF16 ? forward<bf16, true>(a, (cudaStream_t)stream_)
                                       : forward<float, true>(a, (cudaStream_t)stream_));
}

size_t norm_backward_workspace_bytes(int64_t rows, int64_t D) {
    if (rows < 1 || D < 1 || D > kMaxD) return 0;
    return sizeof(float) * (size_t)bwd_blocks(rows) * (size_t)D;
}

ssd_status norm_add_rms_backward(ssd_dtype dtype, const void *dy, const void *h, const float *weight, float eps,
                                 const void *d_stream, void *dx, float *dweight, int64_t rows, int64_t D,
                                 void *workspace, size_t workspace_bytes, void *stream_) {
    record_error("");
    const void *req[] = {dy, h, weight, dx, workspace}, *opt[] = {d_stream, dweight};
    ssd_status st = check(dtype, req, dweight ? 5 : 4, opt, 2, rows, D);
    if (st != SSD_OK) return st;
    if (dweight && workspace_bytes < norm_backward_workspace_bytes(rows, D))
        return norm_fail(SSD_ERR_WORKSPACE, "workspace too small");
    return norm_cuda(dtype == SSD_BF16
                         ? backward<bf16>(dy, h, weight, eps, d_stream, dx, dweight, rows, D, (float *)workspace,
                                          (cudaStream_t)stream_)
                         : backward<float>(dy, h, weight, eps, d_stream, dx, dweight, rows, D, (float *)workspace,
                                           (cudaStream_t)stream_));
}

}  // extern "C"
