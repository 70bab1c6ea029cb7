// norm.cu -- the block's entry norm (include/norm.h): residual addition and
// root-mean-square norm in one pass over the row, the output in the stream's
// type or in e4m3 with scales, and the backward.
//
// All three are streams bound by HBM.  A row is held by TPR threads with NV vectors of
// VEC columns each, vector j of thread t at columns (j TPR + t) VEC, so that every load
// of a warp is contiguous (512 bytes at VEC = 8 in bf16).  VEC is 8 where D is a multiple of
// 8, else 2 or 1: rows then start on the vector's alignment.  Blocks walk the rows: the
// weight stays in registers (read again for every row it is as much L2 traffic as half
// the row), and the next row is loaded, as it is stored, before the sums of this one are
// waited for.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdio.h>

#include "norm.h"
#include "ssd_internal.cuh"

namespace ssd {
namespace {

constexpr float kE4m3Max = 448.f;

// ---- VEC consecutive elements of a row, in 32-bit words as they are stored (VEC sizeof(T) bytes, at most 16 a load)
template <typename T, int VEC>
struct Vec {
    static constexpr int BYTES = VEC * (int)sizeof(T), WORDS = (BYTES + 3) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (BYTES == 32) {
            const uint4 a = __ldg((const uint4 *)p), b = __ldg((const uint4 *)p + 1);
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        } else if constexpr (BYTES == 16) {
            const uint4 a = __ldg((const uint4 *)p);
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        } else if constexpr (BYTES == 8) {
            const uint2 a = __ldg((const uint2 *)p);
            w[0] = a.x, w[1] = a.y;
        } else if constexpr (BYTES == 4) {
            w[0] = __ldg((const uint32_t *)p);
        } else {
            w[0] = __ldg((const unsigned short *)p);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        else
            return __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ void set(const float *f) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], VEC > 1 ? f[2 * i + 1] : 0.f);
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
// Reduction of K values over the TPR threads of a row; every thread gets the results.  `buf` holds K floats
// per warp, twice: `turn` alternates between reductions, so that one barrier each is enough.
template <typename Op, int TPR, int K>
__device__ __forceinline__ void row_reduce(float (&x)[K], float (*buf)[32][K], int &turn) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
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
    __shared__ float buf[2][32][1];
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
    const int t = threadIdx.x % TPR;
    int turn = 0;
    Vec<float, VEC> w[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + t) * VEC;
        w[j].zero();
        if (c < a.D) w[j].load(a.weight + c);
    }
    Vec<T, VEC> x[NV], r[NV];
    const long long first = blockIdx.x * (long long)RPB, step = gridDim.x * (long long)RPB;
    auto load = [&](long long row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            x[j].zero();
            r[j].zero();
            if (row < a.rows && c < a.D) {
                x[j].load((const T *)a.x + row * a.D + c);
                if (a.residual) r[j].load((const T *)a.residual + row * a.D + c);
            }
        }
    };
    load(first + threadIdx.x / TPR);
    for (long long base = first; base < a.rows; base += step) {
        const long long row = base + threadIdx.x / TPR, at = row * a.D;
        const bool live = row < a.rows;
        float f[NV][VEC], ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[j][i] = a.residual ? x[j].get(i) + r[j].get(i) : x[j].get(i);
            x[j].set(f[j]);  // the stream as it is stored is what is normalised
            if (a.stream && live && c < a.D) x[j].store((T *)a.stream + at + c);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                f[j][i] = x[j].get(i);
                ss[0] += f[j][i] * f[j][i];
            }
        }
        load(row + step);
        row_reduce<Sum, TPR, 1>(ss, buf, turn);
        const float rstd = rsqrtf(ss[0] / (float)a.D + a.eps);
        float amax[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                f[j][i] = f[j][i] * rstd * w[j].get(i);
                if (FP8 && c < a.D) amax[0] = max_nan(amax[0], fabsf(f[j][i]));
            }
            if (!FP8 && live && c < a.D) {
                Vec<T, VEC> y;
                y.set(f[j]);
                y.store((T *)a.y + at + c);
            }
            if constexpr (FP8 && VEC == 8) {
                if (a.group) {  // group / 8 neighbouring lanes hold a group's columns of vector j
                    float m = amax[0];
                    for (int o = a.group / 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                    amax[0] = 0.f;
                    const float inv = m == 0.f ? 0.f : kE4m3Max / m;
                    if (live && c < a.D) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) f[j][i] *= inv;
                        st_e4m3<VEC>((uint8_t *)a.y + at + c, f[j]);
                        if (c % a.group == 0) a.scales[row * (a.D / a.group) + c / a.group] = m / kE4m3Max;
                    }
                }
            }
        }
        if constexpr (FP8) {
            if (!a.group) {
                row_reduce<Max, TPR, 1>(amax, buf, turn);
                const float m = amax[0], inv = m == 0.f ? 0.f : kE4m3Max / m;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = (j * TPR + t) * VEC;
                    if (live && c < a.D) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) f[j][i] *= inv;
                        st_e4m3<VEC>((uint8_t *)a.y + at + c, f[j]);
                    }
                }
                if (live && t == 0) a.scales[row] = m / kE4m3Max;
            }
        }
    }
}

// ------------------------------------------------------------------ backward
// A thread's columns are the same in every row, so its share of dweight stays in
// registers and leaves as one partial row per block, which a second kernel adds in
// the blocks' order.
template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(TPR) rms_bwd_kernel(const T *dy, const T *h, const float *weight, float eps,
                                                      const T *d_stream, T *dx, float *part, long long rows, int D) {
    __shared__ float buf[2][32][2];
    const int t = threadIdx.x;
    int turn = 0;
    Vec<float, VEC> w[NV];
    float dw[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + t) * VEC;
        w[j].zero();
        if (c < D) w[j].load(weight + c);
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[j][i] = 0.f;
    }
    Vec<T, VEC> hv[NV], dv[NV], sv[NV], hn[NV], dn[NV], sn[NV];
    auto load = [&](long long row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            hn[j].zero();
            dn[j].zero();
            sn[j].zero();
            if (row < rows && c < D) {
                hn[j].load(h + row * D + c);
                dn[j].load(dy + row * D + c);
                if (d_stream) sn[j].load(d_stream + row * D + c);
            }
        }
    };
    load(blockIdx.x);
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        float sum[2] = {0.f, 0.f};  // h^2 and dy w h
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            hv[j] = hn[j];
            dv[j] = dn[j];
            sv[j] = sn[j];
        }
        load(row + gridDim.x);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                sum[0] += hv[j].get(i) * hv[j].get(i);
                sum[1] += dv[j].get(i) * w[j].get(i) * hv[j].get(i);
            }
        row_reduce<Sum, TPR, 2>(sum, buf, turn);
        const float rstd = rsqrtf(sum[0] / (float)D + eps);
        const float coef = rstd * rstd * (sum[1] / (float)D);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            if (c < D) {
                float out[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float d = dv[j].get(i), x = hv[j].get(i);
                    out[i] = sv[j].get(i) + rstd * (d * w[j].get(i) - x * coef);
                    dw[j][i] += d * x * rstd;
                }
                Vec<T, VEC> o;
                o.set(out);
                o.store(dx + row * D + c);
            }
        }
    }
    if (part) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            Vec<float, VEC> o;
            o.set(dw[j]);
            if (c < D) o.store(part + (long long)blockIdx.x * D + c);
        }
    }
}

// dweight[c] = the sum over the blocks' partial rows: 32 columns a block, 32 rows of threads, fixed order.
__global__ void __launch_bounds__(1024) rms_dweight_reduce(const float *part, float *dweight, int blocks, int D) {
    __shared__ float red[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
    float a = 0.f;
    if (c < D) {
#pragma unroll 4
        for (int i = r; i < blocks; i += 32) a += part[(long long)i * D + c];
    }
    red[r][threadIdx.x & 31] = a;
    __syncthreads();
    if (r == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 32; ++i) a += red[i][threadIdx.x];
        dweight[c] = a;
    }
}

// ------------------------------------------------------------------ host side
constexpr long long kMaxD = 16384;
constexpr int kBwdBlocks = 608;  // four per SM
constexpr int kFwdThreads = 152 * 1280;  // threads that walk the rows

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

unsigned fwd_blocks(long long rows, int rows_per_block, int threads) {
    const long long all = (rows + rows_per_block - 1) / rows_per_block, most = kFwdThreads / threads;
    return (unsigned)(all < most ? all : most);
}
template <typename T, bool FP8>
cudaError_t forward(const NormArgs &a, cudaStream_t s) {
    const int64_t D = a.D;
#define F(V, TPR, NV)                                                                       \
    do {                                                                                    \
        constexpr int rpb = TPR < 128 ? 128 / TPR : 1;                                      \
        add_rms_kernel<T, V, TPR, NV, FP8>                                                  \
            <<<fwd_blocks(a.rows, rpb, TPR * rpb), TPR * rpb, 0, s>>>(a);                   \
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
    rms_dweight_reduce<<<(unsigned)((D + 31) / 32), 1024, 0, s>>>(part, dw, blocks, (int)D);
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
