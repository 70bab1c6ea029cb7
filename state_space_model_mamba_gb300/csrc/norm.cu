// norm.cu -- the block's entry norm (include/norm.h): residual addition and
// root-mean-square norm in one pass over the row, the output in the stream's
// type or in e4m3 with scales, and the backward.
//
// All three are streams bound by HBM.  A row is held by TPR threads with NV vectors of
// VEC columns each, vector j of thread t at columns (j TPR + t) VEC, so that every load
// of a warp is contiguous.  A vector has 16 bytes where D allows (8 columns in bf16, 4 in
// fp32), else VEC is 2 or 1: rows then start on the vector's alignment.  The blocks that the SMs hold at
// once walk the rows: the weight stays in registers (read again for every row it is as much L2
// traffic as half the row), and the next row is loaded, as it is stored, before the sums of this
// one are waited for.  The arithmetic is in pairs, and the residual is added in bf16 itself: at
// 36 instructions a column (scalar, IEEE divisions) the e4m3 form took 63 us where the
// bf16 one, which writes more, took 57.
//
// Measured at 16384 x 2560 in bf16, of a measured copy's 6.69 TB/s:
//   bf16 output 51.9 us (6.5 TB/s), e4m3 with a scale per 128 columns 47.3 us (6.2 TB/s),
//   backward 54.5 us, and 3.9 for dweight's second kernel (5.7 TB/s over both, 0.86 of the copy);
// 24 x 2560: 1.9 us, below a launch.  At 16384 columns, where a row's registers leave no room for the next one, and at
// widths that are no multiple of 16 bytes the rates are lower (backward 3.5 TB/s in bf16, odd widths 1.5 to 5).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdio.h>

#include "norm.h"
#include "ssd_internal.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

using tc::ffma2;
using tc::fmul2;

constexpr float kE4m3Max = 448.f;

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

// e4m3 bytes of VEC floats times `inv`
template <int VEC>
__device__ __forceinline__ void st_e4m3(uint8_t *p, const float2 *f, float inv) {
    if constexpr (VEC == 1) {
        *p = __nv_cvt_float_to_fp8(f[0].x * inv, __NV_SATFINITE, __NV_E4M3);
    } else {
        uint16_t h[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            h[i] = __nv_cvt_float2_to_fp8x2(fmul2(f[i], make_float2(inv, inv)), __NV_SATFINITE, __NV_E4M3);
        if constexpr (VEC == 2)
            *(uint16_t *)p = h[0];
        else if constexpr (VEC == 4)
            *(uint32_t *)p = h[0] | (uint32_t)h[1] << 16;
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
// A group's scale, and what its values are multiplied with to come out as y / scale: the reciprocal, off by one unit
// in the last place at most.  Where that would leave fp32, or the scale is no normal number and so is rounded, values
// and scale go up by 2^64 first, and the reciprocal is that of the scale as it is stored.  Scales that round to 0
// (maxima below 448 halves of the smallest float) come with zeros.
constexpr float kTinyMax = 1e-30f, kUp = 18446744073709551616.f;
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <int N>
__device__ __forceinline__ float e4m3_gain(float m, float &scale, float2 (&f)[N]) {
    scale = m * (1.f / kE4m3Max);
    if (!(m < kTinyMax)) return reciprocal(m) * kE4m3Max;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = fmul2(f[i], make_float2(kUp, kUp));
    return scale == 0.f ? 0.f : reciprocal(scale * kUp);
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
    constexpr int PAIRS = Vec<T, VEC>::PAIRS;
    const long long first = blockIdx.x * (long long)RPB, step = gridDim.x * (long long)RPB;
    auto load = [&](long long row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            x[j].zero();
            r[j].minus_zero();
            if (row < a.rows && c < a.D) {
                x[j].template load<true>((const T *)a.x + row * a.D + c);
                if (a.residual) r[j].template load<true>((const T *)a.residual + row * a.D + c);
            }
        }
    };
    load(first + threadIdx.x / TPR);
    for (long long base = first; base < a.rows; base += step) {
        const long long row = base + threadIdx.x / TPR, at = row * a.D;
        const bool live = row < a.rows;
        float2 f[NV][PAIRS], s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            x[j].add(r[j]);  // the stream as it is stored is what is normalised
            if (a.stream && live && c < a.D) x[j].store((T *)a.stream + at + c);
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                f[j][i] = x[j].get(i);
                s2 = ffma2(f[j][i], f[j][i], s2);
            }
        }
        load(row + step);
        float ss[1] = {s2.x + s2.y};
        row_reduce<Sum, TPR, 1>(ss, buf, turn);
        const float rstd = rsqrtf(ss[0] / (float)a.D + a.eps);
        float amax[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                f[j][i] = fmul2(fmul2(f[j][i], make_float2(rstd, rstd)), w[j].get(i));
                if (FP8 && c < a.D) amax[0] = max_nan(amax[0], max_nan(fabsf(f[j][i].x), fabsf(f[j][i].y)));
            }
            if (!FP8 && live && c < a.D) {
                Vec<T, VEC> y;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) y.set(i, f[j][i]);
                y.store((T *)a.y + at + c);
            }
            if constexpr (FP8 && VEC >= 4) {
                if (a.group) {  // group / VEC neighbouring lanes hold a group's columns of vector j
                    float m = amax[0];
                    for (int o = a.group / (2 * VEC); o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                    amax[0] = 0.f;
                    float scale;
                    const float gain = e4m3_gain(m, scale, f[j]);
                    if (live && c < a.D) {
                        st_e4m3<VEC>((uint8_t *)a.y + at + c, f[j], gain);
                        if (c % a.group == 0) a.scales[row * (a.D / a.group) + c / a.group] = scale;
                    }
                }
            }
        }
        if constexpr (FP8) {
            if (!a.group) {
                row_reduce<Max, TPR, 1>(amax, buf, turn);
                float scale;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = (j * TPR + t) * VEC;
                    const float gain = e4m3_gain(amax[0], scale, f[j]);
                    if (live && c < a.D) st_e4m3<VEC>((uint8_t *)a.y + at + c, f[j], gain);
                }
                if (live && t == 0) a.scales[row] = scale;
            }
        }
    }
}

// ------------------------------------------------------------------ backward
// A thread's columns are the same in every row, so its share of dweight stays in
// registers; the rows of threads of a block add theirs up in order, and one partial row per block
// leaves, which a second kernel adds in the blocks' order.
constexpr int kBwdThreads = 512;  // on an SM at least: 128 registers a thread (at 96 they spill: 78 us for 59; at 140 two blocks of 160: 67)
template <int TPR>
constexpr int kBlock = TPR < 128 ? 128 : TPR;
template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kBlock<TPR>, kBwdThreads / kBlock<TPR> > 1 ? kBwdThreads / kBlock<TPR> : 1)
    rms_bwd_kernel(const T *dy, const T *h, const float *weight, float eps, const T *d_stream, T *dx, float *part,
                   long long rows, int D) {
    constexpr int RPB = kBlock<TPR> / TPR, PAIRS = Vec<T, VEC>::PAIRS;
    constexpr bool kAhead = TPR < 1024;  // registers for the weight and for the next row
    __shared__ float buf[2][32][2];
    __shared__ float2 shares[RPB > 1 ? RPB : 1][RPB > 1 ? TPR * NV * PAIRS : 1];
    const int t = threadIdx.x % TPR;
    int turn = 0;
    Vec<float, VEC> w[NV];
    float2 dw[NV][PAIRS];
    auto load_weight = [&]() {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            w[j].zero();
            if (c < D) w[j].load(weight + c);
        }
    };
    load_weight();
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) dw[j][i] = make_float2(0.f, 0.f);
    Vec<T, VEC> hv[NV], dv[NV], sv[NV], hn[NV], dn[NV], sn[NV];
    auto load = [&](long long row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            hn[j].zero();
            dn[j].zero();
            sn[j].zero();
            if (row < rows && c < D) {
                hn[j].template load<true>(h + row * D + c);
                dn[j].template load<true>(dy + row * D + c);
                if (d_stream) sn[j].template load<true>(d_stream + row * D + c);
            }
        }
    };
    const long long first = blockIdx.x * (long long)RPB, step = gridDim.x * (long long)RPB;
    if (kAhead) load(first + threadIdx.x / TPR);
    for (long long base = first; base < rows; base += step) {
        const long long row = base + threadIdx.x / TPR;
        if (!kAhead) load(row);
        float2 s0 = make_float2(0.f, 0.f), s1 = s0;  // h^2 and dy w h
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            hv[j] = hn[j];
            dv[j] = dn[j];
            sv[j] = sn[j];
        }
        if (kAhead)
            load(row + step);
        else
            load_weight();
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                s0 = ffma2(hv[j].get(i), hv[j].get(i), s0);
                s1 = ffma2(fmul2(dv[j].get(i), w[j].get(i)), hv[j].get(i), s1);
            }
        float sum[2] = {s0.x + s0.y, s1.x + s1.y};
        row_reduce<Sum, TPR, 2>(sum, buf, turn);
        const float rstd = rsqrtf(sum[0] / (float)D + eps);
        const float coef = -rstd * rstd * (sum[1] / (float)D);
        const float2 r2 = make_float2(rstd, rstd), c2 = make_float2(coef, coef);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            if (row < rows && c < D) {
                Vec<T, VEC> o;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    const float2 d = dv[j].get(i), x = hv[j].get(i);
                    o.set(i, ffma2(ffma2(x, c2, fmul2(d, w[j].get(i))), r2, sv[j].get(i)));
                    dw[j][i] = ffma2(fmul2(d, x), r2, dw[j][i]);
                }
                o.store(dx + row * D + c);
            }
        }
    }
    if (part) {
        if constexpr (RPB > 1) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) shares[threadIdx.x / TPR][(j * PAIRS + i) * TPR + t] = dw[j][i];
            __syncthreads();
            if (threadIdx.x >= TPR) return;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < PAIRS; ++i)
                    for (int y = 1; y < RPB; ++y) {
                        const float2 o = shares[y][(j * PAIRS + i) * TPR + t];
                        dw[j][i] = make_float2(dw[j][i].x + o.x, dw[j][i].y + o.y);
                    }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + t) * VEC;
            Vec<float, VEC> o;
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) o.set(i, dw[j][i]);
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
constexpr int kSMs = 152;
constexpr int kBwdBlocks = 4 * kSMs;  // the most whose partial rows the workspace holds

// Blocks of a kernel that the SMs hold at once.  A grid of just these walks the rows: one of 8 blocks per SM where
// 5 fit leaves the last 3 to run by themselves (56 us for 48 at 16384 x 2560 in e4m3).
template <auto Kernel, int THREADS>
int resident_blocks() {
    static const int n = [] {
        int per_sm = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, Kernel, THREADS, 0) != cudaSuccess || per_sm < 1) per_sm = 1;
        return per_sm * kSMs;
    }();
    return n;
}

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

// Calls F(VEC, TPR, NV) with a row's threads: of the counts below the fewest that hold D columns in two vectors of 16 bytes, or
// in four narrow ones; rows too long for 1024 threads of that take more vectors a thread.  The counts are powers of two, and 160
// and 320 for 2560 and 5120 columns in bf16 (1280 and 2560 in fp32): widths between two of them leave threads without a
// column (a quarter of 256 at 1536 columns of fp32, say).
#define NORM_BY_D(F)                                                         \
    do {                                                                     \
        constexpr int kWide = 16 / (int)sizeof(T);                           \
        const int64_t n_ = D % kWide == 0 ? D / kWide : (D % 2 == 0 ? D / 2 : D); \
        if (D % kWide == 0) {                                                \
            if (n_ <= 32) F(kWide, 32, 1);                                   \
            else if (n_ <= 64) F(kWide, 32, 2);                              \
            else if (n_ <= 128) F(kWide, 64, 2);                             \
            else if (n_ <= 256) F(kWide, 128, 2);                            \
            else if (n_ <= 320) F(kWide, 160, 2);                            \
            else if (n_ <= 512) F(kWide, 256, 2);                            \
            else if (n_ <= 640) F(kWide, 320, 2);                            \
            else if (n_ <= 1024) F(kWide, 512, 2);                           \
            else if (n_ <= 2048) F(kWide, 1024, 2);                          \
            else if constexpr (kMaxD > 2048 * kWide) F(kWide, 1024, 4);      \
        } else if (D % 2 == 0) {                                             \
            NORM_NARROW(F, 2);                                               \
        } else {                                                             \
            NORM_NARROW(F, 1);                                               \
        }                                                                    \
    } while (0)
#define NORM_NARROW(F, VEC)                                                  \
    do {                                                                     \
        if (n_ <= 512) F(VEC, 128, 4);                                       \
        else if (n_ <= 1024) F(VEC, 256, 4);                                 \
        else if (n_ <= 2048) F(VEC, 512, 4);                                 \
        else if (n_ <= 4096) F(VEC, 1024, 4);                                \
        else if (n_ <= 8192) F(VEC, 1024, 8);                                \
        else if constexpr (kMaxD > 8192 * VEC) F(VEC, 1024, 16);             \
    } while (0)

template <typename T, bool FP8>
cudaError_t forward(const NormArgs &a, cudaStream_t s) {
    const int64_t D = a.D;
#define F(V, TPR, NV)                                                                              \
    do {                                                                                           \
        constexpr int rpb = TPR < 128 ? 128 / TPR : 1;                                             \
        const long long all = (a.rows + rpb - 1) / rpb;                                            \
        const int most = resident_blocks<add_rms_kernel<T, V, TPR, NV, FP8>, TPR * rpb>();         \
        add_rms_kernel<T, V, TPR, NV, FP8><<<(unsigned)(all < most ? all : most), TPR * rpb, 0, s>>>(a); \
    } while (0)
    NORM_BY_D(F);
#undef F
    return cudaGetLastError();
}
int bwd_blocks(int64_t rows) { return (int)(rows < kBwdBlocks ? rows : kBwdBlocks); }
template <typename T>
cudaError_t backward(const void *dy, const void *h, const float *weight, float eps, const void *ds, void *dx, float *dw,
                     int64_t rows, int64_t D, float *part, cudaStream_t s) {
    int blocks = bwd_blocks(rows);
#define F(V, TPR, NV)                                                                                     \
    do {                                                                                                  \
        const int most = resident_blocks<rms_bwd_kernel<T, V, TPR, NV>, kBlock<TPR>>();                   \
        if (blocks > most) blocks = most;                                                                 \
        rms_bwd_kernel<T, V, TPR, NV><<<blocks, kBlock<TPR>, 0, s>>>((const T *)dy, (const T *)h, weight, eps,    \
                                                             (const T *)ds, (T *)dx, dw ? part : nullptr, \
                                                             rows, (int)D);                               \
    } while (0)
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
