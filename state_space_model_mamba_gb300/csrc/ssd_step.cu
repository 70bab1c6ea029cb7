// ssd_step.cu -- one decoded token of the selective scan (ssd_step, include/ssd.h).
//
// Row p of a state is a recurrence of its own, s <- exp(dt A) s + dt x_p B, y_p = s.C + D x_p.
// 8 lanes hold a row in 16-byte pieces interleaved over the lanes, 16 rows a block; every state element
// is read and written once, and that is what bounds it: HBM.
#include <stdarg.h>
#include <stdio.h>

#include "delta_internal.cuh"

namespace ssd {
namespace {

using delta::load1;
using delta::load4;
using delta::store1;

constexpr int kLanes = 8, kRows = 16, kThreads = kRows * kLanes;

struct StepParams {
    int b, H, P, N, G, hpg;
    const void *x, *B, *C;
    const float *dt, *A, *D;
    float *state;
    long long slots;
    const int32_t *index;
    void *y;
};

// NC = ceil(N / 32) pieces a lane.  Grid: one block per (b, h, 16 rows).
template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) ssd_step_kernel(StepParams p) {
    const int nblk = (p.P + kRows - 1) / kRows, bh = blockIdx.x / nblk, bi = bh / p.H, h = bh % p.H, g = h / p.hpg;
    const int row = (blockIdx.x % nblk) * kRows + threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const bool in = row < p.P;
    const long long slot = p.index ? (long long)p.index[bi] : (long long)bi;
    const long long at = ((long long)bi * p.H + h) * p.P + row;
    if (slot < 0 || slot >= p.slots) {
        if (in && lane == 0) store1((T *)p.y + at, 0.f);
        return;
    }
    float *srow = p.state + ((slot * p.H + h) * p.P + row) * (long long)p.N;
    const long long key = ((long long)bi * p.G + g) * p.N;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 s[NC], B[NC], C[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = 4 * (i * kLanes + lane);
        s[i] = in && c < p.N ? __ldcs((const float4 *)(srow + c)) : zero;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = 4 * (i * kLanes + lane);
        B[i] = c < p.N ? load4((const T *)p.B + key + c) : zero;
        C[i] = c < p.N ? load4((const T *)p.C + key + c) : zero;
    }
    const float dt = __ldg(p.dt + (long long)bi * p.H + h), a = expf(dt * __ldg(p.A + h)), D = __ldg(p.D + h);
    const float x = in ? load1((const T *)p.x + at) : 0.f, u = dt * x;
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        s[i] = make_float4(fmaf(u, B[i].x, a * s[i].x), fmaf(u, B[i].y, a * s[i].y), fmaf(u, B[i].z, a * s[i].z),
                           fmaf(u, B[i].w, a * s[i].w));
        y = fmaf(s[i].x, C[i].x, fmaf(s[i].y, C[i].y, fmaf(s[i].z, C[i].z, fmaf(s[i].w, C[i].w, y))));
    }
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = 4 * (i * kLanes + lane);
        if (in && c < p.N) __stcs((float4 *)(srow + c), s[i]);
    }
    if (in && lane == 0) store1((T *)p.y + at, fmaf(D, x, y));
}

template <typename T>
cudaError_t step(const StepParams &p, cudaStream_t s) {
    const unsigned grid = (unsigned)((long long)p.b * p.H * ((p.P + kRows - 1) / kRows));
    switch ((p.N + 31) / 32) {
        case 1: ssd_step_kernel<T, 1><<<grid, kThreads, 0, s>>>(p); break;
        case 2: ssd_step_kernel<T, 2><<<grid, kThreads, 0, s>>>(p); break;
        case 3: ssd_step_kernel<T, 3><<<grid, kThreads, 0, s>>>(p); break;
        case 4: ssd_step_kernel<T, 4><<<grid, kThreads, 0, s>>>(p); break;
        case 5: ssd_step_kernel<T, 5><<<grid, kThreads, 0, s>>>(p); break;
        case 6: ssd_step_kernel<T, 6><<<grid, kThreads, 0, s>>>(p); break;
        case 7: ssd_step_kernel<T, 7><<<grid, kThreads, 0, s>>>(p); break;
        default: ssd_step_kernel<T, 8><<<grid, kThreads, 0, s>>>(p); break;
    }
    return cudaGetLastError();
}

ssd_status step_fail(ssd_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
ssd_status step_fail(ssd_status st, const char *fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    record_error(msg);
    return st;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" ssd_status ssd_step(const ssd_dims *dims, ssd_dtype dtype, const void *x, const float *dt, const float *A,
                               const void *B, const void *C, const float *D, float *state, int64_t slots,
                               const int32_t *state_index, void *y, void *stream) {
    ssd_status st = ssd_supported(dims, dtype);  // also clears the last error
    if (st != SSD_OK) return st;
    if (dims->seqlen != 1) return step_fail(SSD_ERR_INVALID_ARG, "ssd_step takes one token: seqlen must be 1");
    const void *req[] = {x, dt, A, B, C, D, state, y};
    static const char *const names[] = {"x", "dt", "A", "B", "C", "D", "state", "y"};
    for (int i = 0; i < 8; ++i) {
        if (!req[i]) return step_fail(SSD_ERR_INVALID_ARG, "%s is NULL", names[i]);
        if ((uintptr_t)req[i] & 15u) return step_fail(SSD_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
    }
    if (slots < 1 || slots > (1LL << 31)) return step_fail(SSD_ERR_INVALID_ARG, "slots %lld out of range", (long long)slots);
    if (!state_index && slots < dims->batch)
        return step_fail(SSD_ERR_INVALID_ARG, "%lld slots for a batch of %lld without state_index", (long long)slots,
                         (long long)dims->batch);
    if ((double)dims->batch * dims->nheads > 5.0e8) return step_fail(SSD_ERR_UNSUPPORTED, "problem too large");
    StepParams p;
    p.b = (int)dims->batch;
    p.H = (int)dims->nheads;
    p.P = (int)dims->headdim;
    p.N = (int)dims->dstate;
    p.G = (int)dims->ngroups;
    p.hpg = p.H / p.G;
    p.x = x;
    p.B = B;
    p.C = C;
    p.dt = dt;
    p.A = A;
    p.D = D;
    p.state = state;
    p.slots = slots;
    p.index = state_index;
    p.y = y;
    const cudaError_t e = dtype == SSD_BF16 ? step<bf16>(p, (cudaStream_t)stream) : step<float>(p, (cudaStream_t)stream);
    return e == cudaSuccess ? SSD_OK : step_fail(SSD_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
}
