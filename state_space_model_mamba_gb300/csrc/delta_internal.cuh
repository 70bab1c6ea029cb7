// delta_internal.cuh -- shared definitions of the gated delta rule's kernels
// (include/delta.h; not part of the ABI).
//
// Index conventions: q/k [b, L, G, N], v/o [b, L, H, P], g/beta [b, H, L],
// states [b, H, P, N]; bh = b * H + h.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "delta.h"
#include "ssd_internal.cuh"

namespace ssd {
namespace delta {

constexpr float kMinLogDecay = -1000.f;  // exp of it is 0; keeps differences of sums finite for g = -inf

struct DeltaParams {
    int b, L, H, P, N, G, hpg;
    float scale;
    const void *q, *k, *v;
    const float *g, *beta, *init;
    const int32_t *valid_len;
    void *o;
    float *final_state;
    // backward
    const void *d_o;
    const float *d_final;
    void *dq, *dk, *dv;
    float *dg, *dbeta, *d_init;
    int *status;  // kStatusWords ints at the workspace's start
};

__device__ __forceinline__ int valid_tokens(const DeltaParams &p, int bi) {
    if (!p.valid_len) return p.L;
    const int v = p.valid_len[bi];
    return v < 0 ? 0 : (v > p.L ? p.L : v);
}
// One block writes the call's status words: nothing timed out, how many valid_len entries were clamped.
__device__ __forceinline__ void write_status(const DeltaParams &p, int rows) {
    if (threadIdx.x == 0) {
        int bad = 0;
        if (p.valid_len)
            for (int i = 0; i < rows; ++i) bad += p.valid_len[i] < 0 || p.valid_len[i] > p.L;
        for (int i = 0; i < kStatusWords; ++i) p.status[i] = i == kStatusValidLen ? bad : 0;
    }
}
__device__ __forceinline__ float clamp_log_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }

// Dynamic shared memory of a kernel, asked for once per thread, device and size: a short call is mostly its launches
// (delta_maps.cu).
cudaError_t allow_shared(const void *kernel, int bytes);

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) {
    return __ldg((const float4 *)p);
}
template <>
__device__ __forceinline__ float4 load4<bf16>(const bf16 *p) {
    const uint2 u = __ldg((const uint2 *)p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ float load1(const T *p) {
    return (float)*p;
}
template <typename T>
__device__ __forceinline__ void store1(T *p, float v) {
    *p = (T)v;
}

// ---- token-by-token kernels (delta_simt.cu)
size_t simt_backward_bytes(const delta_dims &d);
cudaError_t launch_simt_forward(const DeltaParams &p, bool is_bf16, cudaStream_t s);
cudaError_t launch_simt_backward(const DeltaParams &p, bool is_bf16, char *ws, cudaStream_t s);
cudaError_t launch_step(const DeltaParams &p, bool is_bf16, float *state, long long slots, const int32_t *index,
                        cudaStream_t s);

}  // namespace delta
}  // namespace ssd
