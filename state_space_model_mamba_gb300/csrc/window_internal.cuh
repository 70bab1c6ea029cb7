// window_internal.cuh -- shared definitions of the window attention kernels
// (include/window.h; not part of the ABI).
//
// Index conventions: q/o/do/dq [b, L, H, P], k/v/dk/dv [b, L, G, P], lse [b, H, L].
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "delta_internal.cuh"
#include "window.h"

namespace ssd {
namespace window {

using delta::load1;
using delta::load4;
using delta::store1;

struct WindowParams {
    int b, L, H, P, G, hpg;
    int W;      // window, at most L
    int sinks;  // none where W is L
    float scale;
    const void *q, *k, *v;
    const int32_t *valid_len;
    void *o;
    float *lse;
    // backward
    const void *d_o;
    void *dq, *dk, *dv;
    float *delta;  // [b, H, L] do . o
    int *status;   // kStatusWords ints at the workspace's start
};

__device__ __forceinline__ int valid_tokens(const WindowParams &p, int bi) {
    if (!p.valid_len) return p.L;
    const int v = p.valid_len[bi];
    return v < 0 ? 0 : (v > p.L ? p.L : v);
}
// One block clears the call's status words and counts the valid_len entries that are clamped.
__device__ __forceinline__ void write_status(const WindowParams &p) {
    if (threadIdx.x == 0) {
        int bad = 0;
        if (p.valid_len)
            for (int i = 0; i < p.b; ++i) bad += p.valid_len[i] < 0 || p.valid_len[i] > p.L;
        for (int i = 0; i < kStatusWords; ++i) p.status[i] = i == kStatusValidLen ? bad : 0;
    }
}
template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float *p, float4 v) {
    *(float4 *)p = v;
}
template <>
__device__ __forceinline__ void store4<bf16>(bf16 *p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *(uint2 *)p = make_uint2(*(const uint32_t *)&a, *(const uint32_t *)&b);
}

// ---- CUDA-core kernels (window_simt.cu)
cudaError_t launch_simt_forward(const WindowParams &p, bool is_bf16, cudaStream_t s);
cudaError_t launch_simt_backward(const WindowParams &p, bool is_bf16, cudaStream_t s);

// ---- tensor-core kernels (window_fwd.cu, window_bwd.cu); the backward's share of the workspace in floats
cudaError_t launch_tile_forward(const WindowParams &p, cudaStream_t s);
size_t tile_backward_floats(long long batch, long long L, long long G, long long P, long long W, long long sinks);
cudaError_t launch_tile_backward(const WindowParams &p, float *parts, cudaStream_t s);

// ---- the ring (window_step.cu)
struct RingParams {
    int b, L, H, P, G, hpg, W, sinks;
    float scale;
    const void *q, *k, *v;
    const int32_t *valid_len, *position, *index;
    void *k_cache, *v_cache, *o;
    long long slots;
};
cudaError_t launch_fill(const RingParams &p, bool is_bf16, cudaStream_t s);
cudaError_t launch_step(const RingParams &p, bool is_bf16, cudaStream_t s);

}  // namespace window
}  // namespace ssd
