// window_simt.cu -- window attention on CUDA cores with fp32 operands: the fp32
// path and WINDOW_FLAG_SIMT.
//
// With x = scale q.k, p = exp(x - lse), D = do.o and dx = p (do.v - D):
//     o = sum_s p v,   dq = scale sum_s dx k,   dk = scale sum_t dx q,   dv = sum_t p do.
// A block holds 16 rows, 4 a warp, and streams tiles of 32 rows of the other side through shared
// memory; in a warp's scores a lane is one row of the tile, in its sums a lane is 4 columns, so both
// read shared memory without conflicts and neither needs a transposed copy.  Rows: queries
// (forward, dq) or keys (dk and dv, over all heads of the group and every query that sees them).
// Every sum has one order.  What bounds them at the sizes that fp32 is for (gradient checks) is
// the chain of a tile's scores, shuffles and sums.
#include "window_internal.cuh"

namespace ssd {
namespace window {
namespace {

constexpr int kRows = 16, kTile = 32, kWarpRows = 4, kThreads = kRows / kWarpRows * 32;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float4 fma4(float a, float4 x, float4 y) {
    return make_float4(fmaf(a, x.x, y.x), fmaf(a, x.y, y.y), fmaf(a, x.z, y.z), fmaf(a, x.w, y.w));
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}
// Rows [first, first + n) of head `head` of a [b, L, heads, P] tensor; rows at or past `end` become zeros.
template <typename T>
__device__ __forceinline__ void load_rows(float *dst, int pitch, const void *src, int bi, int L, int heads, int head, int P,
                                          int first, int n, int end) {
    const int nq = P / 4;
    for (int i = threadIdx.x; i < n * nq; i += kThreads) {
        const int r = i / nq, c = 4 * (i % nq);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (first + r < end) x = load4((const T *)src + (((long long)bi * L + first + r) * heads + head) * P + c);
        *(float4 *)(dst + r * pitch + c) = x;
    }
}
__device__ __forceinline__ bool sees(const WindowParams &p, int t, int s) { return s <= t && (t - s < p.W || s < p.sinks); }
// x[i] = row i of `rows` . row `lane` of `tile`
__device__ __forceinline__ void scores(const float *rows, const float *tile, int pitch, int P, float (&x)[kWarpRows]) {
    const float *mine = tile + (threadIdx.x & 31) * pitch;
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i) x[i] = 0.f;
    for (int c = 0; c < P; c += 4) {
        const float4 k = *(const float4 *)(mine + c);
#pragma unroll
        for (int i = 0; i < kWarpRows; ++i) x[i] = dot4(*(const float4 *)(rows + i * pitch + c), k, x[i]);
    }
}
// acc[i] += sum over the tile's rows of w[i] (lane = row) times 4 columns (lane = columns)
__device__ __forceinline__ void sums(const float (&w)[kWarpRows], const float *tile, int pitch, int P, float4 (&acc)[kWarpRows]) {
    const int c = 4 * (threadIdx.x & 31);
    const float *col = tile + (c < P ? c : 0);
#pragma unroll 8
    for (int j = 0; j < kTile; ++j) {
        const float4 x = *(const float4 *)(col + j * pitch);
#pragma unroll
        for (int i = 0; i < kWarpRows; ++i) acc[i] = fma4(__shfl_sync(0xffffffffu, w[i], j), x, acc[i]);
    }
}
__device__ __forceinline__ void clear(float4 (&acc)[kWarpRows]) {
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// Calls each(first, end) for the key tiles that queries [t0, t1) see: the sinks in front of the
// window of t0, then from there on.
template <class F>
__device__ __forceinline__ void key_tiles(const WindowParams &p, int t0, int t1, F each) {
    const int lo = max(0, t0 - p.W + 1), head = min(p.sinks, lo);
    for (int s = 0; s < head; s += kTile) each(s, head);
    for (int s = lo; s < t1; s += kTile) each(s, t1);
}

// ------------------------------------------------------------------ forward
// Grid: one block per (b, h, 16 queries).
template <typename T>
__global__ void __launch_bounds__(kThreads) window_rows_fwd(WindowParams p) {
    extern __shared__ float4 smem4[];
    const int pitch = p.P + 4, warp = threadIdx.x / 32, lane = threadIdx.x & 31, c = 4 * lane;
    float *Q = (float *)smem4, *K = Q + kRows * pitch, *Vs = K + kTile * pitch;
    const int nblk = (p.L + kRows - 1) / kRows, bh = blockIdx.x / nblk, bi = bh / p.H, h = bh % p.H, g = h / p.hpg;
    const int t0 = (blockIdx.x % nblk) * kRows, V = valid_tokens(p, bi), t1 = min(t0 + kRows, V);
    if (blockIdx.x == 0) write_status(p);
    float4 o[kWarpRows];
    float m[kWarpRows], l[kWarpRows];
    clear(o);
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i) m[i] = -INFINITY, l[i] = 0.f;
    if (t0 < t1) {
        load_rows<T>(Q, pitch, p.q, bi, p.L, p.H, h, p.P, t0, kRows, t1);
        key_tiles(p, t0, t1, [&](int s0, int end) {
            __syncthreads();
            load_rows<T>(K, pitch, p.k, bi, p.L, p.G, g, p.P, s0, kTile, end);
            load_rows<T>(Vs, pitch, p.v, bi, p.L, p.G, g, p.P, s0, kTile, end);
            __syncthreads();
            float x[kWarpRows];
            scores(Q + warp * kWarpRows * pitch, K, pitch, p.P, x);
#pragma unroll
            for (int i = 0; i < kWarpRows; ++i) {
                const int t = t0 + warp * kWarpRows + i, s = s0 + lane;
                x[i] = s < end && sees(p, t, s) ? p.scale * x[i] : -INFINITY;
                const float mn = fmaxf(m[i], warp_max(x[i])), base = mn == -INFINITY ? 0.f : mn;
                const float f = expf(m[i] - base);
                x[i] = expf(x[i] - base);
                l[i] = fmaf(l[i], f, x[i]);
                m[i] = mn;
                o[i] = make_float4(o[i].x * f, o[i].y * f, o[i].z * f, o[i].w * f);
            }
            sums(x, Vs, pitch, p.P, o);
        });
    }
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i) {
        const int t = t0 + warp * kWarpRows + i;
        if (t >= p.L) break;
        const float total = warp_sum(l[i]), inv = t < V ? 1.f / total : 0.f;
        if (c < p.P)
            store4((T *)p.o + (((long long)bi * p.L + t) * p.H + h) * p.P + c,
                   make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv));
        if (p.lse && lane == 0) p.lse[((long long)bi * p.H + h) * p.L + t] = t < V ? m[i] + logf(total) : 0.f;
    }
}

// ------------------------------------------------------------------ backward, dq (and D = do . o)
// Grid: one block per (b, h, 16 queries).
template <typename T>
__global__ void __launch_bounds__(kThreads) window_rows_dq(WindowParams p) {
    extern __shared__ float4 smem4[];
    const int pitch = p.P + 4, warp = threadIdx.x / 32, lane = threadIdx.x & 31, c = 4 * lane;
    float *Q = (float *)smem4, *dO = Q + kRows * pitch, *K = dO + kRows * pitch, *Vs = K + kTile * pitch;
    const int nblk = (p.L + kRows - 1) / kRows, bh = blockIdx.x / nblk, bi = bh / p.H, h = bh % p.H, g = h / p.hpg;
    const int t0 = (blockIdx.x % nblk) * kRows, V = valid_tokens(p, bi), t1 = min(t0 + kRows, V);
    if (blockIdx.x == 0) write_status(p);
    float4 dq[kWarpRows];
    float D[kWarpRows], lse[kWarpRows];
    clear(dq);
    if (t0 < t1) {
        load_rows<T>(Q, pitch, p.q, bi, p.L, p.H, h, p.P, t0, kRows, t1);
        load_rows<T>(dO, pitch, p.d_o, bi, p.L, p.H, h, p.P, t0, kRows, t1);
#pragma unroll
        for (int i = 0; i < kWarpRows; ++i) {
            const int t = t0 + warp * kWarpRows + i;
            const long long at = (((long long)bi * p.L + t) * p.H + h) * p.P + c;
            float d = 0.f;
            if (t < t1 && c < p.P) d = dot4(load4((const T *)p.o + at), load4((const T *)p.d_o + at), 0.f);
            D[i] = warp_sum(d);
            const long long gate = ((long long)bi * p.H + h) * p.L + t;
            lse[i] = t < t1 ? p.lse[gate] : 0.f;
            if (t < t1 && lane == 0) p.delta[gate] = D[i];
        }
        key_tiles(p, t0, t1, [&](int s0, int end) {
            __syncthreads();
            load_rows<T>(K, pitch, p.k, bi, p.L, p.G, g, p.P, s0, kTile, end);
            load_rows<T>(Vs, pitch, p.v, bi, p.L, p.G, g, p.P, s0, kTile, end);
            __syncthreads();
            float x[kWarpRows], dp[kWarpRows];
            scores(Q + warp * kWarpRows * pitch, K, pitch, p.P, x);
            scores(dO + warp * kWarpRows * pitch, Vs, pitch, p.P, dp);
#pragma unroll
            for (int i = 0; i < kWarpRows; ++i) {
                const int t = t0 + warp * kWarpRows + i, s = s0 + lane;
                x[i] = t < t1 && s < end && sees(p, t, s) ? p.scale * expf(p.scale * x[i] - lse[i]) * (dp[i] - D[i]) : 0.f;
            }
            sums(x, K, pitch, p.P, dq);
        });
    }
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i) {
        const int t = t0 + warp * kWarpRows + i;
        if (t < p.L && c < p.P) store4((T *)p.dq + (((long long)bi * p.L + t) * p.H + h) * p.P + c, dq[i]);
    }
}

// ------------------------------------------------------------------ backward, dk and dv
// Grid: one block per (b, g, 16 keys); after window_rows_dq, which leaves D.
template <typename T>
__global__ void __launch_bounds__(kThreads) window_rows_dkv(WindowParams p) {
    extern __shared__ float4 smem4[];
    const int pitch = p.P + 4, warp = threadIdx.x / 32, lane = threadIdx.x & 31, c = 4 * lane;
    float *K = (float *)smem4, *Vs = K + kRows * pitch, *Q = Vs + kRows * pitch, *dO = Q + kTile * pitch;
    const int nblk = (p.L + kRows - 1) / kRows, bg = blockIdx.x / nblk, bi = bg / p.G, g = bg % p.G;
    const int s0 = (blockIdx.x % nblk) * kRows, V = valid_tokens(p, bi), s1 = min(s0 + kRows, V);
    float4 dk[kWarpRows], dv[kWarpRows];
    clear(dk), clear(dv);
    if (s0 < s1) {
        load_rows<T>(K, pitch, p.k, bi, p.L, p.G, g, p.P, s0, kRows, s1);
        load_rows<T>(Vs, pitch, p.v, bi, p.L, p.G, g, p.P, s0, kRows, s1);
        const int last = s0 < p.sinks ? V : (int)min((long long)V, (long long)s1 - 1 + p.W);
        for (int h = g * p.hpg; h < (g + 1) * p.hpg; ++h) {
            const long long gate = ((long long)bi * p.H + h) * p.L;
            for (int t0 = s0; t0 < last; t0 += kTile) {
                __syncthreads();
                load_rows<T>(Q, pitch, p.q, bi, p.L, p.H, h, p.P, t0, kTile, last);
                load_rows<T>(dO, pitch, p.d_o, bi, p.L, p.H, h, p.P, t0, kTile, last);
                __syncthreads();
                const int t = t0 + lane;
                const float lse = t < last ? p.lse[gate + t] : 0.f, D = t < last ? p.delta[gate + t] : 0.f;
                float x[kWarpRows], dp[kWarpRows];
                scores(K + warp * kWarpRows * pitch, Q, pitch, p.P, x);
                scores(Vs + warp * kWarpRows * pitch, dO, pitch, p.P, dp);
#pragma unroll
                for (int i = 0; i < kWarpRows; ++i) {
                    const int s = s0 + warp * kWarpRows + i;
                    x[i] = t < last && s < s1 && sees(p, t, s) ? expf(p.scale * x[i] - lse) : 0.f;
                    dp[i] = x[i] != 0.f ? p.scale * x[i] * (dp[i] - D) : 0.f;
                }
                sums(x, dO, pitch, p.P, dv);
                sums(dp, Q, pitch, p.P, dk);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i) {
        const int s = s0 + warp * kWarpRows + i;
        if (s < p.L && c < p.P) {
            const long long at = (((long long)bi * p.L + s) * p.G + g) * p.P + c;
            store4((T *)p.dk + at, dk[i]);
            store4((T *)p.dv + at, dv[i]);
        }
    }
}

unsigned blocks(const WindowParams &p, int heads) { return (unsigned)((long long)p.b * heads * ((p.L + kRows - 1) / kRows)); }

template <typename T>
cudaError_t forward(const WindowParams &p, cudaStream_t s) {
    const int bytes = (kRows + 2 * kTile) * (p.P + 4) * 4;
    window_rows_fwd<T><<<blocks(p, p.H), kThreads, bytes, s>>>(p);
    return cudaGetLastError();
}
template <typename T>
cudaError_t backward(const WindowParams &p, cudaStream_t s) {
    const int bytes = (2 * kRows + 2 * kTile) * (p.P + 4) * 4;
    constexpr int most = (2 * kRows + 2 * kTile) * 132 * 4;  // asked for once, for every width
    cudaError_t e;
    if ((e = delta::allow_shared((const void *)window_rows_dq<T>, most)) != cudaSuccess) return e;
    if ((e = delta::allow_shared((const void *)window_rows_dkv<T>, most)) != cudaSuccess) return e;
    window_rows_dq<T><<<blocks(p, p.H), kThreads, bytes, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    window_rows_dkv<T><<<blocks(p, p.G), kThreads, bytes, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_simt_forward(const WindowParams &p, bool is_bf16, cudaStream_t s) {
    return is_bf16 ? forward<bf16>(p, s) : forward<float>(p, s);
}
cudaError_t launch_simt_backward(const WindowParams &p, bool is_bf16, cudaStream_t s) {
    return is_bf16 ? backward<bf16>(p, s) : backward<float>(p, s);
}

}  // namespace window
}  // namespace ssd
