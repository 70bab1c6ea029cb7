// window_simt.cu -- window attention on CUDA cores with fp32 operands: the fp32
// path and WINDOW_FLAG_SIMT.
//
// With x = scale q.k, p = exp(x - lse), D = do.o and dx = p (do.v - D):
//     o = sum_s p v,   dq = scale sum_s dx k,   dk = scale sum_t dx q,   dv = sum_t p do.
// A block's 8 warps hold 2 or 4 rows each (WR: 4 where that leaves every SM a block) and stream tiles of 32 rows of the other
// side through shared
// memory, the next tile on its way in registers.  In a warp's scores a lane is one row of the tile; in its sums a lane is
// 4 columns of every n-th row of the tile, n as many as the head's columns leave lanes for, so both
// read shared memory without conflicts and neither needs a transposed copy.  Rows: queries
// (forward, dq) or keys (dk and dv, over all heads of the group and every query that sees them, shared
// among the blocks of a cluster, whose sums are added in the blocks' order).
// Every sum has one order.  What bounds them at the sizes that fp32 is for (gradient checks) is
// the chain of a tile's scores, shuffles and sums: at 129 tokens of 4 heads of 32, window 48, 8 us forward and 22 backward in two
// kernels; at 2 x 4096 tokens of 8 heads of 64, window 1024, 0.81 ms and 2.6, a quarter of the fp32 rate.
#include <cooperative_groups.h>

#include "window_internal.cuh"

namespace ssd {
namespace window {
namespace {

constexpr int kTile = 32, kWarps = 8, kThreads = kWarps * 32;

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
// The scale enters after the sums of dq and dk: before them it would take the terms of a tiny one below the normal numbers.
__device__ __forceinline__ float4 scaled(float a, float4 x) { return make_float4(a * x.x, a * x.y, a * x.z, a * x.w); }
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
// This thread's part of a tile of 32 rows of such a tensor, on its way through registers.
constexpr int kParts = kTile * 32 / kThreads;  // of 4 columns, at most
struct Parts {
    int row[kParts], col[kParts];
    float4 x[kParts];
    __device__ __forceinline__ explicit Parts(int P) {
        const int nq = P / 4;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            const int i = threadIdx.x + k * kThreads, r = i / nq;
            row[k] = r < kTile ? r : -1;
            col[k] = 4 * (i - r * nq);
        }
    }
    template <typename T>
    __device__ __forceinline__ void fetch(const void *src, int bi, int L, int heads, int head, int P, int first, int end) {
        const T *at = (const T *)src + (((long long)bi * L + first) * heads + head) * P;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row[k] >= 0 && first + row[k] < end) x[k] = load4(at + (long long)row[k] * heads * P + col[k]);
        }
    }
    __device__ __forceinline__ void put(float *dst, int pitch) const {
#pragma unroll
        for (int k = 0; k < kParts; ++k)
            if (row[k] >= 0) *(float4 *)(dst + row[k] * pitch + col[k]) = x[k];
    }
};
__device__ __forceinline__ bool sees(const WindowParams &p, int t, int s) { return s <= t && (t - s < p.W || s < p.sinks); }
// x[i] = row i of `rows` . row `lane` of `tile`
template <int WR>
__device__ __forceinline__ void scores(const float *rows, const float *tile, int pitch, int P, float (&x)[WR]) {
    const float *mine = tile + (threadIdx.x & 31) * pitch;
#pragma unroll
    for (int i = 0; i < WR; ++i) x[i] = 0.f;
    for (int c = 0; c < P; c += 4) {
        const float4 k = *(const float4 *)(mine + c);
#pragma unroll
        for (int i = 0; i < WR; ++i) x[i] = dot4(*(const float4 *)(rows + i * pitch + c), k, x[i]);
    }
}
// The lanes of a warp's sums: 4 columns each, of the rows first, first + n, first + 2 n, ..
struct Lanes {
    int c, first, n, quads;
    __device__ __forceinline__ explicit Lanes(int P) {
        const int lane = threadIdx.x & 31;
        quads = P / 4;
        n = 1;
        while (2 * n * quads <= 32) n *= 2;
        first = lane / quads;
        c = 4 * (lane - first * quads);
        if (first >= n) first = n - 1;  // lanes left over repeat the last ones' work, and nobody reads them
    }
    __device__ __forceinline__ bool leads() const { return (threadIdx.x & 31) < quads; }
    // the sum over the lanes of the same columns, in the first of them
    __device__ __forceinline__ float4 total(float4 x) const {
        float4 t = x;
        for (int k = 1; k < n; ++k) {
            const int from = (threadIdx.x + k * quads) & 31;
            const float4 y = make_float4(__shfl_sync(0xffffffffu, x.x, from), __shfl_sync(0xffffffffu, x.y, from),
                                         __shfl_sync(0xffffffffu, x.z, from), __shfl_sync(0xffffffffu, x.w, from));
            t = make_float4(t.x + y.x, t.y + y.y, t.z + y.z, t.w + y.w);
        }
        return t;
    }
};
// acc[i] += sum over this lane's rows of the tile of w[i] (held by lane = row) times its 4 columns
template <int WR>
__device__ __forceinline__ void sums(const float (&w)[WR], const float *tile, int pitch, const Lanes &at, float4 (&acc)[WR]) {
    const float *col = tile + at.c;
#pragma unroll 4
    for (int j = at.first; j < kTile; j += at.n) {
        const float4 x = *(const float4 *)(col + j * pitch);
#pragma unroll
        for (int i = 0; i < WR; ++i) acc[i] = fma4(__shfl_sync(0xffffffffu, w[i], j), x, acc[i]);
    }
}
template <int WR>
__device__ __forceinline__ void clear(float4 (&acc)[WR]) {
#pragma unroll
    for (int i = 0; i < WR; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// The key tiles that queries [t0, t1) see: the sinks in front of the window of t0, then from there on.
struct KeyTiles {
    int lo, head, t1, sinks, n;
    __device__ __forceinline__ KeyTiles(const WindowParams &p, int t0, int t1_) : t1(t1_) {
        lo = max(0, t0 - p.W + 1), head = min(p.sinks, lo);
        sinks = (head + kTile - 1) / kTile;
        n = t0 < t1 ? sinks + (t1 - lo + kTile - 1) / kTile : 0;
    }
    __device__ __forceinline__ int start(int j) const { return j < sinks ? j * kTile : lo + (j - sinks) * kTile; }
    __device__ __forceinline__ int end(int j) const { return j < sinks ? head : t1; }
};

// ------------------------------------------------------------------ forward
// Grid: one block per (b, h, 8 WR queries).
template <typename T, int WR>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) window_rows_fwd(WindowParams p) {
    constexpr int kRows = kWarps * WR;
    extern __shared__ float4 smem4[];
    const int pitch = p.P + 4, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const Lanes at(p.P);
    float *Q = (float *)smem4, *K = Q + kRows * pitch, *Vs = K + kTile * pitch;
    const int nblk = (p.L + kRows - 1) / kRows, bh = blockIdx.x / nblk, bi = bh / p.H, h = bh % p.H, g = h / p.hpg;
    const int t0 = (blockIdx.x % nblk) * kRows, V = valid_tokens(p, bi), t1 = min(t0 + kRows, V);
    if (blockIdx.x == 0) write_status(p);
    float4 o[WR];
    float m[WR], l[WR];
    clear(o);
#pragma unroll
    for (int i = 0; i < WR; ++i) m[i] = -INFINITY, l[i] = 0.f;
    if (t0 < t1) {
        load_rows<T>(Q, pitch, p.q, bi, p.L, p.H, h, p.P, t0, kRows, t1);
        const KeyTiles tiles(p, t0, t1);
        Parts k(p.P), v = k;
        auto fetch = [&](int j) {
            k.fetch<T>(p.k, bi, p.L, p.G, g, p.P, tiles.start(j), tiles.end(j));
            v.fetch<T>(p.v, bi, p.L, p.G, g, p.P, tiles.start(j), tiles.end(j));
        };
        fetch(0);
        for (int j = 0; j < tiles.n; ++j) {
            const int s0 = tiles.start(j), end = tiles.end(j);
            __syncthreads();
            k.put(K, pitch), v.put(Vs, pitch);
            __syncthreads();
            if (j + 1 < tiles.n) fetch(j + 1);
            float x[WR];
            scores(Q + warp * WR * pitch, K, pitch, p.P, x);
#pragma unroll
            for (int i = 0; i < WR; ++i) {
                const int t = t0 + warp * WR + i, s = s0 + lane;
                x[i] = s < end && sees(p, t, s) ? p.scale * x[i] : -INFINITY;
                const float mn = fmaxf(m[i], warp_max(x[i])), base = mn == -INFINITY ? 0.f : mn;
                const float f = expf(m[i] - base);
                x[i] = expf(x[i] - base);
                l[i] = fmaf(l[i], f, x[i]);
                m[i] = mn;
                o[i] = make_float4(o[i].x * f, o[i].y * f, o[i].z * f, o[i].w * f);
            }
            sums(x, Vs, pitch, at, o);
        }
    }
#pragma unroll
    for (int i = 0; i < WR; ++i) {
        const int t = t0 + warp * WR + i;
        if (t >= p.L) break;
        const float total = warp_sum(l[i]), inv = t < V ? 1.f / total : 0.f;
        const float4 y = at.total(o[i]);
        if (at.leads())
            store4((T *)p.o + (((long long)bi * p.L + t) * p.H + h) * p.P + at.c,
                   make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        if (p.lse && lane == 0) p.lse[((long long)bi * p.H + h) * p.L + t] = t < V ? m[i] + logf(total) : 0.f;
    }
}

// ------------------------------------------------------------------ backward, dq (and D = do . o)
// Grid: one block per (b, h, 8 WR queries).
template <typename T, int WR>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) window_rows_dq(WindowParams p) {
    constexpr int kRows = kWarps * WR;
    extern __shared__ float4 smem4[];
    const int pitch = p.P + 4, warp = threadIdx.x / 32, lane = threadIdx.x & 31, c = 4 * lane;
    const Lanes at(p.P);
    float *Q = (float *)smem4, *dO = Q + kRows * pitch, *K = dO + kRows * pitch, *Vs = K + kTile * pitch;
    const int nblk = (p.L + kRows - 1) / kRows, bh = blockIdx.x / nblk, bi = bh / p.H, h = bh % p.H, g = h / p.hpg;
    const int t0 = (blockIdx.x % nblk) * kRows, V = valid_tokens(p, bi), t1 = min(t0 + kRows, V);
    if (blockIdx.x == 0) write_status(p);
    float4 dq[WR];
    float D[WR], lse[WR];
    clear(dq);
    if (t0 < t1) {
        load_rows<T>(Q, pitch, p.q, bi, p.L, p.H, h, p.P, t0, kRows, t1);
        load_rows<T>(dO, pitch, p.d_o, bi, p.L, p.H, h, p.P, t0, kRows, t1);
#pragma unroll
        for (int i = 0; i < WR; ++i) {
            const int t = t0 + warp * WR + i;
            const long long own = (((long long)bi * p.L + t) * p.H + h) * p.P + c;
            float d = 0.f;
            if (t < t1 && c < p.P) d = dot4(load4((const T *)p.o + own), load4((const T *)p.d_o + own), 0.f);
            D[i] = warp_sum(d);
            const long long gate = ((long long)bi * p.H + h) * p.L + t;
            lse[i] = t < t1 ? p.lse[gate] : 0.f;
            if (t < t1 && lane == 0) p.delta[gate] = D[i];
        }
        const KeyTiles tiles(p, t0, t1);
        Parts k(p.P), v = k;
        auto fetch = [&](int j) {
            k.fetch<T>(p.k, bi, p.L, p.G, g, p.P, tiles.start(j), tiles.end(j));
            v.fetch<T>(p.v, bi, p.L, p.G, g, p.P, tiles.start(j), tiles.end(j));
        };
        fetch(0);
        for (int j = 0; j < tiles.n; ++j) {
            const int s0 = tiles.start(j), end = tiles.end(j);
            __syncthreads();
            k.put(K, pitch), v.put(Vs, pitch);
            __syncthreads();
            if (j + 1 < tiles.n) fetch(j + 1);
            float x[WR], dp[WR];
            scores(Q + warp * WR * pitch, K, pitch, p.P, x);
            scores(dO + warp * WR * pitch, Vs, pitch, p.P, dp);
#pragma unroll
            for (int i = 0; i < WR; ++i) {
                const int t = t0 + warp * WR + i, s = s0 + lane;
                x[i] = t < t1 && s < end && sees(p, t, s) ? expf(p.scale * x[i] - lse[i]) * (dp[i] - D[i]) : 0.f;
            }
            sums(x, K, pitch, at, dq);
        }
    }
#pragma unroll
    for (int i = 0; i < WR; ++i) {
        const int t = t0 + warp * WR + i;
        const float4 y = scaled(p.scale, at.total(dq[i]));
        if (t < p.L && at.leads()) store4((T *)p.dq + (((long long)bi * p.L + t) * p.H + h) * p.P + at.c, y);
    }
}

// ------------------------------------------------------------------ backward, dk and dv
// Grid: one cluster per (b, g, 8 WR keys), whose blocks take the tiles of the heads' queries in equal shares; after
// window_rows_dq, which leaves D.
template <typename T, int WR>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) window_rows_dkv(WindowParams p, int splits) {
    constexpr int kRows = kWarps * WR;
    extern __shared__ float4 smem4[];
    const int pitch = p.P + 4, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const Lanes at(p.P);
    float *K = (float *)smem4, *Vs = K + kRows * pitch, *Q = Vs + kRows * pitch, *dO = Q + kTile * pitch;
    const int nblk = (p.L + kRows - 1) / kRows, unit = blockIdx.x / splits, split = blockIdx.x % splits;
    const int bg = unit / nblk, bi = bg / p.G, g = bg % p.G;
    const int s0 = (unit % nblk) * kRows, V = valid_tokens(p, bi), s1 = min(s0 + kRows, V);
    float4 dk[WR], dv[WR];
    clear(dk), clear(dv);
    if (s0 < s1) {
        load_rows<T>(K, pitch, p.k, bi, p.L, p.G, g, p.P, s0, kRows, s1);
        load_rows<T>(Vs, pitch, p.v, bi, p.L, p.G, g, p.P, s0, kRows, s1);
        const int last = s0 < p.sinks ? V : (int)min((long long)V, (long long)s1 - 1 + p.W);
        const int nt = (last - s0 + kTile - 1) / kTile, all = nt * p.hpg, per = (all + splits - 1) / splits;
        const int end = min(all, (split + 1) * per);
        Parts q(p.P), d_o = q;
        float lse = 0.f, D = 0.f;
        auto fetch = [&](int u) {
            const int h = g * p.hpg + u / nt, t0 = s0 + u % nt * kTile, t = t0 + lane;
            q.fetch<T>(p.q, bi, p.L, p.H, h, p.P, t0, last);
            d_o.fetch<T>(p.d_o, bi, p.L, p.H, h, p.P, t0, last);
            const long long gate = ((long long)bi * p.H + h) * p.L + t;
            lse = t < last ? p.lse[gate] : 0.f, D = t < last ? p.delta[gate] : 0.f;
        };
        if (split * per < end) fetch(split * per);
        for (int u = split * per; u < end; ++u) {
            const int t = s0 + u % nt * kTile + lane;
            const float lse_t = lse, D_t = D;
            __syncthreads();
            q.put(Q, pitch), d_o.put(dO, pitch);
            __syncthreads();
            if (u + 1 < end) fetch(u + 1);
            float x[WR], dp[WR];
            scores(K + warp * WR * pitch, Q, pitch, p.P, x);
            scores(Vs + warp * WR * pitch, dO, pitch, p.P, dp);
#pragma unroll
            for (int i = 0; i < WR; ++i) {
                const int s = s0 + warp * WR + i;
                x[i] = t < last && s < s1 && sees(p, t, s) ? expf(p.scale * x[i] - lse_t) : 0.f;
                dp[i] = x[i] != 0.f ? x[i] * (dp[i] - D_t) : 0.f;
            }
            sums(x, dO, pitch, at, dv);
            sums(dp, Q, pitch, at, dk);
        }
    }
#pragma unroll
    for (int i = 0; i < WR; ++i) dk[i] = scaled(p.scale, at.total(dk[i])), dv[i] = at.total(dv[i]);
    if (splits == 1) {
#pragma unroll
        for (int i = 0; i < WR; ++i) {
            const int s = s0 + warp * WR + i;
            if (s < p.L && at.leads()) {
                const long long to = (((long long)bi * p.L + s) * p.G + g) * p.P + at.c;
                store4((T *)p.dk + to, dk[i]);
                store4((T *)p.dv + to, dv[i]);
            }
        }
        return;
    }
    __syncthreads();  // the sums take the keys' place
    if (at.leads()) {
#pragma unroll
        for (int i = 0; i < WR; ++i) {
            *(float4 *)(K + (warp * WR + i) * pitch + at.c) = dk[i];
            *(float4 *)(Vs + (warp * WR + i) * pitch + at.c) = dv[i];
        }
    }
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const int nq = p.P / 4;
    for (int e = split * kThreads + threadIdx.x; e < 2 * kRows * nq; e += splits * kThreads) {
        const int r = e / nq, c = 4 * (e - r * nq), s = s0 + r % kRows;
        if (s >= p.L) continue;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < splits; ++k) {
            const float4 y = *(const float4 *)(cluster.map_shared_rank(K, k) + r * pitch + c);  // K's rows, then V's
            t = make_float4(t.x + y.x, t.y + y.y, t.z + y.z, t.w + y.w);
        }
        store4((T *)(r < kRows ? p.dk : p.dv) + (((long long)bi * p.L + s) * p.G + g) * p.P + c, t);
    }
    cluster.sync();  // nobody leaves while its sums are read
}

long long blocks(const WindowParams &p, int heads, int rows) { return (long long)p.b * heads * ((p.L + rows - 1) / rows); }
// Four rows a warp read a tile for twice as many, and take twice as long over it: where they leave a block for every SM
// (fp32, heads of 64, window 256, forward, two and four rows: 1200 tokens of 24 heads 144 and 115 us, 600 of 8 heads 28 and
// 26.5, of 4 heads 18 and 26).
bool four_rows(const WindowParams &p, int heads) { return blocks(p, heads, 32) >= kSMs; }
constexpr int most_bytes(int rows) { return (rows + kTile) * 2 * 132 * 4; }  // asked for once, for every width

template <typename T, int WR>
cudaError_t forward(const WindowParams &p, cudaStream_t s) {
    constexpr int rows = kWarps * WR;
    const cudaError_t e = delta::allow_shared((const void *)window_rows_fwd<T, WR>, most_bytes(rows));
    if (e != cudaSuccess) return e;
    window_rows_fwd<T, WR><<<(unsigned)blocks(p, p.H, rows), kThreads, (rows + 2 * kTile) * (p.P + 4) * 4, s>>>(p);
    return cudaGetLastError();
}
template <typename T, int WR>
cudaError_t backward_q(const WindowParams &p, cudaStream_t s) {
    constexpr int rows = kWarps * WR;
    const cudaError_t e = delta::allow_shared((const void *)window_rows_dq<T, WR>, most_bytes(rows));
    if (e != cudaSuccess) return e;
    window_rows_dq<T, WR><<<(unsigned)blocks(p, p.H, rows), kThreads, (rows + kTile) * 2 * (p.P + 4) * 4, s>>>(p);
    return cudaGetLastError();
}
template <typename T, int WR>
cudaError_t backward_kv(const WindowParams &p, cudaStream_t s) {
    constexpr int rows = kWarps * WR;
    const cudaError_t e = delta::allow_shared((const void *)window_rows_dkv<T, WR>, most_bytes(rows));
    if (e != cudaSuccess) return e;
    // A cluster's blocks share the queries of a block's keys while there are not two blocks an SM and each has a tile, and where
    // the sinks' or a wide window's queries would keep one block long after the others are done.
    const long long units = blocks(p, p.G, rows), seen = p.sinks || p.L - p.W < rows ? p.L : p.W + rows;
    const long long tiles = p.hpg * ((seen + kTile - 1) / kTile);
    int splits = 1;
    while (splits < 8 && 2 * splits <= tiles && (units * splits < 2 * kSMs || tiles >= 128 * splits)) splits *= 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute cluster = {};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = splits, cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(units * splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (rows + kTile) * 2 * (p.P + 4) * 4;
    cfg.stream = s;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, window_rows_dkv<T, WR>, p, splits);
}
template <typename T>
cudaError_t forward(const WindowParams &p, cudaStream_t s) {
    return four_rows(p, p.H) ? forward<T, 4>(p, s) : forward<T, 2>(p, s);
}
template <typename T>
cudaError_t backward(const WindowParams &p, cudaStream_t s) {
    const cudaError_t e = four_rows(p, p.H) ? backward_q<T, 4>(p, s) : backward_q<T, 2>(p, s);
    if (e != cudaSuccess) return e;
    // the keys of the sinks are seen by every query: far past the window their block is the last to end (16000 tokens of 3 heads
    // of 32, window 16: 650 us with four rows, 412 with two)
    const bool sinks_last = p.sinks && p.L / 4 > p.W + 32;
    return four_rows(p, p.G) && !sinks_last ? backward_kv<T, 4>(p, s) : backward_kv<T, 2>(p, s);
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
