// window_step.cu -- the ring of window attention: a prompt's visible tokens into
// their entries, and one decoded token per request.
//
// The ring makes the mask disappear: what a token sees is every entry written so far, in any
// order, so the step is softmax(scale q K^T) V over min(position + 1, sinks + window) rows of one
// slot.  It reads each row of K and V once and is bound by HBM; what it needs is many loads in flight and few
// launches.  A block takes one key group of one request (all its heads, so a row serves up to 16 of
// them), its warps take tiles of 16 rows.  In bf16 the products run on mma.sync.m16n8k16
// straight from the loaded registers: the order of a product's inner index is free, so a thread's
// fragments are the 16-byte pieces that it loads, and the scores' accumulators are the next product's
// operand.  Probabilities are rounded to bf16 there (2^-8 of each at most; sums stay fp32).  Few
// requests are split over the blocks of a cluster, which join their sums through distributed
// shared memory in the cluster's order: one launch, no workspace, fixed order of sums.
// The new token's own row is taken from the arguments by every block, so the write of its entry
// races with nobody.
#include <cooperative_groups.h>

#include "tc_ptx.cuh"
#include "window_internal.cuh"

namespace cg = cooperative_groups;

namespace ssd {
namespace window {
namespace {

constexpr int kThreads = 128, kStages = 2;
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ prompts into the ring
// One thread per 16 (or 8) bytes of an entry of K and the same of V.
template <typename Vec>
__global__ void __launch_bounds__(256) ring_fill_kernel(RingParams p, int kept, int vecs) {
    const long long i = blockIdx.x * 256ll + threadIdx.x;
    const long long row = i / vecs;
    const int bi = (int)(row / kept), j = (int)(row % kept), c = (int)(i % vecs);
    if (bi >= p.b) return;
    const long long slot = p.index ? (long long)p.index[bi] : (long long)bi;
    int V = p.valid_len ? p.valid_len[bi] : p.L;
    V = V < 0 ? 0 : (V > p.L ? p.L : V);
    if (slot < 0 || slot >= p.slots || j >= V) return;
    const int t = j < p.sinks ? j : j + (V - 1 - j) / p.W * p.W;
    const long long from = ((long long)bi * p.L + t) * vecs + c, to = (slot * ((long long)p.sinks + p.W) + j) * vecs + c;
    const Vec k = __ldg((const Vec *)p.k + from), v = __ldg((const Vec *)p.v + from);
    ((Vec *)p.k_cache)[to] = k;
    ((Vec *)p.v_cache)[to] = v;
}

// ------------------------------------------------------------------ one token
// What a block finds out about its request.
struct Request {
    int bi, g, chunk, split, n, at;  // n entries to read, the new token's is `at`
    long long slot;
    bool live;
    __device__ __forceinline__ Request(const RingParams &p, int splits, int chunks) {
        split = blockIdx.x % splits;
        const int unit = blockIdx.x / splits;
        chunk = unit % chunks;
        g = unit / chunks % p.G;
        bi = unit / chunks / p.G;
        slot = p.index ? (long long)p.index[bi] : (long long)bi;
        const int pos = p.position[bi];
        live = slot >= 0 && slot < p.slots && pos >= 0;
        const long long entries = (long long)p.sinks + p.W;
        n = (int)min((long long)pos + 1, entries);
        at = pos < p.sinks ? pos : p.sinks + (pos - p.sinks) % p.W;
    }
    // first element of the row of entry j
    __device__ __forceinline__ long long entry(const RingParams &p, int j) const {
        return ((slot * ((long long)p.sinks + p.W) + j) * p.G + g) * p.P;
    }
    __device__ __forceinline__ long long own(const RingParams &p) const { return ((long long)bi * p.G + g) * p.P; }
};

// NS partial softmax sums of ROWS heads (NS * ROWS = 64): sums O relative to the exponent m, weights l.
template <int NS, int ROWS>
struct Shares {
    float m[NS][ROWS], l[NS][ROWS], M[ROWS], total[ROWS];
    float O[1];  // [NS][ROWS][P], then [ROWS][P] joined
};
// Joins the block's shares, then the cluster's, and writes the rows of o.
template <typename T, int NS, int ROWS>
__device__ __forceinline__ void join(const RingParams &p, const Request &r, Shares<NS, ROWS> *sh, int splits, int heads) {
    float *joined = sh->O + NS * ROWS * p.P;
    __syncthreads();
    if (threadIdx.x < ROWS) {
        float m = -INFINITY, t = 0.f;
        for (int i = 0; i < NS; ++i) m = fmaxf(m, sh->m[i][threadIdx.x]);
        const float base = m == -INFINITY ? 0.f : m;
        for (int i = 0; i < NS; ++i) {
            const float f = exp2f(sh->m[i][threadIdx.x] - base);
            t += sh->l[i][threadIdx.x] * f;
            sh->m[i][threadIdx.x] = f;
        }
        sh->M[threadIdx.x] = m;
        sh->total[threadIdx.x] = t;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < heads * p.P; e += kThreads) {
        const int row = e / p.P;
        float s = 0.f;
        for (int i = 0; i < NS; ++i) s += sh->m[i][row] * sh->O[i * ROWS * p.P + e];
        joined[e] = s;
    }
    cg::cluster_group cluster = cg::this_cluster();
    if (splits > 1)
        cluster.sync();
    else
        __syncthreads();
    const long long at = ((long long)r.bi * p.H + r.g * p.hpg + r.chunk * ROWS) * p.P;
    for (int e = r.split * kThreads + threadIdx.x; e < heads * p.P; e += splits * kThreads) {
        const int row = e / p.P;
        float m = -INFINITY, s = 0.f, t = 0.f;
        for (int k = 0; k < splits; ++k) m = fmaxf(m, splits > 1 ? cluster.map_shared_rank(sh, k)->M[row] : sh->M[row]);
        const float base = m == -INFINITY ? 0.f : m;
        for (int k = 0; k < splits; ++k) {
            const Shares<NS, ROWS> *from = splits > 1 ? cluster.map_shared_rank(sh, k) : sh;
            const float f = exp2f(from->M[row] - base);
            s += f * from->O[NS * ROWS * p.P + e];
            t += f * from->total[row];
        }
        store1((T *)p.o + at + e, s / t);
    }
    if (splits > 1) cluster.sync();  // nobody leaves while its sums are read
}
template <typename T>
__device__ __forceinline__ void absent(const RingParams &p, const Request &r, int rows, int heads) {
    const long long at = ((long long)r.bi * p.H + r.g * p.hpg + r.chunk * rows) * p.P;
    if (r.split == 0)
        for (int e = threadIdx.x; e < heads * p.P; e += kThreads) store1((T *)p.o + at + e, 0.f);
}
template <typename T>
__device__ __forceinline__ void write_entry(const RingParams &p, const Request &r) {
    if (r.split == 0 && r.chunk == 0)
        for (int c = threadIdx.x; c < p.P; c += kThreads) {
            const long long to = r.entry(p, r.at) + c, from = r.own(p) + c;
            ((T *)p.k_cache)[to] = ((const T *)p.k)[from];
            ((T *)p.v_cache)[to] = ((const T *)p.v)[from];
        }
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *(const uint32_t *)&v;
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// A lane's 16-byte pieces on their way to shared memory, in groups that are waited for in order; what a lane copies it reads
// itself, so that a warp's stages need no barrier.  Rows that are not there become zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// bf16.  NI = ceil(P / 32).  A fragment of m16n8k16 wants inner indices 2c, 2c + 1, 2c + 8, 2c + 9 of lane 4 r + c; it is
// given elements 32 i + 8 c + (0 .. 3) for step 2 i and + (4 .. 7) for step 2 i + 1, of q and k alike.
// A column tile's column n of the second product is column 64 v + 8 n + j of v for tile (v, j).
template <int NI>
__global__ void __launch_bounds__(kThreads, 3) ring_step_mma(RingParams p, int splits, int chunks) {
    extern __shared__ float4 smem4[];
    Shares<4, 16> *sh = (Shares<4, 16> *)smem4;
    constexpr int NV = (NI + 1) / 2;
    const Request r(p, splits, chunks);
    const int heads = min(16, p.hpg - r.chunk * 16);
    if (!r.live) {
        absent<bf16>(p, r, 16, heads);
        return;
    }
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, row = lane >> 2, c = lane & 3;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const float f = p.scale * kLog2e;
    float o[NV][8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) o[v][j][0] = o[v][j][1] = o[v][j][2] = o[v][j][3] = 0.f;
    const int tiles = (r.n + 15) / 16, per = (tiles + splits - 1) / splits, last = min(tiles, (r.split + 1) * per);
    const bf16 *kown = (const bf16 *)p.k + r.own(p), *vown = (const bf16 *)p.v + r.own(p);
    // tiles ahead of the one in work, each 2 NI + 4 NV pieces a lane
    constexpr int kPieces = 2 * NI + 4 * NV;
    const uint32_t ring = tc::smem_u32(smem4) + (uint32_t)(warp * kStages * kPieces * 32 + lane) * 16u;
    auto fetch = [&](int tile, int stage) {
        if (tile < last) {
            const int j0 = tile * 16;
            uint32_t to = ring + (uint32_t)(stage * kPieces * 32) * 16u;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int j = j0 + 8 * x + row;
                const bf16 *src = j == r.at ? kown : (const bf16 *)p.k_cache + r.entry(p, min(j, r.n - 1));
#pragma unroll
                for (int i = 0; i < NI; ++i, to += 512) {
                    const bool in = j < r.n && 32 * i + 8 * c < p.P;
                    copy16(to, src + (in ? 32 * i + 8 * c : 0), in);
                }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int j = j0 + 8 * (x >> 1) + 2 * c + (x & 1);
                const bf16 *src = j == r.at ? vown : (const bf16 *)p.v_cache + r.entry(p, min(j, r.n - 1));
#pragma unroll
                for (int v = 0; v < NV; ++v, to += 512) {
                    const bool in = j < r.n && 64 * v + 8 * row < p.P;
                    copy16(to, src + (in ? 64 * v + 8 * row : 0), in);
                }
            }
        }
        copy_commit();
    };
    constexpr int kStep = kThreads / 32;
    int stage = 0, ahead = r.split * per + warp;
#pragma unroll
    for (int x = 0; x < kStages - 1; ++x, ahead += kStep) fetch(ahead, x);
    uint32_t qa[2 * NI][4];
    {
        const bf16 *q = (const bf16 *)p.q + ((long long)r.bi * p.H + r.g * p.hpg + r.chunk * 16) * p.P;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int col = 32 * i + 8 * c;
            const uint4 x = row < heads && col < p.P ? __ldg((const uint4 *)(q + row * p.P + col)) : zero;
            const uint4 y = row + 8 < heads && col < p.P ? __ldg((const uint4 *)(q + (row + 8) * p.P + col)) : zero;
            qa[2 * i][0] = x.x, qa[2 * i][1] = y.x, qa[2 * i][2] = x.y, qa[2 * i][3] = y.y;
            qa[2 * i + 1][0] = x.z, qa[2 * i + 1][1] = y.z, qa[2 * i + 1][2] = x.w, qa[2 * i + 1][3] = y.w;
        }
    }
    for (int tile = r.split * per + warp; tile < last; tile += kStep, ahead += kStep) {
        const int j0 = tile * 16;
        fetch(ahead, stage == 0 ? kStages - 1 : stage - 1);
        copy_wait<kStages - 1>();
        const uint32_t from = ring + (uint32_t)(stage * kPieces * 32) * 16u;
        stage = stage == kStages - 1 ? 0 : stage + 1;
        uint4 kr[2][NI], vr[4][NV];
#pragma unroll
        for (int x = 0; x < 2 * NI; ++x) kr[x / NI][x % NI] = tc::ld_shared_v4(from + x * 512);
#pragma unroll
        for (int x = 0; x < 4 * NV; ++x) vr[x / NV][x % NV] = tc::ld_shared_v4(from + (2 * NI + x) * 512);
        float s[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                mma(s[x], qa[2 * i], kr[x][i].x, kr[x][i].y);
                mma(s[x], qa[2 * i + 1], kr[x][i].z, kr[x][i].w);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s[x][e] = j0 + 8 * x + 2 * c + (e & 1) < r.n ? f * s[x][e] : -INFINITY;
        }
        float corr[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float mn = fmaxf(m[h], quad_max(fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]))));
            const float base = mn == -INFINITY ? 0.f : mn;
            corr[h] = exp2f(m[h] - base);
            m[h] = mn;
            l[h] *= corr[h];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 2 * h; e < 2 * h + 2; ++e) l[h] += s[x][e] = exp2f(s[x][e] - base);
        }
        const uint32_t pa[4] = {pack2(s[0][0], s[0][1]), pack2(s[0][2], s[0][3]), pack2(s[1][0], s[1][1]), pack2(s[1][2], s[1][3])};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const uint32_t w[4][4] = {{vr[0][v].x, vr[0][v].y, vr[0][v].z, vr[0][v].w}, {vr[1][v].x, vr[1][v].y, vr[1][v].z, vr[1][v].w},
                                      {vr[2][v].x, vr[2][v].y, vr[2][v].z, vr[2][v].w}, {vr[3][v].x, vr[3][v].y, vr[3][v].z, vr[3][v].w}};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                float(&d)[4] = o[v][j];
                d[0] *= corr[0], d[1] *= corr[0], d[2] *= corr[1], d[3] *= corr[1];
                mma(d, pa, __byte_perm(w[0][j >> 1], w[1][j >> 1], sel), __byte_perm(w[2][j >> 1], w[3][j >> 1], sel));
            }
        }
    }
    copy_wait<0>();
    write_entry<bf16>(p, r);  // last: a store waits for its load, and what comes behind it with it
    __syncthreads();  // the shares take the stages' place
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        const int head = row + 8 * h;
        if (c == 0) sh->m[warp][head] = m[h], sh->l[warp][head] = l[h];
        float *dst = sh->O + (warp * 16 + head) * p.P;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int col = 64 * v + 8 * (2 * c + n);
                if (col < p.P) {
                    *(float4 *)(dst + col) = make_float4(o[v][0][2 * h + n], o[v][1][2 * h + n], o[v][2][2 * h + n], o[v][3][2 * h + n]);
                    *(float4 *)(dst + col + 4) = make_float4(o[v][4][2 * h + n], o[v][5][2 * h + n], o[v][6][2 * h + n], o[v][7][2 * h + n]);
                }
            }
    }
    join<bf16, 4, 16>(p, r, sh, splits, heads);
}

// fp32 (and bf16 whose rows are no multiple of 16 bytes): 8 lanes hold a row, 16 rows at a time, 4 heads a block,
// every 8 lanes with sums of their own.
template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) ring_step_rows(RingParams p, int splits, int chunks) {
    extern __shared__ float4 smem4[];
    Shares<16, 4> *sh = (Shares<16, 4> *)smem4;
    const Request r(p, splits, chunks);
    const int heads = min(4, p.hpg - r.chunk * 4);
    if (!r.live) {
        absent<T>(p, r, 4, heads);
        return;
    }
    const int sub = threadIdx.x / 8, lane = threadIdx.x & 7;
    write_entry<T>(p, r);
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float f = p.scale * kLog2e;
    float4 q[4][NC], o[4][NC];
    float m[4], l[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        m[h] = -INFINITY, l[h] = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int col = 32 * i + 4 * lane;
            const long long at = ((long long)r.bi * p.H + r.g * p.hpg + r.chunk * 4 + h) * p.P + col;
            q[h][i] = h < heads && col < p.P ? load4((const T *)p.q + at) : zero;
            o[h][i] = zero;
        }
    }
    const int tiles = (r.n + 15) / 16, per = (tiles + splits - 1) / splits, last = min(tiles, (r.split + 1) * per);
    for (int tile = r.split * per; tile < last; ++tile) {
        const int j = tile * 16 + sub;
        const bool in = j < r.n;
        const T *ks = j == r.at ? (const T *)p.k + r.own(p) : (const T *)p.k_cache + r.entry(p, j);
        const T *vs = j == r.at ? (const T *)p.v + r.own(p) : (const T *)p.v_cache + r.entry(p, j);
        float4 k[NC], v[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int col = 32 * i + 4 * lane;
            k[i] = in && col < p.P ? load4(ks + col) : zero;
            v[i] = in && col < p.P ? load4(vs + col) : zero;
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                x = fmaf(q[h][i].x, k[i].x, fmaf(q[h][i].y, k[i].y, fmaf(q[h][i].z, k[i].z, fmaf(q[h][i].w, k[i].w, x))));
#pragma unroll
            for (int d = 4; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
            x = in ? f * x : -INFINITY;
            const float mn = fmaxf(m[h], x), base = mn == -INFINITY ? 0.f : mn;
            const float corr = exp2f(m[h] - base), e = exp2f(x - base);
            m[h] = mn;
            l[h] = fmaf(l[h], corr, e);
#pragma unroll
            for (int i = 0; i < NC; ++i)
                o[h][i] = make_float4(fmaf(o[h][i].x, corr, e * v[i].x), fmaf(o[h][i].y, corr, e * v[i].y),
                                      fmaf(o[h][i].z, corr, e * v[i].z), fmaf(o[h][i].w, corr, e * v[i].w));
        }
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        if (lane == 0) sh->m[sub][h] = m[h], sh->l[sub][h] = l[h];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int col = 32 * i + 4 * lane;
            if (col < p.P) *(float4 *)(sh->O + (sub * 4 + h) * p.P + col) = o[h][i];
        }
    }
    join<T, 16, 4>(p, r, sh, splits, heads);
}

template <class K>
cudaError_t launch_clusters(K kernel, const RingParams &p, int heads_a_block, int shared, cudaStream_t s) {
    int chunks = (p.hpg + heads_a_block - 1) / heads_a_block, splits = 1;
    const long long units = (long long)p.b * p.G * chunks, entries = (long long)p.sinks + p.W;
    // Two blocks a SM while each keeps 64 rows.  A block's beginning and end are some 7 us, so that halves of full ones do not pay
    // (192 requests of up to 1028 rows: 127 us, in halves 151), nor do blocks of two warps (144) or one (142), nor
    // clusters of 16 for one request.
    while (splits < 8 && units * splits < 2 * kSMs && entries / (2 * splits) >= 64) splits *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = splits;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, splits, chunks);
}
template <int NS, int ROWS>
constexpr int shared_bytes(int P) {
    return (int)sizeof(Shares<NS, ROWS>) + (NS + 1) * ROWS * P * 4;
}
static_assert(shared_bytes<4, 16>(128) <= 49152 && shared_bytes<16, 4>(128) <= 49152, "no attribute asked for");
template <typename T>
cudaError_t step_rows(const RingParams &p, cudaStream_t s) {
    const int shared = shared_bytes<16, 4>(p.P);
    switch ((p.P + 31) / 32) {
        case 1: return launch_clusters(ring_step_rows<T, 1>, p, 4, shared, s);
        case 2: return launch_clusters(ring_step_rows<T, 2>, p, 4, shared, s);
        case 3: return launch_clusters(ring_step_rows<T, 3>, p, 4, shared, s);
        default: return launch_clusters(ring_step_rows<T, 4>, p, 4, shared, s);
    }
}

template <int NI>
cudaError_t step_mma(const RingParams &p, cudaStream_t s) {
    constexpr int ring = kThreads * kStages * (2 * NI + 4 * ((NI + 1) / 2)) * 16, join = shared_bytes<4, 16>(32 * NI);
    constexpr int shared = ring > join ? ring : join;
    const cudaError_t e = delta::allow_shared((const void *)ring_step_mma<NI>, shared);
    return e != cudaSuccess ? e : launch_clusters(ring_step_mma<NI>, p, 16, shared, s);
}

}  // namespace

cudaError_t launch_fill(const RingParams &p, bool is_bf16, cudaStream_t s) {
    const long long bytes = (long long)p.G * p.P * (is_bf16 ? 2 : 4), entries = (long long)p.sinks + p.W;
    const int kept = (int)(entries < p.L ? entries : p.L), wide = bytes % 16 == 0, vecs = (int)(bytes / (wide ? 16 : 8));
    const unsigned grid = (unsigned)(((long long)p.b * kept * vecs + 255) / 256);
    if (wide)
        ring_fill_kernel<uint4><<<grid, 256, 0, s>>>(p, kept, vecs);
    else
        ring_fill_kernel<uint2><<<grid, 256, 0, s>>>(p, kept, vecs);
    return cudaGetLastError();
}

cudaError_t launch_step(const RingParams &p, bool is_bf16, cudaStream_t s) {
    if (!is_bf16) return step_rows<float>(p, s);
    if (p.P % 8) return step_rows<bf16>(p, s);
    switch ((p.P + 31) / 32) {
        case 1: return step_mma<1>(p, s);
        case 2: return step_mma<2>(p, s);
        case 3: return step_mma<3>(p, s);
        default: return step_mma<4>(p, s);
    }
}

}  // namespace window
}  // namespace ssd
