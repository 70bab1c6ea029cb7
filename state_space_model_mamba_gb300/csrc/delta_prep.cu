// delta_prep.cu -- per-chunk matrices of the gated delta rule, all chunks in
// parallel: K K^T and Q K^T of a key group once, then for every head of the group
// the decay-weighted triangles and the triangular inverse (delta_chunk.cuh).
//
// The inverse, per head: the four 16x16 diagonal blocks by forward substitution
// (a thread per column, everything in registers), the blocks below by
//     Tt_ij = -(W + Tt_ii diag(beta_i) W),  W = E_ij + sum_{j<=k<i} E_ik diag(beta_k) Tt_kj
// one diagonal distance after the other, as 16x16 products on the tensor cores
// with tf32 operands split in two (error 2^-21: the inverse is rounded to 2^-17
// only when it is stored).  Substitution of blocks stays accurate for repeated
// keys, where a power series of the triangle would lose every digit.
// What bounds it is the latency of this chain of small steps, about 2500 cycles a
// head; three blocks share an SM to cover it.
#include "delta_chunk.cuh"
#include "delta_mma.cuh"

namespace ssd {
namespace delta {
namespace {

constexpr int kThreads = 128;
constexpr int kLd = 68;       // floats per row of the fp32 matrices: rows 4 banks apart
constexpr int kHeadsPer = 4;  // heads of a group per block

struct PrepSmem {
    union {
        struct {
            __align__(16) unsigned char q[kChunk * 256], k[kChunk * 256];
        };
        struct {
            union {
                struct {
                    float E[kChunk * kLd];
                    float W[3][16 * 20];
                };
                __align__(16) unsigned char tri[4 * kTri];  // written once E is done with
            };
            float T[kChunk * kLd], A[kChunk * kLd];
        };
    };
    float ghi[kChunk], glo[kChunk], beta[kChunk];
    __align__(16) float gates[kGates / 4];
};

// d += a (16x16 at A, columns scaled by sc) times b (16x16 at B), fp32 rows of lda / ldb floats
__device__ __forceinline__ void block_product(float (&d)[2][4], const float *A, int lda, const float *sc, const float *B,
                                              int ldb, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        uint32_t ah[4], al[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = g + (i & 1) * 8, c = ks * 8 + t + (i >> 1) * 4;
            const float x = A[r * lda + c] * sc[c];
            ah[i] = __float_as_uint(x) & 0xFFFFE000u;
            al[i] = __float_as_uint(x - __uint_as_float(ah[i]));
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            uint32_t bh[2], bl[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = B[(ks * 8 + t + i * 4) * ldb + nt * 8 + g];
                bh[i] = __float_as_uint(x) & 0xFFFFE000u;
                bl[i] = __float_as_uint(x - __uint_as_float(bh[i]));
            }
            mma8_tf32(d[nt], al, bh[0], bh[1]);
            mma8_tf32(d[nt], ah, bl[0], bl[1]);
            mma8_tf32(d[nt], ah, bh[0], bh[1]);
        }
    }
}
__device__ __forceinline__ void store_block(float *dst, int ld, const float (&d)[2][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        *(float2 *)(dst + g * ld + nt * 8 + 2 * t) = make_float2(d[nt][0], d[nt][1]);
        *(float2 *)(dst + (g + 8) * ld + nt * 8 + 2 * t) = make_float2(d[nt][2], d[nt][3]);
    }
}
__device__ __forceinline__ void load_block(float (&d)[2][4], const float *src, int ld, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        const float2 a = *(const float2 *)(src + g * ld + nt * 8 + 2 * t), b = *(const float2 *)(src + (g + 8) * ld + nt * 8 + 2 * t);
        d[nt][0] = a.x, d[nt][1] = a.y, d[nt][2] = b.x, d[nt][3] = b.y;
    }
}

// Grid: one block per (b, group, slice of the group's heads, chunk).  NP: dstate padded to 64 or 128.
template <int NP>
__global__ void __launch_bounds__(kThreads, 3) delta_prep_kernel(const ChunkParams cp) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    PrepSmem &s = *(PrepSmem *)smem_raw;
    const DeltaParams &p = cp.p;
    const int slices = (p.hpg + kHeadsPer - 1) / kHeadsPer;
    const int chunk = blockIdx.x % cp.n, slice = blockIdx.x / cp.n % slices;
    const int bg = blockIdx.x / cp.n / slices, bi = bg / p.G, grp = bg % p.G;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    if (blockIdx.x == 0) write_status(p);
    const int V = valid_tokens(p, bi), t0 = chunk * kChunk;
    if (t0 >= V) return;
    constexpr int LINE = NP * 2;

    // q and k rows of the chunk; absent tokens and padding columns are zero
    {
        const uint32_t qs = smem_u32(s.q), ks = smem_u32(s.k);
        for (int i = tid; i < kChunk * (NP / 8); i += kThreads) {
            const int r = i / (NP / 8), c = i % (NP / 8);
            const bool real = t0 + r < V && c * 8 < p.N;
            const long long at = real ? (((long long)bi * p.L + t0 + r) * p.G + grp) * p.N + c * 8 : 0;
            cp_async16(qs + swz<LINE>(r, c), (const bf16 *)p.q + at, real);
            cp_async16(ks + swz<LINE>(r, c), (const bf16 *)p.k + at, real);
        }
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
    }
    // warp w: rows 16 w .. 16 w + 15, columns up to its diagonal block
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[i][e] = qk[i][e] = 0.f;
    {
        const uint32_t qs = smem_u32(s.q), ks = smem_u32(s.k);
#pragma unroll
        for (int st = 0; st < NP / 16; ++st) {
            uint32_t aq[4], ak[4];
            const int ar = 16 * warp + (lane & 15), ac = 2 * st + (lane >> 4);
            ldsm4(aq, qs + swz<LINE>(ar, ac));
            ldsm4(ak, ks + swz<LINE>(ar, ac));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= warp) {
                    uint32_t b[4];
                    ldsm4(b, ks + swz<LINE>(16 * j + (lane & 7) + ((lane >> 4) & 1) * 8, 2 * st + ((lane >> 3) & 1)));
                    mma16(kk[2 * j], ak, b[0], b[1]);
                    mma16(kk[2 * j + 1], ak, b[2], b[3]);
                    mma16(qk[2 * j], aq, b[0], b[1]);
                    mma16(qk[2 * j + 1], aq, b[2], b[3]);
                }
        }
    }

    const int h_end = min((grp + 1) * p.hpg, grp * p.hpg + (slice + 1) * kHeadsPer);
    for (int h = grp * p.hpg + slice * kHeadsPer; h < h_end; ++h) {
        const long long bh = (long long)bi * p.H + h;
        float *gates = s.gates;
        __syncthreads();  // the tiles, or the image of the head before, have been read
        if (warp == 0) {
            // gamma in fp64, kept as hi + lo: differences of it stay exact to fp32 after strong decays
            const int i0 = 2 * lane;
            const long long at = bh * p.L + t0 + i0;
            const bool r0 = t0 + i0 < V, r1 = t0 + i0 + 1 < V;
            const double g0 = r0 ? (double)clamp_log_decay(p.g[at]) : 0.0;
            const double g1 = r1 ? (double)clamp_log_decay(p.g[at + 1]) : 0.0;
            double sum = g0 + g1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            const double c0 = sum - g1, c1 = sum, total = __shfl_sync(0xffffffffu, sum, 31);
            s.ghi[i0] = (float)c0;
            s.glo[i0] = (float)(c0 - (double)(float)c0);
            s.ghi[i0 + 1] = (float)c1;
            s.glo[i0 + 1] = (float)(c1 - (double)(float)c1);
            const float b0 = r0 ? p.beta[at] : 0.f, b1 = r1 ? p.beta[at + 1] : 0.f;
            s.beta[i0] = b0;
            s.beta[i0 + 1] = b1;
            gates[i0] = expf((float)c0);
            gates[i0 + 1] = expf((float)c1);
            gates[kChunk + i0] = expf((float)(total - c0));
            gates[kChunk + i0 + 1] = expf((float)(total - c1));
            gates[2 * kChunk + i0] = b0;
            gates[2 * kChunk + i0 + 1] = b1;
        }
        __syncthreads();
        // E and A
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
            if (nt / 2 <= warp) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int i = 16 * warp + g + 8 * half, j = 8 * nt + 2 * t;
                    const float gi = s.ghi[i], li = s.glo[i];
                    const float d0 = j <= i ? expf((gi - s.ghi[j]) + (li - s.glo[j])) : 0.f;
                    const float d1 = j + 1 <= i ? expf((gi - s.ghi[j + 1]) + (li - s.glo[j + 1])) : 0.f;
                    *(float2 *)(s.E + i * kLd + j) = make_float2(j < i ? d0 * kk[nt][2 * half] : 0.f,
                                                                 j + 1 < i ? d1 * kk[nt][2 * half + 1] : 0.f);
                    *(float2 *)(s.A + i * kLd + j) = make_float2(j <= i ? p.scale * d0 * qk[nt][2 * half] : 0.f,
                                                                 j + 1 <= i ? p.scale * d1 * qk[nt][2 * half + 1] : 0.f);
                }
            }
        __syncthreads();
        // diagonal blocks: column c of block tid / 16
        if (tid < 64) {
            const int o = 16 * (tid >> 4), c = tid & 15;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float a = i > c ? -s.E[(o + i) * kLd + o + c] : 0.f;
#pragma unroll
                for (int m = 0; m < i; ++m) a = fmaf(-s.E[(o + i) * kLd + o + m] * s.beta[o + m], x[m], a);
                x[i] = i > c ? a : 0.f;
                s.T[(o + i) * kLd + o + c] = x[i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int d = 1; d < 4; ++d) {
            if (warp < 4 - d) {
                const int j = warp, i = warp + d;
                float w[2][4];
                load_block(w, s.E + 16 * i * kLd + 16 * j, kLd, lane);
                for (int k = j; k < i; ++k)
                    block_product(w, s.E + 16 * i * kLd + 16 * k, kLd, s.beta + 16 * k, s.T + 16 * k * kLd + 16 * j, kLd, lane);
                store_block(s.W[warp], 20, w, lane);
                __syncwarp();
                block_product(w, s.T + 16 * i * kLd + 16 * i, kLd, s.beta + 16 * i, s.W[warp], 20, lane);
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[nt][e] = -w[nt][e];
                store_block(s.T + 16 * i * kLd + 16 * j, kLd, w, lane);
            }
            __syncthreads();
        }
        // Tt as hi and lo parts, a thread per 16-byte piece
        for (int x = tid; x < 10 * 32; x += kThreads) {
            const int blk = x >> 5, br = blk >= 6 ? 3 : (blk >= 3 ? 2 : (blk >= 1 ? 1 : 0)), bc = blk - br * (br + 1) / 2;
            const int i = 16 * br + ((x >> 1) & 15), c = 2 * bc + (x & 1);
            const float *src = s.T + i * kLd + 8 * c;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split2(src[2 * e], src[2 * e + 1], hi[e], lo[e]);
            *(uint4 *)(s.tri + tri_piece(i, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *(uint4 *)(s.tri + 2 * kTri + tri_piece(i, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        // At = A + A diag(beta) Tt: five block products a warp
        {
            constexpr int nblk[4] = {2, 2, 2, 4};
            constexpr int rows[4][4] = {{3, 0, 0, 0}, {2, 1, 0, 0}, {3, 2, 0, 0}, {3, 1, 2, 3}};
            constexpr int cols[4][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}, {1, 1, 0, 0}, {2, 1, 2, 3}};
            for (int x = 0; x < nblk[warp]; ++x) {
                const int i = rows[warp][x], j = cols[warp][x];
                float w[2][4];
                load_block(w, s.A + 16 * i * kLd + 16 * j, kLd, lane);
                for (int k = j; k <= i; ++k)
                    block_product(w, s.A + 16 * i * kLd + 16 * k, kLd, s.beta + 16 * k, s.T + 16 * k * kLd + 16 * j, kLd, lane);
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t hi, lo;
                        split2(w[nt][2 * half], w[nt][2 * half + 1], hi, lo);
                        unsigned char *dst = s.tri + kTri + tri_piece(16 * i + g + 8 * half, 2 * j + nt) + 4 * t;
                        *(uint32_t *)dst = hi;
                        *(uint32_t *)(dst + 2 * kTri) = lo;
                    }
            }
        }
        __syncthreads();
        uint4 *out = (uint4 *)(cp.img + (bh * cp.n + chunk) * (long long)kImgBytes);
        for (int i = tid; i < kGates / 16; i += kThreads) out[i] = ((const uint4 *)s.gates)[i];
        for (int i = tid; i < 4 * kTri / 16; i += kThreads) out[kImgTri / 16 + i] = ((const uint4 *)s.tri)[i];
    }
}

}  // namespace

cudaError_t launch_chunk_prep(const ChunkParams &c, cudaStream_t s) {
    const DeltaParams &p = c.p;
    const int bytes = (int)sizeof(PrepSmem);
    const unsigned grid = (unsigned)c.n * ((p.hpg + kHeadsPer - 1) / kHeadsPer) * p.b * p.G;
    auto kernel = p.N <= 64 ? delta_prep_kernel<64> : delta_prep_kernel<128>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, bytes, s>>>(c);
    return cudaGetLastError();
}

}  // namespace delta
}  // namespace ssd
