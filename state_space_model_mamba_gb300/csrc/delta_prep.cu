// delta_prep.cu -- per-chunk matrices of the gated delta rule, all chunks in
// parallel (delta_chunk.cuh): K K^T and Q K^T of a key group once, on the tensor
// cores with K stacked on Q, then for every head of the group the decay-weighted
// triangles and the triangular inverse.
//
// With E = D o strict lower (K K^T) and A = scale D o lower (Q K^T),
//     Tt (I + diag(beta) E) = -E      and      At (I + diag(beta) E) = A,
// so both matrices are rows of one right-hand solve with a unit lower triangle, and
// every row is independent: thread i of 128 holds row i of [E; A] as it comes out of
// tensor memory and substitutes from its last column to its first in fp32,
//     y_j = r_j - sum_{m > j} (beta_m y_m) E_mj,
// 16 columns at a time: first the columns already solved (beta y from shared memory,
// column m of all threads side by side; E rows as broadcasts), then the 16 x 16 triangle
// in registers.  Substitution stays accurate for repeated keys, where a power series
// of the triangle would lose every digit.
// What bounds it are the multiply-adds of the two solves, 2000 for each of the rows
// 32 .. 63 and 500 for the others (the backward needs A, not At, and solves half).  Rolled over the blocks: the whole substitution
// unrolled (40 KB of code) waited for instructions half of the time.  Which
// warps get the long rows changes from block to block.
#include "delta_chunk.cuh"
#include "delta_mma.cuh"

namespace ssd {
namespace delta {
namespace {

using namespace tc;

constexpr int kThreads = 128;
constexpr int kHeadsPer = 4;          // heads of a group per block
constexpr int kLdE = 68;              // floats per row of E: 16-byte pieces, rows four banks apart
constexpr uint32_t kAccCols = 64;

struct PrepMaps {
    CUtensorMap k, q;
};

// Grid: one block per (b, group, slice of the group's heads, chunk).
__global__ void __launch_bounds__(kThreads) delta_prep_kernel(const ChunkParams cp, const __grid_constant__ PrepMaps maps) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar_load, bar_mma;
    __shared__ uint32_t s_tmem;
    __shared__ __align__(16) float s_e[kChunk * kLdE];
    __shared__ float2 s_gam[kChunk];   // gamma log2(e), hi and lo
    __shared__ float s_beta[kChunk];
    const DeltaParams &p = cp.p;
    const int slices = (p.hpg + kHeadsPer - 1) / kHeadsPer;
    const int chunk = blockIdx.x % cp.n, slice = blockIdx.x / cp.n % slices;
    const int bg = blockIdx.x / cp.n / slices, bi = bg / p.G, grp = bg % p.G;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0) write_status(p);
    const int V = valid_tokens(p, bi), t0 = chunk * kChunk;
    if (t0 >= V) return;
    const uint32_t kq = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t halves = p.N > 64 ? 2u : 1u;
    // where rows lie changes from block to block, so that the long solves do not always land on the same schedulers
    const uint32_t hash = blockIdx.x * 0x9E3779B1u;
    const int flip = hash >> 31;                          // tokens 32 .. 63 in rows (and columns) 0 .. 31
    const uint32_t k_off = (hash >> 30 & 1) * 8192u;      // K rows behind the Q rows
    if (tid == 0) {
        mbar_init(&bar_load, 1);
        mbar_init(&bar_mma, 1);
        mbar_fence_init();
        mbar_arrive_expect_tx(&bar_load, halves * 16384u);
        for (uint32_t kb = 0; kb < halves; ++kb)
            for (int x = 0; x < 2; ++x) {
                const int tok = t0 + 32 * (x ^ flip);
                tma_tile(kq + kb * 16384u + k_off + 4096u * x, &maps.k, &bar_load, 64 * kb, grp, tok, bi);
                tma_tile(kq + kb * 16384u + (k_off ^ 8192u) + 4096u * x, &maps.q, &bar_load, 64 * kb, grp, tok, bi);
            }
    }
    if (warp == 0) tmem_alloc(&s_tmem, kAccCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;
    bool ok = true;
    if (warp == 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bar_load, 0));
        if (ok && lane == 0) {
            const int nks = (p.N + 15) / 16;
            for (int ks = 0; ks < nks; ++ks)
                mma_bf16(tm, sdesc_kmajor(kq, ks, 16384), sdesc_kmajor(kq + k_off, ks, 16384), idesc_bf16(128, 64, false, false), ks > 0);
            mma_commit(&bar_mma);
        }
        __syncwarp();
    }
    const int i = (tid & 63) ^ (32 * flip);  // the row's token
    const bool keys = (tid < kChunk) == (k_off == 0), live = t0 + i < V;  // rows of absent tokens may hold anything: made zero
    const int h_end = min((grp + 1) * p.hpg, grp * p.hpg + (slice + 1) * kHeadsPer);
    for (int h = grp * p.hpg + slice * kHeadsPer; h < h_end; ++h) {
        const long long bh = (long long)bi * p.H + h;
        char *img = cp.image(bh, chunk);
        if (warp == 0) {
            // gamma in fp64, kept as hi + lo: differences of it stay exact to fp32 after strong decays
            const int i0 = 2 * lane;
            const long long at = bh * p.L + t0 + i0;
            const bool r0 = t0 + i0 < V, r1 = t0 + i0 + 1 < V;
            const float g0 = r0 ? clamp_log_decay(p.g[at]) : 0.f, g1 = r1 ? clamp_log_decay(p.g[at + 1]) : 0.f;
            const float b0 = r0 ? p.beta[at] : 0.f, b1 = r1 ? p.beta[at + 1] : 0.f;
            double sum = (double)g0 + (double)g1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            const double c0 = sum - (double)g1, c1 = sum, total = __shfl_sync(0xffffffffu, sum, 31);
            const double l0 = c0 * 1.4426950408889634, l1 = c1 * 1.4426950408889634;
            const float h0 = (float)l0, h1 = (float)l1;
            s_gam[i0] = make_float2(h0, (float)(l0 - (double)h0));
            s_gam[i0 + 1] = make_float2(h1, (float)(l1 - (double)h1));
            *(float2 *)(s_beta + i0) = make_float2(b0, b1);
            float *gates = (float *)img;
            *(float2 *)(gates + i0) = make_float2(expf((float)c0), expf((float)c1));
            *(float2 *)(gates + kChunk + i0) = make_float2(expf((float)(total - c0)), expf((float)(total - c1)));
            *(float2 *)(gates + 2 * kChunk + i0) = make_float2(b0, b1);
            *(float4 *)(gates + 3 * kChunk + 2 * i0) = make_float4(h0, (float)(l0 - (double)h0), h1, (float)(l1 - (double)h1));
        }
        if (h == grp * p.hpg + slice * kHeadsPer) {
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&bar_mma, 0));
            tc_fence_after();
        }
        if (__syncthreads_and(ok) == 0) break;
        const float2 gi = s_gam[i];
        const int last = i >> 4 | 1;      // warps of rows 0 .. 31 stop after two blocks of columns
        // 16 columns of D o (row of K K^T or Q K^T), zero where j >= i (keys) or j > i
        auto decayed = [&](int jb, float f, float (&r)[16]) {
            float a[16];
            __syncwarp();  // the lanes' rows end at different columns
            tmem_ld16(tmem_addr(tm, 32 * warp, (16 * jb) ^ (32 * flip)), a);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int j = 16 * jb + e;
                const float2 gj = s_gam[j];
                const float d = exp2_approx((gi.x - gj.x) + (gi.y - gj.y));
                r[e] = live && (j < i || (j == i && !keys)) ? f * d * a[e] : 0.f;
            }
        };
        if (keys)
            for (int jb = 0; jb <= (last | 1); ++jb) {
                float r[16];
                decayed(jb, 1.f, r);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *(float4 *)(s_e + i * kLdE + 16 * jb + 4 * e) = make_float4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
            }
        __syncthreads();
        // z[m][row] = beta_m y_m of this thread's row, over the tiles (which the products have read)
        float *z = (float *)(smem_raw + (kq - smem_u32(smem_raw))) + tid;
        const bool bwd = cp.w.states != nullptr;
        char *mat = img + kImgMat + (bwd && !keys ? 2 * kSquare : 0);
        auto store_block = [&](int jb, const float2 *y) {  // hi and lo parts, neighbouring rows on neighbouring addresses
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split2(y[4 * c + e].x, y[4 * c + e].y, hi[e], lo[e]);
                char *dst = mat + (bwd ? square_piece(i, 2 * jb + c) : run_piece(i + (keys ? 0 : kChunk), 2 * jb + c));
                *(uint4 *)dst = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *(uint4 *)(dst + (bwd ? kSquare : kPart)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        };
        // blocks above the diagonal that are stored: zeros
        for (int jb = (i >> 4) + 1; jb < 4; ++jb)
            if (bwd || !keys) {
                const float2 zero[8] = {};
                store_block(jb, zero);
            }
        if (bwd && !keys) {  // the backward takes A itself
            for (int jb = 0; jb <= last; ++jb) {
                float2 y[8];
                decayed(jb, p.scale, (float(&)[16])y);
                if (jb <= (i >> 4)) store_block(jb, y);
            }
        } else
        for (int jb = last; jb >= 0; --jb) {
            float2 y[8];
            if (keys) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 v = *(const float4 *)(s_e + i * kLdE + 16 * jb + 4 * e);
                    y[2 * e] = make_float2(-v.x, -v.y);
                    y[2 * e + 1] = make_float2(-v.z, -v.w);
                }
            } else {
                decayed(jb, p.scale, (float(&)[16])y);
            }
            const float *e0 = s_e + 16 * jb;
#pragma unroll 4
            for (int m = 16 * last + 15; m >= 16 * (jb + 1); --m) {
                const float zm = -z[m * kThreads];
                const float4 *w = (const float4 *)(e0 + m * kLdE);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 v = w[e];
                    y[2 * e] = ffma2(make_float2(v.x, v.y), make_float2(zm, zm), y[2 * e]);
                    y[2 * e + 1] = ffma2(make_float2(v.z, v.w), make_float2(zm, zm), y[2 * e + 1]);
                }
            }
            // the triangle of the block: from the last column, each solved one taken off those before it
            float *yy = (float *)y;
#pragma unroll
            for (int m = 15; m >= 0; --m) {
                const float zm = -s_beta[16 * jb + m] * yy[m];
                z[(16 * jb + m) * kThreads] = -zm;
                const float4 *w = (const float4 *)(e0 + (16 * jb + m) * kLdE);
#pragma unroll
                for (int e = 0; e < (m + 3) / 4; ++e) {
                    const float4 v = w[e];
                    yy[4 * e] = fmaf(zm, v.x, yy[4 * e]);
                    if (4 * e + 1 < m) yy[4 * e + 1] = fmaf(zm, v.y, yy[4 * e + 1]);
                    if (4 * e + 2 < m) yy[4 * e + 2] = fmaf(zm, v.z, yy[4 * e + 2]);
                    if (4 * e + 3 < m) yy[4 * e + 3] = fmaf(zm, v.w, yy[4 * e + 3]);
                }
            }
            if (jb <= (i >> 4)) store_block(jb, y);
        }
        __syncthreads();  // s_e and the gates may be written for the next head
    }
    if (tid == 0) {
        if (!ok) atomicExch(p.status + kStatusCode, (int)SSD_ERR_TIMEOUT);
        mbar_wait(&bar_load, 0);
        mbar_wait(&bar_mma, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tm, kAccCols);
}

}  // namespace

cudaError_t launch_chunk_prep(const ChunkParams &c, cudaStream_t s) {
    const DeltaParams &p = c.p;
    PrepMaps maps;
    cudaError_t e;
    if ((e = map_chunk_tokens(&maps.k, p.k, p.b, p.L, p.G, p.N, 32)) != cudaSuccess) return e;
    if ((e = map_chunk_tokens(&maps.q, p.q, p.b, p.L, p.G, p.N, 32)) != cudaSuccess) return e;
    const int bytes = 1024 + 32768;  // the tiles, then z
    const unsigned grid = (unsigned)c.n * ((p.hpg + kHeadsPer - 1) / kHeadsPer) * p.b * p.G;
    if ((e = cudaFuncSetAttribute(delta_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
    delta_prep_kernel<<<grid, kThreads, bytes, s>>>(c, maps);
    return cudaGetLastError();
}

}  // namespace delta
}  // namespace ssd
