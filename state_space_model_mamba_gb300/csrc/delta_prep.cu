// delta_prep.cu -- per-chunk matrices of the gated delta rule, all chunks in
// parallel (delta_chunk.cuh): K K^T and Q K^T of a key group once, on the tensor
// cores with K stacked on Q, then for every head of the group the decay-weighted
// triangles and the triangular inverse.
//
// With E = D o strict lower (K K^T) and A = scale D o lower (Q K^T),
//     Tt (I + diag(beta) E) = -E      and      At (I + diag(beta) E) = A,
// so both matrices are rows of one right-hand solve with a unit lower triangle, and
// every row is independent: thread i of 128 holds row i of [E; A] as it comes out of
// tensor memory and substitutes from its last column to its first in fp32
// registers,
//     y_j = r_j - sum_{m > j} y_m beta_m E_mj,
// reading diag(beta) E from shared memory as broadcasts.  Substitution stays accurate for
// repeated keys, where a power series of the triangle would lose every digit.
// What bounds it are the 5000 warp-wide multiply-adds of the two solves a head and
// chunk (rows 0 - 31 stop at column 31); a matrix instruction on the 16x16 pieces
// needs fp32 operands in three parts and was slower.
#include "delta_chunk.cuh"
#include "delta_mma.cuh"

namespace ssd {
namespace delta {
namespace {

using namespace tc;

constexpr int kThreads = 128;
constexpr int kHeadsPer = 4;          // heads of a group per block
constexpr int kLdG = 68;              // floats per column of diag(beta) E: 16-byte rows, four banks apart
constexpr uint32_t kAccCols = 64;

struct PrepMaps {
    CUtensorMap k, q;
};

// y_j = r_j - sum_{m > j} y_m g[j][m] for j = M-1 .. 0
template <int M>
__device__ __forceinline__ void solve_row(float (&y)[kChunk], const float *g) {
#pragma unroll
    for (int j = M - 2; j >= 0; --j) {
        float a0 = y[j], a1 = 0.f, a2 = 0.f, a3 = 0.f;
        // the newest value, y[j + 1], comes last
#pragma unroll
        for (int m4 = (M - 1) / 4; m4 >= (j + 1) / 4; --m4) {
            const float4 w = *(const float4 *)(g + j * kLdG + 4 * m4);
            if (4 * m4 + 3 > j) a3 = fmaf(-y[4 * m4 + 3], w.w, a3);
            if (4 * m4 + 2 > j) a2 = fmaf(-y[4 * m4 + 2], w.z, a2);
            if (4 * m4 + 1 > j) a1 = fmaf(-y[4 * m4 + 1], w.y, a1);
            if (4 * m4 > j) a0 = fmaf(-y[4 * m4], w.x, a0);
        }
        y[j] = (a0 + a1) + (a2 + a3);
    }
}

// Grid: one block per (b, group, slice of the group's heads, chunk).
__global__ void __launch_bounds__(kThreads) delta_prep_kernel(const ChunkParams cp, const __grid_constant__ PrepMaps maps) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar_load, bar_mma;
    __shared__ uint32_t s_tmem;
    __shared__ __align__(16) float s_g[kChunk * kLdG];
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
    if (tid == 0) {
        mbar_init(&bar_load, 1);
        mbar_init(&bar_mma, 1);
        mbar_fence_init();
        mbar_arrive_expect_tx(&bar_load, halves * 16384u);
        for (uint32_t kb = 0; kb < halves; ++kb) {
            tma_tile(kq + kb * 16384u, &maps.k, &bar_load, 64 * kb, grp, t0, bi);
            tma_tile(kq + kb * 16384u + 8192u, &maps.q, &bar_load, 64 * kb, grp, t0, bi);
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
                mma_bf16(tm, sdesc_kmajor(kq, ks, 16384), sdesc_kmajor(kq, ks, 16384), idesc_bf16(128, 64, false, false), ks > 0);
            mma_commit(&bar_mma);
        }
        __syncwarp();
    }
    const int i = tid & 63;               // the row's token
    const bool keys = tid < kChunk, live = t0 + i < V;  // rows of absent tokens may hold anything: made zero
    const int h_end = min((grp + 1) * p.hpg, grp * p.hpg + (slice + 1) * kHeadsPer);
    for (int h = grp * p.hpg + slice * kHeadsPer; h < h_end; ++h) {
        const long long bh = (long long)bi * p.H + h;
        char *img = cp.img + (bh * cp.n + chunk) * (long long)kImgBytes;
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
        }
        if (h == grp * p.hpg + slice * kHeadsPer) {
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&bar_mma, 0));
            tc_fence_after();
        }
        if (__syncthreads_and(ok) == 0) break;
        // rows of -E (the key rows) or A
        float y[kChunk];
        const float2 gi = s_gam[i];
        const float f = keys ? -1.f : p.scale;
        const bool low = warp & 1;        // rows 32 .. 63
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q < 2 || low) {
                float a[16];
                tmem_ld16(tmem_addr(tm, 32 * warp, 16 * q), a);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = 16 * q + e;
                    const float2 gj = s_gam[j];
                    const float d = exp2_approx((gi.x - gj.x) + (gi.y - gj.y));
                    y[j] = live && (j < i || (j == i && !keys)) ? f * d * a[e] : 0.f;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) y[16 * q + e] = 0.f;
            }
        }
        if (keys) {  // diag(beta) E by columns
            const float b = -s_beta[i];
#pragma unroll
            for (int j = 0; j < kChunk; ++j)
                if (j < 32 || low) s_g[j * kLdG + i] = b * y[j];
        }
        __syncthreads();
        if (low)
            solve_row<64>(y, s_g);
        else
            solve_row<32>(y, s_g);
        // hi and lo parts: 16-byte pieces, neighbouring rows on neighbouring addresses
        char *tri = img + kImgTri + (keys ? 0 : kTri);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if ((c >> 1) <= (i >> 4)) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split2(y[8 * c + 2 * e], y[8 * c + 2 * e + 1], hi[e], lo[e]);
                char *dst = tri + tri_piece(i, c);
                *(uint4 *)dst = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *(uint4 *)(dst + 2 * kTri) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        __syncthreads();  // s_g and the gates may be written for the next head
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
    if ((e = map_chunk_tokens(&maps.k, p.k, p.b, p.L, p.G, p.N)) != cudaSuccess) return e;
    if ((e = map_chunk_tokens(&maps.q, p.q, p.b, p.L, p.G, p.N)) != cudaSuccess) return e;
    const int bytes = 1024 + (p.N > 64 ? 32768 : 16384);
    const unsigned grid = (unsigned)c.n * ((p.hpg + kHeadsPer - 1) / kHeadsPer) * p.b * p.G;
    if ((e = cudaFuncSetAttribute(delta_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
    delta_prep_kernel<<<grid, kThreads, bytes, s>>>(c, maps);
    return cudaGetLastError();
}

}  // namespace delta
}  // namespace ssd
