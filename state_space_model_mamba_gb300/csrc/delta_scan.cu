// delta_scan.cu -- the serial pass of the chunked gated delta rule
// (delta_chunk.cuh): one block per (b, h, 64 columns of P) walks the chunks in
// order.  Per chunk, three products on the tensor cores, each waiting for the
// one before:
//   1.  [K; Q] S       M = 64 + 64 tokens, K index = N      -> K S and Q S
//   2.  [Tt; At] X     M = 64 + 64 tokens, K index = 64     -> Z = X0 + Tt X,  O = scale e^gamma Q S + At X
//   3.  K^T W          M = N, K index = 64 tokens           -> S' = e^gamma_C S + K^T W
// with X0 = V - e^gamma K S, X = beta X0 and W = beta e^(gamma_C - gamma) Z formed by
// the threads between them.  Stacking K on Q and Tt on At fills the 128 rows of the
// instruction, and the output's rows ride along with the chain's.
//
// Precision: q, k, v are exact in bf16; S, X, W, Tt, At are fp32 values fed as hi + lo
// bf16 parts (2^-17), the hi and lo parts of S and W side by side as one operand of
// twice the columns, so that the left operand is read once.  The state itself stays
// in fp32 registers (thread (n, half) holds row n, 32 columns) and is added to with
// rounding to nearest.
//
// What bounds it is the latency of the chain of three products and three passes of
// the threads.  A block needs 97 KB of shared memory with one set of K, Q tiles, so
// that two chains share an SM and hide in each other's waits; with few chains (one
// block per SM) a second set of K, Q tiles takes the load latency out of the chain.
#include <cuda.h>

#include "delta_chunk.cuh"
#include "delta_mma.cuh"

namespace ssd {
namespace delta {
namespace {

using namespace tc;

constexpr int kCompute = 256;              // eight warps: TMEM lane quarter w % 4, column half w / 4
constexpr int kScanThreads = kCompute + 64;  // and a warp that issues the products, one that issues the copies
constexpr uint32_t kAccCols = 128;

// shared memory from a 1024-byte aligned base
constexpr uint32_t kOffS = 0;              // S hi, S lo: [128 n][64] SW128; X (16 KB) and W (16 KB) in their place
constexpr uint32_t kOffX = 0, kOffW = 16384;
constexpr uint32_t kOffTri = 32768;        // [hi, lo][ks][16 row octets][2][128 bytes]: Tt rows, then At rows
constexpr uint32_t kOffV = 65536;          // [64 tokens][64] SW128
constexpr uint32_t kOffKQ = 73728;         // NB x [2 column halves][K 64 rows, Q 64 rows][64] SW128
constexpr uint32_t kKQBytes = 32768;

// 8 values as one 16-byte piece of row `row` of a hi and of a lo tile (SW128)
__device__ __forceinline__ void store_parts8(uint32_t hi_tile, uint32_t lo_tile, int row, int piece, const float2 *x) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(x[e].x, x[e].y, h[e], l[e]);
    st_shared_v4(hi_tile + sw128_chunk(row, piece), h[0], h[1], h[2], h[3]);
    st_shared_v4(lo_tile + sw128_chunk(row, piece), l[0], l[1], l[2], l[3]);
}

struct ScanMaps {
    CUtensorMap k, q, v;
};

template <int NB>
__global__ void __launch_bounds__(kScanThreads, NB == 1 ? 2 : 1)
    delta_scan_fwd(const ChunkParams cp, const __grid_constant__ ScanMaps maps) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar_kq[2], bar_tri, bar_v;               // copies have landed
    __shared__ uint64_t bar_s, bar_x, bar_w;                     // operands are written (8 warps each)
    __shared__ uint64_t bar_m[3];                                // products are done
    __shared__ uint32_t s_tmem;
    __shared__ int s_err;
    const DeltaParams &p = cp.p;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int nsl = (p.P + 63) / 64, slice = blockIdx.x % nsl, bh = blockIdx.x / nsl, bi = bh / p.H, h = bh % p.H;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int V = valid_tokens(p, bi), nv = (V + kChunk - 1) / kChunk, nks = (p.N + 15) / 16;
    const char *img0 = cp.img + (long long)bh * cp.n * (long long)kImgBytes;
    if (tid == 0) {
        mbar_init(&bar_kq[0], 1);
        mbar_init(&bar_kq[1], 1);
        mbar_init(&bar_tri, 1);
        mbar_init(&bar_v, 1);
        mbar_init(&bar_s, kCompute / 32);
        mbar_init(&bar_x, kCompute / 32);
        mbar_init(&bar_w, kCompute / 32);
        for (int i = 0; i < 3; ++i) mbar_init(&bar_m[i], 1);
        mbar_fence_init();
        s_err = 0;
    }
    if (warp == 0) tmem_alloc(&s_tmem, kAccCols);
    // the row octets of the triangles that no copy writes are zero
    for (int i = tid; i < 32768 / 16; i += kScanThreads) st_shared_v4(base + kOffTri + 16 * i, 0, 0, 0, 0);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;

    if (warp == kCompute / 32) {
        // ---- products
        const uint32_t i1 = idesc_bf16(128, 128, false, true), i2 = idesc_bf16(128, 64, false, true),
                       i3 = idesc_bf16(128, 128, true, true);
        const uint64_t dS = sdesc(base + kOffS, 16384, 1024), dX = sdesc(base + kOffX, 8192, 1024),
                       dW = sdesc(base + kOffW, 8192, 1024), dT = sdesc_tri(base + kOffTri);
        bool ok = true;
        int done = 0;
        for (int c = 0; c < nv; ++c) {
            const uint32_t ph = c & 1, kq = base + kOffKQ + (c % NB) * kKQBytes;
            const uint64_t dK = sdesc(kq, 16, 1024), dKt = sdesc(kq, 16384, 1024);
            ok = mbar_wait(&bar_kq[c % NB], (c / NB) & 1) && mbar_wait(&bar_s, ph);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    if (ks < nks) mma_bf16(tm, sdesc_add(dK, (ks >> 2) * 16384 + (ks & 3) * 32), sdesc_add(dS, ks * 2048), i1, ks > 0);
                mma_commit(&bar_m[0]);
            }
            ok = mbar_wait(&bar_tri, ph) && mbar_wait(&bar_x, ph);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int pass = 0; pass < 3; ++pass)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16(tm, sdesc_add(dT, (pass == 2 ? 16384 : 0) + ks * 4096),
                                 sdesc_add(dX, (pass == 1 ? 8192 : 0) + ks * 2048), i2, true);
                mma_commit(&bar_m[1]);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&bar_w, ph));
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16(tm, sdesc_add(dKt, ks * 2048), sdesc_add(dW, ks * 2048), i3, ks > 0);
                mma_commit(&bar_m[2]);
            }
            __syncwarp();
            done = c + 1;
        }
        if (!ok) s_err = 1;
        if (done) mbar_wait(&bar_m[2], (done - 1) & 1);  // every product has to complete before the block may end
    } else if (warp == kCompute / 32 + 1) {
        // ---- copies
        const int grp = h / p.hpg;
        const uint32_t halves = p.N > 64 ? 2u : 1u;
        int kq_issued = 0, tri_issued = 0, v_issued = 0;
        auto expect_kq = [&](int c) {
            if (lane == 0) mbar_arrive_expect_tx(&bar_kq[c % NB], halves * 16384u);
            kq_issued = c + 1;
        };
        auto load_rows = [&](int c, const CUtensorMap *m, uint32_t off) {
            if (lane == 0)
                for (uint32_t kb = 0; kb < halves; ++kb)
                    tma_tile(base + kOffKQ + (c % NB) * kKQBytes + kb * 16384u + off, m, &bar_kq[c % NB], 64 * kb, grp, c * kChunk, bi);
        };
        auto load_tri = [&](int c) {
            if (lane == 0) mbar_arrive_expect_tx(&bar_tri, 4 * kTri);
            __syncwarp();
            if (lane < 16) {
                const int part = lane >> 3, which = (lane >> 2) & 1, ks = lane & 3;
                bulk_load(base + kOffTri + part * 16384 + ks * 4096 + which * 2048 + 2 * ks * 256,
                          img0 + (long long)c * kImgBytes + kImgTri + (2 * part + which) * kTri + tri_run(ks), tri_run_bytes(ks),
                          &bar_tri);
            }
            tri_issued = c + 1;
        };
        auto load_v = [&](int c) {
            if (lane == 0) {
                mbar_arrive_expect_tx(&bar_v, 8192);
                tma_tile(base + kOffV, &maps.v, &bar_v, 64 * slice, h, c * kChunk, bi);
            }
            v_issued = c + 1;
        };
        for (int c = 0; c < NB && c < nv; ++c) {
            expect_kq(c);
            load_rows(c, &maps.k, 0);
            load_rows(c, &maps.q, 8192);
        }
        if (nv > 0) {
            load_v(0);
            load_tri(0);
        }
        bool ok = true;
        for (int c = 0; c + 1 < nv; ++c) {
            const uint32_t ph = c & 1;
            // V and, by the first product, Q have been read
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_x, ph)))) break;
            if (NB == 1) {
                expect_kq(c + 1);
                load_rows(c + 1, &maps.q, 8192);
            }
            load_v(c + 1);
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[1], ph)))) break;
            load_tri(c + 1);
            if (c + NB < nv) {
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[2], ph)))) break;
                if (NB > 1) {
                    expect_kq(c + NB);
                    load_rows(c + NB, &maps.q, 8192);
                }
                load_rows(c + NB, &maps.k, 0);
            }
        }
        if (!ok) s_err = 1;
        // every copy has to land before the block may end
        for (int c = max(0, kq_issued - NB); c < kq_issued; ++c) mbar_wait(&bar_kq[c % NB], (c / NB) & 1);
        if (tri_issued) mbar_wait(&bar_tri, (tri_issued - 1) & 1);
        if (v_issued) mbar_wait(&bar_v, (v_issued - 1) & 1);
    } else {
        const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;
        const bool keys = quarter < 2;       // rows 0 .. 63: K tokens, 64 .. 127: Q tokens
        const int i = row & 63;              // the row's token
        const uint32_t my = tmem_addr(tm, 32 * quarter, 32 * half);
        const float2 one = make_float2(1.f, 1.f);
        float2 S[16];
        {
            const float *src = p.init ? p.init + ((long long)bh * p.P + slice * 64 + 32 * half) * p.N + row : nullptr;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                ((float *)S)[j] = (src && row < p.N && slice * 64 + 32 * half + j < p.P) ? src[(long long)j * p.N] : 0.f;
        }
        bool ok = true;
        // S as an operand; before the last chunk, K rows of absent tokens are made zero
        auto publish_s = [&](int c) {
#pragma unroll
            for (int j = 0; j < 4; ++j) store_parts8(base + kOffS, base + kOffS + 16384, row, 4 * half + j, S + 4 * j);
            const int live = V - c * kChunk;
            if (live < kChunk) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bar_kq[c % NB], (c / NB) & 1));
                const uint32_t kq = base + kOffKQ + (c % NB) * kKQBytes;
                for (int x = tid; x < 2 * kChunk * 8; x += kCompute)
                    if (((x >> 3) & 63) >= live) st_shared_v4(kq + (x >> 9) * 16384u + (x & 511) * 16u, 0, 0, 0, 0);
            }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_s);
        };
        if (nv > 0) publish_s(0);
        for (int c = 0; c < nv && ok; ++c) {
            const uint32_t ph = c & 1;
            const float *gates = (const float *)(img0 + (long long)c * kImgBytes);
            const float eg = __ldg(gates + i), be = __ldg(gates + 2 * kChunk + i), et = __ldg(gates + kChunk + i);
            const float ec = __ldg(gates + kChunk - 1);
            const bool live = c * kChunk + i < V, partial = V - c * kChunk < kChunk;
            ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[0], ph) && mbar_wait(&bar_v, ph));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float2 a[8], b[8];
                tmem_ld16x2(my + 16 * j, my + 64 + 16 * j, (float *)a, (float *)b);
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = ffma2(b[e], one, a[e]);
                if (keys) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint4 w = ld_shared_v4(base + kOffV + sw128_chunk(i, 4 * half + 2 * j + u));
                        const uint32_t vv[4] = {w.x, w.y, w.z, w.w};
                        float2 xb[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2 x = ffma2(a[4 * u + e], make_float2(-eg, -eg), bf2_to_f2(vv[e]));
                            if (partial && !live) x = make_float2(0.f, 0.f);
                            a[4 * u + e] = x;
                            xb[e] = fmul2(x, make_float2(be, be));
                        }
                        store_parts8(base + kOffX, base + kOffX + 8192, i, 4 * half + 2 * j + u, xb);
                    }
                } else {
                    const float f = p.scale * eg;
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] = fmul2(a[e], make_float2(f, f));
                }
                tmem_st16(my + 16 * j, (const float *)a);
            }
            tmem_wait_st();
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_x);

            ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[1], ph));
            if (!ok) break;
            tc_fence_after();
            {
                float2 a[16];
                tmem_ld32(my, (float *)a);
                if (keys) {
                    const float f = be * et;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        a[e] = fmul2(a[e], make_float2(f, f));
                        if (partial && !live) a[e] = make_float2(0.f, 0.f);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) store_parts8(base + kOffW, base + kOffW + 8192, i, 4 * half + j, a + 4 * j);
                    fence_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_w);
                if (!keys) {
                    const int tok = c * kChunk + i;
                    bf16 *dst = (bf16 *)p.o + (((long long)bi * p.L + tok) * p.H + h) * p.P + slice * 64 + 32 * half;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (tok < p.L && slice * 64 + 32 * half + 8 * j < p.P)
                            *(uint4 *)(dst + 8 * j) =
                                live ? make_uint4(pack_bf2(a[4 * j].x, a[4 * j].y), pack_bf2(a[4 * j + 1].x, a[4 * j + 1].y),
                                                  pack_bf2(a[4 * j + 2].x, a[4 * j + 2].y), pack_bf2(a[4 * j + 3].x, a[4 * j + 3].y))
                                     : make_uint4(0, 0, 0, 0);
                }
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[2], ph));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float2 a[8], b[8];
                tmem_ld16x2(my + 16 * j, my + 64 + 16 * j, (float *)a, (float *)b);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    S[8 * j + e] = ffma2(S[8 * j + e], make_float2(ec, ec), ffma2(b[e], one, a[e]));
            }
            if (c + 1 < nv) publish_s(c + 1);
        }
        if (!ok) s_err = 1;
        // absent tokens past the last chunk
        for (int x = nv * kChunk * 8 + tid; x < p.L * 8; x += kCompute) {
            const int tok = x / 8, cc = x % 8;
            if (slice * 64 + cc * 8 < p.P)
                *(uint4 *)((bf16 *)p.o + (((long long)bi * p.L + tok) * p.H + h) * p.P + slice * 64 + cc * 8) = make_uint4(0, 0, 0, 0);
        }
        if (ok && p.final_state && row < p.N) {
            float *dst = p.final_state + ((long long)bh * p.P + slice * 64 + 32 * half) * p.N + row;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (slice * 64 + 32 * half + j < p.P) dst[(long long)j * p.N] = ((const float *)S)[j];
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && s_err) atomicExch(p.status + kStatusCode, (int)SSD_ERR_TIMEOUT);
    if (warp == 0) tmem_dealloc(tm, kAccCols);
}

}  // namespace

cudaError_t launch_chunk_forward(const ChunkParams &c, cudaStream_t s) {
    const DeltaParams &p = c.p;
    ScanMaps maps;
    cudaError_t e;
    if ((e = map_chunk_tokens(&maps.k, p.k, p.b, p.L, p.G, p.N)) != cudaSuccess) return e;
    if ((e = map_chunk_tokens(&maps.q, p.q, p.b, p.L, p.G, p.N)) != cudaSuccess) return e;
    if ((e = map_chunk_tokens(&maps.v, p.v, p.b, p.L, p.H, p.P)) != cudaSuccess) return e;
    const unsigned grid = (unsigned)(p.b * p.H * ((p.P + 63) / 64));
    const bool one_per_sm = grid <= 152;
    auto kernel = one_per_sm ? delta_scan_fwd<2> : delta_scan_fwd<1>;
    const int bytes = 1024 + (int)kOffKQ + (one_per_sm ? 2 : 1) * (int)kKQBytes;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
    kernel<<<grid, kScanThreads, bytes, s>>>(c, maps);
    return cudaGetLastError();
}

}  // namespace delta
}  // namespace ssd
