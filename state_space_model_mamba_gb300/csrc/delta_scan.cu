// delta_scan.cu -- the serial pass of the chunked gated delta rule
// (delta_chunk.cuh): one block per (b, h, W columns of P) walks the chunks in
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
// bf16 parts, the hi and lo parts of S and W side by side as one operand of twice the
// columns, so that the left operand is read once.  The state itself stays in fp32, in
// tensor memory beside the accumulators, and is added to by the threads with rounding to
// nearest.  What the forward adds to it, W, comes in a third part too (2^-25 of a value): two leave
// 2.5e-6 of the final state, nearly all of its error, where the other operands' second roundings leave 7e-7.
//
// What bounds it is the latency of the chain of three products and three passes of
// the threads.  The rows that carry the chain (K tokens) lie in two of the four lane
// quarters, which only half of the warps may read: 16 warps of 16 columns each hide one
// another's waits there.  A block needs 106 KB of shared memory with one set of K, Q tiles,
// so that two chains share an SM and hide in each other's waits; with few chains (one
// block per SM) a second set of K, Q tiles takes the load latency out of the chain, and
// narrower slices of P (W = 32 or 16 for 64) put more SMs on a chain, each with shorter
// passes and products: they repeat the loads of K and Q and waste part of the
// instruction, so they are taken only where every slice still has an SM of its own.
//
// Measured a chunk: 1.56 us in slices of 16 columns (1 x 131072 x 32 heads, 3.19 ms), 3.1 us
// for the backward's recompute, which also keeps S and Z (4 x 2048 x 24: 99 us); two blocks
// per SM, 8 ragged rows of up to 4096 tokens and 64 heads: 365 us (W in two parts: 341).  The third part in product
// steps of its own, on top of the second's accumulators, took 8 % of a narrow slice's chunk and 33 us of
// the ragged batch; columns of its own, 2 % and 23.  Tried and slower: threads that wait for a block's barrier instead of arriving at one the products' warp waits for.
#include <cuda.h>

#include "delta_chunk.cuh"
#include "delta_mma.cuh"

namespace ssd {
namespace delta {
namespace {

using namespace tc;

// 4 warps for every 16 columns of the slice (TMEM lane quarter w % 4, columns 16 (w / 4) .. + 15),
// a warp that issues the products, one that issues the copies
constexpr int compute_threads(int W) { return 8 * W; }
constexpr int scan_threads(int W) { return compute_threads(W) + 64; }
constexpr uint32_t kTmemCols = 256;

// shared memory from a 1024-byte aligned base
constexpr uint32_t kOffS = 0;              // S hi, S lo: [128 n][64] SW128 each; X and W in their place
constexpr uint32_t kOffX = 0, kOffW = 16384;
// narrow slices: hi and lo parts side by side in the rows of one tile
constexpr uint32_t kOffTri = 32768;        // [hi, lo][ks][16 row octets][2][128 bytes]: Tt rows, then At rows; or squares
constexpr uint32_t kOffV = 65536;          // [64 tokens][64] SW128
constexpr uint32_t kOffKQ = 73728;         // NB x [2 column halves][K 64 rows, Q 64 rows][64] SW128
constexpr uint32_t kKQBytes = 32768;

// 8 values as hi and lo parts of an operand tile with W columns: piece `piece` of row `row`; the lo
// tile lies `lo` bytes behind (W = 64), or the lo columns behind the hi ones
template <int W>
__device__ __forceinline__ void store_operand8(uint32_t tile, uint32_t lo, int row, int piece, const float2 *x) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(x[e].x, x[e].y, h[e], l[e]);
    const uint32_t at = tile + sw128_chunk(row, piece), al = W == 64 ? at + lo : tile + sw128_chunk(row, piece + W / 8);
    st_shared_v4(at, h[0], h[1], h[2], h[3]);
    st_shared_v4(al, l[0], l[1], l[2], l[3]);
}
// in three parts side by side, 64 columns a tile of 8 KB
template <int W>
__device__ __forceinline__ void store_operand8x3(uint32_t tile, int row, int piece, const float2 *x) {
    if constexpr (W == 64) {
        store_parts8(tile, tile + 8192, tile + 16384, row, piece, x);
    } else {
        uint32_t h[4], l[4], r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split3(x[e].x, x[e].y, h[e], l[e], r[e]);
        const uint32_t at = tile + sw128_chunk(row, piece), al = tile + sw128_chunk(row, piece + W / 8),
                       ar = W == 32 ? at + 8192 : tile + sw128_chunk(row, piece + W / 4);
        st_shared_v4(at, h[0], h[1], h[2], h[3]);
        st_shared_v4(al, l[0], l[1], l[2], l[3]);
        st_shared_v4(ar, r[0], r[1], r[2], r[3]);
    }
}
// 16 columns of row `row` of the state
template <int W>
__device__ __forceinline__ void publish_piece(uint32_t planes, int row, int group, const float2 *S) {
    store_operand8<W>(planes, 16384, row, 2 * group, S);
    store_operand8<W>(planes, 16384, row, 2 * group + 1, S + 4);
}
// fp32 rows of a state [P, N] in global memory: element (p, n) at p N + n, lanes along n
__device__ __forceinline__ void load_piece(float2 *S, const float *src, int row, int col, int P, int N) {
#pragma unroll
    for (int j = 0; j < 16; ++j) ((float *)S)[j] = (src && row < N && col + j < P) ? src[(long long)(col + j) * N + row] : 0.f;
}
__device__ __forceinline__ void store_piece(const float2 *S, float *dst, int row, int col, int P, int N) {
    if (!dst || row >= N) return;
#pragma unroll
    for (int j = 0; j < 16; ++j)
        if (col + j < P) dst[(long long)(col + j) * N + row] = ((const float *)S)[j];
}

struct ScanMaps {
    CUtensorMap k, q, v;
};

// The batch row whose length has this rank, longest first: blocks that wait for a place should be the short ones
// (8 rows of 1024 .. 4096 tokens, 64 heads, two blocks per SM: 341 us for 365 in the order given, W in two parts).
__device__ __forceinline__ int longest_first(const DeltaParams &p, int rank, int lane) {
    if (!p.valid_len || p.b > 64) return rank;
    const int v0 = lane < p.b ? valid_tokens(p, lane) : -1, v1 = lane + 32 < p.b ? valid_tokens(p, lane + 32) : -1;
    int r0 = 0, r1 = 0;
    for (int j = 0; j < p.b; ++j) {
        const int v = __shfl_sync(0xffffffffu, j < 32 ? v0 : v1, j & 31);
        r0 += v > v0 || (v == v0 && j < lane);
        r1 += v > v1 || (v == v1 && j < lane + 32);
    }
    const unsigned m0 = __ballot_sync(0xffffffffu, lane < p.b && r0 == rank),
                   m1 = __ballot_sync(0xffffffffu, lane + 32 < p.b && r1 == rank);
    return m0 ? __ffs(m0) - 1 : 31 + __ffs(m1);
}

template <int NB, bool BWD, int W>
__global__ void __launch_bounds__(scan_threads(W), NB == 1 ? 2 : 1)
    delta_scan_fwd(const ChunkParams cp, const __grid_constant__ ScanMaps maps) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar_kq[2], bar_tri, bar_v;               // copies have landed
    __shared__ uint64_t bar_s, bar_x, bar_w;                     // operands are written (by every compute warp)
    __shared__ uint64_t bar_m[3];                                // products are done
    __shared__ uint64_t bar_kept;                                // the backward's copy of S has been taken
    __shared__ uint32_t s_tmem;
    __shared__ int s_err;
    const DeltaParams &p = cp.p;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    constexpr int kCompute = compute_threads(W), kScanThreads = scan_threads(W);
    static_assert(!BWD || W == 64, "the backward's tiles have 64 columns");
    constexpr bool kBeside = NB > 1;
    // W's parts side by side, in the place of X lo too where they take 24 KB; the state behind their accumulators
    constexpr int kParts = BWD ? 2 : 3;
    constexpr uint32_t kAtW = kParts * W > 128 ? kOffX + 8192 : kOffW, kStateCol = kParts * W > 128 ? 192 : 128;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nsl = (p.P + W - 1) / W, slice = blockIdx.x % nsl, unit = blockIdx.x / nsl, h = unit % p.H;
    const int bi = NB == 1 && !BWD ? longest_first(p, unit / p.H, lane) : unit / p.H, bh = bi * p.H + h;
    const int V = valid_tokens(p, bi), nv = (V + kChunk - 1) / kChunk, nks = (p.N + 15) / 16;
    if (tid == 0) {
        mbar_init(&bar_kq[0], 1);
        mbar_init(&bar_kq[1], 1);
        mbar_init(&bar_tri, 1);
        mbar_init(&bar_v, 1);
        mbar_init(&bar_s, kCompute / 32);
        mbar_init(&bar_x, kCompute / 32);
        mbar_init(&bar_w, kCompute / 32);
        for (int i = 0; i < 3; ++i) mbar_init(&bar_m[i], 1);
        mbar_init(&bar_kept, 1);
        mbar_fence_init();
        s_err = 0;
    }
    if (warp == 0) {
        __syncwarp();  // lane 0 may come from a branch of its own
        tmem_alloc(&s_tmem, kTmemCols);
    }
    // the row octets of Tt that no copy writes are zero
    for (int i = tid; !BWD && i < 32768 / 16; i += kScanThreads) st_shared_v4(base + kOffTri + 16 * i, 0, 0, 0, 0);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;

    if (warp == kCompute / 32) {
        // ---- products
        const uint32_t i1 = idesc_bf16(128, 2 * W, false, true), i2 = idesc_bf16(128, W, false, true),
                       i3 = idesc_bf16(128, kParts * W, true, true);
        const uint64_t dS = sdesc(base + kOffS, 16384, 1024), dX = sdesc(base + kOffX, 8192, 1024),
                       dW = sdesc(base + kAtW, 8192, 1024), dT = BWD ? sdesc_plain(base + kOffTri, 1024, 128) : sdesc_plain(base + kOffTri, 128, 256);
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
                // Tt hi X hi and Tt hi X lo (side by side where the threads have the registers to add them), Tt lo X hi
#pragma unroll
                for (int pass = kBeside ? 1 : 0; pass < 3; ++pass)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint32_t at = BWD ? (pass == 2) * kSquare + ks * 2048 : (pass == 2) * 16384 + ks * 4096;
                        if (kBeside)
                            mma_bf16(tm, sdesc_add(dT, at), sdesc_add(dX, ks * 2048), pass == 2 ? i2 : i1, true);
                        else
                            mma_bf16(tm, sdesc_add(dT, at), sdesc_add(dX, (pass == 1) * 8192 + ks * 2048), i2, true);
                    }
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
        const int vcol = slice * W / 64 * 64;  // V comes in tiles of 64 columns
        int kq_issued = 0, tri_issued = 0, v_issued = 0;
        auto expect_kq = [&](int c) {
            if (lane == 0) mbar_arrive_expect_tx(&bar_kq[c % NB], halves * (BWD ? 8192u : 16384u));
            kq_issued = c + 1;
        };
        auto load_rows = [&](int c, const CUtensorMap *m, uint32_t off) {
            if (lane == 0 && !(BWD && off))  // the backward needs no outputs, hence no Q
                for (uint32_t kb = 0; kb < halves; ++kb)
                    tma_tile(base + kOffKQ + (c % NB) * kKQBytes + kb * 16384u + off, m, &bar_kq[c % NB], 64 * kb, grp, c * kChunk, bi);
        };
        auto load_tri = [&](int c) {
            const char *mat = cp.image(bh, c) + kImgMat;
            if (BWD) {  // both parts of Tt; its rows 64 .. 127, of which nothing is read, are what comes behind
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bar_tri, 2 * kSquare);
                    bulk_load(base + kOffTri, mat, 2 * kSquare, &bar_tri);
                }
            } else {
                if (lane == 0) mbar_arrive_expect_tx(&bar_tri, 2 * kPart);
                __syncwarp();
                const int part = lane >> 2, ks = lane & 3;
                if (lane < 8)
                    bulk_load(base + kOffTri + part * 16384 + ks * 4096 + ks * 512, mat + part * kPart + run_at(ks), run_bytes(ks), &bar_tri);
            }
            tri_issued = c + 1;
        };
        auto load_v = [&](int c) {
            if (lane == 0) {
                mbar_arrive_expect_tx(&bar_v, 8192);
                tma_tile(base + kOffV, &maps.v, &bar_v, vcol, h, c * kChunk, bi);
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
        auto keep = [&](int c) {  // S before chunk c, from the operand
            if (!BWD) return true;
            if (!__all_sync(0xffffffffu, mbar_wait(&bar_s, c & 1))) return false;
            if (lane == 0) {
                bulk_store(cp.w.states + ((long long)blockIdx.x * cp.n + c) * kStateTile, base + kOffS, kStateTile);
                bulk_commit();
                bulk_wait_read_all();
                mbar_arrive(&bar_kept);
            }
            __syncwarp();
            return true;
        };
        for (int c = 0; c + 1 < nv; ++c) {
            const uint32_t ph = c & 1;
            if (!(ok = keep(c))) break;
            if (lane == 0) {  // what the next chunk reads, into L2
                prefetch_bulk(cp.image(bh, c + 1), BWD ? kImgMat + 2 * kSquare : kImgFwd);
                if (c + NB < nv)
                    for (uint32_t kb = 0; kb < halves; ++kb) {
                        prefetch_tile(&maps.k, 64 * kb, grp, (c + NB) * kChunk, bi);
                        if (!BWD) prefetch_tile(&maps.q, 64 * kb, grp, (c + NB) * kChunk, bi);
                    }
                prefetch_tile(&maps.v, vcol, h, (c + 1) * kChunk, bi);
            }
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
        if (ok && nv > 0) ok = keep(nv - 1);
        if (BWD && lane == 0) bulk_wait_all();
        if (!ok) s_err = 1;
        // every copy has to land before the block may end
        for (int c = max(0, kq_issued - NB); c < kq_issued; ++c) mbar_wait(&bar_kq[c % NB], (c / NB) & 1);
        if (tri_issued) mbar_wait(&bar_tri, (tri_issued - 1) & 1);
        if (v_issued) mbar_wait(&bar_v, (v_issued - 1) & 1);
    } else {
        const int quarter = warp & 3, group = warp >> 2, row = 32 * quarter + lane;
        const bool keys = quarter < 2;       // rows 0 .. 63: K tokens, 64 .. 127: Q tokens
        const int i = row & 63, col = slice * W + 16 * group;
        const uint32_t ta = tmem_addr(tm, 32 * quarter, 16 * group), tb = ta + W, ts = ta + kStateCol;
        const float2 one = make_float2(1.f, 1.f);
        bool ok = true;
        // the state operand of chunk c is written; before the last chunk, K rows of absent tokens are made zero
        auto published = [&](int c) {
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
        {
            float2 S[8];
            load_piece(S, p.init ? p.init + (long long)bh * p.P * p.N : nullptr, row, col, p.P, p.N);
            __syncwarp();
            tmem_st16(ts, (const float *)S);
            if (nv > 0) publish_piece<W>(base + kOffS, row, group, S);
            tmem_wait_st();
            if (nv > 0) published(0);
        }
        float gn[4] = {0.f, 0.f, 0.f, 0.f};  // the next chunk's gates
        auto load_gates = [&](int c) {
            const float *gates = (const float *)cp.image(bh, c);
            gn[0] = __ldg(gates + i);
            gn[1] = __ldg(gates + 2 * kChunk + i);
            gn[2] = __ldg(gates + kChunk + i);
            gn[3] = __ldg(gates + kChunk - 1);
        };
        if (nv > 0) load_gates(0);
        for (int c = 0; c < nv && ok; ++c) {
            const uint32_t ph = c & 1;
            const float eg = gn[0], be = gn[1], et = gn[2], ec = gn[3];
            if (c + 1 < nv) load_gates(c + 1);
            const int tok = c * kChunk + i;
            const bool live = tok < V, partial = V - c * kChunk < kChunk;
            ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[0], ph) && mbar_wait(&bar_v, ph) && (!BWD || mbar_wait(&bar_kept, ph)));
            if (!ok) break;
            tc_fence_after();
            if (keys || !BWD) {
                float2 a[8], b[8];
                tmem_ld16x2(ta, tb, (float *)a, (float *)b);
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = ffma2(b[e], one, a[e]);
                if (keys) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint4 w = ld_shared_v4(base + kOffV + sw128_chunk(i, (col & 63) / 8 + u));
                        const uint32_t vv[4] = {w.x, w.y, w.z, w.w};
                        float2 xb[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2 x = ffma2(a[4 * u + e], make_float2(-eg, -eg), bf2_to_f2(vv[e]));
                            if (partial && !live) x = make_float2(0.f, 0.f);
                            a[4 * u + e] = x;
                            xb[e] = fmul2(x, make_float2(be, be));
                        }
                        store_operand8<W>(base + kOffX, 8192, i, 2 * group + u, xb);
                    }
                } else {
                    const float f = p.scale * eg;
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] = fmul2(a[e], make_float2(f, f));
                }
                __syncwarp();  // lanes of absent tokens may come from a branch of their own
                tmem_st16(ta, (const float *)a);
                if (kBeside) {
                    const float zero[16] = {};
                    tmem_st16(tb, zero);
                }
                tmem_wait_st();
                if (keys) fence_async_smem();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_x);

            ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[1], ph));
            if (!ok) break;
            tc_fence_after();
            {
                float2 a[8];
                if (kBeside) {
                    float2 b[8];
                    if (keys || !BWD) tmem_ld16x2(ta, tb, (float *)a, (float *)b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] = ffma2(b[e], one, a[e]);
                } else if (keys || !BWD) {
                    tmem_ld16(ta, (float *)a);
                }
                if (keys) {
                    const float f = be * et;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float2 w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (partial && !live) a[4 * u + e] = make_float2(0.f, 0.f);
                            w[e] = fmul2(a[4 * u + e], make_float2(f, f));
                        }
                        if (BWD)
                            store_operand8<W>(base + kOffW, 8192, i, 2 * group + u, w);
                        else
                            store_operand8x3<W>(base + kAtW, i, 2 * group + u, w);
                    }
                    fence_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_w);
                if (BWD && keys) {
                    char *tile = cp.w.errs + ((long long)blockIdx.x * cp.n + c) * kErrTile;
                    store_parts8(tile, 8192, i, 2 * group, a);
                    store_parts8(tile, 8192, i, 2 * group + 1, a + 4);
                }
                if (!BWD && !keys) {
                    bf16 *dst = (bf16 *)p.o + (((long long)bi * p.L + tok) * p.H + h) * p.P + col;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        if (tok < p.L && col + 8 * u < p.P) *(uint4 *)(dst + 8 * u) = live ? pack8(a + 4 * u) : make_uint4(0, 0, 0, 0);
                }
            }
            float2 S[8];
            if (kParts == 3 && kBeside) {
                __syncwarp();  // lanes store rows of their own
                tmem_ld16(ts, (float *)S);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[2], ph));
            if (!ok) break;
            tc_fence_after();
            {
                float2 a[8], b[8];
                if (kParts == 3) {
                    float2 r[8];
                    if (kBeside)
                        tmem_ld16x3(ta, tb, tb + W, (float *)a, (float *)b, (float *)r);
                    else
                        tmem_ld16x2(tb, tb + W, (float *)b, (float *)r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) b[e] = ffma2(r[e], one, b[e]);
                    if (!kBeside) tmem_ld16x2(ta, ts, (float *)a, (float *)S);  // fewer registers at once
                } else {
                    tmem_ld16x3(ta, tb, ts, (float *)a, (float *)b, (float *)S);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) S[e] = ffma2(S[e], make_float2(ec, ec), ffma2(b[e], one, a[e]));
                if (c + 1 < nv) publish_piece<W>(base + kOffS, row, group, S);
                __syncwarp();
                tmem_st16(ts, (const float *)S);
                tmem_wait_st();
                if (c + 1 < nv) published(c + 1);
            }
        }
        if (!ok) s_err = 1;
        // absent tokens past the last chunk
        for (long long x = (long long)nv * kChunk * (W / 8) + tid; !BWD && x < (long long)p.L * (W / 8); x += kCompute) {
            const int tok = (int)(x / (W / 8)), at = slice * W + 8 * (int)(x % (W / 8));
            if (at < p.P) *(uint4 *)((bf16 *)p.o + (((long long)bi * p.L + tok) * p.H + h) * p.P + at) = make_uint4(0, 0, 0, 0);
        }
        if (ok && p.final_state) {
            float2 S[8];
            __syncwarp();
            tmem_ld16(ts, (float *)S);
            store_piece(S, p.final_state + (long long)bh * p.P * p.N, row, col, p.P, p.N);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && s_err) atomicExch(p.status + kStatusCode, (int)SSD_ERR_TIMEOUT);
    if (warp == 0) {
        __syncwarp();  // lane 0 may come from a branch of its own
        tmem_dealloc(tm, kTmemCols);
    }
}

// ------------------------------------------------------------------ reverse
// The adjoint of the scan, chunks in reverse, with dS after the chunk in tensor memory as
// S is in the forward.  With D = s e^gamma dO,
//   0.  A^T dO                          (does not wait for the chain)
//   1.  K dS                            -> dU = A^T dO + e^(gamma_C - gamma) K dS
//   2.  Tt^T (beta dU)                  -> X = dU + Tt^T (beta dU),  dV = beta X
//   3.  K^T (-e^gamma dV) + Q^T D       -> dS = e^gamma_C dS + ...
// and, with what the forward kept, the sums that the gates' gradients are made of
// (delta_chunk.cuh).  D and e^gamma dV, which dS takes up, come in three parts as W does in the forward:
// two left 2.5e-6 of the initial state's gradient.
// One block per SM, with everything that a step reads in flight a step ahead: two sets of
// every tile, D in a place of its own, and Q^T D in an accumulator of its own, formed
// while the chain waits for its threads.  Two blocks per SM (single tiles, 56 registers a
// thread) took as long for two chains as this takes for two in turn.  The forward's S and Z
// read where they are used cost 2 us of a step's 5: Z comes by copy, S into registers, a step ahead.
// Measured: 4.4 us a chunk (4 x 2048 x 24 heads: 145 us, 136 with D and dV in two parts and dS kept in one; 80 chains of 128
// chunks: 564 us; 160 chains on 152 SMs by themselves are two waves, which is why the backward runs halves of the batch on two streams).
constexpr uint32_t kOffX2 = 0, kOffW2 = 8192;                    // in the state's place, as in the forward
constexpr uint32_t kRevTri = 32768, kRevDO = kRevTri + 2 * 32768, kRevD = kRevDO + 2 * 8192, kRevKQ = kRevD + 24576,
                   kRevZ = kRevKQ + 2 * kKQBytes, kRevBytes = kRevZ + kErrTile;
static_assert(kRevBytes + 2048 <= 232448, "shared memory of the reverse scan");
struct RevMaps {
    CUtensorMap k, q, d_o;
};

__global__ void __launch_bounds__(scan_threads(64), 1)
    delta_scan_rev(const ChunkParams cp, const __grid_constant__ RevMaps maps) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar_in[2], bar_z;                        // a step's copies have landed
    __shared__ uint64_t bar_s, bar_x, bar_w;                     // operands are written (by every compute warp)
    __shared__ uint64_t bar_m[3], bar_d;                         // products are done; D is written
    __shared__ uint64_t bar_kept;                                // the backward's copy of S has been taken
    __shared__ uint32_t s_tmem;
    __shared__ int s_err;
    const DeltaParams &p = cp.p;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    constexpr int kCompute = compute_threads(64);
    const int nsl = slices_of(p), slice = blockIdx.x % nsl, bh = blockIdx.x / nsl, bi = bh / p.H, h = bh % p.H;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int V = valid_tokens(p, bi), nv = (V + kChunk - 1) / kChunk, nks = (p.N + 15) / 16;
    if (tid == 0) {
        mbar_init(&bar_in[0], 1);
        mbar_init(&bar_in[1], 1);
        mbar_init(&bar_z, 1);
        mbar_init(&bar_s, kCompute / 32);
        mbar_init(&bar_x, kCompute / 32);
        mbar_init(&bar_w, kCompute / 32);
        for (int i = 0; i < 3; ++i) mbar_init(&bar_m[i], 1);
        mbar_init(&bar_kept, 1);
        mbar_init(&bar_d, kCompute / 64);
        mbar_fence_init();
        s_err = 0;
    }
    constexpr uint32_t kCols = 512, kAcc3 = 256;
    if (warp == 0) {
        __syncwarp();  // lane 0 may come from a branch of its own
        tmem_alloc(&s_tmem, kCols);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;

    if (warp == kCompute / 32) {
        // ---- products; step r is chunk nv - 1 - r
        const uint32_t i0 = idesc_bf16(128, 64, true, true), i1 = idesc_bf16(128, 128, false, true),
                       i2 = idesc_bf16(128, 128, true, true), i3 = idesc_bf16(128, 192, true, true);
        const uint64_t dS = sdesc(base + kOffS, 16384, 1024), dX = sdesc(base + kOffX2, 8192, 1024),
                       dW = sdesc(base + kOffW2, 8192, 1024), dD = sdesc(base + kRevD, 8192, 1024);
        bool ok = true;
        int done = 0;
        auto own = [&](int r) {  // A^T dO of step r
            ok = __all_sync(0xffffffffu, mbar_wait(&bar_in[r & 1], (r >> 1) & 1));
            if (!ok || lane) return;
            const uint64_t dA = sdesc_plain(base + kRevTri + (r & 1) * 32768 + 2 * kSquare, 128, 1024),
                           dO = sdesc(base + kRevDO + (r & 1) * 8192, 8192, 1024);
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16(tm + 128, sdesc_add(dA, part * kSquare + ks * 256), sdesc_add(dO, ks * 2048), i0, part > 0 || ks > 0);
        };
        for (int r = 0; r < nv; ++r) {
            const uint32_t ph = r & 1, kq = base + kRevKQ + (r & 1) * kKQBytes;
            const uint64_t dK = sdesc(kq, 16, 1024), dKt = sdesc(kq, 16384, 1024), dQt = sdesc(kq + 8192, 16384, 1024),
                           dT = sdesc_plain(base + kRevTri + (r & 1) * 32768, 128, 1024);
            ok = mbar_wait(&bar_in[r & 1], (r >> 1) & 1) && mbar_wait(&bar_s, ph);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            if (r == 0) own(0);  // after the rows of absent tokens have been made zero
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    if (ks < nks) mma_bf16(tm, sdesc_add(dK, (ks >> 2) * 16384 + (ks & 3) * 32), sdesc_add(dS, ks * 2048), i1, ks > 0);
                mma_commit(&bar_m[0]);
            }
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_d, ph)))) break;
            tc_fence_after();
            if (lane == 0)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16(tm + kAcc3, sdesc_add(dQt, ks * 2048), sdesc_add(dD, ks * 2048), i3, ks > 0);
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_x, ph)))) break;
            tc_fence_after();
            if (lane == 0) {
                // the products with (beta dU) lo in the columns behind
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16(tm, sdesc_add(dT, part * kSquare + ks * 256), sdesc_add(dX, ks * 2048), part ? i0 : i2, true);
                mma_commit(&bar_m[1]);
            }
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_w, ph)))) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16(tm + kAcc3, sdesc_add(dKt, ks * 2048), sdesc_add(dW, ks * 2048), i3, true);
                mma_commit(&bar_m[2]);
            }
            __syncwarp();
            done = r + 1;
            // the next step's A^T dO, whose accumulator the threads have read
            if (r + 1 < nv) own(r + 1);
            if (!ok) break;
        }
        if (!ok) s_err = 1;
        if (done) mbar_wait(&bar_m[2], (done - 1) & 1);  // every product has to complete before the block may end
    } else if (warp == kCompute / 32 + 1) {
        // ---- copies
        const int grp = h / p.hpg;
        const uint32_t halves = p.N > 64 ? 2u : 1u;
        int issued = 0, z_issued = 0;
        auto load_z = [&](int r) {
            if (lane == 0) {
                mbar_arrive_expect_tx(&bar_z, kErrTile);
                bulk_load(base + kRevZ, cp.w.errs + ((long long)blockIdx.x * cp.n + nv - 1 - r) * kErrTile, kErrTile, &bar_z);
            }
            z_issued = r + 1;
        };
        auto load = [&](int r) {
            if (lane == 0) {
                uint64_t *bar = &bar_in[r & 1];
                const int c = nv - 1 - r, t0 = c * kChunk;
                const uint32_t kq = base + kRevKQ + (r & 1) * kKQBytes;
                mbar_arrive_expect_tx(bar, halves * 16384u + 4 * kSquare + 8192);
                tma_tile(base + kRevDO + (r & 1) * 8192, &maps.d_o, bar, 64 * slice, h, t0, bi);
                bulk_load(base + kRevTri + (r & 1) * 32768, cp.image(bh, c) + kImgMat, 4 * kSquare, bar);
                for (uint32_t kb = 0; kb < halves; ++kb) {
                    tma_tile(kq + kb * 16384u, &maps.k, bar, 64 * kb, grp, t0, bi);
                    tma_tile(kq + kb * 16384u + 8192u, &maps.q, bar, 64 * kb, grp, t0, bi);
                }
            }
            issued = r + 1;
        };
        for (int r = 0; r < 2 && r < nv; ++r) load(r);
        if (nv > 0) load_z(0);
        bool ok = true;
        auto keep = [&](int r) {  // dS after the chunk, from the operand
            if (!__all_sync(0xffffffffu, mbar_wait(&bar_s, r & 1))) return false;
            if (lane == 0) {
                bulk_store(cp.w.dstates + ((long long)blockIdx.x * cp.n + nv - 1 - r) * kDStateTile, base + kOffS, kDStateTile);
                bulk_commit();
                bulk_wait_read_all();
                mbar_arrive(&bar_kept);
            }
            __syncwarp();
            return true;
        };
        for (int r = 0; r + 1 < nv; ++r) {
            const uint32_t ph = r & 1;
            if (!(ok = keep(r))) break;
            if (lane == 0) {  // what the next step reads, into L2
                const int c = nv - 2 - r;
                const long long at = (long long)blockIdx.x * cp.n + c;
                prefetch_bulk(cp.image(bh, c), kGates);
                if (r + 2 < nv) {
                    prefetch_bulk(cp.w.states + (at - 1) * kStateTile, kStateTile);
                    prefetch_bulk(cp.w.errs + (at - 1) * kErrTile, kErrTile);
                }
                if (r + 3 < nv) {
                    const int c3 = c - 2;
                    prefetch_bulk(cp.image(bh, c3), kImgBwd);
                    prefetch_tile(&maps.d_o, 64 * slice, h, c3 * kChunk, bi);
                    for (uint32_t kb = 0; kb < halves; ++kb) {
                        prefetch_tile(&maps.k, 64 * kb, grp, c3 * kChunk, bi);
                        prefetch_tile(&maps.q, 64 * kb, grp, c3 * kChunk, bi);
                    }
                }
            }
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_x, ph)))) break;
            load_z(r + 1);  // Z has been read
            if (r + 2 < nv) {  // the products of this step have read its tiles
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[2], ph)))) break;
                load(r + 2);
            }
        }
        if (ok && nv > 0) ok = keep(nv - 1);
        if (lane == 0) bulk_wait_all();
        if (!ok) s_err = 1;
        // every copy has to land before the block may end
        for (int r = max(0, issued - 2); r < issued; ++r) mbar_wait(&bar_in[r & 1], (r >> 1) & 1);
        if (z_issued) mbar_wait(&bar_z, (z_issued - 1) & 1);
    } else {
        const int quarter = warp & 3, group = warp >> 2, row = 32 * quarter + lane;
        const bool keys = quarter < 2;       // these threads form dU and X; the others D
        const int i = row & 63, col = slice * 64 + 16 * group;
        const uint32_t ta = tmem_addr(tm, 32 * quarter, 16 * group), tb = ta + 64, tu = ta + 128, ts = ta + 192, t3 = ta + kAcc3;
        const float2 one = make_float2(1.f, 1.f);
        bool ok = true;
        // the operand of step r is written; in the first, K, Q and dO rows of absent tokens are made zero
        auto published = [&](int r) {
            const int live = V - (nv - 1 - r) * kChunk;
            if (live < kChunk) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bar_in[r & 1], (r >> 1) & 1));
                const uint32_t kq = base + kRevKQ + (r & 1) * kKQBytes;
                for (int x = tid; x < 4 * kChunk * 8; x += kCompute)
                    if (((x >> 3) & 63) >= live) st_shared_v4(kq + x * 16u, 0, 0, 0, 0);
                for (int x = tid; x < kChunk * 8; x += kCompute)
                    if ((x >> 3) >= live) st_shared_v4(base + kRevDO + (r & 1) * 8192 + x * 16u, 0, 0, 0, 0);
            }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_s);
        };
        {
            float2 S[8];
            load_piece(S, p.d_final ? p.d_final + (long long)bh * p.P * p.N : nullptr, row, col, p.P, p.N);
            __syncwarp();
            tmem_st16(ts, (const float *)S);
            if (nv > 0) publish_piece<64>(base + kOffS, row, group, S);
            tmem_wait_st();
            if (nv > 0) published(0);
        }
        float gn[4] = {0.f, 0.f, 0.f, 0.f};  // the next step's gates
        auto load_gates = [&](int c) {
            if (c < 0) return;
            const float *gates = (const float *)cp.image(bh, c);
            gn[0] = __ldg(gates + i);
            gn[1] = __ldg(gates + 2 * kChunk + i);
            gn[2] = __ldg(gates + kChunk + i);
            gn[3] = __ldg(gates + kChunk - 1);
        };
        load_gates(nv - 1);
        uint4 sr[4];                         // and S before its chunk, this thread's 16 columns: hi, lo parts
        auto load_s = [&](int c) {
            if (c < 0) return;
            const char *tile = cp.w.states + ((long long)blockIdx.x * cp.n + c) * kStateTile;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const char *src = tile + sw128_chunk(row, 2 * group + u);
                sr[u] = __ldg((const uint4 *)src);
                sr[2 + u] = __ldg((const uint4 *)(src + 16384));
            }
        };
        load_s(nv - 1);
        for (int r = 0; r < nv && ok; ++r) {
            const int c = nv - 1 - r;
            const uint32_t ph = r & 1;
            const long long cc = (long long)blockIdx.x * cp.n + c;
            const float eg = gn[0], be = gn[1], et = gn[2], ec = gn[3];
            load_gates(c - 1);
            const int tok = c * kChunk + i;
            if (!keys) {  // D = scale e^gamma dO (bar_s: the rows of absent tokens are zero)
                ok = __all_sync(0xffffffffu, mbar_wait(&bar_in[r & 1], (r >> 1) & 1) && mbar_wait(&bar_s, ph));
                const float f = p.scale * eg;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint4 w = ld_shared_v4(base + kRevDO + (r & 1) * 8192 + sw128_chunk(i, 2 * group + x));
                    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
                    float2 d[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[e] = fmul2(bf2_to_f2(v[e]), make_float2(f, f));
                    store_parts8(base + kRevD, base + kRevD + 8192, base + kRevD + 16384, i, 2 * group + x, d);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_d);
            }
            // e^gamma_C <S, dS>, while the products run
            {
                float2 S[8];
                __syncwarp();  // lane 0 has announced the operand
                tmem_ld16(ts, (float *)S);
                float sum = 0.f;
#pragma unroll
                for (int u = 0; u < 4; ++u) sum = dot8(sr[u], S + 4 * (u & 1), sum);
                load_s(c - 1);
                if (row >= p.N) sum = 0.f;
#pragma unroll
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane == 0) cp.w.ss[cc * 16 + warp] = ec * sum;
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[0], ph) && mbar_wait(&bar_kept, ph) && mbar_wait(&bar_z, ph));
            if (!ok) break;
            tc_fence_after();
            float2 z[8];
            if (keys) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t at = base + kRevZ + sw128_chunk(i, 2 * group + u);
                    join8(ld_shared_v4(at), ld_shared_v4(at + 8192), z + 4 * u);
                }
            }
            float2 ww = make_float2(0.f, 0.f);
            if (keys) {
                float2 a[8], b[8], u[8];
                tmem_ld16x3(ta, tb, tu, (float *)a, (float *)b, (float *)u);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    a[e] = fmul2(ffma2(b[e], one, a[e]), make_float2(et, et));
                    ww = ffma2(z[e], a[e], ww);
                    a[e] = ffma2(u[e], one, a[e]);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float2 xb[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) xb[e] = fmul2(a[4 * x + e], make_float2(be, be));
                    store_parts8(base + kOffX2, base + kOffX2 + 8192, i, 2 * group + x, xb);
                }
                tmem_st16(ta, (const float *)a);
                const float zero[16] = {};
                tmem_st16(tb, zero);
                tmem_wait_st();
                fence_async_smem();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_x);

            ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[1], ph));
            if (!ok) break;
            tc_fence_after();
            if (keys) {
                float2 a[8], b[8];
                tmem_ld16x2(ta, tb, (float *)a, (float *)b);
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = ffma2(b[e], one, a[e]);
                const float f = -eg * be;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float2 w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = fmul2(a[4 * x + e], make_float2(f, f));
                    store_parts8(base + kOffW2, base + kOffW2 + 8192, base + kOffW2 + 16384, i, 2 * group + x, w);
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_w);
                char *lo_tile = cp.w.dv_lo + cc * kDvLoTile;
                bf16 *dst = (bf16 *)p.dv + (((long long)bi * p.L + tok) * p.H + h) * p.P + col;
                float2 zx = make_float2(0.f, 0.f);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        zx = ffma2(z[4 * x + e], a[4 * x + e], zx);
                        const float2 d = fmul2(a[4 * x + e], make_float2(be, be));
                        split2(d.x, d.y, hi[e], lo[e]);
                    }
                    *(uint4 *)(lo_tile + sw128_chunk(i, 2 * group + x)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    if (tok < p.L && col + 8 * x < p.P)
                        *(uint4 *)(dst + 8 * x) = tok < V ? make_uint4(hi[0], hi[1], hi[2], hi[3]) : make_uint4(0, 0, 0, 0);
                }
                const long long sat = ((long long)blockIdx.x * 4 + group) * cp.n * kChunk + tok;
                cp.w.zx[sat] = zx.x + zx.y;
                cp.w.ww[sat] = be * (ww.x + ww.y);
            } else {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_w);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[2], ph));
            if (!ok) break;
            tc_fence_after();
            {
                float2 a[8], b[8], S[8], rest[8];
                tmem_ld16x2(t3 + 64, t3 + 128, (float *)b, (float *)rest);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[e] = ffma2(rest[e], one, b[e]);
                tmem_ld16x2(t3, ts, (float *)a, (float *)S);
#pragma unroll
                for (int e = 0; e < 8; ++e) S[e] = ffma2(S[e], make_float2(ec, ec), ffma2(b[e], one, a[e]));
                if (r + 1 < nv) publish_piece<64>(base + kOffS, row, group, S);
                __syncwarp();
                tmem_st16(ts, (const float *)S);
                tmem_wait_st();
                if (r + 1 < nv) published(r + 1);
            }
        }
        if (!ok) s_err = 1;
        // absent tokens past the last chunk
        for (long long x = (long long)nv * kChunk * 8 + tid; x < (long long)p.L * 8; x += kCompute) {
            const int t = (int)(x / 8), cc = (int)(x % 8);
            if (slice * 64 + cc * 8 < p.P)
                *(uint4 *)((bf16 *)p.dv + (((long long)bi * p.L + t) * p.H + h) * p.P + slice * 64 + cc * 8) = make_uint4(0, 0, 0, 0);
        }
        if (ok && p.d_init) {
            float2 S[8];
            __syncwarp();
            tmem_ld16(ts, (float *)S);
            store_piece(S, p.d_init + (long long)bh * p.P * p.N, row, col, p.P, p.N);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && s_err) atomicExch(p.status + kStatusCode, (int)SSD_ERR_TIMEOUT);
    if (warp == 0) {
        __syncwarp();  // lane 0 may come from a branch of its own
        tmem_dealloc(tm, kCols);
    }
}

}  // namespace

cudaError_t launch_chunk_forward(const ChunkParams &c, cudaStream_t s) {
    const DeltaParams &p = c.p;
    ScanMaps maps;
    cudaError_t e;
    if ((e = map_chunk_tokens(&maps.k, p.k, p.b, p.L, p.G, p.N)) != cudaSuccess) return e;
    if ((e = same_tiles(&maps.q, maps.k, p.q)) != cudaSuccess) return e;
    if ((e = map_chunk_tokens(&maps.v, p.v, p.b, p.L, p.H, p.P)) != cudaSuccess) return e;
    // the narrowest slices that all have an SM of their own; two blocks of full slices per SM where not even those do
    const long long chains = (long long)p.b * p.H;
    int W = 64;
    if (!c.w.states)
        while (W > 16 && chains * ((p.P + W / 2 - 1) / (W / 2)) <= kSMs) W /= 2;
    const long long grid = chains * ((p.P + W - 1) / W);
    const int nb = grid <= kSMs ? 2 : 1, bytes = 1024 + (int)kOffKQ + nb * (int)kKQBytes;
    auto launch = [&](auto kernel, int threads) {
        if ((e = allow_shared((const void *)kernel, bytes)) != cudaSuccess) return e;
        kernel<<<(unsigned)grid, threads, bytes, s>>>(c, maps);
        return cudaGetLastError();
    };
    if (c.w.states) return nb == 2 ? launch(delta_scan_fwd<2, true, 64>, scan_threads(64)) : launch(delta_scan_fwd<1, true, 64>, scan_threads(64));
    if (nb == 1) return launch(delta_scan_fwd<1, false, 64>, scan_threads(64));
    if (W == 64) return launch(delta_scan_fwd<2, false, 64>, scan_threads(64));
    return W == 32 ? launch(delta_scan_fwd<2, false, 32>, scan_threads(32)) : launch(delta_scan_fwd<2, false, 16>, scan_threads(16));
}

cudaError_t launch_chunk_reverse(const ChunkParams &c, cudaStream_t s) {
    const DeltaParams &p = c.p;
    RevMaps maps;
    cudaError_t e;
    if ((e = map_chunk_tokens(&maps.k, p.k, p.b, p.L, p.G, p.N)) != cudaSuccess) return e;
    if ((e = same_tiles(&maps.q, maps.k, p.q)) != cudaSuccess) return e;
    if ((e = map_chunk_tokens(&maps.d_o, p.d_o, p.b, p.L, p.H, p.P)) != cudaSuccess) return e;
    const unsigned grid = (unsigned)(p.b * p.H * slices_of(p));
    const int bytes = 1024 + (int)kRevBytes;
    if ((e = allow_shared((const void *)delta_scan_rev, bytes)) != cudaSuccess) return e;
    delta_scan_rev<<<grid, scan_threads(64), bytes, s>>>(c, maps);
    return cudaGetLastError();
}

}  // namespace delta
}  // namespace ssd
