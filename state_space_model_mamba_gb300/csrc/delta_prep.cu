// delta_prep.cu -- per-chunk matrices of the gated delta rule, all chunks in
// parallel (delta_chunk.cuh): K K^T and Q K^T of a key group once, on the tensor
// cores with K stacked on Q, then for every head of the group the decay-weighted
// triangles and the triangular inverse.
//
// With E = D o strict lower (K K^T) and A = scale D o lower (Q K^T),
//     Tt (I + diag(beta) E) = -E      and      At (I + diag(beta) E) = A,
// so both matrices are rows of one right-hand solve with a unit lower triangle, and
// every row is independent: thread i of 128 holds row i of [E; A] as it comes out of
// tensor memory and substitutes from its last column to its first,
//     y_j = r_j - sum_{m > j} (beta_m y_m) E_mj,
// 16 columns at a time: the 16 x 16 triangle in fp32 registers, its columns' share of all
// columns before them on the tensor cores (beta y and E as hi + lo bf16 parts), which add it
// to the right-hand sides where these lie in tensor memory.  Substitution stays accurate for repeated keys, where a
// power series of the triangle would lose every digit.
// What bounds it is the chain of those steps, each behind a barrier, and 7000 warp
// instructions a head and chunk (8200 before decays and triangles went in pairs, at 40 % of
// the issue slots and 11 % more time) with six blocks on an SM
// (tensor memory would hold eight, shared memory six), four where several heads share a
// block's products.  With the shares in fp32 registers too a head took twice the
// instructions; the whole substitution unrolled waited for instructions half of the time.
// Which warps get the long rows changes from block to block.
// Measured: 12.3 ns a head and chunk (1 x 131072 x 32 heads: 806 us; 4 x 2048 x 24: 47.5 us, 2.7 TB/s).
#include "delta_chunk.cuh"
#include "delta_mma.cuh"

namespace ssd {
namespace delta {
namespace {

using namespace tc;

constexpr int kThreads = 128;
constexpr int kHeadsPer = 6;          // heads of a group per block at most
constexpr int kLdD = 16;              // floats per row of E's diagonal blocks
// over the tiles, once the products have read them: E hi, E lo [64][64] SW128, beta y hi, lo [2 column octets][16 row octets][128]
constexpr uint32_t kOffE = 0, kOffZ = 16384, kOffSmall = 32768;
struct Small {
    float d[kChunk * kLdD];
    float gam[2][kChunk]; // gamma log2(e): hi, lo
    float beta[kChunk];
    uint64_t load, mma, step;
    uint32_t tmem;
};
constexpr uint32_t kBytes = kOffSmall + sizeof(Small);
static_assert(6 * (kBytes + 1024) <= 233472, "six blocks per SM");

struct PrepMaps {
    CUtensorMap k, q;
};

// a sum kept as hi + lo, and its product with log2(e)
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    const float s = a.hi + b.hi, t = s - a.hi, e = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo);
    return Pair{s + e, e - ((s + e) - s)};
}
__device__ __forceinline__ Pair times_log2e(Pair a) {
    constexpr float c = 1.44269504f, c_lo = (float)(1.4426950408889634 - (double)1.44269504f);
    const float p = a.hi * c, e = fmaf(a.hi, c, -p) + fmaf(a.hi, c_lo, a.lo * c);
    return Pair{p + e, e - ((p + e) - p)};
}

// Grid: one block per (b, group, `per` of the group's heads, chunk).
// ALONE: per is 1, and the head's right-hand sides take the products' place in tensor memory.
template <bool ALONE>
__global__ void __launch_bounds__(kThreads, ALONE ? 6 : 4) delta_prep_kernel(const ChunkParams cp, const __grid_constant__ PrepMaps maps, int per,
                                                                                        int status_rows) {
    // no static shared memory and no slack for alignment: the window starts on a 1024-byte boundary
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Small &sm = *(Small *)(smem_raw + kOffSmall);
    uint64_t &bar_load = sm.load, &bar_mma = sm.mma, &bar_step = sm.step;
    float *const s_d = sm.d, *const s_beta = sm.beta;
    float *const s_gh = sm.gam[0], *const s_gl = sm.gam[1];
    // the products, then the right-hand sides
    constexpr uint32_t kAccCols = ALONE ? 64 : 128, kRhs = ALONE ? 0 : 64;
    const DeltaParams &p = cp.p;
    const int slices = (p.hpg + per - 1) / per;
    const int chunk = blockIdx.x % cp.n, slice = blockIdx.x / cp.n % slices;
    const int bg = blockIdx.x / cp.n / slices, bi = bg / p.G, grp = bg % p.G;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0 && status_rows > 0) write_status(p, status_rows);
    const int V = valid_tokens(p, bi), t0 = chunk * kChunk;
    if (t0 >= V) return;
    const uint32_t kq = smem_u32(smem_raw);
    const uint32_t halves = p.N > 64 ? 2u : 1u;
    // where rows lie changes from block to block, so that the long solves do not always land on the same schedulers
    const uint32_t hash = blockIdx.x * 0x9E3779B1u;
    const int flip = hash >> 31;                          // tokens 32 .. 63 in rows (and columns) 0 .. 31
    const uint32_t k_off = (hash >> 30 & 1) * 8192u;      // K rows behind the Q rows
    if (tid == 0) {
        mbar_init(&bar_load, 1);
        mbar_init(&bar_mma, 1);
        mbar_init(&bar_step, 1);
        mbar_fence_init();
        mbar_arrive_expect_tx(&bar_load, halves * 16384u);
        for (uint32_t kb = 0; kb < halves; ++kb)
            for (int x = 0; x < 2; ++x) {
                const int tok = t0 + 32 * (x ^ flip);
                tma_tile(kq + kb * 16384u + k_off + 4096u * x, &maps.k, &bar_load, 64 * kb, grp, tok, bi);
                tma_tile(kq + kb * 16384u + (k_off ^ 8192u) + 4096u * x, &maps.q, &bar_load, 64 * kb, grp, tok, bi);
            }
    }
    if (warp == 0) {
        __syncwarp();  // lane 0 may come from a branch of its own
        tmem_alloc(&sm.tmem, kAccCols);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;
    bool ok = !(kq & 1023u);
    if (warp == 0) {
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&bar_load, 0));
        if (ok && lane == 0) {
            const int nks = (p.N + 15) / 16;
            for (int ks = 0; ks < nks; ++ks)
                mma_bf16(tm, sdesc_kmajor(kq, ks, 16384), sdesc_kmajor(kq + k_off, ks, 16384), idesc_bf16(128, 64, false, false), ks > 0);
            mma_commit(&bar_mma);
        }
        __syncwarp();
    }
    int steps = 0;                        // groups of shares issued
    const int i = (tid & 63) ^ (32 * flip);  // the row's token
    const bool keys = (tid < kChunk) == (k_off == 0), live = t0 + i < V;  // rows of absent tokens may hold anything: made zero
    const int h_end = min((grp + 1) * p.hpg, grp * p.hpg + (slice + 1) * per);
    float2 next_g = make_float2(0.f, 0.f), next_b = next_g;  // the next head's gates of tokens 2 lane, 2 lane + 1
    auto fetch = [&](int h) {
        const long long at = ((long long)bi * p.H + h) * p.L + t0 + 2 * lane;
        const bool r0 = t0 + 2 * lane < V, r1 = t0 + 2 * lane + 1 < V;
        next_g = make_float2(r0 ? clamp_log_decay(p.g[at]) : 0.f, r1 ? clamp_log_decay(p.g[at + 1]) : 0.f);
        next_b = make_float2(r0 ? p.beta[at] : 0.f, r1 ? p.beta[at + 1] : 0.f);
    };
    if (warp == 0) fetch(grp * p.hpg + slice * per);
    for (int h = grp * p.hpg + slice * per; h < h_end; ++h) {
        const long long bh = (long long)bi * p.H + h;
        char *img = cp.image(bh, chunk);
        if (warp == 0) {
            // gamma as hi + lo: differences of it stay exact to fp32 after strong decays
            const int i0 = 2 * lane;
            const float g1 = next_g.y;
            const float2 beta = next_b;
            Pair sum = add(Pair{next_g.x, 0.f}, Pair{g1, 0.f});
            if (h + 1 < h_end) fetch(h + 1);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const Pair up{__shfl_up_sync(0xffffffffu, sum.hi, o), __shfl_up_sync(0xffffffffu, sum.lo, o)};
                if (lane >= o) sum = add(up, sum);
            }
            const Pair c0 = add(sum, Pair{-g1, 0.f}), c1 = sum;
            const Pair total{__shfl_sync(0xffffffffu, sum.hi, 31), __shfl_sync(0xffffffffu, sum.lo, 31)};
            const Pair l0 = times_log2e(c0), l1 = times_log2e(c1);
            *(float2 *)(s_gh + i0) = make_float2(l0.hi, l1.hi);
            *(float2 *)(s_gl + i0) = make_float2(l0.lo, l1.lo);
            *(float2 *)(s_beta + i0) = beta;
            float *gates = (float *)img;
            *(float2 *)(gates + i0) = make_float2(expf(c0.hi), expf(c1.hi));
            *(float2 *)(gates + kChunk + i0) = make_float2(expf((total.hi - c0.hi) + (total.lo - c0.lo)), expf((total.hi - c1.hi) + (total.lo - c1.lo)));
            *(float2 *)(gates + 2 * kChunk + i0) = beta;
            *(float4 *)(gates + 3 * kChunk + 2 * i0) = make_float4(l0.hi, l0.lo, l1.hi, l1.lo);
        }
        if (h == grp * p.hpg + slice * per) {
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&bar_mma, 0));
            tc_fence_after();
        }
        if (__syncthreads_and(ok) == 0) break;
        const float gh = s_gh[i], gl = s_gl[i];
        const int last = i >> 4 | 1;      // warps of rows 0 .. 31 have two blocks of columns
        const int limit = live ? (keys ? i : i + 1) : 0;  // the row's columns that count
        const bool all = t0 + kChunk <= V;
        // 16 columns of f D o (row of K K^T or Q K^T), zero from column `limit` on
        auto decayed = [&](int jb, float f, float2 (&r)[8]) {
            __syncwarp();  // the lanes' rows end at different columns
            tmem_ld16(tmem_addr(tm, 32 * warp, (16 * jb) ^ (32 * flip)), (float *)r);
            const bool whole = all && 16 * jb + 15 < (i & ~31);  // the same for the warp
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 h = *(const float4 *)(s_gh + 16 * jb + 4 * c), l = *(const float4 *)(s_gl + 16 * jb + 4 * c);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float2 minus = make_float2(-1.f, -1.f), one = make_float2(1.f, 1.f);
                    const float2 x = ffma2(u ? make_float2(h.z, h.w) : make_float2(h.x, h.y), minus, make_float2(gh, gh)),
                                 y = ffma2(u ? make_float2(l.z, l.w) : make_float2(l.x, l.y), minus, make_float2(gl, gl)),
                                 d = ffma2(x, one, y);
                    float2 v = fmul2(fmul2(r[2 * c + u], make_float2(f, f)), make_float2(exp2_approx(d.x), exp2_approx(d.y)));
                    if (!whole) {
                        const int j = 16 * jb + 4 * c + 2 * u;
                        v.x = j < limit ? v.x : 0.f;
                        v.y = j + 1 < limit ? v.y : 0.f;
                    }
                    r[2 * c + u] = v;
                }
            }
        };
        const bool bwd = cp.w.states != nullptr, solves = keys || !bwd;
        // where columns 16 jb of a right-hand side lie: in place of the products they come from, or behind them
        auto rhs = [&](int jb) { return tm + kRhs + (uint32_t)(ALONE ? (16 * jb) ^ (32 * flip) : 16 * jb); };
        if (solves)
            for (int jb = 0; jb <= last; ++jb) {
                float2 r[8];
                decayed(jb, keys ? -1.f : p.scale, r);
                __syncwarp();
                tmem_st16(tmem_addr(rhs(jb), 32 * warp, 0), (const float *)r);
                if (keys) {  // -E
                    store_parts8(kq + kOffE, kq + kOffE + 8192, i, 2 * jb, r);
                    store_parts8(kq + kOffE, kq + kOffE + 8192, i, 2 * jb + 1, r + 4);
                    if (jb == i >> 4) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *(float4 *)(s_d + i * kLdD + 4 * e) = make_float4(r[2 * e].x, r[2 * e].y, r[2 * e + 1].x, r[2 * e + 1].y);
                    }
                }
            }
        __syncwarp();
        tmem_wait_st();
        tc_fence_before();
        __syncthreads();
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
        if (bwd && !keys)                 // the backward takes A itself
            for (int jb = 0; jb <= last; ++jb) {
                float2 y[8];
                decayed(jb, p.scale, y);
                if (jb <= (i >> 4)) store_block(jb, y);
            }
        const uint32_t zt = kq + kOffZ + (tid >> 3) * 128 + (tid & 7) * 16;
        for (int jb = 3; jb >= 0; --jb) {
            float2 y[8];
            if (solves && jb <= last) {
                __syncwarp();
                tmem_ld16(tmem_addr(rhs(jb), 32 * warp, 0), (float *)y);
                // the triangle of the block: from the last column, each solved one taken off those before it
                // (pairs of columns; the triangle holds zeros from its diagonal on)
                const float *e0 = s_d + 16 * jb * kLdD;
                float2 z[8];
#pragma unroll
                for (int m = 15; m >= 0; --m) {
                    const float zm = s_beta[16 * jb + m] * (m & 1 ? y[m / 2].y : y[m / 2].x);
                    (m & 1 ? z[m / 2].y : z[m / 2].x) = zm;
                    const float4 *w = (const float4 *)(e0 + m * kLdD);
#pragma unroll
                    for (int e = 0; e < (m + 3) / 4; ++e) {
                        const float4 v = w[e];
                        y[2 * e] = ffma2(make_float2(zm, zm), make_float2(v.x, v.y), y[2 * e]);
                        if (4 * e + 2 < m) y[2 * e + 1] = ffma2(make_float2(zm, zm), make_float2(v.z, v.w), y[2 * e + 1]);
                    }
                }
                if (jb > 0) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) split2(z[4 * c + e].x, z[4 * c + e].y, hi[e], lo[e]);
                        st_shared_v4(zt + c * 2048, hi[0], hi[1], hi[2], hi[3]);
                        st_shared_v4(zt + 4096 + c * 2048, lo[0], lo[1], lo[2], lo[3]);
                    }
                }
            } else if (jb > 0) {
#pragma unroll
                for (int c = 0; c < 4; ++c) st_shared_v4(zt + c * 2048, 0, 0, 0, 0);
            }
            if (jb > 0) {  // the block's share of the columns before it: K = 16, N = 16 jb
                fence_async_smem();
                tc_fence_before();
                __syncthreads();
                if (tid == 0) {
                    tc_fence_after();
                    const uint64_t dZ = sdesc_plain(kq + kOffZ, 2048, 128), dE = sdesc_mnmajor(kq + kOffE, jb, 8192);
                    // columns 0 .. 31, then those behind: apart, where the products lie in the other order
                    for (int c = 0; c < 16 * jb; c += 32) {
                        const uint32_t d = rhs(c / 16), idesc = idesc_bf16(128, min(32, 16 * jb - c), false, true);
                        mma_bf16(d, dZ, sdesc_add(dE, 2 * c), idesc, true);
                        mma_bf16(d, dZ, sdesc_add(dE, 8192 + 2 * c), idesc, true);
                        mma_bf16(d, sdesc_add(dZ, 4096), sdesc_add(dE, 2 * c), idesc, true);
                    }
                    mma_commit(&bar_step);
                }
            }
            if (solves && jb <= (i >> 4)) store_block(jb, y);
            if (jb > 0) {
                __syncwarp();
                ok = __all_sync(0xffffffffu, ok && mbar_wait(&bar_step, steps & 1));
                ++steps;
                tc_fence_after();
            }
        }
        tc_fence_before();
        __syncthreads();  // E and the gates may be written for the next head
    }
    if (tid == 0) {
        if (!ok) atomicExch(p.status + kStatusCode, (int)SSD_ERR_TIMEOUT);
        mbar_wait(&bar_load, 0);
        mbar_wait(&bar_mma, 0);
        if (steps) mbar_wait(&bar_step, (steps - 1) & 1);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) {
        __syncwarp();  // lane 0 may come from a branch of its own
        tmem_dealloc(tm, kAccCols);
    }
}

}  // namespace

cudaError_t launch_chunk_prep(const ChunkParams &c, int status_rows, cudaStream_t s) {
    const DeltaParams &p = c.p;
    PrepMaps maps;
    cudaError_t e;
    if ((e = map_chunk_tokens(&maps.k, p.k, p.b, p.L, p.G, p.N, 32)) != cudaSuccess) return e;
    if ((e = same_tiles(&maps.q, maps.k, p.q)) != cudaSuccess) return e;
    // A block's heads share the two products: equal shares of a group, up to 6 heads (80 heads in 16 groups: one block of
    // 5 took 275 us where blocks of 4 and 1 took 292; 64 heads in 8 groups: 281 us in fours, 284 in eights,
    // 329 alone; all before the arithmetic went in pairs), but one by one while all of them have a place at once.
    const int shares = (p.hpg + kHeadsPer - 1) / kHeadsPer;
    const int per = (long long)c.n * p.b * p.H <= 6 * kSMs ? 1 : (p.hpg + shares - 1) / shares;
    const unsigned grid = (unsigned)c.n * ((p.hpg + per - 1) / per) * p.b * p.G;
    auto launch = [&](auto kernel) {
        if ((e = allow_shared((const void *)kernel, (int)kBytes)) != cudaSuccess) return e;
        kernel<<<grid, kThreads, kBytes, s>>>(c, maps, per, status_rows);
        return cudaGetLastError();
    };
    return per == 1 ? launch(delta_prep_kernel<true>) : launch(delta_prep_kernel<false>);
}

}  // namespace delta
}  // namespace ssd
