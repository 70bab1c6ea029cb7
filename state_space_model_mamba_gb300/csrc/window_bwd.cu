// window_bwd.cu -- window attention, backward, on tcgen05.
//
// With x = scale q.k, p = exp(x - lse), D = do.o and dx = p (do.v - D):
//     dq = scale sum_s dx k,   dk = scale sum_t dx q,   dv = sum_t p do.
// Two kernels make the pairs' p and dx from the inputs again, one per query tile for dq and one per key
// tile for dk and dv, seven products of tiles where one kernel would need five and sums of dq through
// memory in no fixed order (or one that blocks wait for); here every sum has one order.
//
// window_dq_kernel: a block takes query tiles of 128 rows (window_tile.cuh) and streams key tiles of 96:
// S = Q K^T, dP = dO V^T in two buffers each of tensor memory; two groups of four warps, a thread per row and 48
// columns, write dx in bf16 over S, the A operand of dQ += dX K.
//
// window_dkv_kernel: a block takes 128 keys of a group and streams the query rows that see them, 64 at
// a time (tokens times heads, so the heads of the group add up in the accumulators): S^T = K Q^T, dP^T = V dO^T; a thread per
// key and 32 rows writes p over S^T and dx over dP^T, the A operands of dV += P^T dO and dK += dX^T Q.
// Keys that are sinks are seen by every later token: what lies behind their window is cut into segments, items
// of their own whose sums go to the workspace, and a last kernel adds those in order.
//
// An instruction's issue and a wait cost their thread some 55 and 100 cycles, so every kind of product has a thread of
// its own.  p and dx are rounded to bf16 where they enter a product (2^-8 of each at most); sums are fp32.
#include "window_tile.cuh"

namespace ssd {
namespace window {
namespace {

using delta::exp2_approx;
using delta::tma_tile;
using tc::ffma2;
using tc::fmul2;
using tc::tmem_addr;

// ------------------------------------------------------------------ D = do . o
// 8 lanes a row of P (8 columns each in turn), rows in the order of the tensors, 4 a thread whose loads go ahead of the sums
// (one row a thread, numbered in 64 bits: the 130M layer's backward 175 us, so 172; 8 padded rows of up to 4096 tokens of 64 heads of 64
// 1502 and 1474).  The API takes up to 3.2e9 rows, which 32 bits number.
constexpr int kDeltaRows = 4;
template <int KB>
__global__ void __launch_bounds__(256) window_delta_kernel(WindowParams p, uint32_t rows) {
    const uint32_t first = blockIdx.x * (32u * kDeltaRows) + (threadIdx.x >> 3);
    const int lane = threadIdx.x & 7;
    if (blockIdx.x == 0) write_status(p);
    uint4 a[kDeltaRows][KB], b[kDeltaRows][KB];
#pragma unroll
    for (int i = 0; i < kDeltaRows; ++i)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int c = 8 * lane + 64 * kb;
            a[i][kb] = b[i][kb] = make_uint4(0u, 0u, 0u, 0u);
            if (first + 32 * i < rows && c < p.P) {
                const long long at = (long long)(first + 32 * i) * p.P + c;
                a[i][kb] = __ldg((const uint4 *)((const bf16 *)p.o + at));
                b[i][kb] = __ldg((const uint4 *)((const bf16 *)p.d_o + at));
            }
        }
#pragma unroll
    for (int i = 0; i < kDeltaRows; ++i) {
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const uint32_t x[4] = {a[i][kb].x, a[i][kb].y, a[i][kb].z, a[i][kb].w}, y[4] = {b[i][kb].x, b[i][kb].y, b[i][kb].z, b[i][kb].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) acc = ffma2(tc::bf2_to_f2(x[e]), tc::bf2_to_f2(y[e]), acc);
        }
        float s = acc.x + acc.y;
#pragma unroll
        for (int x = 4; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const uint32_t row = first + 32 * i;
        if (row < rows && lane == 0) {
            const uint32_t token = row / (uint32_t)p.H, h = row - token * p.H, bi = token / (uint32_t)p.L, t = token - bi * p.L;
            p.delta[((long long)bi * p.H + h) * p.L + t] = s;
        }
    }
}

struct Maps {
    CUtensorMap q, d_o, k, v;
};

// ------------------------------------------------------------------ dq
constexpr int kDqCompute = 256, kDqThreads = 384, kDqKeys = 96, kDqK = 3, kDqV = 2;  // slots of the rings of K and V tiles
template <int KB>
struct DqLayout {
    static constexpr int kBlock = kDqKeys * 128, kTile = KB * kBlock, kQTile = KB * 16384;
    static constexpr int kOffDO = kQTile, kOffK = 2 * kQTile, kOffV = kOffK + kDqK * kTile, kOffStage = kOffV + kDqV * kTile,
                         kOffBars = kOffStage + 8 * 4096, kBytes = kOffBars + 1024;
    // tensor memory: S of buffer b at 96 b (dx over it, each half over its own columns), dP at 192 + 96 b, dQ at 384
    static constexpr int kS = 0, kDP = 2 * kDqKeys, kDQ = 4 * kDqKeys;
    static_assert(kBytes <= 232448 && kDQ + 64 * KB <= 512, "memory");
};
struct DqBars {
    uint64_t q_full, q_empty, full[2], dp_free[2], ds_full[2], ds_free[2], dq_full, dq_empty, drain, k_full[kDqK], k_empty[kDqK],
        v_full[kDqV], v_empty[kDqV];
    uint32_t tmem;
    int err;
};
static_assert(sizeof(DqBars) <= 1024, "barriers");

using DqItem = QueryItem<kDqKeys>;

// The thread of one of the two products of a pair of tiles: A from `a` (the query tile's rows), B from a ring of SLOTS tiles.
template <int KB, int SLOTS>
__device__ __forceinline__ void dq_scores(const WindowParams &p, int items, int per_row, int T, int ksteps, uint32_t a, uint32_t ring,
                                          uint32_t to, uint64_t *full, uint64_t *free, uint64_t *in_full, uint64_t *in_empty, DqBars &sm) {
    using Lay = DqLayout<KB>;
    const uint64_t d_a = tc::sdesc(a, 16, 1024), d_b = tc::sdesc(ring, 16, 1024);
    const uint32_t idesc0 = tc::idesc_bf16(128, 0, false, false);
    Place<SLOTS> at;
    uint32_t nq = 0, n = 0;
    for (Cursor cur(items, per_row, p); cur.left > 0; cur.next()) {
        const DqItem it(p, cur, T);
        if (it.tiles) wait_bar(&sm.q_full, nq++ & 1, &sm.err);
        for (int j = 0; j < it.tiles; ++j, ++n) {
            wait_bar(&in_full[at.slot], at.phase, &sm.err);
            wait_bar(&free[n & 1], ((n >> 1) & 1) ^ 1, &sm.err);
            tc::tc_fence_after();
            const uint32_t idesc = idesc0 | (uint32_t)((it.count(j) + 15) >> 4) << 18;  // N / 8 from bit 17
            const uint64_t b = delta::sdesc_add(d_b, at.slot * Lay::kTile);
            const uint32_t d = to + (n & 1) * kDqKeys;
#pragma unroll
            for (int ks = 0; ks < 4 * KB; ++ks)
                if (ks < ksteps)
                    tc::mma_bf16(d, delta::sdesc_add(d_a, (ks >> 2) * 16384 + (ks & 3) * 32),
                                 delta::sdesc_add(b, (ks >> 2) * Lay::kBlock + (ks & 3) * 32), idesc, ks > 0);
            tc::mma_commit(&full[n & 1]);
            tc::mma_commit(&in_empty[at.slot]);
            if (j == it.tiles - 1) tc::mma_commit(&sm.q_empty);
            at.next();
        }
    }
    tc::mma_commit(&sm.drain);
    mbar_wait(&sm.drain, 0);
}

template <int KB>
__global__ void __launch_bounds__(kDqThreads, 1) window_dq_kernel(const __grid_constant__ Maps maps, WindowParams p, int items, int per_row) {
    using Lay = DqLayout<KB>;
    extern __shared__ __align__(1024) char smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    DqBars &sm = *(DqBars *)(smem_raw + Lay::kOffBars);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 2);  // the threads of S and of dP
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.full[b], 2);  // S and dP
            mbar_init(&sm.dp_free[b], 8);
            mbar_init(&sm.ds_full[b], 8);
            mbar_init(&sm.ds_free[b], 1);
        }
        mbar_init(&sm.dq_full, 1);
        mbar_init(&sm.dq_empty, 8);
        for (int i = 0; i < kDqK; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 2);  // the threads of S and of dQ
        }
        for (int i = 0; i < kDqV; ++i) {
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        mbar_init(&sm.drain, 3);
        tc::mbar_fence_init();
        sm.err = 0;
    }
    if (warp == 0) {
        __syncwarp();
        tc::tmem_alloc(&sm.tmem, 512);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, sm.tmem, 0);
    const int T = tile_tokens(p), R = p.hpg;
    int *const err = &sm.err;
    const int ksteps = (p.P + 15) / 16;

    if (warp == kDqCompute / 32) {
        // ---- copies
        if (elect()) {
            const uint32_t q_bytes = (uint32_t)(2 * T * R) * 128u * KB;
            Place<kDqK> ak;
            Place<kDqV> av;
            uint32_t nq = 0, nk = 0, nv = 0;
            bool ok = true;
            for (Cursor cur(items, per_row, p); cur.left > 0 && ok; cur.next()) {
                const DqItem it(p, cur, T);
                if (it.tiles) {
                    if (!(ok = wait_copy(&sm.q_empty, (nq & 1) ^ 1, err))) break;
                    ++nq;
                    mbar_arrive_expect_tx(&sm.q_full, q_bytes);
                    for (int kb = 0; kb < KB; ++kb) {
                        tma_tile(base + kb * 16384, &maps.q, &sm.q_full, 64 * kb, it.g * R, it.ta, it.bi);
                        tma_tile(base + Lay::kOffDO + kb * 16384, &maps.d_o, &sm.q_full, 64 * kb, it.g * R, it.ta, it.bi);
                    }
                }
                for (int j = 0; j < it.tiles; ++j) {
                    if (!(ok = wait_copy(&sm.k_empty[ak.slot], ak.phase ^ 1, err))) break;
                    ++nk;
                    mbar_arrive_expect_tx(&sm.k_full[ak.slot], Lay::kTile);
                    for (int kb = 0; kb < KB; ++kb)
                        tma_tile(base + Lay::kOffK + ak.slot * Lay::kTile + kb * Lay::kBlock, &maps.k, &sm.k_full[ak.slot], 64 * kb, it.g,
                                 it.start(j), it.bi);
                    if (!(ok = wait_copy(&sm.v_empty[av.slot], av.phase ^ 1, err))) break;
                    ++nv;
                    mbar_arrive_expect_tx(&sm.v_full[av.slot], Lay::kTile);
                    for (int kb = 0; kb < KB; ++kb)
                        tma_tile(base + Lay::kOffV + av.slot * Lay::kTile + kb * Lay::kBlock, &maps.v, &sm.v_full[av.slot], 64 * kb, it.g,
                                 it.start(j), it.bi);
                    ak.next(), av.next();
                }
            }
            // copies in flight land before the block ends
            for (uint32_t x = nk > kDqK ? nk - kDqK : 0; x < nk; ++x) mbar_wait(&sm.k_full[x % kDqK], (x / kDqK) & 1);
            for (uint32_t x = nv > kDqV ? nv - kDqV : 0; x < nv; ++x) mbar_wait(&sm.v_full[x % kDqV], (x / kDqV) & 1);
            if (nq) mbar_wait(&sm.q_full, (nq - 1) & 1);
        }
        __syncwarp();
    } else if (warp == kDqCompute / 32 + 1) {
        // ---- S = Q K^T
        if (elect())
            dq_scores<KB, kDqK>(p, items, per_row, T, ksteps, base, base + Lay::kOffK, tm + Lay::kS, sm.full, sm.ds_free, sm.k_full, sm.k_empty,
                                sm);
        __syncwarp();
    } else if (warp == kDqCompute / 32 + 2) {
        // ---- dP = dO V^T
        if (elect())
            dq_scores<KB, kDqV>(p, items, per_row, T, ksteps, base + Lay::kOffDO, base + Lay::kOffV, tm + Lay::kDP, sm.full, sm.dp_free,
                                sm.v_full, sm.v_empty, sm);
        __syncwarp();
    } else if (warp == kDqCompute / 32 + 3) {
        // ---- dQ += dX K
        if (elect()) {
            const uint32_t idesc = tc::idesc_bf16(128, (p.P + 15) / 16 * 16, false, true);
            const uint64_t d_k = tc::sdesc(base + Lay::kOffK, Lay::kBlock, 1024);
            Place<kDqK> at;
            uint32_t ni = 0, n = 0;
            for (Cursor cur(items, per_row, p); cur.left > 0; cur.next()) {
                const DqItem it(p, cur, T);
                for (int j = 0; j < it.tiles; ++j, ++n) {
                    if (j == 0) wait_bar(&sm.dq_empty, (ni++ & 1) ^ 1, err);
                    wait_bar(&sm.ds_full[n & 1], (n >> 1) & 1, err);
                    tc::tc_fence_after();
                    const int steps = (it.count(j) + 15) >> 4;
                    const uint64_t k = delta::sdesc_add(d_k, at.slot * Lay::kTile);
                    const uint32_t ds = tm + Lay::kS + (n & 1) * kDqKeys;
#pragma unroll
                    for (int ks = 0; ks < kDqKeys / 16; ++ks)  // dx of the second 48 columns starts where their scores did
                        if (ks < steps)
                            tc::mma_bf16_tmem_a(tm + Lay::kDQ, ds + (ks < 3 ? 8 * ks : 48 + 8 * (ks - 3)), delta::sdesc_add(k, ks * 2048),
                                                idesc, j > 0 || ks > 0);
                    tc::mma_commit(&sm.ds_free[n & 1]);
                    tc::mma_commit(&sm.k_empty[at.slot]);
                    if (j == it.tiles - 1) tc::mma_commit(&sm.dq_full);
                    at.next();
                }
            }
            tc::mma_commit(&sm.drain);
            mbar_wait(&sm.drain, 0);
        }
        __syncwarp();
    } else {
        // ---- dx of columns [48 half, 48 half + 48) of a tile
        const int half = warp >> 2, row = tid & 127, quarter = warp & 3;
        const uint32_t magic = row_magic(R), stage = base + Lay::kOffStage + warp * 4096;
        const uint32_t ts = tmem_addr(tm, 32 * quarter, Lay::kS + 48 * half), tp = tmem_addr(tm, 32 * quarter, Lay::kDP + 48 * half),
                       to = tmem_addr(tm, 32 * quarter, Lay::kDQ);
        const int token = row_token(row, magic), head = row - token * R;
        const float c = p.scale * kLog2e;
        uint32_t n = 0, ni = 0;
        for (Cursor cur(items, per_row, p); cur.left > 0; cur.next()) {
            const DqItem it(p, cur, T);
            const int t = it.ta + token, h = it.g * R + head;
            const bool live = row < T * R && t < it.V;
            float lse2 = 0.f, D = 0.f;
            if (live) {
                const long long at = ((long long)it.bi * p.H + h) * p.L + t;
                lse2 = -kLog2e * __ldg(p.lse + at);
                D = -p.delta[at];
            }
            const int tq = live ? t : it.ta;
            const float2 cc = make_float2(c, c), ll = make_float2(lse2, lse2), DD = make_float2(D, D), one = make_float2(1.f, 1.f);
            for (int j = 0; j < it.tiles; ++j, ++n) {
                const int b = n & 1, nk = it.count(j), s0 = it.start(j), mine = s0 + 48 * half;
                const bool plain = it.plain(p, T, s0, nk);
                wait_warp(&sm.full[b], (n >> 1) & 1, err);
                tc::tc_fence_after();
                float2 x[24], y[24];
                tmem_ld48x2(ts + b * kDqKeys, tp + b * kDqKeys, (float *)x, (float *)y);
                tc::tc_fence_before();
                arrive_first(&sm.dp_free[b], lane);
#pragma unroll
                for (int e = 0; e < 24; ++e) {
                    float2 u = ffma2(x[e], cc, ll);
                    u = make_float2(exp2_approx(u.x), exp2_approx(u.y));
                    x[e] = fmul2(u, ffma2(y[e], one, DD));
                }
                if (!plain) {
                    const int hi = min(nk, tq - s0 + 1) - 48 * half, from = tq - p.W + 1 - mine, sk = p.sinks - mine;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t see = bits_between(-32, hi - 32 * q) & (bits_between(from - 32 * q, 32) | bits_between(-32, sk - 32 * q));
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (16 * q + e >= 24) break;
                            x[16 * q + e].x = see >> (2 * e) & 1 ? x[16 * q + e].x : 0.f;
                            x[16 * q + e].y = see >> (2 * e + 1) & 1 ? x[16 * q + e].y : 0.f;
                        }
                    }
                    __syncwarp();
                }
                uint32_t pk[24];
#pragma unroll
                for (int e = 0; e < 24; ++e) pk[e] = tc::pack_bf2(x[e].x, x[e].y);
                delta::tmem_st16(ts + b * kDqKeys, (const float *)pk);
                tmem_st8(ts + b * kDqKeys + 16, pk + 16);
                delta::tmem_wait_st();
                if (nk & 15) {
                    // rows of K up to the product's step of 16: their dx is 0, so they have to be finite
                    const int rows = 16 - (nk & 15);
                    const uint32_t k = base + Lay::kOffK + n % kDqK * Lay::kTile;
                    for (int e = tid; e < rows * 8 * KB; e += kDqCompute)
                        tc::st_shared_v4(k + (e / (8 * rows)) * Lay::kBlock + (nk + e / 8 % rows) * 128 + (e & 7) * 16, 0, 0, 0, 0);
                    tc::fence_async_smem();
                    __syncwarp();
                }
                tc::tc_fence_before();
                arrive_first(&sm.ds_full[b], lane);
            }
            if (it.tiles) {
                wait_warp(&sm.dq_full, ni++ & 1, err);
                tc::tc_fence_after();
            }
            // columns [64 half, + 64)
            if (half < KB) {
                __syncwarp();
                stage_rows(stage, to + 64 * half, lane, live ? p.scale : 0.f, it.tiles > 0);
            }
            if (it.tiles) {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.dq_empty);
            }
            if (half < KB) {
                __syncwarp();
                store_lines(stage, quarter, lane, (bf16 *)p.dq + (((long long)it.bi * p.L + it.ta) * p.H + it.g * R) * p.P,
                            min(T, p.L - it.ta) * R, 64 * half, p.P,
                            [&](int r) { return row_token(r, magic) * (p.H - R) * p.P + r * p.P; });
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 0) {
        __syncwarp();
        tc::tmem_dealloc(tm, 512);
    }
    if (tid == 0 && sm.err) atomicExch(p.status + kStatusCode, (int)SSD_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ dk and dv
constexpr int kDkvCompute = 256, kDkvThreads = 512, kDkvRows = 64;
template <int KB>
struct DkvLayout {
    static constexpr int kSlots = KB == 2 ? 4 : 6;  // of the ring of query rows, their do and their statistics
    static constexpr int kKTile = KB * 16384, kBlock = kDkvRows * 128, kTile = KB * kBlock;
    static constexpr int kOffV = kKTile, kOffRing = 2 * kKTile, kOffStage = kOffRing + kSlots * 2 * kTile, kOffStats = kOffStage + 8 * 4096,
                         kOffBars = kOffStats + kSlots * 512, kBytes = kOffBars + 1024;
    // tensor memory: S^T of buffer b at 128 b, dP^T at 128 b + 64 (p and dx over them, each half over its own columns)
    static constexpr int kDV = 256, kDK = 256 + 64 * KB;
    static_assert(kBytes <= 232448, "shared memory");
};
struct DkvBars {
    uint64_t kv_full, kv_empty, s_full[2], dp_full[2], p_full[2], dx_full[2], s_free[2], dp_free[2], acc_full, acc_empty, drain, in_full[6], in_empty[6], stats_full[6];
    uint32_t tmem;
    int err;
};
static_assert(sizeof(DkvBars) <= 1024, "barriers");

// How the keys that are sinks are cut: `tiles` tiles of 128 keys, the tokens behind their windows in `segments` of `length`.
struct SinkCut {
    int tiles, segments, length;
};
inline SinkCut sink_cut(long long L, long long W, long long sinks) {
    SinkCut c = {0, 0, 0};
    const long long behind = L - 127 - W;
    if (sinks < 1 || behind < 1) return c;
    // as long as a window item, but no shorter than 1024 tokens, and in all no more than 1024 shares a group: their place is
    // 1 KB a column each, and many tiles of sinks fill the SMs without being cut
    c.tiles = (int)((sinks + 127) / 128);
    const long long most = c.tiles < 1024 ? 1024 / c.tiles : 1, even = (behind + most - 1) / most, least = W + 127 < 1024 ? 1024 : W + 127;
    c.length = (int)(even < least ? least : even);
    c.segments = (int)((behind + c.length - 1) / c.length);
    return c;
}
__host__ __device__ inline size_t sink_floats(const SinkCut &c, long long groups, long long P) {
    return c.segments ? (size_t)groups * c.tiles * (c.segments + 1) * 2 * 128 * P : 0;
}

// 128 keys from k0 and the query tokens [tb, te) that see them: first the sinks' segments, then the rows' tiles, every row's first
// before any other, so that those at a row's end, which fewer tokens see, come last.
struct DkvItem {
    int bi, g, V, k0, tb, te, tiles, part;  // part: the sinks' share that this is, or -1
    __device__ __forceinline__ DkvItem(const WindowParams &p, int index, int T, const SinkCut &cut) {
        const int rows = p.b * p.G, sinks = rows * cut.tiles * cut.segments;
        int tile, segment = 0, row;
        if (index < sinks) {
            row = index % rows;
            tile = index / rows / cut.segments;
            segment = index / rows % cut.segments + 1;
        } else {
            row = (index - sinks) % rows;
            tile = (index - sinks) / rows;
        }
        g = row % p.G;
        bi = row / p.G;
        V = valid_tokens(p, bi);
        k0 = 128 * tile;
        if (segment == 0) {
            tb = k0;
            te = min(V, k0 + 127 + p.W);
        } else {
            const long long from = k0 + 127ll + p.W + (segment - 1ll) * cut.length;
            tb = (int)min(from, (long long)V);
            te = (int)min(from + cut.length, (long long)V);
        }
        part = cut.segments && tile < cut.tiles ? ((bi * p.G + g) * cut.tiles + tile) * (cut.segments + 1) + segment : -1;
        tiles = te > tb ? (te - tb + T - 1) / T : 0;
    }
};

template <int KB>
__global__ void __launch_bounds__(kDkvThreads, 1) window_dkv_kernel(const __grid_constant__ Maps maps, WindowParams p, SinkCut cut, float *parts,
                                                                    int items) {
    using Lay = DkvLayout<KB>;
    constexpr int SLOTS = Lay::kSlots;
    extern __shared__ __align__(1024) char smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    DkvBars &sm = *(DkvBars *)(smem_raw + Lay::kOffBars);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        mbar_init(&sm.kv_full, 1);
        mbar_init(&sm.kv_empty, 2);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.s_full[b], 1);
            mbar_init(&sm.dp_full[b], 1);
            mbar_init(&sm.p_full[b], 8);
            mbar_init(&sm.dx_full[b], 8);
            mbar_init(&sm.s_free[b], 1);
            mbar_init(&sm.dp_free[b], 1);
        }
        mbar_init(&sm.acc_full, 2);  // dV and dK
        mbar_init(&sm.acc_empty, 8);
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&sm.in_full[i], 1);
            mbar_init(&sm.in_empty[i], 2);  // dV and dK, which come behind S^T and dP^T
            mbar_init(&sm.stats_full[i], 1);
        }
        mbar_init(&sm.drain, 4);
        tc::mbar_fence_init();
        sm.err = 0;
    }
    if (warp == 0) {
        __syncwarp();
        tc::tmem_alloc(&sm.tmem, 512);
    }
    // rows past the tokens' of a query tile are never copied and stay 0
    for (int e = tid; e < SLOTS * 2 * Lay::kTile / 16; e += kDkvThreads) tc::st_shared_v4(base + Lay::kOffRing + 16 * e, 0, 0, 0, 0);
    tc::fence_async_smem();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, sm.tmem, 0);
    const int R = p.hpg, T = kDkvRows / R;
    int *const err = &sm.err;

    if (warp == kDkvCompute / 32) {
        // ---- copies
        if (elect()) {
            const uint32_t bytes = (uint32_t)(2 * T * R) * 128u * KB;
            Place<SLOTS> at;
            uint32_t nk = 0, n = 0;
            bool ok = true;
            for (int index = blockIdx.x; index < items && ok; index += gridDim.x) {
                const DkvItem it(p, index, T, cut);
                if (it.tiles) {
                    if (!(ok = wait_copy(&sm.kv_empty, (nk & 1) ^ 1, err))) break;
                    ++nk;
                    mbar_arrive_expect_tx(&sm.kv_full, 2 * Lay::kKTile);
                    for (int kb = 0; kb < KB; ++kb) {
                        tma_tile(base + kb * 16384, &maps.k, &sm.kv_full, 64 * kb, it.g, it.k0, it.bi);
                        tma_tile(base + Lay::kOffV + kb * 16384, &maps.v, &sm.kv_full, 64 * kb, it.g, it.k0, it.bi);
                    }
                }
                for (int j = 0; j < it.tiles; ++j, ++n) {
                    if (!(ok = wait_copy(&sm.in_empty[at.slot], at.phase ^ 1, err))) break;
                    mbar_arrive_expect_tx(&sm.in_full[at.slot], bytes);
                    const uint32_t to = base + Lay::kOffRing + at.slot * 2 * Lay::kTile;
                    for (int kb = 0; kb < KB; ++kb) {
                        tma_tile(to + kb * Lay::kBlock, &maps.q, &sm.in_full[at.slot], 64 * kb, it.g * R, it.tb + j * T, it.bi);
                        tma_tile(to + Lay::kTile + kb * Lay::kBlock, &maps.d_o, &sm.in_full[at.slot], 64 * kb, it.g * R, it.tb + j * T, it.bi);
                    }
                    at.next();
                }
            }
            // copies in flight land before the block ends
            for (uint32_t x = n > SLOTS ? n - SLOTS : 0; x < n; ++x) mbar_wait(&sm.in_full[x % SLOTS], (x / SLOTS) & 1);
            if (nk) mbar_wait(&sm.kv_full, (nk - 1) & 1);
        }
        __syncwarp();
    } else if (warp == kDkvCompute / 32 + 1 || warp == kDkvCompute / 32 + 2) {
        // ---- S^T = K Q^T (first thread), dP^T = V dO^T (second)
        if (elect()) {
            const uint32_t second = warp - (kDkvCompute / 32 + 1);
            const uint32_t idesc = tc::idesc_bf16(128, kDkvRows, false, false);
            const int ksteps = (p.P + 15) / 16;
            const uint64_t d_a = tc::sdesc(base + second * Lay::kOffV, 16, 1024), d_b = tc::sdesc(base + Lay::kOffRing + second * Lay::kTile, 16, 1024);
            uint64_t *const full = second ? sm.dp_full : sm.s_full, *const free = second ? sm.dp_free : sm.s_free;
            Place<SLOTS> at;
            uint32_t nk = 0, n = 0;
            for (int index = blockIdx.x; index < items; index += gridDim.x) {
                const DkvItem it(p, index, T, cut);
                if (it.tiles) wait_bar(&sm.kv_full, nk++ & 1, err);
                for (int j = 0; j < it.tiles; ++j, ++n) {
                    wait_bar(&sm.in_full[at.slot], at.phase, err);
                    wait_bar(&free[n & 1], ((n >> 1) & 1) ^ 1, err);
                    tc::tc_fence_after();
                    const uint64_t b = delta::sdesc_add(d_b, at.slot * 2 * Lay::kTile);
                    const uint32_t d = tm + 128 * (n & 1) + 64 * second;
#pragma unroll
                    for (int ks = 0; ks < 4 * KB; ++ks)
                        if (ks < ksteps)
                            tc::mma_bf16(d, delta::sdesc_add(d_a, (ks >> 2) * 16384 + (ks & 3) * 32),
                                         delta::sdesc_add(b, (ks >> 2) * Lay::kBlock + (ks & 3) * 32), idesc, ks > 0);
                    tc::mma_commit(&full[n & 1]);
                    at.next();
                }
            }
            tc::mma_commit(&sm.drain);
            mbar_wait(&sm.drain, 0);
        }
        __syncwarp();
    } else if (warp == kDkvCompute / 32 + 3 || warp == kDkvCompute / 32 + 5) {
        // ---- dV += P^T dO (first thread), dK += dX^T Q (second)
        if (elect()) {
            const uint32_t second = warp == kDkvCompute / 32 + 5;
            const uint32_t idesc = tc::idesc_bf16(128, (p.P + 15) / 16 * 16, false, true), to = tm + (second ? Lay::kDK : Lay::kDV);
            const uint64_t d_b = tc::sdesc(base + Lay::kOffRing + (second ? 0 : Lay::kTile), Lay::kBlock, 1024);
            uint64_t *const in = second ? sm.dx_full : sm.p_full, *const free = second ? sm.dp_free : sm.s_free;
            Place<SLOTS> at;
            uint32_t ni = 0, n = 0;
            for (int index = blockIdx.x; index < items; index += gridDim.x) {
                const DkvItem it(p, index, T, cut);
                for (int j = 0; j < it.tiles; ++j, ++n) {
                    if (j == 0) wait_bar(&sm.acc_empty, (ni++ & 1) ^ 1, err);
                    wait_bar(&in[n & 1], (n >> 1) & 1, err);
                    tc::tc_fence_after();
                    const uint64_t b = delta::sdesc_add(d_b, at.slot * 2 * Lay::kTile);
                    const uint32_t a = tm + 128 * (n & 1) + 64 * second;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)  // the second 32 rows' values start where their scores did
                        tc::mma_bf16_tmem_a(to, a + (ks & 2) * 16 + (ks & 1) * 8, delta::sdesc_add(b, ks * 2048), idesc, j > 0 || ks > 0);
                    tc::mma_commit(&free[n & 1]);
                    tc::mma_commit(&sm.in_empty[at.slot]);
                    if (j == it.tiles - 1) {
                        tc::mma_commit(&sm.kv_empty);
                        tc::mma_commit(&sm.acc_full);
                    }
                    at.next();
                }
            }
            tc::mma_commit(&sm.drain);
            mbar_wait(&sm.drain, 0);
        }
        __syncwarp();
    } else if (warp == kDkvCompute / 32 + 4) {
        // ---- the rows' statistics: -lse log2(e) (so low where there is no row that p is 0) and -D
        const uint32_t magic = row_magic(R);
        Place<SLOTS> at;
        for (int index = blockIdx.x; index < items; index += gridDim.x) {
            const DkvItem it(p, index, T, cut);
            for (int j = 0; j < it.tiles; ++j) {
                float ll[2] = {-INFINITY, -INFINITY}, dd[2] = {0.f, 0.f};
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = lane + 32 * x, token = row_token(r, magic), t = it.tb + j * T + token;
                    if (r < T * R && t < it.te) {
                        const long long from = ((long long)it.bi * p.H + it.g * R + r - token * R) * p.L + t;
                        ll[x] = -kLog2e * __ldg(p.lse + from);
                        dd[x] = -__ldg(p.delta + from);
                    }
                }
                wait_warp(&sm.in_empty[at.slot], at.phase ^ 1, err);
                float *to = (float *)(smem_raw + Lay::kOffStats) + at.slot * 128;
                to[lane] = ll[0], to[lane + 32] = ll[1], to[64 + lane] = dd[0], to[96 + lane] = dd[1];
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.stats_full[at.slot]);
                at.next();
            }
        }
    } else if (warp < kDkvCompute / 32) {
        // ---- p and dx of rows [32 half, 32 half + 32) of a query tile; then one of the two accumulators
        const int half = warp >> 2, quarter = warp & 3, key = tid & 127;
        const uint32_t stage = base + Lay::kOffStage + warp * 4096;
        const uint32_t ts = tmem_addr(tm, 32 * quarter, 32 * half), ta = tmem_addr(tm, 32 * quarter, half ? Lay::kDK : Lay::kDV);
        const float c = p.scale * kLog2e;
        const float2 cc = make_float2(c, c);
        Place<SLOTS> at;
        uint32_t n = 0, ni = 0;
        for (int index = blockIdx.x; index < items; index += gridDim.x) {
            const DkvItem it(p, index, T, cut);
            const int s = it.k0 + key;
            for (int j = 0; j < it.tiles; ++j, ++n) {
                const int b = n & 1, t0 = it.tb + j * T;
                const bool plain = it.k0 + 127 <= t0 && (t0 + T - 1 - it.k0 < p.W || it.k0 + 128 <= p.sinks) && t0 + T <= it.V;
                wait_warp(&sm.stats_full[at.slot], at.phase, err);
                wait_warp(&sm.s_full[b], (n >> 1) & 1, err);
                tc::tc_fence_after();
                float2 x[16], y[16];
                uint32_t pk[16], see = 0xffffffffu;
                tc::tmem_ld32u(ts + 128 * b, (uint32_t *)x);
                const uint32_t st = base + Lay::kOffStats + at.slot * 512 + half * 128;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint4 l4 = tc::ld_shared_v4(st + 16 * e);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const float2 ll = make_float2(__uint_as_float(z ? l4.z : l4.x), __uint_as_float(z ? l4.w : l4.y));
                        const float2 u = ffma2(x[2 * e + z], cc, ll);
                        x[2 * e + z] = make_float2(exp2_approx(u.x), exp2_approx(u.y));
                    }
                }
                if (!plain) {
                    const int first = max(0, s - t0) * R, last = min(it.te - t0, s < p.sinks ? T : min(T, s + p.W - t0)) * R;
                    see = bits_between(first - 32 * half, last - 32 * half);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        x[e] = make_float2(see & (1u << (2 * e)) ? x[e].x : 0.f, see & (2u << (2 * e)) ? x[e].y : 0.f);
                    if (t0 + T > it.V) {
                        // rows of absent tokens: their p and dx are 0, so q and do have to be finite (dP^T has read them)
                        wait_warp(&sm.dp_full[b], (n >> 1) & 1, err);
                        const int from = (it.V - t0) * R, rows = T * R - from;
                        const uint32_t q = base + Lay::kOffRing + at.slot * 2 * Lay::kTile;
                        for (int e = tid; e < rows * 8 * 2 * KB; e += kDkvCompute)
                            tc::st_shared_v4(q + (e / (8 * rows)) * Lay::kBlock + (from + e / 8 % rows) * 128 + (e & 7) * 16, 0, 0, 0, 0);
                        tc::fence_async_smem();
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) pk[e] = tc::pack_bf2(x[e].x, x[e].y);
                delta::tmem_st16(ts + 128 * b, (const float *)pk);
                delta::tmem_wait_st();
                tc::tc_fence_before();
                arrive_first(&sm.p_full[b], lane);
                wait_warp(&sm.dp_full[b], (n >> 1) & 1, err);
                tc::tc_fence_after();
                tc::tmem_ld32u(ts + 128 * b + 64, (uint32_t *)y);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint4 d4 = tc::ld_shared_v4(st + 256 + 16 * e);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const float2 dd = make_float2(__uint_as_float(z ? d4.z : d4.x), __uint_as_float(z ? d4.w : d4.y));
                        y[2 * e + z] = fmul2(x[2 * e + z], ffma2(y[2 * e + z], make_float2(1.f, 1.f), dd));
                    }
                }
                if (!plain) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        y[e] = make_float2(see & (1u << (2 * e)) ? y[e].x : 0.f, see & (2u << (2 * e)) ? y[e].y : 0.f);
                    __syncwarp();
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) pk[e] = tc::pack_bf2(y[e].x, y[e].y);
                delta::tmem_st16(ts + 128 * b + 64, (const float *)pk);
                delta::tmem_wait_st();
                tc::tc_fence_before();
                arrive_first(&sm.dx_full[b], lane);
                at.next();
            }
            if (it.tiles) {
                wait_warp(&sm.acc_full, ni++ & 1, err);
                tc::tc_fence_after();
            }
            // half 0 stores dV, half 1 dK
            const float f = half ? p.scale : 1.f;
            if (it.part >= 0) {
                float *to = parts + ((size_t)it.part * 2 + half) * 128 * p.P + key * p.P;
                for (int q = 0; q < (p.P + 15) / 16; ++q) {
                    float v[16];
                    if (it.tiles) {
                        __syncwarp();
                        tc::tmem_ld16(ta + 16 * q, v);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = 0.f;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (16 * q + 4 * e < p.P)
                            *(float4 *)(to + 16 * q + 4 * e) = s < it.V ? make_float4(v[4 * e] * f, v[4 * e + 1] * f, v[4 * e + 2] * f, v[4 * e + 3] * f)
                                                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                if (it.tiles) {
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.acc_empty);
                }
            } else {
                bf16 *to = (bf16 *)(half ? p.dk : p.dv) + (((long long)it.bi * p.L + it.k0) * p.G + it.g) * p.P;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    __syncwarp();
                    stage_rows(stage, ta + 64 * kb, lane, s < it.V ? f : 0.f, it.tiles > 0);
                    if (kb == KB - 1 && it.tiles) {
                        tc::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.acc_empty);
                    }
                    __syncwarp();
                    store_lines(stage, quarter, lane, to, min(128, p.L - it.k0), 64 * kb, p.P, [&](int r) { return r * p.G * p.P; });
                }
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 0) {
        __syncwarp();
        tc::tmem_dealloc(tm, 512);
    }
    if (tid == 0 && sm.err) atomicExch(p.status + kStatusCode, (int)SSD_ERR_TIMEOUT);
}

// dk and dv of the sinks' tiles: their shares in order.  One thread per 4 columns.
__global__ void __launch_bounds__(256) window_sinks_kernel(WindowParams p, SinkCut cut, const float *parts, long long n) {
    const long long i = blockIdx.x * 256ll + threadIdx.x;
    const int nq = p.P / 4;
    if (i >= n) return;
    const int c = 4 * (int)(i % nq), row = (int)(i / nq % (128 * cut.tiles)), which = (int)(i / nq / (128 * cut.tiles) % 2);
    const long long bg = i / nq / (128 * cut.tiles) / 2;
    if (row >= p.L) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k <= cut.segments; ++k) {
        const size_t part = (bg * cut.tiles + row / 128) * (cut.segments + 1) + k;
        const float4 x = *(const float4 *)(parts + ((part * 2 + which) * 128 + row % 128) * p.P + c);
        s = make_float4(s.x + x.x, s.y + x.y, s.z + x.z, s.w + x.w);
    }
    store4((bf16 *)(which ? p.dk : p.dv) + ((bg / p.G * p.L + row) * p.G + bg % p.G) * p.P + c, s);
}

template <int KB>
cudaError_t backward(const WindowParams &p, float *parts, cudaStream_t s) {
    cudaError_t e;
    const long long rows = (long long)p.b * p.L * p.H;
    window_delta_kernel<KB><<<(unsigned)((rows + 32 * kDeltaRows - 1) / (32 * kDeltaRows)), 256, 0, s>>>(p, (uint32_t)rows);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    Maps maps;
    {
        const int T = tile_tokens(p), per_row = (p.L + T - 1) / T, items = per_row * p.G * p.b;
        if ((e = map_tokens(&maps.q, p.q, p, p.H, p.hpg, T)) != cudaSuccess) return e;
        if ((e = delta::same_tiles(&maps.d_o, maps.q, p.d_o)) != cudaSuccess) return e;
        if ((e = map_tokens(&maps.k, p.k, p, p.G, 1, kDqKeys)) != cudaSuccess) return e;
        if ((e = delta::same_tiles(&maps.v, maps.k, p.v)) != cudaSuccess) return e;
        if ((e = delta::allow_shared((const void *)window_dq_kernel<KB>, DqLayout<KB>::kBytes)) != cudaSuccess) return e;
        window_dq_kernel<KB><<<tile_grid(p, items, kSMs), kDqThreads, DqLayout<KB>::kBytes, s>>>(maps, p, items, per_row);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const SinkCut cut = sink_cut(p.L, p.W, p.sinks);
    const int T = kDkvRows / p.hpg, items = ((p.L + 127) / 128 + cut.tiles * cut.segments) * p.G * p.b;
    if ((e = map_tokens(&maps.q, p.q, p, p.H, p.hpg, T)) != cudaSuccess) return e;
    if ((e = delta::same_tiles(&maps.d_o, maps.q, p.d_o)) != cudaSuccess) return e;
    if ((e = map_tokens(&maps.k, p.k, p, p.G, 1, 128)) != cudaSuccess) return e;
    if ((e = delta::same_tiles(&maps.v, maps.k, p.v)) != cudaSuccess) return e;
    if ((e = delta::allow_shared((const void *)window_dkv_kernel<KB>, DkvLayout<KB>::kBytes)) != cudaSuccess) return e;
    window_dkv_kernel<KB><<<tile_grid(p, items, kSMs), kDkvThreads, DkvLayout<KB>::kBytes, s>>>(maps, p, cut, parts, items);
    if ((e = cudaGetLastError()) != cudaSuccess || !cut.segments) return e;
    const long long n = (long long)p.b * p.G * 2 * 128 * cut.tiles * (p.P / 4);
    window_sinks_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p, cut, parts, n);
    return cudaGetLastError();
}

}  // namespace

size_t tile_backward_floats(long long batch, long long L, long long G, long long P, long long W, long long sinks) {
    return sink_floats(sink_cut(L, W, sinks), batch * G, P);
}
cudaError_t launch_tile_backward(const WindowParams &p, float *parts, cudaStream_t s) {
    return p.P > 64 ? backward<2>(p, parts, s) : backward<1>(p, parts, s);
}

}  // namespace window
}  // namespace ssd
