// window_fwd.cu -- window attention, forward, on tcgen05.
//
// Blocks stay on their SM, two on each, and take items in turn: a query tile (window_tile.cuh) and the key
// tiles that it sees.  Per pair of tiles S = Q K^T (fp32, tensor memory), the softmax's step, and
// O += P V.  One thread copies (TMA), one issues the products for S and one those for O, and four warps, a thread per row,
// take the softmax.  The two blocks of an SM are what keeps the tensor core in work: one's products run beside the
// other's softmax, first tiles and last stores (one block with two query tiles that share the copies of
// their keys came to the end of both at once, and stood still for a fifth of an item).  S and P have columns of their own in
// a block's half of tensor memory, so that the next S is made as soon as the last one is in registers: 256 columns hold S, P and
// O with 80 keys a tile where O has 128 columns.  Where it has 64 there would be room for more, but a thread's 96 scores leave
// it too few registers (8 padded rows of 1024 to 4096, 64 heads of 64: 481 us of kernel with 80 keys, a tenth more with 96).
// The row maximum is followed lazily: a row's reference only moves to it, and O is only rescaled, where a tile's P add up to
// more than 2^8, so P <= 256 and the passes over O are rare; sums are fp32 and do not care.  Other tiles do not
// look for their maximum (2 x 8192 tokens of 40 heads of 128, window 2048: 437 us, 413 without).
// P is rounded to bf16 (2^-8 of each at most), the sum it is divided by is not.
#include <float.h>

#include <type_traits>

#include "window_tile.cuh"

namespace ssd {
namespace window {
namespace {

using delta::exp2_approx;
using delta::tma_tile;
using tc::ffma2;
using tc::tmem_addr;

// Threads: four warps of softmax, then four of which three issue.  Those give up registers for a softmax thread's
// scores: 128 * 184 + 128 * 72 = 256 * 128, what the block is launched with.  (An instruction costs its issuing thread some 55
// cycles and a wait 100: one thread for all of them could not keep the tensor core in work.)
constexpr int kSoftmax = 128, kThreads = 256, kRegsSoftmax = 184, kRegsIssue = 72;
static_assert(kSoftmax * kRegsSoftmax + (kThreads - kSoftmax) * kRegsIssue <= kThreads * 128, "registers of the launch");
constexpr float kMost = 256.f;  // what a row's P may add up to in a tile

struct Maps {
    CUtensorMap q, k, v;
};

// KB = ceil(P / 64) blocks of 64 columns a tile.
template <int KB>
struct Layout {
    static constexpr int kKeys = 80;  // of a tile
    // Rings of K and of V tiles, apart: a waiting thread tells a phase of a slot from the next one only, so it has to see
    // every use of the slots it waits for (a ring of three slots for both let S begin on a K that had not landed).
    static constexpr int kBlock = kKeys * 128, kTile = KB * kBlock, kK = 2, kV = 2;
    static constexpr int kQTile = KB * 16384;
    static constexpr int kOffK = kQTile, kOffV = kOffK + kK * kTile;
    static constexpr int kOffBars = kOffV + kV * kTile, kBytes = kOffBars + 1024;
    static constexpr int kS = 0, kP = kKeys, kO = 256 - 64 * KB;  // columns of tensor memory
    static_assert(kP + kKeys / 2 <= kO, "tensor memory");
    static_assert(2 * (kBytes + 1024) <= 233472, "shared memory of two blocks");
};
struct Bars {
    uint64_t q_full, q_empty, s_full, s_free, p_full, p_free, o_empty, drain, k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint32_t tmem;
    int err;
};
static_assert(sizeof(Bars) <= 1024, "barriers");

// 32 bytes to an address that is a multiple of 32: a whole sector, where two stores of 16 bytes would be half ones each
__device__ __forceinline__ void store32(void *p, const uint32_t *v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                 "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

template <int KB>
__global__ void __launch_bounds__(kThreads, 2) window_fwd_kernel(const __grid_constant__ Maps maps, WindowParams p, float c,
                                                                 uint32_t negate, int items, int per_row) {
    using Lay = Layout<KB>;
    constexpr int KEYS = Lay::kKeys;
    using It = QueryItem<KEYS>;
    extern __shared__ __align__(1024) char smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    Bars &sm = *(Bars *)(smem_raw + Lay::kOffBars);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        mbar_init(&sm.s_full, 1);
        mbar_init(&sm.s_free, 4);
        mbar_init(&sm.p_full, 4);
        mbar_init(&sm.p_free, 1);
        mbar_init(&sm.o_empty, 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        mbar_init(&sm.drain, 2);
        tc::mbar_fence_init();
        sm.err = 0;
    }
    if (blockIdx.x == 0) write_status(p);
    if (warp == 0) {
        __syncwarp();
        tc::tmem_alloc(&sm.tmem, 256);
    }
    const int T = tile_tokens(p);
    // rows past the tokens' of a query tile are never copied: zeros, so that their sums never ask for a maximum
    for (int e = tid; e < (128 - T * p.hpg) * 8 * KB; e += kThreads)
        tc::st_shared_v4(base + (e % KB) * 16384 + (T * p.hpg) * 128 + e / KB * 16, 0, 0, 0, 0);
    tc::fence_async_smem();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, sm.tmem, 0);
    int *const err = &sm.err;

    if (warp >= kSoftmax / 32) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (warp == kSoftmax / 32) {
            // ---- copies: K a tile ahead of V
            if (elect()) {
                const uint32_t q_bytes = (uint32_t)(T * p.hpg) * 128u * KB;
                Place<Lay::kK> ak;
                Place<Lay::kV> av;
                uint32_t nq = 0, nk = 0, nv = 0;
                bool ok = true;
                for (Cursor cur(items, per_row, p); cur.left > 0 && ok; cur.next()) {
                    const It it(p, cur, T);
                    auto load_k = [&](int j) {
                        if (!(ok = wait_copy(&sm.k_empty[ak.slot], ak.phase ^ 1, err))) return;
                        mbar_arrive_expect_tx(&sm.k_full[ak.slot], Lay::kTile);
                        for (int kb = 0; kb < KB; ++kb)
                            tma_tile(base + Lay::kOffK + ak.slot * Lay::kTile + kb * Lay::kBlock, &maps.k, &sm.k_full[ak.slot], 64 * kb, it.g,
                                     it.start(j), it.bi);
                        ak.next();
                        ++nk;
                    };
                    if (it.tiles) {
                        if (!(ok = wait_copy(&sm.q_empty, (nq & 1) ^ 1, err))) break;
                        mbar_arrive_expect_tx(&sm.q_full, q_bytes);
                        for (int kb = 0; kb < KB; ++kb)
                            tma_tile(base + kb * 16384, &maps.q, &sm.q_full, 64 * kb, it.g * p.hpg, it.ta, it.bi);
                        ++nq;
                        load_k(0);
                    }
                    for (int j = 0; j < it.tiles && ok; ++j) {
                        if (j + 1 < it.tiles) load_k(j + 1);
                        if (!ok || !(ok = wait_copy(&sm.v_empty[av.slot], av.phase ^ 1, err))) break;
                        mbar_arrive_expect_tx(&sm.v_full[av.slot], Lay::kTile);
                        for (int kb = 0; kb < KB; ++kb)
                            tma_tile(base + Lay::kOffV + av.slot * Lay::kTile + kb * Lay::kBlock, &maps.v, &sm.v_full[av.slot], 64 * kb, it.g,
                                     it.start(j), it.bi);
                        av.next();
                        ++nv;
                    }
                }
                // copies in flight land before the block ends
                for (uint32_t x = nk > Lay::kK ? nk - Lay::kK : 0; x < nk; ++x) mbar_wait(&sm.k_full[x % Lay::kK], (x / Lay::kK) & 1);
                for (uint32_t x = nv > Lay::kV ? nv - Lay::kV : 0; x < nv; ++x) mbar_wait(&sm.v_full[x % Lay::kV], (x / Lay::kV) & 1);
                if (nq) mbar_wait(&sm.q_full, (nq - 1) & 1);
            }
            __syncwarp();
        } else if (warp == kSoftmax / 32 + 1) {
            // ---- products S = Q K^T
            if (elect()) {
                const uint32_t i_s0 = tc::idesc_bf16(128, 0, false, false) | negate;
                const int ksteps = (p.P + 15) / 16;
                const uint64_t d_q = tc::sdesc(base, 16, 1024), d_k = tc::sdesc(base + Lay::kOffK, 16, 1024);
                Place<Lay::kK> at;
                uint32_t nq = 0, ns = 0;
                for (Cursor cur(items, per_row, p); cur.left > 0; cur.next()) {
                    const It it(p, cur, T);
                    if (it.tiles) wait_bar(&sm.q_full, nq++ & 1, err);
                    for (int j = 0; j < it.tiles; ++j, ++ns) {
                        wait_bar(&sm.k_full[at.slot], at.phase, err);
                        wait_bar(&sm.s_free, (ns & 1) ^ 1, err);
                        tc::tc_fence_after();
                        const uint32_t i_s = i_s0 | (uint32_t)((it.count(j) + 15) >> 4) << 18;  // N / 8 from bit 17
                        const uint64_t k = delta::sdesc_add(d_k, at.slot * Lay::kTile);
#pragma unroll
                        for (int ks = 0; ks < 4 * KB; ++ks)
                            if (ks < ksteps)
                                tc::mma_bf16(tm + Lay::kS, delta::sdesc_add(d_q, (ks >> 2) * 16384 + (ks & 3) * 32),
                                             delta::sdesc_add(k, (ks >> 2) * Lay::kBlock + (ks & 3) * 32), i_s, ks > 0);
                        tc::mma_commit(&sm.s_full);
                        tc::mma_commit(&sm.k_empty[at.slot]);
                        if (j == it.tiles - 1) tc::mma_commit(&sm.q_empty);
                        at.next();
                    }
                }
                tc::mma_commit(&sm.drain);
                mbar_wait(&sm.drain, 0);
            }
            __syncwarp();
        } else if (warp == kSoftmax / 32 + 2) {
            // ---- products O += P V
            if (elect()) {
                const uint32_t i_pv = tc::idesc_bf16(128, (p.P + 15) / 16 * 16, false, true);
                const uint64_t d_v = tc::sdesc(base + Lay::kOffV, Lay::kBlock, 1024);
                Place<Lay::kV> at;
                uint32_t no = 0, np = 0;
                for (Cursor cur(items, per_row, p); cur.left > 0; cur.next()) {
                    const It it(p, cur, T);
                    if (it.tiles) wait_bar(&sm.o_empty, (no++ & 1) ^ 1, err);
                    for (int j = 0; j < it.tiles; ++j, ++np) {
                        wait_bar(&sm.v_full[at.slot], at.phase, err);
                        wait_bar(&sm.p_full, np & 1, err);
                        tc::tc_fence_after();
                        const int steps = (it.count(j) + 15) >> 4;
                        const uint64_t v = delta::sdesc_add(d_v, at.slot * Lay::kTile);
#pragma unroll
                        for (int ks = 0; ks < KEYS / 16; ++ks)
                            if (ks < steps)
                                tc::mma_bf16_tmem_a(tm + Lay::kO, tm + Lay::kP + 8 * ks, delta::sdesc_add(v, ks * 2048), i_pv, j > 0 || ks > 0);
                        tc::mma_commit(&sm.p_free);
                        tc::mma_commit(&sm.v_empty[at.slot]);
                        at.next();
                    }
                }
                tc::mma_commit(&sm.drain);
                mbar_wait(&sm.drain, 0);
            }
            __syncwarp();
        }
    } else {
        // ---- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int row = tid, R = p.hpg;
        const uint32_t magic = row_magic(R);
        const uint32_t ts = tmem_addr(tm, 32 * warp, Lay::kS), tp = tmem_addr(tm, 32 * warp, Lay::kP), to = tmem_addr(tm, 32 * warp, Lay::kO);
        const int token = row_token(row, magic), head = row - token * R;
        uint32_t ns = 0;  // tiles before
        for (Cursor cur(items, per_row, p); cur.left > 0; cur.next()) {
            const It it(p, cur, T);
            const int t = it.ta + token, h = it.g * R + head;
            const bool in = row < T * R && t < p.L, live = in && t < it.V;
            const int tq = live ? t : it.ta;
            float m = -INFINITY, l = 0.f;
            // tile j, of which the first COLS columns count
            auto tile = [&](int j, int s0, int nk, bool plain, auto columns) {
                constexpr int COLS = decltype(columns)::value;
                wait_warp(&sm.s_full, ns & 1, err);
                tc::tc_fence_after();
                float2 x[COLS / 2];
                if constexpr (COLS == 16)
                    tc::tmem_ld16(ts, (float *)x);
                else
                    tmem_ld80(ts, (float *)x);
                tc::tc_fence_before();
                arrive_first(&sm.s_free, lane);
                if (!plain) {
                    const int hi = min(nk, tq - s0 + 1), from = tq - p.W + 1 - s0, sk = p.sinks - s0;
#pragma unroll
                    for (int q = 0; q < (COLS + 31) / 32; ++q) {
                        const uint32_t see = bits_between(-32, hi - 32 * q) & (bits_between(from - 32 * q, 32) | bits_between(-32, sk - 32 * q));
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (16 * q + e >= COLS / 2) break;
                            float2 &y = x[16 * q + e];
                            y.x = see & (1u << (2 * e)) ? y.x : -INFINITY;
                            y.y = see & (2u << (2 * e)) ? y.y : -INFINITY;
                        }
                    }
                }
                // The exponents are taken with the reference of the tiles before.  None is above 2^8 where their sum is not; where it is,
                // which is rare past the first tiles, they are taken again with the maximum so far.
                const float2 cc = make_float2(c, c), one = make_float2(1.f, 1.f);
                uint32_t pk[COLS / 2];
                float2 sum[2];
                for (;;) {
                    const float ref = m == -INFINITY ? 0.f : -m * c;
                    const float2 rr = make_float2(ref, ref);
                    sum[0] = sum[1] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int e = 0; e < COLS / 2; ++e) {
                        float2 y = ffma2(x[e], cc, rr);
                        y = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                        sum[e & 1] = ffma2(y, one, sum[e & 1]);
                        pk[e] = tc::pack_bf2(y.x, y.y);
                    }
                    sum[0].x = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    if (__all_sync(0xffffffffu, sum[0].x <= kMost && m != -INFINITY)) break;
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < COLS / 2; ++e) mx[e & 3] = max3(mx[e & 3], x[e].x, x[e].y);
                    const float top = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
                    const bool grows = top > m && (m == -INFINITY || sum[0].x > kMost);
                    if (!__any_sync(0xffffffffu, grows)) break;
                    const float f = grows ? (m == -INFINITY ? 0.f : exp2_approx((m - top) * c)) : 1.f;
                    m = grows ? top : m;
                    l *= f;
                    if (j > 0) {
                        wait_warp(&sm.p_free, (ns & 1) ^ 1, err);
                        tc::tc_fence_after();
                        for (int q = 0; q < (p.P + 15) / 16; ++q) {
                            float o[16];
                            __syncwarp();
                            tc::tmem_ld16(to + 16 * q, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= f;
                            delta::tmem_st16(to + 16 * q, o);
                        }
                        delta::tmem_wait_st();
                    }
                }
                // the product with the last P is done
                wait_warp(&sm.p_free, (ns & 1) ^ 1, err);
                tc::tc_fence_after();
                ++ns;
                if constexpr (COLS == 80) tmem_st32(tp, pk);
                tmem_st8(tp + COLS / 2 - 8, pk + COLS / 2 - 8);
                delta::tmem_wait_st();
                l += sum[0].x;
                if (nk & 15) {
                    // rows of V up to the product's step of 16: their probabilities are 0, so they have to be finite
                    // (V's last use of the slot is over, as the product before this one is)
                    const uint32_t at = ns - 1, slot = at % Lay::kV;
                    const int rows = 16 - (nk & 15);
                    wait_warp(&sm.v_full[slot], (at / Lay::kV) & 1, err);
                    const uint32_t v = base + Lay::kOffV + slot * Lay::kTile;
                    for (int e = row; e < rows * 8 * KB; e += kSoftmax)
                        tc::st_shared_v4(v + (e / (8 * rows)) * Lay::kBlock + (nk + e / 8 % rows) * 128 + (e & 7) * 16, 0, 0, 0, 0);
                    tc::fence_async_smem();
                    __syncwarp();
                }
                tc::tc_fence_before();
                arrive_first(&sm.p_full, lane);
            };
            for (int j = 0; j < it.tiles; ++j) {
                const int s0 = it.start(j), nk = it.count(j);
                if (nk <= 16)  // a few sinks
                    tile(j, s0, nk, false, std::integral_constant<int, 16>());
                else
                    tile(j, s0, nk, it.plain(p, T, s0, nk), std::integral_constant<int, KEYS>());
            }
            if (it.tiles) {
                // the last product: p_free's phase that the next item's first tile waits for too
                wait_warp(&sm.p_free, (ns & 1) ^ 1, err);
                tc::tc_fence_after();
            }
            if (in && p.lse) p.lse[((long long)it.bi * p.H + h) * p.L + t] = live ? (m * c + log2f(l)) * kLn2 : 0.f;
            const float inv = live ? 1.f / l : 0.f;
            // O in bf16, a thread its row's next 64 bytes at a time.  The loop stays one: code that runs once an item is fetched from
            // past the instruction caches, and costs more than what it does.
            bf16 *const o = (bf16 *)p.o + (((long long)it.bi * p.L + t) * p.H + h) * p.P;
            const bool wide = p.P % 16 == 0 && ((uintptr_t)p.o & 31) == 0;
#pragma unroll 1
            for (int q = 0; q < p.P; q += 32) {
                float v[32];
                if (it.tiles) {
                    __syncwarp();
                    tc::tmem_ld32u(to + q, (uint32_t *)v);
                }
                uint32_t y[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = live ? tc::pack_bf2(v[2 * e] * inv, v[2 * e + 1] * inv) : 0u;
                if (wide) {
                    if (in && q < p.P) store32(o + q, y);
                    if (in && q + 16 < p.P) store32(o + q + 16, y + 8);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (in && q + 8 * e < p.P) *(uint4 *)(o + q + 8 * e) = make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                }
            }
            if (it.tiles) {
                tc::tc_fence_before();
                __syncwarp();
                arrive_first(&sm.o_empty, lane);
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 0) {
        __syncwarp();
        tc::tmem_dealloc(tm, 256);
    }
    if (tid == 0 && sm.err) atomicExch(p.status + kStatusCode, (int)SSD_ERR_TIMEOUT);
}

template <int KB>
cudaError_t forward(const WindowParams &p, cudaStream_t s) {
    Maps maps;
    const int T = tile_tokens(p);
    cudaError_t e;
    if ((e = map_tokens(&maps.q, p.q, p, p.H, p.hpg, T)) != cudaSuccess) return e;
    if ((e = map_tokens(&maps.k, p.k, p, p.G, 1, Layout<KB>::kKeys)) != cudaSuccess) return e;
    if ((e = delta::same_tiles(&maps.v, maps.k, p.v)) != cudaSuccess) return e;
    if ((e = delta::allow_shared((const void *)window_fwd_kernel<KB>, Layout<KB>::kBytes)) != cudaSuccess) return e;
    const int per_row = (p.L + T - 1) / T, items = per_row * p.G * p.b;
    // the sign of the scale goes into the product, so that the largest score is the largest exponent; a scale of 0 is
    // kept off 0 for the masked ones, by the smallest number there is: no finite score makes more than 2^-20 of it
    const float c = fmaxf(fabsf(p.scale) * kLog2e, FLT_TRUE_MIN);
    window_fwd_kernel<KB><<<tile_grid(p, items, 2 * kSMs), kThreads, Layout<KB>::kBytes, s>>>(maps, p, c, p.scale < 0.f ? 1u << 13 : 0u,
                                                                                               items, per_row);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tile_forward(const WindowParams &p, cudaStream_t s) { return p.P > 64 ? forward<2>(p, s) : forward<1>(p, s); }

}  // namespace window
}  // namespace ssd
