// window_fwd.cu -- window attention, forward, on tcgen05.
//
// Blocks stay on their SM and take items in turn: two query tiles (window_tile.cuh) of one key group
// and the key tiles that they see.  Per pair of tiles S = Q K^T (fp32, tensor memory), the softmax's
// step, and O += P V.  One warp copies (TMA), one issues products, and two groups of four warps, a
// thread per row, take the softmax of one query tile each.  S and P have columns of their own, so a
// group's next S is made as soon as it has its last one in registers, and the tensor core does not wait for the
// softmax's chain of instructions: 512 columns hold two S, two P and two O with 80 keys a tile where O
// has 128 columns, and 128 keys where it has 64.  (With P in place of S, 128 keys a tile, the products of a
// query tile waited for its softmax: 3570 cycles for 2 x 128 x 128 scores at P = 128, of which 2048 are products.)
// The row maximum is followed lazily: a row's reference only moves, and O is only rescaled, where the maximum
// has grown by 2^8 over it, so P <= 256 and the passes over O are rare; sums are fp32 and do not care.
// P is rounded to bf16 (2^-8 of each at most), the sum it is divided by is not.
#include "window_tile.cuh"

namespace ssd {
namespace window {
namespace {

using delta::exp2_approx;
using delta::tma_tile;
using tc::ffma2;
using tc::fmul2;
using tc::tmem_addr;

// Threads: two groups of softmax, then a group whose first warp copies, whose second issues S and whose others issue O.  An
// instruction costs its issuing thread some 55 cycles and a wait 100, so one thread could not keep the tensor core in work.
// That group gives up registers for a softmax thread's scores: 2 * 128 * 216 + 128 * 72 = 384 * 168, what the block is launched with.
constexpr int kSoftmax = 256, kThreads = 384, kRegsSoftmax = 216, kRegsIssue = 72;
static_assert(kSoftmax * kRegsSoftmax + (kThreads - kSoftmax) * kRegsIssue <= kThreads * 168, "registers of the launch");
constexpr float kLazy = 8.f;  // log2 of what P may grow to

struct Maps {
    CUtensorMap q, k, v;
};

// KB = ceil(P / 64) blocks of 64 columns a tile.
template <int KB>
struct Layout {
    static constexpr int kKeys = KB == 2 ? 80 : 128;                            // of a tile
    static constexpr int kBlock = kKeys * 128, kTile = KB * kBlock, kSlots = 6;  // ring of K and V tiles
    static constexpr int kQTile = KB * 16384;
    static constexpr int kOffRing = 2 * kQTile, kOffStage = kOffRing + kSlots * kTile;  // stage: 8 warps x 32 rows x 64 columns
    static constexpr int kOffBars = kOffStage + 8 * 4096, kBytes = kOffBars + 1024;
    // columns of tensor memory: S, P, O of tile i
    static constexpr int kS = 0, kP = 2 * kKeys, kO = 512 - 2 * 64 * KB, kOCols = 64 * KB;
    static_assert(kP + kKeys <= kO, "tensor memory");
    static_assert(kBytes <= 232448 && kSlots % 2 == 0, "shared memory; K in the even slots");
};
struct Bars {
    uint64_t q_full[2], q_empty[2], s_full[2], s_free[2], p_full[2], p_free[2], o_empty[2], drain, kv_full[8], kv_empty[8];
    uint32_t tmem;
    int err;
};
static_assert(sizeof(Bars) <= 1024, "barriers");

// Two query tiles and their keys: tiles [0, tiles_a) are sinks in front of the window, [tiles_a, tiles) the window.
template <int KEYS>
struct Item {
    int bi, g, V, head, lo, end, tiles_a, tiles;
    int ta[2], from[2], last[2];  // first token; first and last window tile that is seen (none: last < from)
    __device__ __forceinline__ Item(const WindowParams &p, const Cursor &c, int T) {
        const int t0 = c.x * 2 * T;
        g = c.g;
        bi = c.b;
        V = valid_tokens(p, bi);
        end = min(t0 + 2 * T, V);
        lo = max(0, t0 - p.W + 1);
        head = min(p.sinks, lo);
        tiles_a = (head + KEYS - 1) / KEYS;
        tiles = t0 < V ? tiles_a + (end - lo + KEYS - 1) / KEYS : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ta[i] = t0 + i * T;
            // sinks inside the window's first tiles: all of them are taken, the masks do the rest
            from[i] = tiles_a + (lo < p.sinks ? 0 : (max(0, ta[i] - p.W + 1) - lo) / KEYS);
            last[i] = on(i) ? tiles_a + (min(ta[i] + T, V) - 1 - lo) / KEYS : -1;
        }
    }
    __device__ __forceinline__ bool on(int i) const { return ta[i] < V; }
    __device__ __forceinline__ int start(int j) const { return j < tiles_a ? j * KEYS : lo + (j - tiles_a) * KEYS; }
    __device__ __forceinline__ int count(int j) const { return min(KEYS, (j < tiles_a ? head : end) - start(j)); }
    __device__ __forceinline__ bool need(int i, int j) const { return j <= last[i] && (j < tiles_a || j >= from[i]); }
};
template <int KB>
__global__ void __launch_bounds__(kThreads, 1) window_fwd_kernel(const __grid_constant__ Maps maps, WindowParams p, float c,
                                                                 uint32_t negate, int items, int per_row) {
    using Lay = Layout<KB>;
    constexpr int KEYS = Lay::kKeys, SLOTS = Lay::kSlots;
    using It = Item<KEYS>;
    extern __shared__ __align__(1024) char smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    Bars &sm = *(Bars *)(smem_raw + Lay::kOffBars);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], 1);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_free[i], 4);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.p_free[i], 1);
            mbar_init(&sm.o_empty[i], 4);
        }
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&sm.kv_full[i], 1);
            mbar_init(&sm.kv_empty[i], i & 1 ? 2 : 1);  // K: the thread of S; V: both threads of O
        }
        mbar_init(&sm.drain, 3);
        tc::mbar_fence_init();
        sm.err = 0;
    }
    if (blockIdx.x == 0) write_status(p);
    if (warp == 0) {
        __syncwarp();
        tc::tmem_alloc(&sm.tmem, 512);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, sm.tmem, 0);
    const int T = tile_tokens(p);
    int *const err = &sm.err;

    if (warp >= kSoftmax / 32) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (warp == kSoftmax / 32) {
            // ---- copies, one thread
            if (elect()) {
                const uint32_t q_bytes = (uint32_t)(T * p.hpg) * 128u * KB;
                Place<SLOTS> at;
                uint32_t nq[2] = {0, 0};
                int loaded = 0;
                for (Cursor cur(items, per_row, p.G); cur.left > 0; cur.next(per_row, p.G)) {
                    const It it(p, cur, T);
                    if (it.tiles == 0) continue;
                    auto load_q = [&](int i) {
                        if (!it.on(i)) return;
                        wait_bar(&sm.q_empty[i], (nq[i] & 1) ^ 1, err);
                        mbar_arrive_expect_tx(&sm.q_full[i], q_bytes);
                        for (int kb = 0; kb < KB; ++kb)
                            tma_tile(base + i * Lay::kQTile + kb * 16384, &maps.q, &sm.q_full[i], 64 * kb, it.g * p.hpg, it.ta[i], it.bi);
                        ++nq[i];
                    };
                    for (int x = 0; x < 2 * it.tiles; ++x) {
                        if (x < 2) load_q(x);
                        wait_bar(&sm.kv_empty[at.slot], at.phase ^ 1, err);
                        mbar_arrive_expect_tx(&sm.kv_full[at.slot], Lay::kTile);
                        for (int kb = 0; kb < KB; ++kb)
                            tma_tile(base + Lay::kOffRing + at.slot * Lay::kTile + kb * Lay::kBlock, x & 1 ? &maps.v : &maps.k,
                                     &sm.kv_full[at.slot], 64 * kb, it.g, it.start(x >> 1), it.bi);
                        at.next();
                        ++loaded;
                    }
                }
                // copies in flight land before the block ends
                for (int x = max(0, loaded - SLOTS); x < loaded; ++x) mbar_wait(&sm.kv_full[x % SLOTS], (x / SLOTS) & 1);
                for (int i = 0; i < 2; ++i)
                    if (nq[i]) mbar_wait(&sm.q_full[i], (nq[i] - 1) & 1);
            }
            __syncwarp();
        } else if (warp == kSoftmax / 32 + 1) {
            // ---- products S = Q K^T, one thread
            if (elect()) {
                const uint32_t i_s0 = tc::idesc_bf16(128, 0, false, false) | negate;
                const int ksteps = (p.P + 15) / 16;
                const uint64_t d_q = tc::sdesc(base, 16, 1024), d_k = tc::sdesc(base + Lay::kOffRing, 16, 1024);
                Place<SLOTS> at;
                uint32_t nq[2] = {0, 0}, ns[2] = {0, 0};
                for (Cursor cur(items, per_row, p.G); cur.left > 0; cur.next(per_row, p.G)) {
                    const It it(p, cur, T);
                    bool loaded[2] = {false, false};
                    for (int j = 0; j < it.tiles; ++j) {
                        wait_bar(&sm.kv_full[at.slot], at.phase, err);
                        const uint32_t i_s = i_s0 | (uint32_t)((it.count(j) + 15) >> 4) << 18;  // N / 8 from bit 17
                        const uint64_t k = delta::sdesc_add(d_k, at.slot * Lay::kTile);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (!it.need(i, j)) continue;
                            if (!loaded[i]) wait_bar(&sm.q_full[i], nq[i] & 1, err);
                            loaded[i] = true;
                            wait_bar(&sm.s_free[i], (ns[i] & 1) ^ 1, err);
                            ++ns[i];
                            tc::tc_fence_after();
                            const uint64_t q = delta::sdesc_add(d_q, i * Lay::kQTile);
#pragma unroll
                            for (int ks = 0; ks < 4 * KB; ++ks)
                                if (ks < ksteps)
                                    tc::mma_bf16(tm + Lay::kS + KEYS * i, delta::sdesc_add(q, (ks >> 2) * 16384 + (ks & 3) * 32),
                                                 delta::sdesc_add(k, (ks >> 2) * Lay::kBlock + (ks & 3) * 32), i_s, ks > 0);
                            tc::mma_commit(&sm.s_full[i]);
                            if (j == it.last[i]) tc::mma_commit(&sm.q_empty[i]);
                        }
                        tc::mma_commit(&sm.kv_empty[at.slot]);
                        at.next(), at.next();
                    }
                    for (int i = 0; i < 2; ++i) nq[i] += it.on(i) && it.tiles;
                }
                tc::mma_commit(&sm.drain);
                mbar_wait(&sm.drain, 0);
            }
            __syncwarp();
        } else {
            // ---- products O += P V of query tile i, one thread
            if (elect()) {
                const int i = warp - (kSoftmax / 32 + 2);
                const uint32_t i_pv = tc::idesc_bf16(128, (p.P + 15) / 16 * 16, false, true);
                const uint64_t d_v = tc::sdesc(base + Lay::kOffRing, Lay::kBlock, 1024);
                const uint32_t to = tm + Lay::kO + Lay::kOCols * i, tp = tm + Lay::kP + KEYS / 2 * i;
                Place<SLOTS> at;
                at.next();
                uint32_t no = 0, np = 0;
                for (Cursor cur(items, per_row, p.G); cur.left > 0; cur.next(per_row, p.G)) {
                    const It it(p, cur, T);
                    bool begun = false;
                    for (int j = 0; j < it.tiles; ++j) {
                        wait_bar(&sm.kv_full[at.slot], at.phase, err);
                        if (it.need(i, j)) {
                            if (!begun) wait_bar(&sm.o_empty[i], (no & 1) ^ 1, err);
                            wait_bar(&sm.p_full[i], np & 1, err);
                            ++np;
                            tc::tc_fence_after();
                            const int steps = (it.count(j) + 15) >> 4;
                            const uint64_t v = delta::sdesc_add(d_v, at.slot * Lay::kTile);
#pragma unroll
                            for (int ks = 0; ks < KEYS / 16; ++ks)
                                if (ks < steps) tc::mma_bf16_tmem_a(to, tp + 8 * ks, delta::sdesc_add(v, ks * 2048), i_pv, begun || ks > 0);
                            tc::mma_commit(&sm.p_free[i]);
                            tc::mma_commit(&sm.kv_empty[at.slot]);
                            begun = true;
                        } else {
                            mbar_arrive(&sm.kv_empty[at.slot]);
                        }
                        at.next(), at.next();
                    }
                    no += it.on(i) && it.tiles;
                }
                tc::mma_commit(&sm.drain);
                mbar_wait(&sm.drain, 0);
            }
            __syncwarp();
        }
    } else {
        // ---- softmax of query tile i
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int i = warp >> 2, row = tid & 127, quarter = warp & 3, R = p.hpg;
        const uint32_t magic = row_magic(R), stage = base + Lay::kOffStage + warp * 4096;
        const uint32_t ts = tmem_addr(tm, 32 * quarter, Lay::kS + KEYS * i), tp = tmem_addr(tm, 32 * quarter, Lay::kP + KEYS / 2 * i),
                       to = tmem_addr(tm, 32 * quarter, Lay::kO + Lay::kOCols * i);
        int n = 0, ns = 0;
        for (Cursor cur(items, per_row, p.G); cur.left > 0; cur.next(per_row, p.G)) {
            const It it(p, cur, T);
            const int token = row_token(row, magic), t = it.ta[i] + token, h = it.g * R + row - token * R;
            const bool in = row < T * R && t < p.L, live = in && t < it.V;
            float m = -INFINITY, l = 0.f;
            if (it.on(i)) {
                const int tq = live ? t : it.ta[i];
                bool begun = false;
                for (int j = it.tiles_a ? 0 : it.from[i]; j <= it.last[i]; j = j + 1 == it.tiles_a ? it.from[i] : j + 1) {
                    const int s0 = it.start(j), nk = it.count(j);
                    // keys that every row sees: none behind the tile's first token, none in front of its last one's window
                    const bool plain = nk == KEYS && s0 + KEYS - 1 <= it.ta[i] && (s0 > it.ta[i] + T - 1 - p.W || s0 + KEYS <= p.sinks);
                    wait_warp(&sm.s_full[i], ns & 1, err);
                    tc::tc_fence_after();
                    float2 x[KEYS / 2];
                    if constexpr (KEYS == 80)
                        tmem_ld80(ts, (float *)x);
                    else
                        tmem_ld128(ts, (float *)x);
                    tc::tc_fence_before();
                    arrive_first(&sm.s_free[i], lane);
                    if (!plain) {
                        const int hi = min(nk, tq - s0 + 1), from = tq - p.W + 1 - s0, sk = p.sinks - s0;
#pragma unroll
                        for (int q = 0; q < (KEYS + 31) / 32; ++q) {  // past nk all of them
                            const uint32_t see = bits_between(-32, hi - 32 * q) &
                                                 (bits_between(from - 32 * q, 32) | bits_between(-32, sk - 32 * q));
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                if (16 * q + e >= KEYS / 2) break;
                                float2 &y = x[16 * q + e];
                                y.x = see >> (2 * e) & 1 ? y.x : -INFINITY;
                                y.y = see >> (2 * e + 1) & 1 ? y.y : -INFINITY;
                            }
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < KEYS / 2; ++e) mx[e & 3] = fmaxf(mx[e & 3], fmaxf(x[e].x, x[e].y));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    // the product with the last P is done: P and O are this group's
                    wait_warp(&sm.p_free[i], (ns & 1) ^ 1, err);
                    tc::tc_fence_after();
                    ++ns;
                    const bool grows = top > m && (m == -INFINITY || (top - m) * c > kLazy);
                    const float f = m == -INFINITY ? 0.f : exp2_approx((m - top) * c);
                    m = grows ? top : m;
                    l = grows ? l * f : l;
                    if (begun && __any_sync(0xffffffffu, grows)) {
                        const float g = grows ? f : 1.f;
                        for (int q = 0; q < (p.P + 15) / 16; ++q) {
                            float o[16];
                            __syncwarp();
                            tc::tmem_ld16(to + 16 * q, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= g;
                            delta::tmem_st16(to + 16 * q, o);
                        }
                        delta::tmem_wait_st();
                    }
                    begun = true;
                    const float ref = m == -INFINITY ? 0.f : -m * c;
                    const float2 cc = make_float2(c, c), rr = make_float2(ref, ref), one = make_float2(1.f, 1.f);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int q = 0; q < (KEYS + 31) / 32; ++q) {
                        constexpr int kLast = KEYS % 32 ? KEYS % 32 / 2 : 16;  // pairs of the last chunk
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (q == KEYS / 32 && e >= kLast) break;
                            float2 y = ffma2(x[16 * q + e], cc, rr);
                            y = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                            sum[e & 1] = ffma2(y, one, sum[e & 1]);
                            pk[e] = tc::pack_bf2(y.x, y.y);
                        }
                        if (q == KEYS / 32)
                            tmem_st8(tp + 16 * q, pk);
                        else
                            delta::tmem_st16(tp + 16 * q, (const float *)pk);
                    }
                    delta::tmem_wait_st();
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    if ((nk & 15) && (i == 0 || !it.need(0, j))) {
                        // rows of V up to the product's step of 16: their probabilities are 0, so they have to be finite
                        const int slot = (n + 2 * j + 1) % SLOTS, rows = 16 - (nk & 15);
                        wait_warp(&sm.kv_full[slot], ((n + 2 * j + 1) / SLOTS) & 1, err);
                        const uint32_t v = base + Lay::kOffRing + slot * Lay::kTile;
                        for (int e = row; e < rows * 8 * KB; e += 128)
                            tc::st_shared_v4(v + (e / (8 * rows)) * Lay::kBlock + (nk + e / 8 % rows) * 128 + (e & 7) * 16, 0, 0, 0, 0);
                        tc::fence_async_smem();
                        __syncwarp();
                    }
                    tc::tc_fence_before();
                    arrive_first(&sm.p_full[i], lane);
                }
                // the last product: p_free's phase that the next item's first tile waits for too
                wait_warp(&sm.p_free[i], (ns & 1) ^ 1, err);
                tc::tc_fence_after();
            }
            n += 2 * it.tiles;
            if (in && p.lse) p.lse[((long long)it.bi * p.H + h) * p.L + t] = live ? (m * c + log2f(l)) * kLn2 : 0.f;
            const float inv = live ? 1.f / l : 0.f;
            // O in bf16, 64 columns at a time through the warp's stage, so that a row leaves as whole lines
            bf16 *const o = (bf16 *)p.o + (((long long)it.bi * p.L + it.ta[i]) * p.H + it.g * R) * p.P;
            const int rows = min(T, p.L - it.ta[i]) * R;  // of the tile that there are
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float v[32];
                    if (it.on(i)) {
                        tc::tmem_ld32u(to + 64 * kb + 32 * q, (uint32_t *)v);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = 0.f;
                    }
                    uint32_t y[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] = live ? tc::pack_bf2(v[2 * e] * inv, v[2 * e + 1] * inv) : 0u;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        tc::st_shared_v4(stage + tc::sw128_chunk(lane, 4 * q + e), y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                }
                __syncwarp();
                if (kb == KB - 1 && it.on(i)) {
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.o_empty[i]);
                }
                const int col = 64 * kb + 8 * (lane & 7);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = 4 * e + (lane >> 3), rr = 32 * quarter + r;
                    const uint4 y = tc::ld_shared_v4(stage + tc::sw128_chunk(r, lane & 7));
                    if (rr < rows && col < p.P) *(uint4 *)(o + row_token(rr, magic) * (p.H - R) * p.P + rr * p.P + col) = y;
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

template <int KB>
cudaError_t forward(const WindowParams &p, cudaStream_t s) {
    Maps maps;
    const int T = tile_tokens(p);
    cudaError_t e;
    if ((e = map_tokens(&maps.q, p.q, p, p.H, p.hpg, T)) != cudaSuccess) return e;
    if ((e = map_tokens(&maps.k, p.k, p, p.G, 1, Layout<KB>::kKeys)) != cudaSuccess) return e;
    if ((e = delta::same_tiles(&maps.v, maps.k, p.v)) != cudaSuccess) return e;
    if ((e = delta::allow_shared((const void *)window_fwd_kernel<KB>, Layout<KB>::kBytes)) != cudaSuccess) return e;
    const int per_row = (p.L + 2 * T - 1) / (2 * T), items = per_row * p.G * p.b;
    // the sign of the scale goes into the product, so that the largest score is the largest exponent; a scale of 0 is
    // kept off 0 for the masked ones
    const float c = fmaxf(fabsf(p.scale) * kLog2e, 1e-30f);
    window_fwd_kernel<KB><<<items < kSMs ? items : kSMs, kThreads, Layout<KB>::kBytes, s>>>(maps, p, c, p.scale < 0.f ? 1u << 13 : 0u,
                                                                                       items, per_row);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tile_forward(const WindowParams &p, cudaStream_t s) { return p.P > 64 ? forward<2>(p, s) : forward<1>(p, s); }

}  // namespace window
}  // namespace ssd
