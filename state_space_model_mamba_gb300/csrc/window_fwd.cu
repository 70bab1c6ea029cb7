// window_fwd.cu -- window attention, forward, on tcgen05.
//
// Blocks stay on their SM and take items in turn: two query tiles (window_tile.cuh) of one key group
// and the key tiles that they see.  Per tile pair S = Q K^T (128 x 128, fp32, tensor memory), the
// softmax's step, and O += P V.  One warp copies (TMA), one issues products, and two groups of four warps, a
// thread per row, take the softmax of one query tile each: while a group works on its S, the tensor core works on
// the other's.  P goes to tensor memory over the S that it came from, as the A operand; O stays there.
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

// Threads: two groups of softmax, then a group whose first two warps copy and issue.  That group gives up registers
// for a softmax thread's 128 scores: 2 * 128 * 216 + 128 * 72 = 384 * 168, what the block is launched with.
constexpr int kSoftmax = 256, kThreads = 384, kRegsSoftmax = 216, kRegsIssue = 72;
static_assert(kSoftmax * kRegsSoftmax + (kThreads - kSoftmax) * kRegsIssue <= kThreads * 168, "registers of the launch");
constexpr float kLazy = 8.f;  // log2 of what P may grow to

struct Maps {
    CUtensorMap q, k, v;
};

// KB = ceil(P / 64) blocks of 64 columns a tile.
template <int KB>
struct Layout {
    static constexpr int kTile = KB * 16384, kSlots = KB == 2 ? 5 : 8;
    static constexpr int kOffRing = 2 * kTile, kOffBars = kOffRing + kSlots * kTile;
    static constexpr int kBytes = kOffBars + 1024;
};
struct Bars {
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], o_empty[2], drain, kv_full[8], kv_empty[8];
    uint32_t tmem;
    int err;
};
static_assert(sizeof(Bars) <= 1024, "barriers");

// Two query tiles and their keys.
struct Item {
    int bi, g, V, head, lo, end, tiles_a, tiles;
    int ta[2], tb[2], first[2], last[2];
    bool on[2];
    __device__ __forceinline__ Item(const WindowParams &p, int index, int per_row) {
        const int T = tile_tokens(p), t0 = index % per_row * 2 * T;
        g = index / per_row % p.G;
        bi = index / per_row / p.G;
        V = __shfl_sync(0xffffffffu, valid_tokens(p, bi), 0);
        end = min(t0 + 2 * T, V);
        lo = max(0, t0 - p.W + 1);
        head = min(p.sinks, lo);
        tiles_a = (head + 127) / 128;
        tiles = t0 < V ? tiles_a + (end - lo + 127) / 128 : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ta[i] = t0 + i * T;
            tb[i] = min(ta[i] + T, V);
            on[i] = ta[i] < V;
            first[i] = max(0, ta[i] - p.W + 1);
            last[i] = on[i] ? tiles_a + (tb[i] - 1 - lo) / 128 : -1;
        }
    }
    __device__ __forceinline__ int start(int j) const { return j < tiles_a ? j * 128 : lo + (j - tiles_a) * 128; }
    __device__ __forceinline__ int count(int j) const { return min(128, (j < tiles_a ? head : end) - start(j)); }
    __device__ __forceinline__ bool need(const WindowParams &p, int i, int j) const {
        if (j > last[i]) return false;
        const int s = start(j);
        return s + count(j) > first[i] || s < p.sinks;
    }
};

template <int KB>
__global__ void __launch_bounds__(kThreads, 1) window_fwd_kernel(const __grid_constant__ Maps maps, WindowParams p, float c,
                                                                 uint32_t negate, int items, int per_row) {
    using Lay = Layout<KB>;
    extern __shared__ __align__(1024) char smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    Bars &sm = *(Bars *)(smem_raw + Lay::kOffBars);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], 1);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.o_full[i], 1);
            mbar_init(&sm.o_empty[i], 4);
        }
        for (int i = 0; i < Lay::kSlots; ++i) {
            mbar_init(&sm.kv_full[i], 1);
            mbar_init(&sm.kv_empty[i], 1);
        }
        mbar_init(&sm.drain, 1);
        tc::mbar_fence_init();
        sm.err = (base & 1023u) ? 1 : 0;
    }
    if (blockIdx.x == 0) write_status(p);
    if (warp == 0) {
        __syncwarp();
        tc::tmem_alloc(&sm.tmem, 512);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, sm.tmem, 0);  // S (and P) of tile i at column 128 i, O at 256 + 128 i
    bool ok = sm.err == 0;

    if (warp >= kSoftmax / 32) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (warp == kSoftmax / 32) {
            // ---- copies
            const uint32_t q_bytes = (uint32_t)(tile_tokens(p) * p.hpg) * 128u * KB;
            int n = 0, nq[2] = {0, 0};
            for (int index = blockIdx.x; index < items && ok; index += gridDim.x) {
                const Item it(p, index, per_row);
                auto load_q = [&](int i) {
                    if (!it.on[i] || !ok) return;
                    ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_empty[i], (nq[i] & 1) ^ 1));
                    if (ok && elect()) {
                        mbar_arrive_expect_tx(&sm.q_full[i], q_bytes);
                        for (int kb = 0; kb < KB; ++kb)
                            tma_tile(base + i * Lay::kTile + kb * 16384, &maps.q, &sm.q_full[i], 64 * kb, it.g * p.hpg, it.ta[i], it.bi);
                    }
                    if (ok) ++nq[i];
                };
                auto load_kv = [&](const CUtensorMap *map, int j) {
                    if (!ok) return;
                    const int slot = n % Lay::kSlots;
                    ok = __all_sync(0xffffffffu, mbar_wait(&sm.kv_empty[slot], ((n / Lay::kSlots) & 1) ^ 1));
                    if (ok && elect()) {
                        mbar_arrive_expect_tx(&sm.kv_full[slot], Lay::kTile);
                        for (int kb = 0; kb < KB; ++kb)
                            tma_tile(base + Lay::kOffRing + slot * Lay::kTile + kb * 16384, map, &sm.kv_full[slot], 64 * kb, it.g,
                                     it.start(j), it.bi);
                    }
                    if (ok) ++n;
                };
                if (it.tiles == 0) continue;
                load_q(0);
                load_kv(&maps.k, 0);
                load_q(1);
                load_kv(&maps.v, 0);
                for (int j = 1; j < it.tiles; ++j) {
                    load_kv(&maps.k, j);
                    load_kv(&maps.v, j);
                }
            }
            if (!ok) sm.err = 1;
            // copies in flight land before the block ends
            for (int x = max(0, n - Lay::kSlots); x < n; ++x) mbar_wait(&sm.kv_full[x % Lay::kSlots], (x / Lay::kSlots) & 1);
            for (int i = 0; i < 2; ++i)
                if (nq[i]) mbar_wait(&sm.q_full[i], (nq[i] - 1) & 1);
        } else if (warp == kSoftmax / 32 + 1) {
            // ---- products
            const uint32_t i_pv = tc::idesc_bf16(128, (p.P + 15) / 16 * 16, false, true);
            const int ksteps = (p.P + 15) / 16;
            // operands are the same for the whole warp and their descriptors differ by constants: an instruction then takes its
            // 64 cycles (measured; with addresses that the compiler takes for a lane's own it takes 104)
            const uint64_t d_q = tc::sdesc_kmajor(base, 0, 16384), d_k = tc::sdesc_kmajor(base + Lay::kOffRing, 0, 16384),
                           d_v = tc::sdesc_mnmajor(base + Lay::kOffRing, 0, 16384);
            int n = 0, nq[2] = {0, 0}, np[2] = {0, 0};
            for (int index = blockIdx.x; index < items && ok; index += gridDim.x) {
                const Item it(p, index, per_row);
                bool pending[2] = {false, false}, begun[2] = {false, false}, loaded[2] = {false, false};
                for (int j = 0; j <= it.tiles && ok && it.tiles; ++j) {
                    const int kslot = n % Lay::kSlots, vslot = (n + Lay::kSlots - 1) % Lay::kSlots;  // K of j, V of j - 1
                    const bool more = j < it.tiles;
                    if (more) ok = __all_sync(0xffffffffu, mbar_wait(&sm.kv_full[kslot], (n / Lay::kSlots) & 1));
                    const int nk = more ? (it.count(j) + 15) / 16 * 16 : 0;
                    const uint32_t i_s = tc::idesc_bf16(128, nk, false, false) | negate;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (pending[i] && ok) {
                            if (!begun[i]) ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_empty[i], (nq[i] & 1) ^ 1));
                            ok = __all_sync(0xffffffffu, ok && mbar_wait(&sm.p_full[i], np[i] & 1) &&
                                                             mbar_wait(&sm.kv_full[vslot], ((n - 1) / Lay::kSlots) & 1));
                            ++np[i];
                            tc::tc_fence_after();
                            if (ok && elect()) {
                                const int steps = (it.count(j - 1) + 15) / 16;
                                const uint64_t v = delta::sdesc_add(d_v, vslot * Lay::kTile);
#pragma unroll
                                for (int ks = 0; ks < 8; ++ks)
                                    if (ks < steps)
                                        tc::mma_bf16_tmem_a(tm + 256 + 128 * i, tm + 128 * i + 8 * ks, delta::sdesc_add(v, ks * 2048), i_pv,
                                                            begun[i] || ks > 0);
                                if (j - 1 == it.last[i]) tc::mma_commit(&sm.o_full[i]);
                            }
                            __syncwarp();
                            begun[i] = true;
                            pending[i] = false;
                        }
                        if (more && ok && it.need(p, i, j)) {
                            if (!loaded[i]) ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_full[i], nq[i] & 1));
                            loaded[i] = true;
                            tc::tc_fence_after();
                            if (ok && elect()) {
                                const uint64_t q = delta::sdesc_add(d_q, i * Lay::kTile), k = delta::sdesc_add(d_k, kslot * Lay::kTile);
#pragma unroll
                                for (int ks = 0; ks < 4 * KB; ++ks)
                                    if (ks < ksteps)
                                        tc::mma_bf16(tm + 128 * i, delta::sdesc_add(q, (ks >> 2) * 16384 + (ks & 3) * 32),
                                                     delta::sdesc_add(k, (ks >> 2) * 16384 + (ks & 3) * 32), i_s, ks > 0);
                                tc::mma_commit(&sm.s_full[i]);
                                if (j == it.last[i]) tc::mma_commit(&sm.q_empty[i]);
                            }
                            __syncwarp();
                            pending[i] = true;
                        }
                    }
                    if (ok && elect()) {
                        if (j > 0) tc::mma_commit(&sm.kv_empty[vslot]);
                        if (more) tc::mma_commit(&sm.kv_empty[kslot]);
                    }
                    __syncwarp();
                    if (more) n += 2;
                }
                for (int i = 0; i < 2; ++i) nq[i] += it.on[i];
            }
            if (!ok) sm.err = 1;
            if (elect()) tc::mma_commit(&sm.drain);
            __syncwarp();
            mbar_wait(&sm.drain, 0);
        }
    } else {
        // ---- softmax of query tile i
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int i = warp >> 2, row = tid & 127, quarter = warp & 3, R = p.hpg, T = tile_tokens(p);
        const uint32_t ts = tmem_addr(tm, 32 * quarter, 128 * i), to = ts + 256;
        int n = 0, ns = 0, no = 0;
        for (int index = blockIdx.x; index < items && ok; index += gridDim.x) {
            const Item it(p, index, per_row);
            const int t = it.ta[i] + row / R, h = it.g * R + row % R;
            const bool in = row < T * R && t < p.L, live = in && t < it.V;
            float m = -INFINITY, l = 0.f;
            if (it.on[i]) {
                const int tq = live ? t : it.ta[i];
                bool begun = false;
                for (int j = 0; j < it.tiles && ok; ++j, n += 2) {
                    if (!it.need(p, i, j)) continue;
                    const int s0 = it.start(j), nk = it.count(j);
                    // keys that every row sees: none behind the tile's first token, none in front of its last one's window
                    const bool plain = nk == 128 && s0 + 127 <= it.ta[i] && (s0 > it.tb[i] - 1 - p.W || s0 + 128 <= p.sinks);
                    ok = __all_sync(0xffffffffu, mbar_wait(&sm.s_full[i], ns & 1));
                    if (!ok) break;
                    tc::tc_fence_after();
                    ++ns;
                    const bool two = nk > 64;
                    float2 x[64];
                    tc::tmem_ld64(ts, (float *)x);
                    if (two) tc::tmem_ld64(ts + 64, (float *)(x + 32));
                    if (!plain) {
                        const int hi = min(nk, tq - s0 + 1), from = tq - p.W + 1 - s0, sk = p.sinks - s0;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (q >= 2 && !two) break;
                            const uint32_t see = bits_between(-32, hi - 32 * q) &
                                                 (bits_between(from - 32 * q, 32) | bits_between(-32, sk - 32 * q));
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float2 &y = x[16 * q + e];
                                y.x = see >> (2 * e) & 1 ? y.x : -INFINITY;
                                y.y = see >> (2 * e + 1) & 1 ? y.y : -INFINITY;
                            }
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], fmaxf(x[e].x, x[e].y));
                    if (two)
#pragma unroll
                        for (int e = 32; e < 64; ++e) mx[e & 3] = fmaxf(mx[e & 3], fmaxf(x[e].x, x[e].y));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const bool grows = top > m && (m == -INFINITY || (top - m) * c > kLazy);
                    if (!begun) {
                        m = top;
                        begun = true;
                    } else if (__any_sync(0xffffffffu, grows)) {  // products up to the last tile's are done: S came behind them
                        const float f = grows ? (m == -INFINITY ? 0.f : exp2_approx((m - top) * c)) : 1.f;
                        if (grows) m = top;
                        l *= f;
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
                    const float ref = m == -INFINITY ? 0.f : -m * c;
                    const float2 cc = make_float2(c, c), rr = make_float2(ref, ref), one = make_float2(1.f, 1.f);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (q >= 2 && !two) break;
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float2 y = ffma2(x[16 * q + e], cc, rr);
                            y = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                            sum[e & 1] = ffma2(y, one, sum[e & 1]);
                            pk[e] = tc::pack_bf2(y.x, y.y);
                        }
                        __syncwarp();
                        delta::tmem_st16(ts + 16 * q, (const float *)pk);
                    }
                    delta::tmem_wait_st();
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    if ((nk & 15) && (i == 0 || !it.need(p, 0, j))) {
                        // rows of V up to the product's step of 16: their probabilities are 0, so they have to be finite
                        const int slot = (n + 1) % Lay::kSlots, rows = 16 - (nk & 15);
                        ok = __all_sync(0xffffffffu, mbar_wait(&sm.kv_full[slot], ((n + 1) / Lay::kSlots) & 1));
                        const uint32_t v = base + Lay::kOffRing + slot * Lay::kTile;
                        for (int e = row; e < rows * 8 * KB; e += 128)
                            tc::st_shared_v4(v + (e / (8 * rows)) * 16384 + (nk + e / 8 % rows) * 128 + (e & 7) * 16, 0, 0, 0, 0);
                        tc::fence_async_smem();
                    }
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_full[i]);
                }
                if (!ok) break;
                ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_full[i], no & 1));
                if (!ok) break;
                tc::tc_fence_after();
                ++no;
            } else {
                n += 2 * it.tiles;
            }
            const float inv = live ? 1.f / l : 0.f;
            bf16 *o = (bf16 *)p.o + (((long long)it.bi * p.L + t) * p.H + h) * p.P;
            for (int q = 0; q < (p.P + 31) / 32; ++q) {
                float v[32];
                if (it.on[i]) {
                    __syncwarp();
                    tc::tmem_ld32u(to + 32 * q, (uint32_t *)v);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = 32 * q + 8 * e;
                    uint4 y = make_uint4(0u, 0u, 0u, 0u);
                    if (live)
                        y = make_uint4(tc::pack_bf2(v[8 * e] * inv, v[8 * e + 1] * inv), tc::pack_bf2(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                                       tc::pack_bf2(v[8 * e + 4] * inv, v[8 * e + 5] * inv), tc::pack_bf2(v[8 * e + 6] * inv, v[8 * e + 7] * inv));
                    if (in && col < p.P) *(uint4 *)(o + col) = y;
                }
            }
            if (it.on[i]) {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.o_empty[i]);
            }
            if (in && p.lse) p.lse[((long long)it.bi * p.H + h) * p.L + t] = live ? (m * c + log2f(l)) * kLn2 : 0.f;
        }
        if (!ok) sm.err = 1;
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
    if ((e = map_tokens(&maps.k, p.k, p, p.G, 1, 128)) != cudaSuccess) return e;
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
