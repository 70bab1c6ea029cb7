// delta_grad.cu -- dq and dk of the chunked gated delta rule, all chunks in
// parallel, and the gates' gradients from the sums that the two scans left.
//
// Per chunk and head, with D_ij = exp(gamma_i - gamma_j), the forward's S (before the
// chunk) and Z, the reverse pass's dS (after the chunk) and dV:
//     Nm_ij = scale D_ij beta_j (dO_i . Z_j), j <= i;    M_ij = -D_ij beta_j (dV_i . Z_j), j < i
//     dQ = scale e^gamma o (dO S^T) + Nm K
//     dK = -e^gamma o (dV S^T) + M K + Nm^T Q + M^T K + (beta e^(gamma_C - gamma) o Z) dS^T
// in three groups of products: [dO; dV] S^T (128 rows); [dO; dV] Z^T and [Q; K] K^T in its
// place, once the threads have added it, times its gate, to the sums; then, on top of the sums,
// whose rows 0 .. 63 are dQ and 64 .. 127 dK,
// [Nm; M] K, [0; W] dS^T with W = beta e^(gamma_C - gamma) o Z, and [0 | (Nm; M)]^T [Q; K] (the
// zero blocks keep the products that are dK's alone off the dQ rows).  The heads of a key
// group are walked by one block, which adds them up in tensor memory: dq and dk are written
// once, in a fixed order.  Every fp32 operand (Z, S, dS, dV, W, Nm, M) comes as hi + lo parts: what a token reads of
// S and what the chunk has written over it cancel, W and dS rounded once were 2.8e-3 of dk where its own rounding is
// 1.7e-3, and the share of dg that passes between tokens of the chunk is made here, as the sums that cross each token,
//     sum_{i >= t} sum_{j < t} P_ij,   P = Nm o Q K^T + M o K K^T:
// row sums less column sums would add up to the same, but leave the rounding of pairs that do not cross t, above
// all of the diagonal, which no decay makes small (heads at g = -8 and -12 throughout: dg 1e-3 and 5e-2 off).
// Two blocks share an SM, hide each other's copies and passes, and stay for the whole
// pass.  What bounds it: an item is 3.4 us of products (48 steps of 128 rows and columns, 20
// narrow ones) and six hand-overs, 7.2 us an item and SM with two in flight (3072 items of 24 heads,
// 4 x 2048: 145 us, 3.2 TB/s).  With W and dS rounded once and crossing sums as differences it took 122; against that,
// sums in registers spilled (64 a thread of 96) and took 150, masks a column at a time 135.
#include "delta_chunk.cuh"
#include "delta_mma.cuh"

namespace ssd {
namespace delta {
namespace {

using namespace tc;

constexpr int kCompute = 256, kThreads = kCompute + 32;
// shared memory: 64 rows of zeros; dV lo, then W hi; S hi, then [Nm; M] hi; Z hi, then 64 rows of zeros; Z lo, then
// W lo; S lo, then dS hi, then dS lo; dO and dV, then [Nm; M] lo; Q and K
constexpr uint32_t kOffZero = 0, kOffW = 8192, kOffSZ = 16384, kOffZ = kOffSZ + 16384, kOffP = kOffSZ, kOffZlo = 40960,
                   kOffDS = 49152, kOffDV = 65536, kOffPlo = kOffDV, kOffQK = 81920, kOffSmall = 114688;
struct alignas(16) Small {
    float beta[kChunk];  // as the image has them, one copy
    float2 gam[kChunk];
    uint64_t qk, in, ds, x, p, m[3], w;
    uint32_t tmem;
    int err;
};
constexpr uint32_t kGateBytes = 3 * kChunk * 4, kGateAt = 2 * kChunk * 4, kPartDS = kDStateTile / 2;
constexpr uint32_t kBytes = kOffSmall + sizeof(Small);
static_assert(2 * (kBytes + 1024) <= 233472, "two blocks per SM");
struct GradMaps {
    CUtensorMap k, q, d_o, dv;
};

// Blocks walk the units (b, group, chunk); within a unit the items (head, slice of 64 columns of P).
__global__ void __launch_bounds__(kThreads, 2) delta_grad_kernel(const ChunkParams cp, const __grid_constant__ GradMaps maps) {
    // no static shared memory and no slack for alignment: the window starts on a 1024-byte boundary
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Small &sm = *(Small *)(smem_raw + kOffSmall);
    uint64_t &bar_qk = sm.qk, &bar_in = sm.in, &bar_ds = sm.ds, &bar_x = sm.x, &bar_p = sm.p, &bar_w = sm.w;
    uint64_t(&bar_m)[3] = sm.m;
    const DeltaParams &p = cp.p;
    const uint32_t base = smem_u32(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nsl = slices_of(p), items = p.hpg * nsl, units = cp.n * p.G * p.b;
    if (tid == 0) {
        mbar_init(&bar_qk, 1);
        mbar_init(&bar_in, 1);
        mbar_init(&bar_ds, 1);
        mbar_init(&bar_p, kCompute / 32);
        mbar_init(&bar_x, kCompute / 32);
        for (int i = 0; i < 3; ++i) mbar_init(&bar_m[i], 1);
        mbar_init(&bar_w, 1);
        mbar_fence_init();
        sm.err = (base & 1023u) ? 1 : 0;
    }
    if (warp == 0) {
        __syncwarp();  // lane 0 may come from a branch of its own
        tmem_alloc(&sm.tmem, 256);
    }
    for (int i = tid; i < 8192 / 16; i += kThreads) st_shared_v4(base + kOffZero + 16 * i, 0, 0, 0, 0);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;
    const uint32_t halves = p.N > 64 ? 2u : 1u;
    bool ok = sm.err == 0;
    int u = 0, n = 0;  // live units and items so far: the barriers' phases

    if (warp == kCompute / 32) {
        // ---- copies and products
        struct Item {
            int chunk, bi, grp, h, slice;
            long long cs;
        };
        // item `it` of unit `unit`; of the next unit that is not all absent, where `it` is past its end
        auto item = [&](int &unit, int it, Item &x) {
            if (it >= items) {
                unit += gridDim.x;
                it = 0;
                while (unit < units && unit % cp.n * kChunk >= valid_tokens(p, unit / cp.n / p.G)) unit += gridDim.x;
            }
            if (unit >= units) return false;
            x.chunk = unit % cp.n;
            x.grp = unit / cp.n % p.G;
            x.bi = unit / cp.n / p.G;
            x.h = x.grp * p.hpg + it / nsl;
            x.slice = it % nsl;
            x.cs = ((long long)x.bi * p.H + x.h) * nsl + x.slice;
            return true;
        };
        auto load_qk = [&](const Item &x) {
            if (lane == 0) {
                mbar_arrive_expect_tx(&bar_qk, halves * 16384u);
                for (uint32_t kb = 0; kb < halves; ++kb) {
                    tma_tile(base + kOffQK + kb * 16384u, &maps.q, &bar_qk, 64 * kb, x.grp, x.chunk * kChunk, x.bi);
                    tma_tile(base + kOffQK + kb * 16384u + 8192u, &maps.k, &bar_qk, 64 * kb, x.grp, x.chunk * kChunk, x.bi);
                }
            }
        };
        auto load_in = [&](const Item &x) {
            if (lane == 0) {
                const char *state = cp.w.states + (x.cs * cp.n + x.chunk) * kStateTile;
                mbar_arrive_expect_tx(&bar_in, 16384 + kStateTile + kErrTile + kDvLoTile + kGateBytes);
                bulk_load(smem_u32(sm.beta), cp.image((long long)x.bi * p.H + x.h, x.chunk) + kGateAt, kGateBytes, &bar_in);
                bulk_load(base + kOffSZ, state, 16384, &bar_in);
                bulk_load(base + kOffZ, cp.w.errs + (x.cs * cp.n + x.chunk) * kErrTile, kErrTile, &bar_in);
                tma_tile(base + kOffDV, &maps.d_o, &bar_in, 64 * x.slice, x.h, x.chunk * kChunk, x.bi);
                tma_tile(base + kOffDV + 8192, &maps.dv, &bar_in, 64 * x.slice, x.h, x.chunk * kChunk, x.bi);
                bulk_load(base + kOffDS, state + 16384, 16384, &bar_in);
                bulk_load(base + kOffW, cp.w.dv_lo + (x.cs * cp.n + x.chunk) * kDvLoTile, kDvLoTile, &bar_in);
            }
        };
        auto prefetch = [&](const Item &x) {  // into L2
            if (lane == 0) {
                prefetch_bulk(cp.w.states + (x.cs * cp.n + x.chunk) * kStateTile, kStateTile);
                prefetch_bulk(cp.w.errs + (x.cs * cp.n + x.chunk) * kErrTile, kErrTile);
                prefetch_bulk(cp.w.dv_lo + (x.cs * cp.n + x.chunk) * kDvLoTile, kDvLoTile);
                prefetch_bulk(cp.w.dstates + (x.cs * cp.n + x.chunk) * kDStateTile, kDStateTile);
                prefetch_bulk(cp.image((long long)x.bi * p.H + x.h, x.chunk), kGates);
                prefetch_tile(&maps.d_o, 64 * x.slice, x.h, x.chunk * kChunk, x.bi);
                prefetch_tile(&maps.dv, 64 * x.slice, x.h, x.chunk * kChunk, x.bi);
            }
        };
        const uint32_t i_c = idesc_bf16(128, 64, false, false),
                       i_b = idesc_bf16(128, 128, false, false), i_d = idesc_bf16(128, 64 * halves, false, true),
                       i_e = idesc_bf16(128, 64 * halves, true, true);
        const uint64_t dDV = sdesc(base + kOffDV, 16, 1024), dSZ = sdesc(base + kOffSZ, 16, 1024),
                       dZ = sdesc(base + kOffZ, 16, 1024), dZlo = sdesc(base + kOffZlo, 16, 1024), dVlo = sdesc(base + kOffZero, 16, 1024),
                       dDS = sdesc(base + kOffDS, 16, 1024), dP = sdesc(base + kOffP, 16, 1024),
                       dPlo = sdesc(base + kOffPlo, 16, 1024), dK = sdesc(base + kOffQK + 8192, 16384, 1024),
                       dQKt = sdesc(base + kOffQK, 16384, 1024), dQK = sdesc(base + kOffQK, 16, 1024),
                       dKk = sdesc(base + kOffQK + 8192, 16, 1024);
        // (zeros | part of P)^T: the 64 zero rows serve both halves of the K index, the second with P 8 KB further away
        auto zeros_p = [&](uint32_t part, int ks) {
            return sdesc(base + kOffZero + (ks & 3) * 2048, part - kOffZero + (ks >> 2) * 8192, 1024);
        };
        const int nks = (p.N + 15) / 16;
        int unit = (int)blockIdx.x - (int)gridDim.x, loaded = 0;
        Item x;
        bool more = ok && item(unit, items, x);
        if (more) {
            load_qk(x);
            load_in(x);
            loaded = 1;
        }
        int qk_loaded = loaded, ds_loaded = 0, done = 0, it = 0;
        while (more) {
            const uint32_t ph = n & 1;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_in, ph)))) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16(tm, sdesc_add(dDV, ks * 32), sdesc_add(dSZ, ks * 32), i_b, ks > 0);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16(tm, sdesc_add(dDV, ks * 32), sdesc_add(dDS, ks * 32), i_b, true);  // S lo
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16(tm, sdesc_add(dVlo, ks * 32), sdesc_add(dSZ, ks * 32), i_b, true);
                mma_commit(&bar_m[0]);
            }
            // the item after this one
            int next_unit = unit, next_it = it + 1;
            Item y;
            const bool next = item(next_unit, next_it, y);
            if (next_it >= items) next_it = 0;
            if (next) prefetch(y);
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[0], ph)))) break;
            auto load_ds = [&](int part) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bar_ds, kPartDS);
                    bulk_load(base + kOffDS, cp.w.dstates + (x.cs * cp.n + x.chunk) * kDStateTile + part * kPartDS, kPartDS, &bar_ds);
                }
                ++ds_loaded;
            };
            load_ds(0);  // in place of S lo
            ok = mbar_wait(&bar_x, ph) && mbar_wait(&bar_qk, u & 1);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16(tm, sdesc_add(dDV, ks * 32), sdesc_add(dZ, ks * 32), i_c, ks > 0);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16(tm, sdesc_add(dDV, ks * 32), sdesc_add(dZlo, ks * 32), i_c, true);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16(tm, sdesc_add(dVlo, ks * 32), sdesc_add(dZ, ks * 32), i_c, true);
                for (int ks = 0; ks < nks; ++ks)
                    mma_bf16(tm + 64, sdesc_add(dQK, (ks >> 2) * 16384 + (ks & 3) * 32),
                             sdesc_add(dKk, (ks >> 2) * 16384 + (ks & 3) * 32), i_c, ks > 0);
                mma_commit(&bar_m[1]);
            }
            ok = mbar_wait(&bar_p, ph) && mbar_wait(&bar_ds, 0);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            if (lane == 0) {
                // W hi, where dV lo was, and W lo, where Z lo was, below zeros; then dS lo takes dS hi's place
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16(tm + 128, sdesc_add(dVlo, ks * 32), sdesc_add(dDS, ks * 32), i_b, true);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16(tm + 128, sdesc_add(dZ, ks * 32), sdesc_add(dDS, ks * 32), i_b, true);
                mma_commit(&bar_w);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16(tm + 128, sdesc_add(dP, ks * 32), sdesc_add(dK, ks * 2048), i_d, true);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16(tm + 128, sdesc_add(dPlo, ks * 32), sdesc_add(dK, ks * 2048), i_d, true);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) mma_bf16(tm + 128, zeros_p(kOffP, ks), sdesc_add(dQKt, ks * 2048), i_e, true);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) mma_bf16(tm + 128, zeros_p(kOffPlo, ks), sdesc_add(dQKt, ks * 2048), i_e, true);
            }
            __syncwarp();
            if ((ok = __all_sync(0xffffffffu, mbar_wait(&bar_w, ph)))) {  // beside the products with Nm and M
                load_ds(1);
                ok = __all_sync(0xffffffffu, mbar_wait(&bar_ds, 1));
                tc_fence_after();
            }
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    if (ok) mma_bf16(tm + 128, sdesc_add(dVlo, ks * 32), sdesc_add(dDS, ks * 32), i_b, true);
                mma_commit(&bar_m[2]);  // whatever failed: the products are waited for
            }
            __syncwarp();
            done = n + 1;
            if (!ok) break;
            if (next) {  // everything has been read
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[2], ph)))) break;
                load_in(y);
                ++loaded;
                if (next_unit != unit) {
                    load_qk(y);
                    ++qk_loaded;
                    ++u;
                }
            }
            more = next;
            unit = next_unit;
            it = next_it;
            x = y;
            ++n;
        }
        if (!ok) sm.err = 1;
        if (qk_loaded) mbar_wait(&bar_qk, (qk_loaded - 1) & 1);
        if (loaded) mbar_wait(&bar_in, (loaded - 1) & 1);
        if (ds_loaded) mbar_wait(&bar_ds, (ds_loaded - 1) & 1);
        if (done) mbar_wait(&bar_m[2], (done - 1) & 1);
    } else {
        const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane, i = row & 63;
        const bool keys = row >= kChunk;     // rows 64 .. 127: dV, M, dK
        for (int unit = blockIdx.x; unit < units && ok; unit += gridDim.x) {
            const int chunk = unit % cp.n, grp = unit / cp.n % p.G, bi = unit / cp.n / p.G;
            const int V = valid_tokens(p, bi), t0 = chunk * kChunk, live_n = V - t0, tok = t0 + i;
            const bool live = i < live_n;
            const uint32_t tx = tmem_addr(tm, 32 * quarter, 64 * half), tr = tx + 128;  // 64 columns of dO S^T and of the sums
            if (live_n > 0) {
                if (live_n < kChunk) {  // q and k rows of absent tokens are made zero
                    ok = __all_sync(0xffffffffu, mbar_wait(&bar_qk, u & 1));
                    for (int x = tid; x < 4 * kChunk * 8; x += kCompute)
                        if (((x >> 3) & 63) >= live_n) st_shared_v4(base + kOffQK + x * 16u, 0, 0, 0, 0);
                    fence_async_smem();  // before the products with them: what is masked below has to be finite
                }
                for (int it = 0; it < items && ok; ++it, ++n) {
                    const uint32_t ph = n & 1;
                    const long long bh = (long long)bi * p.H + grp * p.hpg + it / nsl, cs = bh * nsl + it % nsl;
                    ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[0], ph) && mbar_wait(&bar_in, ph) && mbar_wait(&bar_qk, u & 1));
                    if (!ok) break;
                    tc_fence_after();
                    const int wr = tid & 63, wc = 2 * (tid >> 6);
                    const float2 gi = sm.gam[i], gr = sm.gam[wr], gc = sm.gam[kChunk - 1];
                    const float wf = sm.beta[wr] * exp2_approx((gc.x - gr.x) + (gc.y - gr.y)), eg = exp2_approx(gi.x + gi.y);
                    const float f = keys ? -1.f : p.scale, fa = f * eg;
                    float read = 0.f;
                    if (half < (int)halves) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float2 a[8], b[8];
                            if (it > 0) {
                                tmem_ld16x2(tx + 16 * q, tr + 16 * q, (float *)a, (float *)b);
                            } else {
                                tmem_ld16(tx + 16 * q, (float *)a);
#pragma unroll
                                for (int e = 0; e < 8; ++e) b[e] = make_float2(0.f, 0.f);
                            }
                            // with the row's own q or k: what it reads of S
                            const uint32_t own = base + kOffQK + half * 16384;
#pragma unroll
                            for (int c = 0; c < 2; ++c) read = dot8(ld_shared_v4(own + sw128_chunk(row, 2 * q + c)), a + 4 * c, read);
#pragma unroll
                            for (int e = 0; e < 8; ++e) b[e] = ffma2(a[e], make_float2(fa, fa), b[e]);
                            __syncwarp();
                            tmem_st16(tr + 16 * q, (const float *)b);
                        }
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar_x);
                    (keys ? cp.w.fk : cp.w.fq)[(cs * 2 + half) * cp.n * kChunk + tok] = live ? fa * read : 0.f;
                    ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[1], ph));
                    if (!ok) break;
                    tc_fence_after();
                    // W hi in place of what dV lost, W lo and its zeros in place of Z (16 columns of row tid % 64)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float2 w[4];
                        const uint32_t off = sw128_chunk(wr, wc + c);
                        join8(ld_shared_v4(base + kOffZ + off), ld_shared_v4(base + kOffZlo + off), w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = fmul2(w[e], make_float2(wf, wf));
                        store_parts8(base + kOffW, base + kOffZlo, wr, wc + c, w);
                        st_shared_v4(base + kOffZ + off, 0, 0, 0, 0);
                    }
                    float before = 0.f, cs_[32];  // the row's sum so far; for t a column, what row i >= t has before t
                    const int limit = live ? (keys ? i : i + 1) : 0;  // the row's columns that count
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float2 a[8], b[8];
                        __syncwarp();
                        tmem_ld16x2(tmem_addr(tm, 32 * quarter, 32 * half + 16 * q),
                                    tmem_addr(tm, 32 * quarter, 64 + 32 * half + 16 * q), (float *)a, (float *)b);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int j = 32 * half + 16 * q + 2 * e;
                            const float4 gj = *(const float4 *)(sm.gam + j);
                            const float2 minus = make_float2(-1.f, -1.f), x = ffma2(make_float2(gj.x, gj.y), minus, gi),
                                         y = ffma2(make_float2(gj.z, gj.w), minus, gi);
                            const float2 d = fmul2(make_float2(exp2_approx(x.x + x.y), exp2_approx(y.x + y.y)), *(const float2 *)(sm.beta + j));
                            float2 v = fmul2(fmul2(a[e], make_float2(f, f)), d);
                            v.x = j < limit ? v.x : 0.f;
                            v.y = j + 1 < limit ? v.y : 0.f;
                            a[e] = v;
                            const float2 c = fmul2(v, b[e]);
                            cs_[16 * q + 2 * e] = j <= i ? before : 0.f;
                            cs_[16 * q + 2 * e + 1] = j < i ? before + c.x : 0.f;
                            before += c.x + c.y;
                        }
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            store_parts8(base + kOffP, base + kOffPlo, row, 4 * half + 2 * q + c, a + 4 * c);
                    }
                    fence_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar_p);
                    // column sums over the warp's rows: halves of the columns change hands until lane l has column l
#pragma unroll
                    for (int o = 16; o; o >>= 1) {
                        const bool up = lane & o;
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (e < o) {
                                const float give = up ? cs_[e] : cs_[e + o], keep = up ? cs_[e + o] : cs_[e];
                                cs_[e] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                            }
                    }
                    float *pe = cp.w.pe + (cs * cp.n + chunk) * kCrossSums;
                    if (half == 0) pe[row] = before;
                    pe[128 + quarter * 64 + 32 * half + lane] = cs_[0];
                }
                ++u;
            }
            if (live_n > 0 && ok) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bar_m[2], (n - 1) & 1));
                tc_fence_after();
            }
            bf16 *dst = (bf16 *)(keys ? p.dk : p.dq) + (((long long)bi * p.L + tok) * p.G + grp) * p.N + 64 * half;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float2 r[8];
                if (live_n > 0) {
                    __syncwarp();
                    tmem_ld16(tr + 16 * q, (float *)r);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (ok && tok < p.L && 64 * half + 16 * q + 8 * c < p.N)
                        *(uint4 *)(dst + 16 * q + 8 * c) = live ? pack8(r + 4 * c) : make_uint4(0, 0, 0, 0);
            }
        }
        if (!ok) sm.err = 1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && sm.err) atomicExch(p.status + kStatusCode, (int)SSD_ERR_TIMEOUT);
    if (warp == 0) {
        __syncwarp();  // lane 0 may come from a branch of its own
        tmem_dealloc(tm, 256);
    }
}

// dg and dbeta from the sums (delta_chunk.cuh): a warp per (b, h, chunk), lane l tokens 2 l and 2 l + 1.
__global__ void __launch_bounds__(256) delta_gate_grads(const ChunkParams cp) {
    const DeltaParams &p = cp.p;
    const long long w = blockIdx.x * 8LL + (threadIdx.x >> 5);
    if (w >= (long long)p.b * p.H * cp.n) return;
    const int lane = threadIdx.x & 31, chunk = (int)(w % cp.n), nsl = slices_of(p);
    const long long bh = w / cp.n;
    const int V = valid_tokens(p, (int)(bh / p.H)), t = chunk * kChunk + 2 * lane;
    float2 from = make_float2(0.f, 0.f), to = from, db = from;  // what tokens read, what they write
    float2 cross = from, first = from;  // pairs across a token; what the later half's rows read of the first half
    float ss = 0.f;
    if (chunk * kChunk < V) {
        for (int x = 0; x < 4 * nsl; ++x) {
            const long long at = (bh * nsl * 4 + x) * cp.n * kChunk + t;
            const float2 ww = *(const float2 *)(cp.w.ww + at), zx = *(const float2 *)(cp.w.zx + at);
            to.x += ww.x;
            to.y += ww.y;
            db.x += zx.x;
            db.y += zx.y;
        }
        for (int x = 0; x < 2 * nsl; ++x) {
            const long long at = (bh * nsl * 2 + x) * cp.n * kChunk + t;
            const float2 fq = *(const float2 *)(cp.w.fq + at), fk = *(const float2 *)(cp.w.fk + at);
            from.x += fq.x + fk.x;
            from.y += fq.y + fk.y;
        }
        for (int x = 0; x < nsl; ++x) {
            // the crossing pairs of rows in four quarters, columns of t's own half; the rows' sums over the first half
            const float *pe = cp.w.pe + ((bh * nsl + x) * cp.n + chunk) * kCrossSums + 2 * lane;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float2 c = *(const float2 *)(pe + 128 + 64 * y);
                cross.x += c.x;
                cross.y += c.y;
            }
            if (lane >= 16) {
                const float2 n = *(const float2 *)pe, m = *(const float2 *)(pe + 64);
                first.x += n.x + m.x;
                first.y += n.y + m.y;
            }
            if (lane < 16) ss += cp.w.ss[((bh * nsl + x) * cp.n + chunk) * 16 + lane];
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    float suffix = from.x + from.y, prefix = to.x + to.y, over = first.x + first.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float dn = __shfl_down_sync(0xffffffffu, suffix, o), up = __shfl_up_sync(0xffffffffu, prefix, o),
                    ov = __shfl_down_sync(0xffffffffu, over, o);
        if (lane + o < 32) suffix += dn, over += ov;
        if (lane >= o) prefix += up;
    }
    // the sums without this lane's tokens are its neighbours': its own may be larger by any factor, and would not come off again
    float next = __shfl_down_sync(0xffffffffu, suffix, 1), next_over = __shfl_down_sync(0xffffffffu, over, 1);
    prefix = __shfl_up_sync(0xffffffffu, prefix, 1);
    if (lane == 31) next = next_over = 0.f;
    if (lane == 0) prefix = 0.f;
    next += from.y;
    if (lane >= 16) {  // a token of the second half is crossed by all that the rows from it on have in the first
        cross.x += over;
        cross.y += next_over + first.y;
    }
    const long long at = bh * p.L + t;
    if (t < p.L) {
        p.dg[at] = t < V ? ss + prefix + suffix + cross.x : 0.f;
        p.dbeta[at] = t < V ? db.x : 0.f;
    }
    if (t + 1 < p.L) {
        p.dg[at + 1] = t + 1 < V ? ss + (prefix + to.x) + next + cross.y : 0.f;
        p.dbeta[at + 1] = t + 1 < V ? db.y : 0.f;
    }
}

}  // namespace

cudaError_t launch_chunk_grads(const ChunkParams &c, cudaStream_t s) {
    const DeltaParams &p = c.p;
    GradMaps maps;
    cudaError_t e;
    if ((e = map_chunk_tokens(&maps.k, p.k, p.b, p.L, p.G, p.N)) != cudaSuccess) return e;
    if ((e = same_tiles(&maps.q, maps.k, p.q)) != cudaSuccess) return e;
    if ((e = map_chunk_tokens(&maps.d_o, p.d_o, p.b, p.L, p.H, p.P)) != cudaSuccess) return e;
    if ((e = same_tiles(&maps.dv, maps.d_o, p.dv)) != cudaSuccess) return e;
    const int bytes = (int)kBytes;
    if ((e = allow_shared((const void *)delta_grad_kernel, bytes)) != cudaSuccess) return e;
    // two blocks per SM run at once; as many again for the SMs that other kernels give up later (2.04 ms for 2.11 of the
    // whole backward at 2 x 8192 x 80 heads, where the other half's scan holds SMs; no change elsewhere)
    const int units = c.n * p.G * p.b;
    delta_grad_kernel<<<units < 4 * kSMs ? units : 4 * kSMs, kThreads, bytes, s>>>(c, maps);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    delta_gate_grads<<<(unsigned)(((long long)p.b * p.H * c.n + 7) / 8), 256, 0, s>>>(c);
    return cudaGetLastError();
}

}  // namespace delta
}  // namespace ssd
