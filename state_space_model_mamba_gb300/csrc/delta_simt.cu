// delta_simt.cu -- the gated delta rule token by token on CUDA cores: the fp32
// path, shapes outside the tensor-core kernels, and the one-token step.
//
// Every row p of the state S [P, N] is a recurrence of its own,
//     s <- a s + beta (v_p - a s.k) k,   o_p = scale s.q,
// so rows are spread over the grid: 8 lanes hold one row (N / 8 elements each
// in registers, 4-element pieces interleaved over the lanes so that a row's
// load is one 128-byte line per piece), 32 or 8 rows a block.  What bounds the
// sequence kernels is a warp's own instructions, some 70 a token and three cycles each, in the
// token's order: the sums over the lanes are taken four tokens at a time, and the next tokens are
// loaded meanwhile.  Measured in fp32: 2 x 515 tokens, 4 heads of 32 x 48: 71 us (token by token, without
// loads ahead: 174); its backward, 2 x 129: 15 + 50 + 3 us (44 + 118 + 3).  The step kernel
// reads and writes each state once and is bound by HBM: 192 requests of 80 heads, 64 x 128, 1.01 GB in
// 150 us, 6.7 TB/s, as a copy.
#include <stdio.h>

#include "delta_internal.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace delta {
namespace {

constexpr int kLanes = 8;   // lanes per row
// State rows R per block: 32, or 8 where blocks of 32 would leave SMs without one.  A block's warps share its
// schedulers and shared memory (four tokens' keys are 100 of its cycles for every warp): 2 x 515 tokens of 4 heads,
// 32 rows each, took 92 us in 8 blocks, 74 in 32.
inline int rows_of(long long heads, int P) { return heads * ((P + 31) / 32) < 152 ? 8 : 32; }
// Tokens staged in shared memory at a time, also the tokens between kept states of the backward, whose
// states inside a segment have to fit in shared memory too.
constexpr int tok_of(int nc) { return nc > 4 ? 4 : (nc > 2 ? 8 : 16); }

__device__ __forceinline__ float sum8(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    return x;
}
// in pairs: a warp has a scheduler to itself where heads are few, and each instruction costs it three cycles
using tc::ffma2;
using tc::fmul2;
__device__ __forceinline__ float2 lo2(float4 x) { return make_float2(x.x, x.y); }
__device__ __forceinline__ float2 hi2(float4 x) { return make_float2(x.z, x.w); }
__device__ __forceinline__ float2 dot4(float4 a, float4 b, float2 acc) { return ffma2(hi2(a), hi2(b), ffma2(lo2(a), lo2(b), acc)); }
__device__ __forceinline__ float4 axpy4(float a, float4 x, float4 y) {
    const float2 aa = make_float2(a, a), l = ffma2(aa, lo2(x), lo2(y)), h = ffma2(aa, hi2(x), hi2(y));
    return make_float4(l.x, l.y, h.x, h.y);
}
__device__ __forceinline__ float4 scale4(float a, float4 x) {
    const float2 aa = make_float2(a, a), l = fmul2(aa, lo2(x)), h = fmul2(aa, hi2(x));
    return make_float4(l.x, l.y, h.x, h.y);
}

// Tokens [t0, t0 + nt) of one (b, h, row block) in shared memory: q and k rows
// (N, zero-padded to 32 NC), v (and do) of the block's rows, decay and beta.
template <int NC, bool BWD, int R>
struct Stage {
    static constexpr int kTok = tok_of(NC);
    float4 q[kTok][NC * kLanes], k[kTok][NC * kLanes];
    float v[kTok][R];
    float dO[BWD ? kTok : 1][R];
    float a[kTok], beta[kTok];
};

// A stage on its way to shared memory: a thread's pieces in registers, loaded while the stage before is worked on.
template <typename T, int NC, bool BWD, int R>
struct Fetch {
    static constexpr int kThreads = R * kLanes, kTok = tok_of(NC), kKeys = (kTok * NC * kLanes + kThreads - 1) / kThreads,
                         kVals = (kTok * R + kThreads - 1) / kThreads;
    float4 q[kKeys], k[kKeys];
    float v[kVals], dO[BWD ? kVals : 1], a, beta;
    __device__ __forceinline__ void load(const DeltaParams &p, int bi, int h, int row0, int t0, int nt) {
        const int tid = threadIdx.x % kThreads;
        const int g = h / p.hpg, nq = p.N / 4;
#pragma unroll
        for (int x = 0; x < kKeys; ++x) {
            const int i = tid + x * kThreads, t = i / (NC * kLanes), c = i % (NC * kLanes);
            const long long at = (((long long)bi * p.L + t0 + t) * p.G + g) * p.N + 4 * c;
            q[x] = k[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < nt && c < nq) {
                q[x] = load4((const T *)p.q + at);
                k[x] = load4((const T *)p.k + at);
            }
        }
#pragma unroll
        for (int x = 0; x < kVals; ++x) {
            const int i = tid + x * kThreads, t = i / R, r = i % R;
            const long long at = (((long long)bi * p.L + t0 + t) * p.H + h) * p.P + row0 + r;
            const bool in = t < nt && row0 + r < p.P;
            v[x] = in ? load1((const T *)p.v + at) : 0.f;
            if (BWD) dO[x] = in ? p.scale * load1((const T *)p.d_o + at) : 0.f;
        }
        a = 1.f, beta = 0.f;  // an absent token leaves the state as it is
        if (tid < nt) {
            const long long at = ((long long)bi * p.H + h) * p.L + t0 + tid;
            a = expf(clamp_log_decay(p.g[at]));
            beta = p.beta[at];
        }
    }
    __device__ __forceinline__ void store(Stage<NC, BWD, R> &s) const {
        const int tid = threadIdx.x % kThreads;
#pragma unroll
        for (int x = 0; x < kKeys; ++x) {
            const int i = tid + x * kThreads;
            if (i < kTok * NC * kLanes) {
                (&s.q[0][0])[i] = q[x];
                (&s.k[0][0])[i] = k[x];
            }
        }
#pragma unroll
        for (int x = 0; x < kVals; ++x) {
            const int i = tid + x * kThreads;
            if (i < kTok * R) {
                (&s.v[0][0])[i] = v[x];
                if (BWD) (&s.dO[0][0])[i] = dO[x];
            }
        }
        if (tid < kTok) {
            s.a[tid] = a;
            s.beta[tid] = beta;
        }
    }
};

template <int NC>
__device__ __forceinline__ void load_row(float4 (&s)[NC], const float *src, bool in, int N, int lane) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = 4 * (i * kLanes + lane);
        s[i] = (src && in && c < N) ? *(const float4 *)(src + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
template <int NC>
__device__ __forceinline__ void store_row(const float4 (&s)[NC], float *dst, bool in, int N, int lane) {
    if (!dst || !in) return;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = 4 * (i * kLanes + lane);
        if (c < N) *(float4 *)(dst + c) = s[i];
    }
}

// ------------------------------------------------------------------ forward
// Grid: one block per (b, h, row block).  Without outputs it is the backward's recompute: `kept` gets the
// state before every segment of tok_of(NC) tokens ([b, H, segments, P, N]).
template <typename T, int NC, int R, bool OUT>
__global__ void __launch_bounds__(R * kLanes) delta_rows_fwd(DeltaParams p, float *kept, int nseg) {
    constexpr int kTok = tok_of(NC), kThreads = R * kLanes;
    __shared__ Stage<NC, false, R> stages[2];
    __shared__ float outs[2][kTok][R], gram[kTok / 4][8];
    const int nblk = (p.P + R - 1) / R, bh = blockIdx.x / nblk, bi = bh / p.H, h = bh % p.H;
    const int row0 = (blockIdx.x % nblk) * R;
    const int row = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const bool in = row0 + row < p.P;
    const int V = valid_tokens(p, bi);
    if (blockIdx.x == 0) write_status(p, p.b);
    const long long srow = ((long long)bh * p.P + row0 + row) * p.N;
    float4 s[NC];
    load_row(s, p.init ? p.init + srow : nullptr, in, p.N, lane);
    Fetch<T, NC, false, R> next;
    if (V > 0) {
        next.load(p, bi, h, row0, 0, min(kTok, V));
        next.store(stages[0]);
    }
    __syncthreads();
    for (int t0 = 0, cur = 0; t0 < V; t0 += kTok, cur ^= 1) {
        const int nt = min(kTok, V - t0);
        const Stage<NC, false, R> &st = stages[cur];
        float(*out)[R] = outs[cur];
        if (t0 + kTok < V) next.load(p, bi, h, row0, t0 + kTok, min(kTok, V - t0 - kTok));
        if (!OUT)
            store_row(s, kept + (((long long)bh * nseg + t0 / kTok) * p.P + row0 + row) * p.N, in, p.N, lane);
        // k_i.k_j inside each four tokens, a pair per row of lanes
        constexpr int kPairs = kTok / 4 * 6;
#pragma unroll
        for (int y = 0; y < (kPairs + R - 1) / R; ++y) {  // by whole warps: rows past the last pair take it again
            const int x = min(row + y * R, kPairs - 1);
            const int pair = x % 6, i = pair < 3 ? 0 : (pair < 5 ? 1 : 2), j = pair < 3 ? pair + 1 : (pair < 5 ? pair - 1 : 3);
            float2 g2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < NC; ++c) g2 = dot4(st.k[x / 6 * 4 + i][c * kLanes + lane], st.k[x / 6 * 4 + j][c * kLanes + lane], g2);
            const float g = sum8(g2.x + g2.y);
            if (lane == 0) gram[x / 6][pair] = g;
        }
        __syncthreads();
        // Four tokens a time: the sums s.k of all four from the state before them, one chain of shuffles (beside it
        // those of what the four before have read); what the tokens between write comes in by the pairs' products.
        float od[4] = {0.f, 0.f, 0.f, 0.f};
        for (int t = 0; t < nt; t += 4) {
            float d[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 d2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < NC; ++i) d2 = dot4(s[i], st.k[t + j][i * kLanes + lane], d2);
                d[j] = d2.x + d2.y;
            }
            const float4 a = *(const float4 *)(st.a + t), be = *(const float4 *)(st.beta + t);
            const float *g = gram[t / 4];
            const float g01 = g[0], g02 = g[1], g03 = g[2], g12 = g[3], g13 = g[4], g23 = g[5];
            const float v0 = st.v[t][row], v1 = st.v[t + 1][row], v2 = st.v[t + 2][row], v3 = st.v[t + 3][row];
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    d[j] += __shfl_xor_sync(0xffffffffu, d[j], o);
                    if (OUT) od[j] += __shfl_xor_sync(0xffffffffu, od[j], o);
                }
            if (OUT && t > 0 && lane < 4) out[t - 4 + lane][row] = p.scale * (lane < 2 ? (lane ? od[1] : od[0]) : (lane == 2 ? od[2] : od[3]));
            float u[4];
            u[0] = be.x * (v0 - a.x * d[0]);
            u[1] = be.y * (v1 - a.y * fmaf(u[0], g01, a.x * d[1]));
            u[2] = be.z * (v2 - a.z * fmaf(u[1], g12, a.y * fmaf(u[0], g02, a.x * d[2])));
            u[3] = be.w * (v3 - a.w * fmaf(u[2], g23, a.z * fmaf(u[1], g13, a.y * fmaf(u[0], g03, a.x * d[3]))));
            const float al[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 o2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    s[i] = axpy4(u[j], st.k[t + j][i * kLanes + lane], scale4(al[j], s[i]));
                    if (OUT) o2 = dot4(s[i], st.q[t + j][i * kLanes + lane], o2);
                }
                od[j] = o2.x + o2.y;
            }
        }
#pragma unroll
        for (int j = 0; j < 4 && OUT; ++j) {
            od[j] = sum8(od[j]);
            const int t = (nt - 1) / 4 * 4 + j;
            if (lane == 0 && t < nt) out[t][row] = p.scale * od[j];
        }
        if (t0 + kTok < V) next.store(stages[cur ^ 1]);
        __syncthreads();
        if (OUT)
            for (int i = threadIdx.x; i < nt * R; i += kThreads) {
                const int t = i / R, r = i % R;
                if (row0 + r < p.P)
                    store1((T *)p.o + (((long long)bi * p.L + t0 + t) * p.H + h) * p.P + row0 + r, out[t][r]);
            }
    }
    if (OUT)
        for (long long i = threadIdx.x; i < (long long)(p.L - V) * R; i += kThreads) {  // past 32 bits from 2^28 tokens on
            const int t = V + (int)(i / R), r = (int)(i % R);
            if (row0 + r < p.P) store1((T *)p.o + (((long long)bi * p.L + t) * p.H + h) * p.P + row0 + r, 0.f);
        }
    store_row(s, p.final_state ? p.final_state + srow : nullptr, in, p.N, lane);
}

// ------------------------------------------------------------------ backward
// Reverse over the tokens with the adjoint D of the state in registers.  With
// Sd = a S_{t-1}, z = v - Sd k and S_t = Sd + beta z k^T:
//     D += do q^T;   dbeta = (D k).z;   dz = beta D k = dv;
//     dk = beta z^T D - dz^T Sd;   dq = do^T S_t;   D -= dz k^T;
//     dg = <D, Sd>;   D *= a.
// The states inside a segment are formed again from the kept one and held in
// shared memory, by a second group of threads while the first is on the segment behind where a
// block has few rows (50 us for 66), else by the same threads.  Sums over
// the rows (dq, dk, dbeta, dg) go to per-row-block partials, which
// delta_rows_reduce adds in a fixed order.
struct BwdBuffers {
    float *kept, *part_q, *part_k, *part_g, *part_b;
    int nseg, nblk, items;
};

// shared memory of a block: two stages, and a segment's sums over each warp's rows
template <int NC, int R>
struct BwdShared {
    static constexpr int kThreads = R * kLanes, kParts = R == 8 ? R : R / 4;  // sums of a row, or of a warp's four
    static constexpr int kGroups = R == 8 ? 2 : 1;  // of threads: one a segment ahead with its states, where they fit twice
    Stage<NC, true, R> stage[2];
    float zs[kGroups][tok_of(NC)][R];
    float4 hist[kGroups][tok_of(NC)][NC][kThreads];
    float4 red[2][tok_of(NC)][kParts][NC * kLanes];
    float red1[2][tok_of(NC)][kThreads / 32];
};
static_assert(sizeof(BwdShared<2, 8>) <= 232448 && sizeof(BwdShared<4, 8>) <= 232448 && sizeof(BwdShared<8, 8>) <= 232448 &&
                  sizeof(BwdShared<2, 32>) <= 232448 && sizeof(BwdShared<4, 32>) <= 232448 && sizeof(BwdShared<8, 32>) <= 232448,
              "shared memory of a block");

template <typename T, int NC, int R>
__global__ void __launch_bounds__(R * kLanes * BwdShared<NC, R>::kGroups) delta_rows_bwd(DeltaParams p, BwdBuffers w) {
    constexpr int kSegTok = tok_of(NC), kThreads = R * kLanes, kParts = BwdShared<NC, R>::kParts,
                  kGroups = BwdShared<NC, R>::kGroups;
    extern __shared__ __align__(16) char smem[];
    BwdShared<NC, R> &sm = *(BwdShared<NC, R> *)smem;
    const int tid = threadIdx.x % kThreads, row = tid / kLanes, lane = tid % kLanes, warp = tid / 32;
    const bool ahead = kGroups == 1 || (int)threadIdx.x >= kThreads, back = kGroups == 1 || (int)threadIdx.x < kThreads;
    for (int item = blockIdx.x; item < w.items; item += gridDim.x) {
        const int bh = item / w.nblk, blk = item % w.nblk, bi = bh / p.H, h = bh % p.H, row0 = blk * R;
        const bool in = row0 + row < p.P;
        const int V = valid_tokens(p, bi);
        const long long srow = ((long long)bh * p.P + row0 + row) * p.N;
        const int nseg = (V + kSegTok - 1) / kSegTok;
        float4 D[NC], s[NC], sn[NC];
        load_row(D, p.d_final ? p.d_final + srow : nullptr, in, p.N, lane);
        Fetch<T, NC, true, R> next;
        auto fetch = [&](int seg) {
            next.load(p, bi, h, row0, seg * kSegTok, min(kSegTok, V - seg * kSegTok));
            load_row(sn, w.kept + (((long long)bh * w.nseg + seg) * p.P + row0 + row) * p.N, in, p.N, lane);
        };
        // the states of a segment, from the one kept before it
        auto states = [&](int seg, int buf, int hb) {
            const int nt = min(kSegTok, V - seg * kSegTok);
            const Stage<NC, true, R> &st = sm.stage[buf];
#pragma unroll
            for (int i = 0; i < NC; ++i) s[i] = sn[i];
            if (seg > 0) fetch(seg - 1);
#pragma unroll 2
            for (int t = 0; t < nt; ++t) {
                const float a = st.a[t], be = st.beta[t], v = st.v[t][row];
                float4 k[NC];
                float2 d2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    k[i] = st.k[t][i * kLanes + lane];
                    s[i] = scale4(a, s[i]);
                    sm.hist[hb][t][i][tid] = s[i];
                    d2 = dot4(s[i], k[i], d2);
                }
                const float z = v - sum8(d2.x + d2.y);
                if (lane == 0) sm.zs[hb][t][row] = z;
#pragma unroll
                for (int i = 0; i < NC; ++i) s[i] = axpy4(be * z, k[i], s[i]);
            }
        };
        auto reverse = [&](int seg, int buf, int hb) {
            const int t0 = seg * kSegTok, nt = min(kSegTok, V - t0);
            const Stage<NC, true, R> &st = sm.stage[buf];
            for (int t = nt - 1; t >= 0; --t) {
                const float dO = st.dO[t][row], be = st.beta[t], a = st.a[t], z = sm.zs[hb][t][row];
                float4 k[NC], sd[NC];
                float2 d2 = make_float2(0.f, 0.f), dg2 = d2;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    sd[i] = sm.hist[hb][t][i][tid];
                    k[i] = st.k[t][i * kLanes + lane];
                    D[i] = axpy4(dO, st.q[t][i * kLanes + lane], D[i]);
                    d2 = dot4(D[i], k[i], d2);
                }
                const float d = sum8(d2.x + d2.y);
                const float dz = be * d, bz = be * z;
                if (lane == 0 && in)
                    store1((T *)p.dv + (((long long)bi * p.L + t0 + t) * p.H + h) * p.P + row0 + row, dz);
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    float4 dq = scale4(dO, axpy4(bz, k[i], sd[i]));
                    float4 dk = axpy4(bz, D[i], scale4(-dz, sd[i]));
                    D[i] = axpy4(-dz, k[i], D[i]);
                    dg2 = dot4(D[i], sd[i], dg2);
                    D[i] = scale4(a, D[i]);
                    if (kParts == R / 4) {  // over the warp's four rows
#pragma unroll
                        for (int o = 8; o <= 16; o <<= 1) {
                            dq.x += __shfl_xor_sync(0xffffffffu, dq.x, o);
                            dq.y += __shfl_xor_sync(0xffffffffu, dq.y, o);
                            dq.z += __shfl_xor_sync(0xffffffffu, dq.z, o);
                            dq.w += __shfl_xor_sync(0xffffffffu, dq.w, o);
                            dk.x += __shfl_xor_sync(0xffffffffu, dk.x, o);
                            dk.y += __shfl_xor_sync(0xffffffffu, dk.y, o);
                            dk.z += __shfl_xor_sync(0xffffffffu, dk.z, o);
                            dk.w += __shfl_xor_sync(0xffffffffu, dk.w, o);
                        }
                    }
                    if (kParts == R || (tid & 31) < kLanes) {
                        sm.red[0][t][kParts == R ? row : warp][i * kLanes + lane] = dq;
                        sm.red[1][t][kParts == R ? row : warp][i * kLanes + lane] = dk;
                    }
                }
                // every lane has its share of dg, lane 0 of each row its dbeta
                float dg = dg2.x + dg2.y, db = lane == 0 ? d * z : 0.f;
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    dg += __shfl_xor_sync(0xffffffffu, dg, o);
                    if (o >= 8) db += __shfl_xor_sync(0xffffffffu, db, o);
                }
                if ((tid & 31) == 0) {
                    sm.red1[0][t][warp] = dg;
                    sm.red1[1][t][warp] = db;
                }
            }
        };
        // the segment's sums over its parts, in order
        auto sums = [&](int seg) {
            const int t0 = seg * kSegTok, nt = min(kSegTok, V - t0);
            const long long tok = ((long long)blk * p.b * p.H + bh) * p.L + t0;
            for (int i = threadIdx.x; i < 2 * nt * NC * kLanes; i += kThreads * kGroups) {
                const int c = i % (NC * kLanes), t = i / (NC * kLanes) % nt, which = i / (NC * kLanes) / nt;
                float4 acc = sm.red[which][t][0][c];
#pragma unroll
                for (int x = 1; x < kParts; ++x) {
                    const float4 r = sm.red[which][t][x][c];
                    acc = make_float4(acc.x + r.x, acc.y + r.y, acc.z + r.z, acc.w + r.w);
                }
                if (4 * c < p.N) *(float4 *)((which ? w.part_k : w.part_q) + (tok + t) * p.N + 4 * c) = acc;
            }
            for (int i = threadIdx.x; i < 2 * nt; i += kThreads * kGroups) {
                const int which = i / nt, t = i % nt;
                float acc = 0.f;
                for (int x = 0; x < kThreads / 32; ++x) acc += sm.red1[which][t][x];
                (which ? w.part_b : w.part_g)[tok + t] = acc;
            }
        };
        __syncthreads();  // the item before is done with the stages
        if (nseg > 0 && ahead) {
            fetch(nseg - 1);
            next.store(sm.stage[0]);
        }
        __syncthreads();
        if constexpr (kGroups == 1) {
            for (int seg = nseg - 1, cur = 0; seg >= 0; --seg, cur ^= 1) {
                states(seg, cur, 0);
                __syncwarp();
                reverse(seg, cur, 0);
                if (seg > 0) next.store(sm.stage[cur ^ 1]);
                __syncthreads();
                sums(seg);
                __syncthreads();
            }
        } else {
            // stage[cur] has segment seg, stage[cur ^ 1] the one before it, whose states are formed meanwhile
            if (nseg > 0 && ahead) {
                states(nseg - 1, 0, 0);
                if (nseg > 1) next.store(sm.stage[1]);
            }
            __syncthreads();
            for (int seg = nseg - 1, cur = 0; seg >= 0; --seg, cur ^= 1) {
                if (back)
                    reverse(seg, cur, cur);
                else if (seg > 0)
                    states(seg - 1, cur ^ 1, cur ^ 1);
                __syncthreads();
                if (ahead && seg > 1) next.store(sm.stage[cur]);
                sums(seg);
                __syncthreads();
            }
        }
        if (back) store_row(D, p.d_init ? p.d_init + srow : nullptr, in, p.N, lane);
        for (long long i = threadIdx.x; i < (long long)(p.L - V) * R; i += kThreads * kGroups) {  // past 32 bits from 2^28 tokens on
            const int t = V + (int)(i / R), r = (int)(i % R);
            if (row0 + r < p.P) store1((T *)p.dv + (((long long)bi * p.L + t) * p.H + h) * p.P + row0 + r, 0.f);
        }
    }
}

// dq, dk: the partials of a group's heads and their row blocks; dg, dbeta: of
// the row blocks.  One thread per output element, a fixed order of addition.
template <typename T>
__global__ void delta_rows_reduce(DeltaParams p, BwdBuffers w) {
    const long long nqk = (long long)p.b * p.L * p.G * p.N, ngt = (long long)p.b * p.H * p.L;
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    const long long per = (long long)p.b * p.H * p.L;
    if (i < nqk) {
        const int n = i % p.N, g = (i / p.N) % p.G;
        const long long bt = i / ((long long)p.N * p.G);
        const int t = bt % p.L, bi = bt / p.L;
        float aq = 0.f, ak = 0.f;
        if (t < valid_tokens(p, bi))
            for (int h = g * p.hpg; h < (g + 1) * p.hpg; ++h)
                for (int x = 0; x < w.nblk; ++x) {
                    const long long at = (x * per + ((long long)bi * p.H + h) * p.L + t) * p.N + n;
                    aq += w.part_q[at];
                    ak += w.part_k[at];
                }
        store1((T *)p.dq + i, aq);
        store1((T *)p.dk + i, ak);
    }
    if (i < ngt) {
        const int t = i % p.L, bi = i / ((long long)p.L * p.H);
        float ag = 0.f, ab = 0.f;
        if (t < valid_tokens(p, bi))
            for (int x = 0; x < w.nblk; ++x) {
                ag += w.part_g[x * per + i];
                ab += w.part_b[x * per + i];
            }
        p.dg[i] = ag;
        p.dbeta[i] = ab;
    }
}

// ------------------------------------------------------------------ one token
constexpr int kRows = 32, kThreads = kRows * kLanes;  // of a block
// Grid: one block per (b, h, row block).  Each state element is read and written once, in
// 16-byte pieces, NC of them in flight per thread.
template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) delta_step_kernel(DeltaParams p, float *state, long long slots,
                                                              const int32_t *index) {
    const int nblk = (p.P + kRows - 1) / kRows, bh = blockIdx.x / nblk, bi = bh / p.H, h = bh % p.H, g = h / p.hpg;
    const int row = (blockIdx.x % nblk) * kRows + threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const bool in = row < p.P;
    const long long slot = index ? (long long)index[bi] : (long long)bi;
    const long long vat = ((long long)bi * p.H + h) * p.P + row;
    if (slot < 0 || slot >= slots) {
        if (in && lane == 0) store1((T *)p.o + vat, 0.f);
        return;
    }
    float *srow = state + ((slot * p.H + h) * p.P + row) * (long long)p.N;
    float4 s[NC], k[NC], q[NC];
    load_row(s, srow, in, p.N, lane);
    const long long kat = ((long long)bi * p.G + g) * p.N;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = 4 * (i * kLanes + lane);
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        k[i] = c < p.N ? load4((const T *)p.k + kat + c) : zero;
        q[i] = c < p.N ? load4((const T *)p.q + kat + c) : zero;
    }
    const float a = expf(clamp_log_decay(p.g[bi * (long long)p.H + h])), be = p.beta[bi * (long long)p.H + h];
    const float v = in ? load1((const T *)p.v + vat) : 0.f;
    float2 d = make_float2(0.f, 0.f), od2 = d;
#pragma unroll
    for (int i = 0; i < NC; ++i) d = dot4(s[i], k[i], d);
    const float u = be * (v - a * sum8(d.x + d.y));
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        s[i] = axpy4(u, k[i], scale4(a, s[i]));
        od2 = dot4(s[i], q[i], od2);
    }
    const float od = sum8(od2.x + od2.y);
    store_row(s, srow, in, p.N, lane);
    if (in && lane == 0) store1((T *)p.o + vat, p.scale * od);
}

int row_blocks(int P, int R) { return (P + R - 1) / R; }

size_t up256(size_t v) { return (v + 255) / 256 * 256; }
struct BwdSizes {
    size_t kept, part, gate, total;
    int nseg, nblk, grid, rows;
};
BwdSizes bwd_sizes(long long b, long long L, long long H, long long P, long long N) {
    BwdSizes z;
    const size_t nc = (size_t)(N + 31) / 32;
    const int seg = tok_of((int)nc);
    z.nseg = (int)((L + seg - 1) / seg);
    z.rows = rows_of(b * H, (int)P);
    z.nblk = row_blocks((int)P, z.rows);
    const long long items = b * H * z.nblk;
    const long long most = z.rows == 32 ? 152 : 456;  // a block of 32 rows has an SM to itself
    z.grid = (int)(items < most ? items : most);
    z.kept = up256(4ull * b * H * z.nseg * P * N);
    z.part = up256(4ull * z.nblk * b * H * L * N);
    z.gate = up256(4ull * z.nblk * b * H * L);
    z.total = z.kept + 2 * z.part + 2 * z.gate;
    return z;
}

#define DELTA_BY_NC(CALL)              \
    switch ((p.N + 31) / 32) {         \
        case 1: CALL(1); break;        \
        case 2: CALL(2); break;        \
        case 3: CALL(3); break;        \
        case 4: CALL(4); break;        \
        case 5: CALL(5); break;        \
        case 6: CALL(6); break;        \
        case 7: CALL(7); break;        \
        default: CALL(8); break;       \
    }

template <typename T, int R, bool OUT>
cudaError_t fwd(const DeltaParams &p, float *kept, int nseg, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.b * p.H * row_blocks(p.P, R));
#define CALL(NC) delta_rows_fwd<T, NC, R, OUT><<<grid, R * kLanes, 0, s>>>(p, kept, nseg)
    DELTA_BY_NC(CALL)
#undef CALL
    return cudaGetLastError();
}
template <typename T, int R>
cudaError_t bwd(const DeltaParams &p, char *ws, cudaStream_t s) {
    const BwdSizes z = bwd_sizes(p.b, p.L, p.H, p.P, p.N);
    BwdBuffers w;
    w.kept = (float *)ws;
    w.part_q = (float *)(ws + z.kept);
    w.part_k = (float *)(ws + z.kept + z.part);
    w.part_g = (float *)(ws + z.kept + 2 * z.part);
    w.part_b = (float *)(ws + z.kept + 2 * z.part + z.gate);
    w.nseg = z.nseg;
    w.nblk = z.nblk;
    w.items = p.b * p.H * z.nblk;
    cudaError_t e = fwd<T, R, false>(p, w.kept, w.nseg, s);
    if (e != cudaSuccess) return e;
#define CALL(NC)                                                                                          \
    do {                                                                                                  \
        const int bytes = (int)sizeof(BwdShared<NC, R>);                                                  \
        if ((e = allow_shared((const void *)delta_rows_bwd<T, NC, R>, bytes)) != cudaSuccess) return e;   \
        delta_rows_bwd<T, NC, R><<<z.grid, R * kLanes * BwdShared<NC, R>::kGroups, bytes, s>>>(p, w);                               \
    } while (0)
    DELTA_BY_NC(CALL)
#undef CALL
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const long long nqk = (long long)p.b * p.L * p.G * p.N, ngt = (long long)p.b * p.H * p.L;
    const long long most = nqk > ngt ? nqk : ngt;
    delta_rows_reduce<T><<<(unsigned)((most + 255) / 256), 256, 0, s>>>(p, w);
    return cudaGetLastError();
}
template <typename T>
cudaError_t step(const DeltaParams &p, float *state, long long slots, const int32_t *index, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.b * p.H * row_blocks(p.P, kRows));
#define CALL(NC) delta_step_kernel<T, NC><<<grid, kThreads, 0, s>>>(p, state, slots, index)
    DELTA_BY_NC(CALL)
#undef CALL
    return cudaGetLastError();
}

}  // namespace

size_t simt_backward_bytes(const delta_dims &d) { return bwd_sizes(d.batch, d.seqlen, d.nheads, d.headdim, d.dstate).total; }

cudaError_t launch_simt_forward(const DeltaParams &p, bool is_bf16, cudaStream_t s) {
    if (rows_of((long long)p.b * p.H, p.P) == 8) return is_bf16 ? fwd<bf16, 8, true>(p, nullptr, 0, s) : fwd<float, 8, true>(p, nullptr, 0, s);
    return is_bf16 ? fwd<bf16, 32, true>(p, nullptr, 0, s) : fwd<float, 32, true>(p, nullptr, 0, s);
}
cudaError_t launch_simt_backward(const DeltaParams &p, bool is_bf16, char *ws, cudaStream_t s) {
    if (rows_of((long long)p.b * p.H, p.P) == 8) return is_bf16 ? bwd<bf16, 8>(p, ws, s) : bwd<float, 8>(p, ws, s);
    return is_bf16 ? bwd<bf16, 32>(p, ws, s) : bwd<float, 32>(p, ws, s);
}
cudaError_t launch_step(const DeltaParams &p, bool is_bf16, float *state, long long slots, const int32_t *index,
                        cudaStream_t s) {
    return is_bf16 ? step<bf16>(p, state, slots, index, s) : step<float>(p, state, slots, index, s);
}

}  // namespace delta
}  // namespace ssd
