// norm_group.cu -- the mixers' exit norm (include/norm.h): group norm per token with
// an activation or a gate, and its backward.
//
// A row of D channels in G groups is G rows of w = D / G columns for the statistics, one after the other in
// memory, so the kernels walk rows * G short rows: TPR threads hold one in NV vectors, several short rows a warp.
// Row r has the weights of group r mod G; the grid's stride is a multiple of G, so a thread meets one
// group only and keeps its weights (and their gradients' sums) in registers.  All statistics are
// fp32, the variance is the mean of squares about the mean (two sums, no cancellation).
// Everything is recomputed in the backward from x and the gate: with u the normed input,
// n = (u - mean) rstd, y = n weight + bias and g the gradient of y,
//     dweight = sum g n,  dbias = sum g,  t = g weight,
//     du = rstd (t - [mean of t] - n mean(t n))          ([..] with centring)
// and the gate's or the activation's product rule around it.  Both are streams bound by HBM.
// A thread's sums of dweight and dbias go to a slot each; a second kernel adds the slots in their order.
#include <stdio.h>

#include "norm_rows.cuh"

namespace ssd {
namespace {

using namespace norm_rows;

constexpr long long kMaxD = 16384;

struct GroupArgs {
    const void *x, *gate;
    const float *weight, *bias;
    float eps;
    int act;            // NORM_ACT_*
    bool center, first;
    void *y;            // forward
    const void *dy;     // backward
    void *dx, *dgate;
    float *part;        // [2][slots][D], null: no weight gradients
    long long rows;     // short ones: rows * groups
    int groups, w;
};

// The activation and its derivative; for silu x s and s (1 + x (1 - s)), for sigmoid s and s (1 - s), with s the logistic function of x.
// s = 1 / (1 + exp(-x)) of a pair.  fp32 takes expf; bf16 the approximations of 2^x and of the reciprocal, off by some
// 2^-21 of the result (2^-17 where exp(-x) is 10^35: x log2(e) as rounded) where its rounding is up to 2^-8.  exp(-x) past fp32 is infinite
// and the result 0.
template <typename T>
__device__ __forceinline__ float2 logistic(float2 x) {
    if constexpr (sizeof(T) == 4) {
        return make_float2(__fdividef(1.f, 1.f + expf(-x.x)), __fdividef(1.f, 1.f + expf(-x.y)));
    } else {
        float2 e = fmul2(x, make_float2(-1.4426950408889634f, -1.4426950408889634f));
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
        e = fadd2(e, make_float2(1.f, 1.f));
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
        return e;
    }
}
template <typename T>
__device__ __forceinline__ float2 act2(int act, float2 x) {
    if (act == NORM_ACT_NONE) return x;
    const float2 s = logistic<T>(x);
    return act == NORM_ACT_SILU ? fmul2(x, s) : s;
}
template <typename T>
__device__ __forceinline__ void act2(int act, float2 x, float2 &a, float2 &d) {
    const float2 one = make_float2(1.f, 1.f), minus = make_float2(-1.f, -1.f);
    if (act == NORM_ACT_NONE) {
        a = x;
        d = one;
        return;
    }
    if (act == NORM_ACT_SILU) {
        const float2 s = logistic<T>(x), r = ffma2(s, minus, one);  // 1 - s
        a = fmul2(x, s);
        d = fmul2(s, ffma2(x, r, one));
    } else {
        // s of -|x|, so that 1 - s keeps its bits (where s is next to 1 the difference has none left); of x it is one of the two
        const float2 s = logistic<T>(make_float2(-fabsf(x.x), -fabsf(x.y))), r = ffma2(s, minus, one);
        a = make_float2(x.x > 0.f ? r.x : s.x, x.y > 0.f ? r.y : s.y);
        d = fmul2(s, r);
    }
}

template <int TPR>
constexpr int kBlock = TPR < 256 ? 256 : TPR;

// Blocks of an SM: what the registers of short rows allow, and for long ones that many threads.
template <int TPR, int NV, int VEC>
constexpr int kFwdBlocks = kBlock<TPR> == 256 ? (NV == 1 ? 4 : 2) : (kBlock<TPR> == 512 && NV == 1 ? 2 : 1);
template <int TPR, int NV, int VEC>
constexpr int kBwdBlocks = kBlock<TPR> == 256 && NV == 1 ? 2 : 1;

// The gate's place, known to the compiler for short rows, whose kernels are bound by their instructions (16384 x 5120 in heads of
// 64: 89 us with the place looked up, 83 us known; backward 170 and 139, with three rows ahead).
constexpr int kNoGate = 0, kGateAfter = 1, kGateFirst = 2, kAnyGate = 3;
template <int MODE>
__device__ __forceinline__ bool gated(const GroupArgs &a) {
    return MODE == kAnyGate ? a.gate != nullptr : MODE != kNoGate;
}
template <int MODE>
__device__ __forceinline__ bool gate_first(const GroupArgs &a) {
    return MODE == kAnyGate ? a.first : MODE == kGateFirst;
}

// What both kernels hold of a short row: vectors j of thread t at columns (j TPR + t) VEC.
template <int VEC, int TPR, int NV>
struct Place {
    static constexpr int RPB = kBlock<TPR> / TPR;
    const int t = threadIdx.x % TPR;
    const long long mine = blockIdx.x * (long long)RPB + threadIdx.x / TPR, step = gridDim.x * (long long)RPB;
    __device__ __forceinline__ int col(int j) const { return (j * TPR + t) * VEC; }
};

// mean and rstd of u over the row; u becomes n = (u - mean) rstd, columns outside stay 0.
template <int VEC, int TPR, int NV, int PAIRS>
__device__ __forceinline__ float normalise(float2 (&u)[NV][PAIRS], const GroupArgs &a, const Place<VEC, TPR, NV> &at,
                                           float (*buf)[32][1], int &turn) {
    const float inv = 1.f / (float)a.w;
    if (TPR <= 32 && a.center && a.w == TPR * NV * VEC) {
        // every lane has as many columns: its own mean and squares about it, then lanes in pairs, whose squares about the common
        // mean are the sum of theirs and n / 2 times the difference's; one chain of shuffles in place of two
        constexpr float n = (float)(NV * VEC);
        float2 s2 = make_float2(0.f, 0.f), q2 = s2;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) s2 = fadd2(s2, u[j][i]);
        float mean = (s2.x + s2.y) * (1.f / n);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const float2 d = fadd2(u[j][i], make_float2(-mean, VEC > 1 ? -mean : 0.f));
                q2 = ffma2(d, d, q2);
            }
        float squares = q2.x + q2.y, half = 0.5f * n;
#pragma unroll
        for (int o = 1; o < TPR; o <<= 1) {
            const float m = __shfl_xor_sync(0xffffffffu, mean, o), q = __shfl_xor_sync(0xffffffffu, squares, o), d = m - mean;
            squares = (squares + q) + half * d * d;
            mean = 0.5f * (mean + m);
            half += half;
        }
        const float rstd = rsqrtf(squares * inv + a.eps), off = -mean * rstd;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) u[j][i] = ffma2(u[j][i], make_float2(rstd, rstd), make_float2(off, VEC > 1 ? off : 0.f));
        return rstd;
    }
    if (a.center) {
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) s2 = fadd2(s2, u[j][i]);
        float s[1] = {s2.x + s2.y};
        row_reduce<Sum, TPR, 1>(s, buf, turn);
        const float mean = s[0] * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at.col(j) < a.w)
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) u[j][i] = fadd2(u[j][i], make_float2(-mean, VEC > 1 ? -mean : 0.f));
    }
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) s2 = ffma2(u[j][i], u[j][i], s2);
    float s[1] = {s2.x + s2.y};
    row_reduce<Sum, TPR, 1>(s, buf, turn);
    const float rstd = rsqrtf(s[0] * inv + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) u[j][i] = fmul2(u[j][i], make_float2(rstd, rstd));
    return rstd;
}

// ------------------------------------------------------------------ forward
template <typename T, int VEC, int TPR, int NV, int MODE>
__global__ void __launch_bounds__(kBlock<TPR>, kFwdBlocks<TPR, NV, VEC>) group_norm_kernel(GroupArgs a) {
    __shared__ float buf[2][32][1];
    constexpr int PAIRS = Vec<T, VEC>::PAIRS;
    const Place<VEC, TPR, NV> at;
    int turn = 0;
    Vec<float, VEC> w[NV], b[NV];
    const int off = (int)(at.mine % a.groups) * a.w;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        w[j].zero();
        b[j].zero();
        if (at.col(j) < a.w) {
            w[j].load(a.weight + off + at.col(j));
            if (a.bias) b[j].load(a.bias + off + at.col(j));
        }
    }
    // columns outside stay 0; past the last row the row before stays, and nothing is made of it
    Vec<T, VEC> x[NV], z[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) x[j].zero(), z[j].zero();
    const T *px = (const T *)a.x + at.mine * a.w, *pz = (const T *)a.gate + at.mine * a.w;
    const long long move = at.step * a.w;
    auto load = [&](long long row) {
        if (row < a.rows)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (at.col(j) < a.w) {
                    x[j].template load<true>(px + at.col(j));
                    if (gated<MODE>(a)) z[j].template load<true>(pz + at.col(j));
                }
        px += move, pz += move;
    };
    load(at.mine);
    T *py = (T *)a.y + at.mine * a.w;
    for (long long row = at.mine, base = row - threadIdx.x / TPR; base < a.rows; row += at.step, base += at.step) {
        float2 u[NV][PAIRS], s[NV][PAIRS];  // s: what the normed value is multiplied with
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                u[j][i] = x[j].get(i);
                if (gated<MODE>(a)) s[j][i] = act2<T>(a.act, z[j].get(i));
                if (gate_first<MODE>(a)) u[j][i] = fmul2(u[j][i], s[j][i]);
            }
        load(row + at.step);
        normalise(u, a, at, buf, turn);
        if (row < a.rows)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (at.col(j) >= a.w) continue;
                Vec<T, VEC> y;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    float2 v = ffma2(u[j][i], w[j].get(i), b[j].get(i));
                    if (!gated<MODE>(a))
                        v = act2<T>(a.act, v);
                    else if (!gate_first<MODE>(a))
                        v = fmul2(v, s[j][i]);
                    y.set(i, v);
                }
                y.store(py + at.col(j));
            }
        py += move;
    }
}

// ------------------------------------------------------------------ backward
template <typename T, int VEC, int TPR, int NV, int MODE>
__global__ void __launch_bounds__(kBlock<TPR>, kBwdBlocks<TPR, NV, VEC>) group_norm_bwd_kernel(GroupArgs a) {
    __shared__ float buf[2][32][1], buf2[2][32][2];
    constexpr int PAIRS = Vec<T, VEC>::PAIRS;
    const Place<VEC, TPR, NV> at;
    int turn = 0, turn2 = 0;
    Vec<float, VEC> w[NV], b[NV];
    float2 dw[NV][PAIRS], db[NV][PAIRS];
    const int off = (int)(at.mine % a.groups) * a.w;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        w[j].zero();
        b[j].zero();
        if (at.col(j) < a.w) {
            w[j].load(a.weight + off + at.col(j));
            if (a.bias) b[j].load(a.bias + off + at.col(j));
        }
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) dw[j][i] = db[j][i] = make_float2(0.f, 0.f);
    }
    // columns outside stay 0; past the last row dy is 0, so that nothing is added to the weights' gradients
    constexpr int A = TPR <= 32 && NV == 1 && VEC > 1 ? 3 : 1;  // rows ahead of the one in work
    Vec<T, VEC> xs[A][NV], zs[A][NV], dys[A][NV];
#pragma unroll
    for (int k = 0; k < A; ++k)
#pragma unroll
        for (int j = 0; j < NV; ++j) xs[k][j].zero(), zs[k][j].zero(), dys[k][j].zero();
    const T *px = (const T *)a.x + at.mine * a.w, *pz = (const T *)a.gate + at.mine * a.w, *pdy = (const T *)a.dy + at.mine * a.w;
    const long long move = at.step * a.w;
    auto load = [&](long long row, Vec<T, VEC>(&x)[NV], Vec<T, VEC>(&z)[NV], Vec<T, VEC>(&dy)[NV]) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at.col(j) < a.w) {
                if (row < a.rows) {
                    x[j].template load<true>(px + at.col(j));
                    dy[j].template load<true>(pdy + at.col(j));
                    if (gated<MODE>(a)) z[j].template load<true>(pz + at.col(j));
                } else {
                    dy[j].zero();
                }
            }
        px += move, pz += move, pdy += move;
    };
#pragma unroll
    for (int k = 0; k < A; ++k) load(at.mine + k * at.step, xs[k], zs[k], dys[k]);
    T *pdx = (T *)a.dx + at.mine * a.w, *pdz = (T *)a.dgate + at.mine * a.w;
    const float inv = 1.f / (float)a.w;
    long long row = at.mine;
    auto one = [&](Vec<T, VEC>(&x)[NV], Vec<T, VEC>(&z)[NV], Vec<T, VEC>(&dy)[NV]) {
        // u, then n;  g the gradient of y;  s the gate's activation, d what dgate is multiplied with
        float2 u[NV][PAIRS], g[NV][PAIRS], s[NV][PAIRS], d[NV][PAIRS];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const float2 v = x[j].get(i);
                g[j][i] = dy[j].get(i);
                u[j][i] = v;
                if (gated<MODE>(a)) {
                    act2<T>(a.act, z[j].get(i), s[j][i], d[j][i]);
                    if (gate_first<MODE>(a)) {
                        u[j][i] = fmul2(v, s[j][i]);
                        d[j][i] = fmul2(d[j][i], v);
                    } else {
                        d[j][i] = fmul2(d[j][i], g[j][i]);
                        g[j][i] = fmul2(g[j][i], s[j][i]);
                    }
                }
            }
        load(row + A * at.step, x, z, dy);
        const float rstd = normalise(u, a, at, buf, turn);
        float2 t1 = make_float2(0.f, 0.f), t2 = make_float2(0.f, 0.f);
        const bool live = row < a.rows;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const float2 y = ffma2(u[j][i], w[j].get(i), b[j].get(i));
                if (!gated<MODE>(a)) {
                    float2 act, slope;
                    act2<T>(a.act, y, act, slope);
                    g[j][i] = fmul2(g[j][i], slope);
                } else if (!gate_first<MODE>(a)) {
                    d[j][i] = fmul2(d[j][i], y);  // dgate
                }
                if (live) {  // past the last row n may be NaN (no columns loaded, eps of 0), which dy = 0 does not take out
                    dw[j][i] = ffma2(g[j][i], u[j][i], dw[j][i]);
                    db[j][i] = fadd2(db[j][i], g[j][i]);
                }
                g[j][i] = fmul2(g[j][i], w[j].get(i));
                t1 = fadd2(t1, g[j][i]);
                t2 = ffma2(g[j][i], u[j][i], t2);
            }
        float t[2] = {t1.x + t1.y, t2.x + t2.y};
        row_reduce<Sum, TPR, 2>(t, buf2, turn2);
        const float m1 = a.center ? -t[0] * inv * rstd : 0.f, m2 = -t[1] * inv * rstd;
        if (live)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (at.col(j) >= a.w) continue;
                Vec<T, VEC> dx, dz;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    float2 du = ffma2(g[j][i], make_float2(rstd, rstd), ffma2(u[j][i], make_float2(m2, m2), make_float2(m1, m1)));
                    if (gate_first<MODE>(a)) {
                        d[j][i] = fmul2(d[j][i], du);
                        du = fmul2(du, s[j][i]);
                    }
                    dx.set(i, du);
                    if (gated<MODE>(a)) dz.set(i, d[j][i]);
                }
                dx.store(pdx + at.col(j));
                if (gated<MODE>(a)) dz.store(pdz + at.col(j));
            }
        pdx += move, pdz += move;
        row += at.step;
    };
    for (long long base = row - threadIdx.x / TPR; base < a.rows; base += A * at.step)
#pragma unroll
        for (int k = 0; k < A; ++k) one(xs[k], zs[k], dys[k]);
    if (a.part) {
        const long long D = (long long)a.groups * a.w, slots = at.step / a.groups, slot = at.mine / a.groups;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (at.col(j) >= a.w) continue;
            Vec<float, VEC> o;
            float *to = a.part + slot * D + off + at.col(j);
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) o.set(i, dw[j][i]);
            o.store(to);
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) o.set(i, db[j][i]);
            o.store(to + slots * D);
        }
    }
}

// dweight (blockIdx.y = 0) and dbias (1): the slots' sums, 32 columns and 8 slots at a time.
__global__ void __launch_bounds__(256) group_norm_sum_kernel(const float *part, float *dweight, float *dbias, long long slots,
                                                             int D) {
    __shared__ float share[8][32];
    float *out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    const int lane = threadIdx.x & 31, k = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    const float *src = part + blockIdx.y * slots * D + c;
    float s = 0.f;
    if (c < D)
        for (long long i = k; i < slots; i += 8) s += src[i * D];
    share[k][lane] = s;
    __syncthreads();
    if (k == 0 && c < D) {
        for (int i = 1; i < 8; ++i) s += share[i][lane];
        out[c] = s;
    }
}

// ------------------------------------------------------------------ launches
// The variant of a width, as a call F(VEC, TPR, NV): 16-byte vectors where the width allows, else single
// elements; as few threads as hold the row in one vector each up to 512, then in two or four (single elements: up to 16).
#define GROUP_BY_WIDTH(T, w, F)                                      \
    {                                                                \
        constexpr int kWide = 16 / (int)sizeof(T);                   \
        const int n = (w) % kWide == 0 ? (w) / kWide : (w);          \
        if ((w) % kWide == 0) {                                      \
            if (n <= 4) F(kWide, 4, 1);                              \
            else if (n <= 8) F(kWide, 8, 1);                         \
            else if (n <= 16) F(kWide, 16, 1);                       \
            else if (n <= 32) F(kWide, 32, 1);                       \
            else if (n <= 64) F(kWide, 64, 1);                       \
            else if (n <= 128) F(kWide, 128, 1);                     \
            else if (n <= 256) F(kWide, 256, 1);                     \
            else if (n <= 512) F(kWide, 512, 1);                     \
            else if (n <= 768) F(kWide, 384, 2);                     \
            else if (n <= 1024) F(kWide, 512, 2);                    \
            else if (n <= 2048) F(kWide, 1024, 2);                   \
            else if constexpr (kMaxD > 2048 * kWide) F(kWide, 1024, 4); \
        } else {                                                     \
            if (n <= 128) F(1, 32, 4);                               \
            else if (n <= 1024) F(1, 256, 4);                        \
            else if (n <= 4096) F(1, 1024, 4);                       \
            else F(1, 1024, 16);                                     \
        }                                                            \
    }

long long gcd(long long a, long long b) { return b ? gcd(b, a % b) : a; }
// Blocks: a multiple of what makes the stride a multiple of the groups, as near as that goes to the
// blocks that the SMs hold at once, and no more than there are rows for.
template <int TPR>
long long grid_of(long long rows, int groups, int per_sm) {
    constexpr long long RPB = kBlock<TPR> / TPR;
    const long long unit = groups / gcd(groups, RPB), held = kSMs * per_sm;
    const long long most = (rows + unit * RPB - 1) / (unit * RPB), fit = held / unit;
    return unit * (most < (fit < 1 ? 1 : fit) ? most : (fit < 1 ? 1 : fit));
}
template <int TPR>
long long slots_of(long long rows, int groups, int per_sm) {
    return grid_of<TPR>(rows, groups, per_sm) * (kBlock<TPR> / TPR) / groups;
}

// K<..., MODE> for the gate's place, where a row is held by a warp or less in whole vectors.
#define GROUP_LAUNCH(K, BLOCKS, VEC, TPR, NV)                                                                       \
    do {                                                                                                    \
        const unsigned grid = (unsigned)grid_of<TPR>(a.rows, a.groups, BLOCKS<TPR, NV, VEC>);               \
        if constexpr (TPR <= 32 && VEC > 1) {                                                               \
            if (!a.gate) K<T, VEC, TPR, NV, kNoGate><<<grid, kBlock<TPR>, 0, s>>>(a);                       \
            else if (a.first) K<T, VEC, TPR, NV, kGateFirst><<<grid, kBlock<TPR>, 0, s>>>(a);               \
            else K<T, VEC, TPR, NV, kGateAfter><<<grid, kBlock<TPR>, 0, s>>>(a);                            \
        } else {                                                                                            \
            K<T, VEC, TPR, NV, kAnyGate><<<grid, kBlock<TPR>, 0, s>>>(a);                                   \
        }                                                                                                   \
    } while (0)
template <typename T>
cudaError_t forward(const GroupArgs &a, cudaStream_t s) {
#define CALL(VEC, TPR, NV) GROUP_LAUNCH(group_norm_kernel, kFwdBlocks, VEC, TPR, NV)
    GROUP_BY_WIDTH(T, a.w, CALL)
#undef CALL
    return cudaGetLastError();
}
template <typename T>
long long slots(long long rows, int groups, int w) {
    long long out = 0;
#define CALL(VEC, TPR, NV) out = slots_of<TPR>(rows, groups, kBwdBlocks<TPR, NV, VEC>)
    GROUP_BY_WIDTH(T, w, CALL)
#undef CALL
    return out;
}
template <typename T>
cudaError_t backward(const GroupArgs &a, float *dweight, float *dbias, cudaStream_t s) {
#define CALL(VEC, TPR, NV) GROUP_LAUNCH(group_norm_bwd_kernel, kBwdBlocks, VEC, TPR, NV)
    GROUP_BY_WIDTH(T, a.w, CALL)
#undef CALL
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.part) return e;
    const int D = a.groups * a.w;
    group_norm_sum_kernel<<<dim3((D + 31) / 32, 2), 256, 0, s>>>(a.part, dweight, dbias, slots<T>(a.rows, a.groups, a.w), D);
    return cudaGetLastError();
}

ssd_status group_fail(ssd_status st, const char *msg) {
    record_error(msg);
    return st;
}
ssd_status group_cuda(cudaError_t e) {
    if (e == cudaSuccess) return SSD_OK;
    char msg[256];
    snprintf(msg, sizeof(msg), "launch failed: %s", cudaGetErrorString(e));
    return group_fail(SSD_ERR_CUDA, msg);
}
bool al16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
ssd_status check_shape(ssd_dtype dtype, int activation, uint32_t flags, int64_t rows, int64_t D, int64_t groups) {
    if (dtype != SSD_F32 && dtype != SSD_BF16) return group_fail(SSD_ERR_INVALID_ARG, "unknown dtype");
    if (activation < NORM_ACT_NONE || activation > NORM_ACT_SIGMOID) return group_fail(SSD_ERR_INVALID_ARG, "unknown activation");
    if (flags & ~(uint32_t)(NORM_CENTER | NORM_GATE_FIRST)) return group_fail(SSD_ERR_INVALID_ARG, "unknown flags");
    if (rows < 1 || D < 1 || groups < 1) return group_fail(SSD_ERR_INVALID_ARG, "every dimension must be >= 1");
    if (D % groups) return group_fail(SSD_ERR_INVALID_ARG, "groups must divide the columns");
    if (D > kMaxD) return group_fail(SSD_ERR_UNSUPPORTED, "more than 16384 columns");
    if (rows > (1LL << 31) - 1) return group_fail(SSD_ERR_UNSUPPORTED, "problem too large");
    return SSD_OK;
}
ssd_status check_pointers(const void *const *req, int nreq, const void *const *opt, int nopt) {
    for (int i = 0; i < nreq; ++i)
        if (!req[i] || !al16(req[i])) return group_fail(SSD_ERR_INVALID_ARG, "a required pointer is NULL or not 16-byte aligned");
    for (int i = 0; i < nopt; ++i)
        if (!al16(opt[i])) return group_fail(SSD_ERR_INVALID_ARG, "a pointer is not 16-byte aligned");
    return SSD_OK;
}
GroupArgs group_args(const void *x, const void *gate, const float *weight, const float *bias, float eps, int activation,
                     uint32_t flags, int64_t rows, int64_t D, int64_t groups) {
    GroupArgs a = {};
    a.x = x;
    a.gate = gate;
    a.weight = weight;
    a.bias = bias;
    a.eps = eps;
    a.act = activation;
    a.center = (flags & NORM_CENTER) != 0;
    a.first = (flags & NORM_GATE_FIRST) != 0;
    a.rows = rows * groups;
    a.groups = (int)groups;
    a.w = (int)(D / groups);
    return a;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status norm_group_gated(ssd_dtype dtype, const void *x, const void *gate, const float *weight, const float *bias, float eps,
                            int activation, uint32_t flags, void *y, int64_t rows, int64_t D, int64_t groups, void *stream_) {
    record_error("");
    ssd_status st = check_shape(dtype, activation, flags, rows, D, groups);
    if (st != SSD_OK) return st;
    const void *req[] = {x, weight, y}, *opt[] = {gate, bias};
    if ((st = check_pointers(req, 3, opt, 2)) != SSD_OK) return st;
    if ((flags & NORM_GATE_FIRST) && !gate) return group_fail(SSD_ERR_INVALID_ARG, "NORM_GATE_FIRST without a gate");
    GroupArgs a = group_args(x, gate, weight, bias, eps, activation, flags, rows, D, groups);
    a.y = y;
    return group_cuda(dtype == SSD_BF16 ? forward<bf16>(a, (cudaStream_t)stream_) : forward<float>(a, (cudaStream_t)stream_));
}

size_t norm_group_workspace_bytes(ssd_dtype dtype, int64_t rows, int64_t D, int64_t groups) {
    record_error("");
    if (check_shape(dtype, NORM_ACT_NONE, 0, rows, D, groups) != SSD_OK) return 0;
    const int w = (int)(D / groups);
    return sizeof(float) * 2 * (size_t)D *
           (size_t)(dtype == SSD_BF16 ? slots<bf16>(rows * groups, (int)groups, w) : slots<float>(rows * groups, (int)groups, w));
}

ssd_status norm_group_gated_backward(ssd_dtype dtype, const void *dy, const void *x, const void *gate, const float *weight,
                                     const float *bias, float eps, int activation, uint32_t flags, void *dx, void *dgate,
                                     float *dweight, float *dbias, int64_t rows, int64_t D, int64_t groups, void *workspace,
                                     size_t workspace_bytes, void *stream_) {
    record_error("");
    ssd_status st = check_shape(dtype, activation, flags, rows, D, groups);
    if (st != SSD_OK) return st;
    const void *req[] = {dy, x, weight, dx, workspace}, *opt[] = {gate, bias, dgate, dweight, dbias};
    const bool sums = dweight || dbias;
    if ((st = check_pointers(req, sums ? 5 : 4, opt, 5)) != SSD_OK) return st;
    if ((flags & NORM_GATE_FIRST) && !gate) return group_fail(SSD_ERR_INVALID_ARG, "NORM_GATE_FIRST without a gate");
    if ((gate != nullptr) != (dgate != nullptr)) return group_fail(SSD_ERR_INVALID_ARG, "gate and dgate come together");
    if (sums && workspace_bytes < norm_group_workspace_bytes(dtype, rows, D, groups))
        return group_fail(SSD_ERR_WORKSPACE, "workspace too small");
    GroupArgs a = group_args(x, gate, weight, bias, eps, activation, flags, rows, D, groups);
    a.dy = dy;
    a.dx = dx;
    a.dgate = dgate;
    a.part = sums ? (float *)workspace : nullptr;
    return group_cuda(dtype == SSD_BF16 ? backward<bf16>(a, dweight, dbias, (cudaStream_t)stream_)
                                        : backward<float>(a, dweight, dbias, (cudaStream_t)stream_));
}

}  // extern "C"
