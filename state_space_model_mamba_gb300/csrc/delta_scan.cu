// delta_scan.cu -- the serial pass of the chunked gated delta rule
// (delta_chunk.cuh): one block per (b, h, 64 rows of P) walks the chunks in
// order with the state in registers.
//
// Everything is computed transposed, a warp owning 16 rows of S^T [P, N]:
//     X0^T = V^T - (S^T K^T) e^gamma,   Z^T = X0^T + (X0 beta)^T Tt^T,
//     O^T = (S^T Q^T) scale e^gamma + U^T A^T,   S'^T = e^gamma_C S^T + (U e^(gamma_C-gamma))^T K,
// so that the accumulators of one product are the register operand of the next
// (rows stay in the lane that holds them): state, X0, Z and U never pass through
// shared memory, and the warps of a block share nothing but the loaded tiles.
// The fp32 operands go to the tensor cores as hi + lo bf16 parts (delta_mma.cuh).
#include "delta_chunk.cuh"
#include "delta_mma.cuh"

namespace ssd {
namespace delta {
namespace {

constexpr int kThreads = 128;

template <int NP>
struct ScanStage {
    unsigned char k[kChunk * NP * 2], q[kChunk * NP * 2];
    unsigned char v[kChunk * 128];  // 64 columns; o is staged over it once it has been read
    unsigned char img[kImgFwd];
};

template <int NP>
__device__ __forceinline__ void load_scan_stage(ScanStage<NP> &s, const ChunkParams &cp, int bi, int h, int slice,
                                                int chunk, int V) {
    const DeltaParams &p = cp.p;
    constexpr int LINE = NP * 2;
    const int t0 = chunk * kChunk, grp = h / p.hpg, tid = threadIdx.x;
    const uint32_t ks = smem_u32(s.k), qs = smem_u32(s.q), vs = smem_u32(s.v), is = smem_u32(s.img);
#pragma unroll
    for (int x = 0; x < kChunk * (NP / 8) / kThreads; ++x) {
        const int i = x * kThreads + tid, r = i / (NP / 8), c = i % (NP / 8);
        const bool real = t0 + r < V && c * 8 < p.N;
        const long long at = real ? (((long long)bi * p.L + t0 + r) * p.G + grp) * p.N + c * 8 : 0;
        cp_async16(ks + swz<LINE>(r, c), (const bf16 *)p.k + at, real);
        cp_async16(qs + swz<LINE>(r, c), (const bf16 *)p.q + at, real);
    }
#pragma unroll
    for (int x = 0; x < kChunk * 8 / kThreads; ++x) {
        const int i = x * kThreads + tid, r = i / 8, c = i % 8;
        const bool real = t0 + r < V && slice * 64 + c * 8 < p.P;
        const long long at = real ? (((long long)bi * p.L + t0 + r) * p.H + h) * p.P + slice * 64 + c * 8 : 0;
        cp_async16(vs + swz<128>(r, c), (const bf16 *)p.v + at, real);
    }
    const char *img = cp.img + (((long long)bi * p.H + h) * cp.n + chunk) * (long long)kImgBytes;
#pragma unroll
    for (int x = 0; x < (kImgFwd / 16 + kThreads - 1) / kThreads; ++x) {
        const int i = x * kThreads + tid;
        if (i < kImgFwd / 16) cp_async16(is + 16 * i, img + 16 * i, true);
    }
}

// Rows of fp32 state in accumulator layout: tile nt holds columns 8 nt + 2 t, +1 of rows r and r + 8.
template <int NP>
__device__ __forceinline__ void load_state(float (&s)[NP / 8][4], const float *src, int row, int P, int N, int t) {
#pragma unroll
    for (int nt = 0; nt < NP / 8; ++nt) {
        const int c = 8 * nt + 2 * t;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = row + 8 * half;
            const float2 x = (src && r < P && c < N) ? *(const float2 *)(src + (long long)r * N + c) : make_float2(0.f, 0.f);
            s[nt][2 * half] = x.x;
            s[nt][2 * half + 1] = x.y;
        }
    }
}
template <int NP>
__device__ __forceinline__ void store_state(const float (&s)[NP / 8][4], float *dst, int row, int P, int N, int t) {
    if (!dst) return;
#pragma unroll
    for (int nt = 0; nt < NP / 8; ++nt) {
        const int c = 8 * nt + 2 * t;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = row + 8 * half;
            if (r < P && c < N) *(float2 *)(dst + (long long)r * N + c) = make_float2(s[nt][2 * half], s[nt][2 * half + 1]);
        }
    }
}

template <int NP>
__global__ void __launch_bounds__(kThreads, 2) delta_scan_fwd(const ChunkParams cp) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    ScanStage<NP> *stage = (ScanStage<NP> *)smem_raw;
    constexpr int LINE = NP * 2;
    const DeltaParams &p = cp.p;
    const int nsl = (p.P + 63) / 64, slice = blockIdx.x % nsl, bh = blockIdx.x / nsl, bi = bh / p.H, h = bh % p.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int V = valid_tokens(p, bi), nv = (V + kChunk - 1) / kChunk;
    const int row = slice * 64 + 16 * warp + g;
    const long long sbase = (long long)bh * p.P * p.N;

    float s[NP / 8][4];
    load_state<NP>(s, p.init ? p.init + sbase : nullptr, row, p.P, p.N, t);
    if (nv > 0) load_scan_stage<NP>(stage[0], cp, bi, h, slice, 0, V);
    cp_async_commit();

    for (int c = 0; c < nv; ++c) {
        cp_async_wait<0>();
        __syncthreads();  // this chunk's tiles are complete, the other stage is free
        if (c + 1 < nv) load_scan_stage<NP>(stage[(c + 1) & 1], cp, bi, h, slice, c + 1, V);
        cp_async_commit();
        ScanStage<NP> &st = stage[c & 1];
        const uint32_t ks = smem_u32(st.k), qs = smem_u32(st.q), vs = smem_u32(st.v);
        const uint32_t th = smem_u32(st.img + kImgT), ah_ = smem_u32(st.img + kImgA);
        const float *gates = (const float *)(st.img + kImgGates);

        // S^T K^T and S^T Q^T
        float x[8][4], o[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = o[i][e] = 0.f;
        const int brow = (lane & 7) + ((lane >> 4) & 1) * 8, bcol = (lane >> 3) & 1;
#pragma unroll
        for (int kst = 0; kst < NP / 16; ++kst) {
            uint32_t hi[4], lo[4];
            split_frag(s[2 * kst], s[2 * kst + 1], hi, lo);
            uint32_t b[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) ldsm4(b[j], ks + swz<LINE>(16 * j + brow, 2 * kst + bcol));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mma16(x[2 * j], hi, b[j][0], b[j][1]);
                mma16(x[2 * j + 1], hi, b[j][2], b[j][3]);
            }
            uint32_t bq[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) ldsm4(bq[j], qs + swz<LINE>(16 * j + brow, 2 * kst + bcol));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mma16(o[2 * j], hi, bq[j][0], bq[j][1]);
                mma16(o[2 * j + 1], hi, bq[j][2], bq[j][3]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mma16(x[2 * j], lo, b[j][0], b[j][1]);
                mma16(x[2 * j + 1], lo, b[j][2], b[j][3]);
                mma16(o[2 * j], lo, bq[j][0], bq[j][1]);
                mma16(o[2 * j + 1], lo, bq[j][2], bq[j][3]);
            }
        }
        // X0 = V - e^gamma (K S)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t r[4];
            ldsm4t(r, vs + swz<128>(16 * j + brow, 2 * warp + bcol));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float(&d)[4] = x[2 * j + u];
                const float2 eg = *(const float2 *)(gates + 8 * (2 * j + u) + 2 * t);
                d[0] = __uint_as_float(r[2 * u] << 16) - eg.x * d[0];
                d[1] = __uint_as_float(r[2 * u] & 0xFFFF0000u) - eg.y * d[1];
                d[2] = __uint_as_float(r[2 * u + 1] << 16) - eg.x * d[2];
                d[3] = __uint_as_float(r[2 * u + 1] & 0xFFFF0000u) - eg.y * d[3];
                float(&oo)[4] = o[2 * j + u];
                oo[0] *= p.scale * eg.x;
                oo[1] *= p.scale * eg.y;
                oo[2] *= p.scale * eg.x;
                oo[3] *= p.scale * eg.y;
            }
        }
        // Z = X0 + Tt (beta X0): token blocks from the last, so that a block is an operand before it is added to
        const float *be = gates + 2 * kChunk;
#pragma unroll
        for (int j = 3; j >= 0; --j) {
            uint32_t hi[4], lo[4];
            split_frag(x[2 * j], x[2 * j + 1], *(const float2 *)(be + 16 * j + 2 * t),
                       *(const float2 *)(be + 16 * j + 8 + 2 * t), hi, lo);
#pragma unroll
            for (int i = j; i < 4; ++i) {
                uint32_t bh_[4], bl_[4];
                const uint32_t at = th + blk_at(i, j) * 512 + blk_swz(brow, bcol);
                ldsm4(bh_, at);
                ldsm4(bl_, at + kTri);
                mma16(x[2 * i], hi, bh_[0], bh_[1]);
                mma16(x[2 * i + 1], hi, bh_[2], bh_[3]);
                mma16(x[2 * i], lo, bh_[0], bh_[1]);
                mma16(x[2 * i + 1], lo, bh_[2], bh_[3]);
                mma16(x[2 * i], hi, bl_[0], bl_[1]);
                mma16(x[2 * i + 1], hi, bl_[2], bl_[3]);
            }
        }
        // U = beta Z;  O += U A^T;  S = e^gamma_C S + (U e^(gamma_C - gamma))^T K
        const float ec = gates[kChunk - 1];
#pragma unroll
        for (int nt = 0; nt < NP / 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] *= ec;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t hi[4], lo[4];
            const float2 b0 = *(const float2 *)(be + 16 * j + 2 * t), b1 = *(const float2 *)(be + 16 * j + 8 + 2 * t);
            split_frag(x[2 * j], x[2 * j + 1], b0, b1, hi, lo);
#pragma unroll
            for (int i = j; i < 4; ++i) {
                uint32_t b[4];
                ldsm4(b, ah_ + blk_at(i, j) * 512 + blk_swz(brow, bcol));
                mma16(o[2 * i], hi, b[0], b[1]);
                mma16(o[2 * i + 1], hi, b[2], b[3]);
                mma16(o[2 * i], lo, b[0], b[1]);
                mma16(o[2 * i + 1], lo, b[2], b[3]);
            }
            const float2 e0 = *(const float2 *)(gates + kChunk + 16 * j + 2 * t);
            const float2 e1 = *(const float2 *)(gates + kChunk + 16 * j + 8 + 2 * t);
            split_frag(x[2 * j], x[2 * j + 1], make_float2(b0.x * e0.x, b0.y * e0.y), make_float2(b1.x * e1.x, b1.y * e1.y),
                       hi, lo);
#pragma unroll
            for (int np = 0; np < NP / 16; ++np) {
                uint32_t b[4];
                ldsm4t(b, ks + swz<LINE>(16 * j + (lane & 15), 2 * np + (lane >> 4)));
                mma16(s[2 * np], hi, b[0], b[1]);
                mma16(s[2 * np + 1], hi, b[2], b[3]);
                mma16(s[2 * np], lo, b[0], b[1]);
                mma16(s[2 * np + 1], lo, b[2], b[3]);
            }
        }
        // o: transposed through the warp's own columns of the v tile
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            stsm4t(vs + swz<128>(16 * j + brow, 2 * warp + bcol), tc::pack_bf2(o[2 * j][0], o[2 * j][1]),
                   tc::pack_bf2(o[2 * j][2], o[2 * j][3]), tc::pack_bf2(o[2 * j + 1][0], o[2 * j + 1][1]),
                   tc::pack_bf2(o[2 * j + 1][2], o[2 * j + 1][3]));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 16 * i + (lane >> 1), cc = 2 * warp + (lane & 1), tok = c * kChunk + r;
            if (tok < p.L && slice * 64 + cc * 8 < p.P)
                *(uint4 *)((bf16 *)p.o + (((long long)bi * p.L + tok) * p.H + h) * p.P + slice * 64 + cc * 8) =
                    *(const uint4 *)(st.v + swz<128>(r, cc));
        }
    }
    // absent tokens past the last chunk
    for (int i = nv * kChunk * 8 + threadIdx.x; i < p.L * 8; i += kThreads) {
        const int tok = i / 8, cc = i % 8;
        if (slice * 64 + cc * 8 < p.P)
            *(uint4 *)((bf16 *)p.o + (((long long)bi * p.L + tok) * p.H + h) * p.P + slice * 64 + cc * 8) = make_uint4(0, 0, 0, 0);
    }
    store_state<NP>(s, p.final_state ? p.final_state + sbase : nullptr, row, p.P, p.N, t);
}

}  // namespace

cudaError_t launch_chunk_forward(const ChunkParams &c, cudaStream_t s) {
    const DeltaParams &p = c.p;
    const unsigned grid = (unsigned)(p.b * p.H * ((p.P + 63) / 64));
    const int bytes = 2 * (int)(p.N <= 64 ? sizeof(ScanStage<64>) : sizeof(ScanStage<128>));
    auto kernel = p.N <= 64 ? delta_scan_fwd<64> : delta_scan_fwd<128>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, bytes, s>>>(c);
    return cudaGetLastError();
}

}  // namespace delta
}  // namespace ssd
