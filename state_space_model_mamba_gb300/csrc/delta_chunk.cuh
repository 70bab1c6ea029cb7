// delta_chunk.cuh -- the chunked gated delta rule: layout of what the chunk
// kernels pass to one another (delta_prep.cu, delta_scan.cu, delta_grad.cu).
//
// A chunk is 64 tokens; within it, with gamma the running sum of g,
// D_ij = exp(gamma_i - gamma_j) for j <= i, and S the state before the chunk:
//     E  = D o strict lower (K K^T)
//     (I + E diag(beta)) Z = V - e^gamma o (K S),     U = beta o Z
//     O  = scale e^gamma o (Q S) + A U,               A = scale D o lower (Q K^T)
//     S' = e^gamma_C S + K^T (e^(gamma_C - gamma) o U)
// The inverse is kept as (I + E diag(beta))^-1 = I + Tt diag(beta), Tt strictly
// lower triangular, so that beta = 0 needs no division anywhere:
//     Z = X0 + Tt (beta o X0)  for X0 = V - e^gamma o (K S),
// and, in the backward, X = dU + Tt^T (beta o dU), dV = beta o X.
//
// The chunk image of one (b, h, chunk): lower triangles of 16x16 bf16 blocks
// (10 of 64; blk_at, blk_swz) of Tt and A, each as hi and lo parts, and the gate
// vectors in fp32.
#pragma once
#include "delta_internal.cuh"

namespace ssd {
namespace delta {

constexpr int kChunk = 64;
constexpr int kTri = 10 * 512;                 // bytes of one lower triangle of blocks
constexpr int kGates = 3 * kChunk * 4;         // e^gamma, e^(gamma_C - gamma), beta
// image layout: gates, Tt hi, Tt lo, A hi, A lo.  The forward reads all but A lo.
constexpr int kImgGates = 0, kImgT = kGates, kImgA = kGates + 2 * kTri;
constexpr int kImgFwd = kGates + 3 * kTri, kImgBytes = kGates + 4 * kTri;

struct ChunkParams {
    DeltaParams p;
    int n;           // chunks
    char *img;       // [b, H, n] images
};

inline bool chunk_supported(const delta_dims &d, ssd_dtype t) {
    return t == SSD_BF16 && !(d.flags & DELTA_FLAG_SIMT) && d.headdim % 8 == 0 && d.dstate % 8 == 0 &&
           d.headdim <= 128 && d.dstate <= 128;
}
inline int chunk_count(long long L) { return (int)((L + kChunk - 1) / kChunk); }

cudaError_t launch_chunk_prep(const ChunkParams &c, cudaStream_t s);
cudaError_t launch_chunk_forward(const ChunkParams &c, cudaStream_t s);

}  // namespace delta
}  // namespace ssd
