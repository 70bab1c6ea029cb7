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
// The forward takes A through the inverse, so that one operand (beta o X0) gives both
// the errors and the outputs:  A U = At (beta o X0),  At = A (I + diag(beta) Tt).
//
// The chunk image of one (b, h, chunk) is what the scans copy to shared memory: the
// gate vectors in fp32, then two matrices as hi and lo bf16 parts, kept as the tensor
// core reads them without swizzle, in 8x8 matrices of 128 contiguous bytes.
//   forward:  Tt rows stacked on At rows.  Columns 16 ks .. 16 ks + 15 are one run of the 16 row
//     octets, two matrices each, from octet 2 ks on (the first 2 ks octets of Tt are zero and
//     not stored; those of At are stored, as the run goes on over them): few copies of some
//     kilobytes, for a copy costs its issuing warp some 70 cycles whatever its size.
//   backward: Tt, A as full squares, column octet by column octet, so that the same bytes serve
//     as Tt and, read along the other axis, as Tt^T.
#pragma once
#include <cuda.h>

#include "delta_internal.cuh"

namespace ssd {
namespace delta {

constexpr int kChunk = 64;
// e^gamma, e^(gamma_C - gamma), beta; then pairs gamma log2(e) as hi and lo
constexpr int kGates = 5 * kChunk * 4;
// forward: run ks of a part: its first byte and its length; the 16-byte piece of row i (0 .. 127), columns 8 c .. + 7
__host__ __device__ constexpr int run_bytes(int ks) { return (16 - 2 * ks) * 256; }
__host__ __device__ constexpr int run_at(int ks) { return 4096 * ks - 256 * ks * (ks - 1); }
constexpr int kPart = run_at(4);
__host__ __device__ constexpr int run_piece(int i, int c) {
    return run_at(c >> 1) + ((i >> 3) - (c & ~1)) * 256 + (c & 1) * 128 + (i & 7) * 16;
}
static_assert(kPart == 13312 && run_at(3) + run_bytes(3) == kPart, "runs");
// backward: [Tt hi, Tt lo, A hi, A lo][8 column octets][8 row octets][128 bytes]
constexpr int kSquare = 8192;
__host__ __device__ constexpr int square_piece(int i, int c) { return c * 1024 + (i >> 3) * 128 + (i & 7) * 16; }
// image: gates, then the parts or the squares
constexpr int kImgMat = kGates, kImgFwd = kGates + 2 * kPart, kImgBwd = kGates + 4 * kSquare;

// What the backward's kernels keep, per (b, h) chain and slice of 64 columns of P (chain-slice
// cs = bh * nsl + slice).  Tiles are in the 128-byte swizzle, ready as operands.
//   states [cs, n]          S before every chunk: hi, lo parts [128 n][64] (32 KB)
//   dstates [cs, n]         dS after every chunk: hi, lo parts [128 n][64] (32 KB)
//   errs   [cs, n]          Z: hi, lo parts [64 tokens][64] (16 KB)
//   dv_lo  [cs, n]          what dV lost to its rounding: [64 tokens][64] (8 KB)
// dg is the sum of everything that crosses its token inside the chunk, so that no term carries
// less decay than the result (products of whole rows, do.o - dv.v and <S, dS>, would be the same sum
// but cancel where a head forgets fast, and so would sums that a token's own share is taken off again):
//     dg_t = ss + sum_{j < t} ww_j + sum_{i >= t} (fq_i + fk_i) + sum_{i >= t} sum_{j < t} P_ij
//     ss = e^gamma_C <S, dS>            S before, dS after the chunk    [cs, n, 16], a share of each warp
//     ww = beta Z.(e^(gamma_C - gamma) K dS),  zx = Z.X                 [cs, 4, n * 64], sums over 16 columns
//     fq = q.(scale e^gamma dO S^T),  fk = -k.(e^gamma dV S^T)          [cs, 2, n * 64], over 64 of the keys' columns
//     P = Nm o Q K^T + M o K K^T, as pe                                 [cs, n, 384]:
//       0 .. 127: each row's sum over columns 0 .. 31 (Nm, then M)
//       128 + 64 r + t: over the rows i >= t of quarter r (Nm, Nm, M, M), the columns before t of t's own half
// and dbeta = zx.
struct ChunkBackward {
    char *states, *dstates, *errs, *dv_lo;
    float *ss, *ww, *zx, *fq, *fk, *pe;
};

struct ChunkParams {
    DeltaParams p;
    int n;           // chunks
    int img_bytes;   // kImgFwd or kImgBwd
    char *img;       // [b, H, n] images
    ChunkBackward w; // pointers are null in the forward
    __host__ __device__ char *image(long long bh, int chunk) const { return img + (bh * n + chunk) * (long long)img_bytes; }
};
constexpr int kCrossSums = 384;
constexpr int kStateTile = 32768, kDStateTile = 32768, kErrTile = 16384, kDvLoTile = 8192;
__host__ __device__ __forceinline__ int slices_of(const DeltaParams &p) { return (p.P + 63) / 64; }

inline bool chunk_supported(const delta_dims &d, ssd_dtype t) {
    return t == SSD_BF16 && !(d.flags & DELTA_FLAG_SIMT) && d.headdim % 8 == 0 && d.dstate % 8 == 0 &&
           d.headdim <= 128 && d.dstate <= 128;
}
inline int chunk_count(long long L) { return (int)((L + kChunk - 1) / kChunk); }

// Tensor map of bf16 tiles in the 128-byte swizzle, zeros outside (delta_maps.cu).
cudaError_t encode_tiles(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                         const cuuint32_t *box);
// The map `like` of a tensor with the same shape at another address.
cudaError_t same_tiles(CUtensorMap *m, const CUtensorMap &like, const void *base);
// [b, L, heads, width] bf16: boxes of 64 columns of one head x a chunk's (or fewer) tokens
inline cudaError_t map_chunk_tokens(CUtensorMap *m, const void *ptr, int b, int L, int heads, int width,
                                    int tokens = kChunk) {
    const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)L, (cuuint64_t)b};
    const cuuint64_t strides[3] = {(cuuint64_t)width * 2, (cuuint64_t)heads * width * 2, (cuuint64_t)L * heads * width * 2};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)tokens, 1};
    return encode_tiles(m, ptr, 4, dims, strides, box);
}

// and the status words, over status_rows of valid_len (0: left alone)
cudaError_t launch_chunk_prep(const ChunkParams &c, int status_rows, cudaStream_t s);
cudaError_t launch_chunk_forward(const ChunkParams &c, cudaStream_t s);   // with c.w: the backward's recompute
cudaError_t launch_chunk_reverse(const ChunkParams &c, cudaStream_t s);   // dS, dv and the gates' sums
cudaError_t launch_chunk_grads(const ChunkParams &c, cudaStream_t s);     // dq, dk, dg, dbeta

}  // namespace delta
}  // namespace ssd
