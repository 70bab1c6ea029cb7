// window_tile.cuh -- what the tensor-core kernels of window attention share: how
// queries and keys are cut into tiles, and which pairs of tiles and which elements of them are seen.
//
// A query tile is 128 rows: T = floor(128 / R) tokens times the R = H / G heads of a key group, row
// r = token * R + head, so that heads that share keys share their tiles, and few tokens stick out of a
// window's two edges.  Key tiles are 128 keys: first the sinks in front of the window, from key 0, then
// from the first key of the window on, wherever that is (a copy's token coordinate has no alignment).
#pragma once
#include <cuda.h>

#include "delta_mma.cuh"
#include "window_internal.cuh"

namespace ssd {
namespace window {

using tc::mbar_arrive;
using tc::mbar_arrive_expect_tx;
using tc::mbar_init;
using tc::mbar_wait;
using tc::smem_u32;

constexpr int kTileRows = 128, kSMs = 152;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

inline bool tile_supported(const window_dims &d, ssd_dtype t) {
    return t == SSD_BF16 && !(d.flags & WINDOW_FLAG_SIMT) && d.headdim % 8 == 0 && d.nheads / d.ngroups <= kTileRows;
}
__host__ __device__ __forceinline__ int tile_tokens(const WindowParams &p) { return kTileRows / p.hpg; }

// True in one lane of a converged warp.  Where products and copies are issued behind this instruction the compiler knows
// that one lane is left and takes their operands as they are; behind `lane == 0` it wraps each product in some 400
// bytes of code, and the issuing warp took 104 to 150 cycles for what the tensor core does in 64.
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// bits [lo, hi) of 32, either may be out of range
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
    lo = lo < 0 ? 0 : lo;
    hi = hi > 32 ? 32 : hi;
    if (lo >= hi) return 0u;
    return (0xffffffffu >> (32 - (hi - lo))) << lo;
}

// Tensor maps of [b, L, heads, P] in bf16, 64 columns (128 bytes, swizzled) x `nheads` heads x `tokens` tokens a box.
inline cudaError_t map_tokens(CUtensorMap *m, const void *ptr, const WindowParams &p, int heads, int nheads, int tokens);

}  // namespace window
}  // namespace ssd

#include "delta_chunk.cuh"  // encode_tiles

namespace ssd {
namespace window {
inline cudaError_t map_tokens(CUtensorMap *m, const void *ptr, const WindowParams &p, int heads, int nheads, int tokens) {
    const cuuint64_t dims[4] = {(cuuint64_t)p.P, (cuuint64_t)heads, (cuuint64_t)p.L, (cuuint64_t)p.b};
    const cuuint64_t row = (cuuint64_t)p.P * 2;
    const cuuint64_t strides[3] = {row, heads * row, (cuuint64_t)p.L * heads * row};
    const cuuint32_t box[4] = {64, (cuuint32_t)nheads, (cuuint32_t)tokens, 1};
    return delta::encode_tiles(m, ptr, 4, dims, strides, box);
}
}  // namespace window
}  // namespace ssd
