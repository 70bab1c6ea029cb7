// window_tile.cuh -- what the tensor-core kernels of window attention share: how
// queries and keys are cut into tiles, and which pairs of tiles and which elements of them are seen.
//
// A query tile is 128 rows: T = floor(128 / R) tokens times the R = H / G heads of a key group, row
// r = token * R + head, so that heads that share keys share their tiles, and few tokens stick out of a
// window's two edges.  Key tiles have up to 128 keys: from the first key of the window on, wherever that is (a copy's token
// coordinate has no alignment), and then the sinks in front of it, from key 0 (a few sinks first would make a
// poor first reference of the softmax: 1 x 65536 tokens of 32 heads of 128 967 us, last 886).
#pragma once
#include <cuda.h>

#include "delta_chunk.cuh"  // encode_tiles
#include "delta_mma.cuh"
#include "window_internal.cuh"

namespace ssd {
namespace window {

using tc::mbar_arrive;
using tc::mbar_arrive_expect_tx;
using tc::mbar_init;
using tc::mbar_wait;
using tc::smem_u32;

constexpr int kTileRows = 128;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

inline bool tile_supported(const window_dims &d, ssd_dtype t, bool backward) {
    return t == SSD_BF16 && !(d.flags & WINDOW_FLAG_SIMT) && d.headdim % 8 == 0 && d.nheads / d.ngroups <= (backward ? 64 : kTileRows);
}
__host__ __device__ __forceinline__ int tile_tokens(const WindowParams &p) { return kTileRows / p.hpg; }
// r / R for a row of a tile: with m = ceil(2^16 / R) the product is off by less than r / 2^16 < 1 / R
__device__ __forceinline__ int row_token(int r, uint32_t m) { return (int)((r * m) >> 16); }
__host__ __device__ __forceinline__ uint32_t row_magic(int R) { return (65536u + R - 1) / R; }

// True in one lane of a converged warp.  Where products and copies are issued behind this instruction the compiler knows
// that one lane is left and takes their operands as they are; behind `lane == 0` the issuing warp took 104 to 150 cycles for
// a product that the tensor core does in 64.
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// A wait in two parts: what is over already is a few instructions in line, the rest a loop.  After 2 s, or once any wait
// of the block has given up, it gives up and says so in `err`; the caller goes on, with values that nobody will use, and
// every later wait of the block ends at once.
__device__ __forceinline__ void wait_loop(uint64_t *bar, uint32_t parity, int *err) {
    const uint64_t t0 = tc::global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (tc::mbar_try_wait(bar, parity)) return;
        if ((it & 63u) == 0u && (*(volatile int *)err || tc::global_timer_ns() - t0 > tc::kWaitLimitNs)) {
            *(volatile int *)err = 1;
            return;
        }
    }
}
__device__ __noinline__ inline void wait_long(uint64_t *bar, uint32_t parity, int *err) { wait_loop(bar, parity, err); }
__device__ __forceinline__ void wait_bar(uint64_t *bar, uint32_t parity, int *err) {
    if (!tc::mbar_try_wait(bar, parity)) wait_long(bar, parity, err);
}
// The copying threads' wait: false once a wait of the block has given up, and then nothing more is copied (a barrier that
// nobody waits for would count bytes past its range).
__device__ __forceinline__ bool wait_copy(uint64_t *bar, uint32_t parity, int *err) {
    wait_bar(bar, parity, err);
    return *(volatile int *)err == 0;
}
// The same for whole warps with registers full of values, that a call would have to put away.
__device__ __forceinline__ void wait_warp(uint64_t *bar, uint32_t parity, int *err) {
    if (!tc::mbar_try_wait(bar, parity)) wait_loop(bar, parity, err);
    __syncwarp();
}

// One arrival for the warp, from lane 0, without a branch (each costs a warp some 20 cycles); after a warp-wide
// instruction on tensor memory the lanes need no other meeting point.
__device__ __forceinline__ void arrive_first(uint64_t *bar, int lane) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.eq.s32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(lane)
        : "memory");
}

// The query tiles (place x in the row, key group g, batch row b) of a block: numbers blockIdx.x, + gridDim.x, ... of all of them, counted
// from the rows' ends, every row's last tile before any other: rows advance together, so their windows stay in the L2
// cache, and the tiles at a row's start, which see few keys, come last, where blocks run out of work.  No divisions after the first.
struct Cursor {
    int x, g, b, dx, dg, db, G, B, left;
    __device__ __forceinline__ Cursor(int items, int per_row, const WindowParams &p) : G(p.G), B(p.b) {
        const int rows = G * B;
        x = per_row - 1 - (int)blockIdx.x / rows, g = blockIdx.x % rows % G, b = blockIdx.x % rows / G;
        dx = gridDim.x / rows, dg = gridDim.x % rows % G, db = gridDim.x % rows / G;
        left = (items - 1 - (int)blockIdx.x) / (int)gridDim.x + 1;
    }
    __device__ __forceinline__ void next() {
        x -= dx, g += dg, b += db, --left;
        if (g >= G) g -= G, ++b;
        if (b >= B) b -= B, --x;
    }
};

// Blocks for `items` tiles, at most `most`.  Block i takes tiles i, i + grid, ..., tile n is of batch row n % (G b) / G: where the rows differ
// in length the grid's common divisor with G b is at most G, so that every block comes round all of them (8 padded rows of 8 groups,
// whose 304 blocks met either the even rows or the odd; 16 rows of up to 2048, 32 heads of 128 over 4: 195 us, 187 now).
inline int tile_grid(const WindowParams &p, int items, int most) {
    if (items <= most || !p.valid_len) return items < most ? items : most;
    for (;; --most) {
        int a = p.G * p.b, c = most;
        while (c) {
            const int r = a % c;
            a = c, c = r;
        }
        if (a <= p.G) return most;
    }
}

// A query tile of T tokens and its keys in tiles of KEYS: [0, tiles_w) the window, [tiles_w, tiles) the sinks in front of it.
template <int KEYS>
struct QueryItem {
    int bi, g, V, head, lo, end, tiles_w, tiles, ta;
    __device__ __forceinline__ QueryItem(const WindowParams &p, const Cursor &c, int T) {
        ta = c.x * T;
        g = c.g;
        bi = c.b;
        V = valid_tokens(p, bi);
        end = min(ta + T, V);
        lo = max(0, ta - p.W + 1);
        head = min(p.sinks, lo);
        tiles_w = ta < V ? (end - lo + KEYS - 1) / KEYS : 0;
        tiles = ta < V ? tiles_w + (head + KEYS - 1) / KEYS : 0;
    }
    __device__ __forceinline__ int start(int j) const { return j < tiles_w ? lo + j * KEYS : (j - tiles_w) * KEYS; }
    __device__ __forceinline__ int count(int j) const { return min(KEYS, (j < tiles_w ? end : head) - start(j)); }
    // whether every row sees every key of tile j: none behind the first token, none in front of the last one's window
    __device__ __forceinline__ bool plain(const WindowParams &p, int T, int s0, int nk) const {
        return nk == KEYS && s0 + KEYS - 1 <= ta && (s0 > ta + T - 1 - p.W || s0 + KEYS <= p.sinks);
    }
};
// A place in a ring of SLOTS and the parity of its phase.
template <int SLOTS>
struct Place {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == SLOTS) slot = 0, phase ^= 1;
    }
};

// the largest of three
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// bits [lo, hi) of 32, either may be out of range
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
    lo = lo < 0 ? 0 : lo;
    hi = hi > 32 ? 32 : hi;
    if (lo >= hi) return 0u;
    return (0xffffffffu >> (32 - (hi - lo))) << lo;
}

// 80 consecutive fp32 columns of this warp's 32 lanes, one wait.
__device__ __forceinline__ void tmem_ld80(uint32_t taddr, float *v) {
    uint32_t r[80];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%80];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79}, [%81];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]), "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79])
        : "r"(taddr + 0), "r"(taddr + 64)
        : "memory");
#pragma unroll
    for (int i = 0; i < 80; ++i) v[i] = __uint_as_float(r[i]);
}
// Two sets of 48 columns, one wait.
__device__ __forceinline__ void tmem_ld48x2(uint32_t t0, uint32_t t1, float *v0, float *v1) {
    uint32_t r[96];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%96];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47}, [%97];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79}, [%98];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95}, [%99];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]), "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]), "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]), "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95])
        : "r"(t0 + 0), "r"(t0 + 32), "r"(t1 + 0), "r"(t1 + 32)
        : "memory");
#pragma unroll
    for (int i = 0; i < 48; ++i) v0[i] = __uint_as_float(r[i]), v1[i] = __uint_as_float(r[48 + i]);
}
// 8 and 32 packed 32-bit columns (the caller waits for its stores)
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// A warp's 32 rows x 64 columns in bf16 from its stage to rows of global memory, as whole lines: row r of the tile
// goes to dst + off(r) where r < rows.
template <class F>
__device__ __forceinline__ void store_lines(uint32_t stage, int quarter, int lane, bf16 *dst, int rows, int col, int P, F off) {
    const int c = col + 8 * (lane & 7);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int r = 4 * e + (lane >> 3), rr = 32 * quarter + r;
        const uint4 y = tc::ld_shared_v4(stage + tc::sw128_chunk(r, lane & 7));
        if (rr < rows && c < P) *(uint4 *)(dst + off(rr) + c) = y;
    }
}
// Columns [at, at + 64) of a warp's accumulator rows times f, rounded, to the warp's stage; zeros where f is 0 or none is filled.
__device__ __forceinline__ void stage_rows(uint32_t stage, uint32_t at, int lane, float f, bool filled) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float v[32];
        if (filled) {
            __syncwarp();
            tc::tmem_ld32u(at + 32 * q, (uint32_t *)v);
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0.f;
        }
        uint32_t y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = f != 0.f ? tc::pack_bf2(v[2 * e] * f, v[2 * e + 1] * f) : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            tc::st_shared_v4(stage + tc::sw128_chunk(lane, 4 * q + e), y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
    }
}

// Tensor maps of [b, L, heads, P] in bf16, 64 columns (128 bytes, swizzled) x `nheads` heads x `tokens` tokens a box.
inline cudaError_t map_tokens(CUtensorMap *m, const void *ptr, const WindowParams &p, int heads, int nheads, int tokens) {
    const cuuint64_t dims[4] = {(cuuint64_t)p.P, (cuuint64_t)heads, (cuuint64_t)p.L, (cuuint64_t)p.b};
    const cuuint64_t row = (cuuint64_t)p.P * 2;
    const cuuint64_t strides[3] = {row, heads * row, (cuuint64_t)p.L * heads * row};
    const cuuint32_t box[4] = {64, (cuuint32_t)nheads, (cuuint32_t)tokens, 1};
    return delta::encode_tiles(m, ptr, 4, dims, strides, box);
}
}  // namespace window
}  // namespace ssd
