// delta_api.cu -- the C ABI declared in include/delta.h: argument checks,
// workspace carving and the launch sequences of the gated delta rule.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <map>
#include <memory>
#include <mutex>
#include <type_traits>
#include <utility>

#include "delta_chunk.cuh"

namespace ssd {
namespace delta {
namespace {

ssd_status fail(ssd_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
ssd_status fail(ssd_status st, const char *fmt, ...) {
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    record_error(msg);
    return st;
}
bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

ssd_status validate(const delta_dims *d, ssd_dtype dt) {
    if (!d) return fail(SSD_ERR_INVALID_ARG, "dims is NULL");
    if (dt != SSD_F32 && dt != SSD_BF16) return fail(SSD_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (d->reserved != 0) return fail(SSD_ERR_INVALID_ARG, "dims.reserved must be 0");
    if (d->flags & ~(uint32_t)DELTA_FLAG_SIMT) return fail(SSD_ERR_INVALID_ARG, "unknown flags 0x%x", d->flags);
    if (d->batch < 1 || d->seqlen < 1 || d->nheads < 1 || d->headdim < 1 || d->dstate < 1 || d->ngroups < 1)
        return fail(SSD_ERR_INVALID_ARG, "every dimension must be >= 1");
    if (d->nheads % d->ngroups != 0)
        return fail(SSD_ERR_INVALID_ARG, "nheads (%lld) must be a multiple of ngroups (%lld)", (long long)d->nheads,
                    (long long)d->ngroups);
    if (d->headdim > 128 || d->headdim % 4 != 0)
        return fail(SSD_ERR_UNSUPPORTED, "headdim %lld: need a multiple of 4 <= 128", (long long)d->headdim);
    if (d->dstate > 256 || d->dstate % 4 != 0)
        return fail(SSD_ERR_UNSUPPORTED, "dstate %lld: need a multiple of 4 <= 256", (long long)d->dstate);
    // index and grid limits
    if (d->seqlen > (1LL << 30) || d->batch > (1LL << 24) || d->nheads > (1LL << 20) ||
        (double)d->batch * d->nheads * ((d->seqlen + 63) / 64) > 2.0e9 || (double)d->batch * d->nheads > 2.0e8 ||
        (double)d->batch * d->seqlen * d->nheads * 256.0 > 4.0e11)
        return fail(SSD_ERR_UNSUPPORTED, "problem too large");
    return SSD_OK;
}

ssd_status check_pointers(const void *const *req, const char *const *names, int nreq, const void *const *opt, int nopt) {
    for (int i = 0; i < nreq; ++i) {
        if (!req[i]) return fail(SSD_ERR_INVALID_ARG, "%s is NULL", names[i]);
        if (!aligned16(req[i])) return fail(SSD_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
    }
    for (int i = 0; i < nopt; ++i)
        if (opt[i] && !aligned16(opt[i])) return fail(SSD_ERR_INVALID_ARG, "state pointers must be 16-byte aligned");
    return SSD_OK;
}

ssd_status cuda_status(cudaError_t e) {
    return e == cudaSuccess ? SSD_OK : fail(SSD_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
}

// Nothing thrown below (locks, the table of streams) leaves a C entry.
template <class F>
ssd_status guarded(F launches) {
    try {
        return cuda_status(launches());
    } catch (...) {
        return fail(SSD_ERR_CUDA, "launch failed: a host resource could not be had");
    }
}

constexpr size_t kStatusBytes = 1024;  // status words, then the paths' own buffers

DeltaParams base_params(const delta_dims &d, const void *q, const void *k, const void *v, const float *g,
                        const float *beta, float scale, const float *init, const int32_t *valid_len, void *ws) {
    DeltaParams p;
    memset(&p, 0, sizeof(p));
    p.b = (int)d.batch;
    p.L = (int)d.seqlen;
    p.H = (int)d.nheads;
    p.P = (int)d.headdim;
    p.N = (int)d.dstate;
    p.G = (int)d.ngroups;
    p.hpg = p.H / p.G;
    p.scale = scale;
    p.q = q;
    p.k = k;
    p.v = v;
    p.g = g;
    p.beta = beta;
    p.init = init;
    p.valid_len = valid_len;
    p.status = (int *)ws;
    return p;
}

// The chunked path's buffers behind the status words: the images, then what the backward keeps.
size_t carve(const delta_dims &d, bool backward, char *ws, ChunkParams *c) {
    const size_t n = chunk_count(d.seqlen), chains = (size_t)d.batch * d.nheads, nsl = (d.headdim + 63) / 64, cs = chains * nsl;
    size_t off = kStatusBytes;
    auto take = [&](size_t bytes) {
        char *at = ws + off;
        off += (bytes + 1023) / 1024 * 1024;
        return at;
    };
    const int img_bytes = backward ? kImgBwd : kImgFwd;
    char *img = take(chains * n * img_bytes);
    ChunkBackward w;
    memset(&w, 0, sizeof(w));
    if (backward) {
        w.states = take(cs * n * kStateTile);
        w.dstates = take(cs * n * kDStateTile);
        w.errs = take(cs * n * kErrTile);
        w.dv_lo = take(cs * n * kDvLoTile);
        w.ss = (float *)take(cs * n * 16 * 4);
        for (float **x : {&w.ww, &w.zx}) *x = (float *)take(cs * 4 * n * kChunk * 4);
        for (float **x : {&w.fq, &w.fk}) *x = (float *)take(cs * 2 * n * kChunk * 4);
        w.pe = (float *)take(cs * n * kCrossSums * 4);
    }
    if (c) {
        c->n = (int)n;
        c->img_bytes = img_bytes;
        c->img = img;
        c->w = w;
    }
    return off;
}

// The same problem, batch rows b0 .. b0 + nb - 1 of it.
ChunkParams batch_part(const ChunkParams &all, int b0, int nb) {
    ChunkParams c = all;
    DeltaParams &p = c.p;
    const size_t keys = (size_t)b0 * p.L * p.G * p.N, values = (size_t)b0 * p.L * p.H * p.P, gates = (size_t)b0 * p.H * p.L,
                 state = (size_t)b0 * p.H * p.P * p.N, cs = (size_t)b0 * p.H * slices_of(p);
    auto move = [](auto *&x, size_t bytes) {
        if (x) x = (std::remove_reference_t<decltype(x)>)((char *)x + bytes);
    };
    p.b = nb;
    move(p.q, 2 * keys), move(p.k, 2 * keys), move(p.dq, 2 * keys), move(p.dk, 2 * keys);
    move(p.v, 2 * values), move(p.o, 2 * values), move(p.d_o, 2 * values), move(p.dv, 2 * values);
    move(p.g, 4 * gates), move(p.beta, 4 * gates), move(p.dg, 4 * gates), move(p.dbeta, 4 * gates);
    move(p.init, 4 * state), move(p.final_state, 4 * state), move(p.d_final, 4 * state), move(p.d_init, 4 * state);
    move(p.valid_len, 4 * (size_t)b0);
    move(c.img, (size_t)b0 * p.H * c.n * c.img_bytes);
    ChunkBackward &w = c.w;
    move(w.states, cs * c.n * kStateTile), move(w.dstates, cs * c.n * kDStateTile);
    move(w.errs, cs * c.n * kErrTile), move(w.dv_lo, cs * c.n * kDvLoTile);
    move(w.ss, cs * c.n * 16 * 4);
    move(w.ww, cs * 4 * c.n * kChunk * 4), move(w.zx, cs * 4 * c.n * kChunk * 4);
    move(w.fq, cs * 2 * c.n * kChunk * 4), move(w.fk, cs * 2 * c.n * kChunk * 4);
    move(w.pe, cs * c.n * kCrossSums * 4);
    return c;
}

// A second stream per (device, caller stream), as the scan's backward has one (include/ssd.h): created at the
// first call that takes it, kept until the process exits, with a lock from the fork to the join.
struct SideStream {
    cudaStream_t st = nullptr;
    cudaEvent_t fork = nullptr, join = nullptr;
    std::mutex mu;
};
std::mutex g_side_mu;
std::map<std::pair<int, cudaStream_t>, std::unique_ptr<SideStream>> g_side;
cudaError_t side_stream(cudaStream_t caller, SideStream **out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_side_mu);
    std::unique_ptr<SideStream> &slot = g_side[std::make_pair(dev, caller)];
    if (!slot) {
        std::unique_ptr<SideStream> sd(new SideStream);
        if ((e = cudaStreamCreateWithFlags(&sd->st, cudaStreamNonBlocking)) != cudaSuccess) return e;
        if ((e = cudaEventCreateWithFlags(&sd->fork, cudaEventDisableTiming)) != cudaSuccess) return e;
        if ((e = cudaEventCreateWithFlags(&sd->join, cudaEventDisableTiming)) != cudaSuccess) return e;
        slot = std::move(sd);
    }
    *out = slot.get();
    return cudaSuccess;
}

// The backward of two halves of the batch, each on its own stream.  The scans are serial in the chunks, so a last
// wave of few chains leaves most SMs to themselves for as long as a full one; the other half's kernels fill them,
// those of the gradients above all.  2 x 8192 x 80 heads (160 chains on 152 SMs): 2.11 ms for 2.54 when it was added; 3 x 4096 x 64: 1.28 for
// 1.39; 4 x 8192 x 80: 4.28 for 4.45.  Chains that all run at once anyway gain nothing (4 x 2048 x 24: 453 us for
// 440), short ones not the launches.
bool halves(const ChunkParams &c) {
    return c.p.b >= 2 && (long long)c.p.b * c.p.H * slices_of(c.p) > kSMs && c.n >= 16;
}
cudaError_t backward_halves(const ChunkParams &c, cudaStream_t s) {
    const int b0 = (c.p.b + 1) / 2;
    const ChunkParams part[2] = {batch_part(c, 0, b0), batch_part(c, b0, c.p.b - b0)};
    SideStream *sd = nullptr;
    cudaError_t e = side_stream(s, &sd);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(sd->mu);
    const cudaStream_t on[2] = {s, sd->st};
    if ((e = launch_chunk_prep(part[0], c.p.b, s)) != cudaSuccess) return e;
    if ((e = cudaEventRecord(sd->fork, s)) != cudaSuccess) return e;
    if ((e = cudaStreamWaitEvent(sd->st, sd->fork, 0)) != cudaSuccess) return e;
    e = launch_chunk_prep(part[1], 0, sd->st);
    for (auto step : {launch_chunk_forward, launch_chunk_reverse, launch_chunk_grads})
        for (int i = 0; i < 2 && e == cudaSuccess; ++i) e = step(part[i], on[i]);
    // joined whatever failed: the caller's stream waits for all that runs
    const cudaError_t j = cudaEventRecord(sd->join, sd->st), w = j == cudaSuccess ? cudaStreamWaitEvent(s, sd->join, 0) : j;
    return e != cudaSuccess ? e : w;
}

}  // namespace
}  // namespace delta
}  // namespace ssd

using namespace ssd;
using namespace ssd::delta;

extern "C" {

ssd_status delta_supported(const delta_dims *dims, ssd_dtype dtype) {
    record_error("");
    return validate(dims, dtype);
}

size_t delta_workspace_bytes(const delta_dims *dims, ssd_dtype dtype, int backward) {
    record_error("");
    if (validate(dims, dtype) != SSD_OK) return 0;
    if (chunk_supported(*dims, dtype)) return carve(*dims, backward != 0, nullptr, nullptr);
    return kStatusBytes + (backward ? simt_backward_bytes(*dims) : 0);
}

ssd_status delta_forward(const delta_dims *dims, ssd_dtype dtype, const void *q, const void *k, const void *v,
                         const float *g, const float *beta, float scale, const float *init_state,
                         const int32_t *valid_len, void *o, float *final_state, void *workspace,
                         size_t workspace_bytes, void *stream) {
    record_error("");
    ssd_status st = validate(dims, dtype);
    if (st != SSD_OK) return st;
    const void *req[] = {q, k, v, g, beta, o, workspace};
    static const char *const names[] = {"q", "k", "v", "g", "beta", "o", "workspace"};
    const void *opt[] = {init_state, final_state};
    if ((st = check_pointers(req, names, 7, opt, 2)) != SSD_OK) return st;
    const size_t need = delta_workspace_bytes(dims, dtype, 0);
    if (workspace_bytes < need)
        return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
    DeltaParams p = base_params(*dims, q, k, v, g, beta, scale, init_state, valid_len, workspace);
    p.o = o;
    p.final_state = final_state;
    cudaStream_t cs = (cudaStream_t)stream;
    if (!chunk_supported(*dims, dtype)) return cuda_status(launch_simt_forward(p, dtype == SSD_BF16, cs));
    ChunkParams c;
    c.p = p;
    carve(*dims, false, (char *)workspace, &c);
    return guarded([&] {
        const cudaError_t e = launch_chunk_prep(c, p.b, cs);
        return e != cudaSuccess ? e : launch_chunk_forward(c, cs);
    });
}

ssd_status delta_backward(const delta_dims *dims, ssd_dtype dtype, const void *q, const void *k, const void *v,
                          const float *g, const float *beta, float scale, const float *init_state,
                          const int32_t *valid_len, const void *d_o, const float *d_final_state, void *dq, void *dk,
                          void *dv, float *dg, float *dbeta, float *d_init_state, void *workspace,
                          size_t workspace_bytes, void *stream) {
    record_error("");
    ssd_status st = validate(dims, dtype);
    if (st != SSD_OK) return st;
    const void *req[] = {q, k, v, g, beta, d_o, dq, dk, dv, dg, dbeta, workspace};
    static const char *const names[] = {"q", "k", "v", "g", "beta", "do", "dq", "dk", "dv", "dg", "dbeta", "workspace"};
    const void *opt[] = {init_state, d_final_state, d_init_state};
    if ((st = check_pointers(req, names, 12, opt, 3)) != SSD_OK) return st;
    const size_t need = delta_workspace_bytes(dims, dtype, 1);
    if (workspace_bytes < need)
        return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
    DeltaParams p = base_params(*dims, q, k, v, g, beta, scale, init_state, valid_len, workspace);
    p.d_o = d_o;
    p.d_final = d_final_state;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.dg = dg;
    p.dbeta = dbeta;
    p.d_init = d_init_state;
    cudaStream_t cs = (cudaStream_t)stream;
    if (!chunk_supported(*dims, dtype))
        return cuda_status(launch_simt_backward(p, dtype == SSD_BF16, (char *)workspace + kStatusBytes, cs));
    ChunkParams c;
    c.p = p;
    carve(*dims, true, (char *)workspace, &c);
    return guarded([&] {
        if (halves(c)) return backward_halves(c, cs);
        cudaError_t e = launch_chunk_prep(c, p.b, cs);
        for (auto step : {launch_chunk_forward, launch_chunk_reverse, launch_chunk_grads})
            if (e == cudaSuccess) e = step(c, cs);
        return e;
    });
}

ssd_status delta_step(const delta_dims *dims, ssd_dtype dtype, const void *q, const void *k, const void *v,
                      const float *g, const float *beta, float scale, float *state, int64_t slots,
                      const int32_t *state_index, void *o, void *stream) {
    record_error("");
    ssd_status st = validate(dims, dtype);
    if (st != SSD_OK) return st;
    if (dims->seqlen != 1) return fail(SSD_ERR_INVALID_ARG, "delta_step takes one token: seqlen must be 1");
    const void *req[] = {q, k, v, g, beta, state, o};
    static const char *const names[] = {"q", "k", "v", "g", "beta", "state", "o"};
    if ((st = check_pointers(req, names, 7, nullptr, 0)) != SSD_OK) return st;
    if (slots < 1 || slots > (1LL << 31)) return fail(SSD_ERR_INVALID_ARG, "slots %lld out of range", (long long)slots);
    if (!state_index && slots < dims->batch)
        return fail(SSD_ERR_INVALID_ARG, "%lld slots for a batch of %lld without state_index", (long long)slots,
                    (long long)dims->batch);
    DeltaParams p = base_params(*dims, q, k, v, g, beta, scale, nullptr, nullptr, nullptr);
    p.o = o;
    return cuda_status(launch_step(p, dtype == SSD_BF16, state, slots, state_index, (cudaStream_t)stream));
}

}  // extern "C"
