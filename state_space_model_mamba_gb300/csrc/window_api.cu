// window_api.cu -- the C ABI declared in include/window.h: argument checks,
// workspace carving and the launches of window attention.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "window_tile.cuh"

namespace ssd {
namespace window {
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

ssd_status validate(const window_dims *d, ssd_dtype dt) {
    if (!d) return fail(SSD_ERR_INVALID_ARG, "dims is NULL");
    if (dt != SSD_F32 && dt != SSD_BF16) return fail(SSD_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (d->reserved != 0) return fail(SSD_ERR_INVALID_ARG, "dims.reserved must be 0");
    if (d->flags & ~(uint32_t)WINDOW_FLAG_SIMT) return fail(SSD_ERR_INVALID_ARG, "unknown flags 0x%x", d->flags);
    if (d->batch < 1 || d->seqlen < 1 || d->nheads < 1 || d->headdim < 1 || d->ngroups < 1)
        return fail(SSD_ERR_INVALID_ARG, "every dimension must be >= 1");
    if (d->nheads % d->ngroups != 0)
        return fail(SSD_ERR_INVALID_ARG, "nheads (%lld) must be a multiple of ngroups (%lld)", (long long)d->nheads,
                    (long long)d->ngroups);
    if (d->window < 1) return fail(SSD_ERR_INVALID_ARG, "window %lld: a token sees itself, so need >= 1", (long long)d->window);
    if (d->sinks < 0) return fail(SSD_ERR_INVALID_ARG, "sinks %lld: need >= 0", (long long)d->sinks);
    const int unit = dt == SSD_BF16 && !(d->flags & WINDOW_FLAG_SIMT) ? 8 : 4;
    if (d->headdim > 128 || d->headdim % unit != 0)
        return fail(SSD_ERR_UNSUPPORTED, "headdim %lld: need a multiple of %d <= 128", (long long)d->headdim, unit);
    // index and grid limits
    if (d->seqlen > (1LL << 30) || d->batch > (1LL << 24) || d->nheads > (1LL << 16) || d->window > (1LL << 30) ||
        d->sinks > (1LL << 29) || (double)d->batch * d->nheads * ((d->seqlen + 15) / 16) > 2.0e9 ||
        (double)d->batch * d->seqlen * d->nheads * 128.0 > 4.0e11)
        return fail(SSD_ERR_UNSUPPORTED, "problem too large");
    return SSD_OK;
}

ssd_status check_pointers(const void *const *req, const char *const *names, int nreq) {
    for (int i = 0; i < nreq; ++i) {
        if (!req[i]) return fail(SSD_ERR_INVALID_ARG, "%s is NULL", names[i]);
        if (!aligned16(req[i])) return fail(SSD_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
    }
    return SSD_OK;
}

// The kernels' exponents are of base 2: the scale has to stay finite times log2(e).
ssd_status check_scale(float scale) {
    return isfinite(scale * kLog2e) ? SSD_OK : fail(SSD_ERR_INVALID_ARG, "scale %g is not finite in base 2", (double)scale);
}

ssd_status cuda_status(cudaError_t e) {
    return e == cudaSuccess ? SSD_OK : fail(SSD_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
}
// Nothing thrown below (the tensor maps' entry points are looked up once) leaves a C entry.
template <class F>
ssd_status guarded(F launches) {
    try {
        return cuda_status(launches());
    } catch (...) {
        return fail(SSD_ERR_CUDA, "launch failed: a host resource could not be had");
    }
}

constexpr size_t kStatusBytes = 1024;  // status words, then the backward's buffers

size_t up256(size_t v) { return (v + 255) / 256 * 256; }
// Window and sinks as the kernels take them: at most L, and plain causal where both together leave nobody out.
void fit_window(const window_dims &d, int *W, int *sinks) {
    const bool all = d.window + d.sinks >= d.seqlen;
    *W = (int)(all ? d.seqlen : d.window);
    *sinks = (int)(all ? 0 : d.sinks);
}
// The backward's buffers behind the status words.
size_t carve(const window_dims &d, ssd_dtype dt, char *ws, WindowParams *p, float **parts) {
    const size_t delta = up256(4ull * d.batch * d.nheads * d.seqlen);
    if (p) {
        p->delta = (float *)(ws + kStatusBytes);
        *parts = (float *)(ws + kStatusBytes + delta);
    }
    if (!tile_supported(d, dt, true)) return kStatusBytes + delta;
    int W, sinks;
    fit_window(d, &W, &sinks);
    return kStatusBytes + delta + 4 * tile_backward_floats(d.batch, d.seqlen, d.ngroups, d.headdim, W, sinks);
}

WindowParams base_params(const window_dims &d, const void *q, const void *k, const void *v, float scale,
                         const int32_t *valid_len, void *ws) {
    WindowParams p;
    memset(&p, 0, sizeof(p));
    p.b = (int)d.batch;
    p.L = (int)d.seqlen;
    p.H = (int)d.nheads;
    p.P = (int)d.headdim;
    p.G = (int)d.ngroups;
    p.hpg = p.H / p.G;
    fit_window(d, &p.W, &p.sinks);
    p.scale = scale;
    p.q = q;
    p.k = k;
    p.v = v;
    p.valid_len = valid_len;
    p.status = (int *)ws;
    return p;
}

// The ring's shape and slots.
ssd_status check_ring(const window_dims *d, int64_t slots, const int32_t *index) {
    if (slots < 1 || slots > (1LL << 31)) return fail(SSD_ERR_INVALID_ARG, "slots %lld out of range", (long long)slots);
    if (!index && slots < d->batch)
        return fail(SSD_ERR_INVALID_ARG, "%lld slots for a batch of %lld without cache_index", (long long)slots,
                    (long long)d->batch);
    if ((double)slots * ((double)d->window + (double)d->sinks) * d->ngroups * d->headdim > 4.0e17)
        return fail(SSD_ERR_UNSUPPORTED, "cache too large");
    return SSD_OK;
}
RingParams ring_params(const window_dims &d, const void *k, const void *v, void *k_cache, void *v_cache, int64_t slots,
                       const int32_t *index) {
    RingParams p;
    memset(&p, 0, sizeof(p));
    p.b = (int)d.batch;
    p.L = (int)d.seqlen;
    p.H = (int)d.nheads;
    p.P = (int)d.headdim;
    p.G = (int)d.ngroups;
    p.hpg = p.H / p.G;
    p.W = (int)d.window;
    p.sinks = (int)d.sinks;
    p.k = k;
    p.v = v;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.slots = slots;
    p.index = index;
    return p;
}

}  // namespace
}  // namespace window
}  // namespace ssd

using namespace ssd;
using namespace ssd::window;

extern "C" {

ssd_status window_supported(const window_dims *dims, ssd_dtype dtype) {
    record_error("");
    return validate(dims, dtype);
}

size_t window_workspace_bytes(const window_dims *dims, ssd_dtype dtype, int backward) {
    record_error("");
    if (validate(dims, dtype) != SSD_OK) return 0;
    return backward ? carve(*dims, dtype, nullptr, nullptr, nullptr) : kStatusBytes;
}

ssd_status window_forward(const window_dims *dims, ssd_dtype dtype, const void *q, const void *k, const void *v,
                          float scale, const int32_t *valid_len, void *o, float *lse, void *workspace,
                          size_t workspace_bytes, void *stream) {
    record_error("");
    ssd_status st = validate(dims, dtype);
    if (st != SSD_OK) return st;
    const void *req[] = {q, k, v, o, workspace};
    static const char *const names[] = {"q", "k", "v", "o", "workspace"};
    if ((st = check_pointers(req, names, 5)) != SSD_OK) return st;
    if ((st = check_scale(scale)) != SSD_OK) return st;
    if (lse && !aligned16(lse)) return fail(SSD_ERR_INVALID_ARG, "lse is not 16-byte aligned");
    if (workspace_bytes < kStatusBytes)
        return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, kStatusBytes);
    WindowParams p = base_params(*dims, q, k, v, scale, valid_len, workspace);
    p.o = o;
    p.lse = lse;
    return guarded([&] {
        if (tile_supported(*dims, dtype, false)) return launch_tile_forward(p, (cudaStream_t)stream);
        return launch_simt_forward(p, dtype == SSD_BF16, (cudaStream_t)stream);
    });
}

ssd_status window_backward(const window_dims *dims, ssd_dtype dtype, const void *q, const void *k, const void *v,
                           const void *o, const float *lse, const void *d_o, float scale, const int32_t *valid_len,
                           void *dq, void *dk, void *dv, void *workspace, size_t workspace_bytes, void *stream) {
    record_error("");
    ssd_status st = validate(dims, dtype);
    if (st != SSD_OK) return st;
    const void *req[] = {q, k, v, o, lse, d_o, dq, dk, dv, workspace};
    static const char *const names[] = {"q", "k", "v", "o", "lse", "do", "dq", "dk", "dv", "workspace"};
    if ((st = check_pointers(req, names, 10)) != SSD_OK) return st;
    if ((st = check_scale(scale)) != SSD_OK) return st;
    const size_t need = window_workspace_bytes(dims, dtype, 1);
    if (workspace_bytes < need)
        return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
    WindowParams p = base_params(*dims, q, k, v, scale, valid_len, workspace);
    float *parts = nullptr;
    carve(*dims, dtype, (char *)workspace, &p, &parts);
    p.o = const_cast<void *>(o);
    p.lse = const_cast<float *>(lse);
    p.d_o = d_o;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    return guarded([&] {
        if (tile_supported(*dims, dtype, true)) return launch_tile_backward(p, parts, (cudaStream_t)stream);
        return launch_simt_backward(p, dtype == SSD_BF16, (cudaStream_t)stream);
    });
}

ssd_status window_fill(const window_dims *dims, ssd_dtype dtype, const void *k, const void *v, const int32_t *valid_len,
                       void *k_cache, void *v_cache, int64_t slots, const int32_t *cache_index, void *stream) {
    record_error("");
    ssd_status st = validate(dims, dtype);
    if (st != SSD_OK) return st;
    const void *req[] = {k, v, k_cache, v_cache};
    static const char *const names[] = {"k", "v", "k_cache", "v_cache"};
    if ((st = check_pointers(req, names, 4)) != SSD_OK) return st;
    if ((st = check_ring(dims, slots, cache_index)) != SSD_OK) return st;
    RingParams p = ring_params(*dims, k, v, k_cache, v_cache, slots, cache_index);
    p.valid_len = valid_len;
    return guarded([&] { return launch_fill(p, dtype == SSD_BF16, (cudaStream_t)stream); });
}

ssd_status window_step(const window_dims *dims, ssd_dtype dtype, const void *q, const void *k, const void *v,
                       const int32_t *position, float scale, void *k_cache, void *v_cache, int64_t slots,
                       const int32_t *cache_index, void *o, void *stream) {
    record_error("");
    ssd_status st = validate(dims, dtype);
    if (st != SSD_OK) return st;
    if (dims->seqlen != 1) return fail(SSD_ERR_INVALID_ARG, "window_step takes one token: seqlen must be 1");
    const void *req[] = {q, k, v, k_cache, v_cache, o};
    static const char *const names[] = {"q", "k", "v", "k_cache", "v_cache", "o"};
    if ((st = check_pointers(req, names, 6)) != SSD_OK) return st;
    if ((st = check_scale(scale)) != SSD_OK) return st;
    if (!position) return fail(SSD_ERR_INVALID_ARG, "position is NULL");
    if ((st = check_ring(dims, slots, cache_index)) != SSD_OK) return st;
    RingParams p = ring_params(*dims, k, v, k_cache, v_cache, slots, cache_index);
    p.q = q;
    p.position = position;
    p.o = o;
    p.scale = scale;
    return guarded([&] { return launch_step(p, dtype == SSD_BF16, (cudaStream_t)stream); });
}

}  // extern "C"
