/* delta.h -- C ABI of the gated delta rule, in the same library as the
 * selective scan (libssd.so, ssd.h): a linear recurrence whose write corrects
 * what the state already holds for a key.
 *
 * Per batch b and head h, with key group g = h / (H/G) and a_t = exp(g[b,h,t]):
 *
 *     S_{-1} = init[b,h];   S_t = a_t S_{t-1}
 *                + beta[b,h,t] (v[b,t,h,:] - a_t S_{t-1} k[b,t,g,:]) (outer) k[b,t,g,:]
 *     o[b,t,h,p] = scale sum_r S_t[p,r] q[b,t,g,r]
 *     final_state[b,h] = S_{V-1}
 *
 * where V = valid_len[b] (default L).  Tokens t >= V are absent: no state
 * update, o = 0, and every per-token gradient there is 0; their q, k, v, g,
 * beta and do values are not used (NaN and infinities there do no harm).
 * A NaN or an infinity in a present token's q, k, v, g, beta or do makes no promise for its
 * sequence and key group: the chunked kernels multiply it by stored zeros, so that tokens before it
 * in its chunk (64 tokens) may become NaN too, where the token-by-token kernels leave them alone.
 * Keys are used as given: a layer normalises q and k to unit length before
 * the call, with beta in [0, 1] the recurrence then contracts.
 *
 * Layouts (dense, row-major, contiguous, 16-byte aligned):
 *     q, k, dq, dk           [batch, seqlen, ngroups, dstate]     (T)
 *     v, o, do, dv           [batch, seqlen, nheads, headdim]     (T)
 *     g, beta, dg, dbeta     [batch, nheads, seqlen]              (fp32)
 *     init_state, final_state, d_final_state, d_init_state
 *                            [batch, nheads, headdim, dstate]     (fp32)
 *     valid_len              [batch]                              (int32)
 * T is fp32 for SSD_F32 and bf16 for SSD_BF16.  g is the log of the decay,
 * g <= 0 (values below -1000 act as -1000: a decay of exactly 0); beta is
 * used as given and may be 0.
 *
 * Precision of SSD_BF16: outputs in bf16 are rounded once (1.7e-3 of an output's norm).  The
 * chunked kernels feed fp32 values to the tensor cores as two bf16 parts (2^-17 of a value at most) and what a
 * state takes up as three; of an fp32 output's norm final_state and d_init are below 1e-6 off, dg and dbeta
 * 2e-6 to 5e-6.  DELTA_FLAG_SIMT keeps every operand in fp32: 1e-7 to 3e-7, at the token-by-token
 * kernels' speed.  So does SSD_F32.
 *
 * Memory, streams, errors: as in ssd.h.  The caller owns every buffer, the
 * workspace is sized by delta_workspace_bytes, work is enqueued on `stream`
 * without synchronising, argument errors return before any launch, and
 * ssd_last_error() describes the last failure.  valid_len entries outside
 * [0, seqlen] are clamped; ssd_workspace_status() on the call's workspace
 * reports how many (SSD_ERR_INVALID_ARG).  Results do not depend on the order
 * in which blocks run: the same inputs give the same bits.  A chunked backward
 * of several rows whose chains outnumber the SMs runs half of the batch on a
 * second stream that the library keeps per (device, caller stream) pair,
 * forked from `stream` and joined back into it before the call returns, as the
 * scan's backward does (ssd.h); make a first such call before any capture. */
#ifndef DELTA_GB300_H
#define DELTA_GB300_H

#include <stddef.h>
#include <stdint.h>

#include "ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DELTA_FLAG_NONE 0u
#define DELTA_FLAG_SIMT 1u /* SSD_BF16 only: the token-by-token CUDA-core kernels instead of
                              the chunked tensor-core kernels */

typedef struct {
    int64_t batch;    /* b >= 1 */
    int64_t seqlen;   /* L >= 1 */
    int64_t nheads;   /* H >= 1, value heads */
    int64_t headdim;  /* P, value width of a head */
    int64_t dstate;   /* N, key width */
    int64_t ngroups;  /* G, divides H; q and k are shared by the H/G heads of a group */
    uint32_t flags;   /* DELTA_FLAG_* */
    uint32_t reserved; /* must be 0 */
} delta_dims;

/* SSD_OK when (dims, dtype) can run, else SSD_ERR_INVALID_ARG / _UNSUPPORTED.
 * Limits: headdim <= 128 and a multiple of 4; dstate <= 256 and a multiple of
 * 4.  The chunked tensor-core kernels take SSD_BF16 with headdim and dstate
 * multiples of 8 and at most 128; everything else runs token by token on
 * CUDA cores. */
ssd_status delta_supported(const delta_dims *dims, ssd_dtype dtype);

/* Bytes of workspace delta_forward (backward = 0) or delta_backward
 * (backward = 1) needs; 0 when the arguments are invalid.  The backward keeps a state
 * every 64 tokens (chunked), or every 16, 8 or 4 (token by token, dstate up to 64, 128 or 256), and token by token
 * its key gradients' sums per 32 rows of a head, 8 where heads are few: 0.26 MB a token at 4 heads of 128 x 256. */
size_t delta_workspace_bytes(const delta_dims *dims, ssd_dtype dtype, int backward);

/* Forward: o (and optionally final_state).  init_state may be NULL (zeros),
 * valid_len may be NULL (= seqlen), final_state may be NULL (not written). */
ssd_status delta_forward(const delta_dims *dims, ssd_dtype dtype, const void *q, const void *k, const void *v,
                         const float *g, const float *beta, float scale, const float *init_state,
                         const int32_t *valid_len, void *o, float *final_state, void *workspace,
                         size_t workspace_bytes, void *stream);

/* Backward with recompute: gradients of <do, o> + <d_final_state, final_state>.
 * d_final_state may be NULL (zeros); d_init_state may be NULL (not written).
 * dq and dk are summed over the heads of a group. */
ssd_status delta_backward(const delta_dims *dims, ssd_dtype dtype, const void *q, const void *k, const void *v,
                          const float *g, const float *beta, float scale, const float *init_state,
                          const int32_t *valid_len, const void *d_o, const float *d_final_state, void *dq, void *dk,
                          void *dv, float *dg, float *dbeta, float *d_init_state, void *workspace,
                          size_t workspace_bytes, void *stream);

/* One token of decoding for each of `batch` requests, states updated in place:
 *     q, k [batch, ngroups, dstate]; v, o [batch, nheads, headdim]      (T)
 *     g, beta [batch, nheads] (fp32)
 *     state [slots, nheads, headdim, dstate] (fp32)
 *     state_index [batch] (int32) or NULL: the slot of each request (NULL: slot i,
 *         then slots >= batch)
 * A request whose slot is outside [0, slots) is absent (padding of a captured
 * batch): o = 0, no state is touched.  Two requests must not name one slot.
 * dims->seqlen must be 1. */
ssd_status delta_step(const delta_dims *dims, ssd_dtype dtype, const void *q, const void *k, const void *v,
                      const float *g, const float *beta, float scale, float *state, int64_t slots,
                      const int32_t *state_index, void *o, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DELTA_GB300_H */
