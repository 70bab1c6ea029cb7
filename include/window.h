/* window.h -- C ABI of attention with a sliding window and sinks, in the same
 * library (libssd.so, ssd.h): the sequence mixer that hybrid models put between
 * layers of the scan, with the same padded rows, grouped keys and, for decoding,
 * a state of fixed size per request: a ring of sinks + window entries.
 *
 * Per batch b and query head h, with key group g = h / (H/G) and V = valid_len[b]
 * (default L), token t < V sees token s where
 *     s <= t  and  (t - s < window  or  s < sinks),
 * itself always among them, and
 *     p[t,s]    = softmax over the s that t sees of scale q[b,t,h,:] . k[b,s,g,:]
 *     o[b,t,h]  = sum_s p[t,s] v[b,s,g,:]
 *     lse[b,h,t] = log sum_s exp(scale q . k)
 * window >= seqlen is plain causal attention.  scale is of either sign; it and the scores scale q . k are finite, times log2(e) too.
 * Tokens t >= V are absent:
 * nobody sees them, o, lse and every gradient there are 0, and their q, k, v, o, lse and do values are not
 * used (NaN and infinities there do no harm).  A NaN or an infinity in a present token's
 * k or v makes no promise for the tokens of its row up to 255 before it, which the tensor-core
 * kernels multiply by a stored zero of a probability, nor for those after it.
 *
 * Layouts (dense, row-major, contiguous, 16-byte aligned):
 *     q, o, do, dq           [batch, seqlen, nheads, headdim]     (T)
 *     k, v, dk, dv           [batch, seqlen, ngroups, headdim]    (T)
 *     lse                    [batch, nheads, seqlen]              (fp32)
 *     k_cache, v_cache       [slots, sinks + window, ngroups, headdim] (T)
 *     valid_len, position, cache_index  [batch]                   (int32)
 * T is fp32 for SSD_F32 and bf16 for SSD_BF16.
 *
 * Precision: scores, statistics and sums are fp32, outputs are rounded once.  The tensor-core kernels
 * (SSD_BF16, headdim a multiple of 8) round the probabilities, and in the backward the scores'
 * gradients, to bf16 where they enter a product; the backward's do . o takes o as stored.
 * WINDOW_FLAG_SIMT keeps fp32 operands throughout, at CUDA cores' speed, as SSD_F32 does.
 *
 * Memory, streams, errors: as in ssd.h.  The caller owns every buffer, work is enqueued on
 * `stream` without synchronising, argument errors return before any launch.  The same
 * inputs give the same bits, whatever the order in which blocks run.  valid_len entries outside
 * [0, seqlen] are clamped; ssd_workspace_status() on the call's workspace reports how many. */
#ifndef WINDOW_GB300_H
#define WINDOW_GB300_H

#include <stddef.h>
#include <stdint.h>

#include "ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WINDOW_FLAG_NONE 0u
#define WINDOW_FLAG_SIMT 1u /* SSD_BF16 only: the CUDA-core kernels instead of the tensor-core ones
                               (forward and backward; the step has one form per type) */

typedef struct {
    int64_t batch;    /* b >= 1 */
    int64_t seqlen;   /* L >= 1 */
    int64_t nheads;   /* H >= 1, query heads */
    int64_t headdim;  /* P, width of a head of q, k and v */
    int64_t ngroups;  /* G, divides H; k and v are shared by the H/G heads of a group */
    int64_t window;   /* W >= 1, a token itself among them */
    int64_t sinks;    /* first tokens that stay visible, >= 0 */
    uint32_t flags;   /* WINDOW_FLAG_* */
    uint32_t reserved; /* must be 0 */
} window_dims;

/* SSD_OK when (dims, dtype) can run, else SSD_ERR_INVALID_ARG / _UNSUPPORTED.  Limits: headdim <= 128
 * and a multiple of 4 (SSD_F32, or SSD_BF16 with WINDOW_FLAG_SIMT) or of 8 (SSD_BF16). */
ssd_status window_supported(const window_dims *dims, ssd_dtype dtype);

/* Bytes of workspace window_forward (backward = 0) or window_backward (backward = 1) needs; 0 when
 * the arguments are invalid. */
size_t window_workspace_bytes(const window_dims *dims, ssd_dtype dtype, int backward);

/* Forward: o and, where lse is not NULL, lse.  valid_len may be NULL (= seqlen). */
ssd_status window_forward(const window_dims *dims, ssd_dtype dtype, const void *q, const void *k, const void *v,
                          float scale, const int32_t *valid_len, void *o, float *lse, void *workspace,
                          size_t workspace_bytes, void *stream);

/* Gradients of <do, o> for the forward's o and lse (lse has no gradient of its own).
 * dk and dv are summed over the heads of a group.  do . o takes o as it is stored: in bf16 what
 * that misses (2^-8 of |do| |o| at most) is as large as the gradient of q or k where a token's
 * probabilities all but sit on one key and their gradient all but cancels. */
ssd_status window_backward(const window_dims *dims, ssd_dtype dtype, const void *q, const void *k, const void *v,
                           const void *o, const float *lse, const void *d_o, float scale, const int32_t *valid_len,
                           void *dq, void *dk, void *dv, void *workspace, size_t workspace_bytes, void *stream);

/* The ring.  Token t of a request lies in its slot at entry t where t < sinks, else at
 * sinks + (t - sinks) mod window, so that the entries written are those the next token sees
 * (its own place it takes from the one that leaves the window).
 *
 * window_fill writes the tokens of prompts [batch, seqlen] that tokens from V on see: the
 * first sinks and the last window of the V present ones.  Row i goes to slot cache_index[i]
 * (NULL: slot i); a slot outside [0, slots) marks a row that is not kept.  Other entries are
 * left as they are.  nheads only has to be a multiple of ngroups. */
ssd_status window_fill(const window_dims *dims, ssd_dtype dtype, const void *k, const void *v, const int32_t *valid_len,
                       void *k_cache, void *v_cache, int64_t slots, const int32_t *cache_index, void *stream);

/* One token of decoding for each of `batch` requests: token position[i] (the number of tokens before it) is
 * written to its entry of slot cache_index[i] (NULL: slot i, then slots >= batch) and attends over the
 * min(position + 1, sinks + window) entries written so far.
 *     q, o [batch, nheads, headdim]; k, v [batch, ngroups, headdim]      (T)
 * A request whose slot is outside [0, slots) or whose position is negative is absent (padding of a captured batch):
 * o = 0, nothing is written.  Two requests must not name one slot.  dims->seqlen must be 1. */
ssd_status window_step(const window_dims *dims, ssd_dtype dtype, const void *q, const void *k, const void *v,
                       const int32_t *position, float scale, void *k_cache, void *v_cache, int64_t slots,
                       const int32_t *cache_index, void *o, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* WINDOW_GB300_H */
