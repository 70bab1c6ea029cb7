/* norm.h -- C ABI of the block's entry norm, in the same library (libssd.so):
 * the residual addition and root-mean-square norm in one pass, its output in
 * the stream's type or in 8 bits with scales, and the backward.
 *
 * Per row of D columns:
 *     stream = x + residual            (rounded to T; x itself without a residual)
 *     y      = stream * rstd * weight, rstd = 1 / sqrt(mean(stream^2) + eps)
 * The norm reads the stream as it is stored, so the backward, which reads the
 * stored stream, is the derivative of what the forward computed.  Sums are
 * fp32; T is fp32 (SSD_F32) or bf16 (SSD_BF16); weight is fp32 [D].
 * Rows are dense and contiguous, pointers 16-byte aligned.  Conventions as in
 * ssd.h: caller-owned memory, work enqueued on `stream_` without synchronising,
 * argument errors before any launch, ssd_last_error(). */
#ifndef NORM_GB300_H
#define NORM_GB300_H

#include <stddef.h>
#include <stdint.h>

#include "ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* x, y [rows, D] (T); residual [rows, D] (T) or NULL; stream_out [rows, D] (T),
 * may be NULL without a residual, and may alias x or residual (not y). */
ssd_status norm_add_rms(ssd_dtype dtype, const void *x, const void *residual, const float *weight, float eps,
                        void *y, void *stream_out, int64_t rows, int64_t D, void *stream_);

/* The same with y in e4m3 (one byte each) and fp32 scales [rows, D / group]
 * (group 0: one scale a row): scale = max |y| / 448 over the group, y8 the
 * e4m3 value nearest to y / scale (448 at most, where a scale below fp32's
 * normal numbers was rounded down); a group whose scale is 0 has zeros.
 * group is 0, 32, 64 or 128 and divides D. */
ssd_status norm_add_rms_fp8(ssd_dtype dtype, const void *x, const void *residual, const float *weight, float eps,
                            void *y8, float *scales, void *stream_out, int64_t rows, int64_t D, int64_t group,
                            void *stream_);

/* Backward for dy [rows, D] (T) at the stored stream h, and optionally the
 * gradient d_stream that reaches the stream from behind (may be NULL):
 *     dx = d_stream + rstd (dy w - h rstd^2 mean(dy w h)),  dweight = sum_rows dy h rstd
 * dx is the gradient of both x and residual.  dweight [D] fp32, summed in a
 * fixed order; it may be NULL (not computed). */
size_t norm_backward_workspace_bytes(int64_t rows, int64_t D);
ssd_status norm_add_rms_backward(ssd_dtype dtype, const void *dy, const void *h, const float *weight, float eps,
                                 const void *d_stream, void *dx, float *dweight, int64_t rows, int64_t D,
                                 void *workspace, size_t workspace_bytes, void *stream_);

#ifdef __cplusplus
}
#endif

#endif /* NORM_GB300_H */
