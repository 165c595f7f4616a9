/* qknorm.h -- C ABI of the per-head norms of queries and keys in libmlstm (sm_100a).
 *
 * What stands between a fused projection and a cell: every head's query and key vector
 * is normalized, weighted and rotated by its position, and laid out head by head, in
 * one pass.  For a vector x of D elements:
 *
 *   r = 1 / sqrt(mean(x^2) + eps)     (QKNORM_RMS)   or   1 / sqrt(sum(x^2) + eps)   (QKNORM_L2)
 *   z = r w * x                       (w [D] float32, or NULL for ones)
 *   y = z with its first RD elements rotated: the pair p < RD / 2, elements p and
 *       p + RD / 2 (or 2 p and 2 p + 1 with `interleaved`), turns by the angle
 *       position * inv_freq[p]:  (a, b) -> (a cos - b sin, a sin + b cos).
 *
 * The squares are summed in fp32, which holds those of elements between about 1e-19 and 1e19 / sqrt(D): what eps does
 * not carry has to lie there.  eps may be 0, but a vector of zeros then has no norm (its r is infinite).
 *
 * The angle is formed and reduced in fp64 (a position of 131072 times a frequency of one
 * has no fraction left in fp32); everything else is fp32, rounded once to `dt`.
 *
 * Inputs q [B][S][NHQ][D], k [B][S][NHK][D] with any strides (elements, per batch item,
 * token and head; the D elements of a head are contiguous; aligned to their size), so
 * that slices of a fused projection are read as they lie.  Outputs q_out [B][NHQ][S][D],
 * k_out [B][NHK][S][D], contiguous, the layout of mlstm.h and gdelta.h.  `dt` is the type
 * of all of them.  D a multiple of 8 in [8, 512]; RD even in [0, D] (0: no rotation).
 * positions: device int32 [B][S], or NULL for 0 .. S-1; inv_freq: device float32 [RD / 2].
 * NHQ or NHK may be 0 (that side's pointers are not looked at), at most 4096; B * S < 2^31.
 * Strides of inputs may be 0 or overlap; strides of outputs may not, and no output may
 * overlap an input.  Other conventions as in mlstm.h.
 */
#ifndef QKNORM_H
#define QKNORM_H

#include <stddef.h>

#include "mlstm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum qknorm_kind {
    QKNORM_RMS = 0,
    QKNORM_L2 = 1
} qknorm_kind;

/* Element strides of a [B][S][NH][D] tensor whose last axis is contiguous. */
typedef struct qknorm_strides {
    long long batch, token, head;
} qknorm_strides;

mlstm_status qknorm_fwd(const void *q, qknorm_strides q_strides, const void *k, qknorm_strides k_strides,
                        const float *q_weight, const float *k_weight, const float *inv_freq, const int *positions,
                        mlstm_dtype dt, int B, int S, int NHQ, int NHK, int D, int RD, qknorm_kind kind, float eps,
                        int interleaved, void *q_out, void *k_out, void *stream);

/*
 * Backward pass: from d_q_out [B][NHQ][S][D] and d_k_out [B][NHK][S][D] (contiguous) and
 * the forward's inputs, the gradients dq, dk (any strides, such as the slices of a fused
 * projection's gradient) and, where the pointers are non-NULL, dq_weight, dk_weight [D]
 * float32 (sums over all vectors in a fixed order: the same inputs give the same bits; a
 * NULL weight counts as ones).  positions and inv_freq get no gradient.
 * workspace: qknorm_bwd_workspace_size() bytes, 16-byte aligned; it may be NULL when both
 * weight gradients are.
 */
size_t qknorm_bwd_workspace_size(int B, int S, int NHQ, int NHK, int D);
mlstm_status qknorm_bwd(const void *d_q_out, const void *d_k_out, const void *q, qknorm_strides q_strides,
                        const void *k, qknorm_strides k_strides, const float *q_weight, const float *k_weight,
                        const float *inv_freq, const int *positions, mlstm_dtype dt, int B, int S, int NHQ, int NHK,
                        int D, int RD, qknorm_kind kind, float eps, int interleaved, void *dq,
                        qknorm_strides dq_strides, void *dk, qknorm_strides dk_strides, float *dq_weight,
                        float *dk_weight, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QKNORM_H */
