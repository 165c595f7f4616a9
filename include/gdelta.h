/* gdelta.h -- C ABI of the gated delta rule in libmlstm (sm_100a).
 *
 * The gated delta rule keeps, like the mLSTM cell, a matrix memory S [DK][DV] per
 * value head, but writes the error of the memory's own prediction instead of the
 * value.  Per batch item b, value head h and token t:
 *
 *   S~  = exp(g_t) S_{t-1}                          g_t <= 0: log forget gate
 *   e_t = v_t - S~^T k_t                            what the memory does not predict
 *   S_t = S~ + beta_t k_t e_t^T                     beta_t: write strength
 *   o_t = scale S_t^T q_t
 *
 * Over whole sequences the recurrence runs chunkwise (64 tokens): with a the
 * cumulative sum of g inside the chunk, D_ij = exp(a_i - a_j) and S the state at the
 * chunk's start,
 *   Y = V - e^a K S,   E = T Y,   T = (I + strict_lower(D * K K^T) diag(beta))^-1,
 *   O = scale (e^a Q S + lower(D * Q K^T) beta E),
 *   S' = e^{a_64} S + K^T (e^{a_64 - a} beta E),
 * which equals the recurrence token by token.
 *
 * Conventions are those of mlstm.h: device pointers owned by the caller, contiguous,
 * row-major, 16-byte aligned; work is enqueued on `stream` and nothing synchronizes;
 * bad arguments return an error status before anything is enqueued; the library
 * allocates nothing.  No output may overlap an input or another output, but for the
 * states that a function's comment names.  Layouts:
 *   q, k [B][NH][S][DK]; v, o [B][NHV][S][DV]  in the element type `dt`;
 *   g, beta [B][NHV][S] float32; states [B][NHV][DK][DV] float32.
 * NHV is a multiple of NH: value head h reads query and key head h / (NHV / NH).
 * Supported: DK a multiple of 8 in [8, 128], DV a multiple of 8 in [8, 512]; over
 * sequences B * NHV <= 65535, S <= 2^30 and B * NHV * (S / 64 + 1) < 2^31, for
 * gdelta_step B * NHV * DV / 8 < 2^31.
 * The recurrence is stable for keys of norm at most about one with beta in [0, 2];
 * nothing here normalizes them (qknorm.h does).
 *
 * Real tokens have to be finite (g may be -inf: a full reset).  Over sequences the zeros of a chunk's
 * triangular matrices meet every token of the chunk, so an infinity or NaN in one makes NaN of the
 * outputs of all tokens of its chunk of 64, the earlier ones among them, and of everything behind it; with
 * gradients, of everything.  Other items, and heads that read neither its keys nor its values, are not touched.
 *
 * `lengths` (device int32 [B], or NULL for S everywhere): of item b only the first
 * lengths[b] tokens (clamped to [0, S]) are part of the sequence.  The rows behind
 * are not used, whatever they hold, and the state is the one after the last real
 * token; o and the gradients are 0 there.  lengths[b] == 0 leaves the item's state as
 * it was.
 */
#ifndef GDELTA_H
#define GDELTA_H

#include <stddef.h>

#include "mlstm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Bytes of device workspace gdelta_fwd needs (0 when the arguments are unsupported):
 * a status word, 8 bytes of gates per token of a whole chunk and value head, and per
 * chunk and value head the two 64 x 64 matrices T and the scores in fp32 (32 KB), or
 * on the tensor-core path T and the scores' product with it as bf16 parts (40 KB).
 */
size_t gdelta_fwd_workspace_size(int B, int NH, int NHV, int S, int DK, int DV, mlstm_dtype dt);

/*
 * Forward pass over S tokens from the state S0 (NULL: the zero state).  Writes o and,
 * where it is non-NULL, S_final, which may be S0 itself.  Any S >= 0 (S == 0 copies
 * the state).  workspace: gdelta_fwd_workspace_size() bytes, 256-byte aligned, not
 * shared by two calls in flight.
 *
 * Accuracy: sums and the state are fp32.  On the tensor-core path (bf16 inputs, gdelta_fwd_tensor_path) every
 * fp32 operand that the state comes of enters its products as three bf16 parts, which hold its 24 bits, so that a
 * state from bf16 inputs is as close to an fp64 evaluation as fp32 arithmetic brings it (within 5e-7 where nothing
 * cancels); the scores' product, which only the bf16 o sees, as two.  mlstm_fwd_status on the
 * workspace tells whether every bounded wait of its kernels completed.
 */
mlstm_status gdelta_fwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                        const int *lengths, mlstm_dtype dt, int B, int NH, int NHV, int S, int DK, int DV,
                        float scale, const float *S0, void *o, float *S_final, void *workspace,
                        size_t workspace_bytes, void *stream);

/*
 * 1 when gdelta_fwd runs its products on the tensor cores for this element type and
 * these head sizes, 0 when it runs them in fp32 on the CUDA cores, -1 when the
 * combination is not supported.  No GPU work; a host-side query.
 */
int gdelta_fwd_tensor_path(int DK, int DV, mlstm_dtype dt);

/*
 * One token for every (b, h): updates the state IN PLACE and writes o [B][NHV][DV].
 * q, k [B][NH][DK], v [B][NHV][DV] in `dt`; g, beta [B][NHV] float32 (4-byte aligned
 * is enough for these two).
 */
mlstm_status gdelta_step(float *state, const void *q, const void *k, const void *v, const float *g,
                         const float *beta, mlstm_dtype dt, int B, int NH, int NHV, int DK, int DV, float scale,
                         void *o, void *stream);

/*
 * Backward pass of gdelta_fwd: the gradients of
 *   L = sum of d_o * o over all tokens  +  sum of dS_final * S_final
 * with respect to every input.  d_o [B][NHV][S][DV] in `dt`; dS_final (float32, or
 * NULL for zero); S0 as for gdelta_fwd.  Writes dq, dk [B][NH][S][DK], dv
 * [B][NHV][S][DV] in `dt`, dg, dbeta [B][NHV][S] float32 and, where it is non-NULL,
 * dS0 [B][NHV][DK][DV] float32 (which may be dS_final itself).  dq and dk are the sums
 * over the value heads that share them.  The forward pass is recomputed inside; no
 * atomics: the same inputs give the same bits.
 *
 * dg_t sums the terms that carry exp(g_t) themselves (the state carried across t and
 * the token pairs j < t <= i), not a difference of cumulative sums: strongly
 * forgetting gates keep its accuracy.
 *
 * workspace: gdelta_bwd_workspace_size() bytes, 256-byte aligned, not shared by two
 * calls in flight (the states at the chunks' starts and their gradients, 8 DK DV bytes
 * per chunk and value head, and 8 DV bytes per token and value head make up most of
 * it).  Accuracy on the tensor-core path: dS0 within 6e-7, dg and dbeta within 1.25e-6 of
 * an fp64 evaluation of the same inputs, where they are not what is left of sums that nearly
 * cancel (one key, repeated: as far as inputs moved by a step of fp32 would put fp64 itself).
 */
size_t gdelta_bwd_workspace_size(int B, int NH, int NHV, int S, int DK, int DV, mlstm_dtype dt);
mlstm_status gdelta_bwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                        const int *lengths, const float *S0, const void *d_o, const float *dS_final,
                        mlstm_dtype dt, int B, int NH, int NHV, int S, int DK, int DV, float scale, void *dq,
                        void *dk, void *dv, float *dg, float *dbeta, float *dS0, void *workspace,
                        size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDELTA_H */
