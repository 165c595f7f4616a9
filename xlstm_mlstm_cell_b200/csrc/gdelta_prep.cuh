// gdelta_prep.cuh -- device pieces that the gated delta rule's kernels share: a chunk's cumulative
// gates and the inverse of its unit lower triangular system.
#pragma once

#include "common.cuh"
#include "gdelta_internal.h"

namespace mlstm {
namespace gdelta {

// Tokens of batch item b that are part of its sequence.
MLSTM_DEVINL int live_tokens(const int *lengths, int b, int S)
{
    return lengths ? min(max(lengths[b], 0), S) : S;
}

// a_i - a_j of two cumulative gates held as value and residue: the residues keep the difference
// of neighbouring tokens exact to fp32 after the cumulative sum has grown.
MLSTM_DEVINL float gate_diff(float2 x, float2 y) { return (x.x - y.x) + (x.y - y.y); }

// A log gate below -128 is exp(g) = 0 in fp32; clamping it there keeps a full reset (-inf) out of the
// differences (-inf) - (-inf).  NaN stays NaN.
MLSTM_DEVINL float clamp_gate(float g) { return g < -128.f ? -128.f : g; }

// One warp: the cumulative log gates of a chunk's 64 tokens (`len` of them live, the others 0), summed
// in fp64, times `unit`, and kept as value and residue: tokens 2 lane (a0) and 2 lane + 1 (a1).
MLSTM_DEVINL void chunk_gates(const float *g, int len, int lane, double unit, float2 &a0, float2 &a1)
{
    const double x0 = 2 * lane < len ? (double)clamp_gate(g[2 * lane]) : 0.0;
    const double x1 = 2 * lane + 1 < len ? (double)clamp_gate(g[2 * lane + 1]) : 0.0;
    double sum = x0 + x1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    const double c0 = (sum - x1) * unit, c1 = sum * unit;
    a0.x = (float)c0;
    a0.y = (float)(c0 - (double)a0.x);
    a1.x = (float)c1;
    a1.y = (float)(c1 - (double)a1.x);
}
MLSTM_DEVINL void chunk_gates(const float *g, int len, int lane, float2 *a)
{
    chunk_gates(g, len, lane, 1.0, a[2 * lane], a[2 * lane + 1]);
}
// The same in units of log 2, for exp2f.
MLSTM_DEVINL void chunk_gates_log2(const float *g, int len, int lane, float2 &a0, float2 &a1)
{
    chunk_gates(g, len, lane, 1.4426950408889634074, a0, a1);
}

constexpr int LDT = 68;   // row stride of the 64 x 64 matrices in shared memory (16-byte rows, no bank repeats)

// In place, by `nthr` threads (a multiple of 64, at least 64) of one group that `sync` joins: the unit
// lower triangular matrix I + M, M strictly lower in m [64][LDT], becomes its inverse (the upper part
// and the diagonal of m are written too).  Blocks of 16 are inverted by forward substitution, one
// thread per column; then [A 0; C D]^-1 = [A^-1 0; -D^-1 C A^-1 D^-1] joins them to 32 and to 64.
// Forward substitution keeps the inverse accurate where a power series in M would not (a key that
// repeats makes M's powers large while the inverse stays small).  tmp: 32 * 33 floats.
template <typename Sync>
MLSTM_DEVINL void invert64(float *m, float *tmp, int tid, int nthr, Sync sync)
{
    if (tid < 64) {   // thread (block b, column j) solves (I + M_b) x = e_j
        const int b = tid >> 4, j = tid & 15;
        float *mb = m + (b * 16) * LDT + b * 16;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == j ? 1.f : 0.f;
#pragma unroll
            for (int l = 0; l < i; ++l) s = fmaf(-mb[i * LDT + l], x[l], s);
            x[i] = s;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) mb[i * LDT + j] = x[i];
    }
    for (int i = tid; i < 64 * 64; i += nthr) {   // the upper blocks
        const int r = i >> 6, c = i & 63;
        if ((c >> 4) > (r >> 4)) m[r * LDT + c] = 0.f;
    }
    sync();
    // two joins of 16 -> 32: tmp_p = C A^-1, then C = -D^-1 tmp_p
    for (int i = tid; i < 512; i += nthr) {
        const int p = i >> 8, r = (i >> 4) & 15, c = i & 15;
        const float *C = m + (32 * p + 16) * LDT + 32 * p, *A = m + (32 * p) * LDT + 32 * p;
        float s = 0.f;
#pragma unroll
        for (int l = 0; l < 16; ++l) s = fmaf(C[r * LDT + l], A[l * LDT + c], s);
        tmp[p * 272 + r * 17 + c] = s;
    }
    sync();
    for (int i = tid; i < 512; i += nthr) {
        const int p = i >> 8, r = (i >> 4) & 15, c = i & 15;
        const float *D = m + (32 * p + 16) * LDT + 32 * p + 16;
        float s = 0.f;
#pragma unroll
        for (int l = 0; l < 16; ++l) s = fmaf(-D[r * LDT + l], tmp[p * 272 + l * 17 + c], s);
        m[(32 * p + 16 + r) * LDT + 32 * p + c] = s;
    }
    sync();
    for (int i = tid; i < 1024; i += nthr) {
        const int r = i >> 5, c = i & 31;
        const float *C = m + 32 * LDT, *A = m;
        float s = 0.f;
#pragma unroll 8
        for (int l = 0; l < 32; ++l) s = fmaf(C[r * LDT + l], A[l * LDT + c], s);
        tmp[r * 33 + c] = s;
    }
    sync();
    for (int i = tid; i < 1024; i += nthr) {
        const int r = i >> 5, c = i & 31;
        const float *D = m + 32 * LDT + 32;
        float s = 0.f;
#pragma unroll 8
        for (int l = 0; l < 32; ++l) s = fmaf(-D[r * LDT + l], tmp[l * 33 + c], s);
        m[(32 + r) * LDT + c] = s;
    }
    sync();
}

}  // namespace gdelta
}  // namespace mlstm
