// gdelta_simt.cu -- the gated delta rule chunk by chunk on the CUDA cores in fp32: the path of fp32
// inputs and of every shape the tensor-core kernels do not take.
//
// With a the cumulative log gates of a chunk, D_ij = exp(a_i - a_j), S the state at its start:
//   prep     KK = strict_lower(D * K K^T), P = lower(D * Q K^T), T = (I + KK diag(beta))^-1
//   walk     Y = V - e^a K S,  E = T Y,  U = beta E,  O = scale (e^a Q S + P U),
//            S' = e^{a_64} S + K^T (e^{a_64 - a} U)
//   reverse  dU = scale P^T dO + e^{a_64 - a} K dS',  dV = T^T (beta dU),
//            dS = e^{a_64} dS' + scale Q^T (e^a dO) - K^T (e^a dV)
//   grad     H = dV E^T,  dP = scale (dO E^T) diag(beta),  dA = -H diag(beta),
//            Zq = scale e^a dO S^T,  Zk = -e^a dV S^T,  W = e^{a_64 - a} U dS'^T,
//            dQ = Zq + (dP * D) K,  dK = Zk + W + (dP * D)^T Q + (dA * D + (dA * D)^T) K,
//            dbeta_j = (e^{a_64 - a} W0 . K)_j + sum_i (scale P dO E^T - KK H)_ij,  W0 = E dS'^T,
//            dg_t = sum_{i >= t} (Zq . Q + Zk . K)_i + sum_{j < t} (W . K)_j
//                   + sum_{j < t <= i} (dP * P + dA * KK)_ij + e^{a_64} <S, dS'>
// (dP * D masked to j <= i, dA * D to j < i.)  Only the walks are sequential over the chunks; their
// work splits over value columns, 32 to a CTA.  Products are register tiles of 2 x 4, 4 x 4 or 8 x 8 fed by
// 16-byte shared-memory loads, 512 bytes a warp whether lanes read the same or not; at 128 bytes a cycle and SM these
// bound the walks (8 us a chunk at DK 96, two thirds of it the two products with the state), and the gradients'
// tiles of 8 x 8 sit where loads and fp32 arithmetic take as long.  For few heads the walks leave SMs idle: their
// chain of three products per chunk is what a call then waits for.
#include "gdelta_prep.cuh"
#include "tc_common.cuh"

#include <algorithm>

namespace mlstm {
namespace gdelta {
namespace {

using tc::f2_fma;
using tc::f2_mul;
using tc::f2_pack;
using tc::f2_unpack;
using tc::smem_u32;

constexpr int LDR = 132;   // row stride of [.][128] tiles
constexpr int VT = 32;     // value columns of a walk CTA

MLSTM_DEVINL float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
MLSTM_DEVINL void st4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }

// Rows r < 64 of src (row stride DK, `len` of them live) into columns c0 + r of dst [DK][LDR].
template <typename T>
MLSTM_DEVINL void stage_transposed(const T *src, int len, int DK, float *dst, int c0, int tid, int nthr)
{
    for (int i = tid; i < 64 * (DK / 4); i += nthr) {
        const int r = i & 63, d = (i >> 6) * 4;
        const float4 x = r < len ? load4(src + (size_t)r * DK + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        dst[(d + 0) * LDR + c0 + r] = x.x;
        dst[(d + 1) * LDR + c0 + r] = x.y;
        dst[(d + 2) * LDR + c0 + r] = x.z;
        dst[(d + 3) * LDR + c0 + r] = x.w;
    }
}

MLSTM_DEVINL void fma4x4(float (&acc)[4][4], float4 a, float4 b)
{
    const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
}

// ---------------------------------------------------------------- prep

constexpr size_t PREP_SMEM = sizeof(float) * (128 * LDR + 64 * LDT + 32 * 33 + 64) + sizeof(float2) * 64;

// One CTA per chunk and key head: K K^T and Q K^T once, then the matrices of every value head on it.  Where all of
// them find room at once, one per value head instead (gridDim.z of them): 24 CTAs of three heads took
// 25 us, 72 of one 14.
template <typename T>
__global__ void __launch_bounds__(256, 2)
prep_kernel(const T *__restrict__ q, const T *__restrict__ k, const float *__restrict__ g,
            const float *__restrict__ beta, const int *__restrict__ lengths, int NH, int NHV, int S, int DK,
            Workspace w, bool want_kk)
{
    extern __shared__ __align__(16) float sm[];
    float *kq = sm;                       // [DK][LDR]: K in columns 0..63, Q in 64..127
    float *m = kq + 128 * LDR;            // [64][LDT]
    float *tmp = m + 64 * LDT;
    float *bt = tmp + 32 * 33;            // [64]
    float2 *a = reinterpret_cast<float2 *>(bt + 64);
    const int tid = threadIdx.x, c = blockIdx.x, bh = blockIdx.y, b = bh / NH, group = NHV / NH;
    griddep_wait();
    griddep_launch_dependents();
    if (c == 0 && bh == 0 && blockIdx.z == 0 && tid == 0) *w.status = 0u;
    const int len = min(CH, live_tokens(lengths, b, S) - c * CH);
    if (len <= 0) return;
    const size_t row0 = (size_t)bh * S + c * CH;
    stage_transposed(k + row0 * DK, len, DK, kq, 0, tid, 256);
    stage_transposed(q + row0 * DK, len, DK, kq, 64, tid, 256);
    __syncthreads();
    const int i0 = (tid >> 4) * 4, j0 = (tid & 15) * 4;
    float kk[4][4] = {}, qk[4][4] = {};
    for (int d = 0; d < DK; ++d) {
        const float4 y = ld4(kq + d * LDR + j0);
        fma4x4(kk, ld4(kq + d * LDR + i0), y);
        fma4x4(qk, ld4(kq + d * LDR + 64 + i0), y);
    }
    const int h0 = gridDim.z > 1 ? blockIdx.z : 0, h1 = gridDim.z > 1 ? h0 + 1 : group;
    for (int h = h0; h < h1; ++h) {
        const int bhv = b * NHV + (bh % NH) * group + h;
        const size_t ch = (size_t)bhv * w.NC + c, gt = (size_t)bhv * S + c * CH;
        __syncthreads();
        if (tid < 32) chunk_gates(g + gt, len, tid, a);
        else if (tid < 96) bt[tid - 32] = tid - 32 < len ? beta[gt + tid - 32] : 0.f;
        __syncthreads();
        if (tid < 64) w.A[ch * 64 + tid] = a[tid];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = i0 + r;
            float p[4], x[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int j = j0 + s;
                const float dec = j <= i ? expf(gate_diff(a[i], a[j])) : 0.f;
                p[s] = j <= i ? dec * qk[r][s] : 0.f;
                x[s] = j < i ? dec * kk[r][s] : 0.f;
                m[i * LDT + j] = x[s] * bt[j];
            }
            st4(w.P + ch * 4096 + i * 64 + j0, make_float4(p[0], p[1], p[2], p[3]));
            if (want_kk) st4(w.KK + ch * 4096 + i * 64 + j0, make_float4(x[0], x[1], x[2], x[3]));
        }
        __syncthreads();
        invert64(m, tmp, tid, 256, [] { __syncthreads(); });
        for (int i = tid; i < 64 * 16; i += 256)
            st4(w.T + ch * 4096 + (i >> 4) * 64 + (i & 15) * 4, ld4(m + (i >> 4) * LDT + (i & 15) * 4));
    }
}

// ---------------------------------------------------------------- walks
//
// A CTA of 256 threads runs one value head's chunks over 32 value columns; thread (u = tid / 8, tid % 8) owns the
// tokens 2 u and 2 u + 1 and the state's rows 4 u .. 4 u + 3, four columns each.  The state stays in registers, with
// a copy in shared memory for the products that read all of it.  Everything is row-major as it lies in memory, so
// that the copies are plain and asynchronous: the next chunk's K and Q arrive during the whole of this one, T and P,
// which have no second buffer, during the state's update.  2 x 6 heads of 777 tokens, 96 x 200, take 106 us; with the
// tiles transposed on their way in by the threads, and half the warps at E, the other half at O, they took 211.

constexpr int LDX = 132;   // row stride of K and Q: rows 2 u .. of a warp's four u start 8 banks apart
constexpr int LDW = 68;    // of T and P, likewise

struct Gates { float ea[64], eo[64], bt[64]; };

struct WalkSmem {
    float kq[2][128 * LDX];            // K over Q
    float t[64 * LDW], p[64 * LDW];
    float st[128 * VT];                // the state, or its gradient
    float y[64 * VT], z[64 * VT];      // forward: Y, then U; e^{a_64 - a} U.  Reverse: beta dU; -e^a dV
    float x[64 * VT];                  // reverse: dO, then scale e^a dO
    Gates g[2];
};
static_assert(sizeof(WalkSmem) <= 232448, "one CTA's shared memory");

MLSTM_DEVINL void copy16(float *dst, const float *src, bool on)   // off: zeros
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
MLSTM_DEVINL void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Rows of src (row stride DK, `len` of them live, zeros behind) to dst [64][LDX].
MLSTM_DEVINL void stage_rows(const float *src, int len, int DK, float *dst, int tid)
{
    const int d = (tid & 31) * 4;
    if (d < DK)
        for (int r = tid >> 5; r < 64; r += 8) copy16(dst + r * LDX + d, src + (r < len ? (size_t)r * DK + d : 0), r < len);
}
MLSTM_DEVINL void stage_rows(const __nv_bfloat16 *src, int len, int DK, float *dst, int tid)
{
    const int d = (tid & 31) * 4;
    if (d < DK)
        for (int r = tid >> 5; r < 64; r += 8)
            st4(dst + r * LDX + d, r < len ? load4(src + (size_t)r * DK + d) : make_float4(0.f, 0.f, 0.f, 0.f));
}
MLSTM_DEVINL void stage64(const float *src, float *dst, int tid)
{
    for (int i = tid; i < 64 * 16; i += 256) copy16(dst + (i >> 4) * LDW + (i & 15) * 4, src + i * 4, true);
}

// A chunk's gates, read by thread t < 64 one chunk ahead.
struct GateReg {
    float2 a, last;
    float b;
    MLSTM_DEVINL void read(const Workspace &w, const float *beta, size_t ch, size_t vrow, int len, int t)
    {
        a = w.A[ch * 64 + t];
        last = w.A[ch * 64 + 63];
        b = t < len ? beta[vrow + t] : 0.f;
    }
    MLSTM_DEVINL void put(Gates &g, int t) const
    {
        g.ea[t] = expf(a.x + a.y);
        g.eo[t] = expf(gate_diff(last, a));
        g.bt[t] = b;
    }
};

// Four columns as two packed pairs.
struct Row4 { uint64_t a, b; };
MLSTM_DEVINL Row4 ldr(const float *p)
{
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
    return Row4{v.x, v.y};
}
MLSTM_DEVINL void str(float *p, Row4 v) { *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(v.a, v.b); }
MLSTM_DEVINL Row4 row4(float4 v) { return Row4{f2_pack(v.x, v.y), f2_pack(v.z, v.w)}; }
MLSTM_DEVINL float4 flat(Row4 v)
{
    const float2 a = f2_unpack(v.a), b = f2_unpack(v.b);
    return make_float4(a.x, a.y, b.x, b.y);
}
MLSTM_DEVINL Row4 fma_row(float f, Row4 x, Row4 c)
{
    const uint64_t ff = f2_pack(f, f);
    return Row4{f2_fma(ff, x.a, c.a), f2_fma(ff, x.b, c.b)};
}
MLSTM_DEVINL Row4 mul_row(float f, Row4 x)
{
    const uint64_t ff = f2_pack(f, f);
    return Row4{f2_mul(ff, x.a), f2_mul(ff, x.b)};
}

// acc[r] += sum_{l in [l0, l1)} A[r][l] B[l], rows A of stride lda, B [.][VT] at the thread's columns; l0, l1
// multiples of 4.
template <int R>
MLSTM_DEVINL void rows_times(const float *A, int lda, const float *B, int l0, int l1, Row4 (&acc)[R])
{
#pragma unroll 2
    for (int l = l0; l < l1; l += 4) {
        float4 a[R];
#pragma unroll
        for (int r = 0; r < R; ++r) a[r] = ld4(A + r * lda + l);
        const Row4 b0 = ldr(B + l * VT), b1 = ldr(B + (l + 1) * VT), b2 = ldr(B + (l + 2) * VT), b3 = ldr(B + (l + 3) * VT);
#pragma unroll
        for (int r = 0; r < R; ++r)
            acc[r] = fma_row(a[r].w, b3, fma_row(a[r].z, b2, fma_row(a[r].y, b1, fma_row(a[r].x, b0, acc[r]))));
    }
}
// acc[r] += sum_{l in [l0, l1)} A[l][r] B[l]: rows of A at the first of two neighbouring columns.
MLSTM_DEVINL void cols2_times(const float *A, int lda, const float *B, int l0, int l1, Row4 (&acc)[2])
{
#pragma unroll 4
    for (int l = l0; l < l1; ++l) {
        const float2 a = *reinterpret_cast<const float2 *>(A + l * lda);
        const Row4 b = ldr(B + l * VT);
        acc[0] = fma_row(a.x, b, acc[0]);
        acc[1] = fma_row(a.y, b, acc[1]);
    }
}
// The state's update: four neighbouring columns of A.
MLSTM_DEVINL void cols4_times(const float *A, int lda, const float *B, Row4 (&acc)[4])
{
#pragma unroll 4
    for (int l = 0; l < 64; ++l) {
        const float4 a = ld4(A + l * lda);
        const Row4 b = ldr(B + l * VT);
        acc[0] = fma_row(a.x, b, acc[0]);
        acc[1] = fma_row(a.y, b, acc[1]);
        acc[2] = fma_row(a.z, b, acc[2]);
        acc[3] = fma_row(a.w, b, acc[3]);
    }
}

// KEEP: the backward's recomputation (writes the states at the chunks' starts and E, no outputs).
template <typename T, bool KEEP>
__global__ void __launch_bounds__(256)
walk_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
            const float *__restrict__ beta, const int *__restrict__ lengths, const float *S0, int NH, int NHV,
            int S, int DK, int DV, float scale, Workspace w, T *__restrict__ o, float *S_final)
{
    extern __shared__ __align__(16) unsigned char raw[];
    WalkSmem &sm = *reinterpret_cast<WalkSmem *>(raw);
    constexpr bool ASYNC = sizeof(T) == 4;   // bf16 is widened on its way: no asynchronous copy
    const int tid = threadIdx.x, c0 = blockIdx.x * VT, bhv = blockIdx.y, b = bhv / NHV;
    const int bh = b * NH + (bhv % NHV) / (NHV / NH);
    const int u = tid >> 3, j0 = (tid & 7) * 4, col = c0 + j0, t0 = 2 * u, top = 8 * (tid >> 5) + 8;   // top: behind the warp's tokens
    const bool in = col < DV, mine = in && 4 * u < DK;   // mine: the thread's rows of the state exist
    griddep_wait();
    griddep_launch_dependents();
    const int n = live_tokens(lengths, b, S), nc = (n + CH - 1) / CH;
    auto stage_kq = [&](int c) {
        const size_t at = ((size_t)bh * S + c * CH) * DK;
        stage_rows(k + at, min(CH, n - c * CH), DK, sm.kq[c & 1], tid);
        if (!KEEP) stage_rows(q + at, min(CH, n - c * CH), DK, sm.kq[c & 1] + 64 * LDX, tid);
    };
    auto stage_tp = [&](int c) {
        const size_t at = ((size_t)bhv * w.NC + c) * 4096;
        stage64(w.T + at, sm.t, tid);
        if (!KEEP) stage64(w.P + at, sm.p, tid);
    };
    GateReg gr;
    auto read_gates = [&](int c) {
        if (tid < 64) gr.read(w, beta, (size_t)bhv * w.NC + c, (size_t)bhv * S + c * CH, min(CH, n - c * CH), tid);
    };
    Row4 s[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        s[r] = row4(S0 && mine ? ld4(S0 + ((size_t)bhv * DK + 4 * u + r) * DV + col) : make_float4(0.f, 0.f, 0.f, 0.f));
        str(sm.st + (4 * u + r) * VT + j0, s[r]);
    }
    if (nc > 0) {
        if (ASYNC) stage_kq(0);
        stage_tp(0);
        read_gates(0);
        if (tid < 64) gr.put(sm.g[0], tid);
    }
    for (int c = 0; c < nc; ++c) {
        const int len = min(CH, n - c * CH);
        const size_t ch = (size_t)bhv * w.NC + c, vrow = (size_t)bhv * S + c * CH;
        const float *kq = sm.kq[c & 1];
        const Gates &g = sm.g[c & 1];
        if (!ASYNC) stage_kq(c);
        Row4 vr[2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
            vr[r] = row4(in && t0 + r < len ? load4(v + (vrow + t0 + r) * DV + col) : make_float4(0.f, 0.f, 0.f, 0.f));
        copies_done();
        __syncthreads();
        if (c + 1 < nc) {
            if (ASYNC) stage_kq(c + 1);
            read_gates(c + 1);
        }
        if (KEEP && mine) {
#pragma unroll
            for (int r = 0; r < 4; ++r) st4(w.SC + (ch * DK + 4 * u + r) * DV + col, flat(s[r]));
        }
        Row4 xk[2] = {}, xq[2] = {};
        if (KEEP) {
            rows_times<2>(kq + t0 * LDX, LDX, sm.st + j0, 0, DK, xk);
        } else {   // K and Q on the same rows of the state
            Row4 x[4] = {};
            const float *a = kq + t0 * LDX, *bp = sm.st + j0;
#pragma unroll 2
            for (int l = 0; l < DK; l += 4) {
                const float4 f[4] = {ld4(a + l), ld4(a + LDX + l), ld4(a + 64 * LDX + l), ld4(a + 65 * LDX + l)};
                const Row4 b0 = ldr(bp + l * VT), b1 = ldr(bp + (l + 1) * VT), b2 = ldr(bp + (l + 2) * VT), b3 = ldr(bp + (l + 3) * VT);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    x[r] = fma_row(f[r].w, b3, fma_row(f[r].z, b2, fma_row(f[r].y, b1, fma_row(f[r].x, b0, x[r]))));
            }
            xk[0] = x[0]; xk[1] = x[1]; xq[0] = x[2]; xq[1] = x[3];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = t0 + r;
            str(sm.y + t * VT + j0, t < len ? fma_row(-g.ea[t], xk[r], vr[r]) : Row4{0, 0});
        }
        __syncthreads();
        Row4 e[2] = {};
        rows_times<2>(sm.t + t0 * LDW, LDW, sm.y + j0, 0, top, e);   // T is zero above its diagonal
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = t0 + r;
            if (KEEP && in) st4(w.E + (ch * 64 + t) * DV + col, flat(e[r]));
            e[r] = mul_row(g.bt[t], e[r]);
            str(sm.z + t * VT + j0, mul_row(g.eo[t], e[r]));
            if (!KEEP) str(sm.y + t * VT + j0, e[r]);
        }
        if (c + 1 < nc && tid < 64) gr.put(sm.g[(c + 1) & 1], tid);
        __syncthreads();
        if (!KEEP) {
            Row4 x[2] = {};
            rows_times<2>(sm.p + t0 * LDW, LDW, sm.y + j0, 0, top, x);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int t = t0 + r;
                if (in && t < len) store4(o + (vrow + t) * DV + col, flat(mul_row(scale, fma_row(g.ea[t], xq[r], x[r]))));
            }
            __syncthreads();   // P is read
        }
        if (c + 1 < nc) stage_tp(c + 1);
        if (4 * u < DK) {
#pragma unroll
            for (int r = 0; r < 4; ++r) s[r] = mul_row(g.ea[63], s[r]);
            cols4_times(kq + 4 * u, LDX, sm.z + j0, s);
#pragma unroll
            for (int r = 0; r < 4; ++r) str(sm.st + (4 * u + r) * VT + j0, s[r]);
        }
    }
    if (KEEP) return;
    for (long long i = tid; i < (S - n) * 8ll; i += 256) {   // padding
        const int j = c0 + (int)(i & 7) * 4;
        if (j < DV) store4(o + ((size_t)bhv * S + n + (i >> 3)) * DV + j, make_float4(0.f, 0.f, 0.f, 0.f));
    }
    if (S_final && mine) {
#pragma unroll
        for (int r = 0; r < 4; ++r) st4(S_final + ((size_t)bhv * DK + 4 * u + r) * DV + col, flat(s[r]));
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
reverse_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ d_o,
               const float *__restrict__ beta, const int *__restrict__ lengths, const float *dS_final, int NH,
               int NHV, int S, int DK, int DV, float scale, Workspace w, T *__restrict__ dv, float *dS0)
{
    extern __shared__ __align__(16) unsigned char raw[];
    WalkSmem &sm = *reinterpret_cast<WalkSmem *>(raw);
    constexpr bool ASYNC = sizeof(T) == 4;
    const int tid = threadIdx.x, c0 = blockIdx.x * VT, bhv = blockIdx.y, b = bhv / NHV;
    const int bh = b * NH + (bhv % NHV) / (NHV / NH);
    const int u = tid >> 3, j0 = (tid & 7) * 4, col = c0 + j0, t0 = 2 * u, low = 8 * (tid >> 5);   // low: the warp's first token
    const bool in = col < DV, mine = in && 4 * u < DK;
    griddep_wait();
    griddep_launch_dependents();
    const int n = live_tokens(lengths, b, S), nc = (n + CH - 1) / CH;
    auto stage_kq = [&](int c) {
        const size_t at = ((size_t)bh * S + c * CH) * DK;
        stage_rows(k + at, min(CH, n - c * CH), DK, sm.kq[c & 1], tid);
        stage_rows(q + at, min(CH, n - c * CH), DK, sm.kq[c & 1] + 64 * LDX, tid);
    };
    auto stage_tp = [&](int c) {
        const size_t at = ((size_t)bhv * w.NC + c) * 4096;
        stage64(w.T + at, sm.t, tid);
        stage64(w.P + at, sm.p, tid);
    };
    GateReg gr;
    auto read_gates = [&](int c) {
        if (tid < 64) gr.read(w, beta, (size_t)bhv * w.NC + c, (size_t)bhv * S + c * CH, min(CH, n - c * CH), tid);
    };
    Row4 s[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        s[r] = row4(dS_final && mine ? ld4(dS_final + ((size_t)bhv * DK + 4 * u + r) * DV + col) : make_float4(0.f, 0.f, 0.f, 0.f));
        str(sm.st + (4 * u + r) * VT + j0, s[r]);
    }
    if (nc > 0) {
        if (ASYNC) stage_kq(nc - 1);
        stage_tp(nc - 1);
        read_gates(nc - 1);
        if (tid < 64) gr.put(sm.g[(nc - 1) & 1], tid);
    }
    for (int c = nc - 1; c >= 0; --c) {
        const int len = min(CH, n - c * CH);
        const size_t ch = (size_t)bhv * w.NC + c, vrow = (size_t)bhv * S + c * CH;
        const float *kq = sm.kq[c & 1];
        const Gates &g = sm.g[c & 1];
        if (!ASYNC) stage_kq(c);
        Row4 dor[2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
            dor[r] = row4(in && t0 + r < len ? load4(d_o + (vrow + t0 + r) * DV + col) : make_float4(0.f, 0.f, 0.f, 0.f));
        copies_done();
        __syncthreads();
        if (c > 0) {
            if (ASYNC) stage_kq(c - 1);
            read_gates(c - 1);
        }
        if (mine) {
#pragma unroll
            for (int r = 0; r < 4; ++r) st4(w.DSC + (ch * DK + 4 * u + r) * DV + col, flat(s[r]));
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) str(sm.x + (t0 + r) * VT + j0, dor[r]);
        Row4 x[2] = {}, p[2] = {};
        rows_times<2>(kq + t0 * LDX, LDX, sm.st + j0, 0, DK, x);                    // K dS'
        __syncthreads();
        cols2_times(sm.p + t0, LDW, sm.x + j0, low, 64, p);                         // P^T dO, P lower
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = t0 + r;
            str(sm.y + t * VT + j0, mul_row(g.bt[t], fma_row(scale, p[r], mul_row(g.eo[t], x[r]))));
        }
        __syncthreads();
        Row4 e[2] = {};
        cols2_times(sm.t + t0, LDW, sm.y + j0, low, 64, e);                         // T^T
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = t0 + r;
            if (in) {
                st4(w.DV + (ch * 64 + t) * DV + col, flat(e[r]));
                if (t < len) store4(dv + (vrow + t) * DV + col, flat(e[r]));
            }
            str(sm.z + t * VT + j0, t < len ? mul_row(-g.ea[t], e[r]) : Row4{0, 0});
            str(sm.x + t * VT + j0, mul_row(scale * g.ea[t], dor[r]));
        }
        if (c > 0 && tid < 64) gr.put(sm.g[(c - 1) & 1], tid);
        __syncthreads();
        if (c > 0) stage_tp(c - 1);
        if (4 * u < DK) {
#pragma unroll
            for (int r = 0; r < 4; ++r) s[r] = mul_row(g.ea[63], s[r]);
            cols4_times(kq + 4 * u, LDX, sm.z + j0, s);
            cols4_times(kq + 64 * LDX + 4 * u, LDX, sm.x + j0, s);
#pragma unroll
            for (int r = 0; r < 4; ++r) str(sm.st + (4 * u + r) * VT + j0, s[r]);
        }
    }
    for (long long i = tid; i < (S - n) * 8ll; i += 256) {
        const int j = c0 + (int)(i & 7) * 4;
        if (j < DV) store4(dv + ((size_t)bhv * S + n + (i >> 3)) * DV + j, make_float4(0.f, 0.f, 0.f, 0.f));
    }
    if (dS0 && mine) {
#pragma unroll
        for (int r = 0; r < 4; ++r) st4(dS0 + ((size_t)bhv * DK + 4 * u + r) * DV + col, flat(s[r]));
    }
}

// ---------------------------------------------------------------- gradients of a chunk

constexpr int LDK = 132;   // row stride of K and Q [64][128]
constexpr size_t GRAD_SMEM =
    sizeof(float) * (2 * 64 * LDK + 2 * 64 * LDT + 32 * (LDR + LDT + LDR + LDR) + 5 * 64 + 32) + sizeof(float2) * 64;

// The thread's 8 x 8 tile of a product with 128 columns: rows ra + {0..3}, rb + {0..3}, columns
// 4 (tid & 15) + {0..3} and 64 more.
MLSTM_DEVINL void fma8x8(float (&acc)[8][8], float4 a0, float4 a1, float4 b0, float4 b1)
{
    const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
    const float bv[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
}

MLSTM_DEVINL float half_warp_sum(float x)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// One CTA per chunk and key head, over the value heads on it; dq and dk stay in registers.  Where that leaves half
// the SMs without a CTA, one per value head (gridDim.z of them): each then leaves its share of dq and dk in fp32
// where its states were, which it has read, and sum_heads_kernel adds them in order.  4 key heads of 333 tokens with
// three value heads each, 64 x 72 (24 CTAs or 72): 61 us, 6 of them the
// sum, against 147.
template <typename T>
__global__ void __launch_bounds__(256, 1)
grad_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ d_o,
            const float *__restrict__ beta, const int *__restrict__ lengths, int NH, int NHV, int S, int DK, int DV,
            float scale, Workspace w, T *__restrict__ dq, T *__restrict__ dk, float *__restrict__ dg,
            float *__restrict__ dbeta)
{
    extern __shared__ __align__(16) float sm[];
    float *ks = sm, *qs = ks + 64 * LDK;          // [64][LDK] K, Q, columns behind DK zero
    float *mp = qs + 64 * LDK, *ma = mp + 64 * LDT;   // [64][LDT] dP * D, dA * D
    float *ta = ma + 64 * LDT;                    // [32][LDR] value block: dO in 0..63, dV in 64..127
    float *te = ta + 32 * LDR;                    // [32][LDT] E
    float *ts = te + 32 * LDT;                    // [32][LDR] S transposed
    float *td = ts + 32 * LDR;                    // [32][LDR] dS' transposed
    float *ea = td + 32 * LDR, *eo = ea + 64, *bt = eo + 64, *zin = bt + 64, *zout = zin + 64;
    float *ssum = zout + 64;                      // [32]
    float2 *a = reinterpret_cast<float2 *>(ssum + 32);
    const int tid = threadIdx.x, lane = tid & 31, c = blockIdx.x, bh = blockIdx.y, b = bh / NH, group = NHV / NH;
    const bool split = gridDim.z > 1;
    const int h0 = split ? blockIdx.z : 0, h1 = split ? h0 + 1 : group;
    const int ty = tid >> 4, tx = tid & 15;
    griddep_wait();
    griddep_launch_dependents();
    const int full = min(CH, S - c * CH);
    const int len = min(full, live_tokens(lengths, b, S) - c * CH);
    const size_t row0 = (size_t)bh * S + c * CH;
    const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
    const int first = max(len, 0);
    for (int i = tid; h0 == 0 && i < (full - first) * (DK / 4); i += 256) {   // padding
        const size_t at = (row0 + first) * DK + (size_t)i * 4;
        store4(dq + at, zero4);
        store4(dk + at, zero4);
    }
    for (int h = h0; h < h1; ++h)
        if (tid < full - first) {
            const size_t gt = (size_t)(b * NHV + (bh % NH) * group + h) * S + c * CH + first + tid;
            dg[gt] = 0.f;
            dbeta[gt] = 0.f;
        }
    if (len <= 0) return;
    for (int i = tid; i < 64 * 32; i += 256) {
        const int r = i >> 5, d = (i & 31) * 4;
        const bool ok = r < len && d < DK;
        st4(ks + r * LDK + d, ok ? load4(k + (row0 + r) * DK + d) : zero4);
        st4(qs + r * LDK + d, ok ? load4(q + (row0 + r) * DK + d) : zero4);
    }
    float acc[8][8] = {};   // rows 4 ty + {0..3} of dq, and of dk
    for (int h = h0; h < h1; ++h) {
        const int bhv = b * NHV + (bh % NH) * group + h;
        const size_t ch = (size_t)bhv * w.NC + c, vrow = (size_t)bhv * S + c * CH;
        __syncthreads();
        if (tid < 64) {
            const float2 x = w.A[ch * 64 + tid];
            a[tid] = x;
            ea[tid] = expf(x.x + x.y);
            eo[tid] = expf(gate_diff(w.A[ch * 64 + 63], x));
            bt[tid] = tid < len ? beta[vrow + tid] : 0.f;
        }
        __syncthreads();
        // H = dV E^T and dO E^T (64 x 64 each), then Z = [dO; dV] S^T and W = E dS'^T
        float hx[8][4] = {}, z[8][8] = {}, wv[4][8] = {};
        float sd = 0.f;
        for (int v0 = 0; v0 < DV; v0 += 32) {
            for (int i = tid; i < 64 * 8; i += 256) {
                const int t = i & 63, j = (i >> 6) * 4;
                const bool ok = v0 + j < DV && t < len;
                const float4 x = ok ? load4(d_o + (vrow + t) * DV + v0 + j) : zero4;
                const float4 y = ok ? ld4(w.DV + (ch * 64 + t) * DV + v0 + j) : zero4;
                const float4 e = ok ? ld4(w.E + (ch * 64 + t) * DV + v0 + j) : zero4;
                const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w}, es[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    ta[(j + r) * LDR + t] = xs[r];
                    ta[(j + r) * LDR + 64 + t] = ys[r];
                    te[(j + r) * LDT + t] = es[r];
                }
            }
            for (int i = tid; i < 128 * 8; i += 256) {
                const int d = i & 127, j = (i >> 7) * 4;
                const bool ok = d < DK && v0 + j < DV;
                const float4 x = ok ? ld4(w.SC + (ch * DK + d) * DV + v0 + j) : zero4;
                const float4 y = ok ? ld4(w.DSC + (ch * DK + d) * DV + v0 + j) : zero4;
                sd += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
                ts[(j + 0) * LDR + d] = x.x; ts[(j + 1) * LDR + d] = x.y; ts[(j + 2) * LDR + d] = x.z; ts[(j + 3) * LDR + d] = x.w;
                td[(j + 0) * LDR + d] = y.x; td[(j + 1) * LDR + d] = y.y; td[(j + 2) * LDR + d] = y.z; td[(j + 3) * LDR + d] = y.w;
            }
            __syncthreads();
            for (int l = 0; l < 32; ++l) {
                const float4 x0 = ld4(ta + l * LDR + 4 * ty), x1 = ld4(ta + l * LDR + 64 + 4 * ty);
                const float4 s0 = ld4(ts + l * LDR + 4 * tx), s1 = ld4(ts + l * LDR + 64 + 4 * tx);
                fma8x8(z, x0, x1, s0, s1);
                const float4 e0 = ld4(te + l * LDT + 4 * tx);
                const float xv[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                const float ev[4] = {e0.x, e0.y, e0.z, e0.w};
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) hx[i][j] = fmaf(xv[i], ev[j], hx[i][j]);
                const float4 er = ld4(te + l * LDT + 4 * ty);
                const float4 d0 = ld4(td + l * LDR + 4 * tx), d1 = ld4(td + l * LDR + 64 + 4 * tx);
                const float rv[4] = {er.x, er.y, er.z, er.w};
                const float dv[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) wv[i][j] = fmaf(rv[i], dv[j], wv[i][j]);
            }
            __syncthreads();
        }
        sd = warp_sum(sd);
        if (lane == 0) ssum[tid >> 5] = sd;
        // the inter-chunk terms of dq and dk, and their products with q and k
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 4 * ty + r;
            const float fq = scale * ea[t], fk = -ea[t], fw = eo[t];
            float zi = 0.f, zo = 0.f;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int d = s < 4 ? 4 * tx + s : 60 + 4 * tx + s;
                const float x = fq * z[r][s], y = fk * z[4 + r][s], u = fw * wv[r][s];
                acc[r][s] += x;
                acc[4 + r][s] += y + bt[t] * u;
                zi += x * qs[t * LDK + d] + y * ks[t * LDK + d];
                zo += u * ks[t * LDK + d];
            }
            zi = half_warp_sum(zi);
            zo = half_warp_sum(zo);
            if (tx == 0) { zin[t] = zi; zout[t] = zo; }
        }
        // dP * D and dA * D to mp and ma; first the pairs' shares of the gates' and of beta's gradients
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 4 * ty + r;
            const float4 p4 = ld4(w.P + ch * 4096 + i * 64 + 4 * tx), k4 = ld4(w.KK + ch * 4096 + i * 64 + 4 * tx);
            const float pv[4] = {p4.x, p4.y, p4.z, p4.w}, kv[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int j = 4 * tx + s;
                const float z = scale * hx[r][s] * pv[s] - hx[4 + r][s] * kv[s];   // both zero above the diagonal
                mp[i * LDT + j] = j < i ? bt[j] * z : 0.f;
                ma[i * LDT + j] = z;
            }
        }
        __syncthreads();
        if (tid < 64) {   // row i: the sums over j < t
            float s = 0.f;
            for (int j = 0; j < 64; ++j) {
                const float x = mp[tid * LDT + j];
                mp[tid * LDT + j] = s;
                s += x;
            }
        } else if (tid < 128) {   // column j of the pairs
            const int j = tid - 64;
            float s = zout[j];
            for (int i = j; i < 64; ++i) s += ma[i * LDT + j];
            if (j < len) dbeta[vrow + j] = s;
        }
        __syncthreads();
        if (tid < len) {
            const int t = tid;
            float s = 0.f;
            for (int i = t; i < 64; ++i) s += mp[i * LDT + t] + zin[i];
            for (int j = 0; j < t; ++j) s += bt[j] * zout[j];
            float sdd = 0.f;
            for (int i = 0; i < 8; ++i) sdd += ssum[i];
            dg[vrow + t] = s + ea[63] * sdd;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 4 * ty + r;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int j = 4 * tx + s;
                const float dec = j <= i ? bt[j] * expf(gate_diff(a[i], a[j])) : 0.f;
                mp[i * LDT + j] = j <= i ? scale * dec * hx[r][s] : 0.f;
                ma[i * LDT + j] = j < i ? -dec * hx[4 + r][s] : 0.f;
            }
        }
        __syncthreads();
        // dq_i += sum_j mp_ij k_j;  dk_i += sum_j mp_ji q_j + (ma_ij + ma_ji) k_j
        for (int j = 0; j < 64; ++j) {
            const float4 k0 = ld4(ks + j * LDK + 4 * tx), k1 = ld4(ks + j * LDK + 64 + 4 * tx);
            const float4 q0 = ld4(qs + j * LDK + 4 * tx), q1 = ld4(qs + j * LDK + 64 + 4 * tx);
            const float4 pj = ld4(mp + j * LDT + 4 * ty), aj = ld4(ma + j * LDT + 4 * ty);
            const float pr[4] = {pj.x, pj.y, pj.z, pj.w}, ar[4] = {aj.x, aj.y, aj.z, aj.w};
            const float kv[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
            const float qv[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 4 * ty + r;
                const float x = mp[i * LDT + j], y = ma[i * LDT + j] + ar[r];
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    acc[r][s] = fmaf(x, kv[s], acc[r][s]);
                    acc[4 + r][s] = fmaf(pr[r], qv[s], fmaf(y, kv[s], acc[4 + r][s]));
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int t = 4 * ty + r;
        if (t >= len) continue;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int d = 64 * s + 4 * tx;
            if (d >= DK) continue;
            if (split) {
                const size_t at = ((size_t)(b * NHV + (bh % NH) * group + h0) * w.NC + c) * DK * DV + (size_t)t * DK + d;
                st4(w.SC + at, make_float4(acc[r][4 * s], acc[r][4 * s + 1], acc[r][4 * s + 2], acc[r][4 * s + 3]));
                st4(w.DSC + at, make_float4(acc[4 + r][4 * s], acc[4 + r][4 * s + 1], acc[4 + r][4 * s + 2], acc[4 + r][4 * s + 3]));
                continue;
            }
            store4(dq + (row0 + t) * DK + d, make_float4(acc[r][4 * s], acc[r][4 * s + 1], acc[r][4 * s + 2], acc[r][4 * s + 3]));
            store4(dk + (row0 + t) * DK + d,
                   make_float4(acc[4 + r][4 * s], acc[4 + r][4 * s + 1], acc[4 + r][4 * s + 2], acc[4 + r][4 * s + 3]));
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
sum_heads_kernel(const int *__restrict__ lengths, int NH, int NHV, int S, int DK, int DV, Workspace w, T *__restrict__ dq,
                 T *__restrict__ dk)
{
    const int c = blockIdx.x, bh = blockIdx.y, b = bh / NH, group = NHV / NH;
    griddep_wait();
    griddep_launch_dependents();
    const int len = min(CH, live_tokens(lengths, b, S) - c * CH);
    const size_t first = (size_t)(b * NHV + (bh % NH) * group) * w.NC + c, step = (size_t)w.NC * DK * DV;
    for (int i = threadIdx.x; i < len * (DK / 4); i += 256) {
        const float *x = w.SC + first * DK * DV + (size_t)i * 4, *y = w.DSC + first * DK * DV + (size_t)i * 4;
        float4 q4 = ld4(x), k4 = ld4(y);
        for (int h = 1; h < group; ++h) {
            const float4 a = ld4(x + h * step), e = ld4(y + h * step);
            q4 = make_float4(q4.x + a.x, q4.y + a.y, q4.z + a.z, q4.w + a.w);
            k4 = make_float4(k4.x + e.x, k4.y + e.y, k4.z + e.z, k4.w + e.w);
        }
        const size_t at = ((size_t)bh * S + c * CH) * DK + (size_t)i * 4;
        store4(dq + at, q4);
        store4(dk + at, k4);
    }
}

__global__ void state_copy_kernel(const float *S0, float *S_final, size_t n)
{
    griddep_wait();
    griddep_launch_dependents();
    for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x)
        S_final[i] = S0 ? S0[i] : 0.f;
}

template <typename K>
cudaError_t smem_limit(K kernel, size_t bytes)
{
    return ensure_dynamic_smem((const void *)kernel, (int)bytes);
}

template <typename T>
cudaError_t prep_t(const Args &a, const Workspace &w, bool kk)
{
    cudaError_t e = smem_limit(prep_kernel<T>, PREP_SMEM);
    if (e != cudaSuccess) return e;
    const bool split = (long long)w.NC * a.B * a.NHV <= 2 * 148;
    return launch_kernel(prep_kernel<T>, dim3(w.NC, a.B * a.NH, split ? a.NHV / a.NH : 1), dim3(256), PREP_SMEM, a.stream, 1, (const T *)a.q,
                         (const T *)a.k, a.g, a.beta, a.lengths, a.NH, a.NHV, a.S, a.DK, w, kk);
}

template <typename T, bool KEEP>
cudaError_t walk_t(const Args &a, const Workspace &w, void *o, float *S_final)
{
    cudaError_t e = smem_limit(walk_kernel<T, KEEP>, sizeof(WalkSmem));
    if (e != cudaSuccess) return e;
    return launch_kernel(walk_kernel<T, KEEP>, dim3((a.DV + VT - 1) / VT, a.B * a.NHV), dim3(256), sizeof(WalkSmem), a.stream, 1,
                         (const T *)a.q, (const T *)a.k, (const T *)a.v, a.beta, a.lengths, a.S0, a.NH, a.NHV, a.S,
                         a.DK, a.DV, a.scale, w, (T *)o, S_final);
}

template <typename T>
cudaError_t reverse_t(const Args &a, const Workspace &w, const void *d_o, const float *dS_final, void *dv, float *dS0)
{
    cudaError_t e = smem_limit(reverse_kernel<T>, sizeof(WalkSmem));
    if (e != cudaSuccess) return e;
    return launch_kernel(reverse_kernel<T>, dim3((a.DV + VT - 1) / VT, a.B * a.NHV), dim3(256), sizeof(WalkSmem), a.stream, 1,
                         (const T *)a.q, (const T *)a.k, (const T *)d_o, a.beta, a.lengths, dS_final, a.NH, a.NHV, a.S,
                         a.DK, a.DV, a.scale, w, (T *)dv, dS0);
}

template <typename T>
cudaError_t grad_t(const Args &a, const Workspace &w, const void *d_o, void *dq, void *dk, float *dg, float *dbeta)
{
    cudaError_t e = smem_limit(grad_kernel<T>, GRAD_SMEM);
    if (e != cudaSuccess) return e;
    // the shares take 64 rows of DK where DK rows of DV were
    const bool split = a.NHV > a.NH && a.DV >= 64 && 2ll * w.NC * a.B * a.NH <= 148;
    e = launch_kernel(grad_kernel<T>, dim3(w.NC, a.B * a.NH, split ? a.NHV / a.NH : 1), dim3(256), GRAD_SMEM, a.stream, 1,
                      (const T *)a.q, (const T *)a.k, (const T *)d_o, a.beta, a.lengths, a.NH, a.NHV, a.S, a.DK, a.DV,
                      a.scale, w, (T *)dq, (T *)dk, dg, dbeta);
    if (e != cudaSuccess || !split) return e;
    return launch_kernel(sum_heads_kernel<T>, dim3(w.NC, a.B * a.NH), dim3(256), 0, a.stream, 1, a.lengths, a.NH, a.NHV,
                         a.S, a.DK, a.DV, w, (T *)dq, (T *)dk);
}

}  // namespace

cudaError_t launch_prep(const Args &a, const Workspace &w, bool kk)
{
    return a.bf16 ? prep_t<__nv_bfloat16>(a, w, kk) : prep_t<float>(a, w, kk);
}

cudaError_t launch_walk(const Args &a, const Workspace &w, void *o, float *S_final, bool keep)
{
    if (a.bf16) return keep ? walk_t<__nv_bfloat16, true>(a, w, o, S_final) : walk_t<__nv_bfloat16, false>(a, w, o, S_final);
    return keep ? walk_t<float, true>(a, w, o, S_final) : walk_t<float, false>(a, w, o, S_final);
}

cudaError_t launch_reverse(const Args &a, const Workspace &w, const void *d_o, const float *dS_final, void *dv, float *dS0)
{
    return a.bf16 ? reverse_t<__nv_bfloat16>(a, w, d_o, dS_final, dv, dS0) : reverse_t<float>(a, w, d_o, dS_final, dv, dS0);
}

cudaError_t launch_grad(const Args &a, const Workspace &w, const void *d_o, void *dq, void *dk, float *dg, float *dbeta)
{
    return a.bf16 ? grad_t<__nv_bfloat16>(a, w, d_o, dq, dk, dg, dbeta) : grad_t<float>(a, w, d_o, dq, dk, dg, dbeta);
}

cudaError_t launch_state_copy(const float *S0, float *S_final, size_t n, cudaStream_t stream)
{
    const unsigned grid = (unsigned)std::min<size_t>((n + 255) / 256, 148 * 8);
    return launch_kernel(state_copy_kernel, dim3(grid), dim3(256), 0, stream, 1, S0, S_final, n);
}

}  // namespace gdelta
}  // namespace mlstm
