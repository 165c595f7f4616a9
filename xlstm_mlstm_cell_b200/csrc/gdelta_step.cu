// gdelta_step.cu -- one token of the gated delta rule for every value head, state in place:
//   x = S^T k,  y = S^T q,  u = beta (v - e^g x),  S <- e^g S + k u^T,  o = scale (e^g y + (k . q) u)
//
// Bound by HBM: the fp32 state is read once and written once.  The correction u needs the column sums
// over the whole old state before any of it can be updated, so a CTA takes 32 value columns of a head
// and keeps its DK x 32 tile (16 KB at DK 128) in registers between the sums and the update; o comes
// from the old state's sums too, so one pass serves both.  A thread owns four columns (one 16-byte
// vector) of every 16th row, eight vectors in flight.  8192 heads of 128 x 128 (0.5 GB each way) take 157 us,
// 6.9 TB/s; with 256 threads of four vectors 262 us (the sums over more warps and half the loads in
// flight per thread), with whole rows of 128 columns 276 us; 64 columns of 16 vectors are as fast, with
// half the CTAs for a single sequence.
#include "common.cuh"
#include "gdelta_internal.h"

namespace mlstm {
namespace gdelta {
namespace {


MLSTM_DEVINL float4 fma4(float f, float4 x, float4 acc)
{
    return make_float4(fmaf(f, x.x, acc.x), fmaf(f, x.y, acc.y), fmaf(f, x.z, acc.z), fmaf(f, x.w, acc.w));
}

// Sum over the lanes of a warp that hold the same columns (CG lanes side by side hold different ones).
template <int CG>
MLSTM_DEVINL float4 rows_sum(float4 x)
{
#pragma unroll
    for (int o = CG; o <= 16; o <<= 1) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
        x.z += __shfl_xor_sync(0xffffffffu, x.z, o);
        x.w += __shfl_xor_sync(0xffffffffu, x.w, o);
    }
    return x;
}

// CG threads across (4 CG columns), RG = 128 / ROWS row groups.
template <typename T, int CG, int ROWS>
__global__ void __launch_bounds__(CG * (128 / ROWS))
step_kernel(float *__restrict__ state, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
            const float *__restrict__ g, const float *__restrict__ beta, int NH, int NHV, int DK, int DV, int tiles,
            float scale, T *__restrict__ o)
{
    constexpr int RG = 128 / ROWS, WARPS = CG * RG / 32;
    __shared__ float4 part[WARPS][2][CG];
    __shared__ float kqs[WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bhv = blockIdx.x / tiles, col = (blockIdx.x % tiles) * (4 * CG) + (tid % CG) * 4, r0 = tid / CG;
    const int bh = bhv / NHV * NH + (bhv % NHV) / (NHV / NH);
    const bool in = col < DV;
    griddep_wait();
    griddep_launch_dependents();
    float *sp = state + ((size_t)bhv * DK + r0) * DV + col;
    float4 s[ROWS];
    float kr[ROWS], qr[ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u)
        s[u] = in && r0 + RG * u < DK ? __ldcs(reinterpret_cast<const float4 *>(sp + (size_t)RG * u * DV))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        const bool ok = r0 + RG * u < DK;
        kr[u] = ok ? to_f32(k[(size_t)bh * DK + r0 + RG * u]) : 0.f;
        qr[u] = ok ? to_f32(q[(size_t)bh * DK + r0 + RG * u]) : 0.f;
    }
    const float f = expf(g[bhv]), bt = beta[bhv];
    const float4 v4 = in ? load4(v + (size_t)bhv * DV + col) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    float kq = 0.f;
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        x = fma4(kr[u], s[u], x);
        y = fma4(qr[u], s[u], y);
        kq = fmaf(kr[u], qr[u], kq);
    }
    x = rows_sum<CG>(x);
    y = rows_sum<CG>(y);
#pragma unroll
    for (int o = CG; o <= 16; o <<= 1) kq += __shfl_xor_sync(0xffffffffu, kq, o);
    if (lane < CG) {
        part[warp][0][lane] = x;
        part[warp][1][lane] = y;
        if (lane == 0) kqs[warp] = kq;
    }
    __syncthreads();
    x = y = make_float4(0.f, 0.f, 0.f, 0.f);
    kq = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        x = fma4(1.f, part[w][0][tid % CG], x);
        y = fma4(1.f, part[w][1][tid % CG], y);
        kq += kqs[w];
    }
    const float4 u = make_float4(bt * fmaf(-f, x.x, v4.x), bt * fmaf(-f, x.y, v4.y), bt * fmaf(-f, x.z, v4.z),
                                 bt * fmaf(-f, x.w, v4.w));
    if (!in) return;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
        if (r0 + RG * r < DK)
            __stcs(reinterpret_cast<float4 *>(sp + (size_t)RG * r * DV),
                   make_float4(fmaf(f, s[r].x, kr[r] * u.x), fmaf(f, s[r].y, kr[r] * u.y),
                               fmaf(f, s[r].z, kr[r] * u.z), fmaf(f, s[r].w, kr[r] * u.w)));
    if (r0 == 0)
        store4(o + (size_t)bhv * DV + col,
               make_float4(scale * fmaf(f, y.x, kq * u.x), scale * fmaf(f, y.y, kq * u.y),
                           scale * fmaf(f, y.z, kq * u.z), scale * fmaf(f, y.w, kq * u.w)));
}

template <typename T, int CG, int ROWS>
cudaError_t step_cg(const StepArgs &a)
{
    const int tiles = (a.DV + 4 * CG - 1) / (4 * CG);
    return launch_kernel(step_kernel<T, CG, ROWS>, dim3((unsigned)a.BHV * tiles), dim3(CG * (128 / ROWS)), 0, a.stream, 1,
                         a.state, (const T *)a.q, (const T *)a.k, (const T *)a.v, a.g, a.beta, a.NH, a.NHV, a.DK, a.DV,
                         tiles, a.scale, (T *)a.o);
}

template <typename T>
cudaError_t step_t(const StepArgs &a)
{
    return step_cg<T, 8, 8>(a);
}

}  // namespace

cudaError_t launch_step(const StepArgs &a) { return a.bf16 ? step_t<__nv_bfloat16>(a) : step_t<float>(a); }

}  // namespace gdelta
}  // namespace mlstm
