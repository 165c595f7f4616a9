// qknorm.cu -- norms of queries and keys per head with the position rotation, forward and backward:
//   r = 1 / sqrt(mean|sum(x^2) + eps),  z = r w x,  y = z with pairs of its first RD elements rotated;
//   d = inverse rotation of dy,  dw = sum of d r x,  dx = r (w d - r^2 x mean|sum(w d x)).
//
// Bound by HBM: every vector is read once and written once (the backward reads two).  A CTA takes a few
// tokens with all their query and key heads, so that the tokens' cosines and sines are formed once, in
// shared memory, and serve every head; a group of lanes holds one vector in registers, each lane units of
// VEC + VEC elements chosen so that both elements of a rotated pair sit in the same lane: no exchange but
// the norm's sum over the group.  VEC is the widest vector that sizes, strides and pointers allow.
#include "common.cuh"
#include "qknorm.h"

#include <stdint.h>

#include <algorithm>

namespace mlstm {
namespace qknorm {
namespace {

constexpr int THREADS = 256;
constexpr int SPAN = 8;      // VEC elements times units per lane: a vector of 512 is 32 lanes x 2 x 8

struct Side {                // queries or keys
    const void *x, *dy;
    void *out;               // y or dx
    const float *w;
    qknorm_strides xs, os;
    int heads;
};

struct Params {
    Side side[2];
    const float *inv_freq;
    const int *positions;
    float *part;             // [grid][2][D] partial weight gradients, or NULL
    long long tokens;        // B * S
    int B, S, D, RD, l2, TT, GL;
    float eps;
};

template <typename T, int VEC> struct alignas(sizeof(T) * VEC) Vec { T e[VEC]; };

template <typename T, int VEC>
MLSTM_DEVINL void load_vec(const T *p, float *x)
{
    const Vec<T, VEC> v = *reinterpret_cast<const Vec<T, VEC> *>(p);
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = to_f32(v.e[i]);
}
template <typename T, int VEC>
MLSTM_DEVINL void store_vec(T *p, const float *x)
{
    Vec<T, VEC> v;
#pragma unroll
    for (int i = 0; i < VEC; ++i) v.e[i] = from_f32<T>(x[i]);
    *reinterpret_cast<Vec<T, VEC> *>(p) = v;
}

// A unit is VEC + VEC elements starting at o1 and o2.  Interleaved: 2 VEC neighbours.  Otherwise VEC
// elements of the rotated part's first half with their partners in its second, and behind the rotated
// part likewise (there the halves mean nothing).
template <int VEC, bool INTER>
MLSTM_DEVINL void unit_offsets(int u, int D, int RD, int &o1, int &o2, bool &turn)
{
    if (INTER) {
        o1 = 2 * VEC * u;
        o2 = o1 + VEC;
        turn = o1 < RD;
    } else {
        turn = u * VEC < RD / 2;
        o1 = turn ? u * VEC : RD / 2 + u * VEC;
        o2 = o1 + (turn ? RD / 2 : (D - RD) / 2);
    }
}

// Rotates a unit's pairs; cs holds the token's (cos, sin) of every pair.  sign -1 turns back.
template <int VEC, bool INTER>
MLSTM_DEVINL void rotate(float *x, const float2 *cs, int o1, float sign)
{
    if (INTER && VEC > 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e + 1 < VEC; e += 2) {
                const float2 t = cs[(o1 + h * VEC + e) / 2];
                float &a = x[h * VEC + e], &b = x[h * VEC + e + 1];
                const float c = t.x, s = sign * t.y, a0 = a;
                a = a0 * c - b * s;
                b = a0 * s + b * c;
            }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 t = cs[INTER ? o1 / 2 : o1 + e];
            float &a = x[e], &b = x[VEC + e];
            const float c = t.x, s = sign * t.y, a0 = a;
            a = a0 * c - b * s;
            b = a0 * s + b * c;
        }
    }
}

// The tile's cosines and sines.  The angle is formed in fp64 and brought to [-pi, pi] there, where an
// fp32 sine is accurate to its own rounding.
MLSTM_DEVINL void tile_angles(const Params &p, long long t0, int nt, float2 *cs, int tid)
{
    const int half = p.RD / 2;
    for (int i = tid; i < nt * half; i += THREADS) {
        const int t = i / half, pr = i - t * half;
        const long long tok = t0 + t;
        const int pos = p.positions ? p.positions[tok] : (int)(tok % p.S);
        const double ang = (double)pos * (double)p.inv_freq[pr];
        const double red = ang - 6.283185307179586477 * rint(ang * 0.15915494309189533577);
        float s, c;
        sincosf((float)red, &s, &c);
        cs[t * half + pr] = make_float2(c, s);
    }
}

// One vector (or the vectors of one lane group) forward or backward.  gw: the lane's share of the
// weight's gradient.
template <typename T, int VEC, bool INTER, bool BWD>
MLSTM_DEVINL void one_vector(const Params &p, const Side &sd, long long tok, int head, int gl, bool ok,
                             const float2 *cs, float *gw)
{
    constexpr int NU = SPAN / VEC;
    const int units = p.D / 2 / VEC;
    const int b = (int)(tok / p.S), t = (int)(tok % p.S);
    const T *x = (const T *)sd.x + b * sd.xs.batch + t * sd.xs.token + head * sd.xs.head;
    const size_t row = (((size_t)b * sd.heads + head) * p.S + t) * p.D;   // [B][heads][S][D]
    const T *dy = (const T *)sd.dy + row;
    float xv[NU][2 * VEC], dv[BWD ? NU : 1][2 * VEC];
    float s = 0.f, xd = 0.f;
#pragma unroll
    for (int n = 0; n < NU; ++n) {
        const int u = gl + n * p.GL;
        if (!ok || u >= units) continue;
        int o1, o2;
        bool turn;
        unit_offsets<VEC, INTER>(u, p.D, p.RD, o1, o2, turn);
        load_vec<T, VEC>(x + o1, xv[n]);
        load_vec<T, VEC>(x + o2, xv[n] + VEC);
        if (BWD) {
            load_vec<T, VEC>(dy + o1, dv[n]);
            load_vec<T, VEC>(dy + o2, dv[n] + VEC);
            if (turn) rotate<VEC, INTER>(dv[n], cs, o1, -1.f);
        }
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) {
            s = fmaf(xv[n][e], xv[n][e], s);
            if (BWD) {
                const float w = sd.w ? sd.w[e < VEC ? o1 + e : o2 + e - VEC] : 1.f;
                xd = fmaf(w * dv[n][e], xv[n][e], xd);
            }
        }
    }
    for (int o = p.GL / 2; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        if (BWD) xd += __shfl_xor_sync(0xffffffffu, xd, o);
    }
    const float inv_n = p.l2 ? 1.f : 1.f / (float)p.D;
    const float r = 1.f / sqrtf(fmaf(s, inv_n, p.eps));
    const float back = BWD ? r * r * (xd * inv_n) : 0.f;
    T *out = (T *)sd.out + (BWD ? b * sd.os.batch + t * sd.os.token + head * sd.os.head : (long long)row);
#pragma unroll
    for (int n = 0; n < NU; ++n) {
        const int u = gl + n * p.GL;
        if (!ok || u >= units) continue;
        int o1, o2;
        bool turn;
        unit_offsets<VEC, INTER>(u, p.D, p.RD, o1, o2, turn);
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) {
            const float w = sd.w ? sd.w[e < VEC ? o1 + e : o2 + e - VEC] : 1.f;
            if (BWD) {
                gw[n * 2 * VEC + e] = fmaf(dv[n][e], r * xv[n][e], gw[n * 2 * VEC + e]);
                xv[n][e] = r * (w * dv[n][e] - back * xv[n][e]);
            } else {
                xv[n][e] *= r * w;
            }
        }
        if (!BWD && turn) rotate<VEC, INTER>(xv[n], cs, o1, 1.f);
        store_vec<T, VEC>(out + o1, xv[n]);
        store_vec<T, VEC>(out + o2, xv[n] + VEC);
    }
}

template <typename T, int VEC, bool INTER, bool BWD>
__global__ void __launch_bounds__(THREADS)
qknorm_kernel(const Params p)
{
    extern __shared__ __align__(16) float2 cs[];   // [TT][RD / 2], at the end [groups][D] partial sums
    const int tid = threadIdx.x, gl = tid % p.GL, grp = tid / p.GL, groups = THREADS / p.GL;
    griddep_wait();
    griddep_launch_dependents();
    float gw[BWD ? 2 : 1][BWD ? 2 * SPAN : 1] = {};
    const long long ntiles = (p.tokens + p.TT - 1) / p.TT;
    for (long long tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
        const long long t0 = tile * p.TT;
        const int nt = (int)min((long long)p.TT, p.tokens - t0);
        if (p.RD) {
            __syncthreads();
            tile_angles(p, t0, nt, cs, tid);
            __syncthreads();
        }
#pragma unroll
        for (int sdi = 0; sdi < 2; ++sdi) {
            const Side &sd = p.side[sdi];
            const int rows = nt * sd.heads;
            for (int r0 = 0; r0 < rows; r0 += groups) {   // whole warps stay together for the sums
                const int r = r0 + grp;
                const bool ok = r < rows;
                const int t = ok ? r / sd.heads : 0, head = ok ? r - t * sd.heads : 0;
                one_vector<T, VEC, INTER, BWD>(p, sd, t0 + t, head, gl, ok, cs + t * (p.RD / 2), gw[BWD ? sdi : 0]);
            }
        }
    }
    if (BWD && p.part) {   // the groups' shares of the weights' gradients, added in order
        float *red = reinterpret_cast<float *>(cs);
        const int units = p.D / 2 / VEC;
        for (int sdi = 0; sdi < 2; ++sdi) {
            __syncthreads();
#pragma unroll
            for (int n = 0; n < SPAN / VEC; ++n) {
                const int u = gl + n * p.GL;
                if (u >= units) continue;
                int o1, o2;
                bool turn;
                unit_offsets<VEC, INTER>(u, p.D, p.RD, o1, o2, turn);
#pragma unroll
                for (int e = 0; e < 2 * VEC; ++e)
                    red[grp * p.D + (e < VEC ? o1 + e : o2 + e - VEC)] = gw[BWD ? sdi : 0][BWD ? n * 2 * VEC + e : 0];
            }
            __syncthreads();
            for (int d = tid; d < p.D; d += THREADS) {
                float s = 0.f;
                for (int i = 0; i < groups; ++i) s += red[i * p.D + d];
                p.part[((size_t)blockIdx.x * 2 + sdi) * p.D + d] = s;
            }
        }
    }
}

// dw[side][d] = sum over the CTAs' partials, 32 columns a CTA, 8 rows of it side by side.
__global__ void __launch_bounds__(256)
weight_sum_kernel(const float *__restrict__ part, int n, int D, float *dwq, float *dwk)
{
    __shared__ float red[8][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, sdi = blockIdx.y, d = blockIdx.x * 32 + tx;
    griddep_wait();
    griddep_launch_dependents();
    float s = 0.f;
    if (d < D)
        for (int i = ty; i < n; i += 8) s += part[((size_t)i * 2 + sdi) * D + d];
    red[ty][tx] = s;
    __syncthreads();
    float *dw = sdi ? dwk : dwq;
    if (ty == 0 && d < D && dw) {
        for (int i = 1; i < 8; ++i) s += red[i][tx];
        dw[d] = s;
    }
}

// CTAs of a launch: enough for every SM four times over, no more than there are tiles.
constexpr int MAX_CTAS = 148 * 4;

// The widest vector that divides the parts a unit is cut from and that every address is a multiple of.
int vector_width(const Params &p, int esize, bool inter, bool bwd)
{
    auto fits = [&](int vec) {
        if (inter ? (p.D % (2 * vec) || p.RD % (2 * vec)) : ((p.RD / 2) % vec || ((p.D - p.RD) / 2) % vec)) return false;
        const uintptr_t bytes = (uintptr_t)vec * esize;
        for (const Side &sd : p.side) {
            if (!sd.heads) continue;
            const uintptr_t bits = (uintptr_t)sd.x | (uintptr_t)sd.out | (uintptr_t)sd.dy |
                                   (uintptr_t)((sd.xs.batch | sd.xs.token | sd.xs.head) * esize) |
                                   (bwd ? (uintptr_t)((sd.os.batch | sd.os.token | sd.os.head) * esize) : 0);
            if (bits & (bytes - 1)) return false;
        }
        return true;
    };
    for (int vec = 16 / esize; vec > 1; vec /= 2)
        if (fits(vec)) return vec;
    return 1;
}

template <typename T, int VEC, bool INTER, bool BWD>
cudaError_t launch(Params p, int ctas, cudaStream_t stream)
{
    const int units = p.D / 2 / VEC;
    p.GL = 1;
    while (p.GL < 32 && p.GL < units) p.GL *= 2;
    size_t smem = sizeof(float2) * p.TT * (p.RD / 2);
    if (BWD && p.part) smem = std::max(smem, sizeof(float) * (THREADS / p.GL) * p.D);
    if (smem > 48 * 1024) {
        const cudaError_t e = ensure_dynamic_smem((const void *)qknorm_kernel<T, VEC, INTER, BWD>, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(qknorm_kernel<T, VEC, INTER, BWD>, dim3(ctas), dim3(THREADS), smem, stream, 1, p);
}

template <typename T, int VEC, bool BWD>
cudaError_t launch_inter(const Params &p, bool inter, int ctas, cudaStream_t stream)
{
    return inter ? launch<T, VEC, true, BWD>(p, ctas, stream) : launch<T, VEC, false, BWD>(p, ctas, stream);
}

template <bool BWD>
cudaError_t dispatch(const Params &p, bool bf16, bool inter, int ctas, cudaStream_t stream)
{
    const int vec = vector_width(p, bf16 ? 2 : 4, inter, BWD);
    if (bf16) {
        switch (vec) {
        case 8: return launch_inter<__nv_bfloat16, 8, BWD>(p, inter, ctas, stream);
        case 4: return launch_inter<__nv_bfloat16, 4, BWD>(p, inter, ctas, stream);
        case 2: return launch_inter<__nv_bfloat16, 2, BWD>(p, inter, ctas, stream);
        default: return launch_inter<__nv_bfloat16, 1, BWD>(p, inter, ctas, stream);
        }
    }
    switch (vec) {
    case 4: return launch_inter<float, 4, BWD>(p, inter, ctas, stream);
    case 2: return launch_inter<float, 2, BWD>(p, inter, ctas, stream);
    default: return launch_inter<float, 1, BWD>(p, inter, ctas, stream);
    }
}

// Tokens per tile: one while there are few (a decode step spreads over the GPU), else four.
int tile_tokens(long long tokens) { return tokens <= 2 * MAX_CTAS ? 1 : 4; }
int cta_count(long long tokens)
{
    const int tt = tile_tokens(tokens);
    return (int)std::min<long long>((tokens + tt - 1) / tt, MAX_CTAS);
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

mlstm_status check(const Params &p, mlstm_dtype dt, int NHQ, int NHK, qknorm_kind kind, bool bwd)
{
    if (p.B < 0 || p.S < 0 || NHQ < 0 || NHK < 0 || p.RD < 0 || p.RD > p.D || p.RD % 2) return MLSTM_ERR_INVALID_ARG;
    if (kind != QKNORM_RMS && kind != QKNORM_L2) return MLSTM_ERR_INVALID_ARG;
    if (!(p.eps >= 0.f)) return MLSTM_ERR_INVALID_ARG;
    if (dt != MLSTM_F32 && dt != MLSTM_BF16) return MLSTM_ERR_UNSUPPORTED;
    if (p.D < 8 || p.D > 512 || p.D % 8 || NHQ > 65535 || NHK > 65535) return MLSTM_ERR_UNSUPPORTED;
    if (p.tokens == 0 || NHQ + NHK == 0) return MLSTM_OK;
    const uintptr_t es = dt == MLSTM_BF16 ? 2 : 4;
    for (const Side &sd : p.side) {
        if (!sd.heads) continue;
        if (!sd.x || !sd.out || (bwd && !sd.dy)) return MLSTM_ERR_INVALID_ARG;
        if (!aligned(sd.x, es) || !aligned(sd.w, 4)) return MLSTM_ERR_INVALID_ARG;
        // the contiguous tensors follow the library's 16-byte rule
        if (bwd ? (!aligned(sd.dy, 16) || !aligned(sd.out, es)) : !aligned(sd.out, 16)) return MLSTM_ERR_INVALID_ARG;
    }
    if (p.RD && !p.inv_freq) return MLSTM_ERR_INVALID_ARG;
    if (!aligned(p.inv_freq, 4) || !aligned(p.positions, 4)) return MLSTM_ERR_INVALID_ARG;
    return MLSTM_OK;
}

Side make_side(const void *x, qknorm_strides xs, const void *dy, void *out, qknorm_strides os, const float *w, int heads)
{
    Side s = {x, dy, out, w, xs, os, heads};
    return s;
}

Params make_params(const float *inv_freq, const int *positions, int B, int S, int D, int RD, qknorm_kind kind, float eps)
{
    Params p = {};
    p.inv_freq = inv_freq;
    p.positions = positions;
    p.tokens = B > 0 && S > 0 ? (long long)B * S : 0;
    p.B = B; p.S = S; p.D = D; p.RD = RD;
    p.l2 = kind == QKNORM_L2;
    p.TT = tile_tokens(p.tokens);
    p.eps = eps;
    return p;
}

}  // namespace
}  // namespace qknorm
}  // namespace mlstm

using namespace mlstm;
using namespace mlstm::qknorm;

extern "C" {

mlstm_status qknorm_fwd(const void *q, qknorm_strides q_strides, const void *k, qknorm_strides k_strides,
                        const float *q_weight, const float *k_weight, const float *inv_freq, const int *positions,
                        mlstm_dtype dt, int B, int S, int NHQ, int NHK, int D, int RD, qknorm_kind kind, float eps,
                        int interleaved, void *q_out, void *k_out, void *stream)
{
    Params p = make_params(inv_freq, positions, B, S, D, RD, kind, eps);
    const qknorm_strides none = {0, 0, 0};
    p.side[0] = make_side(q, q_strides, nullptr, q_out, none, q_weight, NHQ);
    p.side[1] = make_side(k, k_strides, nullptr, k_out, none, k_weight, NHK);
    const mlstm_status st = check(p, dt, NHQ, NHK, kind, false);
    if (st != MLSTM_OK || p.tokens == 0 || NHQ + NHK == 0) return st;
    const cudaError_t e = dispatch<false>(p, dt == MLSTM_BF16, interleaved != 0, cta_count(p.tokens),
                                          static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MLSTM_OK : MLSTM_ERR_CUDA;
}

size_t qknorm_bwd_workspace_size(int B, int S, int NHQ, int NHK, int D)
{
    if (B <= 0 || S <= 0 || NHQ < 0 || NHK < 0 || D < 8 || D > 512 || D % 8) return 0;
    return sizeof(float) * 2 * D * (size_t)cta_count((long long)B * S);
}

mlstm_status qknorm_bwd(const void *d_q_out, const void *d_k_out, const void *q, qknorm_strides q_strides,
                        const void *k, qknorm_strides k_strides, const float *q_weight, const float *k_weight,
                        const float *inv_freq, const int *positions, mlstm_dtype dt, int B, int S, int NHQ, int NHK,
                        int D, int RD, qknorm_kind kind, float eps, int interleaved, void *dq,
                        qknorm_strides dq_strides, void *dk, qknorm_strides dk_strides, float *dq_weight,
                        float *dk_weight, void *workspace, size_t workspace_bytes, void *stream)
{
    Params p = make_params(inv_freq, positions, B, S, D, RD, kind, eps);
    p.side[0] = make_side(q, q_strides, d_q_out, dq, dq_strides, q_weight, NHQ);
    p.side[1] = make_side(k, k_strides, d_k_out, dk, dk_strides, k_weight, NHK);
    mlstm_status st = check(p, dt, NHQ, NHK, kind, true);
    if (st != MLSTM_OK) return st;
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return MLSTM_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.tokens == 0 || NHQ + NHK == 0) {   // sums over no vectors
        cudaError_t e = cudaSuccess;
        if (dq_weight) e = cudaMemsetAsync(dq_weight, 0, sizeof(float) * D, s);
        if (dk_weight && e == cudaSuccess) e = cudaMemsetAsync(dk_weight, 0, sizeof(float) * D, s);
        return e == cudaSuccess ? MLSTM_OK : MLSTM_ERR_CUDA;
    }
    const int ctas = cta_count(p.tokens);
    if (dq_weight || dk_weight) {
        if (!workspace || workspace_bytes < sizeof(float) * 2 * D * (size_t)ctas) return MLSTM_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return MLSTM_ERR_INVALID_ARG;
        p.part = static_cast<float *>(workspace);
    }
    cudaError_t e = dispatch<true>(p, dt == MLSTM_BF16, interleaved != 0, ctas, s);
    if (e == cudaSuccess && p.part)
        e = launch_kernel(weight_sum_kernel, dim3((D + 31) / 32, 2), dim3(256), 0, s, 1, p.part, ctas, D, dq_weight,
                          dk_weight);
    return e == cudaSuccess ? MLSTM_OK : MLSTM_ERR_CUDA;
}

}  // extern "C"
