// qknorm.cu -- norms of queries and keys per head with the position rotation, forward and backward:
//   r = 1 / sqrt(mean|sum(x^2) + eps),  z = r w x,  y = z with pairs of its first RD elements rotated;
//   d = inverse rotation of dy,  xh = r x,  dw = sum of d xh,  dx = r (w d - xh mean|sum(w d xh)).
//
// Bound by HBM: every vector is read once and written once (the backward reads two).  A group of lanes
// takes a token and goes through its heads; each lane holds units of VEC + VEC elements of a vector, chosen
// so that both elements of a rotated pair sit in the same lane, and the same pairs for every head: it forms
// their cosines and sines once per token, in registers.  Nothing is exchanged but the norm's sum over the
// group, so warps run on their own and hide one another's latency.  Where there are few tokens (a decode
// step) a token's heads are dealt to several groups.  VEC is the widest vector that sizes, strides and
// pointers allow, at most four elements.
//
// What it costs beyond the bytes is instructions, registers and bytes in flight.  Packed fp32 pairs, one side per CTA,
// four vectors on their way at any time (the next is asked for as soon as one is done with) and lanes without a unit
// that go along instead of branching take the forward pass over 16384 tokens of 16 + 16 heads of 128 (bf16, 268 MB,
// cold) to 61 us (4.4 TB/s) and the backward of 4 x 4096 tokens of 16 + 4 heads (252 MB) to 71 us with the weights'
// sums (3.5 TB/s).  Loading four and then working on four took 67 and 77 us, tokens shared by a CTA with the angles in
// shared memory 74 and 126 us.
#include "common.cuh"
#include "qknorm.h"
#include "tc_common.cuh"

#include <stdint.h>

#include <algorithm>

namespace mlstm {
namespace qknorm {
namespace {

using namespace tc;   // packed fp32 pairs

constexpr int THREADS = 128;
// SPAN: VEC elements times units per lane, 4 for vectors of up to 256 (32 lanes x 2 x 4), 8 beyond.  Wider
// loads (8 bf16) with half the lanes took twice the registers and were slower for it.
// Vectors a group loads before it works on the first of them: what 32 registers hold, at most four.
template <typename T, int VEC, int SPAN, bool BWD>
constexpr int ahead()
{
    constexpr int words = SPAN * 2 / VEC * ((int)sizeof(T) * VEC < 4 ? 1 : (int)sizeof(T) * VEC / 4) * (BWD ? 2 : 1);
    return words >= 32 ? 1 : words >= 16 ? 2 : 4;
}
// CTAs an SM, for the registers that leaves each.
template <typename T, int VEC, int SPAN, bool BWD>
constexpr int resident()
{
    return SPAN == 8 ? (BWD ? 2 : 3) : BWD ? 4 : sizeof(T) == 2 && VEC == 4 ? 6 : 4;
}

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
    unsigned tokens;         // B * S
    int B, S, D, RD, l2;
    int GL, HS;              // lanes of a group; groups that share a token's heads
    float eps;
};

// VEC elements as they lie in memory, in 32-bit words (a single bf16 in the low half of one): eight bf16
// held as eight registers would cost the kernel half its warps.
template <typename T, int VEC>
struct Vec {
    static constexpr int BYTES = (int)sizeof(T) * VEC;
    uint32_t w[BYTES < 4 ? 1 : BYTES / 4];
};
template <typename T, int VEC>
MLSTM_DEVINL Vec<T, VEC> load_vec(const T *p)
{
    Vec<T, VEC> v;
    if constexpr (v.BYTES == 16) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        v.w[0] = u.x; v.w[1] = u.y; v.w[2] = u.z; v.w[3] = u.w;
    } else if constexpr (v.BYTES == 8) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        v.w[0] = u.x; v.w[1] = u.y;
    } else if constexpr (v.BYTES == 4) {
        v.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
        v.w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
    return v;
}

// A unit's 2 VEC values as VEC packed pairs of floats in the order of memory; one element and its partner
// make one pair where VEC is 1.  So a word holds a rotated pair (interleaved, or VEC 1), or two neighbours of
// the same half.
template <typename T, int VEC>
MLSTM_DEVINL void widen(const Vec<T, VEC> (&v)[2], uint64_t (&x)[VEC])
{
    if constexpr (VEC == 1) {
        if constexpr (sizeof(T) == 4) x[0] = f2_pack(__uint_as_float(v[0].w[0]), __uint_as_float(v[1].w[0]));
        else x[0] = f2_pack(__uint_as_float(v[0].w[0] << 16), __uint_as_float(v[1].w[0] << 16));
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const Vec<T, VEC> &u = v[i / (VEC / 2)];
            const int j = i % (VEC / 2);
            if constexpr (sizeof(T) == 4) x[i] = f2_pack(__uint_as_float(u.w[2 * j]), __uint_as_float(u.w[2 * j + 1]));
            else x[i] = f2_from_bf16x2(u.w[j]);
        }
    }
}
template <typename T, int VEC>
MLSTM_DEVINL void narrow(const uint64_t (&x)[VEC], Vec<T, VEC> (&v)[2])
{
    if constexpr (VEC == 1) {
        const float2 f = f2_unpack(x[0]);
        v[0].w[0] = sizeof(T) == 4 ? __float_as_uint(f.x) : bf16x2_bits(f.x, 0.f);
        v[1].w[0] = sizeof(T) == 4 ? __float_as_uint(f.y) : bf16x2_bits(f.y, 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            Vec<T, VEC> &u = v[i / (VEC / 2)];
            const int j = i % (VEC / 2);
            if constexpr (sizeof(T) == 4) {
                const float2 f = f2_unpack(x[i]);
                u.w[2 * j] = __float_as_uint(f.x);
                u.w[2 * j + 1] = __float_as_uint(f.y);
            } else {
                u.w[j] = f2_to_bf16x2(x[i]);
            }
        }
    }
}
template <typename T, int VEC>
MLSTM_DEVINL void store_vec(T *p, const Vec<T, VEC> &v)
{
    if constexpr (v.BYTES == 16) *reinterpret_cast<uint4 *>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    else if constexpr (v.BYTES == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(v.w[0], v.w[1]);
    else if constexpr (v.BYTES == 4) *reinterpret_cast<uint32_t *>(p) = v.w[0];
    else *reinterpret_cast<uint16_t *>(p) = (uint16_t)v.w[0];
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

// Rotates a unit's VEC pairs by cs (cosines and sines); sign -1 turns back.
template <int VEC, bool INTER>
MLSTM_DEVINL void rotate(uint64_t (&x)[VEC], const float2 (&cs)[VEC], float sign)
{
    if constexpr (INTER || VEC == 1) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 v = f2_unpack(x[e]);
            const float s = sign * cs[e].y;
            x[e] = f2_fma(x[e], f2_pack(cs[e].x, cs[e].x), f2_mul(f2_pack(v.y, v.x), f2_pack(-s, s)));
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            const uint64_t c = f2_pack(cs[2 * e].x, cs[2 * e + 1].x), a = x[e], b = x[VEC / 2 + e];
            const uint64_t s = f2_pack(sign * cs[2 * e].y, sign * cs[2 * e + 1].y);
            const uint64_t n = f2_pack(-sign * cs[2 * e].y, -sign * cs[2 * e + 1].y);
            x[e] = f2_fma(a, c, f2_mul(b, n));
            x[VEC / 2 + e] = f2_fma(b, c, f2_mul(a, s));
        }
    }
}

// A group's place: its lane, its token and what it needs of it.
template <int VEC, int SPAN>
struct Place {
    int gl, units, hs;            // units: of a vector
    unsigned b, t;
    float2 cs[SPAN / VEC][VEC];   // of the lane's pairs
};

// The cosines and sines of the lane's pairs.  The angle is formed in fp64, in turns, and brought to half a
// turn there, where an fp32 sine is accurate to its own rounding.
template <int VEC, int SPAN, bool INTER>
MLSTM_DEVINL void angles(const Params &p, unsigned tok, Place<VEC, SPAN> &g)
{
    const double pos = (double)(p.positions ? p.positions[tok] : (int)g.t);
#pragma unroll
    for (int n = 0; n < SPAN / VEC; ++n) {
        int o1, o2;
        bool turn;
        unit_offsets<VEC, INTER>(g.gl + n * p.GL, p.D, p.RD, o1, o2, turn);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float s = 0.f, c = 1.f;
            if (turn && g.gl + n * p.GL < g.units) {
                const double turns = pos * (double)p.inv_freq[(INTER ? o1 / 2 : o1) + e] * 0.15915494309189533577;
                sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
            }
            g.cs[n][e] = make_float2(c, s);
        }
    }
}

// What a lane has loaded of one vector: its units' values and, backward, the gradients of its outputs.
template <typename T, int VEC, int SPAN, bool BWD>
struct Held {
    Vec<T, VEC> x[SPAN / VEC][2], d[BWD ? SPAN / VEC : 1][2];
};

// All of a token's heads of one side.  gw: the lane's share of the weight's gradient.  `on`: the group has a token;
// a warp's groups stay together for the sums either way.  A lane without a unit goes along with the vector's last one,
// counts nothing of it and stores nothing: branches around it cost more than its arithmetic.
template <typename T, int VEC, int SPAN, bool INTER, bool BWD>
MLSTM_DEVINL void one_side(const Params &p, const Side &sd, const Place<VEC, SPAN> &g, bool on, uint64_t *gw)
{
    constexpr int NU = SPAN / VEC, AHEAD = ahead<T, VEC, SPAN, BWD>();
    uint64_t w[NU][VEC];
    bool has[NU];
    int o1[NU], o2[NU];
    bool turn[NU];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
        has[n] = g.gl + n * p.GL < g.units;
        const int u = min(g.gl + n * p.GL, g.units - 1);
        unit_offsets<VEC, INTER>(u, p.D, p.RD, o1[n], o2[n], turn[n]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int f0 = VEC == 1 ? o1[n] : e < VEC / 2 ? o1[n] + 2 * e : o2[n] + 2 * e - VEC;
            const int f1 = VEC == 1 ? o2[n] : f0 + 1;
            w[n][e] = sd.w ? f2_pack(sd.w[f0], sd.w[f1]) : f2_pack(1.f, 1.f);
        }
    }
    // one unit: its first element's offset goes into the pointers
    const int base = NU == 1 ? o1[0] : 0;
    if (NU == 1) {
        o2[0] -= base;
        o1[0] = 0;
    }
    const long long c0 = ((long long)g.b * sd.heads * p.S + g.t) * p.D + base, ch = (long long)p.S * p.D;   // contiguous tensors
    const T *x = (const T *)sd.x + g.b * sd.xs.batch + g.t * sd.xs.token + base + g.hs * sd.xs.head;
    const T *dy = (const T *)sd.dy + c0 + g.hs * ch;
    const long long oh = BWD ? sd.os.head : ch;
    T *out = (T *)sd.out + (BWD ? g.b * sd.os.batch + g.t * sd.os.token + base : c0) + g.hs * oh;
    const float inv_n = p.l2 ? 1.f : 1.f / (float)p.D;
    const long long xstep = p.HS * sd.xs.head, cstep = p.HS * ch, ostep = p.HS * oh;
    using H = Held<T, VEC, SPAN, BWD>;
    auto load = [&](H &v) {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            v.x[n][0] = load_vec<T, VEC>(x + o1[n]);
            v.x[n][1] = load_vec<T, VEC>(x + o2[n]);
            if (BWD) {
                v.d[n][0] = load_vec<T, VEC>(dy + o1[n]);
                v.d[n][1] = load_vec<T, VEC>(dy + o2[n]);
            }
        }
        x += xstep;
        if (BWD) dy += cstep;
    };
    auto work = [&](const H &v, bool live) {
        uint64_t xv[NU][VEC], d[BWD ? NU : 1][VEC], gwd[BWD ? NU : 1][VEC];   // gwd: d without the weight
        float s = 0.f, xd = 0.f;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            uint64_t s2 = 0, xd2 = 0;
            widen<T, VEC>(v.x[n], xv[n]);
            if (BWD) {
                widen<T, VEC>(v.d[n], d[n]);
                if (turn[n]) rotate<VEC, INTER>(d[n], g.cs[n], -1.f);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s2 = f2_fma(xv[n][e], xv[n][e], s2);
                if (BWD) {
                    gwd[n][e] = d[n][e];
                    d[n][e] = f2_mul(w[n][e], d[n][e]);
                    xd2 = f2_fma(d[n][e], xv[n][e], xd2);
                }
            }
            s += has[n] ? f2_unpack(s2).x + f2_unpack(s2).y : 0.f;
            if (BWD) xd += has[n] ? f2_unpack(xd2).x + f2_unpack(xd2).y : 0.f;
        }
        if (!BWD && NU == 1 && !INTER) {   // the shortest body: 61 us, 63 with the steps unrolled
            for (int o = p.GL / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                if (o < p.GL) {
                    s += __shfl_xor_sync(0xffffffffu, s, o);
                    if (BWD) xd += __shfl_xor_sync(0xffffffffu, xd, o);
                }
        }
        const float r = rsqrtf(fmaf(s, inv_n, p.eps));
        // dx = r (w d - (r x) mean|sum(w d (r x))): with r x, whose size is about one, and never r^3, which leaves
        // fp32 where r itself is far inside it
        const float back = BWD ? -r * (r * xd * inv_n) : 0.f;
        const uint64_t r2 = f2_pack(r, r), back2 = f2_pack(back, back);
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            if (!has[n] || !live) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if (BWD) {
                    const uint64_t xh = f2_mul(r2, xv[n][e]);
                    gw[n * VEC + e] = f2_fma(gwd[n][e], xh, gw[n * VEC + e]);
                    xv[n][e] = f2_fma(r2, d[n][e], f2_mul(back2, xh));
                } else {
                    xv[n][e] = f2_mul(xv[n][e], f2_mul(r2, w[n][e]));
                }
            }
            if (!BWD && turn[n]) rotate<VEC, INTER>(xv[n], g.cs[n], 1.f);
            Vec<T, VEC> y[2];
            narrow<T, VEC>(xv[n], y);
            store_vec<T, VEC>(out + o1[n], y[0]);
            store_vec<T, VEC>(out + o2[n], y[1]);
        }
        out += ostep;
    };
    // the next vectors are asked for as soon as one is done with: a group always waits for the oldest of AHEAD
    const int rounds = (sd.heads + p.HS * AHEAD - 1) / (p.HS * AHEAD);   // the same for every group of the warp
    int left = on ? (sd.heads - g.hs + p.HS - 1) / p.HS : 0;
    H v[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        if (k < left) load(v[k]);
#pragma unroll 1
    for (int round = 0; round < rounds; ++round) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            work(v[k], k < left);
            if (k + AHEAD < left) load(v[k]);
        }
        left -= AHEAD;
    }
}

// blockIdx.y: queries or keys.
template <typename T, int VEC, int SPAN, bool INTER, bool BWD>
__global__ void __launch_bounds__(THREADS, (resident<T, VEC, SPAN, BWD>()))
qknorm_kernel(const __grid_constant__ Params p)
{
    extern __shared__ __align__(16) float red[];   // backward: [groups][D]
    const int tid = threadIdx.x, grp = tid / p.GL, groups = THREADS / p.GL;
    const Side &sd = p.side[blockIdx.y];
    Place<VEC, SPAN> g;
    g.gl = tid % p.GL;
    griddep_wait();
    griddep_launch_dependents();
    uint64_t gw[BWD ? SPAN : 1] = {};
    const unsigned long long items = (unsigned long long)p.tokens * p.HS, step = (unsigned long long)gridDim.x * groups;
    // whole warps stay together for the sums: a group without an item goes along
#pragma unroll 1
    for (unsigned long long i0 = (unsigned long long)blockIdx.x * groups; i0 < items; i0 += step) {
        const unsigned long long i = i0 + grp;
        const bool on = i < items;
        const unsigned tok = on ? (unsigned)(p.HS == 1 ? i : i / p.HS) : 0u;
        g.units = p.D / 2 / VEC;
        g.hs = on && p.HS > 1 ? (int)(i - (unsigned long long)tok * p.HS) : 0;
        g.b = tok / (unsigned)p.S;
        g.t = tok - g.b * (unsigned)p.S;
        if (p.RD) angles<VEC, SPAN, INTER>(p, tok, g);
        one_side<T, VEC, SPAN, INTER, BWD>(p, sd, g, on, gw);
    }
    if (BWD && p.part) {   // the groups' shares of the weight's gradient, added in order
        const int units = p.D / 2 / VEC;
#pragma unroll
        for (int n = 0; n < SPAN / VEC; ++n) {
            const int u = g.gl + n * p.GL;
            if (u >= units) continue;
            int o1, o2;
            bool turn;
            unit_offsets<VEC, INTER>(u, p.D, p.RD, o1, o2, turn);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float2 f = f2_unpack(gw[BWD ? n * VEC + e : 0]);
                const int f0 = VEC == 1 ? o1 : e < VEC / 2 ? o1 + 2 * e : o2 + 2 * e - VEC;
                red[grp * p.D + f0] = f.x;
                red[grp * p.D + (VEC == 1 ? o2 : f0 + 1)] = f.y;
            }
        }
        __syncthreads();
        for (int d = tid; d < p.D; d += THREADS) {
            float s = 0.f;
            for (int i = 0; i < groups; ++i) s += red[i * p.D + d];
            p.part[((size_t)blockIdx.x * 2 + blockIdx.y) * p.D + d] = s;
        }
    }
}

// dw[side][d] = sum over the CTAs' partials, 32 columns a CTA, 32 rows of it side by side.
__global__ void __launch_bounds__(1024)
weight_sum_kernel(const float *__restrict__ part, int n, int D, float *dwq, float *dwk)
{
    __shared__ float red[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, sdi = blockIdx.y, d = blockIdx.x * 32 + tx;
    griddep_wait();
    griddep_launch_dependents();
    float s = 0.f;
    if (d < D)
#pragma unroll 8
        for (int i = ty; i < n; i += 32) s += part[((size_t)i * 2 + sdi) * D + d];
    red[ty][tx] = s;
    __syncthreads();
    float *dw = sdi ? dwk : dwq;
    s = warp_sum(red[tx][ty]);   // column ty of the tile
    const int col = blockIdx.x * 32 + ty;
    if (tx == 0 && col < D && dw) dw[col] = s;
}

// CTAs of a backward launch at most: every one leaves partial sums of the weights' gradients.
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
    for (int vec = 4; vec > 1; vec /= 2)
        if (fits(vec)) return vec;
    return 1;
}

template <typename T, int VEC, int SPAN, bool INTER, bool BWD>
cudaError_t launch(Params p, int *ctas, cudaStream_t stream)
{
    const int units = p.D / 2 / VEC, heads = std::max(p.side[0].heads, p.side[1].heads);
    p.GL = 1;
    while (p.GL < 32 && p.GL * (SPAN / VEC) < units) p.GL *= 2;
    const int groups = THREADS / p.GL;
    // a token's heads go to as many groups as it takes to fill the GPU's threads once
    p.HS = (int)std::min<long long>(heads, std::max<long long>(1, 148ll * 1024 / p.GL / p.tokens));
    const unsigned long long need = ((unsigned long long)p.tokens * p.HS + groups - 1) / groups;
    *ctas = (int)std::min<unsigned long long>(need, BWD ? MAX_CTAS : 1ull << 30);
    const size_t smem = BWD && p.part ? sizeof(float) * groups * p.D : 0;
    return launch_kernel(qknorm_kernel<T, VEC, SPAN, INTER, BWD>, dim3((unsigned)*ctas, 2), dim3(THREADS), smem, stream, 1, p);
}

template <typename T, int VEC, bool BWD>
cudaError_t launch_vec(const Params &p, bool inter, int *ctas, cudaStream_t stream)
{
    if (p.D <= 256) return inter ? launch<T, VEC, 4, true, BWD>(p, ctas, stream) : launch<T, VEC, 4, false, BWD>(p, ctas, stream);
    return inter ? launch<T, VEC, 8, true, BWD>(p, ctas, stream) : launch<T, VEC, 8, false, BWD>(p, ctas, stream);
}

template <typename T, bool BWD>
cudaError_t dispatch(const Params &p, bool inter, int *ctas, cudaStream_t stream)
{
    switch (vector_width(p, (int)sizeof(T), inter, BWD)) {
    case 4: return launch_vec<T, 4, BWD>(p, inter, ctas, stream);
    case 2: return launch_vec<T, 2, BWD>(p, inter, ctas, stream);
    default: return launch_vec<T, 1, BWD>(p, inter, ctas, stream);
    }
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

mlstm_status check(const Params &p, mlstm_dtype dt, int NHQ, int NHK, qknorm_kind kind, bool bwd)
{
    if (p.B < 0 || p.S < 0 || NHQ < 0 || NHK < 0 || p.RD < 0 || p.RD > p.D || p.RD % 2) return MLSTM_ERR_INVALID_ARG;
    if (kind != QKNORM_RMS && kind != QKNORM_L2) return MLSTM_ERR_INVALID_ARG;
    if (!(p.eps >= 0.f)) return MLSTM_ERR_INVALID_ARG;
    if (dt != MLSTM_F32 && dt != MLSTM_BF16) return MLSTM_ERR_UNSUPPORTED;
    if (p.D < 8 || p.D > 512 || p.D % 8 || NHQ > 4096 || NHK > 4096) return MLSTM_ERR_UNSUPPORTED;
    if ((long long)p.B * p.S > (1ll << 31) - 1) return MLSTM_ERR_UNSUPPORTED;
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
    Side s = {x, dy, out, heads ? w : nullptr, xs, os, heads};   // without heads nothing of a side is read
    return s;
}

Params make_params(const float *inv_freq, const int *positions, int B, int S, int D, int RD, qknorm_kind kind, float eps)
{
    Params p = {};
    p.inv_freq = inv_freq;
    p.positions = positions;
    p.tokens = B > 0 && S > 0 ? (unsigned)((long long)B * S) : 0u;
    p.B = B; p.S = S; p.D = D; p.RD = RD;
    p.l2 = kind == QKNORM_L2;
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
    int ctas = 0;
    const cudaError_t e = dt == MLSTM_BF16
        ? dispatch<__nv_bfloat16, false>(p, interleaved != 0, &ctas, static_cast<cudaStream_t>(stream))
        : dispatch<float, false>(p, interleaved != 0, &ctas, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MLSTM_OK : MLSTM_ERR_CUDA;
}

size_t qknorm_bwd_workspace_size(int B, int S, int NHQ, int NHK, int D)
{
    if (B <= 0 || S <= 0 || NHQ < 0 || NHK < 0 || D < 8 || D > 512 || D % 8) return 0;
    return sizeof(float) * 2 * D * (size_t)MAX_CTAS;
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
    int ctas = 0;
    if (dq_weight || dk_weight) {
        if (!workspace || workspace_bytes < sizeof(float) * 2 * D * (size_t)MAX_CTAS) return MLSTM_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return MLSTM_ERR_INVALID_ARG;
        p.part = static_cast<float *>(workspace);
    }
    cudaError_t e = dt == MLSTM_BF16 ? dispatch<__nv_bfloat16, true>(p, interleaved != 0, &ctas, s)
                                     : dispatch<float, true>(p, interleaved != 0, &ctas, s);
    if (e == cudaSuccess && p.part)
        e = launch_kernel(weight_sum_kernel, dim3((D + 31) / 32, 2), dim3(1024), 0, s, 1, p.part, ctas, D, dq_weight,
                          dk_weight);
    return e == cudaSuccess ? MLSTM_OK : MLSTM_ERR_CUDA;
}

}  // extern "C"
