// gdelta_grad_tc.cu -- the gated delta rule's gradients of a chunk on tcgen05 (bf16 inputs, see
// gdelta_simt.cu for the formulas): dq, dk, dg and dbeta from the states S at the chunk's start, their
// gradients dS' at its end, E and dV, which the walks left in fp32.
//
//   HX = [dO; dV] E^T     Z = [dO; dV] S^T     W = E dS'^T       reduction over the value columns
//   D += [dP; dA + dA^T] K + [0; dP^T] Q                         reduction over the tokens, all value heads
//   dQ = scale e^a Z_dO + D,  dK = -e^a Z_dV + beta e^{a_64 - a} W + D
//
// dg and dbeta are fp32 outputs, so HX, Z and W take their fp32 operands as three bf16 parts (all 24
// bits) and keep the six products of parts above 2^-24; D only reaches the bf16 dq and dk: two parts.
//
// A persistent CTA takes chunks of a key head one after the other, each over its value heads.  64 value
// columns at a time its 256 worker threads bring the operands from global memory into registers, split them and
// store the parts as swizzled tiles; a ninth warp's thread issues the MMAs.  Z needs [dO; dV] and S, HX and W
// need E and dS' too, so a stage's first two operands are split while the stage before still runs W, the other
// two while Z runs.  TMEM lane = token (dO's rows, dq in lanes 0..63; dV's rows, dk in 64..127): a thread keeps
// its row's 64 columns of dq or dk in registers across the heads.  dP^T and dA^T are the same tiles as dP and dA,
// read MN-major.  Per chunk and value head of 128 x 128: 263 KB, most of it the fp32 states, E and dV, and 168 MMAs.
// 4096 of them take 461 us (2.3 TB/s): a stage's splitting and its MMAs overlap only as far as one set of operands in
// shared memory lets them.
#include "gdelta_prep.cuh"
#include "tc_common.cuh"
#include "tc_fwd.h"

#include <algorithm>
#include <type_traits>

namespace mlstm {
namespace gdelta {
namespace {

using namespace tc;

constexpr int WORKERS = 256, THREADS = WORKERS + 128;   // whole warpgroups, for the register split
constexpr int LDM = 65;                          // row stride of the 64 x 64 fp32 matrices (any row or column at once)
constexpr uint32_t KQ = 0;                       // [2 blocks][128 rows][64]: K over Q
constexpr uint32_t TA = 32768;                   // [dO; dV] values, [0; dV] residues, their residues: 16 KB each
constexpr uint32_t TE = TA + 3 * 16384;          // E's three parts, 64 rows, 8 KB each
constexpr uint32_t TS = TE + 3 * 8192;           // S's three parts, 128 rows, 16 KB each
constexpr uint32_t TD = TS + 3 * 16384;          // dS' likewise
// after the products over the value columns, over TA .. TD:
constexpr uint32_t ZT = TA;                      // 64 rows of zeros
constexpr uint32_t A1 = ZT + 8192;               // [dP; dA] as two parts, 128 rows, 16 KB each
constexpr uint32_t MZ = A1 + 32768;              // fp32 [64][LDM]: scale P * dO E^T, later the pairs' prefix sums
constexpr uint32_t MH = MZ + 64 * LDM * 4;       // -KK * H
constexpr uint32_t GA = TD + 3 * 16384;          // [64] float4: cumulative log2 gate (value, residue), beta, e^a
constexpr uint32_t GO = GA + 1024;               // [64] e^{a_64 - a}
constexpr uint32_t ZI = GO + 256;                // [2][2][64] shares of z_in by column half and row kind
constexpr uint32_t ZO = ZI + 1024;               // [2][64] z_out by column half
constexpr uint32_t SD = ZO + 512;                // [8] shares of <S, dS'>
constexpr uint32_t BAR = SD + 32;
constexpr uint32_t NBAR = 9;
constexpr uint32_t TOTAL = BAR + NBAR * 8 + 16 + 1024;
static_assert(MH + 64 * LDM * 4 <= GA, "the pairs' matrices fit over the operands");
static_assert(TOTAL <= 232448, "one CTA's shared memory");

// TMEM columns
constexpr uint32_t CZ = 0, CW = 128, CH_ = 256, CD = 320, CHS = 448;   // CHS: HX's products of the smaller parts
// An MMA cuts its sum off where fp32 ends, always towards zero, and every one of them adds to the error: HX keeps
// its largest products apart from the others, and Z and W go to the threads' registers, whose additions round,
// after SUM stages.  After every stage, 128 value columns take 535 us where they take 470, for a dg 8e-7 off fp64
// either way; never, 256 columns are 1.4e-6 off.
constexpr int SUM = 2;

struct Params {
    const __nv_bfloat16 *d_o;
    const float *beta;
    const int *lengths;
    __nv_bfloat16 *dq, *dk;
    float *dg, *dbeta;
    int B, NH, NHV, S, DK, DV;
    float scale;
    Workspace w;
};

// Eight values as three bf16 parts (top, middle and last 8 significant bits), 16 bytes each.
MLSTM_DEVINL void split3(const float4 &x, const float4 &y, uint4 (&p)[3])
{
    float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        uint32_t *o = &p[q].x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t u0 = __float_as_uint(v[2 * e]), u1 = __float_as_uint(v[2 * e + 1]);
            o[e] = __byte_perm(u0, u1, 0x7632);
            if (q < 2) {
                v[2 * e] -= __uint_as_float(u0 & 0xffff0000u);
                v[2 * e + 1] -= __uint_as_float(u1 & 0xffff0000u);
            }
        }
    }
}

// 32 values of a row as two bf16 parts (value and rounding residue) into a tile of 128 rows; the residues
// 16 KB behind.
MLSTM_DEVINL void store2(uint8_t *tile, uint32_t row, uint32_t j0, const float (&x)[32])
{
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x0 = x[c * 8 + 2 * e], x1 = x[c * 8 + 2 * e + 1];
            h[e] = pack_bf16(x0, x1);
            l[e] = pack_bf16(x0 - __uint_as_float(h[e] << 16), x1 - __uint_as_float(h[e] & 0xffff0000u));
        }
        const uint32_t off = sw128_chunk(row, j0 + c, 128);
        *reinterpret_cast<uint4 *>(tile + off) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(tile + 16384 + off) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

// N accumulator columns at a time: between two stages, with their operands in registers, or behind the last
using Few = std::integral_constant<int, 16>;
using All = std::integral_constant<int, 32>;

template <int N>
MLSTM_DEVINL void ld(uint32_t taddr, float (&x)[N])
{
    uint32_t r[N];
    if constexpr (N == 16) tmem_ld16(taddr, r);
    else tmem_ld32(taddr, r);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __uint_as_float(r[i]);
}

template <bool LONG>   // more than SUM stages
__global__ void __launch_bounds__(THREADS, 1)
grad_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const Params p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float4 *ga = reinterpret_cast<float4 *>(smem + GA);
    float *go = reinterpret_cast<float *>(smem + GO), *zi = reinterpret_cast<float *>(smem + ZI);
    float *zo = reinterpret_cast<float *>(smem + ZO), *sds = reinterpret_cast<float *>(smem + SD);
    float *mz = reinterpret_cast<float *>(smem + MZ), *mh = reinterpret_cast<float *>(smem + MH);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + BAR);
    // written by the workers: [dO; dV] and S, E, dS', the pairs' tiles, K and Q no longer read; by the MMAs:
    // Z done, HX and W done, D done; by the copies: K and Q
    uint64_t *as_ready = bars, *e_ready = bars + 1, *d_ready = bars + 2, *t_ready = bars + 3, *kq_free = bars + 4,
             *z_done = bars + 5, *w_done = bars + 6, *t_done = bars + 7, *kq_full = bars + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + NBAR), *abort_flag = tmem_slot + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = p.NHV / p.NH, nst = (p.DV + 63) / 64;
    const int items = p.w.NC * p.B * p.NH;   // (chunk, key head), a key head's chunks side by side
    const Workspace &w = p.w;
    WaitCtx wc{abort_flag, w.status};
    if (tid == 0) {
        for (int i = 0; i < 5; ++i) mbar_init(&bars[i], WORKERS / 32);
        for (int i = 5; i < (int)NBAR; ++i) mbar_init(&bars[i], 1);
        *abort_flag = 0u;
        fence_barrier_init();
        tma_prefetch(&tm_q);
        tma_prefetch(&tm_k);
    }
    if (warp == 8) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    griddep_launch_dependents();
    // A wait that gives up sets the abort flag, after which every wait returns at once: all roles run through to
    // the end, with outputs that the status word declares undefined.
    auto live = [&](int item, int &c, int &bh) {
        c = item % w.NC;
        bh = item / w.NC;
        return max(0, min(min(CH, p.S - c * CH), live_tokens(p.lengths, bh / p.NH, p.S) - c * CH));
    };

    // registers: launched with 168 a thread; 2 x 216 + 72 = 3 x 168
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8 && lane == 0) {
            constexpr uint32_t IDN = idesc_bf16(128, 128, 0, 0), IDH = idesc_bf16(128, 64, 0, 0);
            constexpr uint32_t IDD = idesc_bf16(128, 128, 0, 1), IDT = idesc_bf16(128, 128, 1, 1);
            const uint32_t sm = smem_u32(smem);
            uint64_t da = smem_desc(sm + TA, 16, 1024), de = smem_desc(sm + TE, 16, 1024);
            uint64_t ds = smem_desc(sm + TS, 16, 1024), dd = smem_desc(sm + TD, 16, 1024);
            uint64_t a1 = smem_desc(sm + A1, 16, 1024), bk = smem_desc(sm + KQ, 16384, 1024);
            // dP^T and dA^T in lanes 64..127: zeros as the first 64 M, the tile as the others
            uint64_t pt = smem_desc(sm + ZT, A1 - ZT, 1024), pt2 = smem_desc(sm + ZT, A1 + 16384 - ZT, 1024);
            uint64_t at = smem_desc(sm + ZT, A1 + 8192 - ZT, 1024), at2 = smem_desc(sm + ZT, A1 + 24576 - ZT, 1024);
            // the six products of parts, A's and B's, smallest first: the accumulation cuts bits off at the sum's size
            constexpr int PA[6] = {0, 2, 1, 0, 1, 0}, PB[6] = {2, 0, 1, 1, 0, 0};
            uint32_t n = 0, hd = 0, it = 0;   // stages, heads and items so far
            for (int item = blockIdx.x; item < items; item += gridDim.x) {
                int c, bh;
                if (live(item, c, bh) == 0) continue;
                if (it > 0) mbar_wait(kq_free, (it - 1) & 1u, wc);
                mbar_arrive_expect_tx(kq_full, 32768);
                for (int kb = 0; kb < 2; ++kb) {
                    tma_load_3d(smem + KQ + kb * 16384, &tm_k, 64 * kb, c * CH, bh, kq_full);
                    tma_load_3d(smem + KQ + kb * 16384 + 8192, &tm_q, 64 * kb, c * CH, bh, kq_full);
                }
                ++it;
                for (int h = 0; h < group; ++h, ++hd) {
                    for (int s = 0; s < nst; ++s, ++n) {
                        // opaque, or every descriptor of the loop is kept in registers across it
                        asm volatile("" : "+l"(da), "+l"(de), "+l"(ds), "+l"(dd));
                        mbar_wait(as_ready, n & 1u, wc);
                        tc_fence_after();
#pragma unroll
                        for (int q = 0; q < 6; ++q)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_ss(tmem + CZ, da + (uint64_t)(PA[q] * 1024 + k * 2), ds + (uint64_t)(PB[q] * 1024 + k * 2), IDN,
                                       s % SUM + q + k > 0);
                        mbar_wait(e_ready, n & 1u, wc);
                        tc_fence_after();
#pragma unroll
                        for (int q = 0; q < 6; ++q)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_ss(tmem + (q < 5 ? CHS : CH_), da + (uint64_t)(PA[q] * 1024 + k * 2), de + (uint64_t)(PB[q] * 512 + k * 2), IDH,
                                       s + q % 5 + k > 0);
                        mma_commit(z_done);   // and HX: [dO; dV] and S are free
                        mbar_wait(d_ready, n & 1u, wc);
                        tc_fence_after();   // W goes over sums that the workers have just read
                        // E in rows 64..127; the rows in front of a part read what lies before it, into lanes nothing uses
#pragma unroll
                        for (int q = 0; q < 6; ++q)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_ss(tmem + CW, de + (uint64_t)(PA[q] * 512 - 512 + k * 2), dd + (uint64_t)(PB[q] * 1024 + k * 2), IDN,
                                       s % SUM + q + k > 0);
                        mma_commit(w_done);
                    }
                    asm volatile("" : "+l"(a1), "+l"(bk), "+l"(pt), "+l"(pt2), "+l"(at), "+l"(at2));
                    mbar_wait(t_ready, hd & 1u, wc);
                    tc_fence_after();
#pragma unroll
                    for (int q = 1; q >= 0; --q)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            mma_ss(tmem + CD, a1 + (uint64_t)(q * 1024 + k * 2), bk + (uint64_t)(k * 128), IDD, h > 0 || q < 1 || k > 0);
                            mma_ss(tmem + CD, (q ? pt2 : pt) + (uint64_t)(k * 128), bk + (uint64_t)(512 + k * 128), IDT, 1);
                            mma_ss(tmem + CD, (q ? at2 : at) + (uint64_t)(k * 128), bk + (uint64_t)(k * 128), IDT, 1);
                        }
                    mma_commit(t_done);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int quad = warp & 3, half = warp >> 2;
        const int row = quad * 32 + lane, t = row & 63;     // TMEM lane; token
        const bool top = quad < 2;                          // dO's rows and dq, else dV's and dk
        const uint32_t tl = tmem_addr(tmem, quad * 32, 0);
        const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        // a thread's units of 8 values: row u0 + 32 k, columns c8 .. c8 + 7 of the 64
        const int u0 = tid >> 3, c8 = (tid & 7) * 8;
        uint32_t n = 0, hd = 0, it = 0;
        auto arrive = [&](uint64_t *bar) {   // what this thread wrote to shared memory or read of TMEM is done with
            fence_proxy_async();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        auto sync = [] { named_sync(1, WORKERS); };
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            int c, bh;
            const int len = live(item, c, bh), full = min(CH, p.S - c * CH), b = bh / p.NH;
            const size_t row0 = (size_t)bh * p.S + c * CH;
            for (int i = tid; i < (full - len) * (p.DK / 8); i += WORKERS) {   // padding
                const size_t at = (row0 + len) * p.DK + (size_t)i * 8;
                *reinterpret_cast<uint4 *>(p.dq + at) = zero;
                *reinterpret_cast<uint4 *>(p.dk + at) = zero;
            }
            for (int h = 0; h < group; ++h)
                if (tid < full - len) {
                    const size_t gt = (size_t)(b * p.NHV + (bh % p.NH) * group + h) * p.S + c * CH + len + tid;
                    p.dg[gt] = 0.f;
                    p.dbeta[gt] = 0.f;
                }
            if (len == 0) continue;
            uint64_t acc[32];                                   // 64 columns of the thread's row of dq or dk
#pragma unroll
            for (int e = 0; e < 32; ++e) acc[e] = 0;
            for (int h = 0; h < group; ++h, ++hd) {
                const int bhv = b * p.NHV + (bh % p.NH) * group + h;
                const size_t ch = (size_t)bhv * w.NC + c, vrow = (size_t)bhv * p.S + c * CH;
                const float *Sg = w.SC + ch * p.DK * p.DV, *Dg = w.DSC + ch * p.DK * p.DV;
                const float *Eg = w.E + ch * 64 * p.DV, *Vg = w.DV + ch * 64 * p.DV;
                const __nv_bfloat16 *Og = p.d_o + vrow * p.DV;
                uint4 ro[2];
                float4 rv[2][2], re[2][2], rs[4][2], rd[4][2];
                auto load_o = [&](int v0) {
                    const int col = v0 + c8;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        ro[k] = col < p.DV && u0 + 32 * k < len ? *reinterpret_cast<const uint4 *>(Og + (size_t)(u0 + 32 * k) * p.DV + col) : zero;
                };
                auto load_tok = [&](const float *src, int v0, float4 (&x)[2][2]) {
                    const int col = v0 + c8;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            x[k][e] = col < p.DV ? *reinterpret_cast<const float4 *>(src + (size_t)(u0 + 32 * k) * p.DV + col + 4 * e) : zero4;
                };
                auto load_state = [&](const float *src, int v0, float4 (&x)[4][2]) {
                    const int col = v0 + c8;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            x[k][e] = col < p.DV && u0 + 32 * k < p.DK
                                          ? *reinterpret_cast<const float4 *>(src + (size_t)(u0 + 32 * k) * p.DV + col + 4 * e) : zero4;
                };
                auto put = [&](uint32_t tile, uint32_t step, int r, int rows, const float4 (&x)[2]) {
                    uint4 q[3];
                    split3(x[0], x[1], q);
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        *reinterpret_cast<uint4 *>(smem + tile + e * step + sw128_chunk(r, c8 / 8, rows)) = q[e];
                };
                load_o(0);
                load_tok(Vg, 0, rv);
                load_state(Sg, 0, rs);
                float2 gx = make_float2(0.f, 0.f), gl = gx;
                float bt = 0.f;
                if (tid < 64) {
                    gx = w.A[ch * 64 + tid];
                    gl = w.A[ch * 64 + 63];
                    bt = tid < len ? p.beta[vrow + tid] : 0.f;
                }
                if (hd > 0) mbar_wait(t_done, (hd - 1) & 1u, wc);   // the pairs' tiles lie over the operands,
                sync();                                             // and so do the sums' matrices
                if (tid < 64) {
                    ga[tid] = make_float4(gx.x, gx.y, bt, exp2f(gx.x + gx.y));
                    go[tid] = exp2f((gl.x - gx.x) + (gl.y - gx.y));
                }
                // SUM stages' Z and W, 64 columns of the thread's row: onto dq or dk, and their products with q or k.
                float zin = 0.f, zout = 0.f;
                auto fold = [&](auto width, uint32_t tcol, float f, float &sum) {
                    constexpr int N = decltype(width)::value;
#pragma unroll
                    for (int cc = 0; cc < 64 / N; ++cc) {
                        float z[N];
                        ld<N>(tl + tcol + half * 64 + cc * N, z);
#pragma unroll
                        for (int j = 0; j < N / 8; ++j) {   // row t of K (dk) or Q (dq)
                            const uint4 u = *reinterpret_cast<const uint4 *>(
                                smem + KQ + sw128_chunk(top ? 64 + t : t, half * 8 + cc * (N / 8) + j, 128));
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float z0 = z[8 * j + 2 * e], z1 = z[8 * j + 2 * e + 1];
                                const float2 x = unpack_bf16((&u.x)[e]);
                                sum = fmaf(z0, x.x, sum);
                                sum = fmaf(z1, x.y, sum);
                                uint64_t &a = acc[cc * (N / 2) + 4 * j + e];
                                a = f2_fma(f2_pack(f, f), f2_pack(z0, z1), a);
                            }
                        }
                    }
                };
                auto fz = [&] { return top ? p.scale * ga[t].w : -ga[t].w; };
                auto take_kq = [&] {   // K and Q: their padding rows would meet zeros, which NaN survives
                    mbar_wait(kq_full, it & 1u, wc);
                    ++it;
                    if (t >= len) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4 *>(smem + KQ + sw128_chunk(row, half * 8 + j, 128)) = zero;
                    }
                };
                float sd = 0.f;
                for (int s = 0; s < nst; ++s, ++n) {
                    if (s > 0) {
                        mbar_wait(z_done, (n - 1) & 1u, wc);
                        if (LONG && s % SUM == 0) {
                            if (h == 0 && s == SUM) take_kq();
                            tc_fence_after();
                            fold(Few{}, CZ, fz(), zin);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int r = u0 + 32 * k;
                        const uint32_t up = sw128_chunk(r, c8 / 8, 128);
                        *reinterpret_cast<uint4 *>(smem + TA + up) = ro[k];
                        *reinterpret_cast<uint4 *>(smem + TA + 16384 + up) = zero;
                        *reinterpret_cast<uint4 *>(smem + TA + 32768 + up) = zero;
                        put(TA, 16384, 64 + r, 128, rv[k]);
                    }
                    load_tok(Eg, s * 64, re);
#pragma unroll
                    for (int k = 0; k < 4; ++k) put(TS, 16384, u0 + 32 * k, 128, rs[k]);
                    load_state(Dg, s * 64, rd);
                    arrive(as_ready);
                    if (s > 0) {
                        mbar_wait(w_done, (n - 1) & 1u, wc);
                        if (LONG && s % SUM == 0 && !top) {
                            tc_fence_after();
                            fold(Few{}, CW, go[t] * ga[t].z, zout);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) put(TE, 8192, u0 + 32 * k, 64, re[k]);
                    arrive(e_ready);
                    if (s + 1 < nst) {
                        load_o((s + 1) * 64);
                        load_tok(Vg, (s + 1) * 64, rv);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            sd += (rs[k][e].x * rd[k][e].x + rs[k][e].y * rd[k][e].y) + (rs[k][e].z * rd[k][e].z + rs[k][e].w * rd[k][e].w);
                        put(TD, 16384, u0 + 32 * k, 128, rd[k]);
                    }
                    if (s + 1 < nst) load_state(Sg, (s + 1) * 64, rs);
                    arrive(d_ready);
                }
                sd = warp_sum(sd);
                if (lane == 0) sds[warp] = sd;
                if (h == 0 && (!LONG || nst <= SUM)) take_kq();
                // P's or KK's entries of the thread's row, asked for while the last products run; and the next
                // head's operands, or the next chunk's, to L2
                const int j0 = 32 * half;
                const float *src = (top ? w.P : w.KK) + ch * 4096 + t * 64 + j0;
                float pk[32];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 x = *reinterpret_cast<const float4 *>(src + 4 * e);
                    pk[4 * e] = x.x; pk[4 * e + 1] = x.y; pk[4 * e + 2] = x.z; pk[4 * e + 3] = x.w;
                }
                {
                    int nbhv = bhv + 1, nc = c;
                    bool more = h + 1 < group;
                    if (!more && item + (int)gridDim.x < items) {
                        int nbh;
                        more = live(item + gridDim.x, nc, nbh) > 0;
                        nbhv = nbh / p.NH * p.NHV + (nbh % p.NH) * group;
                    }
                    if (more) {
                        const size_t nch = (size_t)nbhv * w.NC + nc;
                        const int lines = p.DV / 32, half_lines = (p.DV + 63) / 64;   // of 128 bytes a row
                        for (int i = tid; i < p.DK * lines; i += WORKERS) {
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(w.SC + nch * p.DK * p.DV + (size_t)i * 32));
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(w.DSC + nch * p.DK * p.DV + (size_t)i * 32));
                        }
                        for (int i = tid; i < 64 * lines; i += WORKERS) {
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(w.E + nch * 64 * p.DV + (size_t)i * 32));
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(w.DV + nch * 64 * p.DV + (size_t)i * 32));
                        }
                        const size_t nv = (size_t)nbhv * p.S + nc * CH;
                        for (int i = tid; i < min(CH, p.S - nc * CH) * half_lines; i += WORKERS)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.d_o + (nv + i / half_lines) * p.DV + (i % half_lines) * 64));
                        if (tid < 128) {
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(w.P + nch * 4096 + tid * 32));
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(w.KK + nch * 4096 + tid * 32));
                        }
                    }
                }
                mbar_wait(z_done, (n - 1) & 1u, wc);
                mbar_wait(w_done, (n - 1) & 1u, wc);
                tc_fence_after();
                fold(All{}, CZ, fz(), zin);
                if (!top) fold(All{}, CW, go[t] * ga[t].z, zout);
                zi[(half * 2 + (top ? 0 : 1)) * 64 + t] = t < len ? fz() * zin : 0.f;
                if (!top) zo[half * 64 + t] = t < len ? go[t] * zout : 0.f;
                const float4 gt = ga[t];
                // the pairs: row t, columns j0 .. j0 + 31.  The operands' tiles are no longer read
                {
                    float x[32];
                    {
                        uint32_t r0[32], r1[32];
                        tmem_ld32(tl + CH_ + j0, r0);
                        tmem_ld32(tl + CHS + j0, r1);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(r0[e]) + __uint_as_float(r1[e]);
                    }
                    float *m1 = (top ? mz : mh) + t * LDM + j0;
                    const float f = top ? p.scale : -1.f;
                    const int lim = top ? t : t - 1;   // P's columns j <= t, KK's j < t
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int j = j0 + e;
                        const float4 gj = ga[j];
                        const bool on = j <= lim;
                        const float dif = on ? (gt.x - gj.x) + (gt.y - gj.y) : 0.f, v = on ? f * x[e] : 0.f;
                        m1[e] = pk[e] * v;
                        x[e] = exp2f(dif) * (gj.z * v);
                    }
                    store2(smem + A1, row, j0 / 8, x);
                    *reinterpret_cast<uint4 *>(smem + ZT + tid * 32) = zero;
                    *reinterpret_cast<uint4 *>(smem + ZT + tid * 32 + 16) = zero;
                }
                arrive(t_ready);
                sync();
                // dbeta_j = z_out_j + sum_i (mz + mh)_ij; a row's prefix sums over j < t', times beta, in place.
                // Four threads a row or column, 16 entries each.
                const int r = tid >> 2, s4 = tid & 3;
                float z16[16], sum = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int i = s4 * 16 + e;
                    sum += mz[i * LDM + r] + mh[i * LDM + r];   // column r
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (s4 == 0 && r < len) p.dbeta[vrow + r] = sum + zo[r] + zo[64 + r];
                float zis = 0.f, zob = 0.f;   // of token tid
                if (tid < 64) {
                    zis = (zi[tid] + zi[64 + tid]) + (zi[128 + tid] + zi[192 + tid]);
                    zob = ga[tid].z * (zo[tid] + zo[64 + tid]);
                }
                sync();
                sum = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = s4 * 16 + e;
                    z16[e] = sum;
                    // the pair of a token with itself decays over no gate
                    sum += j < r ? ga[j].z * (mz[r * LDM + j] + mh[r * LDM + j]) : 0.f;
                }
                float before = 0.f;
#pragma unroll
                for (int o = 1; o < 4; ++o) {
                    const float y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (s4 >= o) before += y;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) mz[r * LDM + s4 * 16 + e] = before + z16[e];
                if (tid < 64) {
                    zi[tid] = zis;
                    zi[64 + tid] = zob;
                }
                sync();
                float dgt = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int i = s4 * 16 + e;   // rows i >= r, and tokens i on either side of r
                    dgt += i >= r ? mz[i * LDM + r] + zi[i] : zi[64 + i];
                }
                dgt += __shfl_xor_sync(0xffffffffu, dgt, 1);
                dgt += __shfl_xor_sync(0xffffffffu, dgt, 2);
                if (s4 == 0 && r < len) {
                    float sum8 = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum8 += sds[i];
                    p.dg[vrow + r] = dgt + ga[63].w * sum8;
                }
            }
            mbar_wait(t_done, (hd - 1) & 1u, wc);
            arrive(kq_free);
            tc_fence_after();
            __nv_bfloat16 *out = (top ? p.dq : p.dk) + (row0 + t) * p.DK + half * 64;
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                float z[32];
                ld<32>(tl + CD + half * 64 + cc * 32, z);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[e] = f2_to_bf16x2(f2_add(acc[cc * 16 + 4 * j + e], f2_pack(z[8 * j + 2 * e], z[8 * j + 2 * e + 1])));
                    if (t < len && half * 64 + cc * 32 + 8 * j < p.DK)
                        *reinterpret_cast<uint4 *>(out + cc * 32 + 8 * j) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*reinterpret_cast<volatile uint32_t *>(abort_flag)) {
        // a wait gave up: let MMAs and copies this CTA may still have in flight finish (bounded)
        const unsigned long long tb = global_timer();
        while (global_timer() - tb < 100000ull) { }
    }
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_grad_tc(const Args &a, const Workspace &w, const Maps &m, const void *d_o, void *dq, void *dk,
                           float *dg, float *dbeta)
{
    auto kernel = a.DV > 64 * SUM ? grad_tc_kernel<true> : grad_tc_kernel<false>;
    cudaError_t e = ensure_dynamic_smem((const void *)kernel, TOTAL);
    if (e != cudaSuccess) return e;
    Params p = {static_cast<const __nv_bfloat16 *>(d_o), a.beta, a.lengths, static_cast<__nv_bfloat16 *>(dq),
                static_cast<__nv_bfloat16 *>(dk), dg, dbeta, a.B, a.NH, a.NHV, a.S, a.DK, a.DV, a.scale, w};
    int sms = 0;
    if ((e = sm_count(&sms)) != cudaSuccess) return e;
    const long long items = (long long)w.NC * a.B * a.NH;
    return launch_kernel(kernel, dim3((unsigned)std::min<long long>(items, sms)), dim3(THREADS), TOTAL, a.stream, 1,
                         m.q, m.k, p);
}

}  // namespace gdelta
}  // namespace mlstm
