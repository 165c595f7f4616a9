// gdelta_tc.cu -- the gated delta rule on the 5th-generation tensor cores (tcgen05), for bf16 inputs with
// 64 <= DK <= 128: the forward pass, and the backward's two walks.
//
// With S the state at a chunk's start (64 tokens) and a its cumulative log gates:
//   prep     KK = strict_lower(D * K K^T), P = lower(D * Q K^T), T = (I + KK diag(beta))^-1,
//            G = scale P diag(beta) T
//   forward  X = [K; Q] S;  Y = V - e^a X_K;  [E - Y; F] = [T - I; G] Y;  O = scale e^a X_Q + F;
//            S' = e^{a_64} S + K^T (e^{a_64 - a} beta E)
//   reverse  X = K dS';  Y = beta e^{a_64 - a} X;  dV - Y = (T - I)^T Y + G^T dO;
//            dS = e^{a_64} dS' - K^T (e^a dV) + Q^T (scale e^a dO)
// G puts the scores' product with the chunk's corrections into the same MMAs as T's, so a chunk is a chain
// of three MMA groups in either direction, each followed by one pass of the epilogue warps over its
// accumulator.  Only that chain is sequential; a CTA runs it for one value head and VT value columns.
//
// Operands.  K and Q are stacked in shared memory, 64 rows each, so that one M = 128 MMA serves both;
// the same tile, read MN-major, is the A operand of the state's update.  The fp32 operands S, Y and the
// state update's enter as three bf16 parts each, which hold all 24 bits, side by side along N: one MMA
// reads A once for all three, and the epilogue adds the parts' columns.  T - I and, backwards, G enter as three parts
// too, each the rounding of what is left; forward G as two, which only the bf16 o sees.  With two parts (2.5e-6 of the
// correction they carry) the state of slowly forgetting gates was 5.5e-7 off where fp32 arithmetic is 1.6e-7, that of a
// key that repeats, whose sums nearly cancel, 3e-5 where it is 5e-7, and there dbeta 1e-4 where it is 5e-6.  The third
// parts cost 0.26 us a chunk forward and 0.6 reverse (four and eight MMAs a chain).  K, Q, dO are exact.
// Without its unit diagonal T leaves Y itself out of the MMA: the threads that formed Y in fp32 add it to the result.
// The fp32 state stays in the epilogue threads' registers, a row (key element) of 16 columns
// each, and takes the update with fp32 additions.
//
// Roles: warp 0 one TMA thread, warp 1 the MMA thread (and the TMEM allocation), then 4 epilogue warps per
// 16 value columns.  TMEM lane = token (K rows in lanes 0..63, Q rows in 64..127) or key element, so gates
// and values are per lane, and no epilogue step exchanges anything between threads.  Every wait is bounded.
#include "gdelta_prep.cuh"
#include "tc_common.cuh"
#include "tc_fwd.h"

namespace mlstm {
namespace gdelta {
namespace {

using namespace tc;

// One contiguous copy global -> shared (16-byte aligned, a multiple of 16 bytes), completing on `bar`.
MLSTM_DEVINL void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Asks for the same bytes to be brought to L2.
MLSTM_DEVINL void bulk_prefetch(const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// Eight pairs of values of a row as three bf16 parts, whose sum is exactly the fp32 value: the top 8
// significant bits, the next 8 and the last 8 (cut off, not rounded, so packing is a byte permutation),
// into a swizzled tile of `rows` rows: 16-byte chunks j0, j0 + 1 of the row, the second and third parts
// `step` and 2 `step` chunks further.
MLSTM_DEVINL void store_parts(uint8_t *tile, uint32_t row, uint32_t j0, uint32_t step, uint32_t rows,
                              const uint64_t (&x)[8])
{
    const uint64_t neg = f2_pack(-1.f, -1.f);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t part[3][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint64_t r = x[c * 4 + e];
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const float2 v = f2_unpack(r);
                const uint32_t u0 = __float_as_uint(v.x), u1 = __float_as_uint(v.y);
                part[q][e] = __byte_perm(u0, u1, 0x7632);
                if (q < 2) r = f2_fma(f2_pack(__uint_as_float(u0 & 0xffff0000u), __uint_as_float(u1 & 0xffff0000u)), neg, r);
            }
        }
#pragma unroll
        for (int q = 0; q < 3; ++q)
            *reinterpret_cast<uint4 *>(tile + sw128_chunk(row, j0 + q * step + c, rows)) =
                make_uint4(part[q][0], part[q][1], part[q][2], part[q][3]);
    }
}

// 16 columns of an accumulator whose operand came in three parts, `step` columns apart: their sum.
MLSTM_DEVINL void load_parts(uint32_t taddr, uint32_t step, uint64_t (&x)[8])
{
    uint32_t h[16], m[16], l[16];
    tmem_ld16(taddr, h);
    tmem_ld16(taddr + step, m);
    tmem_ld16(taddr + 2 * step, l);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        auto two = [&](const uint32_t (&r)[16]) { return f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])); };
        x[i] = f2_add(two(h), f2_add(two(m), two(l)));
    }
}

// ---------------------------------------------------------------- prep

namespace prep {
constexpr int THREADS = 128;
// from 0: [2 blocks][128 rows][64] K over Q, until its product is done; then
constexpr uint32_t MR = 0;                              // [64][LDT] floats: I + KK diag(beta), then T, row-major
constexpr uint32_t MC = MR + 64 * LDT * 4;              // [64][LDT] its transpose
constexpr uint32_t PC = MC + 64 * LDT * 4;              // [64][LDT] transpose of P diag(beta)
constexpr uint32_t AC = PC + 64 * LDT * 4;              // [64] float4: cumulative log2 gate as value and residue, beta
constexpr uint32_t BAR = AC + 1024;
constexpr uint32_t TOTAL = BAR + 32 + 1024;
static_assert(PC >= 32768, "the K, Q tile lies below P");

// acc = sum_{l0 <= l < l1} A[r + 2 i .. ][l] B[l][c + j] on a tile of 2 RP rows x 4 columns, rows in pairs;
// A given transposed (ac[l][r]), B by rows.
template <int RP>
MLSTM_DEVINL void tile(const float *ac, const float *br, int r, int c, int l0, int l1, uint64_t (&acc)[RP][4])
{
#pragma unroll
    for (int i = 0; i < RP; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0;
#pragma unroll 4
    for (int l = l0; l < l1; ++l) {
        uint64_t x[RP];
#pragma unroll
        for (int i = 0; i < RP / 2; ++i) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(ac + l * LDT + r + 4 * i);
            x[2 * i] = v.x;
            x[2 * i + 1] = v.y;
        }
        const float4 y4 = *reinterpret_cast<const float4 *>(br + l * LDT + c);
        const uint64_t y[4] = {f2_pack(y4.x, y4.x), f2_pack(y4.y, y4.y), f2_pack(y4.z, y4.z), f2_pack(y4.w, y4.w)};
#pragma unroll
        for (int i = 0; i < RP; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f2_fma(x[i], y[j], acc[i][j]);
    }
}

// Joins the inverses of two diagonal blocks of N at `at`: with C the block below the first,
// the inverse has -D^-1 C A^-1 in its place.  Thread `tid` of (N / 4)^2, `sync` among all.  The intermediate
// C A^-1 goes to the (zero) block above, which is cleared again.
template <int N, typename Sync>
MLSTM_DEVINL void join(float *mr, float *mc, int at, int tid, bool on, Sync sync)
{
    const int r = (tid / (N / 4)) * 4, c = (tid % (N / 4)) * 4;
    uint64_t acc[2][4];
    if (on) {
        tile<2>(mc + at * LDT + at + N, mr + at * LDT + at, r, c, 0, N, acc);   // C A^-1
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = i & 1 ? -f2_unpack(acc[i >> 1][j]).y : -f2_unpack(acc[i >> 1][j]).x;
            *reinterpret_cast<float4 *>(mr + (at + r + i) * LDT + at + N + c) = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
    sync();
    if (on) tile<2>(mc + (at + N) * LDT + at + N, mr + at * LDT + at + N, r, c, 0, r + 4, acc);   // D^-1 lower
    sync();
    if (on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = i & 1 ? f2_unpack(acc[i >> 1][j]).y : f2_unpack(acc[i >> 1][j]).x;
            *reinterpret_cast<float4 *>(mr + (at + N + r + i) * LDT + at + c) = make_float4(x[0], x[1], x[2], x[3]);
            const float2 lo = f2_unpack(acc[0][i]), hi = f2_unpack(acc[1][i]);
            *reinterpret_cast<float4 *>(mc + (at + c + i) * LDT + at + N + r) = make_float4(lo.x, lo.y, hi.x, hi.y);
            *reinterpret_cast<float4 *>(mr + (at + r + i) * LDT + at + N + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    sync();
}
}  // namespace prep

// One CTA per chunk and key head: [K; Q] K^T once in TMEM, then the matrices of every value head on it.  Where all of
// them find room at once, one per value head instead (gridDim.z of them): 32 CTAs of two heads took 23 us, 64
// of one 13.
// The inverse (diagonal blocks of 16 by substitution,
// then joins, as invert64) and P diag(beta) T run on the CUDA cores in fp32 from shared memory, 4 x 4
// tiles fed by two 16-byte loads per reduction step; four CTAs an SM overlap their short serial parts.
// 8192 chunks of 128 key elements in pairs of value heads take 235 us, 4.2 us of an SM each: half of the
// shared-memory rate, the rest barriers between the joins.  G on the tensor cores needs P and T in three parts each
// (two lose 1e-4 of beta's gradient where keys repeat) and took 305 us with their splitting; CTAs of 64 threads
// 222 to 300 us.
template <bool BACKWARD>
__global__ void __launch_bounds__(prep::THREADS, 4)
prep_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const float *__restrict__ g, const float *__restrict__ beta, const int *__restrict__ lengths, int NH,
               int NHV, int S, int DK, float scale, Workspace w)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *mr = reinterpret_cast<float *>(smem + prep::MR), *mc = reinterpret_cast<float *>(smem + prep::MC);
    float *pc = reinterpret_cast<float *>(smem + prep::PC);
    float4 *ga = reinterpret_cast<float4 *>(smem + prep::AC);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + prep::BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2), *abort_flag = tmem_slot + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = blockIdx.x, bh = blockIdx.y, b = bh / NH, group = NHV / NH;
    WaitCtx wc{abort_flag, w.status};
    if (tid == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        *abort_flag = 0u;
        fence_barrier_init();
        tma_prefetch(&tm_q);
        tma_prefetch(&tm_k);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 64);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    griddep_launch_dependents();
    if (c == 0 && bh == 0 && blockIdx.z == 0 && tid == 0) *w.status = 0u;
    const int len = min(CH, live_tokens(lengths, b, S) - c * CH);
    if (len > 0) {
        bool issued = false;
        if (tid == 0) {
            mbar_arrive_expect_tx(&bars[0], 32768);
            for (int kb = 0; kb < 2; ++kb) {
                tma_load_3d(smem + kb * 16384, &tm_k, 64 * kb, c * CH, bh, &bars[0]);
                tma_load_3d(smem + kb * 16384 + 8192, &tm_q, 64 * kb, c * CH, bh, &bars[0]);
            }
            if (mbar_wait(&bars[0], 0, wc)) {
                constexpr uint32_t ID = idesc_bf16(128, 64, 0, 0);
                const uint64_t d = smem_desc(smem_u32(smem), 16, 1024);
                for (int kk = 0; kk * 16 < DK; ++kk) {   // behind DK both operands are zero
                    const uint64_t dk = d + (uint64_t)((kk >> 2) * 1024 + (kk & 3) * 2);
                    mma_ss(tmem, dk, dk, ID, kk > 0);
                }
                mma_commit(&bars[1]);
                issued = true;
            }
        }
        __syncwarp();
        bool ok = true;
        const int i = tid & 63;   // the thread's row: of K K^T in warps 0 and 1, of Q K^T in 2 and 3
        const bool krow = tid < 64;
        const int h0 = gridDim.z > 1 ? blockIdx.z : 0, h1 = gridDim.z > 1 ? h0 + 1 : group;
        for (int h = h0; h < h1; ++h) {
            const int bhv = b * NHV + (bh % NH) * group + h;
            const size_t ch = (size_t)bhv * w.NC + c, gt = (size_t)bhv * S + c * CH;
            if (warp == 0) {
                float2 a0, a1;
                const float b0 = 2 * lane < len ? beta[gt + 2 * lane] : 0.f;
                const float b1 = 2 * lane + 1 < len ? beta[gt + 2 * lane + 1] : 0.f;
                chunk_gates_log2(g + gt, len, lane, a0, a1);
                if (BACKWARD) {
                    w.A[ch * 64 + 2 * lane] = a0;
                    w.A[ch * 64 + 2 * lane + 1] = a1;
                }
                ga[2 * lane] = make_float4(a0.x, a0.y, b0, 0.f);
                ga[2 * lane + 1] = make_float4(a1.x, a1.y, b1, 0.f);
            }
            __syncthreads();
            if (h == h0) {
                ok = mbar_wait(&bars[1], 0, wc);
                tc_fence_after();
            }
            const float4 ai = ga[i];
            // what the walk needs of the gates: e^a of the token, and beta e^{a_64 - a}
            if (krow) w.GB[ch * 64 + i] = make_float2(exp2f(ai.x + ai.y), ai.z * exp2f((ga[63].x - ai.x) + (ga[63].y - ai.y)));
            // rows and columns behind `len` hold whatever the padding does: selected away
            const int top = i < len ? (krow ? i : i + 1) : 0;
#pragma unroll
            for (int half = 0; half < 4; ++half) {   // 16 columns
                float x[16];
                {
                    uint32_t r[16];
                    tmem_ld16(tmem_addr(tmem, warp * 32, half * 16), r);
                    tmem_wait_ld();
#pragma unroll
                    for (int s = 0; s < 16; ++s) x[s] = __uint_as_float(r[s]);
                }
                // whole blocks above the diagonal need no exponentials
                if (16 * half <= 32 * (warp & 1) + 31) {
#pragma unroll
                    for (int s = 0; s < 16; ++s) {
                        const int j = half * 16 + s;
                        const float4 aj = ga[j];
                        const bool on = j < top;   // selects, not a branch a column
                        const float d = on ? (ai.x - aj.x) + (ai.y - aj.y) : 0.f, y = on ? x[s] : 0.f;
                        x[s] = exp2f(d) * y;
                    }
                } else {
#pragma unroll
                    for (int s = 0; s < 16; ++s) x[s] = 0.f;
                }
                if (BACKWARD) {   // its KK and P
                    float *dst = (krow ? w.KK : w.P) + ch * 4096 + i * 64 + half * 16;
#pragma unroll
                    for (int s = 0; s < 16; s += 4)
                        *reinterpret_cast<float4 *>(dst + s) = make_float4(x[s], x[s + 1], x[s + 2], x[s + 3]);
                }
#pragma unroll
                for (int s = 0; s < 16; ++s) x[s] *= ga[half * 16 + s].z;
                if (krow) {
#pragma unroll
                    for (int s = 0; s < 16; ++s) mc[(half * 16 + s) * LDT + i] = x[s];
#pragma unroll
                    for (int s = 0; s < 16; s += 4)
                        *reinterpret_cast<float4 *>(mr + i * LDT + half * 16 + s) = make_float4(x[s], x[s + 1], x[s + 2], x[s + 3]);
                } else {
#pragma unroll
                    for (int s = 0; s < 16; ++s) pc[(half * 16 + s) * LDT + i] = x[s];
                }
            }
            __syncthreads();
            if (krow) {   // diagonal blocks of 16: thread (block, column j) solves (I + M_b) x = e_j
                const int at = tid & 48, j = tid & 15;
                float x[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float s0 = r == j ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                    for (int l = 0; l < r; l += 4) {   // M is zero from its diagonal on
                        const float4 y = *reinterpret_cast<const float4 *>(mr + (at + r) * LDT + at + l);
                        s0 = fmaf(-y.x, x[l], s0);
                        if (l + 1 < r) s1 = fmaf(-y.y, x[l + 1], s1);
                        if (l + 2 < r) s0 = fmaf(-y.z, x[l + 2], s0);
                        if (l + 3 < r) s1 = fmaf(-y.w, x[l + 3], s1);
                    }
                    x[r] = s0 + s1;
                }
                __syncwarp();
#pragma unroll
                for (int r = 0; r < 16; ++r) mr[(at + r) * LDT + at + j] = x[r];
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    *reinterpret_cast<float4 *>(mc + (at + j) * LDT + at + r) = make_float4(x[r], x[r + 1], x[r + 2], x[r + 3]);
            }
            __syncthreads();
            prep::join<16>(mr, mc, (tid >> 4 & 1) * 32, tid & 15, tid < 32, [] { __syncthreads(); });
            prep::join<32>(mr, mc, 0, tid & 63, tid < 64, [] { __syncthreads(); });
            // G = scale P diag(beta) T and [T - I; G] as two bf16 parts, each a swizzled tile of 128 rows of 64
            uint8_t *tg = w.TG + ch * 32768;
            const int i0 = (tid >> 4) * 8, c0 = (tid & 15) * 4;
            uint64_t acc[4][4];
            prep::tile<4>(pc, mr, i0, c0, 0, i0 + 8, acc);   // from 0: one address for all columns
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float4 t4 = *reinterpret_cast<const float4 *>(mr + (i0 + r) * LDT + c0);
                const float t[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 gp = f2_unpack(acc[r >> 1][e]);
                        y[e] = part ? scale * (r & 1 ? gp.y : gp.x) : i0 + r == c0 + e ? 0.f : t[e];
                    }
                    uint32_t cut[3][2];   // each part the rounding of what is left
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int q = 0; q < 3; ++q) {
                            const uint32_t u = pack_bf16(y[2 * e], y[2 * e + 1]);
                            cut[q][e] = u;
                            y[2 * e] -= __uint_as_float(u << 16);
                            y[2 * e + 1] -= __uint_as_float(u & 0xffff0000u);
                        }
                    const uint32_t off = sw128_offset(64 * part + i0 + r, c0, 128);
                    *reinterpret_cast<uint2 *>(tg + off) = make_uint2(cut[0][0], cut[0][1]);
                    *reinterpret_cast<uint2 *>(tg + 16384 + off) = make_uint2(cut[1][0], cut[1][1]);
                    if (part == 0 || BACKWARD)   // the third part of T - I, and the backward's of G
                        *reinterpret_cast<uint2 *>((part ? w.GL : w.TL) + ch * 8192 + sw128_offset(i0 + r, c0, 64)) =
                            make_uint2(cut[2][0], cut[2][1]);
                }
            }
            __syncthreads();
        }
        if (tid == 0 && !ok) {   // a wait gave up: let the copies and the MMAs of this CTA finish (bounded)
            mbar_wait_drain(&bars[0], 0);
            if (issued) mbar_wait_drain(&bars[1], 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 64);
    }
}

// ---------------------------------------------------------------- walk

// A CTA runs two chains side by side, CW value columns each, on the same K, Q, T and G tiles: while the
// epilogue warps of one pass over an accumulator, the MMAs of the other run.  What bounds a walk is that chain: 2.4 us
// a chunk at CW 16 (32 heads of 16384 tokens, 128 x 128: 615 us, 128 CTAs), 4.3 us at CW 32; with the states
// and E kept 2.7 us, at CW 32 4.6 us (4 x 16 heads of 4096 tokens: 295 us, against 338 in two rounds of CTAs at CW
// 16); reverse 3.9 us.  The tensor pipe is busy a quarter of it, the rest are the epilogues' passes from TMEM over registers to shared memory and the
// waits between the two.  One chain of 32 columns, three or four chains, or 8 columns a thread were no faster.
enum Mode { FORWARD, KEEP, REVERSE };   // KEEP: the forward walk again, for the backward: states and E, no outputs

template <int CW, int KS, int MODE>
struct Walk {
    static constexpr int NCH = 2;                          // chains
    static constexpr int VT = NCH * CW;                    // value columns of the CTA
    static constexpr int EPI = 4 * (CW / 16);              // epilogue warps per chain, 16 columns each
    static constexpr int THREADS = 64 + 32 * NCH * EPI;
    static constexpr int STAGES = 2;
    // A stage: [K; Q] as one or two blocks of 64 columns, then [T - I; G] values and residues, 16 KB each; forward
    // also the third part of T - I, with zeros in G's rows.  With 64 columns a CTA there is room for T - I and G
    // only once: the next chunk's come behind this one's second product with them (single).  Reverse the third parts of
    // T - I and G have one place likewise.  KEEP has
    // no use for Q and G, whose lanes' sums stay unread: K alone, and three parts of T - I, 8 KB each; the MMAs' rows
    // 64..127 are then whatever follows, and so are the state's rows from 64 on with one block.
    static constexpr uint32_t KROWS = MODE == KEEP ? 64 : 128, KB = KROWS * 128, KBLK = KS / 4;
    static constexpr bool SINGLE = MODE == FORWARD && CW == 32;
    static constexpr uint32_t KQ = KBLK * KB;
    static constexpr uint32_t TLOAD = MODE == KEEP ? 24576 : MODE == FORWARD ? 40960 : 32768;
    static constexpr uint32_t TSIZE = TLOAD + (MODE == FORWARD ? 8192 : 0);
    static constexpr uint32_t STAGE = KQ + (SINGLE ? 0 : TSIZE);
    static constexpr uint32_t TOFF = SINGLE ? STAGES * STAGE : KQ;   // of a stage's, or of the only one
    static constexpr uint32_t BLOCKS = (3 * CW + 63) / 64; // blocks of 64 columns that hold an operand's parts
    static constexpr uint32_t SP = STAGES * STAGE + (SINGLE ? TSIZE : 0);   // per chain: S parts, 128 rows
    static constexpr uint32_t YN = SP + NCH * BLOCKS * 16384;   // per chain: Y parts, then the update's, a row per token
    static constexpr uint32_t YROWS = MODE == REVERSE ? 128 : 64;   // (reverse: K's tokens, then Q's)
    static constexpr uint32_t DO = 3 * CW / 8;             // reverse: dO, 64 rows, in the 16-byte chunks behind Y's parts
    static constexpr uint32_t T3 = YN + NCH * BLOCKS * YROWS * 128;   // reverse: the third parts of T - I and G
    // the backward: an epilogue warp's 32 rows of fp32 results on their way out
    static constexpr uint32_t OUT = T3 + (MODE == REVERSE ? 16384 : 0);
    static constexpr uint32_t BAR = OUT + (MODE == FORWARD ? 0 : NCH * EPI * 2048);
    static constexpr uint32_t NBAR = 2 * STAGES + 7 * NCH + 2;
    static constexpr uint32_t TOTAL = BAR + NBAR * 8 + 16 + 1024;
    static_assert(TOTAL <= 232448, "one CTA's shared memory");
    // TMEM columns of a chain: X and [E; F], 3 CW each; D over X, or (reverse) beside them with G^T dO
    static constexpr uint32_t TX = 0, TE = 3 * CW, TD = MODE == REVERSE ? 6 * CW : 0, TG = 9 * CW;
    static constexpr uint32_t TCH = MODE == REVERSE ? 10 * CW : 6 * CW;
    static constexpr uint32_t TMEM_COLS = NCH * TCH > 256 ? 512 : 256;
};

struct WalkParams {
    const __nv_bfloat16 *v;   // reverse: dO
    const float *S0;          // reverse: dS_final
    const int *lengths;
    __nv_bfloat16 *o;         // reverse: dv
    float *S_final;           // reverse: dS0
    int NH, NHV, S, DK, DV;
    float scale;
    Workspace w;
};

template <int CW, int KS, int MODE>
__global__ void __launch_bounds__(Walk<CW, KS, MODE>::THREADS, 1)
walk_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_s, const __grid_constant__ CUtensorMap tm_t, const WalkParams p)
{
    using W = Walk<CW, KS, MODE>;
    static_assert(MODE != REVERSE || CW == 16, "Y's parts leave room for dO");
    constexpr int NST = W::STAGES, NCH = W::NCH;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + W::BAR);
    // per chain: S, Y and N written by the epilogue; X, [E; F] and D finished by the MMAs
    uint64_t *full = bars, *empty = bars + NST, *s_ready = bars + 2 * NST, *x_done = s_ready + NCH, *y_ready = x_done + NCH,
             *e_done = y_ready + NCH, *n_ready = e_done + NCH, *d_done = n_ready + NCH, *o_ready = d_done + NCH,
             *t_full = o_ready + NCH, *t_empty = t_full + 1;   // T - I and G, or their third parts, with one place
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + W::NBAR), *abort_flag = tmem_slot + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bhv = blockIdx.y, b = bhv / p.NHV, bh = b * p.NH + (bhv % p.NHV) / (p.NHV / p.NH);
    WaitCtx wc{abort_flag, p.w.status};
    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int h = 0; h < NCH; ++h) {
            mbar_init(&s_ready[h], W::EPI);
            mbar_init(&x_done[h], 1);
            mbar_init(&y_ready[h], W::EPI / 2);
            mbar_init(&e_done[h], 1);
            mbar_init(&n_ready[h], MODE == REVERSE ? W::EPI / 2 : W::EPI);
            mbar_init(&d_done[h], 1);
            mbar_init(&o_ready[h], W::EPI / 2);
        }
        mbar_init(t_full, 1);
        mbar_init(t_empty, 1);
        *abort_flag = 0u;
        fence_barrier_init();
        tma_prefetch(&tm_q);
        tma_prefetch(&tm_k);
        if (MODE != FORWARD) {
            tma_prefetch(&tm_s);
            tma_prefetch(&tm_t);
        }
    }
    if (MODE == FORWARD) {   // the zeros behind the third part of T - I
        for (uint32_t i = threadIdx.x * 16; i < (W::SINGLE ? 1 : NST) * 8192; i += W::THREADS * 16)
            *reinterpret_cast<uint4 *>(smem + W::TOFF + (i >> 13) * W::STAGE + W::TLOAD + (i & 8191)) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, W::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The reverse walk reads nothing of the forward recomputation launched just before it, only what that one
    // waited for; so it runs beside its last CTAs and waits for it at its own end, for the kernel behind
    if (MODE != REVERSE) griddep_wait();
    griddep_launch_dependents();
    const int n = live_tokens(p.lengths, b, p.S), nc = (n + CH - 1) / CH;

    if (warp == 0) {
        if (lane == 0) {
            for (int c = 0; c < nc; ++c) {
                const int st = c % NST, ci = MODE == REVERSE ? nc - 1 - c : c;
                if (c >= NST && !mbar_wait(&empty[st], (uint32_t)(c / NST - 1) & 1u, wc)) break;
                uint8_t *s = smem + st * W::STAGE;
                const size_t ch = (size_t)bhv * p.w.NC + ci;
                mbar_arrive_expect_tx(&full[st], W::KQ + (W::SINGLE ? 0 : W::TLOAD));
                for (int kb = 0; kb < (int)W::KBLK; ++kb) {
                    tma_load_3d(s + kb * W::KB, &tm_k, 64 * kb, ci * CH, bh, &full[st]);
                    if (MODE != KEEP) tma_load_3d(s + kb * W::KB + 8192, &tm_q, 64 * kb, ci * CH, bh, &full[st]);
                }
                uint64_t *tbar = &full[st];
                uint8_t *tt = s + W::TOFF;
                if (W::SINGLE) {
                    bulk_prefetch(p.w.TG + ch * 32768, 32768);
                    bulk_prefetch(p.w.TL + ch * 8192, 8192);
                    if (c > 0 && !mbar_wait(t_empty, (uint32_t)(c - 1) & 1u, wc)) break;
                    tbar = t_full;
                    tt = smem + W::TOFF;
                    mbar_arrive_expect_tx(t_full, W::TLOAD);
                }
                if (MODE == REVERSE) {
                    bulk_prefetch(p.w.TL + ch * 8192, 8192);
                    bulk_prefetch(p.w.GL + ch * 8192, 8192);
                }
                if (MODE == KEEP) {
                    bulk_load(tt, p.w.TG + ch * 32768, 8192, tbar);
                    bulk_load(tt + 8192, p.w.TG + ch * 32768 + 16384, 8192, tbar);
                    bulk_load(tt + 16384, p.w.TL + ch * 8192, 8192, tbar);
                } else {
                    bulk_load(tt, p.w.TG + ch * 32768, 32768, tbar);
                    if (MODE == FORWARD) bulk_load(tt + 32768, p.w.TL + ch * 8192, 8192, tbar);
                }
                if (MODE == REVERSE) {
                    if (c > 0 && !mbar_wait(t_empty, (uint32_t)(c - 1) & 1u, wc)) break;
                    mbar_arrive_expect_tx(t_full, 16384);
                    bulk_load(smem + W::T3, p.w.TL + ch * 8192, 8192, t_full);
                    bulk_load(smem + W::T3 + 8192, p.w.GL + ch * 8192, 8192, t_full);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // A K-major (X, E) or MN-major (D), B MN-major; N = the parts' columns side by side, so that A is
            // read once for all of them
            constexpr uint32_t IDX = idesc_bf16(128, 3 * CW, 0, 1), IDM = idesc_bf16(128, 2 * CW, 0, 1);
            constexpr uint32_t IDD = idesc_bf16(128, 3 * CW, 1, 1);
            constexpr uint32_t BS = W::BLOCKS * 1024, BY = W::BLOCKS * W::YROWS * 8;   // a chain's operands, 16-byte units
            // reverse: T^T and G^T, M = 64; the 64 M behind read what lies behind, into lanes that nothing uses
            constexpr uint32_t IDG0 = idesc_bf16(128, CW, 0, 1), RES = MODE == KEEP ? 512 : 1024;
            constexpr uint32_t IDTM = idesc_bf16(128, 2 * CW, 1, 1), IDG = idesc_bf16(128, CW, 1, 1);
            const uint64_t atm = smem_desc(smem_u32(smem) + W::TOFF, 8192, 1024);
            const uint64_t at3 = MODE == REVERSE ? smem_desc(smem_u32(smem + W::T3), 8192, 1024) : 0;
            const uint64_t bs = smem_desc(smem_u32(smem + W::SP), 16384, 1024);
            const uint64_t by = smem_desc(smem_u32(smem + W::YN), W::YROWS * 128, 1024);
            const uint64_t ak = smem_desc(smem_u32(smem), 16, 1024), at = smem_desc(smem_u32(smem) + W::TOFF, 16, 1024);
            const uint64_t ad = smem_desc(smem_u32(smem), W::KB, 1024);
            bool ok = true;
            for (int c = 0; c < nc && ok; ++c) {
                const int st = c % NST;
                const uint64_t so = (uint64_t)st * (W::STAGE / 16), to = W::SINGLE ? 0 : so;
                const uint32_t ph = (uint32_t)c & 1u;
                ok = mbar_wait(&full[st], (uint32_t)(c / NST) & 1u, wc);
                auto issue_x = [&](int h) {
                    if (!(ok = ok && mbar_wait(&s_ready[h], ph, wc))) return;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < KS; ++k)
                        mma_ss(tmem + h * W::TCH + W::TX, ak + so + (uint64_t)((k >> 2) * (W::KB / 16) + (k & 3) * 2),
                               bs + (uint64_t)(h * BS + k * 128), IDX, k > 0);
                    mma_commit(&x_done[h]);
                };
                // reverse: G^T dO, and the update's share of Q's tokens; neither waits for the state
                auto issue_q = [&](int h) {
                    if (!(ok = ok && mbar_wait(&o_ready[h], ph, wc))) return;
                    if (h == 0 && !(ok = ok && mbar_wait(t_full, ph, wc))) return;
                    tc_fence_after();
                    const uint64_t bo = by + (uint64_t)(h * BY + W::DO);
                    // smallest first; G's rows lie 8 KB into each part's tile
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss(tmem + h * W::TCH + W::TG, at3 + (uint64_t)(512 + k * 128), bo + (uint64_t)(k * 128), IDG, k > 0);
#pragma unroll
                    for (int k = 7; k >= 0; --k)   // the values' tile, and 16 KB further the residues'
                        mma_ss(tmem + h * W::TCH + W::TG, atm + to + (uint64_t)(512 + (k >> 2) * 1024 + (k & 3) * 128),
                               bo + (uint64_t)((k & 3) * 128), IDG, 1);
#pragma unroll
                    for (int k = 4; k < 8; ++k)
                        mma_ss(tmem + h * W::TCH + W::TD, ad + so + (uint64_t)(k * 128), by + (uint64_t)(h * BY + k * 128), IDD, k > 4);
                };
                auto issue_e = [&](int h) {
                    if (W::SINGLE && h == 0 && !(ok = ok && mbar_wait(t_full, ph, wc))) return;
                    if (!(ok = ok && mbar_wait(&y_ready[h], ph, wc))) return;
                    tc_fence_after();
                    const uint32_t de = tmem + h * W::TCH + W::TE;
                    // An MMA cuts off at the size of the sum it adds to, so products of one size share columns: the values
                    // of T - I and G with Y's three parts; their residues with Y's first two go to the second and third
                    // of these, the third part of T - I with Y's first to the third.  The tokens nearest to the diagonal
                    // come last
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = MODE == REVERSE ? 3 - i : i;
                        mma_ss(de, MODE == REVERSE ? atm + to + (uint64_t)(k * 128) : at + to + (uint64_t)(k * 2),
                               by + (uint64_t)(h * BY + k * 128), MODE == REVERSE ? IDD : IDX, i > 0);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = MODE == REVERSE ? 3 - i : i;
                        mma_ss(de + CW, MODE == REVERSE ? atm + to + (uint64_t)(1024 + k * 128) : at + to + (uint64_t)(RES + k * 2),
                               by + (uint64_t)(h * BY + k * 128), MODE == REVERSE ? IDTM : IDM, 1);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = MODE == REVERSE ? 3 - i : i;
                        mma_ss(de + 2 * CW, MODE == REVERSE ? at3 + (uint64_t)(k * 128) : at + to + (uint64_t)(2 * RES + k * 2),
                               by + (uint64_t)(h * BY + k * 128), MODE == REVERSE ? IDG : IDG0, 1);
                    }
                    mma_commit(&e_done[h]);
                    if ((W::SINGLE || MODE == REVERSE) && h == NCH - 1) mma_commit(t_empty);
                };
                auto issue_d = [&](int h) {
                    if (!(ok = ok && mbar_wait(&n_ready[h], ph, wc))) return;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)   // forward: over X, which every warp has read
                        mma_ss(tmem + h * W::TCH + W::TD, ad + so + (uint64_t)(k * 128), by + (uint64_t)(h * BY + k * 128), IDD,
                               MODE == REVERSE || k > 0);
                    mma_commit(&d_done[h]);
                };
#pragma unroll
                for (int h = 0; h < NCH; ++h) issue_x(h);
#pragma unroll
                for (int h = 0; h < NCH; ++h) {
                    if (MODE == REVERSE) issue_q(h);
                    issue_e(h);
                }
#pragma unroll
                for (int h = 0; h < NCH; ++h) issue_d(h);
                if (ok) mma_commit(&empty[st]);
            }
        }
    } else {
        const int quad = warp & 3, h = (warp - 2) / W::EPI, cg = ((warp - 2) % W::EPI) >> 2;
        const int row = quad * 32 + lane, t = row & 63;        // TMEM lane; token of the chunk
        const bool krow = quad < 2;
        const int col = blockIdx.x * W::VT + h * CW + cg * 16; // first of the thread's 16 value columns
        const uint32_t tl = tmem_addr(tmem, quad * 32, h * W::TCH + cg * 16);
        uint8_t *sp = smem + W::SP + h * W::BLOCKS * 16384, *yn = smem + W::YN + h * W::BLOCKS * W::YROWS * 128;
        uint64_t s[8];                                         // row `row` of the state, in pairs
        const size_t srow = ((size_t)bhv * p.DK + row) * p.DV + col;
        const int live_cols = min(16, p.DV - col);             // a multiple of 8, may be <= 0
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 x = p.S0 && row < p.DK && 4 * e < live_cols ? *reinterpret_cast<const float4 *>(p.S0 + srow + 4 * e)
                                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
            s[2 * e] = f2_pack(x.x, x.y);
            s[2 * e + 1] = f2_pack(x.z, x.w);
        }
        // the warp's 32 rows of 16 fp32 columns to rows r0 .. of chunk ci's array, by way of its buffer
        uint8_t *buf = smem + W::OUT + (warp - 2) * 2048;
        auto send = [&](const CUtensorMap &tm, int r0, int ci, const uint64_t (&x)[8]) {
            if (live_cols <= 0) return;
            if (lane == 0) bulk_wait_read0();
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<ulonglong2 *>(buf + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) = make_ulonglong2(x[2 * e], x[2 * e + 1]);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                tma_store_3d(&tm, buf, col, r0, bhv * p.w.NC + ci);
                bulk_commit();
            }
        };
        for (int c = 0; c < nc; ++c) {
            const uint32_t ph = (uint32_t)c & 1u;
            const int ci = MODE == REVERSE ? nc - 1 - c : c, len = min(CH, n - ci * CH);
            store_parts(sp, row, cg * 2, CW / 8, 128, s);
            fence_proxy_async();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_ready[h]);
            if (MODE != FORWARD && quad * 32 < p.DK) send(tm_s, quad * 32, ci, s);
            // the token's gates and its row of V (reverse: dO, the rows of Q's warps): asked for here, they
            // arrive while X is computed; a load in flight at one of the fences would hold it up.  The next
            // chunk's row is brought to L2
            const int tok = ci * CH + t;
            const float2 *GB = p.w.GB + ((size_t)bhv * p.w.NC + ci) * 64;
            const float2 gt = GB[t];
            const float ef = GB[63].x, ea = gt.x, eo = gt.y;
            const __nv_bfloat16 *v = p.v + ((size_t)bhv * p.S + tok) * p.DV + col;
            const bool vrow = MODE == REVERSE ? !krow : krow;
            uint4 vr[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                vr[e] = vrow && tok < n && 8 * e < live_cols ? *reinterpret_cast<const uint4 *>(v + 8 * e)
                                                             : make_uint4(0u, 0u, 0u, 0u);
            const int ahead = MODE == REVERSE ? -CH : CH;
            if (vrow && live_cols > 0 && tok + ahead >= 0 && tok + ahead < n)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(v + (ptrdiff_t)ahead * p.DV));
            uint64_t x[8], y[8];
            if (MODE == REVERSE && !krow) {   // dO itself, and scale e^a dO behind the K tokens' rows
#pragma unroll
                for (int e = 0; e < 2; ++e) *reinterpret_cast<uint4 *>(yn + sw128_chunk(t, W::DO + e, W::YROWS)) = vr[e];
                const uint64_t f = f2_pack(p.scale * ea, p.scale * ea);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = f2_mul(f, f2_from_bf16x2((&vr[e >> 2].x)[e & 3]));
                store_parts(yn, row, cg * 2, CW / 8, W::YROWS, x);
                if (len < CH) {   // padding, as for K below; the tile has to have landed
                    if (!mbar_wait(&full[c % NST], (uint32_t)(c / NST) & 1u, wc)) break;
                    if (h == 0 && cg == 0 && t >= len) {
#pragma unroll
                        for (int j = 0; j < 2 * KS; ++j)
                            *reinterpret_cast<uint4 *>(smem + (c % NST) * W::STAGE + sw128_chunk(64 + t, j, 128)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_ready[h]);
            }
            if (!mbar_wait(&x_done[h], ph, wc)) break;
            tc_fence_after();
            uint8_t *kq = smem + (c % NST) * W::STAGE;
            if (krow || MODE == FORWARD) load_parts(tl, CW, x);
            if (krow) {
                const float fx = MODE == REVERSE ? eo : -ea;
                const uint64_t f = f2_pack(fx, fx);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = MODE == REVERSE ? f2_mul(f, x[e]) : f2_fma(f, x[e], f2_from_bf16x2((&vr[e >> 2].x)[e & 3]));
                if (t >= len) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = 0;
                }
                store_parts(yn, row, cg * 2, CW / 8, W::YROWS, x);
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&y_ready[h]);
            } else if (MODE != REVERSE) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&n_ready[h]);   // X is read
            }
            if (!mbar_wait(&e_done[h], ph, wc)) break;
            tc_fence_after();
            if (krow || MODE == FORWARD) load_parts(tl + W::TE, CW, y);
            if (krow) {
                if (MODE == REVERSE) {
                    uint32_t go[16];
                    tmem_ld16(tl + W::TG, go);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = f2_add(y[e], f2_pack(__uint_as_float(go[2 * e]), __uint_as_float(go[2 * e + 1])));
                }
                const float fn = MODE == REVERSE ? -ea : eo;
                const uint64_t f = f2_pack(fn, fn);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = f2_add(x[e], y[e]);   // E, or dV
                    y[e] = f2_mul(f, x[e]);
                }
                store_parts(yn, row, cg * 2, CW / 8, W::YROWS, y);
                if (h == 0 && cg == 0 && t >= len) {
                    // padding: its keys meet N's zeros, which NaN would survive.  X of the other chain may still
                    // read them (into lanes that nothing uses); its D is issued after this chain's N arrived
#pragma unroll
                    for (int j = 0; j < 2 * KS; ++j) *reinterpret_cast<uint4 *>(kq + sw128_chunk(t, j, W::KROWS)) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&n_ready[h]);
                if (MODE != FORWARD) send(tm_t, quad * 32, ci, x);
            }
            if (MODE == FORWARD ? !krow && t < len : MODE == REVERSE && krow && t < len) {
                __nv_bfloat16 *o = p.o + ((size_t)bhv * p.S + ci * CH + t) * p.DV + col;
                const uint64_t fe = f2_pack(p.scale * ea, p.scale * ea);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (8 * e >= live_cols) break;
                    uint32_t z[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        z[u] = f2_to_bf16x2(MODE == FORWARD ? f2_fma(fe, x[4 * e + u], y[4 * e + u]) : x[4 * e + u]);
                    *reinterpret_cast<uint4 *>(o + 8 * e) = make_uint4(z[0], z[1], z[2], z[3]);
                }
            }
            if (!mbar_wait(&d_done[h], ph, wc)) break;
            tc_fence_after();
            load_parts(tl + W::TD, CW, y);
            const uint64_t f = f2_pack(ef, ef);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = f2_fma(f, s[e], y[e]);
        }
        if (MODE != FORWARD && lane == 0) bulk_wait0();   // the warp's results are on their way no longer
        if (MODE != KEEP && p.S_final && row < p.DK) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * e < live_cols) {
                    const float2 u = f2_unpack(s[2 * e]), v = f2_unpack(s[2 * e + 1]);
                    *reinterpret_cast<float4 *>(p.S_final + srow + 4 * e) = make_float4(u.x, u.y, v.x, v.y);
                }
        }
        for (int r = n + (int)threadIdx.x - 64; MODE != KEEP && r < p.S; r += W::THREADS - 64) {   // padding rows
            __nv_bfloat16 *o = p.o + ((size_t)bhv * p.S + r) * p.DV + blockIdx.x * W::VT;
            for (int e = 0; e < W::VT && (int)blockIdx.x * W::VT + e < p.DV; e += 8)
                *reinterpret_cast<uint4 *>(o + e) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*reinterpret_cast<volatile uint32_t *>(abort_flag)) {
        // a wait gave up: let MMAs and copies this CTA may still have in flight finish (bounded)
        const unsigned long long tb = global_timer();
        while (global_timer() - tb < 100000ull) { }
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, W::TMEM_COLS);
    }
    if (MODE == REVERSE) griddep_wait();
}

template <int CW, int KS, int MODE>
cudaError_t launch_walk_cw(const Args &a, const Workspace &w, const CUtensorMap (&m)[4], const void *v, const float *S0,
                           void *o, float *S_final)
{
    using W = Walk<CW, KS, MODE>;
    cudaError_t e = ensure_dynamic_smem((const void *)walk_tc_kernel<CW, KS, MODE>, W::TOTAL);
    if (e != cudaSuccess) return e;
    WalkParams p = {static_cast<const __nv_bfloat16 *>(v), S0, a.lengths, static_cast<__nv_bfloat16 *>(o), S_final, a.NH,
                    a.NHV, a.S, a.DK, a.DV, a.scale, w};
    return launch_kernel(walk_tc_kernel<CW, KS, MODE>, dim3((a.DV + W::VT - 1) / W::VT, a.B * a.NHV), dim3(W::THREADS),
                         W::TOTAL, a.stream, 1, m[0], m[1], m[2], m[3], p);
}

template <int MODE>
cudaError_t launch_walk_tc(const Args &a, const Workspace &w, const Maps &qk, const void *v, const float *S0, void *o,
                           float *S_final)
{
    CUtensorMap m[4] = {qk.q, qk.k, qk.q, qk.q};   // q, k, and where the states' and the tokens' results go
    if (MODE != FORWARD && (!tcfwd::make_map_f32(&m[2], MODE == KEEP ? w.SC : w.DSC, a.DV, a.DK, a.B * a.NHV * w.NC) ||
                            !tcfwd::make_map_f32(&m[3], MODE == KEEP ? w.E : w.DV, a.DV, 64, a.B * a.NHV * w.NC)))
        return cudaErrorUnknown;
    // While the GPU has SMs for it a CTA takes 32 columns; 64 take fewer CTAs than twice the time (the epilogue
    // warps of the K tokens, two of the SM's four schedulers, are what a chunk then waits for): a forward call of 192,
    // 256 and 512 CTAs of 32 columns took 405, 427 (4096 tokens) and 378 us (2048), half as many of 64 361, 382 and 331.  The reverse
    // walk always takes 32: Q's share of the update and the results' way out take the shared memory
    const bool narrow = MODE == REVERSE || (long long)a.B * a.NHV * ((a.DV + 31) / 32) <= 148;
    if constexpr (MODE != REVERSE)
        if (!narrow) return a.DK > 64 ? launch_walk_cw<32, 8, MODE>(a, w, m, v, S0, o, S_final)
                                      : launch_walk_cw<32, 4, MODE>(a, w, m, v, S0, o, S_final);
    return a.DK > 64 ? launch_walk_cw<16, 8, MODE>(a, w, m, v, S0, o, S_final)
                     : launch_walk_cw<16, 4, MODE>(a, w, m, v, S0, o, S_final);
}

}  // namespace

bool tc_supported(bool bf16, int DK, int DV) { return bf16 && DK >= 64 && DV >= 32; }

bool make_maps(const Args &a, Maps *m)
{
    return tcfwd::make_map(&m->q, a.q, a.DK, a.S, a.B * a.NH, CH) && tcfwd::make_map(&m->k, a.k, a.DK, a.S, a.B * a.NH, CH);
}

cudaError_t launch_prep_tc(const Args &a, const Workspace &w, const Maps &m)
{
    auto kernel = w.KK ? prep_tc_kernel<true> : prep_tc_kernel<false>;
    const cudaError_t e = ensure_dynamic_smem((const void *)kernel, prep::TOTAL);
    if (e != cudaSuccess) return e;
    const bool split = (long long)w.NC * a.B * a.NHV <= 4 * 148;
    return launch_kernel(kernel, dim3(w.NC, a.B * a.NH, split ? a.NHV / a.NH : 1), dim3(prep::THREADS), prep::TOTAL, a.stream, 1, m.q, m.k,
                         a.g, a.beta, a.lengths, a.NH, a.NHV, a.S, a.DK, a.scale, w);
}

cudaError_t launch_forward_tc(const Args &a, const Workspace &w, const Maps &m, void *o, float *S_final)
{
    return launch_walk_tc<FORWARD>(a, w, m, a.v, a.S0, o, S_final);
}

cudaError_t launch_keep_tc(const Args &a, const Workspace &w, const Maps &m)
{
    return launch_walk_tc<KEEP>(a, w, m, a.v, a.S0, nullptr, nullptr);
}

cudaError_t launch_reverse_tc(const Args &a, const Workspace &w, const Maps &m, const void *d_o, const float *dS_final,
                              void *dv, float *dS0)
{
    return launch_walk_tc<REVERSE>(a, w, m, d_o, dS_final, dv, dS0);
}

}  // namespace gdelta
}  // namespace mlstm
