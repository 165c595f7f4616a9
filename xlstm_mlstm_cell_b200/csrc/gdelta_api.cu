// gdelta_api.cu -- the C ABI of the gated delta rule: argument checks, workspace layout, dispatch.
#include "gdelta_internal.h"

#include <stdint.h>

#include "gdelta.h"

using namespace mlstm;
using namespace mlstm::gdelta;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

mlstm_status check_heads(mlstm_dtype dt, int B, int NH, int NHV, int DK, int DV)
{
    if (B < 0 || NH < 1 || NHV < 1 || NHV % NH != 0) return MLSTM_ERR_INVALID_ARG;
    if (dt != MLSTM_F32 && dt != MLSTM_BF16) return MLSTM_ERR_UNSUPPORTED;
    if (DK < 8 || DK > 128 || DK % 8 != 0 || DV < 8 || DV > 512 || DV % 8 != 0) return MLSTM_ERR_UNSUPPORTED;
    return MLSTM_OK;
}

mlstm_status check_shape(mlstm_dtype dt, int B, int NH, int NHV, int S, int DK, int DV)
{
    if (S < 0) return MLSTM_ERR_INVALID_ARG;
    const mlstm_status st = check_heads(dt, B, NH, NHV, DK, DV);
    if (st != MLSTM_OK) return st;
    if ((long long)B * NHV > 65535 || S > (1 << 30)) return MLSTM_ERR_UNSUPPORTED;
    if ((long long)B * NHV * (S / CH + 1) > 0x7fffffffll) return MLSTM_ERR_UNSUPPORTED;   // chunks, counted in an int
    return MLSTM_OK;
}

// Lays out the workspace (base may be NULL to size it).  Returns the bytes used.
size_t plan(char *base, const Args &a, bool backward, Workspace *w)
{
    Workspace tmp = {};
    if (!w) w = &tmp;
    w->NC = a.S / CH + (a.S % CH != 0);
    const size_t chunks = (size_t)a.B * a.NHV * w->NC;
    size_t off = 0;
    auto take = [&](size_t bytes) -> char * {
        char *p = base ? base + off : nullptr;
        off += (bytes + 255) / 256 * 256;
        return p;
    };
    w->status = reinterpret_cast<uint32_t *>(take(sizeof(uint32_t)));
    const bool tc = tc_supported(a.bf16, a.DK, a.DV);
    if (tc) {
        w->GB = reinterpret_cast<float2 *>(take(sizeof(float2) * 64 * chunks));
        w->TG = reinterpret_cast<uint8_t *>(take(32768 * chunks));
        w->TL = reinterpret_cast<uint8_t *>(take(8192 * chunks));
    } else {
        w->T = reinterpret_cast<float *>(take(sizeof(float) * 4096 * chunks));
    }
    if (!tc || backward) {
        w->A = reinterpret_cast<float2 *>(take(sizeof(float2) * 64 * chunks));
        w->P = reinterpret_cast<float *>(take(sizeof(float) * 4096 * chunks));
    }
    if (backward) {
        if (tc) w->GL = reinterpret_cast<uint8_t *>(take(8192 * chunks));
        w->KK = reinterpret_cast<float *>(take(sizeof(float) * 4096 * chunks));
        w->SC = reinterpret_cast<float *>(take(sizeof(float) * a.DK * a.DV * chunks));
        w->DSC = reinterpret_cast<float *>(take(sizeof(float) * a.DK * a.DV * chunks));
        w->E = reinterpret_cast<float *>(take(sizeof(float) * 64 * a.DV * chunks));
        w->DV = reinterpret_cast<float *>(take(sizeof(float) * 64 * a.DV * chunks));
    }
    return off;
}

mlstm_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MLSTM_OK : MLSTM_ERR_CUDA; }

Args make_args(const void *q, const void *k, const void *v, const float *g, const float *beta, const int *lengths,
               mlstm_dtype dt, int B, int NH, int NHV, int S, int DK, int DV, float scale, const float *S0,
               void *stream)
{
    Args a = {};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.lengths = lengths; a.S0 = S0;
    a.B = B; a.NH = NH; a.NHV = NHV; a.S = S; a.DK = DK; a.DV = DV;
    a.scale = scale;
    a.bf16 = dt == MLSTM_BF16;
    a.stream = static_cast<cudaStream_t>(stream);
    return a;
}

mlstm_status check_workspace(void *workspace, size_t bytes, size_t need)
{
    if (!workspace || bytes < need) return MLSTM_ERR_WORKSPACE;
    return (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0 ? MLSTM_OK : MLSTM_ERR_INVALID_ARG;
}

size_t workspace_size(int B, int NH, int NHV, int S, int DK, int DV, mlstm_dtype dt, bool backward)
{
    if (check_shape(dt, B, NH, NHV, S, DK, DV) != MLSTM_OK) return 0;
    return plan(nullptr, make_args(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, dt, B, NH, NHV, S, DK, DV, 0.f,
                                   nullptr, nullptr), backward, nullptr);
}

}  // namespace

extern "C" {

size_t gdelta_fwd_workspace_size(int B, int NH, int NHV, int S, int DK, int DV, mlstm_dtype dt)
{
    return workspace_size(B, NH, NHV, S, DK, DV, dt, false);
}

size_t gdelta_bwd_workspace_size(int B, int NH, int NHV, int S, int DK, int DV, mlstm_dtype dt)
{
    return workspace_size(B, NH, NHV, S, DK, DV, dt, true);
}

int gdelta_fwd_tensor_path(int DK, int DV, mlstm_dtype dt)
{
    if (check_shape(dt, 1, 1, 1, 1, DK, DV) != MLSTM_OK) return -1;
    return tc_supported(dt == MLSTM_BF16, DK, DV) ? 1 : 0;
}

mlstm_status gdelta_fwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                        const int *lengths, mlstm_dtype dt, int B, int NH, int NHV, int S, int DK, int DV,
                        float scale, const float *S0, void *o, float *S_final, void *workspace,
                        size_t workspace_bytes, void *stream)
{
    mlstm_status st = check_shape(dt, B, NH, NHV, S, DK, DV);
    if (st != MLSTM_OK) return st;
    if (B == 0) return MLSTM_OK;
    if (S > 0 && (!q || !k || !v || !g || !beta || !o)) return MLSTM_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(g) || !aligned16(beta) ||
        !aligned16(S0) || !aligned16(S_final) || !aligned4(lengths))
        return MLSTM_ERR_INVALID_ARG;
    const Args a = make_args(q, k, v, g, beta, lengths, dt, B, NH, NHV, S, DK, DV, scale, S0, stream);
    if ((st = check_workspace(workspace, workspace_bytes, plan(nullptr, a, false, nullptr))) != MLSTM_OK) return st;
    Workspace w = {};
    plan(static_cast<char *>(workspace), a, false, &w);
    if (S == 0) {
        cudaError_t e = cudaMemsetAsync(w.status, 0, sizeof(uint32_t), a.stream);
        if (e == cudaSuccess && S_final && S_final != S0)
            e = launch_state_copy(S0, S_final, (size_t)B * NHV * DK * DV, a.stream);
        return cuda_status(e);
    }
    cudaError_t e;
    if (w.TG) {
        Maps m;
        if (!make_maps(a, &m)) return MLSTM_ERR_CUDA;
        e = launch_prep_tc(a, w, m);
        if (e == cudaSuccess) e = launch_forward_tc(a, w, m, o, S_final);
    } else {
        e = launch_prep(a, w, false);
        if (e == cudaSuccess) e = launch_walk(a, w, o, S_final, false);
    }
    return cuda_status(e);
}

mlstm_status gdelta_step(float *state, const void *q, const void *k, const void *v, const float *g,
                         const float *beta, mlstm_dtype dt, int B, int NH, int NHV, int DK, int DV, float scale,
                         void *o, void *stream)
{
    const mlstm_status st = check_heads(dt, B, NH, NHV, DK, DV);
    if (st != MLSTM_OK) return st;
    if ((long long)B * NHV * (DV / 8) > 0x7fffffffll) return MLSTM_ERR_UNSUPPORTED;   // CTAs, at most one for 8 columns
    if (B == 0) return MLSTM_OK;
    if (!state || !q || !k || !v || !g || !beta || !o) return MLSTM_ERR_INVALID_ARG;
    if (!aligned16(state) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(g) ||
        !aligned4(beta))
        return MLSTM_ERR_INVALID_ARG;
    StepArgs a = {state, q, k, v, g, beta, o, B * NHV, NH, NHV, DK, DV, scale, dt == MLSTM_BF16,
                  static_cast<cudaStream_t>(stream)};
    return cuda_status(gdelta::launch_step(a));
}

mlstm_status gdelta_bwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                        const int *lengths, const float *S0, const void *d_o, const float *dS_final,
                        mlstm_dtype dt, int B, int NH, int NHV, int S, int DK, int DV, float scale, void *dq,
                        void *dk, void *dv, float *dg, float *dbeta, float *dS0, void *workspace,
                        size_t workspace_bytes, void *stream)
{
    mlstm_status st = check_shape(dt, B, NH, NHV, S, DK, DV);
    if (st != MLSTM_OK) return st;
    if (B == 0) return MLSTM_OK;
    if (S > 0 && (!q || !k || !v || !g || !beta || !d_o || !dq || !dk || !dv || !dg || !dbeta))
        return MLSTM_ERR_INVALID_ARG;
    const void *all[] = {q, k, v, g, beta, S0, d_o, dS_final, dq, dk, dv, dg, dbeta, dS0};
    for (const void *p : all)
        if (!aligned16(p)) return MLSTM_ERR_INVALID_ARG;
    if (!aligned4(lengths)) return MLSTM_ERR_INVALID_ARG;
    const Args a = make_args(q, k, v, g, beta, lengths, dt, B, NH, NHV, S, DK, DV, scale, S0, stream);
    if ((st = check_workspace(workspace, workspace_bytes, plan(nullptr, a, true, nullptr))) != MLSTM_OK) return st;
    Workspace w = {};
    plan(static_cast<char *>(workspace), a, true, &w);
    if (S == 0) {
        cudaError_t e = cudaMemsetAsync(w.status, 0, sizeof(uint32_t), a.stream);
        if (e == cudaSuccess && dS0 && dS0 != dS_final)
            e = launch_state_copy(dS_final, dS0, (size_t)B * NHV * DK * DV, a.stream);
        return cuda_status(e);
    }
    cudaError_t e;
    if (w.TG) {
        Maps m;
        if (!make_maps(a, &m)) return MLSTM_ERR_CUDA;
        e = launch_prep_tc(a, w, m);
        if (e == cudaSuccess) e = launch_keep_tc(a, w, m);
        if (e == cudaSuccess) e = launch_reverse_tc(a, w, m, d_o, dS_final, dv, dS0);
        if (e == cudaSuccess) e = launch_grad_tc(a, w, m, d_o, dq, dk, dg, dbeta);
    } else {
        e = launch_prep(a, w, true);
        if (e == cudaSuccess) e = launch_walk(a, w, nullptr, nullptr, true);
        if (e == cudaSuccess) e = launch_reverse(a, w, d_o, dS_final, dv, dS0);
        if (e == cudaSuccess) e = launch_grad(a, w, d_o, dq, dk, dg, dbeta);
    }
    return cuda_status(e);
}

}  // extern "C"
