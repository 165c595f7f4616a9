// gdelta_internal.h -- launch descriptors of the gated delta rule's kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mlstm {
namespace gdelta {

constexpr int CH = 64;   // tokens per chunk

struct Args {
    const void *q, *k, *v;
    const float *g, *beta;
    const int *lengths;
    const float *S0;
    int B, NH, NHV, S, DK, DV;
    float scale;
    bool bf16;
    cudaStream_t stream;
};

// Device workspace, carved from the caller's buffer.  NC = ceil(S / 64) chunks per value head; arrays
// over tokens hold whole chunks, [BHV][NC][64].
struct Workspace {
    uint32_t *status;      // bounded-wait status word (0 = fine)
    int NC;
    float2 *A;             // [BHV][NC][64] cumulative log gate of the chunk as value and residue: natural logarithms,
                           // but on the tensor-core path, whose kernels alone read them there, binary ones
    float *T, *P, *KK;     // [BHV][NC][64][64] (row i, column j); KK the backward only
    float2 *GB;            // tensor-core path: [BHV][NC][64] e^a, and beta e^{a_64 - a}
    uint8_t *TG;           // tensor-core path: [BHV][NC] blocks of 32 KB, T - I and G as bf16 parts
    uint8_t *TL;           // tensor-core path: [BHV][NC] blocks of 8 KB, the third part of T - I
    uint8_t *GL;           // the same of G, the backward only
    // the backward
    float *SC, *DSC;       // [BHV][NC][DK][DV] states at the chunks' starts, gradients at their ends
    float *E, *DV;         // [BHV][NC][64][DV]
};

// The chunk's own matrices: A, T, P and (with `kk`) KK.
cudaError_t launch_prep(const Args &a, const Workspace &w, bool kk);
// Forward walk: o and S_final (`keep` false), or the chunk-start states and E (`keep`).
cudaError_t launch_walk(const Args &a, const Workspace &w, void *o, float *S_final, bool keep);
// Reverse walk: dv, dS0 and the workspace's DSC, DV.
cudaError_t launch_reverse(const Args &a, const Workspace &w, const void *d_o, const float *dS_final, void *dv,
                           float *dS0);
// dq, dk, dg, dbeta of every chunk from the workspace.
cudaError_t launch_grad(const Args &a, const Workspace &w, const void *d_o, void *dq, void *dk, float *dg,
                        float *dbeta);
// The same on the tensor cores, for the shapes that tc_supported names (workspace: GB, TG).  The kernels
// of one call share the tensor maps of q and k.
struct Maps { CUtensorMap q, k; };
bool tc_supported(bool bf16, int DK, int DV);
bool make_maps(const Args &a, Maps *m);
cudaError_t launch_prep_tc(const Args &a, const Workspace &w, const Maps &m);
cudaError_t launch_forward_tc(const Args &a, const Workspace &w, const Maps &m, void *o, float *S_final);
cudaError_t launch_keep_tc(const Args &a, const Workspace &w, const Maps &m);
cudaError_t launch_reverse_tc(const Args &a, const Workspace &w, const Maps &m, const void *d_o, const float *dS_final,
                              void *dv, float *dS0);
cudaError_t launch_grad_tc(const Args &a, const Workspace &w, const Maps &m, const void *d_o, void *dq, void *dk,
                           float *dg, float *dbeta);
cudaError_t launch_state_copy(const float *S0, float *S_final, size_t n, cudaStream_t stream);

struct StepArgs {
    float *state;
    const void *q, *k, *v;
    const float *g, *beta;
    void *o;
    int BHV, NH, NHV, DK, DV;
    float scale;
    bool bf16;
    cudaStream_t stream;
};
cudaError_t launch_step(const StepArgs &a);

}  // namespace gdelta
}  // namespace mlstm
