// Launchers of the norms around a token mixer (mixer_norm.cu, where the formulas are).
#pragma once

#include "internal.cuh"

namespace efla {

struct MixerPrepArgs {
    const void *q, *k;                  // [tokens, Hk, d]
    const void *a, *b;                  // [tokens, H]
    const float *A_log, *dt_bias;       // [H]
    void *q_out, *k_out;                // forward outputs
    float *g_out, *beta_out;
    const void *dq_in, *dk_in;          // backward: gradients of the outputs
    const float *dg_in, *dbeta_in;
    void *dq_out, *dk_out, *da_out, *db_out;
    float *dA_log, *ddt_bias;
    float *ws;                          // backward: mixer_prep_parts(tokens) x 2 H floats
    long long tokens;
    int Hk, H, d;
    efla_dtype dtype;
    float scale, eps;
    cudaStream_t stream;
};
// CTAs a group of 32 heads whose sums the second stage adds: 64 tokens or more each, two CTAs a SM at most.
inline int mixer_prep_parts(long long tokens) {
    const long long n = (tokens + 63) / 64;
    return (int)(n < 1 ? 1 : n < 304 ? n : 304);
}

struct NormGateArgs {
    const void *o, *z;                  // [rows, d]
    const float *w;                     // [d]
    void *y;
    const void *dy;                     // backward
    void *do_, *dz;
    float *dw;
    float *ws;                          // backward: NORM_GATE_PARTS x d floats
    long long rows;
    int d;
    efla_dtype dtype;
    float eps;
    cudaStream_t stream;
};
constexpr int NORM_GATE_PARTS = 152 * 2;  // the CTAs that are resident at once (100 registers a thread)

// out0[i] (i < split), out1[i - split] = the sums over `parts` rows of n floats, in one fixed order (nullptr: not written).
cudaError_t launch_sum_parts(const float *ws, int parts, int n, float *out0, float *out1, int split, cudaStream_t stream);
cudaError_t launch_mixer_prep(const MixerPrepArgs &p, bool bwd);
cudaError_t launch_norm_gate(const NormGateArgs &p, bool bwd);

}  // namespace efla
