// Launchers of the short causal convolution before a token mixer (conv.cu, where the formulas are).
#pragma once

#include <algorithm>

#include "internal.cuh"

namespace efla {

struct ConvArgs {
    const void *x;            // [B, T, D]
    const float *w, *bias;    // [D, W], [D] or nullptr
    const void *state0;       // [N, W - 1, D] or nullptr
    const int32_t *cu_seqlens;
    void *y, *state_T;        // y may be nullptr in the backward
    const void *dy, *dstate_T;  // backward
    void *dx, *dstate0;
    float *dw, *dbias;
    float *ws;                // backward: conv_bwd_parts(..) x D (W + 1) floats
    int B, T, D, W, N;
    efla_dtype dtype;
    int silu;
    cudaStream_t stream;
    int *status;
};

// Vectors a row of a CTA's threads covers (forward: 16 bytes, backward: 4 channels), a power of two up to 32.
inline int conv_lanes(int vecs) {
    int n = 1;
    while (n < vecs && n < 32) n *= 2;
    return n;
}
constexpr int CONV_NT = 256, CONV_BWD_NT = 128;  // threads a CTA; of the backward
// Runs of `run` places of a row extended by the W - 1 of its state, and the CTAs a block of channels that share them:
// one a tile of runs, or as many as are resident at once (three a SM).
inline int conv_bwd_run(efla_dtype t) { return t == EFLA_BF16 ? 32 : 16; }
inline int conv_bwd_runs(int T, int W, int run) { return (int)(((long long)T + W - 1 + run - 1) / run); }
inline int conv_bwd_parts(int B, int T, int D, int W, int run) {
    const int vecs = D / 4, lanes = conv_lanes(vecs), cblocks = (vecs + lanes - 1) / lanes, subs = CONV_BWD_NT / lanes;
    const long long tiles = ((long long)B * conv_bwd_runs(T, W, run) + subs - 1) / subs, most = std::max(1, 152 * 3 / cblocks);
    if (tiles <= most) return (int)std::max(1LL, tiles);
    const long long each = (tiles + most - 1) / most;  // (the same number for nearly all)
    return (int)((tiles + each - 1) / each);
}

cudaError_t launch_conv(const ConvArgs &a);
cudaError_t launch_conv_bwd(const ConvArgs &a);
cudaError_t launch_conv_step(const ConvArgs &a);  // x, y [B, D], state0 == state_T updated in place

}  // namespace efla
