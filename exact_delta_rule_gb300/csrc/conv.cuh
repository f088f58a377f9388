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
// Threads a CTA; of the backward, and the places of its runs.
constexpr int CONV_NT = 256, CONV_BWD_NT = 128, CONV_BWD_ROWS = 37;
// Runs of CONV_BWD_ROWS places of a row extended by the W - 1 of its state, and the CTAs a block of channels that
// share them: all that there are up to six a SM.
inline int conv_bwd_runs(int T, int W) { return (int)(((long long)T + W - 1 + CONV_BWD_ROWS - 1) / CONV_BWD_ROWS); }
inline int conv_bwd_parts(int B, int T, int D, int W) {
    const int vecs = D / 4, lanes = conv_lanes(vecs), cblocks = (vecs + lanes - 1) / lanes, subs = CONV_BWD_NT / lanes;
    const long long tiles = ((long long)B * conv_bwd_runs(T, W) + subs - 1) / subs, most = 152 * 6 / cblocks;
    return (int)std::max(1LL, std::min(tiles, most));
}

cudaError_t launch_conv(const ConvArgs &a);
cudaError_t launch_conv_bwd(const ConvArgs &a);
cudaError_t launch_conv_step(const ConvArgs &a);  // x, y [B, D], state0 == state_T updated in place

}  // namespace efla
