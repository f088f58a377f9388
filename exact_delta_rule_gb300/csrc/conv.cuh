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
    float *ws;                // backward: ConvRuns::parts x D (W + 1) floats
    int B, T, D, W, N;
    efla_dtype dtype;
    int silu;
    cudaStream_t stream;
    int *status;
};

// Vectors of 4 channels that a row of a CTA's threads covers, a power of two up to 32.
inline int conv_lanes(int vecs) {
    int n = 1;
    while (n < vecs && n < 32) n *= 2;
    return n;
}
constexpr int CONV_NT = 256;  // threads a CTA of the forward
constexpr int CONV_BWD_NT = 128, CONV_BWD_CTAS = 3, CONV_BWD_GROUP = 6;  // of the backward; its CTAs a SM; rows a group of copies
// The backward's runs: of `run` places (whole groups) of a row extended by the W - 1 of its state, row_runs a row, and
// `parts` CTAs a block of channels that share them.  Runs are as long as fills the GPU once, twice, .. or four times over,
// whichever takes the fewest places one after the other, 8 more a run for those before it and the start of its copies.
struct ConvRuns {
    int run, row_runs, parts;
};
inline ConvRuns conv_bwd_runs(int B, int T, int D, int W) {
    const int vecs = D / 4, lanes = conv_lanes(vecs), cblocks = (vecs + lanes - 1) / lanes, subs = CONV_BWD_NT / lanes;
    const long long most = std::max(1, 152 * CONV_BWD_CTAS / cblocks), ends = (long long)T + W - 1;
    ConvRuns best{};
    long long least = 0;
    for (int fill = 1; fill <= 4; ++fill) {
        const long long want = std::max(1LL, std::min(fill * most * subs / std::max(1, B), ends / (4 * CONV_BWD_GROUP)));
        const long long run = ((ends + want - 1) / want + CONV_BWD_GROUP - 1) / CONV_BWD_GROUP * CONV_BWD_GROUP;
        const long long row_runs = (ends + run - 1) / run, tiles = std::max(1LL, (B * row_runs + subs - 1) / subs);
        const long long each = (tiles + most - 1) / most, time = each * (run + 8);
        if (fill > 1 && time >= least) continue;
        least = time;
        best.run = (int)run, best.row_runs = (int)row_runs, best.parts = (int)((tiles + each - 1) / each);
    }
    return best;
}

cudaError_t launch_conv(const ConvArgs &a);
cudaError_t launch_conv_bwd(const ConvArgs &a);
cudaError_t launch_conv_step(const ConvArgs &a);  // x, y [B, D], state0 == state_T updated in place

}  // namespace efla
