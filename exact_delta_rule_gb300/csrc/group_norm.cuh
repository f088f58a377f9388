// Launchers of the group norm (group_norm.cu, where the formulas are).
#pragma once

#include <algorithm>

#include "internal.cuh"

namespace efla {

struct GroupNormArgs {
    const void *x;           // [rows, L, C]
    const float *w, *b;      // [C] or nullptr (1, 0)
    void *y;
    float *stats;            // [rows, G, 2]: mean, 1 / sqrt(var + eps); forward: an output or nullptr, backward: an input
    const void *dy;          // backward
    void *dx;
    float *dw, *db;          // [C] or nullptr
    float *ws;               // group_norm_ws(..) floats
    int rows, L, C, G;
    efla_dtype dtype;
    int silu;
    float eps;
    cudaStream_t stream;
};

constexpr int GN_NT = 256;

// Channels of a 16-byte vector, the lanes that hold one group of a row (a power of two), and whether the rows are
// taken whole, a group in the registers of its lanes: L = 1 and groups of whole vectors, 32 at most.
inline int gn_vec(efla_dtype t) { return t == EFLA_BF16 ? 8 : 4; }
inline int gn_team(int vecs) {
    int n = 1;
    while (n < vecs) n *= 2;
    return n;
}
inline bool gn_whole(int L, int C, int G, efla_dtype t) { return L == 1 && C / G % gn_vec(t) == 0 && C / G <= 32 * gn_vec(t); }
// Rows a CTA of the whole-row backward shares out among `parts` CTAs a block of channels: two CTAs a SM.
inline int gn_blocks(int C, int G, efla_dtype t) {
    const int per = 32 / gn_team(C / G / gn_vec(t));
    return (G + per - 1) / per;
}
inline int gn_row_parts(int rows, int C, int G, efla_dtype t) {
    const int most = std::max(1, 304 / gn_blocks(C, G, t));
    return std::max(1, std::min(most, (rows + 7) / 8));
}
// Vectors of a row that a CTA's threads cover in the other kernels, and the chunks its positions come in: CTAs
// enough for four a SM, four positions a thread at least.
inline int gn_lanes(int vecs) { return std::min(32, gn_team(vecs)); }
inline int gn_chunks(int rows, int L, int C, efla_dtype t) {
    const int vecs = C / gn_vec(t), lanes = gn_lanes(vecs), subs = GN_NT / lanes;
    const long long blocks = (long long)rows * ((vecs + lanes - 1) / lanes);
    const long long want = blocks > 0 ? (608 + blocks - 1) / blocks : 1, most = std::max(1, L / (4 * subs));
    return (int)std::max(1LL, std::min(want, most));
}
inline size_t gn_ws(int rows, int L, int C, int G, efla_dtype t, bool bwd) {
    if (gn_whole(L, C, G, t)) return bwd ? (size_t)gn_row_parts(rows, C, G, t) * 2 * C : 0;
    return (size_t)rows * gn_chunks(rows, L, C, t) * 2 * C + (size_t)rows * G * 2;
}

cudaError_t launch_group_norm(const GroupNormArgs &a);
cudaError_t launch_group_norm_bwd(const GroupNormArgs &a);

}  // namespace efla
