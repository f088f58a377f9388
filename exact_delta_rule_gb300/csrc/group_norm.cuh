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
    float *ws;               // gn_ws(..) floats
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
// Rows a CTA of the whole-row backward shares out among `parts` CTAs a block of channels: three CTAs a SM.
inline int gn_blocks(int C, int G, efla_dtype t) {
    const int per = 32 / gn_team(C / G / gn_vec(t));
    return (G + per - 1) / per;
}
inline int gn_row_parts(int rows, int C, int G, efla_dtype t) {
    const int most = std::max(1, 456 / gn_blocks(C, G, t));
    return std::max(1, std::min(most, (rows + 7) / 8));
}
// Vectors of a row that a CTA's threads cover in the other kernels: up to 32, rows cut evenly (40: 20, not 32 and 8), and
// the chunks its positions come in: CTAs enough for four a SM, four positions a thread at least.
inline int gn_lanes(int vecs) {
    const int blocks = std::max(1, (vecs + 31) / 32);
    return std::max(1, (vecs + blocks - 1) / blocks);
}
inline int gn_chunks(int rows, int L, int C, efla_dtype t) {
    const int vecs = C / gn_vec(t), lanes = gn_lanes(vecs), subs = GN_NT / lanes;
    const long long blocks = (long long)rows * ((vecs + lanes - 1) / lanes);
    const long long want = blocks > 0 ? (608 + blocks - 1) / blocks : 1, most = std::max(1, L / (4 * subs));
    return (int)std::max(1LL, std::min(want, most));
}
// The same where the rows are summed over too: chunks of all rows' positions.
inline int gn_column_chunks(int rows, int L, int C, efla_dtype t) {
    const int vecs = C / gn_vec(t), lanes = gn_lanes(vecs), subs = GN_NT / lanes, blocks = (vecs + lanes - 1) / lanes;
    const long long most = std::max(1LL, (long long)rows * L / (4 * subs));
    return (int)std::max(1LL, std::min<long long>(608 / blocks, most));
}
// Samples (rows) that lie in shared memory, one a warp: few elements, or many rows of up to 16 KB.  The warps a CTA.
inline bool gn_warps(int rows, int L, int C, efla_dtype t) {
    const long long n = (long long)L * C;
    return n <= 1024 || (n * (t == EFLA_BF16 ? 2 : 4) <= 16384 && rows >= 608);
}
// Forward, other samples: a tile of whole groups and whole vectors of a sample in the shared memory of a cluster of
// `cluster` CTAs, which share out its positions.  vecs = 0: it does not fit.
struct GnSlab {
    int vecs, tiles, cluster, each;  // vectors a row of the tile; tiles; CTAs; positions a CTA
};
inline GnSlab gn_slab(int rows, int L, int C, int G, efla_dtype t) {
    const int V = gn_vec(t), cg = C / G;
    int unit = cg;  // least common multiple with a vector
    while (unit % V) unit += cg;
    int vecs = unit / V;
    const int units = C / unit;
    if (vecs > GN_NT) return {0, 0, 0, 0};
    for (int m = 1; m <= units && unit / V * m <= 16; ++m)  // up to 256 bytes of a row where groups are small
        if (units % m == 0) vecs = unit / V * m;
    const int tiles = C / V / vecs, subs = GN_NT / vecs;
    const long long bytes = (long long)L * vecs * 16;
    int k = 1;
    while (k < 8 && (bytes / k > 64 * 1024 || ((long long)rows * tiles * k < 152 && L / k > 2 * subs))) k *= 2;
    const int each = (L + k - 1) / k;
    if ((long long)each * vecs * 16 > 160 * 1024) return {0, 0, 0, 0};
    return {vecs, tiles, k, each};
}
// A group of a sample, of whole vectors (two side by side at least where a sample has several positions), in the
// registers of a team of threads, 8192 elements at most: the team's threads and the vectors of each.
struct GnTeam {
    int threads, each;
};
inline GnTeam gn_group(int L, int C, int G, efla_dtype t) {
    const int V = gn_vec(t), cg = C / G;
    const long long n = (long long)L * cg;
    if (cg % V || (L > 1 && cg < 2 * V) || n > 8192 || n <= 32 * V) return {0, 0};
    const int vecs = (int)(n / V);
    return vecs <= 512 ? GnTeam{std::max(64, gn_team(vecs)), 1} : GnTeam{512, vecs <= 1024 ? 2 : 4};
}
// The CTAs of a group, which share its samples: of 256 threads six a SM forward and three backward, of 512 half as
// many, all groups together.
inline int gn_group_parts(int rows, int G, const GnTeam &k, bool bwd) {
    const int at_once = k.threads < GN_NT ? GN_NT / k.threads : 1, most = std::max(1, (k.threads > GN_NT ? (bwd ? 304 : 456) : bwd ? 456 : 912) / G);
    return std::max(1, std::min(most, (rows + at_once - 1) / at_once));
}
// Which way a call goes.
enum class GnWay { ROWS, WARP, GROUP, SLAB, GENERAL };
inline GnWay gn_way(int rows, int L, int C, int G, efla_dtype t, bool bwd) {
    if (gn_whole(L, C, G, t)) return GnWay::ROWS;
    if ((long long)L * C > 1024 && gn_group(L, C, G, t).threads) return GnWay::GROUP;
    if (gn_warps(rows, L, C, t)) return GnWay::WARP;
    return !bwd && gn_slab(rows, L, C, G, t).vecs ? GnWay::SLAB : GnWay::GENERAL;
}
inline size_t gn_ws(int rows, int L, int C, int G, efla_dtype t, bool bwd) {
    const GnWay way = gn_way(rows, L, C, G, t, bwd);
    if (way == GnWay::GENERAL) return (size_t)rows * gn_chunks(rows, L, C, t) * 2 * C + (size_t)rows * G * 2;
    if (!bwd) return 0;
    return 2 * (size_t)C * (way == GnWay::ROWS    ? gn_row_parts(rows, C, G, t)
                            : way == GnWay::GROUP ? gn_group_parts(rows, G, gn_group(L, C, G, t), true)
                                                  : gn_column_chunks(rows, L, C, t));
}

cudaError_t launch_group_norm(const GroupNormArgs &a);
cudaError_t launch_group_norm_bwd(const GroupNormArgs &a);

}  // namespace efla
