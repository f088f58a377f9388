// Group norm with its activation, channels last: x [rows, L, C], G groups of C / G neighbouring channels, statistics
// over the L positions and the channels of a group (L = 1: of a token's heads).
//   n = (x - mean) r,  r = 1 / sqrt(var + eps),   s = w n + b,   y = s or silu(s)
//   ds = dy or dy silu'(s),  dn = ds w,  dx = r (dn - mean(dn) - n mean(dn n)),  dw = sum ds n,  db = sum ds
//
// Bound by HBM: x (and dy) read, y (dx) written.  Which way a call goes:
//   L = 1 and groups of whole vectors up to 32 of them: a group of a row lies in the registers of its lanes, whose sums
//     are shuffles; one pass, the next rows' copies under way (16384 rows of 16 groups of 128, bf16: forward 24 us for
//     134 MB, backward with its sums 38 for 202; 65536 rows 86 and 128, 6.2 TB/s; 92 and 144 with four rows loaded together);
//   groups of whole vectors and up to 8192 elements of a sample: in the registers of 64 to 512 threads; one pass, bound by the
//     exchange of its sums (shuffles, shared memory, barriers) and by issue (16384 rows of 2048 in one group, bf16: forward 38 us, with gradients 92; 51 and
//     189 as a warp's samples; 4096 samples of 16 x 256 in 8 groups 21 and 55; 94 and 238 a warp);
//   samples of few elements, or many of up to 16 KB: one a warp, in shared memory;
//   forward, other samples: tiles of whole groups in the shared memory of a cluster, whose CTAs share out the positions
//     and read one another's sums; one pass (8 maps of 4096 positions x 320 channels in 32 groups: 17 us, three kernels 24; 64 maps 103, 124);
//   the rest in three kernels: sums per channel over chunks of the positions, joined to those of the groups, and
//     applied, where x is found in L2 if it fits (backward of 64 maps of 4096 x 320, bf16: 97 us, 3 and 116; one position
//     at a time and rows cut into 32 vectors and 8: 251, 3 and 167).
// So that neither a mean far from 0 nor a first value far from the others spoils a variance: the three kernels sum a channel to its
// mean and square deviation four positions at a time and join these; a cluster sums x minus the channel's first value, and
// once more from the mean where that value is far from it; where a group is in registers or a warp's memory its mean is taken first.
#include <type_traits>

#include "group_norm.cuh"
#include "mixer_norm.cuh"
#include "vec.cuh"

namespace efla {
namespace {

constexpr int NT = GN_NT;
__host__ __device__ constexpr int gn_group_depth(int each) { return each > 2 ? 2 : 3; }  // samples of the ring

template <bool SILU>
__device__ __forceinline__ float act(float s) { return SILU ? s * quick_sigmoid(s) : s; }
template <bool SILU>
__device__ __forceinline__ float dact(float s) {
    if (!SILU) return 1.f;
    const float g = quick_sigmoid(s);
    return g * fmaf(s, 1.f - g, 1.f);
}

template <int V>
__device__ __forceinline__ void affine(const GroupNormArgs &p, int c0, float (&w)[V], float (&b)[V]) {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
        const float4 ww = p.w ? *reinterpret_cast<const float4 *>(p.w + c0 + e) : make_float4(1.f, 1.f, 1.f, 1.f);
        const float4 bb = p.b ? *reinterpret_cast<const float4 *>(p.b + c0 + e) : make_float4(0.f, 0.f, 0.f, 0.f);
        w[e] = ww.x, w[e + 1] = ww.y, w[e + 2] = ww.z, w[e + 3] = ww.w;
        b[e] = bb.x, b[e + 1] = bb.y, b[e + 2] = bb.z, b[e + 3] = bb.w;
    }
}

// Value e of a vector, by itself.
__device__ __forceinline__ float value(const uint4 &r, int e, float) { return __uint_as_float((&r.x)[e]); }
__device__ __forceinline__ float value(const uint4 &r, int e, __nv_bfloat16) {
    const uint32_t w = (&r.x)[e / 2];
    return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
}

// Mean and sum of squared deviations of a thread's channels over the positions it has seen, a few at a time: those of a
// batch are measured from the mean so far, so that no value, be it the first or one far from all others, costs the others'
// accuracy (a sum of squares from one fixed value, less the square of its mean, would lose it).  The mean is kept as its
// difference from the thread's first position, and so free of how far all of them are from 0.
template <typename T>
struct Running {
    static constexpr int V = Vec<T>::N;
    float first[V], mean[V], dev[V];
    int n = 0;
    __device__ __forceinline__ void start(const uint4 &f) {
        Vec<T>::unpack(f, first);
#pragma unroll
        for (int e = 0; e < V; ++e) mean[e] = dev[e] = 0.f;
    }
    // `have` (1 to M) positions.  With a = sum d, d = f - mean: the mean moves by a / (n + have), dev grows by
    // sum d^2 - a^2 / (n + have), of which at least a fifth of the sum is left (M = 4, d of the very first is 0).
    template <int M>
    __device__ __forceinline__ void add(const uint4 (&f)[M], int have) {
        n += have;
        const float inv = 1.f / (float)n;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float a = 0.f, q = 0.f;
#pragma unroll
            for (int i = 0; i < M; ++i) {
                const float d = i < have ? (value(f[i], e, T()) - first[e]) - mean[e] : 0.f;
                a += d;
                q = fmaf(d, d, q);
            }
            const float move = a * inv;
            mean[e] += move;
            dev[e] += fmaf(-a, move, q);
        }
    }
};
// Pieces of n values each, with their means and deviations, are joined in two walks: a first mean m0 = sum n mean / N; then from
// there what it lacks, rest = sum n (mean - m0), and the deviations.  The mean is m0 + rest / N, which leaves it one rounding of
// its own size, and the deviations from it are less by rest^2 / N (not below 0: pieces that are all the same).
__device__ __forceinline__ void join_end(float m0, float rest, float count, float &mean, float &dev) {
    const float move = rest / count;
    mean = m0 + move;
    dev = fmaf(-rest, move, dev);
    dev = dev < 0.f ? 0.f : dev;
}
// The `channels` channels of a CTA, over `len` > 0 positions, from those of its `subs` threads a vector that have every subs-th of
// them: thread k's at means[k step + at(channel)] and devs[..]; done(channel, mean, dev).  As many neighbouring lanes a channel
// as there are threads for.
template <typename At, typename Done>
__device__ __forceinline__ void join_threads(const float *means, const float *devs, int step, int subs, long long len, int channels, At at,
                                             Done done) {
    int split = 1;
    while (split < 32 && 2 * split * channels <= NT) split *= 2;
    const int part = threadIdx.x % split;
    const float some = (float)(len / subs);
    const int more = (int)(len % subs), have = some > 0.f ? subs : more;
    auto over_lanes = [&](float v) {
        for (int off = 1; off < split; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        return v;
    };
    for (int i0 = 0; i0 < channels; i0 += NT / split) {  // (the same for a CTA)
        const int i = i0 + threadIdx.x / split, off = i < channels ? at(i) : 0;
        float m0 = 0.f, rest = 0.f, mean, dev = 0.f;
#pragma unroll 4
        for (int k = part; k < have; k += split) m0 = fmaf(k < more ? some + 1.f : some, means[k * step + off], m0);
        m0 = over_lanes(m0) / (float)len;
#pragma unroll 4
        for (int k = part; k < have; k += split) {
            const float d = means[k * step + off] - m0, nd = (k < more ? some + 1.f : some) * d;
            rest += nd;
            dev += fmaf(nd, d, devs[k * step + off]);
        }
        rest = over_lanes(rest);
        dev = over_lanes(dev);
        join_end(m0, rest, (float)len, mean, dev);
        if (i < channels && part == 0) done(i, mean, dev);
    }
}

// ------------------------------------------------------------------------------------ whole rows (L = 1)
// A warp holds 32 / TEAM groups of a row, a group in the first C / G / V lanes of its TEAM; a CTA 8 rows of one block
// of groups, and every parts-th 8 rows after them; a warp's rows come through a ring of copies into its threads' own slots.
template <typename T, int TEAM, bool BWD, bool SILU>
__global__ void __launch_bounds__(NT) gn_rows_kernel(GroupNormArgs p, int blocks, int parts) {
    constexpr int V = Vec<T>::N, PER = 32 / TEAM, SUBS = NT / 32, DEPTH = 4;
    constexpr int SLOTS = DEPTH * NT, SUMS = BWD ? SUBS * 32 * V : 0;  // (the sums take the place of the copies)
    constexpr int BYTES = SLOTS * (BWD ? 40 : 16);
    static_assert(SUMS * 4 <= BYTES, "the sums");
    __shared__ __align__(16) uint8_t shared[BYTES];
    uint4 *xs = reinterpret_cast<uint4 *>(shared) + threadIdx.x, *ds = xs + SLOTS;  // slot i at [i NT]
    float2 *ss = reinterpret_cast<float2 *>(shared + SLOTS * 32) + threadIdx.x;
    const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5, l = lane % TEAM;
    const int block = blockIdx.x % blocks, part = blockIdx.x / blocks;
    const int g = block * PER + lane / TEAM, gv = p.C / p.G / V, vecs = p.C / V;
    const bool live = g < p.G && l < gv;
    const int v = live ? g * gv + l : min(g, p.G - 1) * gv;  // (of the same group: what its parameters do stays in it)
    const float inv = 1.f / (float)(p.C / p.G);
    float w[V], b[V], dw[V] = {}, db[V] = {};
    affine(p, v * V, w, b);
    const long long step = (long long)parts * SUBS, first = (long long)part * SUBS + sub;
    // A row's copies, zeros for what is not there: nothing in any sum
    auto fetch_row = [&](long long row, int slot) {
        if (row < p.rows) {
            const long long at = row * vecs + v;
            fetch(xs + slot * NT, static_cast<const uint4 *>(p.x) + at, live);
            if (BWD) {
                fetch(ds + slot * NT, static_cast<const uint4 *>(p.dy) + at, live);
                fetch(ss + slot * NT, reinterpret_cast<const float2 *>(p.stats) + (live ? row * p.G + g : 0), live);
            }
        }
        fetch_commit();
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) fetch_row(first + i * step, i);
    for (long long row0 = first; row0 < p.rows; row0 += step * DEPTH) {  // (the same for a warp)
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            const long long row = row0 + i * step;
            if (row >= p.rows) break;
            fetch_wait(DEPTH - 1);
            const uint4 rx = xs[i * NT], rd = BWD ? ds[i * NT] : rx;
            const float2 st = BWD ? ss[i * NT] : make_float2(0.f, 0.f);
            float x[V];
            Vec<T>::unpack(rx, x);
            if (!BWD) {
                float m = 0.f, q = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) m += x[e];
                m = row_sum<TEAM>(m) * inv;
                const float off = live ? m : 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[e] -= off;
                    q = fmaf(x[e], x[e], q);
                }
                const float r = rsqrtf(row_sum<TEAM>(q) * inv + p.eps);
#pragma unroll
                for (int e = 0; e < V; ++e) x[e] = act<SILU>(fmaf(x[e] * r, w[e], b[e]));
                if (live) {
                    static_cast<uint4 *>(p.y)[row * vecs + v] = Vec<T>::pack(x);
                    if (p.stats && l == 0) reinterpret_cast<float2 *>(p.stats)[row * p.G + g] = make_float2(m, r);
                }
            } else {
                float d[V], s1 = 0.f, s2 = 0.f;
                Vec<T>::unpack(rd, d);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float n = (x[e] - st.x) * st.y;
                    d[e] *= dact<SILU>(fmaf(n, w[e], b[e]));
                    dw[e] = fmaf(d[e], n, dw[e]);
                    db[e] += d[e];
                    d[e] *= w[e];
                    x[e] = n;
                    s1 += d[e];
                    s2 = fmaf(d[e], n, s2);
                }
                s1 = row_sum<TEAM>(s1) * inv;
                s2 = row_sum<TEAM>(s2) * inv;
#pragma unroll
                for (int e = 0; e < V; ++e) x[e] = st.y * (d[e] - s1 - x[e] * s2);
                if (live) static_cast<uint4 *>(p.dx)[row * vecs + v] = Vec<T>::pack(x);
            }
            fetch_row(row + step * DEPTH, i);
        }
    }
    if (BWD) {  // the CTA's sums over its rows, in order: db then dw
        fetch_wait(0);
        float *red = reinterpret_cast<float *>(shared), *out = p.ws + (size_t)part * 2 * p.C;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < V; ++e) red[(sub * 32 + lane) * V + e] = which ? dw[e] : db[e];
            __syncthreads();
            for (int i = threadIdx.x; i < 32 * V; i += NT) {
                const int ln = i / V, gg = block * PER + ln / TEAM, ll = ln % TEAM;
                if (gg >= p.G || ll >= gv) continue;
                float s = 0.f;
#pragma unroll
                for (int k = 0; k < SUBS; ++k) s += red[k * 32 * V + i];
                out[which * p.C + (gg * gv + ll) * V + i % V] = s;
            }
        }
    }
}

// ------------------------------------------------------------------------------------ a group a team
// A group of a sample lies in the registers of TEAM threads, EACH vectors of a thread, its sums are joined through shared
// memory (two barriers forward, one backward).  A CTA has the same group of NTH / TEAM samples at a time, so that a thread's
// channels stay the same, and its samples come through a ring of copies into its own slots.
template <typename T, int TEAM, int EACH, bool BWD, bool SILU>
__global__ void __launch_bounds__(TEAM > NT ? TEAM : NT) gn_group_kernel(GroupNormArgs p, int parts) {
    constexpr int V = Vec<T>::N, NTH = TEAM > NT ? TEAM : NT, TEAMS = NTH / TEAM, DEPTH = gn_group_depth(EACH);
    constexpr int SLOTS = DEPTH * EACH * NTH;
    static_assert(!BWD || SLOTS * 32 >= NTH * EACH * V * 4, "the sums take the place of the copies");
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 joined[2][NTH / 32];
    const int tid = threadIdx.x, team = tid / TEAM, l = tid % TEAM;
    const int g = blockIdx.x % p.G, part = blockIdx.x / p.G, gv = p.C / p.G / V, vecs = p.C / V, total = p.L * gv;
    uint4 *xs = reinterpret_cast<uint4 *>(smem) + tid, *ds = xs + SLOTS;  // vector k of slot i at [(i EACH + k) NTH]
    float2 *ss = reinterpret_cast<float2 *>(smem + (size_t)SLOTS * 32) + tid;
    const float inv = 1.f / ((float)p.L * (float)(p.C / p.G));
    bool live[EACH];
    long long at[EACH];
    float w[EACH][V], b[EACH][V], dw[EACH][V] = {}, db[EACH][V] = {};
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int i = k * TEAM + l;
        live[k] = i < total;
        at[k] = live[k] ? (long long)(i / gv) * vecs + g * gv + i % gv : 0;
        affine(p, (g * gv + i % gv) * V, w[k], b[k]);
    }
    const long long sample = (long long)p.L * vecs, step = (long long)parts * TEAMS, from = (long long)part * TEAMS;
    // A sample's copies, zeros for what is not there: nothing in any sum
    auto fetch_sample = [&](long long row, int slot) {
        const bool real = row < p.rows;
        const long long base = real ? row * sample : 0;
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            fetch(xs + (slot * EACH + k) * NTH, static_cast<const uint4 *>(p.x) + base + at[k], real && live[k]);
            if (BWD) fetch(ds + (slot * EACH + k) * NTH, static_cast<const uint4 *>(p.dy) + base + at[k], real && live[k]);
        }
        if (BWD) fetch(ss + slot * NTH, reinterpret_cast<const float2 *>(p.stats) + (real ? row * p.G + g : 0), real);
        fetch_commit();
    };
    int turn = 0;  // (the buffer of the sums before last is free: every thread has been through a barrier since it read it)
    auto join = [&](float2 v) {  // (forward: of x alone)
        v.x = row_sum<32>(v.x);
        if (BWD) v.y = row_sum<32>(v.y);
        if (tid % 32 == 0) joined[turn][tid / 32] = v;
        __syncthreads();
        v = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < TEAM / 32; ++i) {
            const float2 o = joined[turn][team * (TEAM / 32) + i];
            v.x += o.x;
            if (BWD) v.y += o.y;
        }
        turn ^= 1;
        return v;
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) fetch_sample(from + team + i * step, i);
    int slot = 0;
    for (long long row0 = from; row0 < p.rows; row0 += step) {  // (the same for a CTA)
        const long long row = row0 + team;
        const bool real = row < p.rows;
        fetch_wait(DEPTH - 1);
        float x[EACH][V], d[EACH][V];
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            Vec<T>::unpack(xs[(slot * EACH + k) * NTH], x[k]);
            if (BWD) Vec<T>::unpack(ds[(slot * EACH + k) * NTH], d[k]);
        }
        if (!BWD) {
            float m = 0.f, q = 0.f;
#pragma unroll
            for (int k = 0; k < EACH; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) m += x[k][e];
            m = join(make_float2(m, 0.f)).x * inv;
#pragma unroll
            for (int k = 0; k < EACH; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[k][e] -= live[k] ? m : 0.f;
                    q = fmaf(x[k][e], x[k][e], q);
                }
            const float r = rsqrtf(join(make_float2(q, 0.f)).x * inv + p.eps);
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
#pragma unroll
                for (int e = 0; e < V; ++e) x[k][e] = act<SILU>(fmaf(x[k][e] * r, w[k][e], b[k][e]));
                if (real && live[k]) static_cast<uint4 *>(p.y)[row * sample + at[k]] = Vec<T>::pack(x[k]);
            }
            if (p.stats && real && l == 0) reinterpret_cast<float2 *>(p.stats)[row * p.G + g] = make_float2(m, r);
        } else {
            const float2 st = ss[slot * NTH];
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < EACH; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float n = live[k] ? (x[k][e] - st.x) * st.y : 0.f;
                    d[k][e] *= dact<SILU>(fmaf(n, w[k][e], b[k][e]));
                    dw[k][e] = fmaf(d[k][e], n, dw[k][e]);
                    db[k][e] += d[k][e];
                    d[k][e] *= w[k][e];
                    x[k][e] = n;
                    s.x += d[k][e];
                    s.y = fmaf(d[k][e], n, s.y);
                }
            s = join(s);
            s.x *= inv;
            s.y *= inv;
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
#pragma unroll
                for (int e = 0; e < V; ++e) x[k][e] = st.y * (d[k][e] - s.x - x[k][e] * s.y);
                if (real && live[k]) static_cast<uint4 *>(p.dx)[row * sample + at[k]] = Vec<T>::pack(x[k]);
            }
        }
        fetch_sample(row + DEPTH * step, slot);
        slot = slot + 1 == DEPTH ? 0 : slot + 1;
    }
    if (BWD) {  // the CTA's sums over its samples and their positions, in order: db then dw
        fetch_wait(0);
        float *red = reinterpret_cast<float *>(smem), *out = p.ws + (size_t)part * 2 * p.C + g * gv * V;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < EACH; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) red[((team * EACH + k) * TEAM + l) * V + e] = which ? dw[k][e] : db[k][e];
            __syncthreads();
            for (int c = tid; c < gv * V; c += NTH) {
                float s = 0.f;
                for (int t = 0; t < TEAMS; ++t)
                    for (int i = c / V; i < total; i += gv) s += red[(t * EACH * TEAM + i) * V + c % V];
                out[(size_t)which * p.C + c] = s;
            }
        }
    }
}

// ------------------------------------------------------------------------------------ sums per channel
// Backward: of ds and ds n; forward: the channel's mean and sum of squared deviations.  A CTA takes one chunk of a row's
// positions and a block of its channels: part[row chunks + chunk][2][C].  JOINT (backward): one chunk of the positions of
// all rows.
template <typename T, bool BWD, bool JOINT, bool SILU>
__global__ void __launch_bounds__(NT, BWD ? 0 : 4) gn_sums_kernel(GroupNormArgs p, int lanes, int blocks, int chunks) {
    constexpr int V = Vec<T>::N;
    __shared__ float red[NT][V + 1], red2[BWD ? 1 : NT][V + 1];
    const int tid = threadIdx.x, lane = tid % lanes, sub = tid / lanes, subs = NT / lanes;
    const int block = blockIdx.x % blocks, rc = blockIdx.x / blocks, row = JOINT ? 0 : rc / chunks, chunk = rc % chunks;
    const int vecs = p.C / V, v = block * lanes + lane, cg = p.C / p.G;
    const long long all = JOINT ? (long long)p.rows * p.L : p.L, each = (all + chunks - 1) / chunks;
    const long long from = chunk * each, to = min(all, from + each);
    float a[V] = {}, q[V] = {};
    if (v < vecs && sub < subs) {
        const uint4 *x = static_cast<const uint4 *>(p.x) + (size_t)row * p.L * vecs + v;
        float k[V], r[V], w[V], b[V];
        Running<T> run;
        if (BWD) {
            affine(p, v * V, w, b);
#pragma unroll
            for (int e = 0; e < V && !JOINT; ++e) {
                const float2 st = reinterpret_cast<const float2 *>(p.stats)[(size_t)row * p.G + (v * V + e) / cg];
                k[e] = st.x;
                r[e] = st.y;
            }
        }
        const uint4 *dy = BWD ? static_cast<const uint4 *>(p.dy) + (size_t)row * p.L * vecs + v : nullptr;
        constexpr int AT_ONCE = 4;  // positions whose loads are under way together
        for (long long t1 = from + sub; t1 < to; t1 += (long long)AT_ONCE * subs) {
            uint4 rx[AT_ONCE], rd[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const long long t = t1 + i * subs;
                rx[i] = rd[i] = make_uint4(0, 0, 0, 0);
                if (t < to) {
                    rx[i] = x[(size_t)t * vecs];
                    if (BWD) rd[i] = dy[(size_t)t * vecs];
                }
            }
            if constexpr (!BWD) {
                if (run.n == 0) run.start(rx[0]);
                int have = 1;
#pragma unroll
                for (int i = 1; i < AT_ONCE; ++i) have += t1 + i * subs < to;
                run.add(rx, have);
            } else {
#pragma unroll
                for (int i = 0; i < AT_ONCE; ++i) {
                    const long long t = t1 + i * subs;
                    if (t >= to) break;
                    float f[V], d[V];
                    Vec<T>::unpack(rx[i], f);
                    Vec<T>::unpack(rd[i], d);
                    if (JOINT) {
                        const float2 *stats = reinterpret_cast<const float2 *>(p.stats) + t / p.L * p.G;
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            const float2 st = stats[(v * V + e) / cg];
                            k[e] = st.x;
                            r[e] = st.y;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float n = (f[e] - k[e]) * r[e];
                        d[e] *= dact<SILU>(fmaf(n, w[e], b[e]));
                        a[e] += d[e];
                        q[e] = fmaf(d[e], n, q[e]);
                    }
                }
            }
        }
        if (!BWD && run.n > 0) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                a[e] = run.first[e] + run.mean[e];
                q[e] = run.dev[e];
            }
        }
    }
    if constexpr (!BWD) {  // the threads' means and deviations (of nothing where a thread had no position) to the channel's
#pragma unroll
        for (int e = 0; e < V; ++e) {
            red[tid][e] = a[e];
            red2[tid][e] = q[e];
        }
        __syncthreads();
        if (from < to)
            join_threads(&red[0][0], &red2[0][0], lanes * (V + 1), subs, to - from, min(lanes, vecs - block * lanes) * V,
                         [&](int i) { return i / V * (V + 1) + i % V; },
                         [&](int i, float mean, float dev) {
                             float *to = p.ws + (size_t)rc * 2 * p.C + (size_t)block * lanes * V + i;
                             to[0] = mean;
                             to[p.C] = dev;
                         });
    } else {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < V; ++e) red[tid][e] = which ? q[e] : a[e];
            __syncthreads();
            for (int i = tid; i < lanes * V; i += NT) {
                const int c = (block * lanes + i / V) * V + i % V;
                if (c >= p.C) continue;
                float s = 0.f;
                for (int k = 0; k < subs; ++k) s += red[k * lanes + i / V][i % V];
                p.ws[((size_t)rc * 2 + which) * p.C + c] = s;
            }
        }
    }
}

// Forward: a group's mean and r, by TEAM threads, from its pieces, each the mean and deviations of one channel of one chunk.  (A
// warp a group took 38 us for 2 maps of 65536 x 128 in 8 groups, 304 chunks: 16 warps walk through 4864 pieces each; a CTA a
// group 9.)
template <int TEAM>
__global__ void __launch_bounds__(NT) gn_moments_kernel(GroupNormArgs p, int chunks, float *out) {
    __shared__ float box[3][NT / 32];
    const int tid = threadIdx.x % TEAM, cg = p.C / p.G;
    const long long i = (long long)blockIdx.x * (NT / TEAM) + threadIdx.x / TEAM;
    if (i >= (long long)p.rows * p.G) return;  // (a CTA as a whole where TEAM is one)
    const int row = (int)(i / p.G), c0 = (int)(i % p.G) * cg;
    const float *part = p.ws + (size_t)row * chunks * 2 * p.C;
    auto sum = [&](float v, int which) {
        v = row_sum<32>(v);
        if (TEAM == 32) return v;
        if (tid % 32 == 0) box[which][tid / 32] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < TEAM / 32; ++w) v += box[which][w];
        return v;
    };
    int across = 1;
    while (across < cg && across < TEAM) across *= 2;
    const int each = (int)(((long long)p.L + chunks - 1) / chunks), filled = (p.L + each - 1) / each;
    // this thread's, one after the other: as Running's batches, the mean as its difference from the first
    float n = 0.f, near = 0.f, mean = 0.f, dev = 0.f;
    for (int c = c0 + tid % across; c < c0 + cg; c += across)
#pragma unroll 8
        for (int k = tid / across; k < filled; k += TEAM / across) {
            const float *at = part + (size_t)k * 2 * p.C + c;
            const float one = at[0], q = at[p.C], have = (float)min(p.L - k * each, each);
            if (n == 0.f) near = one;
            const float d = (one - near) - mean, before = n;
            n += have;
            const float move = __fdividef(d * have, n);
            mean += move;
            dev += fmaf(before * d, move, q);
        }
    const float count = (float)p.L * (float)cg, inv = 1.f / count;
    mean += near;
    const float m0 = sum(n * mean, 0) * inv, d = mean - m0, nd = n > 0.f ? n * d : 0.f;
    float first;
    dev = sum(n > 0.f ? fmaf(nd, d, dev) : 0.f, 1);
    join_end(m0, sum(nd, 2), count, first, dev);
    if (tid == 0) reinterpret_cast<float2 *>(out)[i] = make_float2(first, rsqrtf(dev * inv + p.eps));
}

// Backward, a warp a group of a row: mean(dn) and mean(dn n) from the channels' sums.
__global__ void __launch_bounds__(NT) gn_join_kernel(GroupNormArgs p, int chunks, float *out) {
    const int lane = threadIdx.x & 31, cg = p.C / p.G;
    const long long i = (long long)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
    if (i >= (long long)p.rows * p.G) return;
    const int row = (int)(i / p.G), c0 = (int)(i % p.G) * cg;
    const float *part = p.ws + (size_t)row * chunks * 2 * p.C;
    // a channel's sums: of its chunks by 32 / across lanes (of a group of few channels), then over these
    int across = 1;
    while (across < cg && across < 32) across *= 2;
    const bool mine = lane < across;
    auto channel = [&](int c, float &a, float &q) {
        a = q = 0.f;
        if (c < c0 + cg)
#pragma unroll 8
            for (int k = lane / across; k < chunks; k += 32 / across) {
                a += part[(size_t)k * 2 * p.C + c];
                q += part[(size_t)k * 2 * p.C + p.C + c];
            }
        for (int off = across; off < 32; off <<= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, off);
            q += __shfl_xor_sync(0xffffffffu, q, off);
        }
        return mine && c < c0 + cg;
    };
    const float inv = 1.f / ((float)p.L * (float)cg);
    float first = 0.f, second = 0.f;
    for (int c1 = 0; c1 < cg; c1 += across) {
        const int c = c0 + c1 + lane % across;
        float a, q;
        if (!channel(c, a, q)) continue;
        const float w = p.w ? p.w[c] : 1.f;
        first = fmaf(w, a, first);
        second = fmaf(w, q, second);
    }
    first = row_sum<32>(first) * inv;
    second = row_sum<32>(second) * inv;
    if (lane == 0) reinterpret_cast<float2 *>(out)[i] = make_float2(first, second);
}

// y or dx from the groups' values (`means`: backward, what gn_join_kernel gave).  A thread a vector, UNROLL positions.
template <typename T, bool BWD, bool SILU>
__global__ void __launch_bounds__(NT) gn_apply_kernel(GroupNormArgs p, int lanes, int blocks, int tiles, const float *means) {
    constexpr int V = Vec<T>::N, UNROLL = 4;
    const int tid = threadIdx.x, lane = tid % lanes, sub = tid / lanes, subs = NT / lanes;
    const int block = blockIdx.x % blocks, rt = blockIdx.x / blocks, row = rt / tiles, tile = rt % tiles;
    const int vecs = p.C / V, v = block * lanes + lane, cg = p.C / p.G;
    if (v >= vecs || sub >= subs) return;
    const uint4 *x = static_cast<const uint4 *>(p.x) + (size_t)row * p.L * vecs + v;
    const uint4 *dy = BWD ? static_cast<const uint4 *>(p.dy) + (size_t)row * p.L * vecs + v : nullptr;
    uint4 *out = static_cast<uint4 *>(BWD ? p.dx : p.y) + (size_t)row * p.L * vecs + v;
    const int t0 = tile * subs * UNROLL + sub;
    uint4 rx[UNROLL], rd[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const int t = t0 + i * subs;
        rx[i] = rd[i] = make_uint4(0, 0, 0, 0);
        if (t < p.L) {
            rx[i] = x[(size_t)t * vecs];
            if (BWD) rd[i] = dy[(size_t)t * vecs];
        }
    }
    float w[V], b[V], m[V], r[V], s1[V], s2[V];
    affine(p, v * V, w, b);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const size_t g = (size_t)row * p.G + (v * V + e) / cg;
        const float2 st = reinterpret_cast<const float2 *>(p.stats)[g];
        m[e] = st.x;
        r[e] = st.y;
        if (BWD) {
            const float2 mm = reinterpret_cast<const float2 *>(means)[g];
            s1[e] = mm.x;
            s2[e] = mm.y;
        }
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const int t = t0 + i * subs;
        float f[V], d[V];
        Vec<T>::unpack(rx[i], f);
        Vec<T>::unpack(rd[i], d);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float n = (f[e] - m[e]) * r[e], s = fmaf(n, w[e], b[e]);
            f[e] = BWD ? r[e] * (d[e] * dact<SILU>(s) * w[e] - s1[e] - n * s2[e]) : act<SILU>(s);
        }
        if (t < p.L) out[(size_t)t * vecs] = Vec<T>::pack(f);
    }
}

// ------------------------------------------------------------------------------------ a sample a warp
// x (and dy) of a sample in shared memory.  The sums of a group by TEAM lanes (a power of two, at least C / G up to 32)
// that walk through its channels one by one, as a group may begin and end inside a vector; then vector by vector.
// MANY (forward): the mean is a sum of more than 32 values by a lane, up to 1024, and what it lacks by their rounding (four
// deviations at 500 values of 30000, 0.05 apart) comes with the squares: 3 % of the time.
template <typename T, int TEAM, bool BWD, bool SILU, bool MANY>
__global__ void __launch_bounds__(NT) gn_warp_kernel(GroupNormArgs p, int bytes) {
    constexpr int V = Vec<T>::N, PER = 32 / TEAM;
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % TEAM, cg = p.C / p.G;
    const long long row = (long long)blockIdx.x * (blockDim.x / 32) + warp;
    if (row >= p.rows) return;
    const int n = p.L * p.C, vecs = n / V;
    uint8_t *mine = smem + (size_t)warp * bytes;
    T *x = reinterpret_cast<T *>(mine), *dy = x + (BWD ? n : 0);
    float2 *group = reinterpret_cast<float2 *>(mine + (size_t)(BWD ? 2 : 1) * n * sizeof(T)), *means = group + p.G;
    const uint4 *xs = static_cast<const uint4 *>(p.x) + row * vecs, *ys = BWD ? static_cast<const uint4 *>(p.dy) + row * vecs : nullptr;
#pragma unroll 4
    for (int i = lane; i < vecs; i += 32) {
        reinterpret_cast<uint4 *>(x)[i] = xs[i];
        if (BWD) reinterpret_cast<uint4 *>(dy)[i] = ys[i];
    }
    __syncwarp();
    const float inv = 1.f / ((float)p.L * (float)cg);
    float2 *stats = reinterpret_cast<float2 *>(p.stats) + row * p.G;
    for (int g0 = 0; g0 < p.G; g0 += PER) {
        const int g = g0 + lane / TEAM;
        float first = 0.f, second = 0.f;
        if (!BWD) {
            if (g < p.G)
                for (int t = 0; t < p.L; ++t)
                    for (int c = l; c < cg; c += TEAM) first += to_f32(x[t * p.C + g * cg + c]);
            const float m0 = row_sum<TEAM>(first) * inv;
            float rest = 0.f;
            if (g < p.G)
                for (int t = 0; t < p.L; ++t)
                    for (int c = l; c < cg; c += TEAM) {
                        const float d = to_f32(x[t * p.C + g * cg + c]) - m0;
                        if (MANY) rest += d;
                        second = fmaf(d, d, second);
                    }
            first = m0;
            second = row_sum<TEAM>(second) * inv;
            if (MANY) {  // as join_end
                const float move = row_sum<TEAM>(rest) * inv;
                first += move;
                second = fmaf(-move, move, second);
                second = second < 0.f ? 0.f : second;
            }
            second = rsqrtf(second + p.eps);
            if (g < p.G && l == 0) {
                group[g] = make_float2(first, second);
                if (p.stats) stats[g] = make_float2(first, second);
            }
        } else {
            const float2 st = g < p.G ? stats[g] : make_float2(0.f, 0.f);
            if (g < p.G)
                for (int t = 0; t < p.L; ++t)
                    for (int c = l; c < cg; c += TEAM) {
                        const int ch = g * cg + c;
                        const float w = p.w ? p.w[ch] : 1.f, m = (to_f32(x[t * p.C + ch]) - st.x) * st.y;
                        const float dn = to_f32(dy[t * p.C + ch]) * dact<SILU>(fmaf(m, w, p.b ? p.b[ch] : 0.f)) * w;
                        first += dn;
                        second = fmaf(dn, m, second);
                    }
            first = row_sum<TEAM>(first) * inv;
            second = row_sum<TEAM>(second) * inv;
            if (g < p.G && l == 0) {
                group[g] = st;
                means[g] = make_float2(first, second);
            }
        }
    }
    __syncwarp();
    uint4 *out = static_cast<uint4 *>(BWD ? p.dx : p.y) + row * vecs;
    const int per = p.C / V;
    for (int i = lane; i < vecs; i += 32) {
        const int c0 = i % per * V;
        int g = c0 / cg, next = (g + 1) * cg;
        float f[V], d[V], w[V], b[V];
        Vec<T>::unpack(reinterpret_cast<const uint4 *>(x)[i], f);
        if (BWD) Vec<T>::unpack(reinterpret_cast<const uint4 *>(dy)[i], d);
        affine(p, c0, w, b);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (c0 + e == next) {
                ++g;
                next += cg;
            }
            const float2 st = group[g];
            const float m = (f[e] - st.x) * st.y, s = fmaf(m, w[e], b[e]);
            f[e] = BWD ? st.y * (d[e] * dact<SILU>(s) * w[e] - means[g].x - m * means[g].y) : act<SILU>(s);
        }
        out[i] = Vec<T>::pack(f);
    }
}

// ------------------------------------------------------------------------------------ a sample a cluster
// Forward: a tile of a sample's channels (whole groups) in the shared memory of a cluster, read once.  Each CTA
// takes `each` positions: per channel the sums of x - K and (x - K)^2 (K its first value here), joined to a mean and
// square deviation per group, which the CTAs read from one another and join in the order of their ranks.  Where a K turns
// out to be five and a half deviations or more from its channel's mean, so that the difference of the sums loses five bits or
// more (a first position far from all others), the CTA goes over its positions once more from the means.  (At four deviations
// one channel in 10^4 of ordinary values would do so, and with it nearly every call: 0.7 us of 16.8 at 8 x 4096 x 320.)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ float2 cluster_read(const float2 *own, int rank) {
    uint32_t at;
    float2 v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(own))), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}
template <typename T, bool SILU>
__global__ void __launch_bounds__(NT) gn_slab_kernel(GroupNormArgs p, GnSlab s) {
    constexpr int V = Vec<T>::N;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, rank = blockIdx.x % s.cluster, unit = blockIdx.x / s.cluster, row = unit / s.tiles, tile = unit % s.tiles;
    const int cg = p.C / p.G, tc = s.vecs * V, groups = tc / cg, c0 = tile * tc, vecs = p.C / V;
    const int subs = NT / s.vecs, v = tid % s.vecs, sub = tid / s.vecs;
    const int from = min(p.L, rank * s.each), len = min(p.L, from + s.each) - from;
    uint4 *slab = reinterpret_cast<uint4 *>(smem);
    float *red = reinterpret_cast<float *>(smem + (size_t)s.each * s.vecs * 16);  // [NT][V + 1], then sums [2][tc]
    float *sums = red + NT * (V + 1), *centers = sums + 2 * tc;
    float2 *part = reinterpret_cast<float2 *>(centers + tc), *all = part + groups;  // a group's mean and deviation; mean and r
    const bool works = sub < subs;
    const uint4 *x = static_cast<const uint4 *>(p.x) + ((size_t)row * p.L + from) * vecs + c0 / V + v;
    if (works)
        for (int t = sub; t < len; t += subs)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(slab + t * s.vecs + v))),
                         "l"(x + (size_t)t * vecs)
                         : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
    float w[V], b[V];
    affine(p, c0 + v * V, w, b);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    const T *first = reinterpret_cast<const T *>(slab);
    bool again = false;
    auto center = [&](int c) { return again ? centers[c] : to_f32(first[c]); };
    for (;;) {
        float a[V] = {}, q[V] = {}, k[V] = {};
        if (len > 0)
#pragma unroll
            for (int e = 0; e < V; ++e) k[e] = center(v * V + e);
        if (works) {
#pragma unroll 4
            for (int t = sub; t < len; t += subs) {
                float f[V];
                Vec<T>::unpack(slab[t * s.vecs + v], f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    f[e] -= k[e];
                    a[e] += f[e];
                    q[e] = fmaf(f[e], f[e], q[e]);
                }
            }
        }
        bool far = false;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < V; ++e) red[tid * (V + 1) + e] = which ? q[e] : a[e];
            __syncthreads();
            for (int i = tid; i < tc; i += NT) {
                float z = 0.f;
                for (int j = 0; j < subs; ++j) z += red[(j * s.vecs + i / V) * (V + 1) + i % V];
                sums[which * tc + i] = z;
                if (which) far |= fmaf(-sums[i], sums[i] / (float)max(len, 1), z) < z * (1.f / 32.f);
            }
        }
        if (!__syncthreads_or(far) || again) break;
        again = true;
        for (int i = tid; i < tc; i += NT) centers[i] = to_f32(first[i]) + sums[i] / (float)len;
        __syncthreads();
    }
    for (int g = tid / 32; g < groups; g += NT / 32) {
        const int lane = tid & 31;
        const float per = len > 0 ? 1.f / (float)len : 0.f;
        float m = 0.f, dev = 0.f;
        if (len > 0) {
            for (int c = g * cg + lane; c < (g + 1) * cg; c += 32) m += fmaf(sums[c], per, center(c));
            m = row_sum<32>(m) / (float)cg;
            for (int c = g * cg + lane; c < (g + 1) * cg; c += 32) {
                const float cm = sums[c] * per, off = (center(c) - m) + cm;
                dev += fmaxf(fmaf(-sums[c], cm, sums[tc + c]), 0.f) + (float)len * off * off;
            }
            dev = row_sum<32>(dev);
        }
        if (lane == 0) part[g] = make_float2(m, dev);
    }
    cluster_arrive();
    cluster_wait();
    for (int g = tid; g < groups; g += NT) {
        float m = 0.f, dev = 0.f;
        for (int r = 0; r < s.cluster; ++r) {
            const int n = min(p.L, (r + 1) * s.each) - min(p.L, r * s.each);
            m = fmaf((float)n, cluster_read(part + g, r).x, m);
        }
        m /= (float)p.L;
        for (int r = 0; r < s.cluster; ++r) {
            const int n = min(p.L, (r + 1) * s.each) - min(p.L, r * s.each);
            const float2 o = cluster_read(part + g, r);
            if (n > 0) dev += fmaf((float)n * (float)cg * (o.x - m), o.x - m, o.y);
        }
        const float r = rsqrtf(dev / ((float)p.L * (float)cg) + p.eps);
        all[g] = make_float2(m, r);
        if (p.stats && rank == 0) reinterpret_cast<float2 *>(p.stats)[(size_t)row * p.G + c0 / cg + g] = make_float2(m, r);
    }
    cluster_arrive();  // (no CTA leaves while another may read from it)
    __syncthreads();
    if (works) {
        float m[V], r[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float2 st = all[(v * V + e) / cg];
            m[e] = st.x;
            r[e] = st.y;
        }
        uint4 *y = static_cast<uint4 *>(p.y) + ((size_t)row * p.L + from) * vecs + c0 / V + v;
#pragma unroll 4
        for (int t = sub; t < len; t += subs) {
            float f[V];
            Vec<T>::unpack(slab[t * s.vecs + v], f);
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = act<SILU>(fmaf((f[e] - m[e]) * r[e], w[e], b[e]));
            y[(size_t)t * vecs] = Vec<T>::pack(f);
        }
    }
    cluster_wait();
}

template <typename T, bool SILU>
cudaError_t slab(const GroupNormArgs &a, const GnSlab &s) {
    constexpr int V = Vec<T>::N;
    const int tc = s.vecs * V;
    const size_t smem = (size_t)s.each * s.vecs * 16 + (size_t)NT * (V + 1) * 4 + 3 * tc * 4 + (size_t)tc / (a.C / a.G) * 16;
    const cudaError_t e = allow_smem(gn_slab_kernel<T, SILU>, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = s.cluster, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)a.rows * s.tiles * s.cluster), cfg.blockDim = dim3(NT), cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream, cfg.attrs = &attr, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gn_slab_kernel<T, SILU>, a, s);
}

template <typename T, bool BWD, bool SILU>
cudaError_t warps(const GroupNormArgs &a) {
    const int cg = a.C / a.G, team = std::min(32, gn_team(cg));
    const int bytes = (int)(((size_t)(BWD ? 2 : 1) * a.L * a.C * sizeof(T) + (size_t)a.G * (BWD ? 16 : 8) + 15) / 16 * 16);
    const int count = std::max(1, std::min({8, (int)(64 * 1024 / bytes), (a.rows + 151) / 152}));
    auto go = [&](auto kernel) {
        const cudaError_t e = allow_smem(kernel, (size_t)count * bytes);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)((a.rows + count - 1) / count), 32 * count, (size_t)count * bytes, a.stream>>>(a, bytes);
        return cudaGetLastError();
    };
    auto teams = [&](auto many) {
        constexpr bool MANY = decltype(many)::value;
        return team == 1    ? go(gn_warp_kernel<T, 1, BWD, SILU, MANY>)
               : team == 2  ? go(gn_warp_kernel<T, 2, BWD, SILU, MANY>)
               : team == 4  ? go(gn_warp_kernel<T, 4, BWD, SILU, MANY>)
               : team == 8  ? go(gn_warp_kernel<T, 8, BWD, SILU, MANY>)
               : team == 16 ? go(gn_warp_kernel<T, 16, BWD, SILU, MANY>)
                            : go(gn_warp_kernel<T, 32, BWD, SILU, MANY>);
    };
    cudaError_t e = !BWD && a.L * ((cg + team - 1) / team) > 32 ? teams(std::bool_constant<!BWD>{}) : teams(std::false_type{});
    if constexpr (BWD) {
        if (e != cudaSuccess || (!a.dw && !a.db)) return e;
        const int vecs = a.C / Vec<T>::N, lanes = gn_lanes(vecs), blocks = (vecs + lanes - 1) / lanes;
        const int chunks = gn_column_chunks(a.rows, a.L, a.C, a.dtype);
        gn_sums_kernel<T, true, true, SILU><<<(unsigned)chunks * blocks, NT, 0, a.stream>>>(a, lanes, blocks, chunks);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        return launch_sum_parts(a.ws, chunks, 2 * a.C, a.db, a.dw, a.C, a.stream);
    }
    return e;
}

template <typename T, bool BWD, bool SILU>
cudaError_t whole(const GroupNormArgs &a) {
    const int team = gn_team(a.C / a.G / Vec<T>::N), blocks = gn_blocks(a.C, a.G, a.dtype);
    const int parts = BWD ? gn_row_parts(a.rows, a.C, a.G, a.dtype) : (a.rows + 63) / 64;
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)parts * blocks, NT, 0, a.stream>>>(a, blocks, parts);
        return cudaGetLastError();
    };
    cudaError_t e = team == 1    ? go(gn_rows_kernel<T, 1, BWD, SILU>)
                    : team == 2  ? go(gn_rows_kernel<T, 2, BWD, SILU>)
                    : team == 4  ? go(gn_rows_kernel<T, 4, BWD, SILU>)
                    : team == 8  ? go(gn_rows_kernel<T, 8, BWD, SILU>)
                    : team == 16 ? go(gn_rows_kernel<T, 16, BWD, SILU>)
                                 : go(gn_rows_kernel<T, 32, BWD, SILU>);
    if (e != cudaSuccess || !BWD) return e;
    return launch_sum_parts(a.ws, parts, 2 * a.C, a.db, a.dw, a.C, a.stream);
}

template <typename T, bool BWD, bool SILU>
cudaError_t group(const GroupNormArgs &a) {
    const GnTeam k = gn_group(a.L, a.C, a.G, a.dtype);
    const int parts = gn_group_parts(a.rows, a.G, k, BWD), threads = std::max(k.threads, NT);
    const size_t smem = (size_t)gn_group_depth(k.each) * threads * (k.each * (BWD ? 32 : 16) + (BWD ? 8 : 0));
    auto go = [&](auto kernel) {
        const cudaError_t e = allow_smem(kernel, smem);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)parts * a.G, threads, smem, a.stream>>>(a, parts);
        return cudaGetLastError();
    };
    cudaError_t e = cudaErrorInvalidValue;
    if constexpr (sizeof(T) == 4) {
        if (k.each == 4) e = go(gn_group_kernel<T, 512, 4, BWD, SILU>);
    }
    if (k.each < 4)
        e = k.each == 2        ? go(gn_group_kernel<T, 512, 2, BWD, SILU>)
            : k.threads == 512 ? go(gn_group_kernel<T, 512, 1, BWD, SILU>)
            : k.threads == 256 ? go(gn_group_kernel<T, 256, 1, BWD, SILU>)
            : k.threads == 128 ? go(gn_group_kernel<T, 128, 1, BWD, SILU>)
                               : go(gn_group_kernel<T, 64, 1, BWD, SILU>);
    if (e != cudaSuccess || !BWD) return e;
    return launch_sum_parts(a.ws, parts, 2 * a.C, a.db, a.dw, a.C, a.stream);
}

template <typename T, bool BWD, bool SILU>
cudaError_t general(GroupNormArgs a) {
    const int vecs = a.C / Vec<T>::N, lanes = gn_lanes(vecs), blocks = (vecs + lanes - 1) / lanes;
    const int chunks = gn_chunks(a.rows, a.L, a.C, a.dtype), tiles = (a.L + NT / lanes * 4 - 1) / (NT / lanes * 4);
    float *joined = a.ws + (size_t)a.rows * chunks * 2 * a.C;
    if (!BWD && a.stats) joined = a.stats;
    gn_sums_kernel<T, BWD, false, SILU><<<(unsigned)(a.rows * chunks) * blocks, NT, 0, a.stream>>>(a, lanes, blocks, chunks);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long groups = (long long)a.rows * a.G, of_warps = (groups + NT / 32 - 1) / (NT / 32);
    if (BWD)
        gn_join_kernel<<<(unsigned)of_warps, NT, 0, a.stream>>>(a, chunks, joined);
    else if (groups >= 152 * NT / 32)  // (a warp for every group keeps the GPU as busy)
        gn_moments_kernel<32><<<(unsigned)of_warps, NT, 0, a.stream>>>(a, chunks, joined);
    else
        gn_moments_kernel<NT><<<(unsigned)groups, NT, 0, a.stream>>>(a, chunks, joined);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (!BWD) a.stats = joined;
    gn_apply_kernel<T, BWD, SILU><<<(unsigned)(a.rows * tiles) * blocks, NT, 0, a.stream>>>(a, lanes, blocks, tiles, joined);
    if ((e = cudaGetLastError()) != cudaSuccess || !BWD) return e;
    return launch_sum_parts(a.ws, a.rows * chunks, 2 * a.C, a.db, a.dw, a.C, a.stream);
}

template <typename T, bool BWD, bool SILU>
cudaError_t path(const GroupNormArgs &a) {
    switch (gn_way(a.rows, a.L, a.C, a.G, a.dtype, BWD)) {
        case GnWay::ROWS: return whole<T, BWD, SILU>(a);
        case GnWay::WARP: return warps<T, BWD, SILU>(a);
        case GnWay::GROUP: return group<T, BWD, SILU>(a);
        case GnWay::SLAB:
            if constexpr (!BWD) return slab<T, SILU>(a, gn_slab(a.rows, a.L, a.C, a.G, a.dtype));
            break;
        case GnWay::GENERAL: break;
    }
    return general<T, BWD, SILU>(a);
}
template <bool BWD>
cudaError_t types(const GroupNormArgs &a) {
    if (a.silu) return a.dtype == EFLA_BF16 ? path<__nv_bfloat16, BWD, true>(a) : path<float, BWD, true>(a);
    return a.dtype == EFLA_BF16 ? path<__nv_bfloat16, BWD, false>(a) : path<float, BWD, false>(a);
}

}  // namespace

cudaError_t launch_group_norm(const GroupNormArgs &a) { return types<false>(a); }
cudaError_t launch_group_norm_bwd(const GroupNormArgs &a) {
    if (a.rows > 0 && a.L > 0) return types<true>(a);
    return launch_sum_parts(a.ws, 0, 2 * a.C, a.db, a.dw, a.C, a.stream);  // the sums over no rows
}

}  // namespace efla
