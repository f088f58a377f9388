// Group norm with its activation, channels last: x [rows, L, C], G groups of C / G neighbouring channels, statistics
// over the L positions and the channels of a group (L = 1: of a token's heads).
//   n = (x - mean) r,  r = 1 / sqrt(var + eps),   s = w n + b,   y = s or silu(s)
//   ds = dy or dy silu'(s),  dn = ds w,  dx = r (dn - mean(dn) - n mean(dn n)),  dw = sum ds n,  db = sum ds
//
// Bound by HBM: x (and dy) read, y (dx) written.  With L = 1 a group of a row lies in the registers of up to 32
// lanes, whose sums are shuffles: one pass.  Otherwise sums per channel are taken over chunks of the positions
// (kernel 1), joined to those of the groups (kernel 2, which is small) and applied (kernel 3, which finds x in L2
// where it fits).  A channel's sums are those of x minus the channel's first value, and channels join by their means
// and square deviations, so that a mean far from 0 costs no accuracy.
#include "group_norm.cuh"
#include "mixer_norm.cuh"
#include "vec.cuh"

namespace efla {
namespace {

constexpr int NT = GN_NT;

// To 2 + 1.2 |x| ulp, as the output gate's.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ float act(float s, int silu) { return silu ? s * sigmoid(s) : s; }
__device__ __forceinline__ float dact(float s, int silu) {
    if (!silu) return 1.f;
    const float g = sigmoid(s);
    return g * fmaf(s, 1.f - g, 1.f);
}

template <int V>
__device__ __forceinline__ void affine(const GroupNormArgs &p, int c0, float (&w)[V], float (&b)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        w[e] = p.w ? p.w[c0 + e] : 1.f;
        b[e] = p.b ? p.b[c0 + e] : 0.f;
    }
}

// ------------------------------------------------------------------------------------ whole rows (L = 1)
// A warp holds 32 / TEAM groups of a row, a group in the first C / G / V lanes of its TEAM; a CTA 8 rows of one block
// of groups, and every parts-th 8 rows after them.
template <typename T, int TEAM, bool BWD>
__global__ void __launch_bounds__(NT) gn_rows_kernel(GroupNormArgs p, int blocks, int parts) {
    constexpr int V = Vec<T>::N, PER = 32 / TEAM, SUBS = NT / 32, UNROLL = 4;
    __shared__ float red[BWD ? SUBS : 1][BWD ? 32 * V : 1];
    const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5, l = lane % TEAM;
    const int block = blockIdx.x % blocks, part = blockIdx.x / blocks;
    const int g = block * PER + lane / TEAM, gv = p.C / p.G / V, vecs = p.C / V;
    const bool live = g < p.G && l < gv;
    const int v = live ? g * gv + l : 0;
    const float inv = 1.f / (float)(p.C / p.G);
    float w[V], b[V], dw[V] = {}, db[V] = {};
    affine(p, v * V, w, b);
    const long long step = (long long)parts * SUBS;
    for (long long row0 = (long long)part * SUBS + sub; row0 < p.rows; row0 += step * UNROLL) {  // (the same for a warp)
        uint4 rx[UNROLL], rd[UNROLL];
        float2 st[UNROLL];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const long long row = row0 + i * step;
            rx[i] = rd[i] = make_uint4(0, 0, 0, 0);
            st[i] = make_float2(0.f, 0.f);
            if (live && row < p.rows) {
                rx[i] = static_cast<const uint4 *>(p.x)[row * vecs + v];
                if (BWD) {
                    rd[i] = static_cast<const uint4 *>(p.dy)[row * vecs + v];
                    st[i] = reinterpret_cast<const float2 *>(p.stats)[row * p.G + g];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const long long row = row0 + i * step;
            if (row >= p.rows) break;
            float x[V];
            Vec<T>::unpack(rx[i], x);
            if (!BWD) {
                float m = 0.f, q = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) m += x[e];
                m = row_sum<TEAM>(m) * inv;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[e] = live ? x[e] - m : 0.f;
                    q = fmaf(x[e], x[e], q);
                }
                const float r = rsqrtf(row_sum<TEAM>(q) * inv + p.eps);
#pragma unroll
                for (int e = 0; e < V; ++e) x[e] = act(fmaf(x[e] * r, w[e], b[e]), p.silu);
                if (live) {
                    static_cast<uint4 *>(p.y)[row * vecs + v] = Vec<T>::pack(x);
                    if (p.stats && l == 0) reinterpret_cast<float2 *>(p.stats)[row * p.G + g] = make_float2(m, r);
                }
            } else {
                float d[V], s1 = 0.f, s2 = 0.f;
                Vec<T>::unpack(rd[i], d);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float n = (x[e] - st[i].x) * st[i].y;
                    d[e] *= dact(fmaf(n, w[e], b[e]), p.silu);
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
                for (int e = 0; e < V; ++e) x[e] = st[i].y * (d[e] - s1 - x[e] * s2);
                if (live) static_cast<uint4 *>(p.dx)[row * vecs + v] = Vec<T>::pack(x);
            }
        }
    }
    if (BWD) {  // the CTA's sums over its rows, in order: db then dw
        float *out = p.ws + (size_t)part * 2 * p.C;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < V; ++e) red[sub][lane * V + e] = which ? dw[e] : db[e];
            __syncthreads();
            for (int i = threadIdx.x; i < 32 * V; i += NT) {
                const int ln = i / V, gg = block * PER + ln / TEAM, ll = ln % TEAM;
                if (gg >= p.G || ll >= gv) continue;
                float s = 0.f;
#pragma unroll
                for (int k = 0; k < SUBS; ++k) s += red[k][i];
                out[which * p.C + (gg * gv + ll) * V + i % V] = s;
            }
        }
    }
}

// ------------------------------------------------------------------------------------ sums per channel
// Forward: of x - K and (x - K)^2 with K the channel's first value of the row; backward: of ds and ds n.  A CTA
// takes one chunk of a row's positions and a block of its channels: part[row chunks + chunk][2][C].
template <typename T, bool BWD>
__global__ void __launch_bounds__(NT) gn_sums_kernel(GroupNormArgs p, int lanes, int blocks, int chunks) {
    constexpr int V = Vec<T>::N;
    __shared__ float red[NT][V + 1];
    const int tid = threadIdx.x, lane = tid % lanes, sub = tid / lanes, subs = NT / lanes;
    const int block = blockIdx.x % blocks, rc = blockIdx.x / blocks, row = rc / chunks, chunk = rc % chunks;
    const int vecs = p.C / V, v = block * lanes + lane, cg = p.C / p.G;
    const int each = (p.L + chunks - 1) / chunks, from = chunk * each, to = min(p.L, from + each);
    float a[V] = {}, q[V] = {};
    if (v < vecs) {
        const uint4 *x = static_cast<const uint4 *>(p.x) + (size_t)row * p.L * vecs + v;
        float k[V], r[V], w[V], b[V];
        if (BWD) {
            affine(p, v * V, w, b);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float2 st = reinterpret_cast<const float2 *>(p.stats)[(size_t)row * p.G + (v * V + e) / cg];
                k[e] = st.x;
                r[e] = st.y;
            }
        } else {
            Vec<T>::unpack(x[0], k);
        }
        const uint4 *dy = BWD ? static_cast<const uint4 *>(p.dy) + (size_t)row * p.L * vecs + v : nullptr;
#pragma unroll 4
        for (int t = from + sub; t < to; t += subs) {
            float f[V], d[V];
            Vec<T>::unpack(x[(size_t)t * vecs], f);
            if (BWD) Vec<T>::unpack(dy[(size_t)t * vecs], d);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (BWD) {
                    const float n = (f[e] - k[e]) * r[e];
                    d[e] *= dact(fmaf(n, w[e], b[e]), p.silu);
                    a[e] += d[e];
                    q[e] = fmaf(d[e], n, q[e]);
                } else {
                    const float s = f[e] - k[e];
                    a[e] += s;
                    q[e] = fmaf(s, s, q[e]);
                }
            }
        }
    }
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

// A warp a group of a row: its mean and r from the channels' sums; backward: mean(dn) and mean(dn n).
template <typename T, bool BWD>
__global__ void __launch_bounds__(NT) gn_join_kernel(GroupNormArgs p, int chunks, float *out) {
    const int lane = threadIdx.x & 31, cg = p.C / p.G;
    const long long i = (long long)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
    if (i >= (long long)p.rows * p.G) return;
    const int row = (int)(i / p.G), c0 = (int)(i % p.G) * cg;
    const float *part = p.ws + (size_t)row * chunks * 2 * p.C;
    auto channel = [&](int c, float &a, float &q) {
        a = q = 0.f;
        for (int k = 0; k < chunks; ++k) {
            a += part[(size_t)k * 2 * p.C + c];
            q += part[(size_t)k * 2 * p.C + p.C + c];
        }
    };
    const float inv = 1.f / ((float)p.L * (float)cg);
    float first = 0.f, second = 0.f;
    if (BWD) {
        for (int c = c0 + lane; c < c0 + cg; c += 32) {
            float a, q;
            channel(c, a, q);
            const float w = p.w ? p.w[c] : 1.f;
            first = fmaf(w, a, first);
            second = fmaf(w, q, second);
        }
        first = row_sum<32>(first) * inv;
        second = row_sum<32>(second) * inv;
    } else {
        const T *x = static_cast<const T *>(p.x) + (size_t)row * p.L * p.C;
        const float per = 1.f / (float)p.L;
        float sum = 0.f;
        for (int c = c0 + lane; c < c0 + cg; c += 32) {
            float a, q;
            channel(c, a, q);
            sum += fmaf(a, per, to_f32(x[c]));
        }
        first = row_sum<32>(sum) / (float)cg;
        float dev = 0.f;
        for (int c = c0 + lane; c < c0 + cg; c += 32) {
            float a, q;
            channel(c, a, q);
            const float m = a * per, off = (to_f32(x[c]) - first) + m;
            dev += fmaxf(fmaf(-a, m, q), 0.f) + (float)p.L * off * off;
        }
        second = rsqrtf(row_sum<32>(dev) * inv + p.eps);
    }
    if (lane == 0) reinterpret_cast<float2 *>(out)[i] = make_float2(first, second);
}

// y or dx from the groups' values (`means`: backward, what gn_join_kernel gave).  A thread a vector, UNROLL positions.
template <typename T, bool BWD>
__global__ void __launch_bounds__(NT) gn_apply_kernel(GroupNormArgs p, int lanes, int blocks, int tiles, const float *means) {
    constexpr int V = Vec<T>::N, UNROLL = 4;
    const int tid = threadIdx.x, lane = tid % lanes, sub = tid / lanes, subs = NT / lanes;
    const int block = blockIdx.x % blocks, rt = blockIdx.x / blocks, row = rt / tiles, tile = rt % tiles;
    const int vecs = p.C / V, v = block * lanes + lane, cg = p.C / p.G;
    if (v >= vecs) return;
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
            f[e] = BWD ? r[e] * (d[e] * dact(s, p.silu) * w[e] - s1[e] - n * s2[e]) : act(s, p.silu);
        }
        if (t < p.L) out[(size_t)t * vecs] = Vec<T>::pack(f);
    }
}

template <typename T, bool BWD>
cudaError_t whole(const GroupNormArgs &a) {
    const int team = gn_team(a.C / a.G / Vec<T>::N), blocks = gn_blocks(a.C, a.G, a.dtype);
    const int parts = BWD ? gn_row_parts(a.rows, a.C, a.G, a.dtype) : (a.rows + 31) / 32;
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)parts * blocks, NT, 0, a.stream>>>(a, blocks, parts);
        return cudaGetLastError();
    };
    cudaError_t e = team == 1    ? go(gn_rows_kernel<T, 1, BWD>)
                    : team == 2  ? go(gn_rows_kernel<T, 2, BWD>)
                    : team == 4  ? go(gn_rows_kernel<T, 4, BWD>)
                    : team == 8  ? go(gn_rows_kernel<T, 8, BWD>)
                    : team == 16 ? go(gn_rows_kernel<T, 16, BWD>)
                                 : go(gn_rows_kernel<T, 32, BWD>);
    if (e != cudaSuccess || !BWD) return e;
    return launch_sum_parts(a.ws, parts, 2 * a.C, a.db, a.dw, a.C, a.stream);
}

template <typename T, bool BWD>
cudaError_t general(GroupNormArgs a) {
    const int vecs = a.C / Vec<T>::N, lanes = gn_lanes(vecs), blocks = (vecs + lanes - 1) / lanes;
    const int chunks = gn_chunks(a.rows, a.L, a.C, a.dtype), tiles = (a.L + NT / lanes * 4 - 1) / (NT / lanes * 4);
    float *joined = a.ws + (size_t)a.rows * chunks * 2 * a.C;
    if (!BWD && a.stats) joined = a.stats;
    gn_sums_kernel<T, BWD><<<(unsigned)(a.rows * chunks) * blocks, NT, 0, a.stream>>>(a, lanes, blocks, chunks);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    gn_join_kernel<T, BWD><<<(unsigned)(((long long)a.rows * a.G + NT / 32 - 1) / (NT / 32)), NT, 0, a.stream>>>(a, chunks, joined);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (!BWD) a.stats = joined;
    gn_apply_kernel<T, BWD><<<(unsigned)(a.rows * tiles) * blocks, NT, 0, a.stream>>>(a, lanes, blocks, tiles, joined);
    if ((e = cudaGetLastError()) != cudaSuccess || !BWD) return e;
    return launch_sum_parts(a.ws, a.rows * chunks, 2 * a.C, a.db, a.dw, a.C, a.stream);
}

template <bool BWD>
cudaError_t types(const GroupNormArgs &a) {
    if (gn_whole(a.L, a.C, a.G, a.dtype)) return a.dtype == EFLA_BF16 ? whole<__nv_bfloat16, BWD>(a) : whole<float, BWD>(a);
    return a.dtype == EFLA_BF16 ? general<__nv_bfloat16, BWD>(a) : general<float, BWD>(a);
}

}  // namespace

cudaError_t launch_group_norm(const GroupNormArgs &a) { return types<false>(a); }
cudaError_t launch_group_norm_bwd(const GroupNormArgs &a) {
    if (a.rows > 0 && a.L > 0) return types<true>(a);
    return launch_sum_parts(a.ws, 0, 2 * a.C, a.db, a.dw, a.C, a.stream);  // the sums over no rows
}

}  // namespace efla
