// Short causal convolution over the tokens of every channel, before a token mixer (W = 2, 3 or 4 taps):
//   s_t = bias + sum_{j < W} w_j x_{t-W+1+j},   y = s or silu(s) = s sigmoid(s)
// the W - 1 inputs before a sequence's first token from its state (or 0), the last W - 1 of state and
// sequence kept as the next state.  Reverse mode, ds = dy or dy silu'(s), silu'(s) = g (1 + s (1 - g)) with
// g = sigmoid(s):
//   dx_t = sum_j w_j ds_{t+W-1-j},  dw_j = sum_t ds_t x_{t-W+1+j},  dbias = sum_t ds_t
// on rows extended by the state: place e = t + W - 1 >= 0, dfull_e = sum_j w_j ds_{e-j} (ds = 0 outside the
// row), plus dstate_T's at the last W - 1 places; the first W - 1 are dstate0.
//
// Bound by HBM: x is read and y written once.  A thread takes 4 channels and walks down a run of tokens with the last
// W - 1 rows in registers, so a row is read once by its run and again only as the W - 1 rows before the next.  Rows
// come into the thread's own slots of shared memory by asynchronous copies, a group of them at a time and the next groups under
// way.  Code for groups inside their row is straight (packed sequences go token by token); channels go in pairs, in packed arithmetic.  Runs of the forward
// are 32 tokens at most; those of the backward, which computes the gradients of the tokens before a run again, as
// long as fills the GPU.  Arithmetic is fp32, each output rounded once; the sums over tokens go in two stages of fixed order.
// 8 x 2048 tokens, W = 4, silu, bf16: forward of 6144 channels 70 us (403 MB, 5.8 TB/s), of 2048 26 (134 MB); backward with
// its sums of 6144 115 us (604 MB, 5.2 TB/s), of 2048 45 (201 MB, 4.5 TB/s; 66 in runs of 32 places), in fp32 72 (403 MB, 5.6 TB/s).
// The backward's threads need 148 registers: three CTAs of 128 a SM take 45 us, four with 128 registers 47, five 54, seven of
// 64 threads 52; groups of 12 rows 48 to 53.
#include <algorithm>
#include <type_traits>

#include "conv.cuh"
#include "mixer_norm.cuh"
#include "vec.cuh"

namespace efla {
namespace {

constexpr int NT = CONV_NT;
constexpr int FOUND = 32;  // long sequences that a CTA of the packed forward fills in together
template <typename T>
constexpr int conv_bwd_depth = sizeof(T) == 2 ? 3 : 2;  // groups of the backward's ring: 48 KB a CTA
template <typename T>
constexpr int BATCH = sizeof(T) == 2 ? 8 : 4;  // rows of a group of copies, of which a thread's run has four at most

// V channels of a row.
template <typename T, int V>
struct Pack;
template <typename T>
struct Pack<T, 8> {
    uint4 r;
};
template <>
struct Pack<float, 4> {
    uint4 r;
};
template <>
struct Pack<__nv_bfloat16, 4> {
    uint2 r;
};
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, 8> &p, float (&x)[8]) { Vec<__nv_bfloat16>::unpack(p.r, x); }
__device__ __forceinline__ void unpack(const Pack<float, 4> &p, float (&x)[4]) { Vec<float>::unpack(p.r, x); }
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, 4> &p, float (&x)[4]) {
    x[0] = __uint_as_float(p.r.x << 16);
    x[1] = __uint_as_float(p.r.x & 0xffff0000u);
    x[2] = __uint_as_float(p.r.y << 16);
    x[3] = __uint_as_float(p.r.y & 0xffff0000u);
}
__device__ __forceinline__ void pack(const float (&x)[8], Pack<__nv_bfloat16, 8> &p) { p.r = Vec<__nv_bfloat16>::pack(x); }
__device__ __forceinline__ void pack(const float (&x)[4], Pack<float, 4> &p) { p.r = Vec<float>::pack(x); }
__device__ __forceinline__ void pack(const float (&x)[4], Pack<__nv_bfloat16, 4> &p) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    p.r = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// Four channels as two pairs.
__device__ __forceinline__ void unpack(const Pack<float, 4> &p, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(p.r.x), __uint_as_float(p.r.y));
    x[1] = make_float2(__uint_as_float(p.r.z), __uint_as_float(p.r.w));
}
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, 4> &p, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(p.r.x << 16), __uint_as_float(p.r.x & 0xffff0000u));
    x[1] = make_float2(__uint_as_float(p.r.y << 16), __uint_as_float(p.r.y & 0xffff0000u));
}
__device__ __forceinline__ void pack(const float2 (&x)[2], Pack<float, 4> &p) {
    p.r = make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
}
__device__ __forceinline__ void pack(const float2 (&x)[2], Pack<__nv_bfloat16, 4> &p) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0].x, x[0].y), b = __floats2bfloat162_rn(x[1].x, x[1].y);
    p.r = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// Row `row` of p [rows, vecs], vector v.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load(const void *p, long long row, int vecs, int v) {
    return static_cast<const Pack<T, V> *>(p)[row * vecs + v];
}
template <typename T, int V>
__device__ __forceinline__ void store(void *p, long long row, int vecs, int v, const float (&x)[V]) {
    Pack<T, V> r;
    pack(x, r);
    static_cast<Pack<T, V> *>(p)[row * vecs + v] = r;
}

template <int W, int V>
struct Taps {
    float w[V][W], bias[V];
    __device__ __forceinline__ void load(const ConvArgs &p, int c0) {  // (V W floats from a multiple of 16 bytes)
        float f[V * W];
#pragma unroll
        for (int i = 0; i < V * W / 4; ++i) {
            const float4 r = reinterpret_cast<const float4 *>(p.w + (size_t)c0 * W)[i];
            f[4 * i] = r.x, f[4 * i + 1] = r.y, f[4 * i + 2] = r.z, f[4 * i + 3] = r.w;
        }
#pragma unroll
        for (int c = 0; c < V; ++c) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[c][j] = f[c * W + j];
            bias[c] = p.bias ? p.bias[c0 + c] : 0.f;
        }
    }
};

// The same of four channels as two pairs.
template <int W>
struct Taps4 {
    float2 w[2][W], bias[2];
    __device__ __forceinline__ void load(const ConvArgs &p, int c0) {
        Taps<W, 4> t;
        t.load(p, c0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[h][j] = make_float2(t.w[2 * h][j], t.w[2 * h + 1][j]);
            bias[h] = make_float2(t.bias[2 * h], t.bias[2 * h + 1]);
        }
    }
};

// ------------------------------------------------------------------------------------ forward
// CTAs [0, work_ctas): runs of `rows` tokens x a block of the channels; the others copy the states.  PACKED: the
// runs are of all tokens, and first[i], seq[i] say where the sequence of the CTA's token i begins and which it is
// (-1: none).  Otherwise they are of the rows, row_runs each.
template <typename T, int W, bool PACKED, bool SILU>
__global__ void __launch_bounds__(NT, 3) conv_fwd_kernel(ConvArgs p, int vecs, int lanes, int cblocks, unsigned work_ctas, int rows,
                                                      int row_runs) {
    constexpr int V = 4, BATCH = efla::BATCH<T>;
    const int tid = threadIdx.x;
    if (blockIdx.x >= work_ctas) {  // state_T: place j of a sequence's last W - 1 inputs
        const long long e = (long long)(blockIdx.x - work_ctas) * NT + tid;
        if (e >= (long long)p.N * (W - 1) * vecs) return;
        const int v = (int)(e % vecs), j = (int)(e / vecs % (W - 1));
        const int n = (int)(e / vecs / (W - 1));
        long long lo, hi;
        if (PACKED) {
            lo = p.cu_seqlens[n], hi = p.cu_seqlens[n + 1];
            if (lo < 0 || hi < lo || hi > p.T) {
                if (v == 0 && j == 0) atomicExch(p.status, (int)EFLA_ERR_INVALID_ARG);
                return;
            }
        } else {
            lo = (long long)n * p.T, hi = lo + p.T;
        }
        const long long at = hi - (W - 1) + j;
        Pack<T, V> r{};
        if (at >= lo)
            r = load<T, V>(p.x, at, vecs, v);
        else if (p.state0)
            r = load<T, V>(p.state0, (long long)n * (W - 1) + (at - lo + W - 1), vecs, v);
        static_cast<Pack<T, V> *>(p.state_T)[e] = r;
        return;
    }
    extern __shared__ __align__(16) uint8_t shared[];
    Pack<T, V> *slots = reinterpret_cast<Pack<T, V> *>(shared) + tid;  // row i of this thread's run at [i NT]
    const int subs = NT / lanes, tile = blockIdx.x / cblocks, sub = tid / lanes;
    int *first = reinterpret_cast<int *>(shared + (size_t)rows * NT * sizeof(Pack<T, V>)), *seq = first + rows * subs;
    long long t0 = 0, begin, end, lo = 0;
    int n = 0;
    if (PACKED) {
        const int tile_rows = rows * subs;
        t0 = (long long)tile * tile_rows;
        __shared__ int found, list[FOUND][4];  // long sequences of the tile: from, to, number, first token
        for (int i = tid; i < tile_rows; i += NT) seq[i] = -1;
        if (tid == 0) found = 0;
        __syncthreads();
        for (int i = tid; i < p.N; i += NT) {
            const long long l = p.cu_seqlens[i], h = p.cu_seqlens[i + 1];
            if (l < 0 || h < l || h > p.T) {
                if (blockIdx.x == 0) atomicExch(p.status, (int)EFLA_ERR_INVALID_ARG);
                continue;
            }
            const int from = (int)(max(l, t0) - t0), to = (int)(min(h, t0 + tile_rows) - t0);
            const int at = to - from > 16 ? atomicAdd(&found, 1) : FOUND;
            if (at < FOUND) {
                list[at][0] = from, list[at][1] = to, list[at][2] = i, list[at][3] = (int)l;
                continue;
            }
            for (int t = from; t < to; ++t) {
                first[t] = (int)l;
                seq[t] = i;
            }
        }
        __syncthreads();
        for (int f = 0; f < min(found, FOUND); ++f)
            for (int t = list[f][0] + tid; t < list[f][1]; t += NT) {
                first[t] = list[f][3];
                seq[t] = list[f][2];
            }
        __syncthreads();
        begin = t0 + (long long)sub * rows;
        end = begin + rows < p.T ? begin + rows : p.T;
    } else {
        const long long run = (long long)tile * subs + sub;
        if (run >= (long long)p.B * row_runs) return;
        n = (int)(run / row_runs);
        lo = (long long)n * p.T;
        begin = lo + run % row_runs * rows;
        end = begin + rows < lo + p.T ? begin + rows : lo + p.T;
    }
    const int v = (blockIdx.x % cblocks) * lanes + tid % lanes;
    if (v >= vecs || begin >= end) return;
    const int count = (int)(end - begin);
    {
        const Pack<T, V> *from = static_cast<const Pack<T, V> *>(p.x) + begin * vecs + v;
        for (int t = 0; t < count; t += BATCH) {
#pragma unroll
            for (int k = 0; k < BATCH; ++k) fetch(slots + (t + k) * NT, from + (size_t)(t + k < count ? t + k : 0) * vecs, t + k < count);
            fetch_commit();
        }
    }
    float2 win[W - 1][2];
    // the W - 1 inputs before token t of the sequence n that begins at lo
    auto before = [&](long long t) {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const long long at = t - (W - 1) + i;
            Pack<T, V> r{};
            if (at >= lo)
                r = load<T, V>(p.x, at, vecs, v);
            else if (p.state0)
                r = load<T, V>(p.state0, (long long)n * (W - 1) + (at - lo + W - 1), vecs, v);
            unpack(r, win[i]);
        }
    };
    if (PACKED)
        lo = -1;  // no sequence yet
    else
        before(begin);
    Taps4<W> taps;
    taps.load(p, v * V);
    auto token = [&](const Pack<T, V> &raw, Pack<T, V> *to) {
        float2 x[2], s[2];
        unpack(raw, x);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float2 a = taps.bias[h];
#pragma unroll
            for (int i = 0; i < W - 1; ++i) a = __ffma2_rn(taps.w[h][i], win[i][h], a);
            a = __ffma2_rn(taps.w[h][W - 1], x[h], a);
            s[h] = SILU ? __fmul2_rn(a, quick_sigmoid(a)) : a;
#pragma unroll
            for (int i = 0; i + 1 < W - 1; ++i) win[i][h] = win[i + 1][h];
            win[W - 2][h] = x[h];
        }
        Pack<T, V> r;
        pack(s, r);
        *to = r;
    };
    Pack<T, V> *to = static_cast<Pack<T, V> *>(p.y) + begin * vecs + v;
    int left = (count + BATCH - 1) / BATCH;
    for (int t = 0; t < count; t += BATCH, to += (size_t)BATCH * vecs) {
        fetch_wait(--left);
        if (!PACKED && t + BATCH <= count) {  // straight code for whole batches
#pragma unroll
            for (int k = 0; k < BATCH; ++k) token(slots[(t + k) * NT], to + (size_t)k * vecs);
            continue;
        }
#pragma unroll 1
        for (int k = 0; k < BATCH; ++k) {
            if (t + k >= count) break;
            if (PACKED) {
                n = seq[begin + t + k - t0];
                if (n < 0) {
                    lo = -1;
                    continue;
                }
                if (lo != first[begin + t + k - t0]) {
                    lo = first[begin + t + k - t0];
                    before(begin + t + k);
                }
            }
            token(slots[(t + k) * NT], to + (size_t)k * vecs);
        }
    }
}

// ------------------------------------------------------------------------------------ backward
// A CTA: `lanes` vectors of 4 channels x NT / lanes runs of R places of an extended row, and every parts-th such tile after
// it; row_runs runs a row.  Place e needs ds_e and the W - 1 before, so those before a run are computed again; x and dy
// come through a ring of groups of G rows in the thread's own slots, G a multiple of every window's length.
template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(CONV_BWD_NT, CONV_BWD_CTAS) conv_bwd_kernel(ConvArgs p, int vecs, int lanes, int cblocks, ConvRuns plan) {
    constexpr int V = 4, G = CONV_BWD_GROUP, DEPTH = conv_bwd_depth<T>, NT = CONV_BWD_NT;
    extern __shared__ __align__(16) uint8_t shared[];
    Pack<T, V> *xs = reinterpret_cast<Pack<T, V> *>(shared) + threadIdx.x, *ys = xs + DEPTH * G * NT;  // row i at [i NT]
    const int tid = threadIdx.x, lane = tid % lanes, sub = tid / lanes, subs = NT / lanes;
    const int cb = blockIdx.x % cblocks, tile = blockIdx.x / cblocks, v = cb * lanes + lane;
    const long long runs = (long long)p.B * plan.row_runs, step = (long long)plan.parts * subs;
    const int ends = p.T + W - 1;
    float2 dw[2][W] = {}, db[2] = {};
    Taps4<W> taps;
    if (v < vecs) taps.load(p, v * V);
    for (long long run = (long long)tile * subs + sub; v < vecs && run < runs; run += step) {
        const int b = (int)(run / plan.row_runs), e0 = (int)(run % plan.row_runs) * plan.run;
        const int e1 = e0 + min(plan.run, ends - e0);  // (a run is longer than what the longest row leaves below 2^31)
        const long long row = (long long)b * p.T;
        const Pack<T, V> *x0 = static_cast<const Pack<T, V> *>(p.x) + row * vecs + v, *y0 = static_cast<const Pack<T, V> *>(p.dy) + row * vecs + v;
        auto fetch_group = [&](int t0, int slot) {  // rows t0 .. of x and dy; past the row's end zeros
            if (t0 < e1) {
                const Pack<T, V> *x = x0 + (size_t)t0 * vecs, *y = y0 + (size_t)t0 * vecs;
                Pack<T, V> *xt = xs + slot * G * NT, *yt = ys + slot * G * NT;
                if (t0 + G <= p.T) {
#pragma unroll
                    for (int k = 0; k < G; ++k) {
                        fetch(xt + k * NT, x + (size_t)k * vecs, true);
                        fetch(yt + k * NT, y + (size_t)k * vecs, true);
                    }
                } else {
#pragma unroll 1
                    for (int k = 0; k < G; ++k) {
                        const bool real = t0 + k < p.T;
                        fetch(xt + k * NT, real ? x + (size_t)k * vecs : x0, real);
                        fetch(yt + k * NT, real ? y + (size_t)k * vecs : y0, real);
                    }
                }
            }
            fetch_commit();
        };
#pragma unroll
        for (int q = 0; q < DEPTH; ++q) fetch_group(e0 + q * G, q);
        float2 win[W - 1][2], old[W - 1][2];  // x at t - (W - 1) .. t - 1, ds of the W - 1 tokens before t
        // ds of token t, whose newest input is x (`real`: t is in the row); with `own` into dw and dbias too
        auto token = [&](const float2(&x)[2], float2(&ds)[2], bool real, bool own) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (SILU) {
                    float2 a = taps.bias[h];
#pragma unroll
                    for (int i = 0; i < W - 1; ++i) a = __ffma2_rn(taps.w[h][i], win[i][h], a);
                    a = __ffma2_rn(taps.w[h][W - 1], x[h], a);
                    const float2 one = make_float2(1.f, 1.f), g = quick_sigmoid(a);
                    const float2 slope = __fmul2_rn(g, __ffma2_rn(a, __ffma2_rn(g, make_float2(-1.f, -1.f), one), one));
                    if (real) ds[h] = __fmul2_rn(ds[h], slope);
                }
                if (own) {
#pragma unroll
                    for (int i = 0; i < W - 1; ++i) dw[h][i] = __ffma2_rn(ds[h], win[i][h], dw[h][i]);
                    dw[h][W - 1] = __ffma2_rn(ds[h], x[h], dw[h][W - 1]);
                    db[h] = __fadd2_rn(db[h], ds[h]);
                }
            }
        };
        // place e = t: d += sum_j w_j ds_{t-j}
        auto place_sum = [&](const float2(&ds)[2], float2(&d)[2]) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                d[h] = __ffma2_rn(taps.w[h][0], ds[h], d[h]);
#pragma unroll
                for (int j = 1; j < W; ++j) d[h] = __ffma2_rn(taps.w[h][j], old[W - 1 - j][h], d[h]);
            }
        };
        auto shift = [&](const float2(&x)[2], const float2(&ds)[2]) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i + 1 < W - 1; ++i) {
                    win[i][h] = win[i + 1][h];
                    old[i][h] = old[i + 1][h];
                }
                win[W - 2][h] = x[h];
                old[W - 2][h] = ds[h];
            }
        };
        // The tokens before the run: their inputs (of the state before token 0) and ds
        {
            const Pack<T, V> *state = p.state0 ? static_cast<const Pack<T, V> *>(p.state0) + (long long)b * (W - 1) * vecs + v : nullptr;
            Pack<T, V> xr[2 * (W - 1)], yr[W - 1];
#pragma unroll
            for (int i = 0; i < 2 * (W - 1); ++i) {
                const int t = e0 - 2 * (W - 1) + i;
                xr[i] = {};
                if (t >= 0 && t < p.T)
                    xr[i] = x0[(size_t)t * vecs];
                else if (t < 0 && t + W - 1 >= 0 && state)
                    xr[i] = state[(size_t)(t + W - 1) * vecs];
            }
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                const int t = e0 - (W - 1) + i;
                yr[i] = {};
                if (t >= 0 && t < p.T) yr[i] = y0[(size_t)t * vecs];
            }
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                unpack(xr[i], win[i]);
                old[i][0] = old[i][1] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                const int t = e0 - (W - 1) + i;
                float2 x[2], ds[2];
                unpack(xr[W - 1 + i], x);
                unpack(yr[i], ds);
                token(x, ds, t >= 0 && t < p.T, false);
                shift(x, ds);
            }
        }
        Pack<T, V> *to = static_cast<Pack<T, V> *>(p.dx) + (row + e0 - (W - 1)) * vecs + v;  // (at place e0; used from place W - 1 on)
        int slot = 0;
#pragma unroll 1
        for (int t0 = e0; t0 < e1; t0 += G, to += (size_t)G * vecs) {
            fetch_wait(DEPTH - 1);
            const Pack<T, V> *xq = xs + slot * G * NT, *yq = ys + slot * G * NT;
            if (t0 >= W - 1 && t0 + G <= p.T) {  // all of it tokens of the row: straight code
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    float2 x[2], ds[2], d[2] = {};
                    unpack(xq[k * NT], x);
                    unpack(yq[k * NT], ds);
                    token(x, ds, true, true);
                    place_sum(ds, d);
                    shift(x, ds);
                    Pack<T, V> r;
                    pack(d, r);
                    to[(size_t)k * vecs] = r;
                }
            } else {
#pragma unroll 1
                for (int t = t0; t < min(t0 + G, e1); ++t) {
                    float2 x[2], ds[2], d[2] = {};
                    unpack(xq[(t - t0) * NT], x);
                    unpack(yq[(t - t0) * NT], ds);  // 0 past the row
                    token(x, ds, t < p.T, true);
                    if (p.dstate_T && t >= p.T) unpack(load<T, V>(p.dstate_T, (long long)b * (W - 1) + t - p.T, vecs, v), d);
                    place_sum(ds, d);
                    Pack<T, V> r;
                    pack(d, r);
                    if (t >= W - 1)
                        to[(size_t)(t - t0) * vecs] = r;
                    else if (p.dstate0)
                        static_cast<Pack<T, V> *>(p.dstate0)[((long long)b * (W - 1) + t) * vecs + v] = r;
                    shift(x, ds);
                }
            }
            fetch_group(t0 + DEPTH * G, slot);
            slot = slot + 1 == DEPTH ? 0 : slot + 1;
        }
        fetch_wait(0);
    }
    // the CTA's sums over its runs, in order: [D][W] then [D] of part `tile`
    float4 *red = reinterpret_cast<float4 *>(shared);  // (every thread is done with its slots)
    const int sums = p.dbias ? W + 1 : W;
    float *part = p.ws + (size_t)tile * p.D * sums;
    __syncthreads();
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        const float2 lo = j < W ? dw[0][j < W ? j : 0] : db[0], hi = j < W ? dw[1][j < W ? j : 0] : db[1];
        red[j * NT + tid] = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
    __syncthreads();
    for (int i = tid; i < sums * lanes * V; i += NT) {
        const int j = i / (lanes * V), l = i / V % lanes, c = i % V, ch = (cb * lanes + l) * V + c;
        if (ch >= p.D) continue;
        float s = 0.f;
        for (int q = 0; q < subs; ++q) s += reinterpret_cast<const float *>(red + j * NT + q * lanes + l)[c];
        part[j < W ? (size_t)ch * W + j : (size_t)p.D * W + ch] = s;
    }
}

// ------------------------------------------------------------------------------------ one token
// A thread a vector of ROWS sequences, whose weights it reads once.
constexpr int STEP_NT = 128;
template <typename T, int V, int W, int ROWS>
__global__ void __launch_bounds__(STEP_NT) conv_step_kernel(ConvArgs p, int vecs) {
    const long long e = (long long)blockIdx.x * STEP_NT + threadIdx.x;
    const int v = (int)(e % vecs);
    const long long b0 = e / vecs * ROWS;
    if (b0 >= p.B) return;
    Pack<T, V> raw[ROWS][W];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (b0 + r >= p.B) break;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) raw[r][i] = load<T, V>(p.state0, (b0 + r) * (W - 1) + i, vecs, v);
        raw[r][W - 1] = load<T, V>(p.x, b0 + r, vecs, v);
    }
    Taps<W, V> taps;
    taps.load(p, v * V);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const long long b = b0 + r;
        if (b >= p.B) break;
        float s[V];
#pragma unroll
        for (int c = 0; c < V; ++c) s[c] = taps.bias[c];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float x[V];
            unpack(raw[r][i], x);
#pragma unroll
            for (int c = 0; c < V; ++c) s[c] = fmaf(taps.w[c][i], x[c], s[c]);
            if (i > 0) static_cast<Pack<T, V> *>(p.state_T)[(b * (W - 1) + i - 1) * vecs + v] = raw[r][i];
        }
        if (p.silu) {
#pragma unroll
            for (int c = 0; c < V; ++c) s[c] *= quick_sigmoid(s[c]);
        }
        store<T, V>(p.y, b, vecs, v, s);
    }
}

template <typename T, int W>
cudaError_t fwd(const ConvArgs &a) {
    constexpr int V = 4;
    const int vecs = a.D / V, lanes = conv_lanes(vecs), cblocks = (vecs + lanes - 1) / lanes, subs = NT / lanes;
    // Tokens a thread: four batches (3 rows of halo in 32 or 16) where that still leaves two CTAs a SM, down to 8.
    const long long tokens = (long long)a.B * a.T;
    int rows = 4 * BATCH<T>;
    while (rows > 8 && tokens * vecs < 2LL * 152 * NT * rows) rows /= 2;
    const int row_runs = (a.T + rows - 1) / rows;
    const long long runs = a.cu_seqlens ? (tokens + rows - 1) / rows : (long long)a.B * row_runs;
    const long long work = std::max((runs + subs - 1) / subs * cblocks, a.cu_seqlens ? 1LL : 0LL);  // (the first CTA looks at all bounds)
    const long long copies = a.state_T ? ((long long)a.N * (W - 1) * vecs + NT - 1) / NT : 0;
    if (work + copies == 0) return cudaSuccess;
    const size_t slots = (size_t)rows * NT * sizeof(Pack<T, V>);
    auto go = [&](auto kernel, size_t smem) {
        const cudaError_t e = allow_smem(kernel, smem);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)(work + copies), NT, smem, a.stream>>>(a, vecs, lanes, cblocks, (unsigned)work, rows, row_runs);
        return cudaGetLastError();
    };
    if (a.cu_seqlens)
        return go(a.silu ? conv_fwd_kernel<T, W, true, true> : conv_fwd_kernel<T, W, true, false>,
                  slots + 2 * rows * subs * sizeof(int));
    return go(a.silu ? conv_fwd_kernel<T, W, false, true> : conv_fwd_kernel<T, W, false, false>, slots);
}
template <typename T, int W>
cudaError_t bwd(const ConvArgs &a) {
    const int vecs = a.D / 4, lanes = conv_lanes(vecs), cblocks = (vecs + lanes - 1) / lanes;
    const ConvRuns plan = conv_bwd_runs(a.B, a.T, a.D, a.W);
    constexpr size_t smem = (size_t)2 * conv_bwd_depth<T> * CONV_BWD_GROUP * CONV_BWD_NT * sizeof(Pack<T, 4>);
    static_assert(smem >= (W + 1) * CONV_BWD_NT * sizeof(float4), "the sums");
    auto go = [&](auto kernel) {
        const cudaError_t e = allow_smem(kernel, smem);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)plan.parts * cblocks, CONV_BWD_NT, smem, a.stream>>>(a, vecs, lanes, cblocks, plan);
        return cudaGetLastError();
    };
    const cudaError_t e = go(a.silu ? conv_bwd_kernel<T, W, true> : conv_bwd_kernel<T, W, false>);
    if (e != cudaSuccess) return e;
    return launch_sum_parts(a.ws, plan.parts, a.D * (a.dbias ? W + 1 : W), a.dw, a.dbias, a.D * W, a.stream);
}
template <typename T, int W>
cudaError_t step(const ConvArgs &a) {
    constexpr int V = Vec<T>::N;
    const int vecs = a.D / V;
    auto ctas = [&](int rows) { return (unsigned)(((long long)(a.B + rows - 1) / rows * vecs + STEP_NT - 1) / STEP_NT); };
    if (ctas(4) >= 152)
        conv_step_kernel<T, V, W, 4><<<ctas(4), STEP_NT, 0, a.stream>>>(a, vecs);
    else
        conv_step_kernel<T, V, W, 1><<<ctas(1), STEP_NT, 0, a.stream>>>(a, vecs);
    return cudaGetLastError();
}

template <typename T>
cudaError_t taps(const ConvArgs &a, int which) {
    auto go = [&](auto w) {
        constexpr int W = decltype(w)::value;
        return which == 0 ? fwd<T, W>(a) : which == 1 ? bwd<T, W>(a) : step<T, W>(a);
    };
    return a.W == 2 ? go(std::integral_constant<int, 2>{}) : a.W == 3 ? go(std::integral_constant<int, 3>{})
                                                                      : go(std::integral_constant<int, 4>{});
}
cudaError_t types(const ConvArgs &a, int which) {
    return a.dtype == EFLA_BF16 ? taps<__nv_bfloat16>(a, which) : taps<float>(a, which);
}

}  // namespace

cudaError_t launch_conv(const ConvArgs &a) { return types(a, 0); }
cudaError_t launch_conv_bwd(const ConvArgs &a) { return types(a, 1); }
cudaError_t launch_conv_step(const ConvArgs &a) { return types(a, 2); }

}  // namespace efla
