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
// W - 1 rows in registers, so a row is read once by its run and again only as the W - 1 rows before the next.  A run
// comes into the thread's own slots of shared memory by asynchronous copies, four groups of them under way; the backward
// refills a group for the next run as soon as it is done with it.  Code for runs inside their row is straight.
// Arithmetic is fp32, each output rounded once; the sums over tokens go in two stages of fixed order.
// 8 x 2048 tokens, W = 4, silu, bf16: forward of 6144 channels 78 us (403 MB, 5.2 TB/s), of 2048 27 (134 MB); backward of 2048 62
// (201 MB, 3.2 TB/s).  An element of the forward is 17 instructions and one of the backward 33, 0.62 and
// 0.54 of what issues: the copies no longer limit them.
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

// An asynchronous copy of a Pack into this thread's slot of shared memory; zeros where it is not live.
template <typename P>
__device__ __forceinline__ void fetch(P *dst, const P *src, bool live) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (sizeof(P) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(live ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(src), "r"(live ? 8 : 0) : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most `left` (0 to 3) of the latest groups are under way.
__device__ __forceinline__ void fetch_wait(int left) {
    if (left >= 3)
        asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (left == 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (left == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
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
// A CTA: `lanes` vectors of 4 channels x NT / lanes runs of R places of an extended row (with the W - 1 before them), and every
// parts-th such tile after it; row_runs runs a row.
template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(CONV_BWD_NT, 3) conv_bwd_kernel(ConvArgs p, int vecs, int lanes, int cblocks, int parts, int row_runs) {
    constexpr int V = 4, BATCH = efla::BATCH<T>, NT = CONV_BWD_NT, R = 4 * BATCH;
    extern __shared__ __align__(16) uint8_t shared[];
    constexpr int XS = R + 2 * (W - 1);  // slots of x: tokens from e0 - 2 (W - 1) on; of dy: from e0 - (W - 1) on
    Pack<T, V> *xs = reinterpret_cast<Pack<T, V> *>(shared) + threadIdx.x, *ys = xs + XS * NT;  // slot i at [i NT]
    const int tid = threadIdx.x, lane = tid % lanes, sub = tid / lanes, subs = NT / lanes;
    const int cb = blockIdx.x % cblocks, tile = blockIdx.x / cblocks, v = cb * lanes + lane;
    const long long runs = (long long)p.B * row_runs, step = (long long)parts * subs;
    const int ends = p.T + W - 1;
    float2 dw[2][W] = {}, db[2] = {};
    Taps4<W> taps;
    if (v < vecs) taps.load(p, v * V);
    // Group q of a run's copies: its batch q, and the first with what comes before it.  A group is fetched for the next
    // run as soon as this one is done with its slots, so three are always under way behind the one that is needed.
    auto fetch_group = [&](long long run, int q) {
        if (v < vecs && run < runs) {
            const int b = (int)(run / row_runs), e0 = (int)(run % row_runs) * R;
            const long long at = (long long)b * p.T * vecs + v;
            const Pack<T, V> *x = static_cast<const Pack<T, V> *>(p.x) + at, *y = static_cast<const Pack<T, V> *>(p.dy) + at;
            if (e0 >= 2 * (W - 1) && e0 + R <= p.T) {
                x += (long long)(e0 + q * BATCH) * vecs;
                y += (long long)(e0 + q * BATCH) * vecs;
                if (q == 0) {
#pragma unroll
                    for (int i = 0; i < 2 * (W - 1); ++i) fetch(xs + i * NT, x + (long long)(i - 2 * (W - 1)) * vecs, true);
#pragma unroll
                    for (int i = 0; i < W - 1; ++i) fetch(ys + i * NT, y + (long long)(i - (W - 1)) * vecs, true);
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    fetch(xs + (2 * (W - 1) + q * BATCH + k) * NT, x + (size_t)k * vecs, true);
                    fetch(ys + (W - 1 + q * BATCH + k) * NT, y + (size_t)k * vecs, true);
                }
            } else {
                const Pack<T, V> *state = p.state0 ? static_cast<const Pack<T, V> *>(p.state0) + (long long)b * (W - 1) * vecs + v : nullptr;
                const int from = q == 0 ? 0 : 2 * (W - 1) + q * BATCH, to = 2 * (W - 1) + (q + 1) * BATCH;
#pragma unroll 1
                for (int i = from; i < to; ++i) {
                    const int t = e0 - 2 * (W - 1) + i, j = i - (W - 1);
                    const bool real = t >= 0 && t < p.T, old = t < 0 && t + W - 1 >= 0 && state;
                    fetch(xs + i * NT, real ? x + (size_t)t * vecs : old ? state + (size_t)(t + W - 1) * vecs : x, real || old);
                    if (j >= 0) fetch(ys + j * NT, real ? y + (size_t)t * vecs : y, real);
                }
            }
        }
        fetch_commit();
    };
    const long long run0 = (long long)tile * subs + sub;
#pragma unroll
    for (int q = 0; q < 4; ++q) fetch_group(run0, q);
    for (long long run = run0; v < vecs && run < runs; run += step) {
        const int b = (int)(run / row_runs);
        const int e0 = (int)(run % row_runs) * R, tb0 = e0 - (W - 1), e1 = min(e0 + R, ends);
        const long long row = (long long)b * p.T;
        float2 win[W - 1][2], old[W - 1][2] = {};  // x at t - (W - 1) .. t - 1, ds of the W - 1 tokens before t
        fetch_wait(3);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) unpack(xs[i * NT], win[i]);
        // ds of token t, whose newest input is x, into the window; with `own` into dw and dbias too
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
        if (e0 >= 2 * (W - 1) && e0 + R <= p.T) {  // all of it tokens of the row: straight code
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {  // the tokens before the run: their ds
                float2 x[2], ds[2];
                unpack(xs[(W - 1 + i) * NT], x);
                unpack(ys[i * NT], ds);
                token(x, ds, true, false);
                shift(x, ds);
            }
            Pack<T, V> *to = static_cast<Pack<T, V> *>(p.dx) + (size_t)(row + tb0) * vecs + v;
#pragma unroll 1
            for (int q = 0; q < 4; ++q, to += (size_t)BATCH * vecs) {
                if (q > 0) fetch_wait(3);
                const Pack<T, V> *xq = xs + (2 * (W - 1) + q * BATCH) * NT, *yq = ys + (W - 1 + q * BATCH) * NT;
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
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
                fetch_group(run + step, q);
            }
            continue;
        }
        fetch_wait(0);
        auto put = [&](void *to, long long at, const float2(&d)[2]) {
            Pack<T, V> r;
            pack(d, r);
            static_cast<Pack<T, V> *>(to)[at * vecs + v] = r;
        };
#pragma unroll 1
        for (int t = tb0; t < e1; ++t) {  // token t's newest input is at place t + W - 1 of the extended row
            float2 x[2], ds[2];
            unpack(xs[(t - tb0 + W - 1) * NT], x);
            unpack(ys[(t - tb0) * NT], ds);  // 0 outside the row
            token(x, ds, t >= 0 && t < p.T, t >= e0);
            if (t >= e0) {
                float2 d[2] = {};
                if (p.dstate_T && t >= p.T) unpack(load<T, V>(p.dstate_T, (long long)b * (W - 1) + t - p.T, vecs, v), d);
                place_sum(ds, d);
                if (t >= W - 1)
                    put(p.dx, row + t - (W - 1), d);
                else if (p.dstate0)
                    put(p.dstate0, (long long)b * (W - 1) + t, d);
            }
            shift(x, ds);
        }
#pragma unroll 1
        for (int q = 0; q < 4; ++q) fetch_group(run + step, q);
    }
    fetch_wait(0);
    float(*red)[V + 1] = reinterpret_cast<float(*)[V + 1]>(shared);  // (the slots are done with)
    // the CTA's sums over its runs, in order: [D][W] then [D] of part `tile`
    const int sums = p.dbias ? W + 1 : W;
    float *part = p.ws + (size_t)tile * p.D * sums;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        if (j == sums) break;
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 r = j < W ? dw[h][j < W ? j : 0] : db[h];
            red[tid][2 * h] = r.x;
            red[tid][2 * h + 1] = r.y;
        }
        __syncthreads();
        for (int i = tid; i < lanes * V; i += NT) {
            const int l = i / V, c = i % V, ch = (cb * lanes + l) * V + c;
            if (ch >= p.D) continue;
            float s = 0.f;
            for (int q = 0; q < subs; ++q) s += red[q * lanes + l][c];
            part[j < W ? (size_t)ch * W + j : (size_t)p.D * W + ch] = s;
        }
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

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
    return bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) : cudaSuccess;
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
    const long long work = (runs + subs - 1) / subs * cblocks;
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
    constexpr int RUN = 4 * BATCH<T>;  // conv_bwd_run(a.dtype)
    const int parts = conv_bwd_parts(a.B, a.T, a.D, a.W, RUN);
    const size_t smem = (size_t)(2 * RUN + 3 * (W - 1)) * CONV_BWD_NT * sizeof(Pack<T, 4>);
    auto go = [&](auto kernel) {
        const cudaError_t e = allow_smem(kernel, smem);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)parts * cblocks, CONV_BWD_NT, smem, a.stream>>>(a, vecs, lanes, cblocks, parts, conv_bwd_runs(a.T, a.W, RUN));
        return cudaGetLastError();
    };
    const cudaError_t e = go(a.silu ? conv_bwd_kernel<T, W, true> : conv_bwd_kernel<T, W, false>);
    if (e != cudaSuccess) return e;
    return launch_sum_parts(a.ws, parts, a.D * (a.dbias ? W + 1 : W), a.dw, a.dbias, a.D * W, a.stream);
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
