// Selective state space scan, forward (ssm.cuh has the formulas).
//
// The work is N exponentials and 3 N multiply-adds a token and channel, on inputs and outputs of a few bytes: bound
// by the exponential unit (32 a clock and SM) and the fp32 pipe (128), not by HBM.  So a thread keeps 16 entries of
// one channel's state in registers over all tokens of its segment (N / 16 lanes a channel, their shares of C . h
// added by shuffles) and computes delta itself; only B and C, which all channels share, go through shared memory as
// fp32.  Multiply-adds run packed in pairs, which leaves the issue slots to the exponentials.  Inputs come in
// stages of 16 tokens by asynchronous copies two stages ahead; B and C of the next stage are converted while this
// one is computed, so a stage costs one barrier.
#include "ssm.cuh"

namespace efla {
namespace {

constexpr int NT = SSM_NT, TOK = SSM_TOK, PER = SSM_PER, STAGES = 3;

// CARRY: end state and sum of delta of a segment from h = 0, no outputs.
template <typename T, int NSUB, bool CARRY>
struct Scan {
    static constexpr int N = NSUB * PER, CT = NT / NSUB;
    static constexpr int ROW = CT * sizeof(T), BROW = N * sizeof(T);        // bytes a token
    static constexpr int X = 0, DT = TOK * ROW, Z = 2 * TOK * ROW, B = 3 * TOK * ROW, C = B + TOK * BROW;
    static constexpr int STAGE = C + TOK * BROW, CVT = 2 * TOK * N * 4;      // bytes a stage; of B and C as fp32
    static constexpr int SMEM = STAGES * STAGE + 2 * CVT;
};

// Where entry n of token t's B or C lies: the lanes of a channel read 16 bytes each side by side.
template <int NSUB>
__device__ __forceinline__ int cvt_at(int n) { return ((n % PER / 4) * NSUB + n / PER) * 4 + n % 4; }

template <typename T, int NSUB, bool CARRY>
__global__ void __launch_bounds__(NT) ssm_fwd_kernel(SsmArgs p, int tiles) {
    using K = Scan<T, NSUB, CARRY>;
    constexpr int N = K::N, CT = K::CT;
    extern __shared__ __align__(16) uint8_t smem[];
    float *cvt = reinterpret_cast<float *>(smem + STAGES * K::STAGE);  // [2][B, C][TOK][N]
    const int tid = threadIdx.x, tile = blockIdx.x % tiles, slot = blockIdx.x / tiles;
    SsmSpan span;
    if (p.cu_seqlens) {
        if (!ssm_packed_span(p, slot, tile == 0, span)) return;
    } else {
        span = ssm_row_span(p, slot);
    }
    const int each = p.D / p.G, tpg = tiles / p.G, g = tile / tpg, c0 = g * each + tile % tpg * CT;
    const int have = min(CT, (g + 1) * each - c0);  // channels of the tile
    const int c = tid / NSUB, sub = tid % NSUB, d = c0 + c;
    const bool live = c < have;

    float2 rate[PER / 2], h[PER / 2];
    float bias = 0.f, skip = 0.f, total = 0.f;
    const size_t at = (size_t)(live ? d : 0) * N + sub * PER;
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) {
        const float2 a = reinterpret_cast<const float2 *>(p.A_log + at)[i];
        rate[i] = make_float2(ssm_rate(a.x), ssm_rate(a.y));
        h[i] = make_float2(0.f, 0.f);
    }
    if (live) {
        if (p.dt_bias) bias = p.dt_bias[d];
        if (p.Dskip) skip = p.Dskip[d];
        const float *h0 = CARRY ? nullptr : p.seg ? p.state + (size_t)slot * p.D * N : p.S0 ? p.S0 + (size_t)span.seq * p.D * N : nullptr;
        if (h0) {
#pragma unroll
            for (int i = 0; i < PER / 2; ++i) h[i] = reinterpret_cast<const float2 *>(h0 + at)[i];
        }
    }

    const uint8_t *xg = static_cast<const uint8_t *>(p.x) + (size_t)c0 * sizeof(T);
    const uint8_t *dg = static_cast<const uint8_t *>(p.dt) + (size_t)c0 * sizeof(T);
    const uint8_t *zg = p.z ? static_cast<const uint8_t *>(p.z) + (size_t)c0 * sizeof(T) : nullptr;
    const uint8_t *bg = static_cast<const uint8_t *>(p.Bm) + (size_t)g * N * sizeof(T);
    const uint8_t *cg = static_cast<const uint8_t *>(p.Cm) + (size_t)g * N * sizeof(T);
    const size_t pitch = (size_t)p.D * sizeof(T), bpitch = (size_t)p.G * N * sizeof(T);
    const int pieces = have * (int)sizeof(T) / 16;
    auto load = [&](int s) {
        const long long t0 = span.lo + (long long)s * TOK;
        if (t0 < span.hi) {
            uint8_t *st = smem + s % STAGES * K::STAGE;
            load_tile<K::ROW / 16>(st + K::X, xg, pitch, t0, span.hi, pieces);
            load_tile<K::ROW / 16>(st + K::DT, dg, pitch, t0, span.hi, pieces);
            load_tile<K::BROW / 16>(st + K::B, bg, bpitch, t0, span.hi, K::BROW / 16);
            if (!CARRY) {
                if (zg) load_tile<K::ROW / 16>(st + K::Z, zg, pitch, t0, span.hi, pieces);
                load_tile<K::BROW / 16>(st + K::C, cg, bpitch, t0, span.hi, K::BROW / 16);
            }
        }
        cp_async_commit();
    };
    auto convert = [&](int s) {
        const uint8_t *st = smem + s % STAGES * K::STAGE;
        float *to = cvt + (s & 1) * 2 * TOK * N;
#pragma unroll
        for (int k = 0; k < TOK * N / NT; ++k) {
            const int i = k * NT + tid, t = i / N, n = i % N;
            to[t * N + cvt_at<NSUB>(n)] = to_f32(reinterpret_cast<const T *>(st + K::B)[i]);
            if (!CARRY) to[TOK * N + t * N + cvt_at<NSUB>(n)] = to_f32(reinterpret_cast<const T *>(st + K::C)[i]);
        }
    };

    const int stages = (int)((span.hi - span.lo + TOK - 1) / TOK);
    load(0);
    load(1);
    cp_async_wait<1>();
    __syncthreads();
    if (stages > 0) convert(0);
    for (int s = 0; s < stages; ++s) {
        cp_async_wait<0>();
        __syncthreads();  // stage s + 1 has arrived, B and C of stage s are converted, stage s - 1 is done with
        if (s + 1 < stages) convert(s + 1);
        load(s + 2);
        const uint8_t *st = smem + s % STAGES * K::STAGE;
        const float *bc = cvt + (s & 1) * 2 * TOK * N + sub * 4;
        const long long t0 = span.lo + (long long)s * TOK;
        const int count = (int)min((long long)TOK, span.hi - t0);
        if (!CARRY && p.keep && live) {
            const int row = (int)(t0 / p.T), nk = (p.T + TOK - 1) / TOK;
            float2 *k = reinterpret_cast<float2 *>(p.keep + ((size_t)row * nk + (size_t)(t0 - (long long)row * p.T) / TOK) * p.D * N + at);
#pragma unroll
            for (int i = 0; i < PER / 2; ++i) k[i] = h[i];
        }
#pragma unroll 4
        for (int t = 0; t < count; ++t) {
            const float x = to_f32(reinterpret_cast<const T *>(st + K::X)[t * CT + c]);
            const float delta = softplus(to_f32(reinterpret_cast<const T *>(st + K::DT)[t * CT + c]) + bias);
            const float u = delta * x;
            const float2 delta2 = make_float2(delta, delta), u2 = make_float2(u, u);
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int j = 0; j < PER / 4; ++j) {
                const float4 b = *reinterpret_cast<const float4 *>(bc + t * N + j * NSUB * 4);
                const float2 e0 = __fmul2_rn(delta2, rate[2 * j]), e1 = __fmul2_rn(delta2, rate[2 * j + 1]);
                h[2 * j] = __ffma2_rn(make_float2(ssm_ex2(e0.x), ssm_ex2(e0.y)), h[2 * j], __fmul2_rn(u2, make_float2(b.x, b.y)));
                h[2 * j + 1] = __ffma2_rn(make_float2(ssm_ex2(e1.x), ssm_ex2(e1.y)), h[2 * j + 1], __fmul2_rn(u2, make_float2(b.z, b.w)));
                if (!CARRY) {
                    const float4 cc = *reinterpret_cast<const float4 *>(bc + TOK * N + t * N + j * NSUB * 4);
                    acc[0] = __ffma2_rn(h[2 * j], make_float2(cc.x, cc.y), acc[0]);
                    acc[1] = __ffma2_rn(h[2 * j + 1], make_float2(cc.z, cc.w), acc[1]);
                }
            }
            if (CARRY) {
                total += delta;
            } else {
                float y = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
#pragma unroll
                for (int off = 1; off < NSUB; off <<= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
                y = fmaf(skip, x, y);
                if (p.z) {
                    const float z = to_f32(reinterpret_cast<const T *>(st + K::Z)[t * CT + c]);
                    y *= z * ssm_sigmoid(z);
                }
                if (live && sub == 0 && p.y) static_cast<T *>(p.y)[(size_t)(t0 + t) * p.D + d] = from_f32<T>(y);
            }
        }
    }
    if (!live) return;
    if (CARRY) {
        float2 *to = reinterpret_cast<float2 *>(p.state + (size_t)slot * p.D * N + at);
#pragma unroll
        for (int i = 0; i < PER / 2; ++i) to[i] = h[i];
        if (sub == 0) p.sum[(size_t)slot * p.D + d] = total;
    } else if (p.S_T && !p.seg) {
        float2 *to = reinterpret_cast<float2 *>(p.S_T + (size_t)span.seq * p.D * N + at);
#pragma unroll
        for (int i = 0; i < PER / 2; ++i) to[i] = h[i];
    }
}

// Start states of a row's or sequence's segments from their local end states, in place, and its last state.
// A thread an entry of the state; blockIdx.y the row.
__global__ void __launch_bounds__(NT) ssm_combine_kernel(SsmArgs p) {
    __shared__ int box[NT / 32];
    const int row = blockIdx.y, tid = threadIdx.x;
    int first, segs;
    if (p.cu_seqlens) {
        long long lo, hi;
        segs = ssm_segments(p, row, lo, hi);
        if (segs < 0) return;
        int n = 0;
        for (int i = tid; i < row; i += NT) n += max(0, ssm_segments(p, i, lo, hi));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
        if ((tid & 31) == 0) box[tid >> 5] = n;
        __syncthreads();
        first = 0;
        for (int w = 0; w < NT / 32; ++w) first += box[w];
        if (first + segs > p.slots) return;  // sequences that overlap
    } else {
        segs = (p.T + p.seg - 1) / p.seg;
        first = row * segs;
    }
    const size_t e = (size_t)blockIdx.x * NT + tid, size = (size_t)p.D * p.N;
    if (e >= size) return;
    const float rate = ssm_rate(p.A_log[e]);
    float h = p.S0 ? p.S0[row * size + e] : 0.f;
    float *state = p.state + first * size + e;
    const float *sum = p.sum + (size_t)first * p.D + e / p.N;
#pragma unroll 8
    for (int s = 0; s < segs; ++s) {
        const float local = state[s * size];
        state[s * size] = h;
        h = fmaf(ssm_ex2(rate * sum[(size_t)s * p.D]), h, local);
    }
    if (p.S_T) p.S_T[row * size + e] = h;
}

template <typename T, int NSUB, bool CARRY>
cudaError_t run(const SsmArgs &a, long long slots, int tiles) {
    using K = Scan<T, NSUB, CARRY>;
    if (K::SMEM > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(ssm_fwd_kernel<T, NSUB, CARRY>, cudaFuncAttributeMaxDynamicSharedMemorySize, K::SMEM);
        if (e != cudaSuccess) return e;
    }
    ssm_fwd_kernel<T, NSUB, CARRY><<<(unsigned)(slots * tiles), NT, K::SMEM, a.stream>>>(a, tiles);
    return cudaGetLastError();
}

template <typename T, int NSUB>
cudaError_t forward(const SsmArgs &a) {
    const int tiles = ssm_tiles(a.D, a.N, a.G);
    const long long slots = a.seg ? a.slots : a.nseq;
    if (a.seg) {
        cudaError_t e = run<T, NSUB, true>(a, slots, tiles);
        if (e != cudaSuccess) return e;
        const dim3 grid((unsigned)(((size_t)a.D * a.N + NT - 1) / NT), a.nseq);
        ssm_combine_kernel<<<grid, NT, 0, a.stream>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return run<T, NSUB, false>(a, slots, tiles);
}

template <typename T>
cudaError_t states(const SsmArgs &a) {
    return a.N == 16 ? forward<T, 1>(a) : a.N == 32 ? forward<T, 2>(a) : a.N == 64 ? forward<T, 4>(a) : forward<T, 8>(a);
}

// ------------------------------------------------------------------------------------ one token
// HBM bound: the state is read and written once (8 N bytes a channel; everything else is a few).  A thread has four
// entries of one channel's state and takes ROWS sequences, so that the rates are computed once for them.
constexpr int STEP_NT = 128;
template <typename T, int N, int ROWS>
__global__ void __launch_bounds__(STEP_NT) ssm_step_kernel(SsmArgs p) {
    constexpr int LN = N / 4, CT = STEP_NT / LN;
    const int tid = threadIdx.x, l = tid % LN, blocks = (p.D + CT - 1) / CT;
    const int d = blockIdx.x % blocks * CT + tid / LN, b0 = blockIdx.x / blocks * ROWS;
    const bool live = d < p.D;
    const int dd = live ? d : p.D - 1, each = p.D / p.G, g = dd / each;
    float4 h[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
        if (b0 + r < p.B) h[r] = *reinterpret_cast<const float4 *>(p.S0 + ((size_t)(b0 + r) * p.D + dd) * N + 4 * l);
    const float4 al = *reinterpret_cast<const float4 *>(p.A_log + (size_t)dd * N + 4 * l);
    const float rate[4] = {ssm_rate(al.x), ssm_rate(al.y), ssm_rate(al.z), ssm_rate(al.w)};
    const float bias = p.dt_bias ? p.dt_bias[dd] : 0.f, skip = p.Dskip ? p.Dskip[dd] : 0.f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int b = b0 + r;
        if (b >= p.B) break;
        const size_t e = (size_t)b * p.D + dd, m = ((size_t)b * p.G + g) * N + 4 * l;
        const float x = to_f32(static_cast<const T *>(p.x)[e]);
        const float delta = softplus(to_f32(static_cast<const T *>(p.dt)[e]) + bias), u = delta * x;
        const T *B = static_cast<const T *>(p.Bm) + m, *C = static_cast<const T *>(p.Cm) + m;
        float hv[4] = {h[r].x, h[r].y, h[r].z, h[r].w}, y = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hv[i] = fmaf(ssm_ex2(delta * rate[i]), hv[i], u * to_f32(B[i]));
            y = fmaf(hv[i], to_f32(C[i]), y);
        }
#pragma unroll
        for (int off = 1; off < LN; off <<= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
        y = fmaf(skip, x, y);
        if (p.z) {
            const float z = to_f32(static_cast<const T *>(p.z)[e]);
            y *= z * ssm_sigmoid(z);
        }
        if (live) {
            *reinterpret_cast<float4 *>(p.S_T + e * N + 4 * l) = make_float4(hv[0], hv[1], hv[2], hv[3]);
            if (l == 0) static_cast<T *>(p.y)[e] = from_f32<T>(y);
        }
    }
}

template <typename T, int N>
cudaError_t step(const SsmArgs &a) {
    constexpr int ROWS = 4;
    const long long blocks = (a.D + STEP_NT / (N / 4) - 1) / (STEP_NT / (N / 4));
    if (a.B * blocks <= 304 * ROWS)
        ssm_step_kernel<T, N, 1><<<(unsigned)(a.B * blocks), STEP_NT, 0, a.stream>>>(a);
    else
        ssm_step_kernel<T, N, ROWS><<<(unsigned)((a.B + ROWS - 1) / ROWS * blocks), STEP_NT, 0, a.stream>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t step_states(const SsmArgs &a) {
    return a.N == 16 ? step<T, 16>(a) : a.N == 32 ? step<T, 32>(a) : a.N == 64 ? step<T, 64>(a) : step<T, 128>(a);
}

}  // namespace

int ssm_segment(long long rows, int T, int tiles) {
    // Enough CTAs for two a SM, but segments of 64 tokens at least.
    const long long units = rows * tiles, want = 152 * 2;
    if (units <= 0 || 2 * units > want || T < 128) return 0;
    const long long parts = std::min<long long>(want / units, (T + 63) / 64);
    const long long seg = (T + parts - 1) / parts;
    return (int)((seg + SSM_TOK - 1) / SSM_TOK * SSM_TOK);
}

cudaError_t launch_ssm_scan(const SsmArgs &a) { return a.dtype == EFLA_BF16 ? states<__nv_bfloat16>(a) : states<float>(a); }
cudaError_t launch_ssm_step(const SsmArgs &a) {
    return a.dtype == EFLA_BF16 ? step_states<__nv_bfloat16>(a) : step_states<float>(a);
}

}  // namespace efla
