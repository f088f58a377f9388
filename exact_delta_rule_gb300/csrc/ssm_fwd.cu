// Selective state space scan, forward (ssm.cuh has the formulas).
//
// The work is N exponentials and 3 N multiply-adds a token and channel, on inputs and outputs of a few bytes: HBM is far
// from its bound (8 x 2048 tokens of 4096 channels, N = 16, bf16: 409 us for 540 MB).  A warp's token of 32 x 16 entries
// is 118 instructions and takes 170 clocks of a scheduler that has many, 191 each with two, 326 with one.
// What takes them is neither issue (0.65) nor the exponential unit (leaving the exponentials out changes nothing) but
// the registers' read ports: a packed multiply-add of three different operands takes 2.4 to 3 clocks, one with a
// constant 2, so 32 of them are 85 of the 170; gates and outputs are 50, copies and conversions 12.
//
// A thread keeps 2 channels x 8 entries of the state in registers over all tokens of its segment, so that B and C, which
// all channels share, are read from shared memory (as fp32) once for both channels; multiply-adds run packed in pairs of
// entries, and what the next token needs before it meets the state is computed between this one's
// multiply-adds (8 % at 19456 channels).  Tokens go in groups of four, 16 in straight code.  Their softplus
// and gate are shared out among the N / 8 lanes of a pair of channels: the lane that computes a token's delta also gets
// its sum of C . h and writes its output; a lane keeps its own channel first, so that two lanes swap what belongs to
// the other without selecting.  A CTA is one warp (two for N = 128): 8 x 2048 tokens of 4096 channels are 1024 warps, 6.7
// a SM.  Other splits of the state, at that size: 1 channel x 8 entries 449 us, 1 x 16 406 to 524, 2 x 4 427; eight tokens
// in straight code 443, four 540 (copies between registers).
// Inputs come in stages of 16 tokens by asynchronous copies two stages ahead; B and C of the next stage are converted
// while this one is computed, so a stage costs one barrier.
#include "ssm.cuh"
#include "vec.cuh"

namespace efla {
namespace {

constexpr int TOK = SSM_TOK, PER = 8, STAGES = 3;

// CARRY: end state and sum of delta of a segment from h = 0, no outputs.
template <typename T, int N_, bool CARRY>
struct Scan {
    static constexpr int N = N_, NT = ssm_fwd_threads(N), CT = ssm_fwd_channels(N), SUB = N / PER;
    static constexpr int TL = SUB / 2 < 4 ? SUB / 2 : 4, LOC = 4 / TL;  // lanes that share four tokens; tokens a lane
    static constexpr int ROW = CT * sizeof(T), BROW = N * sizeof(T);        // bytes a token
    static constexpr int X = 0, DT = TOK * ROW, Z = 2 * TOK * ROW, B = 3 * TOK * ROW, C = B + TOK * BROW;
    static constexpr int STAGE = C + TOK * BROW, CVT = 2 * TOK * N * 4;      // bytes a stage; of B and C as fp32
    static constexpr int SMEM = STAGES * STAGE + 2 * CVT;
};

__device__ __forceinline__ void unpack8(const __nv_bfloat16 *src, float4 &a, float4 &b) {
    const uint4 r = *reinterpret_cast<const uint4 *>(src);
    a = make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
    b = make_float4(__uint_as_float(r.z << 16), __uint_as_float(r.z & 0xffff0000u), __uint_as_float(r.w << 16), __uint_as_float(r.w & 0xffff0000u));
}
__device__ __forceinline__ void unpack8(const float *src, float4 &a, float4 &b) {
    a = reinterpret_cast<const float4 *>(src)[0];
    b = reinterpret_cast<const float4 *>(src)[1];
}

// Sums of y[0..3] over the SUB / 2 lanes that differ in the bits above the lowest: token k's ends in the lanes of
// (sub / 2) % TL = k % TL, at out[k / TL].
template <int SUB, int LOC>
__device__ __forceinline__ void owner_sums(const float (&y)[4], int sub, float (&out)[LOC]) {
    if constexpr (SUB == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = y[k];
    } else if constexpr (SUB == 4) {
        const bool up = sub & 2;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            out[i] = (up ? y[2 * i + 1] : y[2 * i]) + __shfl_xor_sync(0xffffffffu, up ? y[2 * i] : y[2 * i + 1], 2);
    } else {
        const bool b1 = sub & 4, b0 = sub & 2;
        const float v0 = (b1 ? y[2] : y[0]) + __shfl_xor_sync(0xffffffffu, b1 ? y[0] : y[2], 4);
        const float v1 = (b1 ? y[3] : y[1]) + __shfl_xor_sync(0xffffffffu, b1 ? y[1] : y[3], 4);
        out[0] = (b0 ? v1 : v0) + __shfl_xor_sync(0xffffffffu, b0 ? v0 : v1, 2);
        #pragma unroll
        for (int off = 8; off < SUB; off <<= 1) out[0] += __shfl_xor_sync(0xffffffffu, out[0], off);
    }
}

template <typename T, int N, bool CARRY>
__global__ void __launch_bounds__(ssm_fwd_threads(N)) ssm_fwd_kernel(SsmArgs p, int tiles) {
    using K = Scan<T, N, CARRY>;
    constexpr int NT = K::NT, CT = K::CT, SUB = K::SUB, TL = K::TL, LOC = K::LOC;
    extern __shared__ __align__(16) uint8_t smem[];
    float *cvt = reinterpret_cast<float *>(smem + STAGES * K::STAGE);  // [2][B, C][TOK][N]
    const int tid = threadIdx.x, tile = blockIdx.x % tiles, slot = blockIdx.x / tiles;
    SsmSpan span;
    if (p.cu_seqlens) {
        if (!ssm_packed_span<NT>(p, slot, tile == 0, span)) return;
    } else {
        span = ssm_row_span(p, slot);
    }
    const int each = p.D / p.G, tpg = tiles / p.G, g = tile / tpg, c0 = g * each + tile % tpg * CT;
    const int have = min(CT, (g + 1) * each - c0);  // channels of the tile
    // this lane's channel, and of the other (its partner lane's) the same entries
    const int sub = tid % SUB, c = tid / SUB * 2 + (sub & 1), d = c0 + c, mine = sub / 2 % TL;
    const bool live = c < have;  // (tiles have a multiple of 4 channels)

    float2 rate[2][PER / 2], h[2][PER / 2];
    float bias = 0.f, skip = 0.f, total = 0.f;
    size_t at[2];
    const float *h0 = CARRY ? nullptr : p.seg ? p.state + (size_t)slot * p.D * N : p.S0 ? p.S0 + (size_t)span.seq * p.D * N : nullptr;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        at[q] = (size_t)(live ? c0 + (c ^ q) : 0) * N + sub * PER;
#pragma unroll
        for (int i = 0; i < PER / 2; ++i) {
            const float2 a = reinterpret_cast<const float2 *>(p.A_log + at[q])[i];
            rate[q][i] = make_float2(ssm_rate(a.x), ssm_rate(a.y));
            h[q][i] = live && h0 ? reinterpret_cast<const float2 *>(h0 + at[q])[i] : make_float2(0.f, 0.f);
        }
    }
    if (live) {
        if (p.dt_bias) bias = p.dt_bias[d];
        if (p.Dskip) skip = p.Dskip[d];
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
            load_tile<K::ROW / 16, NT>(st + K::X, xg, pitch, t0, span.hi, pieces);
            load_tile<K::ROW / 16, NT>(st + K::DT, dg, pitch, t0, span.hi, pieces);
            load_tile<K::BROW / 16, NT>(st + K::B, bg, bpitch, t0, span.hi, K::BROW / 16);
            if (!CARRY) {
                if (zg) load_tile<K::ROW / 16, NT>(st + K::Z, zg, pitch, t0, span.hi, pieces);
                load_tile<K::BROW / 16, NT>(st + K::C, cg, bpitch, t0, span.hi, K::BROW / 16);
            }
        }
        cp_async_commit();
    };
    // Entry n of a token's B or C goes to ((n % 8 / 4) SUB + n / 8) 4 + n % 4: the lanes of a channel read 16 bytes side by side.
    auto convert = [&](int s) {
        const uint8_t *st = smem + s % STAGES * K::STAGE;
        float4 *to = reinterpret_cast<float4 *>(cvt + (s & 1) * 2 * TOK * N);
        constexpr int V = TOK * N / 8;  // eights of B; those of C follow
        static_assert(V % NT == 0, "whole passes");
#pragma unroll
        for (int k = 0; k < (CARRY ? 1 : 2) * V / NT; ++k) {
            const int i = k * NT + tid;
            const int t = i % V / (N / 8), e = i % (N / 8);
            float4 a, b;
            unpack8(reinterpret_cast<const T *>(st + (i < V ? K::B : K::C)) + t * N + 8 * e, a, b);
            float4 *at = to + (i / V * TOK + t) * (N / 4) + e;
            at[0] = a;
            at[SUB] = b;
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
            float *k = p.keep + ((size_t)row * nk + (size_t)(t0 - (long long)row * p.T) / TOK) * p.D * N;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < PER / 4; ++i)
                    reinterpret_cast<float4 *>(k + at[q])[i] = make_float4(h[q][2 * i].x, h[q][2 * i].y, h[q][2 * i + 1].x, h[q][2 * i + 1].y);
        }
        // x, delta and u = delta x of this lane's channel and tokens of a group: those of number `mine`, + TL, ..
        auto gates = [&](int tg, float(&x)[LOC], float(&delta)[LOC], float(&u)[LOC]) {
            float v[LOC];
#pragma unroll
            for (int i = 0; i < LOC; ++i) {
                const int t = tg + mine + i * TL;
                x[i] = to_f32(reinterpret_cast<const T *>(st + K::X)[t * CT + c]);
                v[i] = to_f32(reinterpret_cast<const T *>(st + K::DT)[t * CT + c]) + bias;
            }
            if constexpr (LOC > 1) {
#pragma unroll
                for (int i = 0; i < LOC; i += 2) {
                    const float2 r = softplus2(make_float2(v[i], v[i + 1]));
                    v[i] = r.x;
                    v[i + 1] = r.y;
                }
            } else {
                v[0] = softplus(v[0]);
            }
#pragma unroll
            for (int i = 0; i < LOC; ++i) {
                delta[i] = tg + mine + i * TL < count ? v[i] : 0.f;  // (past the end: a token that changes nothing)
                u[i] = delta[i] * x[i];
            }
        };
        // delta and u of token t of the group, of this lane's channel and of the other.
        auto steps = [&](int t, const float(&delta)[LOC], const float(&u)[LOC], float2(&dk)[2], float2(&uk)[2]) {
            const int k = t % 4;
            float d0 = delta[k / TL], u0 = u[k / TL], d1, u1;
            if (TL > 1) {  // from the lane of this token
                const int from = (threadIdx.x & 31 & ~(SUB - 1)) | (k % TL * 2) | (sub & 1);
                d1 = __shfl_sync(0xffffffffu, d0, from ^ 1);
                u1 = __shfl_sync(0xffffffffu, u0, from ^ 1);
                d0 = __shfl_sync(0xffffffffu, d0, from);
                u0 = __shfl_sync(0xffffffffu, u0, from);
            } else {
                d1 = __shfl_xor_sync(0xffffffffu, d0, 1);
                u1 = __shfl_xor_sync(0xffffffffu, u0, 1);
            }
            if (CARRY) total += d0;
            dk[0] = make_float2(d0, d0), dk[1] = make_float2(d1, d1);
            uk[0] = make_float2(u0, u0), uk[1] = make_float2(u1, u1);
        };
        auto fetch = [&](const float *from, float2(&v)[PER / 2]) {
#pragma unroll
            for (int j = 0; j < PER / 4; ++j) {
                const float4 r = *reinterpret_cast<const float4 *>(from + j * SUB * 4);
                v[2 * j] = make_float2(r.x, r.y);
                v[2 * j + 1] = make_float2(r.z, r.w);
            }
        };
        float x[LOC], delta[LOC], u[LOC];
        float2 a[2][PER / 2], ub[2][PER / 2], cc[PER / 2];
        gates(0, x, delta, u);
        {
            float2 dk[2], uk[2], b[PER / 2];
            steps(0, delta, u, dk, uk);
            fetch(bc, b);
            if (!CARRY) fetch(bc + TOK * N, cc);
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < PER / 2; ++i) {
                    const float2 e = ssm_exponent(dk[q], rate[q][i]);
                    a[q][i] = make_float2(ssm_ex2(e.x), ssm_ex2(e.y));
                    ub[q][i] = __fmul2_rn(uk[q], b[i]);
                }
        }
#pragma unroll
        for (int tg = 0; tg < TOK; tg += 4) {
            if (tg >= count) break;
            float xn[LOC], dn[LOC], un[LOC], y[4];
            if (tg + 4 < TOK) gates(tg + 4, xn, dn, un);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = tg + k;
                const bool more = t + 1 < TOK;
                float2 dk[2], uk[2], b[PER / 2], cn[PER / 2], acc[2], e[2][PER / 2];
                if (more) {
                    if (k < 3)
                        steps(t + 1, delta, u, dk, uk);
                    else
                        steps(t + 1, dn, un, dk, uk);
                    fetch(bc + (t + 1) * N, b);
                    if (!CARRY) fetch(bc + (TOK + t + 1) * N, cn);
                    e[0][0] = ssm_exponent(dk[0], rate[0][0]);
                }
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int i = 0; i < PER / 2; ++i) {
                        // this token's state and output between the exponentials of the next
                        constexpr int HALF = PER / 2;
                        const int nq = (q * HALF + i + 1) / HALF, ni = (i + 1) % HALF;
                        float2 an;
                        if (more) an.x = ssm_ex2_here(e[q][i].x);
                        h[q][i] = __ffma2_rn(a[q][i], h[q][i], ub[q][i]);
                        if (more) {
                            if (nq < 2) e[nq][ni] = ssm_exponent(dk[nq], rate[nq][ni]);
                            an.y = ssm_ex2_here(e[q][i].y);
                            ub[q][i] = __fmul2_rn(uk[q], b[i]);
                            a[q][i] = an;
                        }
                        if (!CARRY) acc[q] = i ? __ffma2_rn(h[q][i], cc[i], acc[q]) : __fmul2_rn(h[q][0], cc[0]);
                    }
                if (!CARRY) y[k] = acc[0].x + acc[0].y + __shfl_xor_sync(0xffffffffu, acc[1].x + acc[1].y, 1);
#pragma unroll
                for (int i = 0; i < PER / 2; ++i) cc[i] = cn[i];
            }
            if (!CARRY) {
                float out[LOC];
                owner_sums<SUB, LOC>(y, sub, out);
#pragma unroll
                for (int i = 0; i < LOC; ++i) {
                    const int t = tg + mine + i * TL;
                    out[i] = fmaf(skip, x[i], out[i]);
                    if (p.z) {
                        const float z = to_f32(reinterpret_cast<const T *>(st + K::Z)[t * CT + c]);
                        out[i] *= z * ssm_sigmoid(z);
                    }
                    if (live && sub < 8 && t < count && p.y) static_cast<T *>(p.y)[(size_t)(t0 + t) * p.D + d] = from_f32<T>(out[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < LOC; ++i) {
                x[i] = xn[i];
                delta[i] = dn[i];
                u[i] = un[i];
            }
        }
    }
    if (!live) return;
    float *end = CARRY ? p.state + (size_t)slot * p.D * N : p.S_T && !p.seg ? p.S_T + (size_t)span.seq * p.D * N : nullptr;
    if (end) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < PER / 2; ++i) reinterpret_cast<float2 *>(end + at[q])[i] = h[q][i];
    }
    if (CARRY && sub < 2) p.sum[(size_t)slot * p.D + d] = total;
}

// Start states of a row's or sequence's segments from their local end states, in place, and its last state.
// A thread an entry of the state; blockIdx.y the row.
constexpr int COMBINE_NT = 128;
__global__ void __launch_bounds__(COMBINE_NT) ssm_combine_kernel(SsmArgs p) {
    constexpr int NT = COMBINE_NT;
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
        segs = ssm_pieces(p.T, p.seg);
        first = row * segs;
    }
    const size_t e = (size_t)blockIdx.x * NT + tid, size = (size_t)p.D * p.N;
    if (e >= size) return;
    const float rate = ssm_rate(p.A_log[e]);
    float h = p.S0 ? p.S0[row * size + e] : 0.f;
    float *state = p.state + first * size + e;
    const float *sum = p.sum + (size_t)first * p.D + e / p.N;
    constexpr int BATCH = 8;  // (all loaded before the first is written back)
    for (int s0 = 0; s0 < segs; s0 += BATCH) {
        float local[BATCH], decay[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            local[i] = decay[i] = 0.f;
            if (s0 + i < segs) {
                local[i] = state[(s0 + i) * size];
                decay[i] = ssm_ex2(rate * sum[(size_t)(s0 + i) * p.D]);
            }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (s0 + i < segs) {
                state[(s0 + i) * size] = h;
                h = fmaf(decay[i], h, local[i]);
            }
    }
    if (p.S_T) p.S_T[row * size + e] = h;
}

template <typename T, int N, bool CARRY>
cudaError_t run(const SsmArgs &a, long long slots, int tiles) {
    using K = Scan<T, N, CARRY>;
    const cudaError_t e = allow_smem(ssm_fwd_kernel<T, N, CARRY>, K::SMEM);
    if (e != cudaSuccess) return e;
    ssm_fwd_kernel<T, N, CARRY><<<(unsigned)(slots * tiles), K::NT, K::SMEM, a.stream>>>(a, tiles);
    return cudaGetLastError();
}

template <typename T, int N>
cudaError_t forward(const SsmArgs &a) {
    const int tiles = ssm_fwd_tiles(a.D, a.N, a.G);
    const long long slots = a.seg ? a.slots : a.nseq;
    if (a.seg) {
        cudaError_t e = run<T, N, true>(a, slots, tiles);
        if (e != cudaSuccess) return e;
        const dim3 grid((unsigned)(((size_t)a.D * a.N + COMBINE_NT - 1) / COMBINE_NT), a.nseq);
        ssm_combine_kernel<<<grid, COMBINE_NT, 0, a.stream>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return run<T, N, false>(a, slots, tiles);
}

template <typename T>
cudaError_t states(const SsmArgs &a) {
    return a.N == 16 ? forward<T, 16>(a) : a.N == 32 ? forward<T, 32>(a) : a.N == 64 ? forward<T, 64>(a) : forward<T, 128>(a);
}

// ------------------------------------------------------------------------------------ one token
// HBM bound: the state is read and written once (8 N bytes a channel; everything else is a few).  A thread has four
// entries of one channel's state and takes ROWS sequences, so that the rates are computed once for them; all that it
// reads is under way before the first is used.  Of a row's scalars (softplus, gate, the output) each of four threads
// has one row's and hands them to the others: 256 sequences of 4096 channels, N = 16: 24 us (143 MB, 5.9 TB/s, what a
// multiplication in place reaches), in L2 18; 30 and 22 with every thread computing all four rows' scalars.
constexpr int STEP_NT = 128;
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 r = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
template <typename T, int N, int ROWS>
__global__ void __launch_bounds__(STEP_NT) ssm_step_kernel(SsmArgs p) {
    static_assert(ROWS == 1 || ROWS == 4, "a row for each of four threads");
    constexpr int LN = N / 4, CT = STEP_NT / LN;
    constexpr unsigned FULL = 0xffffffffu;
    const int tid = threadIdx.x, l = tid % LN, blocks = (p.D + CT - 1) / CT;
    const int d = blockIdx.x % blocks * CT + tid / LN, b0 = blockIdx.x / blocks * ROWS;
    const bool live = d < p.D;
    const int dd = live ? d : p.D - 1, each = p.D / p.G, g = dd / each;
    float4 h[ROWS], B[ROWS], C[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int b = min(b0 + r, p.B - 1);  // (a row past the last: the last again, not written)
        const size_t e = (size_t)b * p.D + dd, m = ((size_t)b * p.G + g) * N + 4 * l;
        h[r] = *reinterpret_cast<const float4 *>(p.S0 + e * N + 4 * l);
        B[r] = load4(static_cast<const T *>(p.Bm) + m);
        C[r] = load4(static_cast<const T *>(p.Cm) + m);
    }
    const int mine = l % ROWS;  // the row whose scalars are this thread's
    const size_t own = (size_t)min(b0 + mine, p.B - 1) * p.D + dd;
    const float x = to_f32(static_cast<const T *>(p.x)[own]), dt = to_f32(static_cast<const T *>(p.dt)[own]);
    const float z = p.z ? to_f32(static_cast<const T *>(p.z)[own]) : 0.f;
    const float4 al = *reinterpret_cast<const float4 *>(p.A_log + (size_t)dd * N + 4 * l);
    const float rate[4] = {ssm_rate(al.x), ssm_rate(al.y), ssm_rate(al.z), ssm_rate(al.w)};
    const float bias = p.dt_bias ? p.dt_bias[dd] : 0.f, skip = p.Dskip ? p.Dskip[dd] : 0.f;
    const float step = softplus(dt + bias), in = step * x;
    float y[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const float delta = __shfl_sync(FULL, step, r, ROWS), u = __shfl_sync(FULL, in, r, ROWS);
        h[r].x = fmaf(ssm_ex2(ssm_exponent(delta, rate[0])), h[r].x, u * B[r].x);
        h[r].y = fmaf(ssm_ex2(ssm_exponent(delta, rate[1])), h[r].y, u * B[r].y);
        h[r].z = fmaf(ssm_ex2(ssm_exponent(delta, rate[2])), h[r].z, u * B[r].z);
        h[r].w = fmaf(ssm_ex2(ssm_exponent(delta, rate[3])), h[r].w, u * B[r].w);
        y[r] = fmaf(h[r].x, C[r].x, h[r].y * C[r].y) + fmaf(h[r].z, C[r].z, h[r].w * C[r].w);
        if (live && b0 + r < p.B) *reinterpret_cast<float4 *>(p.S_T + ((size_t)(b0 + r) * p.D + dd) * N + 4 * l) = h[r];
    }
    // Sums over the state: with four rows, half of them go to the neighbour at each of two exchanges, so that row l ends here.
    float sum = y[0];
    if constexpr (ROWS == 4) {
        const bool odd = l & 1, high = l & 2;
        const float a = (odd ? y[1] : y[0]) + __shfl_xor_sync(FULL, odd ? y[0] : y[1], 1);
        const float c = (odd ? y[3] : y[2]) + __shfl_xor_sync(FULL, odd ? y[2] : y[3], 1);
        sum = (high ? c : a) + __shfl_xor_sync(FULL, high ? a : c, 2);
    }
#pragma unroll
    for (int off = ROWS; off < LN; off <<= 1) sum += __shfl_xor_sync(FULL, sum, off);
    sum = fmaf(skip, x, sum);
    if (p.z) sum *= z * ssm_sigmoid(z);
    if (live && l < ROWS && b0 + l < p.B) static_cast<T *>(p.y)[own] = from_f32<T>(sum);
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

namespace {
// How many segments to cut a row of T tokens into: the number of the least estimated time.  A token costs one(w) clocks
// on a unit of the GPU (of which there are `places`) that has w of the `work` pieces of a row's length, all rows
// together; cutting costs `carry` of that again, and `step` a segment (its state through HBM: 8 bytes an entry).  Rows of
// uneven lengths take longer by `uneven` / w: the more pieces a unit has, the more they even out.
template <typename F>
int cut(long long work, int T, int places, F one, double carry, double step, double uneven) {
    if (work <= 0) return 0;
    int best = 1;
    double least = 0.;
    const int most = std::max(1, std::min(T / 64, 4096));
    for (int p = 1; p <= most; p += 1 + p / 32) {
        const long long w = (work * p + places - 1) / places;
        const int tokens = ((T + p - 1) / p + SSM_TOK - 1) / SSM_TOK * SSM_TOK;
        const double t = tokens * one(w) * (p > 1 ? 1. + carry : 1.) * (1. + uneven / w) + step * p;
        if (p == 1 || t < least) best = p, least = t;
    }
    if (best == 1) return 0;
    return ((T + best - 1) / best + SSM_TOK - 1) / SSM_TOK * SSM_TOK;
}
}  // namespace

// (Of packed sequences only the mean length is known here: below 128 tokens of it nothing is cut, so one long sequence among
// many short ones runs as long as its tokens one after the other.  200 of 20 tokens and one of 12000, 2048 channels, N = 16,
// bf16: 2.3 ms; the long one in a call of its own 0.21.)
// A scheduler (608) with one warp takes 326 clocks a token, with more 183 each; the carry kernel 0.55 of the scan's
// (8 x 2048 tokens of 2432, 4864 and 7296 channels, N = 16: 347, 407 and 567 us whole).
int ssm_segment(long long rows, int T, int D, int N, bool uneven) {
    if (rows > 65535) return 0;  // (the combine kernel's grid; rows enough without)
    return cut(rows * (((long long)D * N + 511) / 512), T, 608, [](long long w) { return w == 1 ? 326. : 183. * w; }, 0.55,
               600. + 0.0023 * rows * D * N, uneven ? 2. : 0.);
}
// A SM (152) with two CTAs takes 1528 clocks for a token of both, with one 1086; the carry 0.2 of that.
int ssm_bwd_segment(long long rows, int T, int D, int N, int tiles) {
    if (rows > 65535) return 0;
    return cut(rows * tiles, T, 152, [](long long w) { return w / 2 * 1528. + w % 2 * 1086.; }, 0.2, 600. + 0.0092 * rows * D * N, 0.);
}

cudaError_t launch_ssm_scan(const SsmArgs &a) { return a.dtype == EFLA_BF16 ? states<__nv_bfloat16>(a) : states<float>(a); }
cudaError_t launch_ssm_step(const SsmArgs &a) {
    return a.dtype == EFLA_BF16 ? step_states<__nv_bfloat16>(a) : step_states<float>(a);
}

}  // namespace efla
