// Selective state space scan, reverse mode (ssm.cuh has the forward's formulas).  With g_t = dy_t silu(z_t) and
// u_t = delta_t x_t, from the last token to the first (l: the gradient of h_t):
//   l_t = g_t C_t + a_{t+1} l_{t+1},  a_t = e^{A delta_t}         dC_t = sum_d g_t h_t,  dB_t = sum_d l_t u_t
//   du_t = l_t . B_t,  w_t = a_t l_t h_{t-1},  ddelta_t = w_t . A + du_t x_t,   dA = sum_t w_t delta_t
//   dx = du delta + D g,  ddt = ddelta sigmoid(dt + dt_bias),  dz = dy (C . h + D x) silu'(z),
//   dA_log = A dA,  dD = sum g x,  ddt_bias = sum ddt,  dS0 = a_1 l_1
//
// The forward keeps the state at every 16th token.  A CTA takes its segment's chunks of 16 tokens from last to first:
// from the kept state it recomputes h up to each quarter of the chunk (three are set aside in shared memory), then,
// last quarter first, recomputes the quarter's four tokens with h and a of each in registers, and goes back over them.
//
// About 19 multiply-adds and 1.75 exponentials an entry of the state, 360 instructions a warp's token of 32 x 16
// entries: bound like the forward by issue and the registers' read ports (114 packed multiply-adds), at the two warps a
// scheduler that 255 registers leave.  8 x 2048 tokens of 2048 channels, N = 16, bf16: 640 us.  A thread
// has 4 channels x 4 entries: a token's sums over the entries (of du, ddelta and y; over the N / 4 lanes of a
// channel) and over the channels (of dB and dC; over the others) then take 14 shuffles for 16 entries, the fewest of
// all splits of 16; their first step needs no selecting (reduce4).  Elementwise work goes in pairs of channels, by each
// warp on its own channels, so a chunk costs two barriers.  Sums over the four warps of a CTA go through shared memory and
// those over the CTAs through the workspace, all in a fixed order.
#include "mixer_norm.cuh"
#include "ssm.cuh"
#include "vec.cuh"

namespace efla {
namespace {

constexpr int NT = SSM_BWD_NT, TOK = SSM_TOK, WARPS = NT / 32;
constexpr float LN2 = 0.693147181f;

template <typename T, int LN>
struct Back {
    static constexpr int N = 4 * LN, CG = 32 / LN, CT = WARPS * CG * 4;  // entries; channel quads a warp; channels a CTA
    static constexpr int ROW = CT * sizeof(T), BROW = N * sizeof(T);
    static constexpr int X = 0, DT = TOK * ROW, Z = 2 * TOK * ROW, DY = 3 * TOK * ROW, B = 4 * TOK * ROW, C = B + TOK * BROW;
    static constexpr int STAGE = C + TOK * BROW;                 // bytes of a chunk's inputs; two of them
    static constexpr int F = 2 * STAGE, FROW = TOK * CT * 4;     // fp32 [TOK][CT]: delta, u then du, g then ddelta, C . h
    static constexpr int BC = F + 4 * FROW;                      // B, C as fp32, every value twice: [2][TOK][N] float2
    static constexpr int KEPT = BC + 2 * TOK * N * 8;            // three states a thread: [3][4][NT] float4
    static constexpr int RED = KEPT + 3 * 4 * NT * 16;           // a warp's dB and dC: [WARPS][TOK][2 N]
    static constexpr int SMEM = RED + WARPS * TOK * 2 * N * 4;
};

// Two neighbouring channels.
__device__ __forceinline__ float2 load2(const float *p) { return *reinterpret_cast<const float2 *>(p); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16 *p) {
    const uint32_t r = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}
__device__ __forceinline__ void store2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
}

// Sums of four values over L lanes, `stride` apart.  A lane has them in slots: slots 0, 1 are the values 2 b, 2 b + 1 with b
// the uppermost bit of the lane's number among the L, slots 2, 3 the other two (L = 1: in order) - so that a lane
// keeps slots 0, 1 and hands over 2, 3 without selecting.  For L >= 4 the lane ends with that value in v[0] that the two
// upper bits of its number name, for L = 2 with two in v[0], v[1], for L = 1 with all four.
template <int L, int STRIDE>
__device__ __forceinline__ void reduce4(float (&v)[4], int lane) {
    if (L >= 2) {
        constexpr int M = L / 2 * STRIDE;
        v[0] += __shfl_xor_sync(0xffffffffu, v[2], M);
        v[1] += __shfl_xor_sync(0xffffffffu, v[3], M);
    }
    if (L >= 4) {
        constexpr int M = L / 4 * STRIDE;
        const bool up = lane & M;
        const float s0 = up ? v[0] : v[1], k0 = up ? v[1] : v[0];
        v[0] = k0 + __shfl_xor_sync(0xffffffffu, s0, M);
    }
#pragma unroll
    for (int m = L / 8; m > 0; m >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], m * STRIDE);
}
// Which of the four reduce4 leaves in this lane (L >= 4), and whether the lane is the first with it.
template <int L, int STRIDE>
__device__ __forceinline__ int reduced_index(int lane) {
    return 2 * ((lane / (L / 2 * STRIDE)) & 1) + ((lane / (L / 4 * STRIDE)) & 1);
}

template <typename T, int LN>
__global__ void __launch_bounds__(NT) ssm_bwd_kernel(SsmBwdArgs p, int tiles) {
    using K = Back<T, LN>;
    constexpr int N = K::N, CG = K::CG, CT = K::CT;
    extern __shared__ __align__(16) uint8_t smem[];
    const SsmArgs &f = p.f;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nq = lane % LN, cg = lane / LN;
    const int tile = blockIdx.x % tiles, slot = blockIdx.x / tiles;
    const SsmSpan span = ssm_row_span(f, slot);
    const int each = f.D / f.G, tpg = tiles / f.G, group = tile / tpg, c0 = group * each + tile % tpg * CT;
    const int have = min(CT, (group + 1) * each - c0);
    const int ch = warp * CG * 4 + cg * 4;  // this thread's first channel of the tile
    const bool live = ch < have;            // (tiles have a multiple of 4 channels)
    const size_t dn = (size_t)f.D * N;

    float *delta_s = reinterpret_cast<float *>(smem + K::F), *u_s = delta_s + TOK * CT, *g_s = u_s + TOK * CT, *y_s = g_s + TOK * CT;
    const float4 *b_s = reinterpret_cast<const float4 *>(smem + K::BC), *c_s = b_s + TOK * N / 2;
    float4 *kept = reinterpret_cast<float4 *>(smem + K::KEPT) + tid;
    float *red = reinterpret_cast<float *>(smem + K::RED);

    // which of a token's sums reduce4 leaves in this lane: LEFT entries of dB and dC from bc_at, one channel's at ch_at
    constexpr int LEFT = CG >= 4 ? 1 : 4 / CG;
    const bool bc_writes = CG < 8 || (cg & 1) == 0, ch_writes = nq % (LN / 4) == 0;
    const int bc_at = 4 * nq + (CG >= 4 ? reduced_index<CG < 4 ? 4 : CG, LN>(lane) : CG == 2 ? 2 * cg : 0);
    const int ch_at = ch + reduced_index<LN, 1>(lane);

    // the slots' order (reduce4): pair q of channels is ch + 2 (q ^ cflip), + 1; slot i of entries is 4 nq + (i ^ 2 nflip)
    const int cflip = lane / (LN / 2) & 1, nflip = CG >= 2 ? lane / ((CG >= 2 ? CG / 2 : 1) * LN) & 1 : 0;
    float2 rate[2][4], l[2][4], dA[2][4];
    auto place = [&](int c, int i) { return (size_t)(c0 + ch + (c ^ 2 * cflip)) * N + 4 * nq + (i ^ 2 * nflip); };
    auto entry = [&](const float *base, int c, int i) { return base[place(c, i)]; };
    const float *l0 = f.seg ? f.state + slot * dn : p.dS_T ? p.dS_T + span.seq * dn : nullptr;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rate[q][i] = live ? make_float2(ssm_rate(entry(f.A_log, 2 * q, i)), ssm_rate(entry(f.A_log, 2 * q + 1, i))) : make_float2(0.f, 0.f);
            l[q][i] = live && l0 ? make_float2(entry(l0, 2 * q, i), entry(l0, 2 * q + 1, i)) : make_float2(0.f, 0.f);
            dA[q][i] = make_float2(0.f, 0.f);
        }
    // elementwise work, a warp on its own channels: channels ec, ec + 1 of the tile, tokens et, et + TSTEP, ..
    constexpr int CW = CT / WARPS, TSTEP = 64 / CW;
    const int ec = warp * CW + 2 * (lane % (CW / 2)), et = lane / (CW / 2), ed = c0 + ec;
    const bool elive = ec < have;
    float2 bias = make_float2(0.f, 0.f), skip = bias, sum_D = bias, sum_dt = bias;
    if (elive && f.dt_bias) bias = *reinterpret_cast<const float2 *>(f.dt_bias + ed);
    if (elive && f.Dskip) skip = *reinterpret_cast<const float2 *>(f.Dskip + ed);

    const size_t esz = sizeof(T), pitch = f.D * esz, bpitch = (size_t)f.G * N * esz;
    auto at_tile = [&](const void *base) { return static_cast<const uint8_t *>(base) + (size_t)c0 * esz; };
    const uint8_t *xg = at_tile(f.x), *dg = at_tile(f.dt), *zg = f.z ? at_tile(f.z) : nullptr, *yg = at_tile(p.dy);
    const uint8_t *bg = static_cast<const uint8_t *>(f.Bm) + (size_t)group * N * esz, *cgm = static_cast<const uint8_t *>(f.Cm) + (size_t)group * N * esz;
    const int pieces = have * (int)esz / 16;
    auto load = [&](int s) {
        if (s >= 0) {
            const long long t0 = span.lo + (long long)s * TOK;
            uint8_t *st = smem + (s & 1) * K::STAGE;
            load_tile<K::ROW / 16, NT>(st + K::X, xg, pitch, t0, span.hi, pieces);
            load_tile<K::ROW / 16, NT>(st + K::DT, dg, pitch, t0, span.hi, pieces);
            if (zg) load_tile<K::ROW / 16, NT>(st + K::Z, zg, pitch, t0, span.hi, pieces);
            load_tile<K::ROW / 16, NT>(st + K::DY, yg, pitch, t0, span.hi, pieces);
            load_tile<K::BROW / 16, NT>(st + K::B, bg, bpitch, t0, span.hi, K::BROW / 16);
            load_tile<K::BROW / 16, NT>(st + K::C, cgm, bpitch, t0, span.hi, K::BROW / 16);
        }
        cp_async_commit();
    };

    const int chunks = (int)((span.hi - span.lo + TOK - 1) / TOK), nk = (f.T + TOK - 1) / TOK;
    const long long row0 = (long long)span.seq * f.T;
    // dB and dC of the tile over the chunk that begins at t0, a token's 2 N values side by side
    auto sum_warps = [&](long long t0) {
        const int n = (int)min((long long)TOK, span.hi - t0) * 2 * N;
        float *part = p.part + ((size_t)tile * f.B * f.T + t0) * 2 * N;
        for (int i = tid; i < n; i += NT) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) v += red[w * TOK * 2 * N + i];
            part[i] = v;
        }
    };
    load(chunks - 1);
    for (int s = chunks - 1; s >= 0; --s) {
        const uint8_t *st = smem + (s & 1) * K::STAGE;
        const long long t0 = span.lo + (long long)s * TOK;
        const int count = (int)min((long long)TOK, span.hi - t0);
        // the chunk's start state
        float2 h[2][4];
        const float *h0 = f.keep + ((size_t)span.seq * nk + (size_t)(t0 - row0) / TOK) * dn;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) h[q][i] = live ? make_float2(entry(h0, 2 * q, i), entry(h0, 2 * q + 1, i)) : make_float2(0.f, 0.f);
        cp_async_wait<0>();
        __syncthreads();  // the chunk's inputs are here, the one before is done with
        load(s - 1);
        if (s + 1 < chunks) sum_warps(t0 + TOK);
        auto in = [&](int what, int t) { return load2(reinterpret_cast<const T *>(st + what) + t * CT + ec); };
        auto at = [&](float *base, int t) { return reinterpret_cast<float2 *>(base + t * CT + ec); };
#pragma unroll 4
        for (int t = et; t < TOK; t += TSTEP) {  // past the row's end: a token that changes nothing
            const bool real = t < count;
            float2 delta = softplus2(__fadd2_rn(in(K::DT, t), bias)), g = in(K::DY, t);
            if (f.z) {
                const float2 z = in(K::Z, t);
                g = __fmul2_rn(g, __fmul2_rn(z, make_float2(ssm_sigmoid(z.x), ssm_sigmoid(z.y))));
            }
            if (!real) delta = g = make_float2(0.f, 0.f);
            *at(delta_s, t) = delta;
            *at(u_s, t) = __fmul2_rn(delta, in(K::X, t));
            *at(g_s, t) = g;
        }
#pragma unroll
        for (int k = 0; k < TOK * N / NT; ++k) {
            const int i = k * NT + tid;
            const float b = to_f32(reinterpret_cast<const T *>(st + K::B)[i]), c = to_f32(reinterpret_cast<const T *>(st + K::C)[i]);
            reinterpret_cast<float2 *>(smem + K::BC)[i] = make_float2(b, b);
            reinterpret_cast<float2 *>(smem + K::BC)[TOK * N + i] = make_float2(c, c);
        }
        __syncthreads();
        // four values of channels ch .. ch + 3 as two pairs; four entries of B or C, each twice
        auto quad = [&](const float *base, int t, float2(&v)[2]) {
            v[0] = *reinterpret_cast<const float2 *>(base + t * CT + ch + 2 * cflip);
            v[1] = *reinterpret_cast<const float2 *>(base + t * CT + ch + 2 * (cflip ^ 1));
        };
        auto four = [&](const float4 *base, int t, float2(&v)[4]) {
            const float4 r0 = base[t * (N / 2) + 2 * nq + nflip], r1 = base[t * (N / 2) + 2 * nq + (nflip ^ 1)];
            v[0] = make_float2(r0.x, r0.y);
            v[1] = make_float2(r0.z, r0.w);
            v[2] = make_float2(r1.x, r1.y);
            v[3] = make_float2(r1.z, r1.w);
        };
        // h at the start of the quarters 1, 2, 3
#pragma unroll 1
        for (int k = 0; k < 3; ++k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * k + j;
                float2 dl[2], u[2], b[4];
                quad(delta_s, t, dl);
                quad(u_s, t, u);
                four(b_s, t, b);
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 e = ssm_exponent(dl[q], rate[q][i]);
                        h[q][i] = __ffma2_rn(make_float2(ssm_ex2(e.x), ssm_ex2(e.y)), h[q][i], __fmul2_rn(u[q], b[i]));
                    }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                kept[(k * 4 + j) * NT] = make_float4(h[j / 2][2 * (j & 1)].x, h[j / 2][2 * (j & 1)].y, h[j / 2][2 * (j & 1) + 1].x, h[j / 2][2 * (j & 1) + 1].y);
        }
#pragma unroll 2  // (1109 -> 1084 us of training 8 x 2048 x 2048; all four no longer fit the instruction cache: 1200)
        for (int k = 3; k >= 0; --k) {
            float2 a[4][2][4], hp[4][2][4];
            float2 dAq[2][4];  // dA of these four tokens: a sum of four at a time into the long one halves its rounding
            float rB[4][LEFT], rC[4][LEFT], rU[4], rD[4], rY[4];  // a token's sums, as reduce4 leaves them
            if (k > 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 r = kept[((k - 1) * 4 + j) * NT];
                    h[j / 2][2 * (j & 1)] = make_float2(r.x, r.y);
                    h[j / 2][2 * (j & 1) + 1] = make_float2(r.z, r.w);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[q][i] = live ? make_float2(entry(h0, 2 * q, i), entry(h0, 2 * q + 1, i)) : make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * k + j;
                float2 dl[2], u[2], g[2], b[4], c[4], y[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                quad(delta_s, t, dl);
                quad(u_s, t, u);
                quad(g_s, t, g);
                four(b_s, t, b);
                four(c_s, t, c);
                float dC[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float2 e = ssm_exponent(dl[q], rate[q][i]);
                        a[j][q][i] = make_float2(ssm_ex2(e.x), ssm_ex2(e.y));
                        hp[j][q][i] = h[q][i];
                        h[q][i] = __ffma2_rn(a[j][q][i], h[q][i], __fmul2_rn(u[q], b[i]));
                        y[q] = __ffma2_rn(h[q][i], c[i], y[q]);
                        acc = __ffma2_rn(g[q], h[q][i], acc);
                    }
                    dC[i] = acc.x + acc.y;
                }
                reduce4<CG, LN>(dC, lane);
#pragma unroll
                for (int i = 0; i < LEFT; ++i) rC[j][i] = dC[i];
                float ys[4] = {y[0].x, y[0].y, y[1].x, y[1].y};
                reduce4<LN, 1>(ys, lane);
                rY[j] = ys[0];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // (stored at the end: a store between would hold up the next token's loads)
                const int t = 4 * k + j;
                if (bc_writes) {
#pragma unroll
                    for (int i = 0; i < LEFT; ++i) red[(warp * TOK + t) * 2 * N + N + bc_at + i] = rC[j][i];
                }
                if (ch_writes) y_s[t * CT + ch_at] = rY[j];
            }
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                const int t = 4 * k + j;
                float2 dl[2], u[2], g[2], b[4], c[4], du[2], dd[2];
                quad(delta_s, t, dl);
                quad(u_s, t, u);
                quad(g_s, t, g);
                four(b_s, t, b);
                four(c_s, t, c);
                du[0] = du[1] = dd[0] = dd[1] = make_float2(0.f, 0.f);
                float dB[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        l[q][i] = __ffma2_rn(g[q], c[i], l[q][i]);
                        acc = __ffma2_rn(l[q][i], u[q], acc);
                        du[q] = __ffma2_rn(l[q][i], b[i], du[q]);
                        l[q][i] = __fmul2_rn(l[q][i], a[j][q][i]);
                        const float2 w = __fmul2_rn(l[q][i], hp[j][q][i]);
                        dAq[q][i] = j == 3 ? __fmul2_rn(w, dl[q]) : __ffma2_rn(w, dl[q], dAq[q][i]);
                        if (j == 0) dA[q][i] = __fadd2_rn(dA[q][i], dAq[q][i]);
                        dd[q] = __ffma2_rn(w, rate[q][i], dd[q]);
                    }
                    dB[i] = acc.x + acc.y;
                }
                reduce4<CG, LN>(dB, lane);
#pragma unroll
                for (int i = 0; i < LEFT; ++i) rB[j][i] = dB[i];
                float v0[4] = {du[0].x, du[0].y, du[1].x, du[1].y}, v1[4] = {dd[0].x, dd[0].y, dd[1].x, dd[1].y};
                reduce4<LN, 1>(v0, lane);
                reduce4<LN, 1>(v1, lane);
                rU[j] = v0[0];
                rD[j] = v1[0];
            }
            __syncwarp();  // every lane has read u and g of these tokens
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * k + j;
                if (bc_writes) {
#pragma unroll
                    for (int i = 0; i < LEFT; ++i) red[(warp * TOK + t) * 2 * N + bc_at + i] = rB[j][i];
                }
                if (ch_writes) {
                    u_s[t * CT + ch_at] = rU[j];
                    g_s[t * CT + ch_at] = rD[j];
                }
            }
        }
        __syncwarp();
        if (elive) {
            float2 chunk_D = make_float2(0.f, 0.f), chunk_dt = chunk_D;
#pragma unroll 4
            for (int t = et; t < count; t += TSTEP) {
                const float2 x = in(K::X, t), dt = __fadd2_rn(in(K::DT, t), bias), du = *at(u_s, t), dd = *at(g_s, t);
                float2 g = in(K::DY, t);
                const size_t to = (size_t)(t0 + t) * f.D + ed;
                if (f.z) {
                    const float2 z = in(K::Z, t), y = __ffma2_rn(skip, x, *at(y_s, t)), sg = make_float2(ssm_sigmoid(z.x), ssm_sigmoid(z.y));
                    const float2 slope = __fmul2_rn(sg, make_float2(fmaf(z.x, 1.f - sg.x, 1.f), fmaf(z.y, 1.f - sg.y, 1.f)));
                    store2(static_cast<T *>(p.dz) + to, __fmul2_rn(__fmul2_rn(g, y), slope));
                    g = __fmul2_rn(g, __fmul2_rn(z, sg));
                }
                // ddelta = ln2 (w . rate) + du x
                const float2 ddelta = __ffma2_rn(du, x, make_float2(LN2 * dd.x, LN2 * dd.y));
                // (a slope of 0, of dt = -infinity: 0 whatever ddelta is, which a large A takes out of range)
                const float2 rise = make_float2(ssm_sigmoid(dt.x), ssm_sigmoid(dt.y));
                const float2 ddt = make_float2(rise.x == 0.f ? 0.f : ddelta.x * rise.x, rise.y == 0.f ? 0.f : ddelta.y * rise.y);
                store2(static_cast<T *>(p.dx) + to, __ffma2_rn(du, *at(delta_s, t), __fmul2_rn(skip, g)));
                store2(static_cast<T *>(p.ddt) + to, ddt);
                chunk_D = __ffma2_rn(g, x, chunk_D);
                chunk_dt = __fadd2_rn(chunk_dt, ddt);
            }
            sum_D = __fadd2_rn(sum_D, chunk_D);
            sum_dt = __fadd2_rn(sum_dt, chunk_dt);
        }
    }
    if (live) {
        float *out = p.sums + slot * dn;
        const bool first = p.dS0 && span.first;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const size_t e = place(2 * q, i);
                out[e] = LN2 * rate[q][i].x * dA[q][i].x;
                out[e + N] = LN2 * rate[q][i].y * dA[q][i].y;
                if (first) {
                    p.dS0[span.seq * dn + e] = l[q][i].x;
                    p.dS0[span.seq * dn + e + N] = l[q][i].y;
                }
            }
    }
    __syncthreads();
    if (chunks > 0) sum_warps(span.lo);
#pragma unroll
    for (int m = CW / 2; m < 32; m <<= 1) {
        sum_D.x += __shfl_xor_sync(0xffffffffu, sum_D.x, m);
        sum_D.y += __shfl_xor_sync(0xffffffffu, sum_D.y, m);
        sum_dt.x += __shfl_xor_sync(0xffffffffu, sum_dt.x, m);
        sum_dt.y += __shfl_xor_sync(0xffffffffu, sum_dt.y, m);
    }
    if (elive && et == 0) {
        *reinterpret_cast<float2 *>(p.sums2 + (size_t)slot * 2 * f.D + ed) = sum_D;
        *reinterpret_cast<float2 *>(p.sums2 + (size_t)slot * 2 * f.D + f.D + ed) = sum_dt;
    }
}

// The gradient that each segment hands to the token before it, from l = 0 at its end, and its sum of delta.  Threads
// as in the forward: 16 entries of a channel.
template <typename T, int NSUB>
struct Carry {
    static constexpr int N = NSUB * 16, CT = NT / NSUB, ROW = CT * sizeof(T), BROW = N * sizeof(T);
    static constexpr int DT = 0, Z = TOK * ROW, DY = 2 * TOK * ROW, C = 3 * TOK * ROW, STAGE = C + TOK * BROW;
    static constexpr int SMEM = 2 * STAGE + TOK * N * 4;
};
template <typename T, int NSUB>
__global__ void __launch_bounds__(NT) ssm_bwd_carry_kernel(SsmBwdArgs p, int tiles) {
    using K = Carry<T, NSUB>;
    constexpr int N = K::N, CT = K::CT, PER = 16;
    extern __shared__ __align__(16) uint8_t smem[];
    const SsmArgs &f = p.f;
    float *cvt = reinterpret_cast<float *>(smem + 2 * K::STAGE);
    const int tid = threadIdx.x, tile = blockIdx.x % tiles, slot = blockIdx.x / tiles;
    const SsmSpan span = ssm_row_span(f, slot);
    const int each = f.D / f.G, tpg = tiles / f.G, group = tile / tpg, c0 = group * each + tile % tpg * CT;
    const int have = min(CT, (group + 1) * each - c0), c = tid / NSUB, sub = tid % NSUB, d = c0 + c;
    const bool live = c < have;
    float2 rate[PER / 2], l[PER / 2];
    const size_t at = (size_t)(live ? d : 0) * N + sub * PER;
    const float bias = live && f.dt_bias ? f.dt_bias[d] : 0.f;
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) {
        const float2 a = reinterpret_cast<const float2 *>(f.A_log + at)[i];
        rate[i] = make_float2(ssm_rate(a.x), ssm_rate(a.y));
        l[i] = make_float2(0.f, 0.f);
    }
    const size_t esz = sizeof(T), pitch = f.D * esz, bpitch = (size_t)f.G * N * esz;
    auto at_tile = [&](const void *base) { return static_cast<const uint8_t *>(base) + (size_t)c0 * esz; };
    const uint8_t *dg = at_tile(f.dt), *zg = f.z ? at_tile(f.z) : nullptr, *yg = at_tile(p.dy);
    const uint8_t *cg = static_cast<const uint8_t *>(f.Cm) + (size_t)group * N * esz;
    const int pieces = have * (int)esz / 16;
    auto load = [&](int s) {
        if (s >= 0) {
            const long long t0 = span.lo + (long long)s * TOK;
            uint8_t *st = smem + (s & 1) * K::STAGE;
            load_tile<K::ROW / 16, NT>(st + K::DT, dg, pitch, t0, span.hi, pieces);
            if (zg) load_tile<K::ROW / 16, NT>(st + K::Z, zg, pitch, t0, span.hi, pieces);
            load_tile<K::ROW / 16, NT>(st + K::DY, yg, pitch, t0, span.hi, pieces);
            load_tile<K::BROW / 16, NT>(st + K::C, cg, bpitch, t0, span.hi, K::BROW / 16);
        }
        cp_async_commit();
    };
    const int chunks = (int)((span.hi - span.lo + TOK - 1) / TOK);
    load(chunks - 1);
    for (int s = chunks - 1; s >= 0; --s) {
        const uint8_t *st = smem + (s & 1) * K::STAGE;
        const int count = (int)min((long long)TOK, span.hi - span.lo - (long long)s * TOK);
        cp_async_wait<0>();
        __syncthreads();
        load(s - 1);
#pragma unroll
        for (int k = 0; k < TOK * N / NT; ++k) {
            const int i = k * NT + tid, n = i % N;
            cvt[i - n + ((n % PER / 4) * NSUB + n / PER) * 4 + n % 4] = to_f32(reinterpret_cast<const T *>(st + K::C)[i]);
        }
        __syncthreads();
        auto in = [&](int what, int t) { return to_f32(reinterpret_cast<const T *>(st + what)[t * CT + c]); };
#pragma unroll 4
        for (int t = count - 1; t >= 0; --t) {
            const float delta = softplus(in(K::DT, t) + bias);
            float g = in(K::DY, t);
            if (f.z) {
                const float z = in(K::Z, t);
                g *= z * ssm_sigmoid(z);
            }
            total += delta;
            const float2 delta2 = make_float2(delta, delta), g2 = make_float2(g, g);
#pragma unroll
            for (int j = 0; j < PER / 4; ++j) {
                const float4 v = *reinterpret_cast<const float4 *>(cvt + t * N + (j * NSUB + sub) * 4);
                const float2 e0 = ssm_exponent(delta2, rate[2 * j]), e1 = ssm_exponent(delta2, rate[2 * j + 1]);
                l[2 * j] = __fmul2_rn(make_float2(ssm_ex2(e0.x), ssm_ex2(e0.y)), __ffma2_rn(g2, make_float2(v.x, v.y), l[2 * j]));
                l[2 * j + 1] = __fmul2_rn(make_float2(ssm_ex2(e1.x), ssm_ex2(e1.y)), __ffma2_rn(g2, make_float2(v.z, v.w), l[2 * j + 1]));
            }
        }
    }
    if (!live) return;
    float2 *to = reinterpret_cast<float2 *>(f.state + (size_t)slot * f.D * N + at);
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) to[i] = l[i];
    if (sub == 0) f.sum[(size_t)slot * f.D + d] = total;
}

// The gradient of the state at each segment's end, in place of what the segment alone hands on.
__global__ void __launch_bounds__(NT) ssm_bwd_combine_kernel(SsmBwdArgs p) {
    const SsmArgs &f = p.f;
    const int row = blockIdx.y, segs = ssm_pieces(f.T, f.seg);
    const size_t e = (size_t)blockIdx.x * NT + threadIdx.x, size = (size_t)f.D * f.N;
    if (e >= size) return;
    const float rate = ssm_rate(f.A_log[e]);
    float l = p.dS_T ? p.dS_T[row * size + e] : 0.f;
    float *state = f.state + (size_t)row * segs * size + e;
    const float *sum = f.sum + (size_t)row * segs * f.D + e / f.N;
    constexpr int BATCH = 8;  // (all loaded before the first is written back)
    for (int s0 = segs - 1; s0 >= 0; s0 -= BATCH) {
        float local[BATCH], decay[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            local[i] = decay[i] = 0.f;
            if (s0 - i >= 0) {
                local[i] = state[(s0 - i) * size];
                decay[i] = ssm_ex2(rate * sum[(size_t)(s0 - i) * f.D]);
            }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (s0 - i >= 0) {
                state[(s0 - i) * size] = l;
                l = fmaf(decay[i], l, local[i]);
            }
    }
}

// dB, dC [tokens, G, N] = the sums of their tiles' shares.
template <typename T>
__global__ void __launch_bounds__(256) ssm_bc_kernel(const float *part, T *dB, T *dC, long long tokens, int N, int G, int tpg) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;  // of [tokens][G][2 N]
    if (i >= tokens * G * 2 * N) return;
    const int n = (int)(i % (2 * N)), g = (int)(i / (2 * N) % G);
    const long long t = i / (2 * N) / G;
    const float *src = part + ((size_t)g * tpg * tokens + t) * 2 * N + n;
    float v = 0.f;
#pragma unroll 8
    for (int k = 0; k < tpg; ++k) v += src[(size_t)k * tokens * 2 * N];
    const size_t at = ((size_t)t * G + g) * N;
    if (n < N)
        dB[at + n] = from_f32<T>(v);
    else
        dC[at + n - N] = from_f32<T>(v);
}

template <typename T, int NSUB>
cudaError_t backward(const SsmBwdArgs &a) {
    using KB = Back<T, 4 * NSUB>;
    using KC = Carry<T, NSUB>;
    const SsmArgs &f = a.f;
    const int tiles = ssm_bwd_tiles(f.D, f.N, f.G), slots = f.slots;
    const long long tokens = (long long)f.B * f.T;
    cudaError_t e = allow_smem(ssm_bwd_kernel<T, 4 * NSUB>, KB::SMEM);
    if (e != cudaSuccess) return e;
    if (f.seg && slots > 0) {
        if ((e = allow_smem(ssm_bwd_carry_kernel<T, NSUB>, KC::SMEM)) != cudaSuccess) return e;
        ssm_bwd_carry_kernel<T, NSUB><<<(unsigned)slots * tiles, NT, KC::SMEM, f.stream>>>(a, tiles);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        ssm_bwd_combine_kernel<<<dim3((unsigned)(((size_t)f.D * f.N + NT - 1) / NT), f.B), NT, 0, f.stream>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (slots > 0) {
        ssm_bwd_kernel<T, 4 * NSUB><<<(unsigned)slots * tiles, NT, KB::SMEM, f.stream>>>(a, tiles);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (tokens > 0) {
        const long long n = tokens * f.G * 2 * f.N;
        ssm_bc_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, f.stream>>>(a.part, static_cast<T *>(a.dB), static_cast<T *>(a.dC),
                                                                            tokens, f.N, f.G, tiles / f.G);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return launch_sum_parts(a.sums, slots, f.D * f.N, a.dA_log, nullptr, f.D * f.N, f.stream);
}

template <typename T>
cudaError_t states(const SsmBwdArgs &a) {
    const int N = a.f.N;
    const cudaError_t e = N == 16 ? backward<T, 1>(a) : N == 32 ? backward<T, 2>(a) : N == 64 ? backward<T, 4>(a) : backward<T, 8>(a);
    if (e != cudaSuccess || (!a.dD && !a.ddt_bias)) return e;
    return launch_sum_parts(a.sums2, a.f.slots, 2 * a.f.D, a.dD, a.ddt_bias, a.f.D, a.f.stream);
}

}  // namespace

cudaError_t launch_ssm_bwd(const SsmBwdArgs &a) { return a.f.dtype == EFLA_BF16 ? states<__nv_bfloat16>(a) : states<float>(a); }

}  // namespace efla
