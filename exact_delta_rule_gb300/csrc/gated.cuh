// Gated delta rule: argument blocks of its launchers and the decay arithmetic its kernels share.
//
//   S_t = e^{g_t} (I - alpha_t k_t k_t^T) S_{t-1} + alpha_t k_t v_t^T,   o_t = S_t^T q_t
//
// In a chunk with start state S, G_t the running sum of g and Gamma_ts = e^{G_t - G_s} (s <= t),
// u_t = alpha_t (v_t - e^{g_t} S_{t-1}^T k_t) gives S_t = e^{G_t} S + sum_{s <= t} Gamma_ts k_s u_s^T:
//   (I + diag(alpha) L) U = diag(alpha) R,  R = V - diag(e^G) K S,  L = strictly-lower(Gamma o K K^T)
//   O  = diag(e^G) Q S + P U,               P = (Gamma o Q K^T) o M_incl
//   S' = e^{G_C} S + K^T diag(c) U,         c_s = e^{G_C - G_s}
// Every exponent is a sum of g over a stretch of tokens, so for g <= 0 no factor exceeds 1.
#pragma once

#include <algorithm>

#include "internal.cuh"

namespace efla {

// Value head h reads the query and key head h / (H / Hk).
struct GatedFwdArgs {
    const void *q, *k, *v;
    const float *g, *beta, *S0;
    const int32_t *cu_seqlens;
    void *o;      // may be nullptr: no outputs wanted
    float *S_T;   // may be nullptr
    int B, T, Hk, H, dk, dv, N;
    efla_dtype in_dtype, o_dtype;
    int euler;
    cudaStream_t stream;
    int *status;
    void *ws = nullptr;  // training: the workspace of the backward, filled by the forward (rows of [B, T] only)
};

struct GatedBwdArgs {
    const void *q, *k, *v;
    const float *g, *beta, *S0;
    const void *dO;  // in_dtype
    const float *dST;
    void *dq, *dk, *dv;  // in_dtype
    float *dg, *dbeta, *dS0;
    int B, T, Hk, H, dk_dim, dv_dim;
    efla_dtype in_dtype;
    int euler;
    cudaStream_t stream;
    int *status;
    void *ws;
};

struct GatedDecodeArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    float *S;
    void *o;
    int B, m, Hk, H, dk, dv;
    efla_dtype in_dtype, o_dtype;
    int euler;
    cudaStream_t stream;
};

// Workspace of the backward (bytes from its base, every region 256-byte aligned).  nc = ceil(T / 64).
//   states and dse [B H][nc]: the state at the start of every chunk and the gradient of the state at
//     its end, d_k x d_v x 4 bytes each (tensor cores: 64 KB tiles whatever the head sizes);
//   w [B H][nc]: T'' = (I + diag(alpha) L)^{-1} diag(alpha) of every chunk (the tensor-core path: the
//     inverse without diag(alpha)), 64 x 64 x 4 bytes;
//   p [B H][nc]: P likewise (CUDA-core path only);
//   sdot [B H][nc][4]: partial sums of <S, dS'> of every chunk (CUDA-core path only);
//   part [2][B T H][d_k] fp32: dq and dk of every value head (where key heads are shared);
//   tok [B H][nc]: dY hi, dO and dY lo of every chunk as operand tiles, 48 KB (tensor-core path,
//     gated_bwd_tc.cu).
struct GatedWs {
    size_t states, dse, w, p, sdot, part, tok, bytes;
};
// Which kernels take a forward or backward: bf16 inputs the tensor cores, at every size (features up to
// 128 are zeros that TMA fills in).  Even where that is most of the work they are ahead of the CUDA-core
// kernels, which take fp32 inputs only.  Forward and forward with backward in us, bf16 on the tensor cores /
// the same shape in fp32 on CUDA cores:
//   d_k = d_v = 32, 2 heads of 32 tokens  12 / 13, 36 / 45;   8 x 2048 tokens of 16 heads  160 / 452, 629 / 1572
//   d_k = d_v = 64                        12 / 17, 37 / 72;                                162 / 1111, 634 / 3429
// What it costs is memory: the tiles are those of 128 features, so the workspace of 8 x 2048 tokens of 16 heads
// is 768 MiB at d = 32, 64 and 128 alike, where the fp32 layout takes 160, 256 and 640.
inline bool gated_tc(efla_dtype in_dtype) { return in_dtype == EFLA_BF16; }
inline GatedWs gated_ws(int B, int T, int Hk, int H, int dk, int dv, efla_dtype in_dtype) {
    const size_t units = (size_t)B * H, nc = ((size_t)T + 63) / 64, tok = (size_t)B * T * H;
    const bool tc = gated_tc(in_dtype);
    const size_t mat = tc ? 65536 : (size_t)dk * dv * 4;
    GatedWs w;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t r = at;
        at += (n + 255) / 256 * 256;
        return r;
    };
    w.states = take(units * nc * mat);
    w.dse = take(units * nc * mat);
    w.w = take(units * nc * 64 * 64 * 4);
    w.p = take(tc ? 0 : units * nc * 64 * 64 * 4);
    w.sdot = take(tc ? 0 : units * nc * 4 * sizeof(float));
    w.part = take(Hk != H ? 2 * tok * dk * sizeof(float) : 0);
    w.tok = take(tc ? units * nc * 49152 : 0);
    w.bytes = T > 0 && units > 0 ? at : 0;
    return w;
}

// CUDA cores, fp32 inputs (gated_simt.cu); the backward of T = 0 whatever the type.
cudaError_t launch_gated_chunk_simt(const GatedFwdArgs &a);
cudaError_t launch_gated_bwd_simt(const GatedBwdArgs &a);
// Tensor cores: bf16 inputs (chunk_tc.cu).
cudaError_t launch_gated_chunk_tc(const GatedFwdArgs &a, const char **why);
cudaError_t launch_gated_bwd_tc(const GatedBwdArgs &a, const char **why);  // T > 0 (gated_bwd_tc.cu)
cudaError_t launch_gated_decode_tokens_tc(const GatedDecodeArgs &a, const char **why);  // (decode_tc.cu)
// dq, dk [B T Hk][d] = the sums over each key head's value heads of part [2][B T H][d] (fp32), in
// the input type, one fixed order of addition.
cudaError_t launch_gated_reduce_heads(const GatedBwdArgs &a, const float *part);
// One token per sequence; m tokens per sequence (gated_decode.cu).
cudaError_t launch_gated_decode_step(const GatedDecodeArgs &a);
cudaError_t launch_gated_decode_tokens(const GatedDecodeArgs &a);

// 2^x (one MUFU instruction, relative error about 2^-22; underflows to 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// An unevaluated sum hi + lo of two floats, and the sum of two of them to about 2^-46 (the error of
// the floats' own sum, recovered exactly).
struct Sum2 {
    float h, l;
};
__device__ __forceinline__ Sum2 add2(Sum2 a, Sum2 b) {
    const float s = a.h + b.h, t = s - a.h, e = ((a.h - (s - t)) + (b.h - t)) + (a.l + b.l);
    const float h = s + e;
    return {h, e - (h - s)};
}
__device__ __forceinline__ float diff2(Sum2 a, Sum2 b) { return (a.h - b.h) + (a.l - b.l); }
// A gate in units of log2.  A gate of -inf (or below -700) is taken as -700: e^-700 is 0 in fp32, and
// sums stay finite.
__device__ __forceinline__ Sum2 gate2(float g) {
    constexpr float L_HI = 1.44269504f, L_LO = 1.92596299e-8f;  // log2(e) = L_HI + L_LO
    g = g < -700.f ? -700.f : g;
    const float h = g * L_HI;
    return {h, fmaf(g, L_HI, -h) + g * L_LO};
}
__device__ __forceinline__ Sum2 shfl_up2(Sum2 x, int off) {
    return {__shfl_up_sync(0xffffffffu, x.h, off), __shfl_up_sync(0xffffffffu, x.l, off)};
}
__device__ __forceinline__ Sum2 shfl2(Sum2 x, int lane) {
    return {__shfl_sync(0xffffffffu, x.h, lane), __shfl_sync(0xffffffffu, x.l, lane)};
}

// A sum of gates (log2) as its nearest whole number and the rest, to 2^-25: what is left of a difference
// of two such pairs keeps that accuracy however far the sums are from 0.
constexpr float WHOLE = 12582912.f;  // 1.5 2^23: a sum with it is rounded to a whole number, held in its low bits
__device__ __forceinline__ float2 whole_rest(Sum2 G) {
    const float n = (G.h + WHOLE) - WHOLE;
    return make_float2(n, (G.h - n) + G.l);
}
// 2^(a - b) of two such pairs to the accuracy of ex2 (as one float an exponent of 64 or more is 2^-18 off):
// the whole part goes into the exponent by itself.  0 below 2^-127, infinity from 2^128.
__device__ __forceinline__ float from_quarter(float na, float ra, float nb, float rb) {
    const uint32_t n = __float_as_uint(fminf(fmaxf(na - nb, -127.f), 128.f) + WHOLE);
    return ex2(ra - rb) * __uint_as_float((n + 127u) << 23);
}

// The decays of a chunk's 64 tokens from its gates (0 past the chunk's end), by one warp: lane l holds
// tokens 2 l and 2 l + 1.  Writes, token t at [t stride], G_t (log2) as whole_rest to gw and gr, and to dn
// e^{G_m - G_t} with m = DECAY_MID the ninth token of t's quarter of 16; to eg[t] e^{G_t} and to ec[t]
// e^{G_C - G_t}.  Returns (in every lane) whether every dn lies between 2^-100 and 2^60: then Gamma_ts =
// e^{G_t - G_m} dn_s for s in quarter m and t >= s costs a product an entry (from_quarter gives the first
// factor); otherwise, and without dn (nullptr), pair_decay takes the difference of the sums, an exponential an
// entry.
// Within these bounds neither factor overflows for t >= s, and the first one's underflow (2^-126) leaves
// out only Gamma below 2^-66.  Measured from its middle a quarter may decay by up to 2^120.
// The running sum is kept to about 2^-46: a plain 32-bit sum of 64 gates of size 2 is off by 2^-17 in
// the exponent, more than every other rounding of the chunk.  For the same reason the exponents of the two
// factors, which may both be far from 1 where their product is not, are taken in two parts.
constexpr int DECAY_MID = 8;
__device__ __forceinline__ bool chunk_decay(float g0, float g1, int lane, float *gw, float *gr, float *dn, int stride,
                                            float *eg, float *ec) {
    const Sum2 a = gate2(g0), b = gate2(g1);
    Sum2 G1 = add2(a, b);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const Sum2 x = shfl_up2(G1, off), y = add2(G1, x);
        if (lane >= off) G1 = y;
    }
    Sum2 G0 = shfl_up2(G1, 1);  // G_{2 l - 1}
    if (lane == 0) G0 = {0.f, 0.f};
    G0 = add2(G0, a);
    const float2 w0 = whole_rest(G0), w1 = whole_rest(G1);
    const Sum2 last = shfl2(G1, 31);
    const int t = 2 * lane;
    gw[t * stride] = w0.x;
    gw[(t + 1) * stride] = w1.x;
    gr[t * stride] = w0.y;
    gr[(t + 1) * stride] = w1.y;
    eg[t] = ex2(G0.h + G0.l);
    eg[t + 1] = ex2(G1.h + G1.l);
    ec[t] = ex2(diff2(last, G0));
    ec[t + 1] = ex2(diff2(last, G1));
    if (!dn) return false;
    const int mid = (lane & 24) + DECAY_MID / 2;
    const float mn = __shfl_sync(0xffffffffu, w0.x, mid), mr = __shfl_sync(0xffffffffu, w0.y, mid);
    const float d0 = from_quarter(mn, mr, w0.x, w0.y), d1 = from_quarter(mn, mr, w1.x, w1.y);
    dn[t * stride] = d0;
    dn[(t + 1) * stride] = d1;
    return __all_sync(0xffffffffu, fminf(d0, d1) > 0x1p-100f && fmaxf(d0, d1) < 0x1p60f);
}

// The same for a block of 16 tokens, one per lane (lanes 16-31 take part with g = 0 and write nothing).
__device__ __forceinline__ void block_decay16(float g, int lane, float *gh, float *gl, float *eg, float *ec) {
    Sum2 G = gate2(g);
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) {
        const Sum2 x = shfl_up2(G, off), y = add2(G, x);
        if (lane >= off) G = y;
    }
    const Sum2 last = shfl2(G, 15);
    if (lane < 16) {
        gh[lane] = G.h;
        gl[lane] = G.l;
        eg[lane] = ex2(G.h + G.l);
        ec[lane] = ex2(diff2(last, G));
    }
}
// A beta of magnitude below 2^-90 writes nothing (the chunk kernels of bf16 inputs): u_t is 0, and so is dv_t.
// Where alpha_t divides - dalpha_t is (dY U^T)_tt / alpha_t with U = T diag(alpha) R, whose row t is
// proportional to alpha_t - it is 2^-90, in T too: exact for dalpha, and 2^-90 of a token's size off in dq and dk.
constexpr float BETA_MIN = 0x1p-90f;
__device__ __forceinline__ bool writes_nothing(float b) { return fabsf(b) < BETA_MIN; }
__device__ __forceinline__ float live_beta(float b) { return writes_nothing(b) ? BETA_MIN : b; }
// alpha where it divides: the exact gate's is beta itself where beta lambda is so small
// that the difference is lost (2^-25), as (1 - e^{-beta lambda}) / lambda is 0 once beta lambda is below the
// smallest float.
__device__ __forceinline__ float live_alpha(float b, float lam, int euler) {
    return euler || fabsf(b * lam) < 0x1p-25f ? b : efla_alpha(b, lam, 0);
}
// Gamma_ts from the two sums, each given in two parts (whole_rest, or the two floats of a Sum2).
__device__ __forceinline__ float pair_decay(float ht, float lt, float hs, float ls) { return ex2((ht - hs) + (lt - ls)); }

}  // namespace efla
