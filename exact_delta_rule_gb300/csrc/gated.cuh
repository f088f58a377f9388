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
    int *status;
};

// Workspace of the backward (bytes from its base, every region 256-byte aligned).  nc = ceil(T / 64).
//   states and dse [B H][nc]: the state at the start of every chunk and the gradient of the state at
//     its end, d_k x d_v x 4 bytes each;
//   w [B H][nc]: T'' = (I + diag(alpha) L)^{-1} diag(alpha) of every chunk (the tensor-core path: the
//     inverse without diag(alpha)), 64 x 64 x 4 bytes;
//   p [B H][nc]: P likewise (CUDA-core path only);
//   sdot [B H][nc][4]: partial sums of <S, dS'> of every chunk;
//   part [2][B T H][d_k] fp32: dq and dk of every value head (where key heads are shared);
//   tok: per-token scratch of the tensor-core path: dY [B T H][128] as bf16 hi, then lo (gated_bwd_tc.cu).
struct GatedWs {
    size_t states, dse, w, p, sdot, part, tok, bytes;
};
inline bool gated_tc(efla_dtype in_dtype, int dk, int dv) { return in_dtype == EFLA_BF16 && dk == 128 && dv == 128; }
inline GatedWs gated_ws(int B, int T, int Hk, int H, int dk, int dv, efla_dtype in_dtype) {
    const size_t units = (size_t)B * H, nc = ((size_t)T + 63) / 64, mat = (size_t)dk * dv * 4;
    const size_t tok = (size_t)B * T * H;
    const bool tc = gated_tc(in_dtype, dk, dv);
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
    w.sdot = take(units * nc * 4 * sizeof(float));
    w.part = take(Hk != H ? 2 * tok * dk * sizeof(float) : 0);
    w.tok = take(tc ? tok * 128 * (2 + 2) : 0);
    w.bytes = T > 0 && units > 0 ? at : 0;
    return w;
}

// CUDA cores, every supported shape (gated_simt.cu).
cudaError_t launch_gated_chunk_simt(const GatedFwdArgs &a);
cudaError_t launch_gated_bwd_simt(const GatedBwdArgs &a);
// Tensor cores: bf16, d_k = d_v = 128, gated_tc() (chunk_tc.cu).
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

// G_t of a chunk's 64 tokens in units of log2, as the unevaluated sum hi + lo of two floats, and
// the two factors every token needs, by one warp (64 values of g, 0 past the chunk's end; lane l
// holds tokens 2 l and 2 l + 1; token t's two floats go to gh[t stride] and gl[t stride]).  The running sum is taken in 64 bits: a difference G_t - G_s of
// two far sums is then exact to about 2^-46 of the sums, where a 32-bit sum of 64 gates of size 2
// would already be off by 2^-17 in the exponent, more than every other rounding of the chunk.
// A gate of -inf (or below -700) is taken as -700: e^-700 is 0 in fp32, and sums stay finite.
__device__ __forceinline__ void chunk_decay(float g0, float g1, int lane, float *gh, float *gl, int stride,
                                            float *eg, float *ec) {
    constexpr double LOG2E = 1.4426950408889634;
    const double a = (double)(g0 < -700.f ? -700.f : g0) * LOG2E, b = (double)(g1 < -700.f ? -700.f : g1) * LOG2E;
    double s = a + b;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += x;
    }
    const double last = __shfl_sync(0xffffffffu, s, 31), G1 = s, G0 = s - b;
    const float h0 = (float)G0, h1 = (float)G1;
    gh[2 * lane * stride] = h0;
    gh[(2 * lane + 1) * stride] = h1;
    gl[2 * lane * stride] = (float)(G0 - (double)h0);
    gl[(2 * lane + 1) * stride] = (float)(G1 - (double)h1);
    eg[2 * lane] = ex2(h0);  // (rounding the exponent x costs 2^-25 |x| of a factor 2^x)
    eg[2 * lane + 1] = ex2(h1);
    ec[2 * lane] = ex2((float)(last - G0));
    ec[2 * lane + 1] = ex2((float)(last - G1));
}
// The same for a block of 16 tokens, one per lane (lanes 16-31 take part with g = 0 and write nothing).
__device__ __forceinline__ void block_decay16(float g, int lane, float *gh, float *gl, float *eg, float *ec) {
    const double a = (double)(g < -700.f ? -700.f : g) * 1.4426950408889634;
    double s = a;
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += x;
    }
    const double last = __shfl_sync(0xffffffffu, s, 15);
    const float h = (float)s;
    if (lane < 16) {
        gh[lane] = h;
        gl[lane] = (float)(s - (double)h);
        eg[lane] = ex2(h);
        ec[lane] = ex2((float)(last - s));
    }
}
// Gamma_ts from the two sums.
__device__ __forceinline__ float pair_decay(float ht, float lt, float hs, float ls) { return ex2((ht - hs) + (lt - ls)); }

}  // namespace efla
