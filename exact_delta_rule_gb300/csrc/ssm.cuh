// Selective state space scan: argument blocks of its launchers and the arithmetic its kernels share.
//
//   delta_t = softplus(dt_t + dt_bias),   A = -e^{A_log}
//   h_t = e^{A delta_t} h_{t-1} + delta_t x_t B_t,   y_t = (C_t . h_t + D x_t) silu(z_t)
//
// per channel d of D with a state h of N entries; B_t and C_t [G, N] are shared by the D / G channels of a group.
//
// Long rows are cut into segments where the channels alone do not fill the GPU: first each segment's end state
// from h = 0 and its sum of delta (the carry kernel), then, segment after segment,
// h_end = e^{A sum delta} h_start + local (the combine kernel), then all segments at once from their start states.
// That costs the exponentials a second time, without the outputs: 0.55 of the scan.
#pragma once

#include <algorithm>

#include "internal.cuh"

namespace efla {

constexpr int SSM_TOK = 16;   // tokens a stage; the training forward keeps the state at the start of each

struct SsmArgs {
    const void *x, *dt, *z;              // [B, T, D]; z may be nullptr
    const float *A_log, *Dskip, *dt_bias;  // [D, N], [D], [D]; the last two may be nullptr
    const void *Bm, *Cm;                 // [B, T, G, N]
    const float *S0;                     // [nseq, D, N] or nullptr
    const int32_t *cu_seqlens;
    void *y;
    float *S_T;                          // may be nullptr
    int B, T, D, N, G, nseq;
    efla_dtype dtype;
    cudaStream_t stream;
    int *status;
    int seg = 0;             // tokens a segment, a multiple of SSM_TOK; 0: rows are not cut
    int slots = 0;           // segments: of all rows, or the most that cu_seqlens can make
    float *state = nullptr;  // [slots, D, N]: a segment's local end state, then its start state
    float *sum = nullptr;    // [slots, D]: its sum of delta
    float *keep = nullptr;   // training: [B, ceil(T / SSM_TOK), D, N], the state at the start of each stage
};

struct SsmBwdArgs {
    SsmArgs f;               // inputs, f.keep filled by the forward; f.state and f.sum: scratch of the segments
    const void *dy;
    const float *dS_T;       // may be nullptr
    void *dx, *ddt, *dz, *dB, *dC;        // dz nullptr where z is
    float *dA_log, *dD, *ddt_bias, *dS0;  // dD, ddt_bias, dS0 may be nullptr
    float *part;             // [channel tiles, B T, 2 N]: a tile's share of dB and dC
    float *sums;             // [slots][D N]: a segment's share of dA_log
    float *sums2;            // [slots][2 D]: of dD and ddt_bias
};

// Threads a CTA and its channels, 16 entries of the state a thread.  Tiles do not cross a group, and a tile's row of a
// token is 16 bytes or more.
constexpr int ssm_fwd_threads(int N) { return N == 128 ? 64 : 32; }
constexpr int ssm_fwd_channels(int N) { return ssm_fwd_threads(N) * 16 / N; }
constexpr int SSM_BWD_NT = 128;
constexpr int ssm_bwd_channels(int N) { return SSM_BWD_NT * 16 / N; }
inline int ssm_tiles(int D, int G, int channels) { return G * ((D / G + channels - 1) / channels); }
inline int ssm_fwd_tiles(int D, int N, int G) { return ssm_tiles(D, G, ssm_fwd_channels(N)); }
inline int ssm_bwd_tiles(int D, int N, int G) { return ssm_tiles(D, G, ssm_bwd_channels(N)); }
// Tokens a segment (0: rows stay whole) for `rows` rows of T tokens, D channels and N entries: of the forward (uneven:
// T is the mean of sequences of unknown lengths), and of the backward.
int ssm_segment(long long rows, int T, int D, int N, bool uneven);
int ssm_bwd_segment(long long rows, int T, int D, int N, int tiles);

// Segments of `seg` tokens in a row of T, 1 where seg is 0.  (T + seg - 1 would pass 2^31 for the longest rows.)
__host__ __device__ inline int ssm_pieces(int T, int seg) { return seg ? T / seg + (T % seg != 0) : 1; }

// Workspace of the training pair, in bytes from its base (16-byte aligned regions).
struct SsmWs {
    int seg, slots, bwd_seg, bwd_slots;
    size_t keep, part, sums, sums2, state, sum, bytes;
};
inline SsmWs ssm_ws(int B, int T, int D, int N, int G) {
    SsmWs w{};
    const int tiles = ssm_bwd_tiles(D, N, G);
    w.seg = ssm_segment(B, T, D, N, false);
    w.slots = B * ssm_pieces(T, w.seg);
    w.bwd_seg = ssm_bwd_segment(B, T, D, N, tiles);
    w.bwd_slots = B * ssm_pieces(T, w.bwd_seg);
    size_t at = 0;
    auto take = [&](size_t floats) {
        const size_t r = at;
        at += (floats * 4 + 255) / 256 * 256;
        return r;
    };
    const size_t tok = (size_t)B * T, dn = (size_t)D * N;
    const size_t cut = std::max(w.seg ? w.slots : 0, w.bwd_seg ? w.bwd_slots : 0);  // (the forward is done with its own)
    w.keep = take((size_t)B * ((T + SSM_TOK - 1) / SSM_TOK) * dn);
    w.part = take(tok * tiles * 2 * N);
    w.sums = take(w.bwd_slots * dn);
    w.sums2 = take((size_t)w.bwd_slots * 2 * D);
    w.state = take(cut * dn);
    w.sum = take(cut * D);
    w.bytes = at;
    return w;
}

cudaError_t launch_ssm_scan(const SsmArgs &a);
cudaError_t launch_ssm_bwd(const SsmBwdArgs &a);
cudaError_t launch_ssm_step(const SsmArgs &a);  // x, dt, z, y [B, D], Bm, Cm [B, G, N], S0 == S_T in place

// 2^x (one MUFU instruction, relative error 1.5e-7 at most, 6e-8 rms, for x <= 0; underflows to 0).
__device__ __forceinline__ float ssm_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The same, kept where it is written among other such.
__device__ __forceinline__ float ssm_ex2_here(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float LOG2E = 1.44269504f;

// log(1 + e^t) = max(t, 0) + log1p(u), u = e^{-|t|} in [0, 1]; log1p(u) = u P(u) with P of degree 9 fitted to
// log1p(u) / u on [0, 1] for the smallest largest relative error (5e-9; 1.5e-7 with fp32 coefficients and
// arithmetic).
__device__ __forceinline__ float softplus(float t) {
    const float u = ssm_ex2(-fabsf(t) * LOG2E);
    float p = -0.0032439809292554855f;
    p = fmaf(p, u, 0.019851263612508774f);
    p = fmaf(p, u, -0.056959159672260284f);
    p = fmaf(p, u, 0.10603617131710052f);
    p = fmaf(p, u, -0.15305569767951965f);
    p = fmaf(p, u, 0.19675931334495544f);
    p = fmaf(p, u, -0.24954132735729218f);
    p = fmaf(p, u, 0.3332996368408203f);
    p = fmaf(p, u, -0.4999990165233612f);
    p = fmaf(p, u, 1.f);
    return fmaf(p, u, fmaxf(t, 0.f));
}
__device__ __forceinline__ float ssm_sigmoid(float x) {
    float y;  // (1 / infinity is 0)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + ssm_ex2(-x * LOG2E)));
    return y;
}
// The same for two, packed.
__device__ __forceinline__ float2 softplus2(float2 t) {
    auto two = [](float c) { return make_float2(c, c); };
    const float2 a = __fmul2_rn(make_float2(-fabsf(t.x), -fabsf(t.y)), two(LOG2E)), u = make_float2(ssm_ex2(a.x), ssm_ex2(a.y));
    float2 p = __ffma2_rn(two(-0.0032439809292554855f), u, two(0.019851263612508774f));
    p = __ffma2_rn(p, u, two(-0.056959159672260284f));
    p = __ffma2_rn(p, u, two(0.10603617131710052f));
    p = __ffma2_rn(p, u, two(-0.15305569767951965f));
    p = __ffma2_rn(p, u, two(0.19675931334495544f));
    p = __ffma2_rn(p, u, two(-0.24954132735729218f));
    p = __ffma2_rn(p, u, two(0.3332996368408203f));
    p = __ffma2_rn(p, u, two(-0.4999990165233612f));
    p = __ffma2_rn(p, u, two(1.f));
    return __ffma2_rn(p, u, make_float2(fmaxf(t.x, 0.f), fmaxf(t.y, 0.f)));
}
// A token's exponent in units of log2, rate delta.  The exponential instruction's results are 0.6e-8 to 2.7e-8 too small
// in the mean for exponents of 2^-13 to -1, which a state that many of them carry would add up; 2.1e-8 more in the
// exponent leaves -1.3e-8 to 0.9e-8 (1e-6 in place of 2e-6 of a state that 100 tokens carry), and 0 remains 0 or 2^0 = 1.
constexpr float EX2_MEAN = 2.1e-8f;
__device__ __forceinline__ float ssm_exponent(float delta, float rate) { return fmaf(delta, rate, EX2_MEAN); }
__device__ __forceinline__ float2 ssm_exponent(float2 delta, float2 rate) {
    return __ffma2_rn(delta, rate, make_float2(EX2_MEAN, EX2_MEAN));
}
// A in units of log2: e^{A delta} = 2^{rate delta}.  Held at the lowest finite number, which a_log = 88.4 reaches: a token
// of delta = 0 has to keep the state, and 0 times an infinite rate would be NaN.
__device__ __forceinline__ float ssm_rate(float a_log) {
    constexpr float LOWEST = -3.402823466e38f;
    const float rate = -expf(a_log) * LOG2E;
    return rate < LOWEST ? LOWEST : rate;  // (a NaN stays one)
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Tokens [t0, t0 + SSM_TOK) of src, the first `have` of CHUNKS 16-byte pieces each, to dst; zeros for the others and
// from token hi on.  By NT threads.  (Whole tiles, nearly all, without a test and a 64-bit product a piece.)
template <int CHUNKS, int NT>
__device__ __forceinline__ void load_tile(uint8_t *dst, const uint8_t *src, size_t pitch, long long t0, long long hi, int have) {
    constexpr int PASSES = (SSM_TOK * CHUNKS + NT - 1) / NT;
    static_assert(NT % CHUNKS == 0, "a pass takes whole tokens");
    const int t = threadIdx.x / CHUNKS, c = threadIdx.x % CHUNKS;
    src += (size_t)t0 * pitch;
    if (SSM_TOK * CHUNKS % NT == 0 && t0 + SSM_TOK <= hi && have == CHUNKS) {
        const uint32_t off = t * (uint32_t)pitch + 16 * c;
#pragma unroll
        for (int k = 0; k < PASSES; ++k) cp_async16(dst + 16 * (k * NT + threadIdx.x), src + k * (NT / CHUNKS) * pitch + off, true);
        return;
    }
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
        const int tk = t + k * (NT / CHUNKS);
        if (tk >= SSM_TOK) break;
        const bool live = t0 + tk < hi && c < have;
        cp_async16(dst + 16 * (k * NT + threadIdx.x), live ? src + (size_t)tk * pitch + 16 * c : src, live);
    }
}

// Which tokens [lo, hi) of [B T] a segment covers, and whether it is its row's or sequence's first.
struct SsmSpan {
    int seq;
    long long lo, hi;
    bool first;
};

// Segment `slot` of rows of T tokens, `seg` tokens each.
__device__ __forceinline__ SsmSpan ssm_row_span(const SsmArgs &p, int slot) {
    const int per = ssm_pieces(p.T, p.seg), row = slot / per, s = slot % per;
    const long long row0 = (long long)row * p.T, lo = row0 + (long long)s * p.seg;
    const long long hi = s + 1 < per ? lo + p.seg : row0 + p.T;
    return {row, lo, hi, s == 0};
}

// Segments of sequence n of cu_seqlens: max(1, ceil(length / seg)), -1 if it is malformed.
__device__ __forceinline__ int ssm_segments(const SsmArgs &p, int n, long long &lo, long long &hi) {
    lo = p.cu_seqlens[n], hi = p.cu_seqlens[n + 1];
    if (lo < 0 || hi < lo || hi > p.T) return -1;
    return p.seg && hi > lo ? (int)((hi - lo + p.seg - 1) / p.seg) : 1;
}

// Segment `slot` of packed sequences, all segments of a sequence after those of the ones before it.  By all threads
// of a CTA; false if there is none.  A malformed sequence has none and is reported by the CTA that `reports`; one whose segments
// are not all among p.slots (behind sequences that overlap) is left out, here and where segments are joined.
template <int NT>
__device__ __forceinline__ bool ssm_packed_span(const SsmArgs &p, int slot, bool reports, SsmSpan &out) {
    __shared__ long long box[4];
    __shared__ int sums[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long lo, hi;
    if (!p.seg) {
        if (ssm_segments(p, slot, lo, hi) < 0) {
            if (tid == 0 && reports) atomicExch(p.status, (int)EFLA_ERR_INVALID_ARG);
            return false;
        }
        out = {slot, lo, hi, true};
        return true;
    }
    reports = reports && slot == 0;
    if (tid == 0) box[0] = -1;
    __syncthreads();
    long long before = 0;
    for (int base = 0; base < p.nseq && (before <= slot || reports); base += NT) {
        const int n = base + tid;
        int segs = n < p.nseq ? ssm_segments(p, n, lo, hi) : 0;
        if (segs < 0) {
            segs = 0;
            if (reports) atomicExch(p.status, (int)EFLA_ERR_INVALID_ARG);
        }
        int run = segs;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, run, off);
            if (lane >= off) run += y;
        }
        if (lane == 31) sums[warp] = run;
        __syncthreads();
        long long start = before + run - segs;
        for (int w = 0; w < warp; ++w) start += sums[w];
        if (slot >= start && slot < start + segs && start + segs <= p.slots) {
            const int s = (int)(slot - start);
            box[0] = n;
            box[1] = lo + (long long)s * p.seg;
            box[2] = s + 1 < segs ? box[1] + p.seg : hi;
            box[3] = s == 0;
        }
        for (int w = 0; w < NT / 32; ++w) before += sums[w];
        __syncthreads();
    }
    if (box[0] < 0) return false;
    out = {(int)box[0], box[1], box[2], box[3] != 0};
    return true;
}

}  // namespace efla
