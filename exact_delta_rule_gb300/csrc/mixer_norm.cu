// The norms around a gated token mixer, forward and backward, as streaming kernels.
//
// Before it (rows q, k of d_k per token and key head; gates per token and value head):
//   q^ = scale q r_q, k^ = k r_k,  r = rsqrt(||x||^2 + eps)
//   g = -e^{A_log} softplus(a + dt_bias),  beta = sigmoid(b)
//   dx = r (dy' - x^ (x^ . dy')) with x^ = r x, dy' = dy (times scale for q)
//   da = -dg e^{A_log} sigmoid(a + dt_bias),  db = dbeta sigmoid(b) sigmoid(-b)
//   dA_log = sum dg g,  ddt_bias = sum da              (over the tokens of a head)
// After it (rows of d): with n = o r, r = rsqrt(mean(o^2) + eps), s = sigmoid(z)
//   y = n w z s;  dn = dy w z s,  do = r (dn - n mean(dn n)),  dz = dy n w s (1 + z (1 - s)),
//   dw = sum dy n z s                                  (over the rows)
//
// Bound by HBM: every input is read and every output written once.  A row is held by
// d * sizeof(T) / 16 lanes, one 16-byte vector each, so a warp's access is 512 contiguous bytes and
// the row sums are 2 to 5 shuffles; each thread has UNROLL rows in flight.  Arithmetic is fp32 whatever
// the type, each output rounded once.  The sums over tokens (dA_log, ddt_bias, dw) go in two stages of
// fixed order - per thread and CTA into a workspace, then one CTA over those - so that a result does
// not depend on the order in which CTAs finish.
#include <algorithm>

#include "mixer_norm.cuh"
#include "vec.cuh"

namespace efla {
namespace {

constexpr int NT = 256;

// The output gate's, to 2 + 1.2 |x| ulp (__expf): 1e-6 of the value at |x| = 5.  The prep's gates, which the recurrence
// multiplies up, take expf and a rounded division.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

template <typename T, int D>
struct Rows {
    static constexpr int N = Vec<T>::N, LPR = D / N, RPB = NT / LPR;  // lanes a row, rows a CTA and pass
};

// ------------------------------------------------------------------------------------ before: forward
// CTAs [0, row_ctas) take the 2 n rows of q, then k; the others the n H gates.
template <typename T, int D, int UNROLL>
__global__ void __launch_bounds__(NT) prep_fwd_kernel(MixerPrepArgs p, unsigned row_ctas) {
    using R = Rows<T, D>;
    if (blockIdx.x < row_ctas) {
        const long long rows = p.tokens * p.Hk;
        const long long base = (long long)blockIdx.x * R::RPB * UNROLL + threadIdx.x / R::LPR;
        const int lane = threadIdx.x % R::LPR;
        uint4 raw[UNROLL];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const long long r = base + i * R::RPB;
            const uint4 *src = reinterpret_cast<const uint4 *>(r < rows ? p.q : p.k);
            raw[i] = r < 2 * rows ? src[(r < rows ? r : r - rows) * R::LPR + lane] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const long long r = base + i * R::RPB;
            float x[R::N], s = 0.f;
            Vec<T>::unpack(raw[i], x);
#pragma unroll
            for (int e = 0; e < R::N; ++e) s = fmaf(x[e], x[e], s);
            s = row_sum<R::LPR>(s);
            const float f = rsqrtf(s + p.eps) * (r < rows ? p.scale : 1.f);
#pragma unroll
            for (int e = 0; e < R::N; ++e) x[e] *= f;
            if (r < 2 * rows)
                reinterpret_cast<uint4 *>(r < rows ? p.q_out : p.k_out)[(r < rows ? r : r - rows) * R::LPR + lane] = Vec<T>::pack(x);
        }
    } else {
        const long long e = (long long)(blockIdx.x - row_ctas) * NT + threadIdx.x;
        if (e >= p.tokens * p.H) return;
        const int h = (int)(e % p.H);
        const float t = to_f32(static_cast<const T *>(p.a)[e]) + p.dt_bias[h];
        const float b = to_f32(static_cast<const T *>(p.b)[e]);
        p.g_out[e] = -expf(p.A_log[h]) * (fmaxf(t, 0.f) + log1pf(expf(-fabsf(t))));
        p.beta_out[e] = 1.f / (1.f + expf(-b));
    }
}

// ------------------------------------------------------------------------------------ before: backward
template <typename T, int D, int UNROLL>
__global__ void __launch_bounds__(NT) prep_bwd_kernel(MixerPrepArgs p, unsigned row_ctas, int parts) {
    using R = Rows<T, D>;
    if (blockIdx.x < row_ctas) {
        const long long rows = p.tokens * p.Hk;
        const long long base = (long long)blockIdx.x * R::RPB * UNROLL + threadIdx.x / R::LPR;
        const int lane = threadIdx.x % R::LPR;
        uint4 raw[UNROLL], grad[UNROLL];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const long long r = base + i * R::RPB, at = (r < rows ? r : r - rows) * R::LPR + lane;
            raw[i] = grad[i] = make_uint4(0, 0, 0, 0);
            if (r < 2 * rows) {
                raw[i] = reinterpret_cast<const uint4 *>(r < rows ? p.q : p.k)[at];
                grad[i] = reinterpret_cast<const uint4 *>(r < rows ? p.dq_in : p.dk_in)[at];
            }
        }
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const long long r = base + i * R::RPB, at = (r < rows ? r : r - rows) * R::LPR + lane;
            float x[R::N], d[R::N], s = 0.f, xd = 0.f;
            Vec<T>::unpack(raw[i], x);
            Vec<T>::unpack(grad[i], d);
#pragma unroll
            for (int e = 0; e < R::N; ++e) {
                s = fmaf(x[e], x[e], s);
                xd = fmaf(x[e], d[e], xd);
            }
            s = row_sum<R::LPR>(s);
            xd = row_sum<R::LPR>(xd);
            const float f = rsqrtf(s + p.eps), c = f * (r < rows ? p.scale : 1.f), m = f * f * xd;
#pragma unroll
            for (int e = 0; e < R::N; ++e) x[e] = c * fmaf(-m, x[e], d[e]);
            if (r < 2 * rows) reinterpret_cast<uint4 *>(r < rows ? p.dq_out : p.dk_out)[at] = Vec<T>::pack(x);
        }
        return;
    }
    // gates: part `part` of the tokens, heads h0 .. h0 + 31; lane = (token sub-row, head) with HP heads a row
    __shared__ float red[2][NT];
    const int gx = blockIdx.x - row_ctas, part = gx % parts, h0 = gx / parts * 32;
    const int heads = min(32, p.H - h0);
    int HP = 1;
    while (HP < heads) HP *= 2;
    const int hl = threadIdx.x & (HP - 1), sub = threadIdx.x / HP, nsub = NT / HP, h = h0 + hl;
    float sA = 0.f, sD = 0.f;
    if (hl < heads) {
        const float rate = expf(p.A_log[h]), bias = p.dt_bias[h];
        for (long long tok = (long long)part * nsub + sub; tok < p.tokens; tok += (long long)parts * nsub) {
            const long long e = tok * p.H + h;
            const float t = to_f32(static_cast<const T *>(p.a)[e]) + bias, b = to_f32(static_cast<const T *>(p.b)[e]);
            const float dg = p.dg_in[e], dbeta = p.dbeta_in[e];
            const float g = -rate * (fmaxf(t, 0.f) + log1pf(expf(-fabsf(t))));
            const float eb = expf(-fabsf(b)), c = 1.f / (1.f + eb);  // (1 - sigmoid(b) would cancel for large b)
            const float da = -dg * rate / (1.f + expf(-t));
            static_cast<T *>(p.da_out)[e] = from_f32<T>(da);
            static_cast<T *>(p.db_out)[e] = from_f32<T>(dbeta * (eb * c) * c);
            sA = fmaf(dg, g, sA);
            sD += da;
        }
    }
    red[0][threadIdx.x] = sA;
    red[1][threadIdx.x] = sD;
    __syncthreads();
    if (threadIdx.x < heads) {
        float a = 0.f, d = 0.f;
        for (int s = 0; s < nsub; ++s) {
            a += red[0][s * HP + threadIdx.x];
            d += red[1][s * HP + threadIdx.x];
        }
        p.ws[(size_t)part * 2 * p.H + h0 + threadIdx.x] = a;
        p.ws[(size_t)part * 2 * p.H + p.H + h0 + threadIdx.x] = d;
    }
}

// out[i] = sum over parts of ws[part][i], i < n.  A warp reads 32 entries (a line) of every 32nd part and
// the CTA's 32 warps are added in order (304 parts of 128: 4.5 us).
// Programmatic launch: its CTAs may be set up while the kernel before it ends, and wait here for that
// kernel's results.  (That kernel gives no earlier signal, so the two do not overlap beyond this.)
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float *__restrict__ ws, int parts, int n,
                                                         float *__restrict__ out0, float *__restrict__ out1, int split) {
    __shared__ float red[32][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int i = blockIdx.x * 32 + lane;
    float s = 0.f;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (i < n) {
#pragma unroll 4
        for (int p = warp; p < parts; p += 32) s += __ldcg(ws + (size_t)p * n + i);
    }
    red[warp][lane] = s;
    __syncthreads();
    i = blockIdx.x * 32 + warp;
    s = row_sum<32>(red[lane][warp]);
    if (lane == 0 && i < n) {
        if (i < split && out0) out0[i] = s;
        if (i >= split && out1) out1[i - split] = s;
    }
}

}  // namespace

cudaError_t launch_sum_parts(const float *ws, int parts, int n, float *out0, float *out1, int split, cudaStream_t stream) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((n + 31) / 32), cfg.blockDim = dim3(1024), cfg.stream = stream, cfg.attrs = &attr, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sum_parts_kernel, ws, parts, n, out0, out1, split);
}

namespace {

// ------------------------------------------------------------------------------------ after: forward
template <typename T, int D, int UNROLL>
__global__ void __launch_bounds__(NT) norm_fwd_kernel(NormGateArgs p) {
    using R = Rows<T, D>;
    const int lane = threadIdx.x % R::LPR;
    const long long base = (long long)blockIdx.x * R::RPB * UNROLL + threadIdx.x / R::LPR;
    uint4 ro[UNROLL], rz[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const long long r = base + i * R::RPB;
        ro[i] = rz[i] = make_uint4(0, 0, 0, 0);
        if (r < p.rows) {
            ro[i] = static_cast<const uint4 *>(p.o)[r * R::LPR + lane];
            rz[i] = static_cast<const uint4 *>(p.z)[r * R::LPR + lane];
        }
    }
    float w[R::N];
#pragma unroll
    for (int e = 0; e < R::N; e += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(p.w + lane * R::N + e);
        w[e] = f.x;
        w[e + 1] = f.y;
        w[e + 2] = f.z;
        w[e + 3] = f.w;
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const long long r = base + i * R::RPB;
        float o[R::N], z[R::N], s = 0.f;
        Vec<T>::unpack(ro[i], o);
        Vec<T>::unpack(rz[i], z);
#pragma unroll
        for (int e = 0; e < R::N; ++e) s = fmaf(o[e], o[e], s);
        const float rn = rsqrtf(row_sum<R::LPR>(s) * (1.f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < R::N; ++e) o[e] = o[e] * rn * w[e] * (z[e] * sigmoid(z[e]));
        if (r < p.rows) static_cast<uint4 *>(p.y)[r * R::LPR + lane] = Vec<T>::pack(o);
    }
}

// ------------------------------------------------------------------------------------ after: backward
// Persistent CTAs: each thread keeps dw of its columns over the rows it meets.
template <typename T, int D, int UNROLL>
__global__ void __launch_bounds__(NT, 2) norm_bwd_kernel(NormGateArgs p) {
    using R = Rows<T, D>;
    __shared__ float red[NT / 32][D];  // a warp's sums over its rows of a pass, then added in order
    const int lane = threadIdx.x % R::LPR, sub = threadIdx.x / R::LPR;
    float w[R::N], dw[R::N] = {};
#pragma unroll
    for (int e = 0; e < R::N; ++e) w[e] = p.w[lane * R::N + e];
    const long long step = (long long)gridDim.x * R::RPB * UNROLL;
    // (the bound is the same in every thread of a CTA: the shuffles need whole warps)
    for (long long blk = (long long)blockIdx.x * R::RPB * UNROLL; blk < p.rows; blk += step) {
        const long long base = blk + sub;
        uint4 ro[UNROLL], rz[UNROLL], rd[UNROLL];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const long long r = base + i * R::RPB;
            ro[i] = rz[i] = rd[i] = make_uint4(0, 0, 0, 0);
            if (r < p.rows) {
                ro[i] = static_cast<const uint4 *>(p.o)[r * R::LPR + lane];
                rz[i] = static_cast<const uint4 *>(p.z)[r * R::LPR + lane];
                rd[i] = static_cast<const uint4 *>(p.dy)[r * R::LPR + lane];
            }
        }
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const long long r = base + i * R::RPB;
            float o[R::N], z[R::N], d[R::N], s = 0.f;
            Vec<T>::unpack(ro[i], o);
            Vec<T>::unpack(rz[i], z);
            Vec<T>::unpack(rd[i], d);
#pragma unroll
            for (int e = 0; e < R::N; ++e) s = fmaf(o[e], o[e], s);
            const float rn = rsqrtf(row_sum<R::LPR>(s) * (1.f / D) + p.eps);
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < R::N; ++e) {
                const float sg = sigmoid(z[e]), n = o[e] * rn, dn = d[e] * n;
                dw[e] = fmaf(dn, z[e] * sg, dw[e]);
                const float dz = dn * w[e] * sg * fmaf(z[e], 1.f - sg, 1.f);
                d[e] *= w[e] * z[e] * sg;  // dn
                o[e] = n;
                z[e] = dz;
                m = fmaf(d[e], n, m);
            }
            m = row_sum<R::LPR>(m) * (1.f / D);
#pragma unroll
            for (int e = 0; e < R::N; ++e) o[e] = rn * fmaf(-m, o[e], d[e]);
            if (r < p.rows) {
                static_cast<uint4 *>(p.do_)[r * R::LPR + lane] = Vec<T>::pack(o);
                static_cast<uint4 *>(p.dz)[r * R::LPR + lane] = Vec<T>::pack(z);
            }
        }
    }
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int e = 0; e < R::N; ++e) {  // rows of a warp: lanes a multiple of LPR apart hold the same columns
        float x = dw[e];
#pragma unroll
        for (int off = R::LPR; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        if ((threadIdx.x & 31) < R::LPR) red[warp][lane * R::N + e] = x;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += NT) {
        float x = 0.f;
#pragma unroll
        for (int v = 0; v < NT / 32; ++v) x += red[v][c];
        p.ws[(size_t)blockIdx.x * D + c] = x;
    }
}

// Rows in flight a thread.  8 x 2048 tokens of 16 heads of 128, bf16, against 6.79 TB/s of a copy:
//   prep forward 36 us (268 MB), backward 60 (403 MB);  norm forward 30 us (201 MB), backward 55 (336 MB)
// Fewer rows with more CTAs a SM give the norm's backward 52 to 56, three CTAs a SM of 4 rows spill: 70.
constexpr int UF = 4;

template <typename T, int D>
cudaError_t prep_launch(const MixerPrepArgs &p, bool bwd) {
    using R = Rows<T, D>;
    const long long rows = 2 * p.tokens * p.Hk;
    const unsigned row_ctas = (unsigned)((rows + R::RPB * UF - 1) / (R::RPB * UF));
    if (!bwd) {
        const unsigned gate_ctas = (unsigned)((p.tokens * p.H + NT - 1) / NT);
        prep_fwd_kernel<T, D, UF><<<row_ctas + gate_ctas, NT, 0, p.stream>>>(p, row_ctas);
        return cudaGetLastError();
    }
    const int parts = mixer_prep_parts(p.tokens);
    prep_bwd_kernel<T, D, UF><<<row_ctas + parts * ((p.H + 31) / 32), NT, 0, p.stream>>>(p, row_ctas, parts);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_sum_parts(p.ws, parts, 2 * p.H, p.dA_log, p.ddt_bias, p.H, p.stream);
}
template <typename T>
cudaError_t prep_d(const MixerPrepArgs &p, bool bwd) {
    return p.d == 32 ? prep_launch<T, 32>(p, bwd) : p.d == 64 ? prep_launch<T, 64>(p, bwd) : prep_launch<T, 128>(p, bwd);
}

template <typename T, int D>
cudaError_t norm_launch(const NormGateArgs &p, bool bwd) {
    using R = Rows<T, D>;
    const long long passes = (p.rows + R::RPB * UF - 1) / (R::RPB * UF);
    if (!bwd) {
        norm_fwd_kernel<T, D, UF><<<(unsigned)passes, NT, 0, p.stream>>>(p);
        return cudaGetLastError();
    }
    const int parts = (int)std::min<long long>(passes, NORM_GATE_PARTS);
    norm_bwd_kernel<T, D, UF><<<parts, NT, 0, p.stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_sum_parts(p.ws, parts, D, p.dw, nullptr, D, p.stream);
}
template <typename T>
cudaError_t norm_d(const NormGateArgs &p, bool bwd) {
    return p.d == 32 ? norm_launch<T, 32>(p, bwd) : p.d == 64 ? norm_launch<T, 64>(p, bwd) : norm_launch<T, 128>(p, bwd);
}

}  // namespace

cudaError_t launch_mixer_prep(const MixerPrepArgs &p, bool bwd) {
    if (p.tokens == 0 && !bwd) return cudaSuccess;
    if (p.tokens == 0) {  // the sums over no tokens
        cudaError_t e = cudaMemsetAsync(p.dA_log, 0, p.H * sizeof(float), p.stream);
        return e == cudaSuccess ? cudaMemsetAsync(p.ddt_bias, 0, p.H * sizeof(float), p.stream) : e;
    }
    return p.dtype == EFLA_BF16 ? prep_d<__nv_bfloat16>(p, bwd) : prep_d<float>(p, bwd);
}

cudaError_t launch_norm_gate(const NormGateArgs &p, bool bwd) {
    if (p.rows == 0) return bwd ? cudaMemsetAsync(p.dw, 0, p.d * sizeof(float), p.stream) : cudaSuccess;
    return p.dtype == EFLA_BF16 ? norm_d<__nv_bfloat16>(p, bwd) : norm_d<float>(p, bwd);
}

}  // namespace efla
