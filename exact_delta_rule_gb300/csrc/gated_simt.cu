// Gated delta rule in chunks of 64 tokens on CUDA cores in fp32: forward, training forward and
// backward of fp32 inputs (bf16 inputs take the tensor cores).  The formulas of the forward are in
// gated.cuh.
//
// Backward, with dS' the gradient of a chunk's end state and dO of its outputs:
//   G   = P^T dO + diag(c) K dS'          (the gradient of U)
//   dR  = W^T G,  dV = dR                 (W = T'', U = W R)
//   dS  = e^{G_C} dS' + Q^T diag(e^G) dO - K^T diag(e^G) dR
//   dY  = G - L^T dR,  Z = R - L U,  dalpha_t = dY_t . Z_t,  dbeta = dalpha dalpha/dbeta
//   dP' = Gamma o (dO U^T) o M_incl,  dL' = -Gamma o strictly-lower(dR U^T)
//   dQ  = diag(e^G) dO S^T + dP' K
//   dK  = -diag(e^G) dR S^T + diag(c) U dS'^T + dP'^T Q + (dL' + dL'^T + diag(2 dalpha dalpha/dlambda)) K
//   dg_t = e^{G_C} <S, dS'> + sum_{r >= t} a_r + sum_{s < t} w_s + sum_{r >= t > s} M_rs, where
//     a_r = dO_r . (e^{G_r} S^T q_r) - dR_r . (e^{G_r} S^T k_r),  w_s = c_s U_s . (dS'^T k_s),
//     M_rs = dP'_rs (q_r . k_s) + dL'_rs (k_r . k_s)
// dg_t is the sum over every path that the decay of token t scales: from the start state or a write
// before t to a read from t on or to the end state.  The shorter form with running sums of
// q . dq - v . dv is equal, but there the paths that do not cross t (each token's read of its own
// write among them) cancel only up to rounding, which at e^g << 1 leaves nothing of dg; here every
// term carries the factor e^{g_t}.
//
// What bounds it: fp32 FMA issue (128 a clock and SM) and the shared-memory reads that feed it; the
// state pass is serial over chunks.  The d_v columns of the state are independent of one another,
// so the serial kernels run one CTA per 32 columns (four times the CTAs of one per head at d_v = 128).
// A forward of 256 tokens of 2 heads of 32: 55 us; a training step of 2 x 300 tokens of 4 heads of 64: 209.
#include "gated.cuh"
#include "tri_inverse.cuh"

namespace efla {
namespace {

constexpr int C = 64;
constexpr int NT = 256;
constexpr int LC = C + 4;  // row stride of the C x C matrices (a multiple of 4 for the inverse)
constexpr int J = 32;      // columns of d_v per slab
constexpr int LJ = J + 4;

__device__ __forceinline__ float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ void st4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }

// ROWS x COLS of a row-major tensor (row stride `stride` elements) into shared memory [ROWS][ld] as
// fp32, rows at or past `valid` as zeros; every load of a thread is issued before its first store.
template <int ROWS, int COLS>
__device__ __forceinline__ void load_block(float *dst, int ld, const float *src, size_t stride, int valid) {
    constexpr int VPR = COLS / 4, NV = (ROWS * VPR + NT - 1) / NT;
    float4 r[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int v = threadIdx.x + n * NT, row = v / VPR, col = (v % VPR) * 4;
        r[n] = row < ROWS && row < valid ? __ldg(reinterpret_cast<const float4 *>(src + (size_t)row * stride + col))
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int v = threadIdx.x + n * NT, row = v / VPR, col = (v % VPR) * 4;
        if (row < ROWS) st4(dst + row * ld + col, r[n]);
    }
}

// The same for a whole matrix.
template <int ROWS, int COLS>
__device__ __forceinline__ void load_mat(float *dst, int ld, const float *src, size_t stride) {
    load_block<ROWS, COLS>(dst, ld, src, stride, ROWS);
}

// Per-token quantities of a chunk in shared memory.
struct Rows {
    float gw[C], gr[C], eg[C], ec[C];  // chunk_decay
    float al[C], invn[C], gn[C];         // alpha, 1/n, gamma/n
    float dadb[C], dadl[C], lam[C], bt[C];
};

// gates of the chunk: warp 0 the decays, threads 0-63 beta (0 past the end); no barrier
template <typename A>
__device__ __forceinline__ void load_gates(const A &a, Rows &R, size_t row0, int valid) {
    const int tid = threadIdx.x;
    if (tid < 32) {
        const int t = 2 * tid;
        const float g0 = t < valid ? a.g[row0 + (size_t)t * a.H] : 0.f;
        const float g1 = t + 1 < valid ? a.g[row0 + (size_t)(t + 1) * a.H] : 0.f;
        chunk_decay(g0, g1, tid, R.gw, R.gr, nullptr, 1, R.eg, R.ec);
    } else if (tid >= 64 && tid < 64 + C) {
        const int t = tid - 64;
        R.bt[t] = t < valid ? a.beta[row0 + (size_t)t * a.H] : 0.f;
    }
}

// From K, Q [C][LK] and the gates: Ab = L (strictly lower) where `keep_l`, Pm = P and W = T''
// ([C][LC]); alpha and (with `grads`) its derivatives into R.  Ends with a barrier.
template <int DK>
__device__ __forceinline__ void chunk_matrices(const float *Ks, const float *Qs, Rows &R, float *Ab, float *Pm, float *W,
                                               int valid, int euler, bool grads) {
    constexpr int LK = DK + 4;
    const int tid = threadIdx.x, r4 = tid >> 4, c4 = tid & 15;
    float kk[4][4] = {}, qk[4][4] = {};
#pragma unroll 2
    for (int i = 0; i < DK; i += 4) {
        float4 kt[4], qt[4], ks[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            kt[r] = ld4(Ks + (r4 + 16 * r) * LK + i);
            qt[r] = ld4(Qs + (r4 + 16 * r) * LK + i);
            ks[r] = ld4(Ks + (c4 + 16 * r) * LK + i);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                kk[r][c] = fmaf(kt[r].x, ks[c].x, fmaf(kt[r].y, ks[c].y, fmaf(kt[r].z, ks[c].z, fmaf(kt[r].w, ks[c].w, kk[r][c]))));
                qk[r][c] = fmaf(qt[r].x, ks[c].x, fmaf(qt[r].y, ks[c].y, fmaf(qt[r].z, ks[c].z, fmaf(qt[r].w, ks[c].w, qk[r][c]))));
            }
    }
    if (r4 == c4) {
#pragma unroll
        for (int r = 0; r < 4; ++r) R.lam[r4 + 16 * r] = kk[r][r];
    }
    __syncthreads();
    if (tid < C) {
        const float lam = R.lam[tid], bt = R.bt[tid];
        const bool live = tid < valid && lam > 0.f;
        const float in = live ? rsqrtf(lam) : 0.f;
        const float gam = !live ? 0.f : euler ? bt * lam : -expm1f(-bt * lam);
        R.al[tid] = tid < valid ? efla_alpha(bt, lam, euler) : 0.f;
        R.invn[tid] = in;
        R.gn[tid] = gam * in;
        if (grads) {
            float db = 0.f, dl = 0.f;
            if (tid < valid) gate_grad(bt, lam, euler, db, dl);
            R.dadb[tid] = db;
            R.dadl[tid] = dl;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int t = r4 + 16 * r, s = c4 + 16 * c;
            const float d = s <= t ? pair_decay(R.gw[t], R.gr[t], R.gw[s], R.gr[s]) : 0.f;
            const float l = s < t ? d * kk[r][c] : 0.f;
            if (Ab) Ab[t * LC + s] = l;
            Pm[t * LC + s] = s <= t ? d * qk[r][c] : 0.f;
            if (W) W[t * LC + s] = s < t ? R.gn[t] * l * R.invn[s] : 0.f;
        }
    __syncthreads();
    if (!W) return;
    invert_unit_lower<1, LC>(W, tid);  // ends with a barrier over all 256 threads
    // W = diag(1/n) T~ diag(gamma/n); a zero key's row keeps u_t = alpha_t r_t
    for (int e = tid; e < C * C; e += NT) {
        const int t = e / C, s = e % C;
        W[t * LC + s] = s < t    ? R.invn[t] * W[t * LC + s] * R.gn[s]
                        : s == t ? (R.invn[t] > 0.f ? R.gn[t] * R.invn[t] : R.al[t])
                                 : 0.f;
    }
    __syncthreads();
}

// ------------------------------------------------------------------------------------ forward
template <int DK>
constexpr size_t fwd_smem_floats() {
    return 2 * (size_t)C * (DK + 4) + 2 * (size_t)C * LC + (size_t)DK * LJ + 2 * (size_t)C * LJ + sizeof(Rows) / 4;
}

// One CTA per (sequence, head, slab of 32 columns of d_v).  With a.ws the chunk-start states, T''
// and P of every chunk go into the workspace (the matrices from slab 0).
template <typename TOut, int DK>
__global__ void __launch_bounds__(NT, 1) gated_fwd_kernel(GatedFwdArgs a, GatedWs L) {
    extern __shared__ __align__(16) float sm[];
    constexpr int LK = DK + 4;
    float *Ks = sm, *Qs = Ks + C * LK, *Pm = Qs + C * LK, *W = Pm + C * LC, *S = W + C * LC, *Rs = S + DK * LJ;
    float *Us = Rs + C * LJ;
    Rows &R = *reinterpret_cast<Rows *>(Us + C * LJ);
    const int tid = threadIdx.x;
    const int slabs = a.dv / J, slab = blockIdx.x % slabs, unit = blockIdx.x / slabs;
    const int n = unit / a.H, h = unit % a.H, hk = h / (a.H / a.Hk), j0 = slab * J;
    long b, bos, eos;
    if (a.cu_seqlens) {
        b = 0;
        bos = a.cu_seqlens[n];
        eos = a.cu_seqlens[n + 1];
        if (bos < 0 || eos < bos || eos > a.T) {  // malformed bounds: flag and touch nothing
            if (tid == 0) atomicExch(a.status, (int)EFLA_ERR_INVALID_ARG);
            return;
        }
    } else {
        b = n;
        bos = 0;
        eos = a.T;
    }
    const float *q = static_cast<const float *>(a.q), *k = static_cast<const float *>(a.k), *v = static_cast<const float *>(a.v);
    TOut *o = static_cast<TOut *>(a.o);
    const size_t sbase = (size_t)unit * DK * a.dv + j0;
    const int nc = (int)((eos - bos + C - 1) / C);
    char *ws = static_cast<char *>(a.ws);
    float *states = ws ? reinterpret_cast<float *>(ws + L.states) + (size_t)unit * nc * DK * a.dv + j0 : nullptr;
    auto put_state = [&](float *dst) {
        for (int e = tid; e < DK * (J / 4); e += NT) {
            const int i = e / (J / 4), c4 = (e % (J / 4)) * 4;
            st4(dst + (size_t)i * a.dv + c4, ld4(S + i * LJ + c4));
        }
    };
    for (int e = tid; e < DK * (J / 4); e += NT) {
        const int i = e / (J / 4), c4 = (e % (J / 4)) * 4;
        st4(S + i * LJ + c4, a.S0 ? ld4(a.S0 + sbase + (size_t)i * a.dv + c4) : make_float4(0, 0, 0, 0));
    }
    const int ts = tid >> 2, jq = (tid & 3) * 8;  // row and columns of this thread in the C x J tiles
    for (int c = 0; c < nc; ++c) {
        const long t0 = bos + (long)c * C;
        const int valid = (int)min((long)C, eos - t0);
        const size_t tok0 = (size_t)b * a.T + (size_t)t0, row0 = tok0 * a.H + h, rowk = tok0 * a.Hk + hk;
        __syncthreads();  // the previous chunk is done with every buffer; S is complete
        if (ws) put_state(states + (size_t)c * DK * a.dv);
        load_block<C, DK>(Ks, LK, k + rowk * DK, (size_t)a.Hk * DK, valid);
        load_block<C, DK>(Qs, LK, q + rowk * DK, (size_t)a.Hk * DK, valid);
        load_block<C, J>(Rs, LJ, v + row0 * a.dv + j0, (size_t)a.H * a.dv, valid);
        load_gates(a, R, row0, valid);
        __syncthreads();
        chunk_matrices<DK>(Ks, Qs, R, nullptr, Pm, W, valid, a.euler, false);
        if (ws && slab == 0) {
            float *wd = reinterpret_cast<float *>(ws + L.w) + ((size_t)unit * nc + c) * C * C;
            float *pd = reinterpret_cast<float *>(ws + L.p) + ((size_t)unit * nc + c) * C * C;
            for (int e = 4 * tid; e < C * C; e += 4 * NT) {
                st4(wd + e, ld4(W + (e / C) * LC + e % C));
                st4(pd + e, ld4(Pm + (e / C) * LC + e % C));
            }
        }
        float x[8] = {}, y[8] = {};  // rows of K S and Q S
#pragma unroll 2
        for (int i = 0; i < DK; i += 4) {
            const float4 kt = ld4(Ks + ts * LK + i), qt = ld4(Qs + ts * LK + i);
            const float kv[4] = {kt.x, kt.y, kt.z, kt.w}, qv[4] = {qt.x, qt.y, qt.z, qt.w};
#pragma unroll
            for (int ii = 0; ii < 4; ++ii) {
                const float4 s0 = ld4(S + (i + ii) * LJ + jq), s1 = ld4(S + (i + ii) * LJ + jq + 4);
                const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    x[m] = fmaf(kv[ii], sv[m], x[m]);
                    y[m] = fmaf(qv[ii], sv[m], y[m]);
                }
            }
        }
        const float eg = R.eg[ts];
        {  // R = V - e^G K S (this thread's own elements)
            float *rp = Rs + ts * LJ + jq;
            const float4 v0 = ld4(rp), v1 = ld4(rp + 4);
            st4(rp, make_float4(fmaf(-eg, x[0], v0.x), fmaf(-eg, x[1], v0.y), fmaf(-eg, x[2], v0.z), fmaf(-eg, x[3], v0.w)));
            st4(rp + 4, make_float4(fmaf(-eg, x[4], v1.x), fmaf(-eg, x[5], v1.y), fmaf(-eg, x[6], v1.z), fmaf(-eg, x[7], v1.w)));
        }
        __syncthreads();
        float u[8] = {};
        for (int s = 0; s <= ts; ++s) {  // U = T'' R
            const float wv = W[ts * LC + s];
            const float4 a0 = ld4(Rs + s * LJ + jq), a1 = ld4(Rs + s * LJ + jq + 4);
            const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
            for (int m = 0; m < 8; ++m) u[m] = fmaf(wv, av[m], u[m]);
        }
        st4(Us + ts * LJ + jq, make_float4(u[0], u[1], u[2], u[3]));
        st4(Us + ts * LJ + jq + 4, make_float4(u[4], u[5], u[6], u[7]));
        __syncthreads();
        if (o && ts < valid) {  // O = e^G Q S + P U
#pragma unroll
            for (int m = 0; m < 8; ++m) y[m] *= eg;
            for (int s = 0; s <= ts; ++s) {
                const float pv = Pm[ts * LC + s];
                const float4 a0 = ld4(Us + s * LJ + jq), a1 = ld4(Us + s * LJ + jq + 4);
                const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
                for (int m = 0; m < 8; ++m) y[m] = fmaf(pv, av[m], y[m]);
            }
            TOut *op = o + (row0 + (size_t)ts * a.H) * a.dv + j0 + jq;
#pragma unroll
            for (int m = 0; m < 8; ++m) op[m] = from_f32<TOut>(y[m]);
        }
        {  // S = e^{G_C} S + K^T diag(c) U: thread (i, column group)
            constexpr int CG = NT / DK < 1 ? 1 : NT / DK, CW = J / CG;  // column groups, columns a thread
            const int i = tid % DK, cg = (tid / DK) * CW;
            const float el = R.eg[C - 1];
            float s[CW];
#pragma unroll
            for (int m = 0; m < CW; ++m) s[m] = el * S[i * LJ + cg + m];
            for (int t = 0; t < valid; ++t) {
                const float kc = Ks[t * LK + i] * R.ec[t];
#pragma unroll
                for (int m = 0; m < CW; m += 4) {
                    const float4 uv = ld4(Us + t * LJ + cg + m);
                    s[m] = fmaf(kc, uv.x, s[m]);
                    s[m + 1] = fmaf(kc, uv.y, s[m + 1]);
                    s[m + 2] = fmaf(kc, uv.z, s[m + 2]);
                    s[m + 3] = fmaf(kc, uv.w, s[m + 3]);
                }
            }
#pragma unroll
            for (int m = 0; m < CW; ++m) S[i * LJ + cg + m] = s[m];
        }
    }
    __syncthreads();
    if (a.S_T) put_state(a.S_T + sbase);
}

// ------------------------------------------------------------------------------------ state gradients
template <int DK>
constexpr size_t state_smem_floats() {
    return 2 * (size_t)C * (DK + 4) + 2 * (size_t)C * LC + (size_t)DK * LJ + 2 * (size_t)C * LJ + sizeof(Rows) / 4;
}

// Sum over the CTA (one value a thread), the result in every thread; red: NT / 32 floats.
__device__ __forceinline__ float block_sum(float x, float *red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) s += red[w];
    return s;
}

// One CTA per (b, h, slab of 32 columns) walks the chunks in reverse: dS' of every chunk and this
// slab's share of <S, dS'> into the workspace, dS0 at the end.
template <int DK>
__global__ void __launch_bounds__(NT, 1) gated_bwd_state_kernel(GatedBwdArgs a, GatedWs L) {
    extern __shared__ __align__(16) float sm[];
    __shared__ float red[NT / 32];
    constexpr int LK = DK + 4;
    float *Ks = sm, *Qs = Ks + C * LK, *Pm = Qs + C * LK, *W = Pm + C * LC, *dS = W + C * LC, *dOs = dS + DK * LJ;
    float *Gs = dOs + C * LJ;
    Rows &R = *reinterpret_cast<Rows *>(Gs + C * LJ);
    const int tid = threadIdx.x;
    const int dv = a.dv_dim, slabs = dv / J, slab = blockIdx.x % slabs, unit = blockIdx.x / slabs, j0 = slab * J;
    const int b = unit / a.H, h = unit % a.H, hk = h / (a.H / a.Hk);
    const int nc = (a.T + C - 1) / C;
    const float *q = static_cast<const float *>(a.q), *k = static_cast<const float *>(a.k), *dO = static_cast<const float *>(a.dO);
    char *ws = static_cast<char *>(a.ws);
    const float *states = reinterpret_cast<const float *>(ws + L.states) + (size_t)unit * nc * DK * dv + j0;
    float *dse = reinterpret_cast<float *>(ws + L.dse) + (size_t)unit * nc * DK * dv + j0;
    float *sdot = reinterpret_cast<float *>(ws + L.sdot) + (size_t)unit * nc * 4;
    const size_t sbase = (size_t)unit * DK * dv + j0;
    for (int e = tid; e < DK * J; e += NT) {
        const int i = e / J, j = e % J;
        dS[i * LJ + j] = a.dST ? a.dST[sbase + (size_t)i * dv + j] : 0.f;
    }
    const int ts = tid >> 2, jq = (tid & 3) * 8;
    for (int c = nc - 1; c >= 0; --c) {
        const int valid = min(C, a.T - c * C);
        const size_t tok0 = (size_t)b * a.T + (size_t)c * C, row0 = tok0 * a.H + h, rowk = tok0 * a.Hk + hk;
        __syncthreads();
        float dot = 0.f;
        for (int e = tid; e < DK * (J / 4); e += NT) {
            const int i = e / (J / 4), c4 = (e % (J / 4)) * 4;
            const float4 d = ld4(dS + i * LJ + c4), s = ld4(states + (size_t)c * DK * dv + (size_t)i * dv + c4);
            st4(dse + (size_t)c * DK * dv + (size_t)i * dv + c4, d);
            dot = fmaf(d.x, s.x, fmaf(d.y, s.y, fmaf(d.z, s.z, fmaf(d.w, s.w, dot))));
        }
        dot = block_sum(dot, red);
        if (tid == 0) sdot[c * 4 + slab] = dot;
        load_block<C, DK>(Ks, LK, k + rowk * DK, (size_t)a.Hk * DK, valid);
        load_block<C, DK>(Qs, LK, q + rowk * DK, (size_t)a.Hk * DK, valid);
        load_block<C, J>(dOs, LJ, dO + row0 * dv + j0, (size_t)a.H * dv, valid);
        load_mat<C, C>(W, LC, reinterpret_cast<const float *>(ws + L.w) + ((size_t)unit * nc + c) * C * C, C);
        load_mat<C, C>(Pm, LC, reinterpret_cast<const float *>(ws + L.p) + ((size_t)unit * nc + c) * C * C, C);
        load_gates(a, R, row0, valid);
        __syncthreads();
        float x[8] = {};
#pragma unroll 2
        for (int i = 0; i < DK; i += 4) {
            const float4 kt = ld4(Ks + ts * LK + i);
            const float kv[4] = {kt.x, kt.y, kt.z, kt.w};
#pragma unroll
            for (int ii = 0; ii < 4; ++ii) {
                const float4 s0 = ld4(dS + (i + ii) * LJ + jq), s1 = ld4(dS + (i + ii) * LJ + jq + 4);
                const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                for (int m = 0; m < 8; ++m) x[m] = fmaf(kv[ii], sv[m], x[m]);
            }
        }
#pragma unroll
        for (int m = 0; m < 8; ++m) x[m] *= R.ec[ts];
        for (int s = ts; s < valid; ++s) {
            const float pv = Pm[s * LC + ts];
            const float4 a0 = ld4(dOs + s * LJ + jq), a1 = ld4(dOs + s * LJ + jq + 4);
            const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
            for (int m = 0; m < 8; ++m) x[m] = fmaf(pv, av[m], x[m]);
        }
        st4(Gs + ts * LJ + jq, make_float4(x[0], x[1], x[2], x[3]));
        st4(Gs + ts * LJ + jq + 4, make_float4(x[4], x[5], x[6], x[7]));
        __syncthreads();
        float r[8] = {};
        for (int s = ts; s < C; ++s) {
            const float wv = W[s * LC + ts];
            const float4 a0 = ld4(Gs + s * LJ + jq), a1 = ld4(Gs + s * LJ + jq + 4);
            const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
            for (int m = 0; m < 8; ++m) r[m] = fmaf(wv, av[m], r[m]);
        }
        __syncthreads();
        st4(Gs + ts * LJ + jq, make_float4(r[0], r[1], r[2], r[3]));
        st4(Gs + ts * LJ + jq + 4, make_float4(r[4], r[5], r[6], r[7]));
        __syncthreads();
        {  // dS = e^{G_C} dS' + Q^T diag(e^G) dO - K^T diag(e^G) dR
            constexpr int CG = NT / DK < 1 ? 1 : NT / DK, CW = J / CG;
            const int i = tid % DK, cg = (tid / DK) * CW;
            const float el = R.eg[C - 1];
            float s[CW];
#pragma unroll
            for (int m = 0; m < CW; ++m) s[m] = el * dS[i * LJ + cg + m];
            for (int t = 0; t < valid; ++t) {
                const float qe = Qs[t * LK + i] * R.eg[t], ke = -Ks[t * LK + i] * R.eg[t];
#pragma unroll
                for (int m = 0; m < CW; m += 4) {
                    const float4 ov = ld4(dOs + t * LJ + cg + m), rv = ld4(Gs + t * LJ + cg + m);
                    s[m] = fmaf(qe, ov.x, fmaf(ke, rv.x, s[m]));
                    s[m + 1] = fmaf(qe, ov.y, fmaf(ke, rv.y, s[m + 1]));
                    s[m + 2] = fmaf(qe, ov.z, fmaf(ke, rv.z, s[m + 2]));
                    s[m + 3] = fmaf(qe, ov.w, fmaf(ke, rv.w, s[m + 3]));
                }
            }
#pragma unroll
            for (int m = 0; m < CW; ++m) dS[i * LJ + cg + m] = s[m];
        }
    }
    __syncthreads();
    if (a.dS0)
        for (int e = tid; e < DK * J; e += NT) {
            const int i = e / J, j = e % J;
            a.dS0[sbase + (size_t)i * dv + j] = dS[i * LJ + j];
        }
}

// ------------------------------------------------------------------------------------ per-chunk gradients
template <int DK>
constexpr size_t grad_smem_floats() {
    return 2 * (size_t)C * (DK + 4) + 3 * (size_t)C * LC + 2 * (size_t)DK * LJ + 6 * (size_t)C * LJ + sizeof(Rows) / 4 +
           3 * C;
}

// One CTA per (b, h, chunk): every token's gradients from the chunk's S and dS'.  Where key heads
// are shared (Hk < H) dq and dk of each value head go to part in fp32.
template <int DK>
__global__ void __launch_bounds__(NT, 1) gated_bwd_grad_kernel(GatedBwdArgs a, GatedWs L) {
    extern __shared__ __align__(16) float sm[];
    constexpr int LK = DK + 4;
    constexpr int TI = DK / 16;
    float *Ks = sm, *Qs = Ks + C * LK, *Ab = Qs + C * LK, *Pm = Ab + C * LC, *W = Pm + C * LC;
    float *Ssl = W + C * LC, *dSsl = Ssl + DK * LJ, *Vsl = dSsl + DK * LJ, *dOsl = Vsl + C * LJ, *Rs = dOsl + C * LJ;
    float *Us = Rs + C * LJ, *Gs = Us + C * LJ, *dRs = Gs + C * LJ;
    Rows &R = *reinterpret_cast<Rows *>(dRs + C * LJ);
    float *dal = reinterpret_cast<float *>(&R + 1), *ra = dal + C, *rw = ra + C;  // dalpha, a, w
    float *Ms = Vsl;  // at the end: M [C][LC]
    const int tid = threadIdx.x, dv = a.dv_dim;
    const int nc = (a.T + C - 1) / C, unit = blockIdx.x / nc, c = blockIdx.x % nc;
    const int b = unit / a.H, h = unit % a.H, hk = h / (a.H / a.Hk);
    const int valid = min(C, a.T - c * C);
    const float *q = static_cast<const float *>(a.q), *k = static_cast<const float *>(a.k), *v = static_cast<const float *>(a.v);
    const float *dO = static_cast<const float *>(a.dO);
    char *ws = static_cast<char *>(a.ws);
    const float *Sc = reinterpret_cast<const float *>(ws + L.states) + ((size_t)unit * nc + c) * DK * dv;
    const float *dSe = reinterpret_cast<const float *>(ws + L.dse) + ((size_t)unit * nc + c) * DK * dv;
    const size_t tok0 = (size_t)b * a.T + (size_t)c * C, row0 = tok0 * a.H + h, rowk = tok0 * a.Hk + hk;
    load_block<C, DK>(Ks, LK, k + rowk * DK, (size_t)a.Hk * DK, valid);
    load_block<C, DK>(Qs, LK, q + rowk * DK, (size_t)a.Hk * DK, valid);
    load_gates(a, R, row0, valid);
    __syncthreads();
    chunk_matrices<DK>(Ks, Qs, R, Ab, Pm, nullptr, valid, a.euler, true);
    load_mat<C, C>(W, LC, reinterpret_cast<const float *>(ws + L.w) + ((size_t)unit * nc + c) * C * C, C);

    const int ts = tid >> 2, jq = (tid & 3) * 8;
    const int r4 = tid >> 4, c4 = tid & 15;
    float dP[4][4] = {}, dLr[4][4] = {}, dQ[4][TI] = {}, dK[4][TI] = {};
    float dal_part = 0.f, a_part = 0.f, w_part = 0.f;
    const float eg = R.eg[ts], ec = R.ec[ts];
    float eg4[4], ec4[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        eg4[r] = R.eg[r4 + 16 * r];
        ec4[r] = R.ec[r4 + 16 * r];
    }

#pragma unroll 1
    for (int j0 = 0; j0 < dv; j0 += J) {
        __syncthreads();  // the previous slab's buffers are free
        load_mat<DK, J>(Ssl, LJ, Sc + j0, dv);
        load_mat<DK, J>(dSsl, LJ, dSe + j0, dv);
        load_block<C, J>(Vsl, LJ, v + row0 * dv + j0, (size_t)a.H * dv, valid);
        load_block<C, J>(dOsl, LJ, dO + row0 * dv + j0, (size_t)a.H * dv, valid);
        __syncthreads();
        float x[8] = {}, gk[8] = {}, y[8] = {};  // row ts, columns jq ..: e^G K S, c K dS', e^G Q S
        {  // R = V - e^G K S and G = P^T dO + c K dS'
            float g[8];
#pragma unroll 1
            for (int i = 0; i < DK; i += 4) {
                const float4 kt = ld4(Ks + ts * LK + i), qt = ld4(Qs + ts * LK + i);
                const float kv[4] = {kt.x, kt.y, kt.z, kt.w}, qv[4] = {qt.x, qt.y, qt.z, qt.w};
#pragma unroll
                for (int ii = 0; ii < 4; ++ii) {
                    const float4 s0 = ld4(Ssl + (i + ii) * LJ + jq), s1 = ld4(Ssl + (i + ii) * LJ + jq + 4);
                    const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
                    const float4 d0 = ld4(dSsl + (i + ii) * LJ + jq), d1 = ld4(dSsl + (i + ii) * LJ + jq + 4);
                    const float dv8[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
#pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        x[m] = fmaf(kv[ii], sv[m], x[m]);
                        y[m] = fmaf(qv[ii], sv[m], y[m]);
                        gk[m] = fmaf(kv[ii], dv8[m], gk[m]);
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                x[m] *= eg;
                y[m] *= eg;
                g[m] = gk[m] *= ec;
            }
#pragma unroll 1
            for (int s = ts; s < valid; ++s) {
                const float pv = Pm[s * LC + ts];
                const float4 o0 = ld4(dOsl + s * LJ + jq), o1 = ld4(dOsl + s * LJ + jq + 4);
                const float ov[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
#pragma unroll
                for (int m = 0; m < 8; ++m) g[m] = fmaf(pv, ov[m], g[m]);
            }
            const float4 v0 = ld4(Vsl + ts * LJ + jq), v1 = ld4(Vsl + ts * LJ + jq + 4);
            st4(Rs + ts * LJ + jq, make_float4(v0.x - x[0], v0.y - x[1], v0.z - x[2], v0.w - x[3]));
            st4(Rs + ts * LJ + jq + 4, make_float4(v1.x - x[4], v1.y - x[5], v1.z - x[6], v1.w - x[7]));
            st4(Gs + ts * LJ + jq, make_float4(g[0], g[1], g[2], g[3]));
            st4(Gs + ts * LJ + jq + 4, make_float4(g[4], g[5], g[6], g[7]));
        }
        __syncthreads();
        {  // U = W R and dR = W^T G
            float u[8] = {}, r[8] = {};
#pragma unroll 1
            for (int s = 0; s <= ts; ++s) {
                const float wv = W[ts * LC + s];
                const float4 a0 = ld4(Rs + s * LJ + jq), a1 = ld4(Rs + s * LJ + jq + 4);
                const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
                for (int m = 0; m < 8; ++m) u[m] = fmaf(wv, av[m], u[m]);
            }
#pragma unroll 1
            for (int s = ts; s < C; ++s) {
                const float wv = W[s * LC + ts];
                const float4 a0 = ld4(Gs + s * LJ + jq), a1 = ld4(Gs + s * LJ + jq + 4);
                const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
                for (int m = 0; m < 8; ++m) r[m] = fmaf(wv, av[m], r[m]);
            }
            st4(Us + ts * LJ + jq, make_float4(u[0], u[1], u[2], u[3]));
            st4(Us + ts * LJ + jq + 4, make_float4(u[4], u[5], u[6], u[7]));
            st4(dRs + ts * LJ + jq, make_float4(r[0], r[1], r[2], r[3]));
            st4(dRs + ts * LJ + jq + 4, make_float4(r[4], r[5], r[6], r[7]));
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                a_part = fmaf(dOsl[ts * LJ + jq + m], y[m], fmaf(-r[m], x[m], a_part));
                w_part = fmaf(u[m], gk[m], w_part);
            }
            if (ts < valid) {  // dv = dR
                float *dvp = static_cast<float *>(a.dv) + (row0 + (size_t)ts * a.H) * dv + j0 + jq;
#pragma unroll
                for (int m = 0; m < 8; ++m) dvp[m] = r[m];
            }
        }
        __syncthreads();
        {  // dalpha_t += sum_j (G - L^T dR)[t][j] (R - L U)[t][j]
            float y[8], z[8];
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                y[m] = Gs[ts * LJ + jq + m];
                z[m] = Rs[ts * LJ + jq + m];
            }
#pragma unroll 1
            for (int s = ts + 1; s < valid; ++s) {
                const float lv = Ab[s * LC + ts];
                const float4 a0 = ld4(dRs + s * LJ + jq), a1 = ld4(dRs + s * LJ + jq + 4);
                const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
                for (int m = 0; m < 8; ++m) y[m] = fmaf(-lv, av[m], y[m]);
            }
#pragma unroll 1
            for (int s = 0; s < ts; ++s) {
                const float lv = Ab[ts * LC + s];
                const float4 a0 = ld4(Us + s * LJ + jq), a1 = ld4(Us + s * LJ + jq + 4);
                const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
                for (int m = 0; m < 8; ++m) z[m] = fmaf(-lv, av[m], z[m]);
            }
#pragma unroll
            for (int m = 0; m < 8; ++m) dal_part = fmaf(y[m], z[m], dal_part);
        }
        {  // dP += dO U^T, dLr += dR U^T; dQ += e^G dO S^T, dK += -e^G dR S^T + c U dS'^T
#pragma unroll 1
            for (int jj = 0; jj < J; jj += 4) {
                float4 o4[4], r4v[4], u4[4], uc[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    o4[r] = ld4(dOsl + (r4 + 16 * r) * LJ + jj);
                    r4v[r] = ld4(dRs + (r4 + 16 * r) * LJ + jj);
                    u4[r] = ld4(Us + (r4 + 16 * r) * LJ + jj);
                    uc[r] = ld4(Us + (c4 + 16 * r) * LJ + jj);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc) {
                        dP[r][cc] = fmaf(o4[r].x, uc[cc].x, fmaf(o4[r].y, uc[cc].y, fmaf(o4[r].z, uc[cc].z, fmaf(o4[r].w, uc[cc].w, dP[r][cc]))));
                        dLr[r][cc] = fmaf(r4v[r].x, uc[cc].x, fmaf(r4v[r].y, uc[cc].y, fmaf(r4v[r].z, uc[cc].z, fmaf(r4v[r].w, uc[cc].w, dLr[r][cc]))));
                    }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    o4[r] = make_float4(eg4[r] * o4[r].x, eg4[r] * o4[r].y, eg4[r] * o4[r].z, eg4[r] * o4[r].w);
                    r4v[r] = make_float4(eg4[r] * r4v[r].x, eg4[r] * r4v[r].y, eg4[r] * r4v[r].z, eg4[r] * r4v[r].w);
                    u4[r] = make_float4(ec4[r] * u4[r].x, ec4[r] * u4[r].y, ec4[r] * u4[r].z, ec4[r] * u4[r].w);
                }
#pragma unroll
                for (int cc = 0; cc < TI; ++cc) {
                    const float4 s4 = ld4(Ssl + (c4 + 16 * cc) * LJ + jj);
                    const float4 e4 = ld4(dSsl + (c4 + 16 * cc) * LJ + jj);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        dQ[r][cc] = fmaf(o4[r].x, s4.x, fmaf(o4[r].y, s4.y, fmaf(o4[r].z, s4.z, fmaf(o4[r].w, s4.w, dQ[r][cc]))));
                        float x = dK[r][cc];
                        x = fmaf(-r4v[r].x, s4.x, fmaf(-r4v[r].y, s4.y, fmaf(-r4v[r].z, s4.z, fmaf(-r4v[r].w, s4.w, x))));
                        x = fmaf(u4[r].x, e4.x, fmaf(u4[r].y, e4.y, fmaf(u4[r].z, e4.z, fmaf(u4[r].w, e4.w, x))));
                        dK[r][cc] = x;
                    }
                }
            }
        }
    }
    dal_part += __shfl_xor_sync(0xffffffffu, dal_part, 1);
    dal_part += __shfl_xor_sync(0xffffffffu, dal_part, 2);
    a_part += __shfl_xor_sync(0xffffffffu, a_part, 1);
    a_part += __shfl_xor_sync(0xffffffffu, a_part, 2);
    w_part += __shfl_xor_sync(0xffffffffu, w_part, 1);
    w_part += __shfl_xor_sync(0xffffffffu, w_part, 2);
    __syncthreads();  // every slab done: Pm, Ab and W are free
    if ((tid & 3) == 0) {
        dal[ts] = dal_part;
        ra[ts] = a_part;
        rw[ts] = w_part;
    }
    // M, then dP' (inclusive lower) into Pm, dL' = -strictly-lower(dLr) into W, both times Gamma
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
            const int t = r4 + 16 * r, s = c4 + 16 * cc;
            const float d = s <= t ? pair_decay(R.gw[t], R.gr[t], R.gw[s], R.gr[s]) : 0.f;
            Ms[t * LC + s] = s < t ? fmaf(dP[r][cc], Pm[t * LC + s], -dLr[r][cc] * Ab[t * LC + s]) : 0.f;
            Pm[t * LC + s] = s <= t ? d * dP[r][cc] : 0.f;
            W[t * LC + s] = s < t ? -d * dLr[r][cc] : 0.f;
        }
    __syncthreads();
    for (int e = tid; e < C * C; e += NT) {  // dL' + dL'^T into Ab
        const int t = e / C, s = e % C;
        Ab[t * LC + s] = W[t * LC + s] + W[s * LC + t];
    }
    __syncthreads();
#pragma unroll 1
    for (int s = 0; s < valid; ++s) {  // dQ += dP' K, dK += dP'^T Q + (dL' + dL'^T) K
        float pr[4], pc[4], lr[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = r4 + 16 * r;
            pr[r] = Pm[t * LC + s];
            pc[r] = Pm[s * LC + t];
            lr[r] = Ab[t * LC + s];
        }
#pragma unroll
        for (int cc = 0; cc < TI; ++cc) {
            const float kv = Ks[s * LK + c4 + 16 * cc], qv = Qs[s * LK + c4 + 16 * cc];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dQ[r][cc] = fmaf(pr[r], kv, dQ[r][cc]);
                dK[r][cc] = fmaf(pc[r], qv, fmaf(lr[r], kv, dK[r][cc]));
            }
        }
    }
    const bool shared_heads = a.Hk != a.H;
    float *pq = reinterpret_cast<float *>(ws + L.part), *pk = pq + (size_t)a.B * a.T * a.H * DK;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int t = r4 + 16 * r;
        const float dl2 = 2.f * dal[t] * R.dadl[t];
        const size_t rowv = row0 + (size_t)t * a.H, rowo = rowk + (size_t)t * a.Hk;
#pragma unroll
        for (int cc = 0; cc < TI; ++cc) {
            const int i = c4 + 16 * cc;
            const float dk = fmaf(dl2, Ks[t * LK + i], dK[r][cc]);
            if (t < valid) {
                if (shared_heads) {
                    pq[rowv * DK + i] = dQ[r][cc];
                    pk[rowv * DK + i] = dk;
                } else {
                    static_cast<float *>(a.dq)[rowo * DK + i] = dQ[r][cc];
                    static_cast<float *>(a.dk)[rowo * DK + i] = dk;
                }
            }
        }
    }
    if (tid < valid) a.dbeta[row0 + (size_t)tid * a.H] = dal[tid] * R.dadb[tid];
    {  // M row ts -> its exclusive prefix sums R_r(t) = sum_{s < t} M_rs (16 columns a thread)
        float *m = Ms + ts * LC + (tid & 3) * 16, p = 0.f, x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            x[e] = p;
            p += m[e];
        }
        float before = 0.f;
#pragma unroll
        for (int w = 0; w < 3; ++w) {
            const float y = __shfl_sync(0xffffffffu, p, (tid & 28) + w);
            if (w < (tid & 3)) before += y;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) m[e] = before + x[e];
    }
    __syncthreads();
    {  // dg_t: column t of R from row t on, the suffix of a and the prefix of w (a quarter of the rows a thread)
        float s = 0.f;
        for (int r = (tid & 3) * 16; r < (tid & 3) * 16 + 16; ++r)
            s += r >= ts ? ra[r] + Ms[r * LC + ts] : rw[r];
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if ((tid & 3) == 0 && ts < valid) {
            const float *sd = reinterpret_cast<const float *>(ws + L.sdot) + ((size_t)unit * nc + c) * 4;
            float through = 0.f;
            for (int j = 0; j < dv / J; ++j) through += sd[j];
            a.dg[row0 + (size_t)ts * a.H] = fmaf(R.eg[C - 1], through, s);
        }
    }
}

static_assert(fwd_smem_floats<128>() * 4 <= 232448 && state_smem_floats<128>() * 4 + 64 <= 232448 &&
                  grad_smem_floats<128>() * 4 <= 232448,
              "shared memory of a CTA");

// ------------------------------------------------------------------------------------ shared key heads
// One thread per four features of a key head's token: adds the H / Hk value heads in order.
template <typename TOut>
__global__ void __launch_bounds__(256) reduce_heads_kernel(const float *__restrict__ part, TOut *__restrict__ dq,
                                                           TOut *__restrict__ dk, size_t tokens, int Hk, int rep, int d) {
    const size_t n4 = tokens * Hk * d / 4;
    const size_t plane = tokens * Hk * rep * d;
    for (size_t e = blockIdx.x * (size_t)blockDim.x + threadIdx.x; e < 2 * n4; e += (size_t)gridDim.x * blockDim.x) {
        const bool is_k = e >= n4;
        const size_t x = (is_k ? e - n4 : e) * 4, row = x / d, i = x % d;  // row = token * Hk + key head
        const float *src = part + (is_k ? plane : 0) + row * rep * d + i;
        float4 s = ld4(src);
        for (int r = 1; r < rep; ++r) {
            const float4 y = ld4(src + (size_t)r * d);
            s.x += y.x;
            s.y += y.y;
            s.z += y.z;
            s.w += y.w;
        }
        TOut *dst = (is_k ? dk : dq) + x;
        dst[0] = from_f32<TOut>(s.x);
        dst[1] = from_f32<TOut>(s.y);
        dst[2] = from_f32<TOut>(s.z);
        dst[3] = from_f32<TOut>(s.w);
    }
}

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename TOut, int DK>
cudaError_t fwd_launch(const GatedFwdArgs &a) {
    const size_t bytes = fwd_smem_floats<DK>() * 4;
    const GatedWs L = gated_ws(a.B, a.T, a.Hk, a.H, a.dk, a.dv, a.in_dtype);
    cudaError_t e = allow_smem(gated_fwd_kernel<TOut, DK>, bytes);
    if (e != cudaSuccess) return e;
    gated_fwd_kernel<TOut, DK><<<(unsigned)((long)a.N * a.H * (a.dv / J)), NT, bytes, a.stream>>>(a, L);
    return cudaGetLastError();
}
template <typename TOut>
cudaError_t fwd_dk(const GatedFwdArgs &a) {
    return a.dk == 32 ? fwd_launch<TOut, 32>(a) : a.dk == 64 ? fwd_launch<TOut, 64>(a) : fwd_launch<TOut, 128>(a);
}

template <int DK>
cudaError_t bwd_launch(const GatedBwdArgs &a) {
    const GatedWs L = gated_ws(a.B, a.T, a.Hk, a.H, a.dk_dim, a.dv_dim, a.in_dtype);
    const size_t b1 = state_smem_floats<DK>() * 4, b2 = grad_smem_floats<DK>() * 4;
    const long units = (long)a.B * a.H, nc = (a.T + C - 1) / C;
    cudaError_t e = allow_smem(gated_bwd_state_kernel<DK>, b1);
    if (e == cudaSuccess) e = allow_smem(gated_bwd_grad_kernel<DK>, b2);
    if (e != cudaSuccess) return e;
    gated_bwd_state_kernel<DK><<<(unsigned)(units * (a.dv_dim / J)), NT, b1, a.stream>>>(a, L);
    if ((e = cudaGetLastError()) != cudaSuccess || nc == 0) return e;
    gated_bwd_grad_kernel<DK><<<(unsigned)(units * nc), NT, b2, a.stream>>>(a, L);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return a.Hk == a.H ? cudaSuccess
                       : launch_gated_reduce_heads(a, reinterpret_cast<const float *>(static_cast<char *>(a.ws) + L.part));
}

}  // namespace

cudaError_t launch_gated_chunk_simt(const GatedFwdArgs &a) {
    if (a.N == 0) return cudaSuccess;
    return a.o_dtype == EFLA_BF16 ? fwd_dk<__nv_bfloat16>(a) : fwd_dk<float>(a);
}

cudaError_t launch_gated_bwd_simt(const GatedBwdArgs &a) {
    if ((long)a.B * a.H == 0) return cudaSuccess;
    switch (a.dk_dim) {
        case 32: return bwd_launch<32>(a);
        case 64: return bwd_launch<64>(a);
        default: return bwd_launch<128>(a);
    }
}

cudaError_t launch_gated_reduce_heads(const GatedBwdArgs &a, const float *part) {
    const size_t tokens = (size_t)a.B * a.T, n = tokens * a.Hk * a.dk_dim / 2;
    if (n == 0) return cudaSuccess;
    const unsigned grid = (unsigned)std::min<size_t>((n + 255) / 256, 152 * 16);
    const int rep = a.H / a.Hk;
    if (a.in_dtype == EFLA_BF16)
        reduce_heads_kernel<<<grid, 256, 0, a.stream>>>(part, static_cast<__nv_bfloat16 *>(a.dq),
                                                         static_cast<__nv_bfloat16 *>(a.dk), tokens, a.Hk, rep, a.dk_dim);
    else
        reduce_heads_kernel<<<grid, 256, 0, a.stream>>>(part, static_cast<float *>(a.dq), static_cast<float *>(a.dk),
                                                         tokens, a.Hk, rep, a.dk_dim);
    return cudaGetLastError();
}

}  // namespace efla
