// Gated delta rule, one token per sequence: S <- e^g (I - alpha k k^T) S + alpha k v^T, o = S^T q with the
// updated state, S in place.  In one pass over S, with Sd = e^g S:
//   x = Sd^T k, y = Sd^T q, u = alpha (v - x), S = Sd + k u^T, o = y + (q . k) u.
//
// HBM bound: S is read and written once (8 d_k d_v bytes a head; the vectors are 0.8 % of it).  A CTA
// of 256 threads holds the rows of S for COLS of the d_v columns in registers, read and written once
// with 16-byte accesses; the column sums over the row groups go through shared memory.  The columns
// are independent, so COLS trades CTAs for the repeated reading of k and q: with COLS = d_v a step of
// 8192 heads streams at the copy rate (158 us, 1.08 GB), while fewer heads than SMs leave SMs idle and
// the load latency of a 64 KB state bare; then 32 columns a CTA (a row of it is still one 128-byte line).
// d = 128, bf16, 32 columns / d_v a CTA: 8 heads 2.3 / 3.2 us, 32 2.7 / 3.5, 128 5.1 / 5.3, 256 8.8 / 8.3,
// 2048 48 / 45.
#include "gated.cuh"

namespace efla {
namespace {

constexpr int NT = 256;

template <int DK, int COLS, typename TIn, typename TOut>
__global__ void __launch_bounds__(NT) gated_decode_kernel(const TIn *__restrict__ q, const TIn *__restrict__ k,
                                                          const TIn *__restrict__ v, const float *__restrict__ g,
                                                          const float *__restrict__ beta, float *__restrict__ S,
                                                          TOut *__restrict__ o, int H, int rep, int dv, int euler) {
    constexpr int CG = COLS / 4, RG = NT / CG, ROWS = DK / RG;  // column groups, row groups, rows a thread
    static_assert(ROWS >= 1 && ROWS * RG == DK, "unsupported decode shape");
    __shared__ float ks[DK], qs[DK];
    __shared__ float red_x[RG][COLS], red_y[RG][COLS];
    __shared__ float us[COLS];
    __shared__ float scal[2];
    const int slabs = dv / COLS, unit = blockIdx.x / slabs, j0 = (blockIdx.x % slabs) * COLS;  // unit = b H + h
    const int b = unit / H, h = unit % H;
    const size_t rowk = (size_t)b * (H / rep) + h / rep;
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG;

    float *Su = S + (size_t)unit * DK * dv + j0 + 4 * cg;
    float4 reg[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) reg[r] = *reinterpret_cast<const float4 *>(Su + (size_t)(rg + r * RG) * dv);
    const float gt = g[unit], bt = beta[unit];
    float vt = 0.f;
    if (tid < COLS) vt = to_f32(v[(size_t)unit * dv + j0 + tid]);
    if (tid < DK) {
        ks[tid] = to_f32(k[rowk * DK + tid]);
        qs[tid] = to_f32(q[rowk * DK + tid]);
    }
    const float eg = expf(gt);
    __syncthreads();
    if (tid < 32) {
        float lam = 0.f, qk = 0.f;
#pragma unroll
        for (int i = tid; i < DK; i += 32) {
            lam = fmaf(ks[i], ks[i], lam);
            qk = fmaf(qs[i], ks[i], qk);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            lam += __shfl_xor_sync(0xffffffffu, lam, off);
            qk += __shfl_xor_sync(0xffffffffu, qk, off);
        }
        if (tid == 0) {
            scal[0] = efla_alpha(bt, lam, euler);
            scal[1] = qk;
        }
    }
    float px[4] = {}, py[4] = {};
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const float ki = ks[rg + r * RG], qi = qs[rg + r * RG];
        float4 &s = reg[r];
        s = make_float4(eg * s.x, eg * s.y, eg * s.z, eg * s.w);
        const float s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            px[c] = fmaf(ki, s4[c], px[c]);
            py[c] = fmaf(qi, s4[c], py[c]);
        }
    }
    *reinterpret_cast<float4 *>(&red_x[rg][4 * cg]) = make_float4(px[0], px[1], px[2], px[3]);
    *reinterpret_cast<float4 *>(&red_y[rg][4 * cg]) = make_float4(py[0], py[1], py[2], py[3]);
    __syncthreads();
    if (tid < COLS) {
        float x = 0.f, y = 0.f;
#pragma unroll 8
        for (int r = 0; r < RG; ++r) {
            x += red_x[r][tid];
            y += red_y[r][tid];
        }
        const float u = scal[0] * (vt - x);
        us[tid] = u;
        o[(size_t)unit * dv + j0 + tid] = from_f32<TOut>(fmaf(scal[1], u, y));
    }
    __syncthreads();
    const float4 u4 = *reinterpret_cast<const float4 *>(&us[4 * cg]);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const float ki = ks[rg + r * RG];
        const float4 s = reg[r];
        *reinterpret_cast<float4 *>(Su + (size_t)(rg + r * RG) * dv) =
            make_float4(fmaf(ki, u4.x, s.x), fmaf(ki, u4.y, s.y), fmaf(ki, u4.z, s.z), fmaf(ki, u4.w, s.w));
    }
}

template <int DK, int COLS, typename TIn, typename TOut>
cudaError_t step_launch(const GatedDecodeArgs &a) {
    gated_decode_kernel<DK, COLS, TIn, TOut><<<(unsigned)((long)a.B * a.H * (a.dv / COLS)), NT, 0, a.stream>>>(
        static_cast<const TIn *>(a.q), static_cast<const TIn *>(a.k), static_cast<const TIn *>(a.v), a.g, a.beta, a.S,
        static_cast<TOut *>(a.o), a.H, a.H / a.Hk, a.dv, a.euler);
    return cudaGetLastError();
}

template <int DK, int COLS>
cudaError_t step_types(const GatedDecodeArgs &a) {
    const bool ib = a.in_dtype == EFLA_BF16, ob = a.o_dtype == EFLA_BF16;
    if (ib) return ob ? step_launch<DK, COLS, __nv_bfloat16, __nv_bfloat16>(a) : step_launch<DK, COLS, __nv_bfloat16, float>(a);
    return ob ? step_launch<DK, COLS, float, __nv_bfloat16>(a) : step_launch<DK, COLS, float, float>(a);
}

template <int DK>
cudaError_t step_cols(const GatedDecodeArgs &a) {
    if (a.dv == 32 || (long)a.B * a.H < 152) return step_types<DK, 32>(a);  // fewer heads than SMs
    return a.dv == 64 ? step_types<DK, 64>(a) : step_types<DK, 128>(a);
}

}  // namespace

cudaError_t launch_gated_decode_step(const GatedDecodeArgs &a) {
    if (a.B == 0) return cudaSuccess;
    return a.dk == 32 ? step_cols<32>(a) : a.dk == 64 ? step_cols<64>(a) : step_cols<128>(a);
}

}  // namespace efla
