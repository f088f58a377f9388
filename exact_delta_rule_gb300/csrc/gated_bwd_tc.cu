// Backward of the gated delta rule on the sm_103a tensor cores (tcgen05 + TMEM + TMA): bf16, d_k = d_v =
// 128, chunks of 64, rows of [B, T], after the training forward (chunk_tc.cu), which leaves in the
// workspace, as bf16 hi/lo operand tiles, every chunk's start state (S^T, rows = d_v) and
// T = (I + diag(alpha) L)^{-1}.  The formulas are in gated_simt.cu; here they are taken through
//   dY = T^T G,  dR = diag(alpha) dY,  U = T diag(alpha) R,
// which needs no second matrix and gives dalpha without forming Z = R - L U or keeping G:
//   dalpha_t = dY_t . R_t - sum_s L_ts (dY U^T)_ts.
//
// 1. State pass (state_kernel): one CTA per (b, h) walks the chunks in reverse with dS^T fp32 in TMEM,
//    lane j = column j of d_v, everything transposed as in the forward:
//      G^T  = (dS'^T K^T) diag(c) + dO^T P       dY^T = G^T T
//      dS^T = e^{G_C} dS'^T + (dO^T diag(e^G)) Q - (dY^T diag(alpha e^G)) K
//    It writes dS' of every chunk as an operand tile, dv = diag(alpha) dY, and dY as bf16 hi and lo.
//    The serial chain is dS' split -> dS'^T K^T -> G split -> dY -> dY split -> dS and all the state
//    warps do; the prep warps form P and diag(e^G) dO, and, once dS' is split, sum <S, dS'> and scale
//    dS' by e^{G_C} in TMEM, beside the chain.
// 2. Gradient pass (grad_kernel): persistent CTAs over the (b, h, chunk) items, all independent:
//      P0  Gram [K; Q] K^T; L = Gamma o strictly-lower(K K^T) and P kept in registers
//      P2  X^T = S^T K^T;  R^T = V^T - X^T diag(e^G);  U^T = (diag(alpha) R)^T T^T;  dY . R
//      P3  [dY; dO] U^T;  dS' U^T;  [S dY^T | S dO^T] and a from them
//      P4  dalpha, dg, and the operands dP' = Gamma o dP, E = dL' + dL'^T + diag(2 dalpha dalpha/dlambda)
//      P5  dP' K;  dP'^T Q + E K
//      P6  dq = e^G (S dO^T) + dP' K,  dk = -alpha e^G (S dY^T) + c (dS' U^T) + (dP'^T Q + E K)
//    Products with different row factors keep their own accumulators and are joined where they are read
//    out.  The next item's K, Q, S and its first two products are under way while this one ends.  Sums
//    over features or rows are taken by shuffles and per-warp slots in a fixed order.
//    The kernel is bound by the CUDA-core phases between the products and by fetching their code, so
//    those share loops where they can.
//
// dO and the inputs are exact bf16; every other operand is split into two bf16 parts rounded to nearest
// (2^-18), fp32 accumulation.  Every wait is bounded; on expiry the CTA records EFLA_ERR_DEVICE_TIMEOUT
// and leaves.
#include <algorithm>

#include "gated.cuh"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace efla {
namespace {
using namespace ptx;
using namespace tc;

constexpr int C = 64;
constexpr int D = 128;
constexpr uint64_t DRAIN_NS = 2000000000ull;

// x[0..15] as bf16 hi and lo of row `row`, columns col0 .. col0 + 15 (col0 + 15 < 64) of a swizzled
// [.][64] tile (hi at `tile`, lo at tile + lo_off).
__device__ __forceinline__ void put16(uint8_t *tile, uint32_t lo_off, int row, int col0, const float *x) {
    uint32_t hh[8], ll[8];
    split_pack_rn<8>(x, hh, ll);
#pragma unroll
    for (int h8 = 0; h8 < 2; ++h8) {
        const uint32_t off = swz_offset(row, col0 + 8 * h8, 0);
        *reinterpret_cast<uint4 *>(tile + off) = make_uint4(hh[4 * h8], hh[4 * h8 + 1], hh[4 * h8 + 2], hh[4 * h8 + 3]);
        *reinterpret_cast<uint4 *>(tile + lo_off + off) = make_uint4(ll[4 * h8], ll[4 * h8 + 1], ll[4 * h8 + 2], ll[4 * h8 + 3]);
    }
}

// ======================================================================================= state pass
namespace st {

constexpr int NSTAGE = 2;
constexpr uint32_t STAGE_BYTES = 49152;  // [K;Q] [2 cb][128 rows][64] (32 KB), dO [2 cb][64 rows][64] (16 KB)
constexpr uint32_t OFF_DO = 32768;       // within a stage
constexpr uint32_t OFF_TPP = NSTAGE * STAGE_BYTES;  // per chunk parity: T hi, lo, P hi, lo, [64][64] bf16 each
constexpr uint32_t TPP_BYTES = 32768;
constexpr uint32_t OFF_DRS = OFF_TPP + 2 * TPP_BYTES;  // dv, dY hi, dY lo on their way to HBM, [2 cb][64 rows][64] each
constexpr uint32_t OFF_DEC = OFF_DRS + 3 * 16384;      // {G hi, lo} [64], then per parity e^G [64], c [64], alpha [64]
constexpr uint32_t DEC_LD = 192;
constexpr uint32_t OFF_BAR = OFF_DEC + 512 + 2 * DEC_LD * 4;
constexpr uint32_t OFF_MISC = OFF_BAR + 256;
constexpr uint32_t SMEM_ALLOC = OFF_MISC + 16 + 1024;
static_assert(OFF_TPP % 1024 == 0 && OFF_DRS % 1024 == 0 && SMEM_ALLOC <= 232448, "shared memory layout");

constexpr uint32_t TM_S = 0;     // dS^T fp32 (128)
constexpr uint32_t TM_SA = 128;  // dS'^T hi (64) | lo (64)
constexpr uint32_t TM_X = 256;   // dS'^T K^T fp32 (64); then G^T hi (32) | lo (32); then -diag(alpha e^G) dY hi | lo
constexpr uint32_t TM_G = 320;   // Gram rows [K; Q] K^T fp32 (64)
constexpr uint32_t TM_G2 = 384;  // dO^T P fp32 (64); then dY^T
constexpr uint32_t TM_DO = 448;  // diag(e^G) dO hi (32) | lo (32)
constexpr int BAR_PREP = 2, BAR_STATE = 3;

struct Params {
    CUtensorMap map_q, map_k, map_do, map_dv, map_yh, map_yl;  // [B, T, heads, 128] bf16, box 64 x 1 x 64 x 1, 128B swizzle
    const float *gate, *beta, *dST;
    uint8_t *dse;
    const uint8_t *states, *tpp;
    float *dS0, *sdot;
    int *status;
    int T, H, rep;
    int euler, debug_stall;
    unsigned long long wait_ns;
};

struct Bars {
    uint64_t tma_full[NSTAGE], s_free[NSTAGE];
    uint64_t g_done, g_free;
    uint64_t gate_ready[2];  // decays of a chunk written
    uint64_t prep_ready[2];  // P written and T landed
    uint64_t t_full[2], tpp_free[2];
    uint64_t do_ready;       // diag(e^G) dO written (128 arrivals)
    uint64_t sc_ready;       // dS' read from TMEM by the prep warps and scaled (128 arrivals)
    uint64_t x_done, u_done, s_done;
    uint64_t s_prep;         // as s_done, for the prep warps
    uint64_t sa_ready, r_ready, u_ready;
    uint64_t drain, never;
};
static_assert(sizeof(Bars) <= 256, "mbarrier block exceeds its slot");

// Tokens t0, t0 + 1 of column j (this lane) into the staging tiles ([2 column blocks][64 tokens][64],
// 128-byte swizzle; dv, then dY hi and lo 16 KB apart).  Lanes j and j ^ 1 hold neighbouring columns:
// for dv each writes one token's word, for dY the even lane the hi words and the odd lane the lo.
__device__ __forceinline__ void stage_pair(uint8_t *stg, int j, int t0, float y0, float y1, float v0, float v1) {
    const bool odd = (j & 1) != 0;
    const float y[2] = {y0, y1};
    uint32_t hi[1], lo[1];
    split_pack_rn<1>(y, hi, lo);  // tokens t0 (low half), t0 + 1
    const __nv_bfloat162 vv = __floats2bfloat162_rn(v0, v1);
    const uint32_t v = *reinterpret_cast<const uint32_t *>(&vv);
    const uint32_t rv = __shfl_xor_sync(0xffffffffu, v, 1), ry = __shfl_xor_sync(0xffffffffu, odd ? hi[0] : lo[0], 1);
    const uint32_t o0 = swz_offset(t0, j & ~1, 8192), o1 = swz_offset(t0 + 1, j & ~1, 8192);
    *reinterpret_cast<uint32_t *>(stg + (odd ? o1 : o0)) = odd ? __byte_perm(rv, v, 0x7632) : __byte_perm(v, rv, 0x5410);
    uint8_t *d = stg + (odd ? 32768 : 16384);
    const uint32_t a = odd ? ry : hi[0], b = odd ? lo[0] : ry;  // columns j & ~1 and (j & ~1) + 1
    *reinterpret_cast<uint32_t *>(d + o0) = __byte_perm(a, b, 0x5410);
    *reinterpret_cast<uint32_t *>(d + o1) = __byte_perm(a, b, 0x7632);
}

__global__ void __launch_bounds__(320, 1) state_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars *bars = reinterpret_cast<Bars *>(sm + OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + OFF_MISC + 4);
    float *gsum = reinterpret_cast<float *>(sm + OFF_DEC), *dec = gsum + 128;

    const int tid = threadIdx.x, warp = tid >> 5;
    const uint64_t wait_ns = p.wait_ns;
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / p.rep;
    const int nchunks = (p.T + C - 1) / C;  // >= 1
    const size_t ubase = (size_t)blockIdx.x * D * D;
    auto chunk_of = [&](int it) { return nchunks - 1 - it; };  // reverse order

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->tma_full[i], 1);
            mbar_init(&bars->s_free[i], 1);
            mbar_init(&bars->gate_ready[i], 1);
            mbar_init(&bars->prep_ready[i], 1);
            mbar_init(&bars->t_full[i], 1);
            mbar_init(&bars->tpp_free[i], 1);
        }
        mbar_init(&bars->g_done, 1);
        mbar_init(&bars->g_free, 1);
        mbar_init(&bars->do_ready, 128);
        mbar_init(&bars->sc_ready, 128);
        mbar_init(&bars->x_done, 1);
        mbar_init(&bars->u_done, 1);
        mbar_init(&bars->s_done, 1);
        mbar_init(&bars->s_prep, 1);
        mbar_init(&bars->sa_ready, 128);
        mbar_init(&bars->r_ready, 128);
        mbar_init(&bars->u_ready, 128);
        mbar_init(&bars->drain, 1);
        mbar_init(&bars->never, 1);
        fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t s_sm = smem_u32(sm);
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);

    if (tid >= 128 && tid < 256) {
        // =============================== prep warpgroup ===============================
        // Gram row r is TMEM lane r: rows 0-63 (K K^T) give alpha, rows 64-127 (Q K^T) P; warp 4 forms the
        // decays.  For the work on dO and dS' thread = lane = column of d_v.
        const int lane = tid & 31, row = tid - 128;
        const bool leader = tid == 128;
        auto load_g = [&](int it, int odd) {
            const int t = it < nchunks ? chunk_of(it) * C + 2 * lane + odd : p.T;
            return warp == 4 && t < p.T ? p.gate[((size_t)b * p.T + t) * p.H + h] : 0.f;
        };
        auto load_beta = [&](int it) {
            const int t = it < nchunks ? chunk_of(it) * C + row : p.T;
            return row < C && t < p.T ? p.beta[((size_t)b * p.T + t) * p.H + h] : 0.f;
        };
        float g0 = load_g(0, 0), g1 = load_g(0, 1), bt = load_beta(0);
        bool ok = true;
        for (int it = 0; it < nchunks; ++it) {
            const int buf = it & 1, st = it % NSTAGE;
            float *eg = dec + buf * DEC_LD;
            // (chunk it - 2, the last reader of this parity's decays, is complete: s_prep below)
            if (warp == 4) chunk_decay(g0, g1, lane, gsum, gsum + 1, 2, eg, eg + 64);
            const float bcur = bt;
            g0 = load_g(it + 1, 0);
            g1 = load_g(it + 1, 1);
            bt = load_beta(it + 1);
            ok = ok && wait_bar_warp(&bars->g_done, it & 1, abort_flag, wait_ns);
            if (it >= 2) ok = ok && wait_bar_warp(&bars->tpp_free[buf], ((it - 2) >> 1) & 1, abort_flag, wait_ns);
            tc_fence_after();
            float x[2][32];
            if (ok && row >= C) {
                tmem_ld32(lane_base + TM_G, x[0]);
                tmem_ld32(lane_base + TM_G + 32, x[1]);
                tmem_ld_wait();
            } else if (ok) {  // alpha of token `row`: its lambda is the diagonal of K K^T
                float lam = 0.f;
                if (!p.euler) {
                    tmem_ld32(lane_base + TM_G + (row & 32), x[0]);
                    tmem_ld_wait();
#pragma unroll
                    for (int s = 0; s < 32; ++s) lam = s == lane ? x[0][s] : lam;
                }
                eg[128 + row] = efla_alpha(bcur, lam, p.euler);  // (beta is 0 past the end)
            }
            tc_fence_before();
            if (named_bar_any(BAR_PREP, 128, !ok || *abort_flag)) {  // decays visible; also spreads an abort
                *abort_flag = 1;
                break;
            }
            if (leader) {
                mbar_arrive(&bars->g_free);
                mbar_arrive(&bars->gate_ready[buf]);
            }
            if (row >= C) {  // P = Gamma o Q K^T, inclusive lower triangle
                const int t = row - C;
                const float2 gt = reinterpret_cast<const float2 *>(gsum)[t];
                uint8_t *phi = sm + OFF_TPP + buf * TPP_BYTES + 16384;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int c16 = 0; c16 < 32; c16 += 16) {
                        float y[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int s = 32 * hf + c16 + e;
                            const float2 gs = reinterpret_cast<const float2 *>(gsum)[s];
                            y[e] = s <= t ? x[hf][c16 + e] * pair_decay(gt.x, gt.y, gs.x, gs.y) : 0.f;
                        }
                        put16(phi, 8192, t, 32 * hf + c16, y);
                    }
            }
            fence_proxy_async_smem();
            named_bar(BAR_PREP, 128);
            if (leader) {
                ok = wait_bar(&bars->t_full[buf], (it >> 1) & 1, abort_flag, wait_ns);
                mbar_arrive(&bars->prep_ready[buf]);
                if (!ok) *abort_flag = 1;
            }
            ok = __all_sync(0xffffffffu, ok);
            // diag(e^G) dO of this chunk once the previous chunk's state update has read TM_DO
            ok = wait_bar_warp(&bars->tma_full[st], (it / NSTAGE) & 1, abort_flag, wait_ns) && ok;
            if (it > 0) ok = wait_bar_warp(&bars->s_prep, (it - 1) & 1, abort_flag, wait_ns) && ok;
            if (ok) {
                tc_fence_after();
                const uint8_t *src = sm + st * STAGE_BYTES + OFF_DO;
#pragma unroll 1
                for (int hf = 0; hf < 2; hf = opaque(hf + 1)) {
                    float y[32], f[32];
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        y[e] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(src + swz_offset(e, row, 8192) + hf * 4096) << 16);
                    load32(eg + 32 * hf, f);
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] *= f[e];
                    split_pack_rn<16>(y, hi, lo);
                    tmem_st16u(lane_base + TM_DO + 16 * hf, hi);
                    tmem_st16u(lane_base + TM_DO + 32 + 16 * hf, lo);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars->do_ready);
            }
            // <S, dS'> and dS' times e^{G_C} in TM_S (row = column j of d_v), once the state warps have read dS'
            ok = ok && wait_bar_warp(&bars->sa_ready, it & 1, abort_flag, wait_ns);
            if (ok) {
                tc_fence_after();
                const uint8_t *src = p.states + ((size_t)blockIdx.x * nchunks + chunk_of(it)) * 65536 + row * 16;
                const float el = eg[C - 1];
                float2 dot = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int g = 0; g < 4; g = opaque(g + 1)) {
                    uint4 sh[4], sl[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        sh[q] = __ldcg(reinterpret_cast<const uint4 *>(src + g * 8192 + q * 2048));
                        sl[q] = __ldcg(reinterpret_cast<const uint4 *>(src + 32768 + g * 8192 + q * 2048));
                    }
                    float sv[32];
                    tmem_ld32(lane_base + TM_S + g * 32, sv);
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t wh[4] = {sh[q].x, sh[q].y, sh[q].z, sh[q].w}, wl[4] = {sl[q].x, sl[q].y, sl[q].z, sl[q].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 xx = make_float2(sv[8 * q + 2 * e], sv[8 * q + 2 * e + 1]);
                            dot = __ffma2_rn(make_float2(__uint_as_float(wh[e] << 16), __uint_as_float(wh[e] & 0xffff0000u)), xx, dot);
                            dot = __ffma2_rn(make_float2(__uint_as_float(wl[e] << 16), __uint_as_float(wl[e] & 0xffff0000u)), xx, dot);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) sv[i] *= el;
                    tmem_st32(lane_base + TM_S + g * 32, sv);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars->sc_ready);
                float d = dot.x + dot.y;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
                if (lane == 0) p.sdot[((size_t)blockIdx.x * nchunks + chunk_of(it)) * 4 + (warp & 3)] = d;
            }
        }
    } else if (tid < 128) {
        // =============================== state warpgroup ===============================
        const int j = tid;
        {  // dS_T -> TMEM (dS^T: lane j holds column j)
            float r[32];
#pragma unroll 1
            for (int g = 0; g < 4; g = opaque(g + 1)) {
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = p.dST ? p.dST[ubase + (size_t)(g * 32 + i) * D + j] : 0.f;
                tmem_st32(lane_base + TM_S + g * 32, r);
            }
            tmem_st_wait();
        }
        bool ok = true;
        uint8_t *stg = sm + OFF_DRS;
        // A failed wait skips the work up to the chunk's consensus barrier, which every thread of the
        // warpgroup reaches, so that the warpgroup leaves together.
        for (int it = 0; it < nchunks; ++it) {
            if (it > 0) ok = wait_bar_warp(&bars->s_done, (it - 1) & 1, abort_flag, wait_ns);
            const int c = chunk_of(it);
            const float *eg = dec + (it & 1) * DEC_LD, *ec = eg + 64, *al = eg + 128;
            if (ok) {
                tc_fence_after();
                uint8_t *dse = p.dse + ((size_t)blockIdx.x * nchunks + c) * 65536;
#pragma unroll 1
                for (int g = 0; g < 4; g = opaque(g + 1)) {  // dS'^T -> bf16 hi/lo operand, and to HBM as a tile
                    float sv[32];
                    uint32_t hi[16], lo[16];
                    tmem_ld32(lane_base + TM_S + g * 32, sv);
                    tmem_ld_wait();
                    split_pack_rn<16>(sv, hi, lo);
                    tmem_st16u(lane_base + TM_SA + g * 16, hi);
                    tmem_st16u(lane_base + TM_SA + 64 + g * 16, lo);
                    put_state_row(dse, g, j, hi, lo);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars->sa_ready);
                ok = wait_bar_warp(&bars->gate_ready[it & 1], (it >> 1) & 1, abort_flag, wait_ns);
                ok = ok && wait_bar_warp(&bars->x_done, it & 1, abort_flag, wait_ns);
            }
            if (ok) {  // G^T = (dS'^T K^T) diag(c) + dO^T P; its split overwrites TM_X once all of it is in registers
                tc_fence_after();
                uint32_t hi[16], lo[16];
                float x[64], f[32];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float(&xa)[32] = *reinterpret_cast<float(*)[32]>(x + 32 * hf);
                    float y[32];
                    tmem_ld32(lane_base + TM_X + 32 * hf, xa);
                    tmem_ld32(lane_base + TM_G2 + 32 * hf, y);
                    load32(ec + 32 * hf, f);
                    tmem_ld_wait();
#pragma unroll
                    for (int t = 0; t < 32; ++t) xa[t] = fmaf(f[t], xa[t], y[t]);
                }
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    split_pack_rn<16>(x + 32 * hf, hi, lo);
                    tmem_st16u(lane_base + TM_X + 16 * hf, hi);
                    tmem_st16u(lane_base + TM_X + 32 + 16 * hf, lo);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars->r_ready);
                ok = wait_bar_warp(&bars->u_done, it & 1, abort_flag, wait_ns);
            }
            if (ok) {  // -diag(alpha e^G) dY -> operand
                tc_fence_after();
#pragma unroll 1
                for (int hf = 0; hf < 2; hf = opaque(hf + 1)) {
                    uint32_t hi[16], lo[16];
                    float x[32], f[32], f2[32];
                    tmem_ld32(lane_base + TM_G2 + 32 * hf, x);
                    load32(eg + 32 * hf, f);
                    load32(al + 32 * hf, f2);
                    tmem_ld_wait();
#pragma unroll
                    for (int t = 0; t < 32; ++t) f[t] *= -f2[t] * x[t];
                    split_pack_rn<16>(f, hi, lo);
                    tmem_st16u(lane_base + TM_X + 16 * hf, hi);
                    tmem_st16u(lane_base + TM_X + 32 + 16 * hf, lo);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars->u_ready);
            }
            // dv and dY, staged and stored by TMA (rows past the end are clipped) once the previous chunk's stores
            // have read the staging; TM_G2 is written again only after the next chunk's sa_ready
            if (tid == 0) bulk_wait_read0();
            if (named_bar_any(BAR_STATE, 128, !ok)) {
                ok = false;
                break;
            }
#pragma unroll 1
            for (int q = 0; q < 4; q = opaque(q + 1)) {
                float x[16];
                tmem_ld16(lane_base + TM_G2 + 16 * q, x);
                tmem_ld_wait();
                uint8_t *dst = stg + q * 2048;  // 16 tokens are two groups of 8 rows
#pragma unroll
                for (int t = 0; t < 16; t += 2)
                    stage_pair(dst, j, t, x[t], x[t + 1], al[16 * q + t] * x[t], al[16 * q + t + 1] * x[t + 1]);
            }
            fence_proxy_async_smem();
            named_bar(BAR_STATE, 128);
            if (tid == 0) {
                for (int cb = 0; cb < 2; ++cb) {
                    tma_store_4d(&p.map_dv, stg + cb * 8192, cb * 64, h, c * C, b);
                    tma_store_4d(&p.map_yh, stg + 16384 + cb * 8192, cb * 64, h, c * C, b);
                    tma_store_4d(&p.map_yl, stg + 32768 + cb * 8192, cb * 64, h, c * C, b);
                }
                bulk_commit();
            }
        }
        if (ok) {
            ok = wait_bar_warp(&bars->s_done, (nchunks - 1) & 1, abort_flag, wait_ns);
            if (ok && p.dS0) {
                tc_fence_after();
#pragma unroll 1
                for (int g = 0; g < 4; g = opaque(g + 1)) {
                    float sv[32];
                    tmem_ld32(lane_base + TM_S + g * 32, sv);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) p.dS0[ubase + (size_t)(g * 32 + i) * D + j] = sv[i];
                }
            }
        }
        if (tid == 0) bulk_wait0();  // the stores have completed before the CTA leaves
        if (!ok) *abort_flag = 1;
    } else if (tid == 288) {
        // ============================ TMA producer (one thread) ============================
        prefetch_tensormap(&p.map_q);
        prefetch_tensormap(&p.map_k);
        prefetch_tensormap(&p.map_do);
        int issued = 0, t_issued = 0;
        for (int it = 0; it < nchunks; ++it) {
            const int st = it % NSTAGE, buf = it & 1;
            if (it >= 2 && !wait_bar(&bars->tpp_free[buf], ((it - 2) >> 1) & 1, abort_flag, wait_ns)) break;
            mbar_arrive_expect_tx(&bars->t_full[buf], 16384);
            bulk_load(sm + OFF_TPP + buf * TPP_BYTES, p.tpp + ((size_t)blockIdx.x * nchunks + chunk_of(it)) * 16384, 16384,
                      &bars->t_full[buf]);
            t_issued = it + 1;
            if (it >= NSTAGE && !wait_bar(&bars->s_free[st], ((it - NSTAGE) / NSTAGE) & 1, abort_flag, wait_ns)) break;
            uint8_t *dst = sm + st * STAGE_BYTES;
            const int tok = chunk_of(it) * C;
            mbar_arrive_expect_tx(&bars->tma_full[st], STAGE_BYTES);
            for (int cb = 0; cb < 2; ++cb) {
                tma_load_4d(dst + cb * 16384, &p.map_k, &bars->tma_full[st], cb * 64, hk, tok, b);
                tma_load_4d(dst + cb * 16384 + 8192, &p.map_q, &bars->tma_full[st], cb * 64, hk, tok, b);
                tma_load_4d(dst + OFF_DO + cb * 8192, &p.map_do, &bars->tma_full[st], cb * 64, h, tok, b);
            }
            issued = it + 1;
        }
        // the last loads have landed before the CTA can leave (bounded; matters after an abort)
        for (int cc = max(0, issued - NSTAGE); cc < issued; ++cc) {
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait_sleep(&bars->tma_full[cc % NSTAGE], (cc / NSTAGE) & 1, 20000) && globaltimer_ns() - t0 < DRAIN_NS) {
            }
        }
        for (int cc = max(0, t_issued - 2); cc < t_issued; ++cc) {
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait_sleep(&bars->t_full[cc & 1], (cc >> 1) & 1, 20000) && globaltimer_ns() - t0 < DRAIN_NS) {
            }
        }
    } else if (warp == 8) {
        // =============================== MMA warp ===============================
        bool ok = true;
        int g_next = 0;
        // Gram rows of chunks up to `limit`, each once the prep has read the previous one and its stage has
        // landed; with `block` false only what is ready now
        auto issue_grams = [&](int limit, bool block) {
            while (ok && g_next <= limit && g_next < nchunks) {
                if (!block) {
                    const bool ready = (g_next == 0 || mbar_test(&bars->g_free, (g_next - 1) & 1)) &&
                                       mbar_test(&bars->tma_full[g_next % NSTAGE], (g_next / NSTAGE) & 1);
                    if (!__all_sync(0xffffffffu, ready)) break;
                } else {
                    if (g_next > 0 && !(ok = wait_bar_warp(&bars->g_free, (g_next - 1) & 1, abort_flag, wait_ns))) break;
                    if (!(ok = wait_bar_warp(&bars->tma_full[g_next % NSTAGE], (g_next / NSTAGE) & 1, abort_flag, wait_ns))) break;
                }
                tc_fence_after();
                const uint32_t kq = s_sm + (g_next % NSTAGE) * STAGE_BYTES;
                const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 0);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
                    mma_bf16_e(tmem + TM_G, smem_desc(kq + off, 16, 1024), smem_desc(kq + off, 16, 1024), idesc, ks > 0);
                }
                mma_commit_e(&bars->g_done);
                ++g_next;
            }
        };
        if (p.debug_stall) ok = wait_bar_warp(&bars->never, 0, abort_flag, wait_ns);
        issue_grams(0, true);
        for (int it = 0; it < nchunks && ok; ++it) {
            const int st = it % NSTAGE, buf = it & 1;
            const uint32_t kq_s = s_sm + st * STAGE_BYTES, dO_s = kq_s + OFF_DO;
            const uint32_t tp = s_sm + OFF_TPP + buf * TPP_BYTES, pb = tp + 16384;
            if (!(ok = wait_bar_warp(&bars->tma_full[st], (it / NSTAGE) & 1, abort_flag, wait_ns))) break;
            if (!(ok = wait_bar_warp(&bars->sa_ready, it & 1, abort_flag, wait_ns))) break;
            tc_fence_after();
            {  // dS'^T K^T (the chain)
                const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 0);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
                        mma_bf16_ts_e(tmem + TM_X, tmem + TM_SA + part * 64 + ks * 8, smem_desc(kq_s + off, 16, 1024), idesc,
                                      (part | ks) != 0);
                    }
            }
            issue_grams(it + 1, false);
            if (!(ok = wait_bar_warp(&bars->prep_ready[buf], (it >> 1) & 1, abort_flag, wait_ns))) break;
            tc_fence_after();
            issue_grams(it + 1, false);
            {  // dO^T P: dO^T (M = j) and P (N = t) read as MN-major operands, K = s
                const uint32_t idesc = idesc_bf16_f32(128, 64, 1, 1);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t ad = smem_desc(dO_s + ks * 2048, 8192, 1024);
                    mma_bf16_e(tmem + TM_G2, ad, smem_desc(pb + ks * 2048, 8192, 1024), idesc, ks > 0);
                    mma_bf16_e(tmem + TM_G2, ad, smem_desc(pb + 8192 + ks * 2048, 8192, 1024), idesc, 1);
                }
                mma_commit_e(&bars->x_done);
            }
            if (!(ok = wait_bar_warp(&bars->r_ready, it & 1, abort_flag, wait_ns))) break;
            tc_fence_after();
            {  // dY^T = G^T T (T read as an MN-major operand, K = s), over dO^T P, which the state warps have read
                const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 1);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t th = smem_desc(tp + ks * 2048, 8192, 1024), tl = smem_desc(tp + 8192 + ks * 2048, 8192, 1024);
                    mma_bf16_ts_e(tmem + TM_G2, tmem + TM_X + ks * 8, th, idesc, ks > 0);
                    mma_bf16_ts_e(tmem + TM_G2, tmem + TM_X + ks * 8, tl, idesc, 1);
                    mma_bf16_ts_e(tmem + TM_G2, tmem + TM_X + 32 + ks * 8, th, idesc, 1);
                }
                mma_commit_e(&bars->u_done);
                mma_commit_e(&bars->tpp_free[buf]);
            }
            if (!(ok = wait_bar_warp(&bars->do_ready, it & 1, abort_flag, wait_ns))) break;
            if (!(ok = wait_bar_warp(&bars->sc_ready, it & 1, abort_flag, wait_ns))) break;
            tc_fence_after();
            {  // dS^T += (diag(e^G) dO)^T Q, behind dY in the pipe
                const uint32_t idesc = idesc_bf16_f32(128, 128, 0, 1);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16_ts_e(tmem + TM_S, tmem + TM_DO + part * 32 + ks * 8,
                                      smem_desc(kq_s + 8192 + ks * 2048, 16384, 1024), idesc, 1);
            }
            issue_grams(it + 2, false);
            if (!(ok = wait_bar_warp(&bars->u_ready, it & 1, abort_flag, wait_ns))) break;
            tc_fence_after();
            {  // dS^T += (-diag(alpha e^G) dY)^T K (the chain)
                const uint32_t idesc = idesc_bf16_f32(128, 128, 0, 1);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16_ts_e(tmem + TM_S, tmem + TM_X + part * 32 + ks * 8,
                                      smem_desc(kq_s + ks * 2048, 16384, 1024), idesc, 1);
                mma_commit_e(&bars->s_done);
                mma_commit_e(&bars->s_prep);
                mma_commit_e(&bars->s_free[st]);
            }
            issue_grams(it + 1, true);  // (the next chunk's, if it was not ready above)
        }
        if (!ok) *abort_flag = 1;
        mma_commit_e(&bars->drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait_sleep(&bars->drain, 0, 20000) && globaltimer_ns() - t0 < DRAIN_NS) {
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag && tid == 0) atomicExch(p.status, (int)EFLA_ERR_DEVICE_TIMEOUT);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace st

// ======================================================================================= gradient pass
namespace gr {

constexpr int NW = 256;       // CUDA-core threads (warps 0-7)
constexpr int NTH = NW + 32;  // and the MMA / TMA warp
constexpr int BAR_W = 1;

// Shared memory (bytes).  No room is left for alignment slack: the array is declared 1024-byte aligned
// and the kernel refuses to run on another base.
constexpr uint32_t OFF_KQ = 0;         // two items' [K; Q]: 2 column blocks x 128 rows, 32 KB each
constexpr uint32_t OFF_ROD = 65536;    // [dY hi; dO]: 2 column blocks x 128 rows, 32 KB
constexpr uint32_t OFF_YL = 98304;     // dY lo: 2 column blocks x 64 rows, 16 KB
constexpr uint32_t OFF_SS = 114688;    // S^T, later dS'^T, hi | lo (put_state_row's layout), 64 KB
constexpr uint32_t OFF_W = 180224;     // T hi | lo [64][64]; later dP' hi | lo
constexpr uint32_t OFF_UT = 196608;    // U^T hi | lo [128][64], 32 KB; V before it in the second half, E hi | lo
                                       // after it in the first; then dq and dk on their way out
constexpr uint32_t OFF_ROW = 229376;   // fp32 rows, struct RowData
constexpr uint32_t LO_128 = 32768, LO_UT = 16384, LO_64 = 8192;
constexpr uint32_t OFF_V = OFF_UT + 16384;  // V: 2 column blocks x 64 rows
// scratch over [dY hi; dO] once its products are complete: dL' [64][65], then sums
constexpr int DL_LD = 65;
constexpr uint32_t OFF_DL = OFF_ROD;
constexpr uint32_t OFF_PART = OFF_ROD + 64 * DL_LD * 4;  // fp32 [4 sums][8 warps][32], row sums [2 halves][128]
static_assert(64 * DL_LD * 4 + 4 * 8 * 32 * 4 + 256 * 4 <= 32768 && OFF_PART % 16 == 0, "scratch leaves its region");

struct RowData {
    float2 g[C];              // G_t hi, lo
    float eg[C], ec[C];
    float al[C], dadb[C], dadl[C];
};
constexpr uint32_t OFF_BAR = OFF_ROW + sizeof(RowData);
constexpr uint32_t OFF_MISC = OFF_BAR + 256;
constexpr uint32_t SMEM_ALLOC = OFF_MISC + 16;
static_assert(OFF_BAR % 16 == 0 && SMEM_ALLOC <= 232448, "shared memory layout");

// TMEM columns (fp32, 64 each, unless split: hi in the first 32 columns, lo in the next 32)
constexpr uint32_t TM_P = 0;     // [dY hi; dO] U^T; then (dP' K)^T
constexpr uint32_t TM_D2 = 64;   // (dS' U^T) as [feature][token]
constexpr uint32_t TM_E = 128;   // (dP'^T Q + E K)^T
constexpr uint32_t TM_RS = 192;  // (diag(alpha) R)^T split; then dY lo U^T (lanes 0-63)
constexpr uint32_t TM_U = 256;   // Gram -> U^T
constexpr uint32_t TM_X = 320;   // X^T
constexpr uint32_t TM_DK = 384;  // S dY^T, adjacent to
constexpr uint32_t TM_DQ = 448;  // S dO^T: one N = 128 product fills both

struct Params {
    CUtensorMap map_q, map_k, map_v, map_do, map_yh, map_yl, map_dq, map_dk;
    const float *gate, *beta, *sdot;
    const uint8_t *states, *dse, *tpp;
    float *part;                   // [2][B, T, H, 128] in place of dq, dk where key heads are shared
    float *dbeta, *dg;
    size_t plane;                  // elements of one part
    int *status;
    int T, H, rep, items;
    int euler, debug_stall;
    unsigned long long wait_ns;
};

struct Bars {
    uint64_t tma_kq[2], tma_rod, s_full, d_full, t_full, v_full;
    uint64_t g, m1a, m1b, u, b, d2, m2;       // products complete
    uint64_t w_u, w_p3, w_p5, w_free, w_out;  // operands written / accumulators read / outputs staged (8 arrivals)
    uint64_t drain, never;
};
static_assert(sizeof(Bars) <= 256, "mbarrier block exceeds its slot");

// Sum over the 32 lanes of a warp of x[0..31]: lane l returns the sum of x[l].
__device__ __forceinline__ float lane_reduce_scatter(float (&x)[32], int lane) {
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) {
        const bool up = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float send = up ? x[i] : x[i + w];
            const float keep = up ? x[i + w] : x[i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
        }
    }
    return x[0];
}

struct Item {
    int b, h, hk, t0, valid;
    size_t row0;
};
__device__ __forceinline__ Item item_of(const Params &p, int w, int nc) {
    Item it;
    const int unit = w / nc, c = w - unit * nc;
    it.b = unit / p.H;
    it.h = unit - it.b * p.H;
    it.hk = it.h / p.rep;
    it.t0 = c * C;
    it.valid = min(C, p.T - it.t0);
    it.row0 = ((size_t)it.b * p.T + (size_t)it.t0) * p.H + it.h;
    return it;
}

__device__ __forceinline__ float bf16_at(const uint8_t *p) { return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(p) << 16); }

__global__ void __launch_bounds__(NTH, 1) grad_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = smem_raw;
    if (smem_u32(sm) & 1023u) {  // (the operand layout needs the base aligned)
        if (threadIdx.x == 0) atomicExch(p.status, (int)EFLA_ERR_CUDA);
        return;
    }
    Bars *bars = reinterpret_cast<Bars *>(sm + OFF_BAR);
    RowData &R = *reinterpret_cast<RowData *>(sm + OFF_ROW);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + OFF_MISC + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nc = (p.T + C - 1) / C;
    const uint64_t wait_ns = p.wait_ns;
    const uint32_t s_sm = smem_u32(sm);

    if (tid == 0) {
        uint64_t *one[] = {&bars->tma_kq[0], &bars->tma_kq[1], &bars->tma_rod, &bars->s_full, &bars->d_full, &bars->t_full,
                           &bars->v_full, &bars->g, &bars->m1a, &bars->m1b, &bars->u, &bars->b, &bars->d2, &bars->m2,
                           &bars->drain, &bars->never};
        for (uint64_t *x : one) mbar_init(x, 1);
        uint64_t *eight[] = {&bars->w_u, &bars->w_p3, &bars->w_p5, &bars->w_free, &bars->w_out};
        for (uint64_t *x : eight) mbar_init(x, 8);
        fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 8) {
        // ============================ MMA / TMA warp ============================
        const bool leader = lane == 0;
        const uint32_t rod = s_sm + OFF_ROD, yl = s_sm + OFF_YL, ss = s_sm + OFF_SS, wt = s_sm + OFF_W, ut = s_sm + OFF_UT;
        if (leader) {
            const CUtensorMap *maps[] = {&p.map_q, &p.map_k, &p.map_v, &p.map_do, &p.map_yh, &p.map_yl};
            for (const CUtensorMap *m : maps) prefetch_tensormap(m);
        }
        bool ok = true;
        // the parity of each kind of load that may still be in flight (-1: none), for the drain at the end
        int kq_pending[2] = {-1, -1}, rod_pending = -1, s_pending = -1, d_pending = -1, t_pending = -1, v_pending = -1;
        auto wait = [&](uint64_t *bar, int parity) {
            ok = ok && wait_bar_warp(bar, parity, abort_flag, wait_ns);
            tc_fence_after();
            return ok;
        };
        auto load_tile = [&](uint64_t *bar, uint32_t off, const uint8_t *src, uint32_t bytes) {
            if (leader) {
                mbar_arrive_expect_tx(bar, bytes);
                bulk_load(sm + off, src, bytes, bar);
            }
            __syncwarp();
        };
        // loads of the n-th item of this CTA (work item w)
        auto load_kq = [&](int w, int n) {
            if (leader) {
                const Item I = item_of(p, w, nc);
                uint64_t *bar = &bars->tma_kq[n & 1];
                mbar_arrive_expect_tx(bar, 2 * 16384);
                for (int cb = 0; cb < 2; ++cb) {
                    uint8_t *dst = sm + OFF_KQ + (n & 1) * 32768 + cb * 16384;
                    tma_load_4d(dst, &p.map_k, bar, cb * 64, I.hk, I.t0, I.b);
                    tma_load_4d(dst + 8192, &p.map_q, bar, cb * 64, I.hk, I.t0, I.b);
                }
            }
            kq_pending[n & 1] = (n >> 1) & 1;
            __syncwarp();
        };
        auto load_s = [&](int w, int n) {
            load_tile(&bars->s_full, OFF_SS, p.states + (size_t)w * 65536, 65536);
            s_pending = n & 1;
        };
        auto load_t_rod = [&](int w, int n) {
            load_tile(&bars->t_full, OFF_W, p.tpp + (size_t)w * 16384, 16384);
            t_pending = n & 1;
            if (leader) {
                const Item I = item_of(p, w, nc);
                mbar_arrive_expect_tx(&bars->tma_rod, 6 * 8192);
                for (int cb = 0; cb < 2; ++cb) {
                    tma_load_4d(sm + OFF_ROD + cb * 16384, &p.map_yh, &bars->tma_rod, cb * 64, I.h, I.t0, I.b);
                    tma_load_4d(sm + OFF_ROD + cb * 16384 + 8192, &p.map_do, &bars->tma_rod, cb * 64, I.h, I.t0, I.b);
                    tma_load_4d(sm + OFF_YL + cb * 8192, &p.map_yl, &bars->tma_rod, cb * 64, I.h, I.t0, I.b);
                }
            }
            rod_pending = n & 1;
            __syncwarp();
        };
        auto load_v = [&](int w, int n) {
            if (leader) {
                const Item I = item_of(p, w, nc);
                mbar_arrive_expect_tx(&bars->v_full, 2 * 8192);
                for (int cb = 0; cb < 2; ++cb)
                    tma_load_4d(sm + OFF_V + cb * 8192, &p.map_v, &bars->v_full, cb * 64, I.h, I.t0, I.b);
            }
            v_pending = n & 1;
            __syncwarp();
        };
        // Gram [K; Q] K^T of item n into TM_U, X^T = S^T K^T (tile rows = d_v: a K-major A) into TM_X
        auto issue_gram = [&](int n) {
            if (!wait(&bars->tma_kq[n & 1], (n >> 1) & 1)) return;
            kq_pending[n & 1] = -1;
            if (leader) {
                const uint32_t kq = s_sm + OFF_KQ + (n & 1) * 32768;
                const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 0);
#pragma unroll 1
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
                    mma_bf16(tmem + TM_U, smem_desc(kq + off, 16, 1024), smem_desc(kq + off, 16, 1024), idesc, ks > 0);
                }
                mma_commit(&bars->g);
            }
            __syncwarp();
        };
        auto issue_x = [&](int n) {
            if (!wait(&bars->s_full, n & 1)) return;
            s_pending = -1;
            if (leader) {
                const uint32_t kq = s_sm + OFF_KQ + (n & 1) * 32768;
                const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 0);
#pragma unroll 1
                for (int i = 0; i < 16; ++i) {
                    const uint32_t off = ((i & 7) >> 2) * 16384 + (i & 3) * 32;
                    mma_bf16(tmem + TM_X, smem_desc_plain(ss + (i >> 3) * LO_128 + (i & 7) * 4096, 2048, 128),
                             smem_desc(kq + off, 16, 1024), idesc, i > 0);
                }
                mma_commit(&bars->m1a);
            }
            __syncwarp();
        };
        if (p.debug_stall) ok = wait_bar_warp(&bars->never, 0, abort_flag, wait_ns);
        if (ok) {  // (the grid has no CTA without an item)
            load_kq(blockIdx.x, 0);
            load_s(blockIdx.x, 0);
            load_v(blockIdx.x, 0);
            load_t_rod(blockIdx.x, 0);
            issue_gram(0);
            if (ok) issue_x(0);
        }
        int n = 0;
        for (int w = blockIdx.x; w < p.items && ok; w += gridDim.x, ++n) {
            const int ph = n & 1, w1 = w + (int)gridDim.x;
            const bool more = w1 < p.items;
            const uint32_t kq = s_sm + OFF_KQ + ph * 32768;
            if (more) load_kq(w1, n + 1);  // (that buffer's last products, item n - 1's, are complete)
            if (!wait(&bars->tma_rod, ph)) break;
            rod_pending = -1;
            if (n > 0 && !wait(&bars->w_free, ph ^ 1)) break;  // the previous item's results are read out
            if (leader) {  // [S dY^T | S dO^T]: S read from the S^T tile as an MN-major A, K = j; dY lo only against S hi
                const uint32_t id128 = idesc_bf16_f32(128, 128, 1, 0), id64 = idesc_bf16_f32(128, 64, 1, 0);
#pragma unroll 1
                for (int i = 0; i < 16; ++i) {
                    const uint32_t boff = ((i & 7) >> 2) * 16384 + (i & 3) * 32;
                    mma_bf16(tmem + TM_DK, smem_desc_plain(ss + (i >> 3) * LO_128 + (i & 7) * 256, 128, 2048),
                             smem_desc(rod + boff, 16, 1024), id128, i > 0);
                }
#pragma unroll 1
                for (int ks = 0; ks < 8; ++ks)
                    mma_bf16(tmem + TM_DK, smem_desc_plain(ss + ks * 256, 128, 2048),
                             smem_desc(yl + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024), id64, 1);
                mma_commit(&bars->m1b);
            }
            __syncwarp();
            if (!wait(&bars->m1b, ph)) break;  // S is read: dS' replaces it
            load_tile(&bars->d_full, OFF_SS, p.dse + (size_t)w * 65536, 65536);
            d_pending = ph;
            if (!wait(&bars->t_full, ph)) break;
            t_pending = -1;
            if (!wait(&bars->w_u, ph)) break;  // V read, (diag(alpha) R)^T written
            v_pending = -1;
            if (leader) {  // U^T = (diag(alpha) R)^T T^T
                const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 0);
#pragma unroll 1
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t bh = smem_desc(wt + ks * 32, 16, 1024), bl = smem_desc(wt + LO_64 + ks * 32, 16, 1024);
                    mma_bf16_ts(tmem + TM_U, tmem + TM_RS + ks * 8, bh, idesc, ks > 0);
                    mma_bf16_ts(tmem + TM_U, tmem + TM_RS + ks * 8, bl, idesc, 1);
                    mma_bf16_ts(tmem + TM_U, tmem + TM_RS + 32 + ks * 8, bh, idesc, 1);
                }
                mma_commit(&bars->u);
            }
            __syncwarp();
            if (!wait(&bars->w_p3, ph)) break;  // U^T tile written
            if (leader) {  // [dY hi; dO] U^T and (into TM_RS, rows 0-63 meant) dY lo U^T: B[t][j] = U^T[j][t] (MN-major)
                const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 1);
#pragma unroll 1
                for (int i = 0; i < 16; ++i) {
                    const uint32_t aoff = ((i & 7) >> 2) * 16384 + (i & 3) * 32;
                    mma_bf16(tmem + TM_P, smem_desc(rod + aoff, 16, 1024),
                             smem_desc(ut + (i >> 3) * LO_UT + (i & 7) * 2048, 8192, 1024), idesc, i > 0);
                }
#pragma unroll 1
                for (int ks = 0; ks < 8; ++ks)
                    mma_bf16(tmem + TM_RS, smem_desc(yl + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024),
                             smem_desc(ut + ks * 2048, 8192, 1024), idesc, ks > 0);
                mma_commit(&bars->b);
            }
            __syncwarp();
            if (!wait(&bars->d_full, ph)) break;
            d_pending = -1;
            if (leader) {  // dS' U^T: dS' read from the dS'^T tile as an MN-major A
                const uint32_t idesc = idesc_bf16_f32(128, 64, 1, 1);
#pragma unroll 1
                for (int i = 0; i < 24; ++i) {
                    const int pr = i >> 3, ks = i & 7;  // hi x hi, hi x lo, lo x hi
                    mma_bf16(tmem + TM_D2, smem_desc_plain(ss + (pr == 2 ? LO_128 : 0) + ks * 256, 128, 2048),
                             smem_desc(ut + (pr == 1 ? LO_UT : 0) + ks * 2048, 8192, 1024), idesc, i > 0);
                }
                mma_commit(&bars->d2);
            }
            __syncwarp();
            if (more) issue_gram(n + 1);
            if (!ok || !wait(&bars->d2, ph)) break;
            if (more) load_s(w1, n + 1);
            if (!wait(&bars->w_p5, ph)) break;  // dP' and E written, the accumulators below read
            if (leader) {  // (dP' K)^T = K^T dP'^T;  (dP'^T Q + E K)^T = Q^T dP' + K^T E
                const uint32_t id_kn = idesc_bf16_f32(128, 64, 1, 0), id_mn = idesc_bf16_f32(128, 64, 1, 1);
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    const int ks = i & 3;
                    const uint32_t lo = (i >> 2) * LO_64;
                    const uint64_t kt = smem_desc(kq + ks * 2048, 16384, 1024);         // K^T (M = i, K = s)
                    const uint64_t qt = smem_desc(kq + 8192 + ks * 2048, 16384, 1024);  // Q^T
                    mma_bf16(tmem + TM_P, kt, smem_desc(wt + lo + ks * 32, 16, 1024), id_kn, i > 0);      // dP'[t][s]
                    mma_bf16(tmem + TM_E, qt, smem_desc(wt + lo + ks * 2048, 8192, 1024), id_mn, i > 0);  // dP'[s][t]
                    mma_bf16(tmem + TM_E, kt, smem_desc(ut + lo + ks * 32, 16, 1024), id_kn, 1);          // E[t][s]
                }
                mma_commit(&bars->m2);
            }
            __syncwarp();
            if (more) issue_x(n + 1);
            if (!ok || !wait(&bars->m2, ph)) break;
            if (more) load_t_rod(w1, n + 1);
            if (!wait(&bars->w_out, ph)) break;  // dq and dk staged (or written)
            if (leader && !p.part) {
                const Item I = item_of(p, w, nc);
                for (int cb = 0; cb < 2; ++cb) {  // (rows past the sequence end are clipped)
                    tma_store_4d(&p.map_dq, sm + OFF_UT + cb * 8192, cb * 64, I.h, I.t0, I.b);
                    tma_store_4d(&p.map_dk, sm + OFF_UT + 16384 + cb * 8192, cb * 64, I.h, I.t0, I.b);
                }
                bulk_commit();
                bulk_wait_read0();
            }
            __syncwarp();
            if (more) load_v(w1, n + 1);
        }
        if (!ok) *abort_flag = 1;
        if (leader) {  // every product, load and store issued has completed before TMEM and the CTA go (bounded)
            mma_commit(&bars->drain);
            const uint64_t ts = globaltimer_ns();
            auto settle = [&](uint64_t *bar, int parity) {
                while (parity >= 0 && !mbar_try_wait_sleep(bar, parity, 20000) && globaltimer_ns() - ts < DRAIN_NS) {
                }
            };
            settle(&bars->drain, 0);
            settle(&bars->tma_kq[0], kq_pending[0]);
            settle(&bars->tma_kq[1], kq_pending[1]);
            settle(&bars->tma_rod, rod_pending);
            settle(&bars->s_full, s_pending);
            settle(&bars->d_full, d_pending);
            settle(&bars->t_full, t_pending);
            settle(&bars->v_full, v_pending);
            bulk_wait0();
        }
        __syncwarp();
    } else {
        // ============================ CUDA-core warps ============================
        float *dLs = reinterpret_cast<float *>(sm + OFF_DL);
        float *part = reinterpret_cast<float *>(sm + OFF_PART);  // sums {dY . R, a, w, M's columns} [8 warps][32]
        float *rsum = part + 4 * 8 * 32;                         // [2][128] row sums of M (rows >= 64) and of L o dY U^T
        // TMEM: this thread reads and writes lane `ln`, the columns of token half `hf`
        const int hf = warp >> 2, ln = (warp & 3) * 32 + lane, col0 = 32 * hf;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const bool gate_thr = ln < C && (ln >> 5) == hf;  // holds K K^T[t][t] for t = ln
        const int tr = ln & (C - 1);                      // the row of this thread in the C x C matrices
        // element (token col0 + e, feature ln) of a [tokens][128] tile whose column blocks are `cb` bytes apart
        auto feat = [&](int e, uint32_t cb) { return (uint32_t)(ln >> 6) * cb + hf * 4096u + swz_offset(e, ln & 63, 0); };
        bool ok = true;
        int it = 0;
        auto wait = [&](uint64_t *bar, int parity) {
            ok = ok && wait_bar_warp(bar, parity, abort_flag, wait_ns);
            tc_fence_after();
        };
        auto arrive = [&](uint64_t *bar) {  // one arrival per warp, what it wrote or read before ordered first
            tmem_st_wait();
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        // gates and step sizes are loaded an item ahead: warp 7 the gates of tokens 2 l, 2 l + 1
        float g0 = 0.f, g1 = 0.f, bt = 0.f;
        auto load_gates = [&](int w) {
            if (w >= p.items) return;
            const Item I = item_of(p, w, nc);
            const int t = 2 * lane;
            if (warp == 7) {
                g0 = t < I.valid ? p.gate[I.row0 + (size_t)t * p.H] : 0.f;
                g1 = t + 1 < I.valid ? p.gate[I.row0 + (size_t)(t + 1) * p.H] : 0.f;
            }
            if (gate_thr) bt = ln < I.valid ? p.beta[I.row0 + (size_t)ln * p.H] : 0.f;
        };
        load_gates(blockIdx.x);
        for (int w = blockIdx.x; w < p.items; w += gridDim.x, ++it) {
            const int ph = it & 1;
            const Item I = item_of(p, w, nc);
            const int valid = I.valid;
            const size_t row0 = I.row0;
            const uint8_t *KQ = sm + OFF_KQ + ph * 32768;
            // ------------------------------ P0: decays, gate terms, L and P ------------------------------
            named_bar(BAR_W, NW);  // every warp is done with the previous item's row data
            if (warp == 7) chunk_decay(g0, g1, lane, &R.g[0].x, &R.g[0].y, 2, R.eg, R.ec);
            named_bar(BAR_W, NW);
            wait(&bars->g, ph);
            float m[32];  // Gamma o Gram of row tr, this half's columns: L (ln < 64) or P, strictly below the diagonal
            if (ok) {
                tmem_ld32(lane_base + TM_U + col0, m);
                tmem_ld_wait();
                if (gate_thr) {
                    const int t = ln;
                    float lam = 0.f;
#pragma unroll
                    for (int s = 0; s < 32; ++s) lam = (s == (t & 31)) ? m[s] : lam;
                    float db = 0.f, dl = 0.f;
                    if (t < valid) gate_grad(bt, lam, p.euler, db, dl);
                    R.dadb[t] = db;
                    R.dadl[t] = dl;
                    R.al[t] = efla_alpha(bt, lam, p.euler);  // (0 past the end: beta is)
                }
                const float2 gt = R.g[tr];
#pragma unroll
                for (int s = 0; s < 32; ++s) {
                    const float2 gs = R.g[col0 + s];
                    m[s] = col0 + s < tr ? m[s] * pair_decay(gt.x, gt.y, gs.x, gs.y) : 0.f;
                }
            }
            load_gates(w + gridDim.x);
            if (named_bar_any(BAR_W, NW, !ok)) break;  // every CUDA-core warp leaves together
            // ------------------------------ P2: R^T; dY . R ------------------------------
            float s_yr = 0.f;
            wait(&bars->v_full, ph);
            wait(&bars->m1a, ph);
            if (ok) {
                float r[32], f[32];
                tmem_ld32(lane_base + TM_X + col0, r);
                load32(R.eg + col0, f);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = fmaf(-f[e], r[e], bf16_at(sm + OFF_V + feat(e, 8192)));
                load32(R.al + col0, f);
#pragma unroll
                for (int e = 0; e < 32; ++e) f[e] *= r[e];
                uint32_t hh[16], ll[16];
                split_pack_rn<16>(f, hh, ll);
                tmem_st16u(lane_base + TM_RS + 16 * hf, hh);
                tmem_st16u(lane_base + TM_RS + 32 + 16 * hf, ll);
                arrive(&bars->w_u);
                wait(&bars->tma_rod, ph);
                if (ok) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        r[e] *= bf16_at(sm + OFF_ROD + feat(e, 16384)) + bf16_at(sm + OFF_YL + feat(e, 8192));
                    s_yr = lane_reduce_scatter(r, lane);
                }
            }
            // ------------------------------ P3: the U^T tile ------------------------------
            wait(&bars->u, ph);
            if (ok) {
                float u[32];
                tmem_ld32(lane_base + TM_U + col0, u);
                tmem_ld_wait();
                put16(sm + OFF_UT, LO_UT, ln, col0, u);
                put16(sm + OFF_UT, LO_UT, ln, col0 + 16, u + 16);
                arrive(&bars->w_p3);
            }
            // ------------------------------ P4: dalpha, dg, operands ------------------------------
            float s_a = 0.f, s_w = 0.f, s_m = 0.f, m_first = 0.f;
            wait(&bars->m1b, ph);
            if (ok) {  // a_t = e^{G_t} (q_t . (S dO_t) - alpha_t k_t . (S dY_t)): this warp's 32 features
                float x[32], y[32], f[32];
                tmem_ld32(lane_base + TM_DQ + col0, x);
                tmem_ld32(lane_base + TM_DK + col0, y);
                load32(R.al + col0, f);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const uint8_t *kp = KQ + feat(e, 16384);
                    x[e] = fmaf(bf16_at(kp + 8192), x[e], -f[e] * y[e] * bf16_at(kp));
                }
                s_a = R.eg[col0 + lane] * lane_reduce_scatter(x, lane);
            }
            wait(&bars->b, ph);
            if (ok) {
                float x[32];
                tmem_ld32(lane_base + TM_P + col0, x);
                if (ln < C) {  // (whole warps) dY lo U^T joins
                    float y[32];
                    tmem_ld32(lane_base + TM_RS + col0, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int s = 0; s < 32; ++s) x[s] += y[s];
                }
                tmem_ld_wait();
                // dL = -diag(alpha) (dY U^T): M_ts = dP_ts P_ts and dL_ts L_ts (s < t; m is 0 elsewhere), here still
                // without the row's factor -alpha_t, which the sums over s take at the end
                const float2 gr = R.g[tr];
                const float fac = ln < C ? -R.al[tr] : 1.f;
                float total = 0.f;
#pragma unroll
                for (int s = 0; s < 32; ++s) {
                    const float v = m[s] * x[s];
                    m[s] = col0 + s <= tr ? fac * total : 0.f;  // exclusive prefix sum along the row, from this half's first column
                    total += v;
                    const float2 gs = R.g[col0 + s];
                    x[s] = col0 + s <= tr ? fac * x[s] * pair_decay(gr.x, gr.y, gs.x, gs.y) : 0.f;
                }
                m_first = total;
                if (ln < C) {  // dL' = Gamma o dL, strictly below the diagonal, row t
#pragma unroll
                    for (int s = 0; s < 32; ++s) dLs[tr * DL_LD + col0 + s] = col0 + s < tr ? x[s] : 0.f;
                } else {       // dP' = Gamma o dP, row t
                    put16(sm + OFF_W, LO_64, tr, col0, x);
                    put16(sm + OFF_W, LO_64, tr, col0 + 16, x + 16);
                }
                s_m = lane_reduce_scatter(m, lane);  // columns over this warp's rows
            }
            wait(&bars->d2, ph);
            if (ok) {  // w_t = c_t k_t . (dS' u_t)
                float x[32];
                tmem_ld32(lane_base + TM_D2 + col0, x);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] *= bf16_at(KQ + feat(e, 16384));
                s_w = R.ec[col0 + lane] * lane_reduce_scatter(x, lane);
                part[warp * 32 + lane] = s_yr;
                part[256 + warp * 32 + lane] = s_a;
                part[512 + warp * 32 + lane] = s_w;
                part[768 + warp * 32 + lane] = s_m;
                rsum[hf * 128 + ln] = m_first;
            }
            if (named_bar_any(BAR_W, NW, !ok)) break;
            {  // E = dL' + dL'^T + diag(2 dalpha dalpha/dlambda)
                const int t = tid >> 2, s0 = (tid & 3) * 16;
                const float *pd = part + (t >> 5) * 128 + (t & 31);
                const float dal = ((pd[0] + pd[32]) + (pd[64] + pd[96])) - (rsum[t] + rsum[128 + t]);
                const float dg = 2.f * dal * R.dadl[t];
                float x[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] = dLs[t * DL_LD + s0 + e] + dLs[(s0 + e) * DL_LD + t] + (s0 + e == t ? dg : 0.f);
                put16(sm + OFF_UT, LO_64, t, s0, x);
                if ((tid & 3) == 0 && t < valid) p.dbeta[row0 + (size_t)t * p.H] = dal * R.dadb[t];
            }
            if (warp == 0) {  // dg: lane l has tokens 2 l and 2 l + 1
                auto total = [&](int which, int t) {
                    const float *x = part + which * 256 + (t >> 5) * 128 + (t & 31);
                    return (x[0] + x[32]) + (x[64] + x[96]);
                };
                const int t = 2 * lane;
                const float a0 = total(1, t), a1 = total(1, t + 1), w0 = total(2, t), w1 = total(2, t + 1);
                // rows of the second half: what their first 32 columns hold belongs to every column t >= 32
                const float f0 = rsum[C + t] - R.al[t] * rsum[t], f1 = rsum[C + t + 1] - R.al[t + 1] * rsum[t + 1];
                float sa = a0 + a1, sf = f0 + f1, sw = w0 + w1;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const float x = __shfl_down_sync(0xffffffffu, sa, off), y = __shfl_down_sync(0xffffffffu, sf, off);
                    const float z = __shfl_up_sync(0xffffffffu, sw, off);
                    if (lane + off < 32) {
                        sa += x;
                        sf += y;
                    }
                    if (lane >= off) sw += z;
                }
                const float4 th = *reinterpret_cast<const float4 *>(p.sdot + (size_t)w * 4);
                const float through = R.eg[C - 1] * ((th.x + th.y) + (th.z + th.w));
                const float up = lane >= 16 ? 1.f : 0.f;
                float before = __shfl_up_sync(0xffffffffu, sw, 1);  // w of the lanes before
                if (lane == 0) before = 0.f;
                // (suffix sums at the odd token are taken from the next lane, not by subtraction)
                float sa_n = __shfl_down_sync(0xffffffffu, sa, 1), sf_n = __shfl_down_sync(0xffffffffu, sf, 1);
                if (lane == 31) sa_n = sf_n = 0.f;
                const float dg0 = through + sa + before + total(3, t) + up * sf;
                const float dg1 = through + (a1 + sa_n) + (before + w0) + total(3, t + 1) + up * (f1 + sf_n);
                if (t < valid) p.dg[row0 + (size_t)t * p.H] = dg0;
                if (t + 1 < valid) p.dg[row0 + (size_t)(t + 1) * p.H] = dg1;
            }
            arrive(&bars->w_p5);
            // ------------------------------ P6 ------------------------------
            wait(&bars->m2, ph);
            if (ok) {
                float dq[32], dk[32], x[32], f[32];
                tmem_ld32(lane_base + TM_DQ + col0, dq);
                tmem_ld32(lane_base + TM_P + col0, x);
                load32(R.eg + col0, f);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) dq[e] = fmaf(f[e], dq[e], x[e]);
                tmem_ld32(lane_base + TM_DK + col0, x);
                tmem_ld32(lane_base + TM_E + col0, dk);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] *= -f[e];
                load32(R.al + col0, f);
#pragma unroll
                for (int e = 0; e < 32; ++e) dk[e] = fmaf(f[e], x[e], dk[e]);
                tmem_ld32(lane_base + TM_D2 + col0, x);
                load32(R.ec + col0, f);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->w_free);  // everything is in registers
#pragma unroll
                for (int e = 0; e < 32; ++e) dk[e] = fmaf(f[e], x[e], dk[e]);
                if (p.part) {
                    float *o = p.part + (row0 + (size_t)col0 * p.H) * D + ln;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (col0 + e < valid) {
                            o[(size_t)e * p.H * D] = dq[e];
                            o[p.plane + (size_t)e * p.H * D] = dk[e];
                        }
                } else {  // staged as bf16 tiles; lanes ln and ln ^ 1 pair up, the even one writes dq, the odd one dk
                    const bool odd = (lane & 1) != 0;
                    uint8_t *dst = sm + OFF_UT + (odd ? 16384 : 0) + (ln >> 6) * 8192 + hf * 4096;
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const __nv_bfloat162 a = __floats2bfloat162_rn(dq[e], dq[e + 1]), b = __floats2bfloat162_rn(dk[e], dk[e + 1]);
                        const uint32_t aq = *reinterpret_cast<const uint32_t *>(&a), bk = *reinterpret_cast<const uint32_t *>(&b);
                        const uint32_t recv = __shfl_xor_sync(0xffffffffu, odd ? aq : bk, 1);
                        const uint32_t lo = odd ? recv : aq, hi = odd ? bk : recv;  // columns ln & ~1 and (ln & ~1) + 1
                        *reinterpret_cast<uint32_t *>(dst + swz_offset(e, (ln & 62), 0)) = __byte_perm(lo, hi, 0x5410);
                        *reinterpret_cast<uint32_t *>(dst + swz_offset(e + 1, (ln & 62), 0)) = __byte_perm(lo, hi, 0x7632);
                    }
                }
                arrive(&bars->w_out);
            }
        }
        if (!ok) *abort_flag = 1;
    }

    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) atomicExch(p.status, (int)EFLA_ERR_DEVICE_TIMEOUT);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace gr

template <typename K>
cudaError_t allow_smem(K kernel, uint32_t bytes, int dev, bool (&done)[64]) {
    if (dev < 64 && done[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

}  // namespace

cudaError_t launch_gated_bwd_tc(const GatedBwdArgs &a, const char **why) {
    const long units = (long)a.B * a.H, nc = (a.T + C - 1) / C, items = units * nc;
    const GatedWs L = gated_ws(a.B, a.T, a.Hk, a.H, a.dk_dim, a.dv_dim, a.in_dtype);
    char *ws = static_cast<char *>(a.ws);
    const size_t n = (size_t)a.B * a.T * a.H * D;
    __nv_bfloat16 *y_hi = reinterpret_cast<__nv_bfloat16 *>(ws + L.tok), *y_lo = y_hi + n;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) {
        *why = "querying the SM count";
        return e;
    }
    static bool st_done[64] = {}, gr_done[64] = {};
    if ((e = allow_smem(st::state_kernel, st::SMEM_ALLOC, dev, st_done)) != cudaSuccess ||
        (e = allow_smem(gr::grad_kernel, gr::SMEM_ALLOC, dev, gr_done)) != cudaSuccess) {
        *why = "setting the gated backward kernels' shared memory";
        return e;
    }
    st::Params s;
    gr::Params p;
    memset(&s, 0, sizeof s);
    memset(&p, 0, sizeof p);
    if (!bwd_row_map(&s.map_q, a.q, a.B, a.T, a.Hk) || !bwd_row_map(&s.map_k, a.k, a.B, a.T, a.Hk) ||
        !bwd_row_map(&s.map_do, a.dO, a.B, a.T, a.H) || !bwd_row_map(&s.map_dv, a.dv, a.B, a.T, a.H) ||
        !bwd_row_map(&s.map_yh, y_hi, a.B, a.T, a.H) || !bwd_row_map(&s.map_yl, y_lo, a.B, a.T, a.H) ||
        !bwd_row_map(&p.map_v, a.v, a.B, a.T, a.H) || !bwd_row_map(&p.map_dq, a.dq, a.B, a.T, a.Hk) ||
        !bwd_row_map(&p.map_dk, a.dk, a.B, a.T, a.Hk)) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    s.gate = a.g;
    s.beta = a.beta;
    s.dST = a.dST;
    s.dse = reinterpret_cast<uint8_t *>(ws + L.dse);
    s.tpp = reinterpret_cast<const uint8_t *>(ws + L.w);
    s.dS0 = a.dS0;
    s.states = reinterpret_cast<const uint8_t *>(ws + L.states);
    s.sdot = reinterpret_cast<float *>(ws + L.sdot);
    s.euler = a.euler;
    s.status = a.status;
    s.T = a.T;
    s.H = a.H;
    s.rep = a.H / a.Hk;
    s.wait_ns = wait_limit_ns();
    s.debug_stall = (debug_stall() & STALL_BWD_STATE) ? 1 : 0;
    *why = "tcgen05 gated state-gradient kernel launch";
    st::state_kernel<<<(unsigned)units, 320, st::SMEM_ALLOC, a.stream>>>(s);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    p.map_q = s.map_q;
    p.map_k = s.map_k;
    p.map_do = s.map_do;
    p.map_yh = s.map_yh;
    p.map_yl = s.map_yl;
    p.gate = a.g;
    p.beta = a.beta;
    p.sdot = s.sdot;
    p.states = s.states;
    p.dse = s.dse;
    p.tpp = s.tpp;
    p.part = a.Hk == a.H ? nullptr : reinterpret_cast<float *>(ws + L.part);
    p.plane = n;
    p.dbeta = a.dbeta;
    p.dg = a.dg;
    p.status = a.status;
    p.T = a.T;
    p.H = a.H;
    p.rep = s.rep;
    p.items = (int)items;
    p.euler = a.euler;
    p.wait_ns = s.wait_ns;
    p.debug_stall = (debug_stall() & STALL_BWD_GRAD) ? 1 : 0;
    *why = "tcgen05 gated gradient kernel launch";
    gr::grad_kernel<<<(unsigned)std::min<long>(items, sms), gr::NTH, gr::SMEM_ALLOC, a.stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess || !p.part) return e;
    *why = "gated head-sum kernel launch";
    return launch_gated_reduce_heads(a, p.part);
}

}  // namespace efla
