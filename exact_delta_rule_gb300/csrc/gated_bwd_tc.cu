// Backward of the gated delta rule on the sm_103a tensor cores (tcgen05 + TMEM + TMA): bf16, d_k = d_v =
// 128, chunks of 64, rows of [B, T], after the training forward (chunk_tc.cu), which leaves every chunk's
// start state S and T'' in the workspace as bf16 hi/lo operand tiles.  The formulas are in gated_simt.cu.
//
// 1. State pass (state_kernel): one CTA per (b, h) walks the chunks in reverse with dS^T fp32 in TMEM,
//    lane j = column j of d_v, everything transposed as in the forward:
//      G^T  = (dS'^T K^T) diag(c) + dO^T P       dR^T = G^T T''
//      dS^T = e^{G_C} dS'^T + (dO^T diag(e^G)) Q - (dR^T diag(e^G)) K
//    It writes dS' of every chunk as an operand tile, G (fp32) and dR: its high part is dv, the rounding
//    of dR to bf16, its low part goes to the workspace beside it.
//    The serial chain is dS' split -> dS'^T K^T -> G split -> dR -> dR split -> dS; the decays that are
//    factors of rows ride on the splits, e^{G_C} is applied to TMEM while the tensor core forms dS'^T K^T,
//    and the operand diag(e^G) dO is formed by the prep warps beside it.
// 2. Gradient pass (grad_kernel): persistent CTAs over the (b, h, chunk) items, all independent:
//      P0  Gram [K; Q] K^T; L = Gamma o strictly-lower(K K^T) as a tile, L and P kept in registers; <S, dS'>
//      P1  X^T = S^T K^T;  [S dR^T | S dO^T]
//      P2  R^T = V^T - X^T diag(e^G);  U^T = R^T T''^T
//      P3  -Z^T = -R^T + U^T L^T;  -dY^T = -G^T + dR^T L;  [dR; dO] U^T;  dS' U^T
//      P4  dalpha, dg and the operands dP' = Gamma o dP, E = dL' + dL'^T + diag(2 dalpha dalpha/dlambda)
//      P5  dP' K;  dP'^T Q + E K
//      P6  dq = e^G (S dO^T) + dP' K,  dk = -e^G (S dR^T) + c (dS' U^T) + (dP'^T Q + E K)
//    The products with different row factors keep their own accumulators and are joined when they are
//    read out.  Sums over features or rows are taken by shuffles and per-warp slots in a fixed order.
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
constexpr uint32_t OFF_TPP = NSTAGE * STAGE_BYTES;  // per chunk parity: T'' hi, lo, P hi, lo, [64][64] bf16 each
constexpr uint32_t TPP_BYTES = 32768;
constexpr uint32_t OFF_DRS = OFF_TPP + 2 * TPP_BYTES;  // dR hi, lo on their way to HBM, [2 cb][64 rows][64] each
constexpr uint32_t OFF_DEC = OFF_DRS + 32768;          // {G hi, lo} [64], then per parity e^G [64], c [64]
constexpr uint32_t OFF_BAR = OFF_DEC + 512 + 1024;
constexpr uint32_t OFF_MISC = OFF_BAR + 256;
constexpr uint32_t SMEM_ALLOC = OFF_MISC + 16 + 1024;
static_assert(OFF_TPP % 1024 == 0 && OFF_DRS % 1024 == 0 && SMEM_ALLOC <= 232448, "shared memory layout");

constexpr uint32_t TM_S = 0;     // dS^T fp32 (128)
constexpr uint32_t TM_SA = 128;  // dS'^T hi (64) | lo (64); then dR^T fp32 (64) and -diag(e^G) dR hi (32) | lo (32)
constexpr uint32_t TM_X = 256;   // dS'^T K^T fp32 (64); then G^T hi (32) | lo (32)
constexpr uint32_t TM_G = 320;   // Gram rows [K; Q] K^T fp32 (64)
constexpr uint32_t TM_G2 = 384;  // dO^T P fp32 (64)
constexpr uint32_t TM_DO = 448;  // diag(e^G) dO hi (32) | lo (32)
constexpr int BAR_PREP = 2, BAR_STATE = 3;

struct Params {
    CUtensorMap map_q, map_k, map_do, map_dv, map_lo;  // [B, T, heads, 128] bf16, box 64 x 1 x 64 x 1, 128B swizzle
    const float *gate, *dST;
    uint8_t *dse;
    const uint8_t *tpp;
    float *dS0, *g_out;
    int *status;
    int T, H, rep;
    int debug_stall;
    unsigned long long wait_ns;
};

struct Bars {
    uint64_t tma_full[NSTAGE], s_free[NSTAGE];
    uint64_t g_done, g_free;
    uint64_t gate_ready[2];  // decays of a chunk written
    uint64_t prep_ready[2];  // P written and T'' landed
    uint64_t t_full[2], tpp_free[2];
    uint64_t do_ready;       // diag(e^G) dO written (128 arrivals)
    uint64_t x_done, u_done, s_done;
    uint64_t s_prep;         // as s_done, for the prep warps
    uint64_t sa_ready, r_ready, u_ready;
    uint64_t drain, never;
};
static_assert(sizeof(Bars) <= 256, "mbarrier block exceeds its slot");

// Tokens 0-63 of column j (this lane) as bf16 hi and lo into the staging tiles of the TMA stores ([2
// column blocks][64 tokens][64], 128-byte swizzle, lo 16 KB behind hi).  Lanes j and j ^ 1 pair up: the
// even lane writes the hi word of columns j, j + 1, the odd lane the lo.
__device__ __forceinline__ void stage_split(uint8_t *stg, int j, const float (&x0)[32], const float (&x1)[32]) {
    const bool odd = (j & 1) != 0;
    uint8_t *dst = stg + (odd ? 16384u : 0u);
#pragma unroll
    for (int t = 0; t < 64; ++t) {
        uint32_t h16, l16;
        split1_rn(t < 32 ? x0[t] : x1[t - 32], h16, l16);
        const uint32_t recv = __shfl_xor_sync(0xffffffffu, odd ? h16 : l16, 1);
        *reinterpret_cast<uint32_t *>(dst + swz_offset(t, j & ~1, 8192)) = odd ? ((recv & 0xffffu) | (l16 << 16)) : (h16 | (recv << 16));
    }
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
        // Gram row r is TMEM lane r: rows 64-127 (Q K^T) are read by warps 6 and 7; warp 4 forms the decays;
        // all four form diag(e^G) dO (thread = lane = feature of d_v).
        const int lane = tid & 31, row = tid - 128;
        const bool leader = tid == 128;
        auto load_g = [&](int it, int odd) {
            const int t = it < nchunks ? chunk_of(it) * C + 2 * lane + odd : p.T;
            return warp == 4 && t < p.T ? p.gate[((size_t)b * p.T + t) * p.H + h] : 0.f;
        };
        float g0 = load_g(0, 0), g1 = load_g(0, 1);
        bool ok = true;
        for (int it = 0; it < nchunks; ++it) {
            const int buf = it & 1, st = it % NSTAGE;
            float *eg = dec + buf * 128;
            // (chunk it - 2, the last reader of this parity's decays, is complete: s_prep below)
            if (warp == 4) chunk_decay(g0, g1, lane, gsum, gsum + 1, 2, eg, eg + 64);
            g0 = load_g(it + 1, 0);
            g1 = load_g(it + 1, 1);
            ok = ok && wait_bar_warp(&bars->g_done, it & 1, abort_flag, wait_ns);
            if (it >= 2) ok = ok && wait_bar_warp(&bars->tpp_free[buf], ((it - 2) >> 1) & 1, abort_flag, wait_ns);
            tc_fence_after();
            float x[2][32];
            if (ok && row >= C) {
                tmem_ld32(lane_base + TM_G, x[0]);
                tmem_ld32(lane_base + TM_G + 32, x[1]);
                tmem_ld_wait();
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
            // diag(e^G) dO of this chunk once the previous chunk's state update has read TM_DO
            ok = __all_sync(0xffffffffu, ok);
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
                        y[e] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(src + swz_offset(32 * hf + e, row, 8192)) << 16);
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
            const int c = chunk_of(it), valid = min(C, p.T - c * C);
            const size_t row0 = ((size_t)b * p.T + (size_t)c * C) * p.H + h;
            const float *eg = dec + (it & 1) * 128, *ec = eg + 64;
            float x0[32], x1[32];
            if (ok) {
                tc_fence_after();
#pragma unroll 1
                for (int g = 0; g < 4; g = opaque(g + 1)) {  // dS'^T -> bf16 hi/lo operand
                    float sv[32];
                    uint32_t hi[16], lo[16];
                    tmem_ld32(lane_base + TM_S + g * 32, sv);
                    tmem_ld_wait();
                    split_pack_rn<16>(sv, hi, lo);
                    tmem_st16u(lane_base + TM_SA + g * 16, hi);
                    tmem_st16u(lane_base + TM_SA + 64 + g * 16, lo);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars->sa_ready);
                ok = wait_bar_warp(&bars->gate_ready[it & 1], (it >> 1) & 1, abort_flag, wait_ns);
                // dS' of this chunk to HBM and e^{G_C} dS' into TMEM while the tensor core forms dS'^T K^T
                if (ok) decay_state_rows(p.dse + ((size_t)blockIdx.x * nchunks + c) * 65536, lane_base + TM_S, 0, 4, j, eg[C - 1]);
                ok = ok && wait_bar_warp(&bars->x_done, it & 1, abort_flag, wait_ns);
            }
            if (ok) {  // G^T = (dS'^T K^T) diag(c) + dO^T P
                tc_fence_after();
                uint32_t hi[16], lo[16];
                float y[32], f[32];
                tmem_ld32(lane_base + TM_X, x0);
                tmem_ld32(lane_base + TM_X + 32, x1);
                tmem_ld32(lane_base + TM_G2, y);
                load32(ec, f);
                tmem_ld_wait();
#pragma unroll
                for (int t = 0; t < 32; ++t) x0[t] = fmaf(f[t], x0[t], y[t]);
                tmem_ld32(lane_base + TM_G2 + 32, y);
                load32(ec + 32, f);
                tmem_ld_wait();
#pragma unroll
                for (int t = 0; t < 32; ++t) x1[t] = fmaf(f[t], x1[t], y[t]);
                split_pack_rn<16>(x0, hi, lo);
                tmem_st16u(lane_base + TM_X, hi);
                tmem_st16u(lane_base + TM_X + 32, lo);
                split_pack_rn<16>(x1, hi, lo);
                tmem_st16u(lane_base + TM_X + 16, hi);
                tmem_st16u(lane_base + TM_X + 48, lo);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars->r_ready);
                float *go = p.g_out + row0 * D + j;  // for the gradient pass, sent while the tensor core forms dR
#pragma unroll
                for (int t = 0; t < 32; ++t)
                    if (t < valid) go[(size_t)t * p.H * D] = x0[t];
#pragma unroll
                for (int t = 0; t < 32; ++t)
                    if (32 + t < valid) go[(size_t)(32 + t) * p.H * D] = x1[t];
                ok = wait_bar_warp(&bars->u_done, it & 1, abort_flag, wait_ns);
            }
            if (ok) {  // -diag(e^G) dR -> operand
                tc_fence_after();
                uint32_t hi[16], lo[16];
                float f[32];
                tmem_ld32(lane_base + TM_SA, x0);
                tmem_ld32(lane_base + TM_SA + 32, x1);
                load32(eg, f);
                tmem_ld_wait();
#pragma unroll
                for (int t = 0; t < 32; ++t) f[t] *= -x0[t];
                split_pack_rn<16>(f, hi, lo);
                tmem_st16u(lane_base + TM_SA + 64, hi);
                tmem_st16u(lane_base + TM_SA + 96, lo);
                load32(eg + 32, f);
#pragma unroll
                for (int t = 0; t < 32; ++t) f[t] *= -x1[t];
                split_pack_rn<16>(f, hi, lo);
                tmem_st16u(lane_base + TM_SA + 80, hi);
                tmem_st16u(lane_base + TM_SA + 112, lo);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars->u_ready);
            }
            // dR as bf16 hi (= dv) and lo, staged and stored by TMA (rows past the end are clipped) once the
            // previous chunk's stores have read the staging
            if (tid == 0) bulk_wait_read0();
            if (named_bar_any(BAR_STATE, 128, !ok)) {
                ok = false;
                break;
            }
            stage_split(stg, j, x0, x1);
            fence_proxy_async_smem();
            named_bar(BAR_STATE, 128);
            if (tid == 0) {
                for (int cb = 0; cb < 2; ++cb) {
                    tma_store_4d(&p.map_dv, stg + cb * 8192, cb * 64, h, c * C, b);
                    tma_store_4d(&p.map_lo, stg + 16384 + cb * 8192, cb * 64, h, c * C, b);
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
            {  // dR^T = G^T T'' (T'' read as an MN-major operand, K = s), into TM_SA
                const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 1);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t th = smem_desc(tp + ks * 2048, 8192, 1024), tl = smem_desc(tp + 8192 + ks * 2048, 8192, 1024);
                    mma_bf16_ts_e(tmem + TM_SA, tmem + TM_X + ks * 8, th, idesc, ks > 0);
                    mma_bf16_ts_e(tmem + TM_SA, tmem + TM_X + ks * 8, tl, idesc, 1);
                    mma_bf16_ts_e(tmem + TM_SA, tmem + TM_X + 32 + ks * 8, th, idesc, 1);
                }
                mma_commit_e(&bars->u_done);
                mma_commit_e(&bars->tpp_free[buf]);
            }
            if (!(ok = wait_bar_warp(&bars->do_ready, it & 1, abort_flag, wait_ns))) break;
            tc_fence_after();
            {  // dS^T += (diag(e^G) dO)^T Q, behind dR in the pipe (the state warpgroup scaled dS before r_ready)
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
            {  // dS^T += (-diag(e^G) dR)^T K (the chain)
                const uint32_t idesc = idesc_bf16_f32(128, 128, 0, 1);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16_ts_e(tmem + TM_S, tmem + TM_SA + 64 + part * 32 + ks * 8,
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
constexpr uint32_t OFF_KQ = 0;        // [K; Q]: 2 column blocks x 128 rows, 32 KB
constexpr uint32_t OFF_ROD = 32768;   // [dR; dO] hi | lo: 2 column blocks x 128 rows each (dO's lo rows stay zero)
constexpr uint32_t OFF_SS = 98304;    // S, later dS', hi | lo: 2 column blocks x 128 rows each
constexpr uint32_t OFF_W = 163840;    // T'' hi | lo [64][64]; later dP' hi | lo
constexpr uint32_t OFF_L = 180224;    // L hi | lo [64][64]; later E hi | lo
constexpr uint32_t OFF_UT = 196608;   // U^T hi | lo [128][64]
constexpr uint32_t OFF_ROW = 229376;  // fp32 rows, struct RowData
constexpr uint32_t LO_128 = 32768, LO_UT = 16384, LO_64 = 8192;
// scratch over the hi part of [dR; dO] once its products are complete: dL' [64][65], then per-warp sums
constexpr int DL_LD = 65;
constexpr uint32_t OFF_DL = OFF_ROD;
constexpr uint32_t OFF_PART = OFF_ROD + 64 * DL_LD * 4;  // fp32 [4 sums][8 warps][32], then M's first-half row sums [128]
static_assert(64 * DL_LD * 4 + 4 * 8 * 32 * 4 + 128 * 4 <= LO_128 && OFF_PART % 16 == 0, "scratch leaves the hi part");

struct RowData {
    float2 g[C];              // G_t hi, lo
    float eg[C], ec[C];
    float dadb[C], dadl[C], dal[C];
    float sdot[8];            // <S, dS'>, a warp each
};
constexpr uint32_t OFF_BAR = OFF_ROW + sizeof(RowData);
constexpr uint32_t OFF_MISC = OFF_BAR + 256;
constexpr uint32_t SMEM_ALLOC = OFF_MISC + 16;
static_assert(OFF_BAR % 16 == 0 && SMEM_ALLOC <= 232448, "shared memory layout");

// TMEM columns (fp32, 64 each, unless split: hi in the first 32 columns, lo in the next 32)
constexpr uint32_t TM_P = 0;     // [dR; dO] U^T; then (dP' K)^T
constexpr uint32_t TM_D2 = 64;   // (dS' U^T) as [feature][token]
constexpr uint32_t TM_X = 128;   // X^T -> -R^T -> -Z^T; then (dP'^T Q + E K)^T
constexpr uint32_t TM_RS = 192;  // R^T split
constexpr uint32_t TM_U = 256;   // Gram -> U^T -> -G^T -> -dY^T
constexpr uint32_t TM_US = 320;  // U^T split
constexpr uint32_t TM_DK = 384;  // S dR^T, adjacent to
constexpr uint32_t TM_DQ = 448;  // S dO^T: one N = 128 product fills both

struct Params {
    CUtensorMap map_q, map_k, map_do, map_dv, map_lo;
    const __nv_bfloat16 *v;
    const float *gate, *beta;
    const uint8_t *states, *dse, *tpp;
    const float *g;                // G of every token
    __nv_bfloat16 *dq, *dk;        // [B, T, Hk, 128]
    float *part;                   // [2][B, T, H, 128] instead, where key heads are shared
    float *dbeta, *dg;
    size_t plane;                  // elements of one part
    int *status;
    int T, H, rep, items;
    int euler, debug_stall;
    unsigned long long wait_ns;
};

struct Bars {
    uint64_t tma_kq, tma_rod, s_full, d_full, t_full;
    uint64_t g, m1a, m1b, u, a, b, d2, m2;    // products complete
    uint64_t w_s, w_u, w_p3, w_p5, w_free;    // CUDA-core warps done with an input / operands written (8 arrivals)
    uint64_t drain, never;
};
static_assert(sizeof(Bars) <= 256, "mbarrier block exceeds its slot");

__device__ __forceinline__ void tsplit32(uint32_t lane_base, uint32_t base, int h, const float (&x)[32]) {
    uint32_t hh[16], ll[16];
    split_pack_rn<16>(x, hh, ll);
    tmem_st16u(lane_base + base + 16 * h, hh);
    tmem_st16u(lane_base + base + 32 + 16 * h, ll);
}

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

// sum of (hi + lo)(hi' + lo') over eight bf16 pairs
__device__ __forceinline__ float dot8(const uint4 &h, const uint4 &l, const uint4 &h2, const uint4 &l2) {
    const uint32_t a[4] = {h.x, h.y, h.z, h.w}, b[4] = {l.x, l.y, l.z, l.w}, c[4] = {h2.x, h2.y, h2.z, h2.w},
                   d[4] = {l2.x, l2.y, l2.z, l2.w};
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s0 = fmaf(__uint_as_float(a[i] << 16) + __uint_as_float(b[i] << 16),
                  __uint_as_float(c[i] << 16) + __uint_as_float(d[i] << 16), s0);
        s1 = fmaf(__uint_as_float(a[i] & 0xffff0000u) + __uint_as_float(b[i] & 0xffff0000u),
                  __uint_as_float(c[i] & 0xffff0000u) + __uint_as_float(d[i] & 0xffff0000u), s1);
    }
    return s0 + s1;
}

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
        uint64_t *one[] = {&bars->tma_kq, &bars->tma_rod, &bars->s_full, &bars->d_full, &bars->t_full, &bars->g, &bars->m1a,
                           &bars->m1b, &bars->u, &bars->a, &bars->b, &bars->d2, &bars->m2, &bars->drain, &bars->never};
        for (uint64_t *x : one) mbar_init(x, 1);
        uint64_t *eight[] = {&bars->w_s, &bars->w_u, &bars->w_p3, &bars->w_p5, &bars->w_free};
        for (uint64_t *x : eight) mbar_init(x, 8);
        fence_mbar_init();
        *abort_flag = 0;
    }
    // dO is exact bf16: its rows of the lo part are zero for every item
    for (int e = tid; e < 2 * 64 * 8; e += NTH) {
        const int cb = e >> 9, x = e & 511;
        *reinterpret_cast<uint4 *>(sm + OFF_ROD + LO_128 + cb * 16384 + 8192 + x * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
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
        const uint32_t kq = s_sm + OFF_KQ, rod = s_sm + OFF_ROD, ss = s_sm + OFF_SS;
        const uint32_t wt = s_sm + OFF_W, l = s_sm + OFF_L, ut = s_sm + OFF_UT;
        if (leader) {
            prefetch_tensormap(&p.map_q);
            prefetch_tensormap(&p.map_k);
            prefetch_tensormap(&p.map_do);
            prefetch_tensormap(&p.map_dv);
            prefetch_tensormap(&p.map_lo);
        }
        bool ok = true;
        int it = 0, kq_pending = -1, rod_pending = -1, s_pending = -1, d_pending = -1, t_pending = -1;
        auto load_tile = [&](uint64_t *bar, uint32_t off, const uint8_t *src, uint32_t bytes) {
            if (leader) {
                mbar_arrive_expect_tx(bar, bytes);
                bulk_load(sm + off, src, bytes, bar);
            }
            __syncwarp();
        };
        auto wait = [&](uint64_t *bar, int parity) {
            ok = ok && wait_bar_warp(bar, parity, abort_flag, wait_ns);
            tc_fence_after();
            return ok;
        };
        if (p.debug_stall) ok = wait_bar_warp(&bars->never, 0, abort_flag, wait_ns);
        for (int w = blockIdx.x; w < p.items; w += gridDim.x, ++it) {
            const int ph = it & 1;
            if (!ok) break;
            const Item I = item_of(p, w, nc);
            // the previous item's last products are complete: every operand tile is free
            if (it > 0 && !wait(&bars->m2, ph ^ 1)) break;
            if (leader) {
                mbar_arrive_expect_tx(&bars->tma_kq, 2 * 16384);
                for (int cb = 0; cb < 2; ++cb) {
                    tma_load_4d(sm + OFF_KQ + cb * 16384, &p.map_k, &bars->tma_kq, cb * 64, I.hk, I.t0, I.b);
                    tma_load_4d(sm + OFF_KQ + cb * 16384 + 8192, &p.map_q, &bars->tma_kq, cb * 64, I.hk, I.t0, I.b);
                }
            }
            kq_pending = ph;
            __syncwarp();
            load_tile(&bars->s_full, OFF_SS, p.states + (size_t)w * 65536, 65536);
            s_pending = ph;
            load_tile(&bars->t_full, OFF_W, p.tpp + (size_t)w * 16384, 16384);
            t_pending = ph;
            if (leader) {  // dR (rows 0-63, hi and lo) and dO (rows 64-127, hi)
                mbar_arrive_expect_tx(&bars->tma_rod, 6 * 8192);
                for (int cb = 0; cb < 2; ++cb) {
                    uint8_t *x = sm + OFF_ROD + cb * 16384;
                    tma_load_4d(x, &p.map_dv, &bars->tma_rod, cb * 64, I.h, I.t0, I.b);
                    tma_load_4d(x + LO_128, &p.map_lo, &bars->tma_rod, cb * 64, I.h, I.t0, I.b);
                    tma_load_4d(x + 8192, &p.map_do, &bars->tma_rod, cb * 64, I.h, I.t0, I.b);
                }
            }
            rod_pending = ph;
            __syncwarp();
            if (!wait(&bars->tma_kq, ph)) break;
            kq_pending = -1;
            if (leader) {  // Gram [K; Q] K^T
                const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 0);
#pragma unroll 1
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
                    mma_bf16(tmem + TM_U, smem_desc(kq + off, 16, 1024), smem_desc(kq + off, 16, 1024), idesc, ks > 0);
                }
                mma_commit(&bars->g);
            }
            __syncwarp();
            if (!wait(&bars->s_full, ph)) break;
            s_pending = -1;
            if (it > 0 && !wait(&bars->w_free, ph ^ 1)) break;  // the previous item's results are read out
            if (leader) {  // X^T = S^T K^T: S^T read as an MN-major A (M = j), K = i
                const uint32_t idesc = idesc_bf16_f32(128, 64, 1, 0);
#pragma unroll 1
                for (int part = 0; part < 2; ++part)
#pragma unroll 1
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t boff = (ks >> 2) * 16384 + (ks & 3) * 32;
                        mma_bf16(tmem + TM_X, smem_desc(ss + part * LO_128 + ks * 2048, 16384, 1024),
                                 smem_desc(kq + boff, 16, 1024), idesc, (part | ks) != 0);
                    }
                mma_commit(&bars->m1a);
            }
            __syncwarp();
            if (!wait(&bars->tma_rod, ph)) break;
            rod_pending = -1;
            if (leader) {  // [S dR^T | S dO^T]: one N = 128 product, K = j; S hi x lo only against dR (N = 64)
                const uint32_t id128 = idesc_bf16_f32(128, 128, 0, 0), id64 = idesc_bf16_f32(128, 64, 0, 0);
#pragma unroll 1
                for (int pr = 0; pr < 3; ++pr) {  // S hi x hi, S lo x hi, S hi x lo
                    const uint32_t a_lo = pr == 1 ? LO_128 : 0, b_lo = pr == 2 ? LO_128 : 0;
#pragma unroll 1
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
                        mma_bf16(tmem + TM_DK, smem_desc(ss + a_lo + off, 16, 1024), smem_desc(rod + b_lo + off, 16, 1024),
                                 pr == 2 ? id64 : id128, (pr | ks) != 0);
                    }
                }
                mma_commit(&bars->m1b);
            }
            __syncwarp();
            if (!wait(&bars->m1b, ph)) break;
            if (!wait(&bars->w_s, ph)) break;  // the S tile is read by everyone: dS' replaces it
            load_tile(&bars->d_full, OFF_SS, p.dse + (size_t)w * 65536, 65536);
            d_pending = ph;
            if (!wait(&bars->w_u, ph)) break;  // R^T split written, zero keys' T'' entries set (after t_full)
            t_pending = -1;
            if (leader) {  // U^T = R^T T''^T
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
            if (!wait(&bars->w_p3, ph)) break;  // U^T split and tile, -G^T written
            if (!wait(&bars->d_full, ph)) break;
            d_pending = -1;
            if (leader) {
                {  // -Z^T += U^T L^T: B[t][s] = L[t][s] (K-major)
                    const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 0);
#pragma unroll 1
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t bh = smem_desc(l + ks * 32, 16, 1024), bl = smem_desc(l + LO_64 + ks * 32, 16, 1024);
                        mma_bf16_ts(tmem + TM_X, tmem + TM_US + ks * 8, bh, idesc, 1);
                        mma_bf16_ts(tmem + TM_X, tmem + TM_US + ks * 8, bl, idesc, 1);
                        mma_bf16_ts(tmem + TM_X, tmem + TM_US + 32 + ks * 8, bh, idesc, 1);
                    }
                }
                {  // -dY^T += dR^T L: A[j][s] = dR[s][j] (rows 0-63 of the tile, MN-major), B[t][s] = L[s][t] (MN-major)
                    const uint32_t idesc = idesc_bf16_f32(128, 64, 1, 1);
#pragma unroll 1
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t ah = smem_desc(rod + ks * 2048, 16384, 1024), al = smem_desc(rod + LO_128 + ks * 2048, 16384, 1024);
                        const uint64_t bh = smem_desc(l + ks * 2048, 8192, 1024), bl = smem_desc(l + LO_64 + ks * 2048, 8192, 1024);
                        mma_bf16(tmem + TM_U, ah, bh, idesc, 1);
                        mma_bf16(tmem + TM_U, ah, bl, idesc, 1);
                        mma_bf16(tmem + TM_U, al, bh, idesc, 1);
                    }
                }
                mma_commit(&bars->a);
                // [dR; dO] U^T, then dS' U^T: B[t][j] = U^T[j][t] (MN-major), K = j
                const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 1);
#pragma unroll 1
                for (int pr = 0; pr < 3; ++pr) {  // hi x hi, hi x lo, lo x hi
                    const uint32_t a_lo = pr == 2 ? LO_128 : 0, b_lo = pr == 1 ? LO_UT : 0;
#pragma unroll 1
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t aoff = a_lo + (ks >> 2) * 16384 + (ks & 3) * 32;
                        mma_bf16(tmem + TM_P, smem_desc(rod + aoff, 16, 1024), smem_desc(ut + b_lo + ks * 2048, 8192, 1024),
                                 idesc, (pr | ks) != 0);
                    }
                }
                mma_commit(&bars->b);
#pragma unroll 1
                for (int pr = 0; pr < 3; ++pr) {
                    const uint32_t a_lo = pr == 2 ? LO_128 : 0, b_lo = pr == 1 ? LO_UT : 0;
#pragma unroll 1
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t aoff = a_lo + (ks >> 2) * 16384 + (ks & 3) * 32;
                        mma_bf16(tmem + TM_D2, smem_desc(ss + aoff, 16, 1024), smem_desc(ut + b_lo + ks * 2048, 8192, 1024),
                                 idesc, (pr | ks) != 0);
                    }
                }
                mma_commit(&bars->d2);
            }
            __syncwarp();
            if (!wait(&bars->w_p5, ph)) break;  // dP' and E tiles written, the accumulators below read
            if (leader) {  // (dP' K)^T = K^T dP'^T;  (dP'^T Q + E K)^T = Q^T dP' + K^T E
                const uint32_t id_kn = idesc_bf16_f32(128, 64, 1, 0), id_mn = idesc_bf16_f32(128, 64, 1, 1);
#pragma unroll 1
                for (int part = 0; part < 2; ++part)
#pragma unroll 1
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t kt = smem_desc(kq + ks * 2048, 16384, 1024);         // K^T (M = i, K = s)
                        const uint64_t qt = smem_desc(kq + 8192 + ks * 2048, 16384, 1024);  // Q^T
                        const uint32_t lo = part * LO_64;
                        mma_bf16(tmem + TM_P, kt, smem_desc(wt + lo + ks * 32, 16, 1024), id_kn, (part | ks) != 0);      // dP'[t][s]
                        mma_bf16(tmem + TM_X, qt, smem_desc(wt + lo + ks * 2048, 8192, 1024), id_mn, (part | ks) != 0);  // dP'[s][t]
                        mma_bf16(tmem + TM_X, kt, smem_desc(l + lo + ks * 32, 16, 1024), id_kn, 1);                      // E[t][s]
                    }
                mma_commit(&bars->m2);
            }
            __syncwarp();
        }
        if (!ok) *abort_flag = 1;
        if (leader) {  // every product and load issued has completed before TMEM and the CTA go (bounded)
            mma_commit(&bars->drain);
            const uint64_t ts = globaltimer_ns();
            auto settle = [&](uint64_t *bar, int parity) {
                while (parity >= 0 && !mbar_try_wait_sleep(bar, parity, 20000) && globaltimer_ns() - ts < DRAIN_NS) {
                }
            };
            settle(&bars->drain, 0);
            settle(&bars->tma_kq, kq_pending);
            settle(&bars->tma_rod, rod_pending);
            settle(&bars->s_full, s_pending);
            settle(&bars->d_full, d_pending);
            settle(&bars->t_full, t_pending);
        }
        __syncwarp();
    } else {
        // ============================ CUDA-core warps ============================
        float *dLs = reinterpret_cast<float *>(sm + OFF_DL);
        float *part = reinterpret_cast<float *>(sm + OFF_PART);  // sums {dalpha, a, w, M's columns} [8 warps][32]
        float *half_sum = part + 4 * 8 * 32;                     // [128]
        // TMEM: this thread reads and writes lane `ln`, the columns of token half `hf`
        const int hf = warp >> 2, ln = (warp & 3) * 32 + lane, col0 = 32 * hf;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const bool gate_thr = ln < C && (ln >> 5) == hf;  // holds K K^T[t][t] for t = ln
        const int tr = ln & (C - 1);                      // the row of this thread in the C x C matrices
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
        for (int w = blockIdx.x; w < p.items; w += gridDim.x, ++it) {
            const int ph = it & 1;
            const Item I = item_of(p, w, nc);
            const int valid = I.valid;
            const size_t row0 = I.row0;
            const float bt = gate_thr && ln < valid ? p.beta[row0 + (size_t)ln * p.H] : 0.f;
            // ------------------------------ P0: decays, <S, dS'>, gate terms, L ------------------------------
            named_bar(BAR_W, NW);  // every warp is done with the previous item's row data
            if (warp == 7) {
                const int t = 2 * lane;
                const float g0 = t < valid ? p.gate[row0 + (size_t)t * p.H] : 0.f;
                const float g1 = t + 1 < valid ? p.gate[row0 + (size_t)(t + 1) * p.H] : 0.f;
                chunk_decay(g0, g1, lane, &R.g[0].x, &R.g[0].y, 2, R.eg, R.ec);
            }
            named_bar(BAR_W, NW);
            wait(&bars->g, ph);
            bool zero_key = false;  // this gate thread's key is zero: T''[t][t] = alpha_t (the forward has 0)
            float alpha = 0.f;
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
                    zero_key = t < valid && !(lam > 0.f);
                    alpha = efla_alpha(bt, lam, p.euler);
                }
                const float2 gt = R.g[tr];
#pragma unroll
                for (int s = 0; s < 32; ++s) {
                    const float2 gs = R.g[col0 + s];
                    m[s] = col0 + s < tr ? m[s] * pair_decay(gt.x, gt.y, gs.x, gs.y) : 0.f;
                }
                if (ln < C) {
                    put16(sm + OFF_L, LO_64, tr, col0, m);
                    put16(sm + OFF_L, LO_64, tr, col0 + 16, m + 16);
                }
            }
            wait(&bars->s_full, ph);
            if (ok) {  // <S, dS'>: S from its tile, dS' from HBM (the same layout; its bulk copy follows)
                const uint4 *sh = reinterpret_cast<const uint4 *>(sm + OFF_SS), *sl = sh + 2048;
                const uint4 *dh = reinterpret_cast<const uint4 *>(p.dse + (size_t)w * 65536), *dl = dh + 2048;
                float s = 0.f;
#pragma unroll
                for (int x = 0; x < 8; x += 4) {
                    uint4 a[4], b[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        a[y] = __ldcg(dh + tid + (x + y) * NW);
                        b[y] = __ldcg(dl + tid + (x + y) * NW);
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y) s += dot8(sh[tid + (x + y) * NW], sl[tid + (x + y) * NW], a[y], b[y]);
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
                if (lane == 0) R.sdot[warp] = s;
            }
            arrive(&bars->w_s);
            if (named_bar_any(BAR_W, NW, !ok)) break;  // every CUDA-core warp leaves together
            // ------------------------------ P2: R^T ------------------------------
            float gt[32];
            wait(&bars->m1a, ph);
            wait(&bars->t_full, ph);
            if (ok && zero_key) {  // u_t = alpha_t r_t for a zero key
                uint32_t h16, l16;
                split1_rn(alpha, h16, l16);
                const uint32_t off = swz_offset(ln, ln, 0);
                *reinterpret_cast<uint16_t *>(sm + OFF_W + off) = (uint16_t)h16;
                *reinterpret_cast<uint16_t *>(sm + OFF_W + LO_64 + off) = (uint16_t)l16;
            }
            if (ok) {
                // rows past the chunk's end load its last row (always in bounds) and are zeroed after, so that all
                // loads are unconditional and in flight together
                const __nv_bfloat16 *vc = p.v + row0 * D + ln;
                __nv_bfloat16 vr[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) vr[e] = __ldcg(vc + (size_t)min(col0 + e, valid - 1) * p.H * D);
#pragma unroll
                for (int e = 0; e < 32; ++e) gt[e] = __ldcg(p.g + (row0 + (size_t)min(col0 + e, valid - 1) * p.H) * D + ln);
                float r[32], xt[32], f[32];
                tmem_ld32(lane_base + TM_X + col0, xt);
                load32(R.eg + col0, f);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    r[e] = fmaf(-f[e], xt[e], col0 + e < valid ? __bfloat162float(vr[e]) : 0.f);
                    xt[e] = -r[e];
                }
                tmem_st32(lane_base + TM_X + col0, xt);
                tsplit32(lane_base, TM_RS, hf, r);
            }
            arrive(&bars->w_u);
            // ------------------------------ P3 operands ------------------------------
            wait(&bars->u, ph);
            if (ok) {
#pragma unroll
                for (int e = 0; e < 32; ++e) gt[e] = col0 + e < valid ? -gt[e] : 0.f;
                float u[32];
                tmem_ld32(lane_base + TM_U + col0, u);
                tmem_ld_wait();
                tsplit32(lane_base, TM_US, hf, u);
                put16(sm + OFF_UT, LO_UT, ln, col0, u);
                put16(sm + OFF_UT, LO_UT, ln, col0 + 16, u + 16);
                tmem_st32(lane_base + TM_U + col0, gt);  // -G^T over U^T (read above)
            }
            arrive(&bars->w_p3);
            // ------------------------------ P4: dalpha, dg, operands ------------------------------
            float s_dal = 0.f, s_a = 0.f, s_w = 0.f, s_m = 0.f, m_first = 0.f;
            {  // a_t = e^{G_t} (q_t . (S dO_t) - k_t . (S dR_t)): this warp's 32 features
                wait(&bars->m1b, ph);
                if (ok) {
                    float x[32], y[32], f[32];
                    tmem_ld32(lane_base + TM_DQ + col0, x);
                    tmem_ld32(lane_base + TM_DK + col0, y);
                    load32(R.eg + col0, f);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint8_t *kp = sm + OFF_KQ + (ln >> 6) * 16384 + swz_offset(col0 + e, ln & 63, 0);
                        const float k = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(kp) << 16);
                        const float q = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(kp + 8192) << 16);
                        x[e] = f[e] * fmaf(q, x[e], -k * y[e]);
                    }
                    s_a = lane_reduce_scatter(x, lane);
                }
            }
            wait(&bars->a, ph);
            if (ok) {  // dalpha_t = sum over j of dY^T[j][t] Z^T[j][t]
                float y[32], z[32];
                tmem_ld32(lane_base + TM_U + col0, y);
                tmem_ld32(lane_base + TM_X + col0, z);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] *= z[e];  // (both negated)
                s_dal = lane_reduce_scatter(y, lane);
            }
            wait(&bars->b, ph);
            if (ok) {
                float x[32];
                tmem_ld32(lane_base + TM_P + col0, x);
                tmem_ld_wait();
                const float2 gr = R.g[tr];
                const float sign = ln < C ? -1.f : 1.f;  // dL = -dR U^T
#pragma unroll
                for (int s = 0; s < 32; ++s) {  // M_ts = dP_ts P_ts and dL_ts L_ts, s < t (m is 0 elsewhere)
                    m[s] *= sign * x[s];
                    const float2 gs = R.g[col0 + s];
                    x[s] = col0 + s <= tr ? sign * x[s] * pair_decay(gr.x, gr.y, gs.x, gs.y) : 0.f;
                }
                if (ln < C) {  // dL' = Gamma o dL, strictly below the diagonal, row t
#pragma unroll
                    for (int s = 0; s < 32; ++s) dLs[tr * DL_LD + col0 + s] = col0 + s < tr ? x[s] : 0.f;
                } else {       // dP' = Gamma o dP, row t
                    put16(sm + OFF_W, LO_64, tr, col0, x);
                    put16(sm + OFF_W, LO_64, tr, col0 + 16, x + 16);
                }
                // exclusive prefix sums along the row (from this half's first column), where s <= t
#pragma unroll
                for (int s = 0; s < 32; ++s) {
                    const float v = m[s];
                    m[s] = col0 + s <= tr ? m_first : 0.f;
                    m_first += v;
                }
                s_m = lane_reduce_scatter(m, lane);  // columns over this warp's rows
            }
            wait(&bars->d2, ph);
            if (ok) {  // w_t = c_t k_t . (dS' u_t)
                float x[32], f[32];
                tmem_ld32(lane_base + TM_D2 + col0, x);
                load32(R.ec + col0, f);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const uint8_t *kp = sm + OFF_KQ + (ln >> 6) * 16384 + swz_offset(col0 + e, ln & 63, 0);
                    x[e] *= f[e] * __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(kp) << 16);
                }
                s_w = lane_reduce_scatter(x, lane);
                part[warp * 32 + lane] = s_dal;
                part[256 + warp * 32 + lane] = s_a;
                part[512 + warp * 32 + lane] = s_w;
                part[768 + warp * 32 + lane] = s_m;
                if (hf == 0) half_sum[ln] = m_first;
            }
            if (named_bar_any(BAR_W, NW, !ok)) break;
            {  // E = dL' + dL'^T + diag(2 dalpha dalpha/dlambda)
                const int t = tid >> 2, s0 = (tid & 3) * 16;
                const float *pd = part + (t >> 5) * 128 + (t & 31);
                const float dal = (pd[0] + pd[32]) + (pd[64] + pd[96]);
                const float dg = 2.f * dal * R.dadl[t];
                float x[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] = dLs[t * DL_LD + s0 + e] + dLs[(s0 + e) * DL_LD + t] + (s0 + e == t ? dg : 0.f);
                put16(sm + OFF_L, LO_64, t, s0, x);
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
                const float f0 = half_sum[t] + half_sum[C + t], f1 = half_sum[t + 1] + half_sum[C + t + 1];
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
                float through = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) through += R.sdot[i];
                through *= R.eg[C - 1];
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
                tmem_ld32(lane_base + TM_X + col0, dk);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) dk[e] = fmaf(-f[e], x[e], dk[e]);
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
                } else {  // (one value head a key head: Hk = H)
                    const size_t o = (row0 + (size_t)col0 * p.H) * D + ln;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (col0 + e < valid) {
                            p.dq[o + (size_t)e * p.H * D] = __float2bfloat16_rn(dq[e]);
                            p.dk[o + (size_t)e * p.H * D] = __float2bfloat16_rn(dk[e]);
                        }
                }
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
    float *g_tok = reinterpret_cast<float *>(ws + L.tok);
    void *dr_lo = g_tok + n;
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
        !bwd_row_map(&s.map_lo, dr_lo, a.B, a.T, a.H)) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    s.gate = a.g;
    s.dST = a.dST;
    s.dse = reinterpret_cast<uint8_t *>(ws + L.dse);
    s.tpp = reinterpret_cast<const uint8_t *>(ws + L.w);
    s.dS0 = a.dS0;
    s.g_out = g_tok;
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
    p.map_dv = s.map_dv;
    p.map_lo = s.map_lo;
    p.v = static_cast<const __nv_bfloat16 *>(a.v);
    p.gate = a.g;
    p.beta = a.beta;
    p.states = reinterpret_cast<const uint8_t *>(ws + L.states);
    p.dse = s.dse;
    p.tpp = s.tpp;
    p.g = g_tok;
    p.dq = static_cast<__nv_bfloat16 *>(a.dq);
    p.dk = static_cast<__nv_bfloat16 *>(a.dk);
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
