// Backward of the gated delta rule on the sm_103a tensor cores (tcgen05 + TMEM + TMA): bf16, d_k, d_v up to
// 128 (tiles of 128, the rest zeros that TMA fills in), chunks of 64, rows of [B, T], after the training forward (chunk_tc.cu), which leaves in the
// workspace, as bf16 hi/lo operand tiles, every chunk's start state (S^T, rows = d_v) and
// T = (I + diag(alpha) L)^{-1}.  The formulas are in gated_simt.cu; here they are taken through
//   dY = T^T G,  dR = diag(alpha) dY,  U = T diag(alpha) R,
// which needs no second matrix and gives dalpha without forming Z = R - L U or keeping G:
//   dalpha_t = dY_t . Z_t = (dY U^T)_tt / alpha_t         (live_beta, live_alpha keep alpha off 0)
//
// 1. State pass (state_kernel): one CTA per (b, h) walks the chunks in reverse with dS^T fp32 in TMEM,
//    lane j = column j of d_v, everything transposed as in the forward:
//      G^T  = (dS'^T K^T) diag(c) + dO^T P       dY^T = G^T T
//      dS^T = e^{G_C} dS'^T + (dO^T diag(e^G)) Q - (dY^T diag(alpha e^G)) K
//    It writes dv = diag(alpha) dY and, as operand tiles, dS' and [dY hi; dO; dY lo] of every chunk, all but
//    dv in a layout that a thread owning a lane writes with whole lines (put_state_row).
//    The serial chain is dS' split -> dS'^T K^T -> G split -> dY -> dY split -> dS and all that the
//    state warps do; beside it the prep warps form P and diag(e^G) dO and scale the split dS' by e^{G_C}
//    in TMEM, and the output warps write everything out.
// 2. Gradient pass (grad_kernel): persistent CTAs over the (b, h, chunk) items, all independent:
//      P0  Gram [K; Q] K^T; L = Gamma o strictly-lower(K K^T) and P; <S, dS'>
//      P2  X^T = S^T K^T;  R^T = V^T - X^T diag(e^G);  U^T = (diag(alpha) R)^T T^T
//      P3  [S dY^T | S dO^T];  [dY; dO] U^T;  dS' U^T
//      P4  dalpha, dg, and the operands dP' = Gamma o dP, E = dL' + dL'^T + diag(2 dalpha dalpha/dlambda)
//      P5  dP' K;  dP'^T Q + E K
//      P6  dq = e^G (S dO^T) + dP' K,  dk = -alpha e^G (S dY^T) + c (dS' U^T) + (dP'^T Q + E K)
//    Products with different row factors keep their own accumulators and are joined where they are read
//    out.  The next item's K, Q, S and its first two products are under way while this one ends.  Sums
//    over features or rows are taken by shuffles and per-warp slots in a fixed order.
//
// 8 x 2048 tokens of 16 heads of 128 (4096 items): state pass 163 us (765 MB, 4.7 TB/s), gradient pass
// 285 us (1.1 GB, 4 TB/s).  Both are bound by the latency of their CUDA-core phases, with the memory
// traffic of the tiles between the passes not far behind: forming <S, dS'> in the state pass, which
// reads 64 KB more a chunk there, gives 197 and 270.  What they cost most was not arithmetic: register spills (the few KB of L1 left beside the operand tiles turn each into an L2
// access), code beyond the instruction cache (all roles fetch at once: unrolled MMA issue alone was 50
// KB) and scattered 16-byte accesses to HBM.  Hence the rolled issue loops, 16 columns a thread in the
// gradient pass, the update rule as a template argument, and the tile layout.
//
// dO and the inputs are exact bf16; every other operand is split into two bf16 parts rounded to nearest
// (2^-17 at most), fp32 accumulation.  Every wait is bounded; on expiry the CTA records EFLA_ERR_DEVICE_TIMEOUT
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
constexpr uint32_t OFF_DRS = OFF_TPP + 2 * TPP_BYTES;  // dv on its way to HBM, [2 cb][64 rows][64]
constexpr uint32_t OFF_DEC = OFF_DRS + 16384;      // {G whole, rest, dn, -} [64], then of four chunks e^G [64], c [64], alpha [64]
constexpr uint32_t DEC_LD = 192;
constexpr uint32_t OFF_BAR = OFF_DEC + 1024 + 4 * DEC_LD * 4;
constexpr uint32_t OFF_MISC = OFF_BAR + 256;
constexpr uint32_t SMEM_ALLOC = OFF_MISC + 16 + 1024;
static_assert(OFF_TPP % 1024 == 0 && OFF_DRS % 1024 == 0 && SMEM_ALLOC <= 232448, "shared memory layout");

constexpr uint32_t TM_S = 0;     // dS^T fp32 (128)
constexpr uint32_t TM_SA = 128;  // dS'^T hi (64) | lo (64)
constexpr uint32_t TM_X = 256;   // dS'^T K^T fp32 (64); then G^T and then -diag(alpha e^G) dY, split in place (split_half)
constexpr uint32_t TM_G = 320;   // Gram rows [K; Q] K^T fp32 (64)
constexpr uint32_t TM_G2 = 384;  // dO^T P fp32 (64); then dY^T
constexpr uint32_t TM_DO = 448;  // diag(e^G) dO hi (32) | lo (32)
constexpr int BAR_PREP = 2, BAR_OUT = 3;
constexpr int THREADS = 448;

struct Params {
    CUtensorMap map_q, map_k, map_do, map_dv;  // [B, T, heads, d] bf16, box 64 x 1 x 64 x 1, 128B swizzle
    const float *gate, *beta, *dST;
    uint8_t *dse, *rod;  // tiles of every chunk: dS'^T; dY hi, dO, dY lo
    const uint8_t *tpp;
    float *dS0;
    int *status;
    int T, H, rep, dk, dv;
    int debug_stall;
    unsigned long long wait_ns;
};

struct Bars {
    uint64_t tma_full[NSTAGE], s_free[NSTAGE];
    uint64_t g_done, g_free;
    uint64_t gate_ready[2];  // decays of a chunk written
    uint64_t prep_ready[2];  // P written and T landed
    uint64_t t_full[2], tpp_free[2];
    uint64_t do_ready;       // diag(e^G) dO written (128 arrivals)
    uint64_t sc_ready;       // dS' scaled by the prep warps (128 arrivals)
    uint64_t sa_read;        // the output warps have read the split dS' (128 arrivals)
    uint64_t y_read;         // ... and dY (128 arrivals)
    uint64_t x_done, u_done, s_done;
    uint64_t s_prep;         // as s_done, for the prep warps
    uint64_t sa_ready, r_ready, u_ready;
    uint64_t drain, never;
};
static_assert(sizeof(Bars) <= 256, "mbarrier block exceeds its slot");

// dv of tokens t0, t0 + 1 of column j (this lane) into the staging tile ([2 column blocks][64 tokens][64],
// 128-byte swizzle).  Lanes j and j ^ 1 hold neighbouring columns: each writes one token's word.
__device__ __forceinline__ void stage_pair(uint8_t *stg, int j, int t0, uint32_t v) {
    const bool odd = (j & 1) != 0;
    const uint32_t rv = __shfl_xor_sync(0xffffffffu, v, 1);
    *reinterpret_cast<uint32_t *>(stg + swz_offset(odd ? t0 + 1 : t0, j & ~1, 8192)) =
        odd ? __byte_perm(rv, v, 0x7632) : __byte_perm(v, rv, 0x5410);
}

template <bool EULER>
__global__ void __launch_bounds__(THREADS, 1) state_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars *bars = reinterpret_cast<Bars *>(sm + OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + OFF_MISC + 4);
    float *gsum = reinterpret_cast<float *>(sm + OFF_DEC), *dec = gsum + 256;

    const int tid = threadIdx.x, warp = tid >> 5;
    const uint64_t wait_ns = p.wait_ns;
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / p.rep;
    const int nchunks = (p.T + C - 1) / C;  // >= 1
    const size_t ubase = (size_t)blockIdx.x * p.dk * p.dv;
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
        mbar_init(&bars->sa_read, 128);
        mbar_init(&bars->y_read, 128);
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
        for (int e = row; e < 2 * 1024; e += 128)  // both P buffers
            *reinterpret_cast<uint4 *>(sm + OFF_TPP + (e >> 10) * TPP_BYTES + 16384 + (e & 1023) * 16) = make_uint4(0, 0, 0, 0);
        named_bar(BAR_PREP, 128);
        bool ok = true;
        for (int it = 0; it < nchunks; ++it) {
            const int buf = it & 1, st = it % NSTAGE;
            float *eg = dec + (it & 3) * DEC_LD;  // (chunk it - 4's readers are done: s_prep of chunk it - 2 was waited for)
            if (warp == 4) {
                const bool fast = chunk_decay(g0, g1, lane, gsum, gsum + 1, gsum + 2, 4, eg, eg + 64);
                if (lane == 0) gsum[3] = fast ? 1.f : 0.f;
            }
            const float bcur = bt;
            g0 = load_g(it + 1, 0);
            g1 = load_g(it + 1, 1);
            bt = load_beta(it + 1);
            ok = ok && wait_bar_warp(&bars->g_done, it & 1, abort_flag, wait_ns);
            if (it >= 2) ok = ok && wait_bar_warp(&bars->tpp_free[buf], ((it - 2) >> 1) & 1, abort_flag, wait_ns);
            tc_fence_after();
            if (ok && row < C) {  // alpha of token `row`: its lambda is the diagonal of K K^T
                float lam = 0.f;
                if (!EULER) {
                    float x[32];
                    tmem_ld32(lane_base + TM_G + (row & 32), x);
                    tmem_ld_wait();
#pragma unroll
                    for (int s = 0; s < 32; ++s) lam = s == lane ? x[s] : lam;
                }
                eg[128 + row] = writes_nothing(bcur) ? 0.f : live_alpha(bcur, lam, EULER);
            }
            if (named_bar_any(BAR_PREP, 128, !ok || *abort_flag)) {  // decays visible; also spreads an abort
                *abort_flag = 1;
                break;
            }
            if (leader) mbar_arrive(&bars->gate_ready[buf]);
            if (row >= C) {  // P = Gamma o Q K^T, inclusive lower triangle
                const int t = row - C;
                const float4 gt = reinterpret_cast<const float4 *>(gsum)[t];
                const bool fast = gsum[3] != 0.f;
                uint8_t *phi = sm + OFF_TPP + buf * TPP_BYTES + 16384;
                // (16-column blocks above a warp's rows stay the zeros they were set to at the start)
#pragma unroll 2
                for (int q = 0; q < (row >= 96 ? 4 : 2); ++q) {
                    float x[16];
                    tmem_ld16(lane_base + TM_G + 16 * q, x);
                    const float *gs = gsum + 64 * q;
                    const float up = from_quarter(gt.x, gt.y, gs[4 * DECAY_MID], gs[4 * DECAY_MID + 1]);
                    tmem_ld_wait();
                    if (fast) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] *= up * gs[4 * e + 2];
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] *= pair_decay(gt.x, gt.y, gs[4 * e], gs[4 * e + 1]);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = 16 * q + e <= t ? x[e] : 0.f;
                    put16(phi, 8192, t, 16 * q, x);
                }
            }
            tc_fence_before();
            fence_proxy_async_smem();
            named_bar(BAR_PREP, 128);
            if (leader) {
                mbar_arrive(&bars->g_free);  // the Gram rows have been read
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
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {  // dO itself -> its tile
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = __byte_perm(__float_as_uint(y[e + 2 * i]), __float_as_uint(y[e + 2 * i + 1]), 0x7632);
                        *reinterpret_cast<uint4 *>(p.rod + ((size_t)blockIdx.x * nchunks + chunk_of(it)) * 49152 + 16384 +
                                                   (4 * hf + e / 8) * 2048 + row * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
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
            // dS' times e^{G_C} in TM_S, once the state warps have read it
            ok = ok && wait_bar_warp(&bars->sa_ready, it & 1, abort_flag, wait_ns);
            if (ok) {
                tc_fence_after();
                const float el = eg[C - 1];
#pragma unroll 1
                for (int g = 0; g < 4; g = opaque(g + 1)) {
                    float sv[32];
                    tmem_ld32(lane_base + TM_S + g * 32, sv);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) sv[i] *= el;
                    tmem_st32(lane_base + TM_S + g * 32, sv);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars->sc_ready);
            }
        }
    } else if (tid >= 320) {
        // =============================== output warpgroup ===============================
        // Thread = lane = column j of d_v.
        const int lane = tid & 31, j = (warp & 3) * 32 + lane;
        uint8_t *stg = sm + OFF_DRS;
        bool ok = true;
        for (int it = 0; it < nchunks; ++it) {
            const int c = chunk_of(it);
            uint8_t *dst = p.dse + ((size_t)blockIdx.x * nchunks + c) * 65536;
            uint8_t *rod = p.rod + ((size_t)blockIdx.x * nchunks + c) * 49152 + j * 16;
            const float *al = dec + (it & 3) * DEC_LD + 128;
            ok = ok && wait_bar_warp(&bars->sa_ready, it & 1, abort_flag, wait_ns);
            if (ok) {  // dS'^T as the gradient pass's tile
                tc_fence_after();
#pragma unroll 1
                for (int g = 0; g < 4; g = opaque(g + 1)) {
                    float h[16], l[16];
                    tmem_ld16(lane_base + TM_SA + g * 16, h);
                    tmem_ld16(lane_base + TM_SA + 64 + g * 16, l);
                    tmem_ld_wait();
                    put_state_row(dst, g, j, reinterpret_cast<const uint32_t(&)[16]>(h), reinterpret_cast<const uint32_t(&)[16]>(l));
                }
                tc_fence_before();
                mbar_arrive(&bars->sa_read);
                ok = wait_bar_warp(&bars->u_done, it & 1, abort_flag, wait_ns);
                tc_fence_after();
            }
            // dY hi and lo into their tiles; dv staged and stored by TMA (rows past the end are clipped) once the
            // previous chunk's store has read the staging.  A failed wait skips the work up to this barrier, which every thread of the
            // warpgroup reaches, so that it leaves together.
            if (j == 0) bulk_wait_read0();
            if (named_bar_any(BAR_OUT, 128, !ok)) {
                ok = false;
                break;
            }
            float y[64];
            tmem_ld32(lane_base + TM_G2, *reinterpret_cast<float(*)[32]>(y));
            tmem_ld32(lane_base + TM_G2 + 32, *reinterpret_cast<float(*)[32]>(y + 32));
            tmem_ld_wait();
            tc_fence_before();
            mbar_arrive(&bars->y_read);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float *x = y + 16 * q;
                uint32_t hi[8], lo[8];
                split_pack_rn<8>(x, hi, lo);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    *reinterpret_cast<uint4 *>(rod + (2 * q + i) * 2048) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                    *reinterpret_cast<uint4 *>(rod + 32768 + (2 * q + i) * 2048) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                }
                uint8_t *d = stg + q * 2048;  // 16 tokens are two groups of 8 rows
#pragma unroll
                for (int t = 0; t < 16; t += 2) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(al[16 * q + t] * x[t], al[16 * q + t + 1] * x[t + 1]);
                    stage_pair(d, j, t, *reinterpret_cast<const uint32_t *>(&v));
                }
            }
            fence_proxy_async_smem();
            named_bar(BAR_OUT, 128);
            if (j == 0) {
                for (int cb = 0; cb * 64 < p.dv; ++cb) tma_store_4d(&p.map_dv, stg + cb * 8192, cb * 64, h, c * C, b);
                bulk_commit();
            }
        }
        if (j == 0) bulk_wait0();  // the stores have completed before the CTA leaves
        if (!ok) *abort_flag = 1;
    } else if (tid < 128) {
        // =============================== state warpgroup ===============================
        const int j = tid;
        {  // dS_T -> TMEM (dS^T: lane j holds column j)
            float r[32];
#pragma unroll 1
            for (int g = 0; g < 4; g = opaque(g + 1)) {
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = p.dST && g * 32 < p.dk && j < p.dv ? p.dST[ubase + (size_t)(g * 32 + i) * p.dv + j] : 0.f;
                tmem_st32(lane_base + TM_S + g * 32, r);
            }
            tmem_st_wait();
        }
        bool ok = true;
        for (int it = 0; it < nchunks && ok; ++it) {
            if (it > 0) ok = wait_bar_warp(&bars->s_done, (it - 1) & 1, abort_flag, wait_ns);
            const float *eg = dec + (it & 3) * DEC_LD, *ec = eg + 64, *al = eg + 128;
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
                ok = ok && wait_bar_warp(&bars->x_done, it & 1, abort_flag, wait_ns);
            }
            if (ok) {  // G^T = (dS'^T K^T) diag(c) + dO^T P, split in place
                tc_fence_after();
#pragma unroll 1
                for (int hf = 0; hf < 2; hf = opaque(hf + 1)) {
                    float x[32], y[32], f[32];
                    tmem_ld32(lane_base + TM_X + 32 * hf, x);
                    tmem_ld32(lane_base + TM_G2 + 32 * hf, y);
                    load32(ec + 32 * hf, f);
                    tmem_ld_wait();
#pragma unroll
                    for (int t = 0; t < 32; ++t) x[t] = fmaf(f[t], x[t], y[t]);
                    split_half(lane_base + TM_X, hf, x);
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
                    float x[32], f[32];
                    tmem_ld32(lane_base + TM_G2 + 32 * hf, x);
                    load32(eg + 32 * hf, f);
                    tmem_ld_wait();
#pragma unroll
                    for (int t = 0; t < 32; ++t) x[t] *= -f[t];
                    load32(al + 32 * hf, f);
#pragma unroll
                    for (int t = 0; t < 32; ++t) x[t] *= f[t];
                    split_half(lane_base + TM_X, hf, x);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars->u_ready);
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
                    for (int i = 0; i < 32; ++i)
                        if (g * 32 < p.dk && j < p.dv) p.dS0[ubase + (size_t)(g * 32 + i) * p.dv + j] = sv[i];
                }
            }
        }
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
                run_gram(tmem + TM_G, smem_desc(s_sm + (g_next % NSTAGE) * STAGE_BYTES, 16, 1024), 16384,
                         idesc_bf16_f32(128, 64, 0, 0));
                mma_commit_e(&bars->g_done);
                ++g_next;
            }
        };
        if (p.debug_stall) ok = wait_bar_warp(&bars->never, 0, abort_flag, wait_ns);
        for (int it = 0; it < nchunks && ok; ++it) {
            issue_grams(it, true);  // (the first chunk's; a later one's if it was not ready below)
            if (!ok) break;
            const int st = it % NSTAGE, buf = it & 1;
            const uint32_t kq_s = s_sm + st * STAGE_BYTES, dO_s = kq_s + OFF_DO;
            const uint32_t tp = s_sm + OFF_TPP + buf * TPP_BYTES, pb = tp + 16384;
            if (!(ok = wait_bar_warp(&bars->tma_full[st], (it / NSTAGE) & 1, abort_flag, wait_ns))) break;
            if (!(ok = wait_bar_warp(&bars->sa_ready, it & 1, abort_flag, wait_ns))) break;
            tc_fence_after();
            // dS'^T K^T (the chain)
            run_ts_kmajor(tmem + TM_X, tmem + TM_SA, smem_desc(kq_s, 16, 1024), 16384, idesc_bf16_f32(128, 64, 0, 0), 0);
            if (!(ok = wait_bar_warp(&bars->prep_ready[buf], (it >> 1) & 1, abort_flag, wait_ns))) break;
            // (TM_G2: the output warps have read the previous chunk's dY)
            if (it > 0 && !(ok = wait_bar_warp(&bars->y_read, (it - 1) & 1, abort_flag, wait_ns))) break;
            tc_fence_after();
            {  // dO^T P: dO^T (M = j) and P (N = t) read as MN-major operands, K = s
                const uint32_t idesc = idesc_bf16_f32(128, 64, 1, 1);
                const uint64_t ad = smem_desc(dO_s, 8192, 1024), bp = smem_desc(pb, 8192, 1024);
                mma4_ss(tmem + TM_G2, ad, 128, bp, 128, idesc, 0);
                mma4_ss(tmem + TM_G2, ad, 128, bp + (8192 >> 4), 128, idesc, 1);
                mma_commit_e(&bars->x_done);
            }
            if (!(ok = wait_bar_warp(&bars->r_ready, it & 1, abort_flag, wait_ns))) break;
            tc_fence_after();
            {  // dY^T = G^T T (T read as an MN-major operand, K = s), over dO^T P, which the state warps have read
                const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 1);
                const uint64_t th = smem_desc(tp, 8192, 1024);
                run_ts_halves(tmem + TM_G2, tmem + TM_X, th, 128, idesc, 0);
                run_ts_halves(tmem + TM_G2, tmem + TM_X, th + (8192 >> 4), 128, idesc, 1);
                run_ts_halves(tmem + TM_G2, tmem + TM_X + 16, th, 128, idesc, 1);
                mma_commit_e(&bars->u_done);
                mma_commit_e(&bars->tpp_free[buf]);
            }
            if (!(ok = wait_bar_warp(&bars->do_ready, it & 1, abort_flag, wait_ns))) break;
            if (!(ok = wait_bar_warp(&bars->sc_ready, it & 1, abort_flag, wait_ns))) break;
            if (!(ok = wait_bar_warp(&bars->sa_read, it & 1, abort_flag, wait_ns))) break;
            tc_fence_after();
            // dS^T += (diag(e^G) dO)^T Q, behind dY in the pipe (hi and lo: 8 K steps of adjacent columns, Q's 4 twice)
            const uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 1);
#pragma unroll 1
            for (int part = 0; part < 2; part = opaque(part + 1))
                run_ts(tmem + TM_S, tmem + TM_DO + part * 32, smem_desc(kq_s + 8192, 16384, 1024), 128, idesc_s, 1);
            issue_grams(it + 1, false);  // (the prep has read this chunk's by now)
            if (!(ok = wait_bar_warp(&bars->u_ready, it & 1, abort_flag, wait_ns))) break;
            tc_fence_after();
            {  // dS^T += (-diag(alpha e^G) dY)^T K (the chain)
#pragma unroll 1
                for (int part = 0; part < 2; part = opaque(part + 1))
                    run_ts_halves(tmem + TM_S, tmem + TM_X + part * 16, smem_desc(kq_s, 16384, 1024), 128, idesc_s, 1);
                mma_commit_e(&bars->s_done);
                mma_commit_e(&bars->s_prep);
                mma_commit_e(&bars->s_free[st]);
            }
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

constexpr int NW = 512;       // CUDA-core threads (warps 0-15)
constexpr int NTH = NW + 32;  // and the MMA / TMA warp
constexpr int BAR_W = 1;

// Shared memory (bytes).  No room is left for alignment slack: the array is declared 1024-byte aligned
// and the kernel refuses to run on another base.
constexpr uint32_t OFF_KQ = 0;         // two items' [K; Q]: 2 column blocks x 128 rows, 32 KB each
constexpr uint32_t OFF_ROD = 65536;    // [dY hi; dO], 16 chunks of 8 tokens x 128 j (the state pass's tile), 32 KB
constexpr uint32_t OFF_YL = 98304;     // dY lo, 8 such chunks, 16 KB
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
constexpr uint32_t OFF_PART = OFF_ROD + 64 * DL_LD * 4;  // fp32 [2][16 warps][32], [4 quarters][128], [2 + 4][64]
static_assert(64 * DL_LD * 4 + (2 * 16 * 32 + 512 + 6 * 64) * 4 <= 32768 && OFF_PART % 16 == 0, "scratch leaves its region");

struct RowData {
    float4 g[C];              // G_t (whole_rest) and dn_t (chunk_decay), d alpha / d beta
    float eg[C], ec[C];
    float al[C], dadl[C];
    float gate[C], beta[C];   // the next item's, copied in asynchronously
    float sdot[16];           // <S, dS'>, a warp each
};
constexpr uint32_t OFF_BAR = OFF_ROW + sizeof(RowData);
constexpr uint32_t OFF_MISC = OFF_BAR + 192;
constexpr uint32_t SMEM_ALLOC = OFF_MISC + 16;  // tmem base, abort flag, whether the item's dn may be used
static_assert(OFF_BAR % 16 == 0 && SMEM_ALLOC <= 232448, "shared memory layout");

// TMEM columns (fp32, 64 each, unless split: hi in the first 32 columns, lo in the next 32)
constexpr uint32_t TM_P = 0;     // [dY hi; dO] U^T; then (dP' K)^T
constexpr uint32_t TM_D2 = 64;   // (dS' U^T) as [feature][token]
constexpr uint32_t TM_E = 128;   // Gamma o Gram below the diagonal; then (dP'^T Q + E K)^T
constexpr uint32_t TM_RS = 192;  // (diag(alpha) R)^T split; then dY lo U^T (lanes 0-63)
constexpr uint32_t TM_U = 256;   // Gram -> U^T
constexpr uint32_t TM_X = 320;   // X^T
constexpr uint32_t TM_DK = 384;  // S dY^T, adjacent to
constexpr uint32_t TM_DQ = 448;  // S dO^T: one N = 128 product fills both

struct Params {
    CUtensorMap map_q, map_k, map_v, map_dq, map_dk;
    const float *gate, *beta;
    const uint8_t *states, *dse, *rod, *tpp;
    float *part;                   // [2][B, T, H, dk] in place of dq, dk where key heads are shared
    float *dbeta, *dg;
    size_t plane;                  // elements of one part
    int *status;
    int T, H, rep, items, dk;
    int debug_stall;
    unsigned long long wait_ns;
};

struct Bars {
    uint64_t tma_kq[2], rod_full, s_full, d_full, t_full, v_full;
    uint64_t g, m1a, m1b, u, b, d2, m2;            // products complete
    uint64_t w_s, w_u, w_p3, w_p5, w_free, w_out;  // S read / operands written / accumulators read / outputs staged (16 arrivals)
    uint64_t drain, never;
};
static_assert(sizeof(Bars) <= 192, "mbarrier block exceeds its slot");

// Sums over the 32 lanes of a warp of a[0..15] and b[0..15]: lane l < 16 returns that of a[l], lane 16 +
// l that of b[l] (31 shuffles).  a is overwritten.
__device__ __forceinline__ float reduce_pair(float (&a)[16], const float (&b)[16], int lane) {
    const bool hi = (lane & 16) != 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float send = hi ? a[i] : b[i], keep = hi ? b[i] : a[i];
        a[i] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
    }
#pragma unroll
    for (int w = 8; w >= 1; w >>= 1) {
        const bool up = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float send = up ? a[i] : a[i + w], keep = up ? a[i + w] : a[i];
            a[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
        }
    }
    return a[0];
}

// The work items w, w + gridDim.x, ... of a CTA: chunk c of head h of row b, advanced without divisions.
struct Items {
    int w, b, h, c;
    int sb, sh, sc;  // a step of gridDim.x items
    __device__ __forceinline__ Items(int w0, int step, int nc, int H) : w(w0) {
        const int u = w0 / nc, su = step / nc;
        c = w0 - u * nc, b = u / H, h = u - b * H;
        sc = step - su * nc, sb = su / H, sh = su - sb * H;
    }
    __device__ __forceinline__ void next(int step, int nc, int H) {
        w += step, c += sc, h += sh, b += sb;
        if (c >= nc) c -= nc, ++h;
        if (h >= H) h -= H, ++b;
    }
    __device__ __forceinline__ size_t row0(int T, int H) const { return ((size_t)b * T + (size_t)c * C) * H + h; }
};

__device__ __forceinline__ float bf16_at(const uint8_t *p) { return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(p) << 16); }

template <bool EULER>
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
    const int nc = (p.T + C - 1) / C, grid = (int)gridDim.x;
    const uint64_t wait_ns = p.wait_ns;
    const uint32_t s_sm = smem_u32(sm);

    if (tid == 0) {
        uint64_t *first = &bars->tma_kq[0];
        for (int i = 0; i < (int)(sizeof(Bars) / 8); ++i) {
            uint64_t *x = first + i;
            mbar_init(x, x >= &bars->w_s && x <= &bars->w_out ? NW / 32 : 1);
        }
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

    if (warp == NW / 32) {
        // ============================ MMA / TMA warp ============================
        // The whole warp runs converged; lane 0 issues copies, an elected lane the products.
        const bool leader = lane == 0;
        const uint32_t ss = s_sm + OFF_SS;
        const uint64_t rod_d = smem_desc_plain(s_sm + OFF_ROD, 128, 2048), yl_d = smem_desc_plain(s_sm + OFF_YL, 128, 2048);
        const uint64_t s_mn = smem_desc_plain(ss, 128, 2048), s_k = smem_desc_plain(ss, 2048, 128);
        const uint64_t ut_d = smem_desc(s_sm + OFF_UT, 8192, 1024), ut_k = smem_desc(s_sm + OFF_UT, 16, 1024);
        const uint64_t w_k = smem_desc(s_sm + OFF_W, 16, 1024), w_mn = smem_desc(s_sm + OFF_W, 8192, 1024);
        bool ok = true;
        // the parity of each kind of load that may still be in flight (-1: none), for the drain at the end
        int kq0_pending = -1, kq1_pending = -1, rod_pending = -1, s_pending = -1, d_pending = -1, t_pending = -1, v_pending = -1;
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
        Items N(blockIdx.x, grid, nc, p.H);         // the next item ...
        int iw = 0, ib = 0, ih = 0, ic = 0;         // ... and this one's place
        // The loop is entered a step early, as the end of an item -1: what it does there for the next item
        // starts the first one.  (One copy of that code, and none of it runs twice.)
        for (int n = -1; ok; ++n) {
            const int ph = n & 1, nx = ph ^ 1;
            const uint32_t kq = s_sm + OFF_KQ + ph * 32768, kq1 = s_sm + OFF_KQ + nx * 32768;
            const bool more = N.w < p.items;
            if (n < 0 && p.debug_stall && !(ok = wait_bar_warp(&bars->never, 0, abort_flag, wait_ns))) break;
            if (more) {  // (that buffer's last products, item n - 1's, are complete)
                if (leader) {
                    uint64_t *bar = &bars->tma_kq[nx];
                    mbar_arrive_expect_tx(bar, 2 * 16384);
                    const int hk = N.h / p.rep;
                    for (int cb = 0; cb < 2; ++cb) {
                        uint8_t *dst = sm + OFF_KQ + nx * 32768 + cb * 16384;
                        tma_load_4d(dst, &p.map_k, bar, cb * 64, hk, N.c * C, N.b);
                        tma_load_4d(dst + 8192, &p.map_q, bar, cb * 64, hk, N.c * C, N.b);
                    }
                    // dS' of that item is read from the L2 twice, and soon
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.dse + (size_t)N.w * 65536), "r"(65536) : "memory");
                }
                (nx ? kq1_pending : kq0_pending) = ((n + 1) >> 1) & 1;
                __syncwarp();
            }
            if (n >= 0) {
                if (!wait(&bars->rod_full, ph)) break;
                rod_pending = -1;
                if (n > 0 && !wait(&bars->w_free, nx)) break;  // the previous item's results are read out
                {  // [S dY^T | S dO^T]: S read from the S^T tile as an MN-major A, K = j; dY lo only against S hi
                    const uint32_t id128 = idesc_bf16_f32(128, 128, 1, 1), id64 = idesc_bf16_f32(128, 64, 1, 1);
#pragma unroll 1
                    for (int i = 0; i < 4; i = opaque(i + 1))
                        mma4_ss(tmem + TM_DK, s_mn + (i >> 1) * (LO_128 >> 4) + (i & 1) * 64, 16, rod_d + (i & 1) * 64, 16, id128, i);
#pragma unroll 1
                    for (int i = 0; i < 2; i = opaque(i + 1)) mma4_ss(tmem + TM_DK, s_mn + i * 64, 16, yl_d + i * 64, 16, id64, 1);
                    mma_commit_e(&bars->m1b);
                }
                if (!wait(&bars->m1b, ph) || !wait(&bars->w_s, ph)) break;  // S is read: dS' replaces it
                load_tile(&bars->d_full, OFF_SS, p.dse + (size_t)iw * 65536, 65536);
                d_pending = ph;
                if (!wait(&bars->t_full, ph)) break;
                t_pending = -1;
                if (!wait(&bars->w_u, ph)) break;  // V read, (diag(alpha) R)^T written
                v_pending = -1;
                {  // U^T = (diag(alpha) R)^T T^T
                    const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 0);
#pragma unroll 1
                    for (int i = 0; i < 3; i = opaque(i + 1))  // hi x hi, hi x lo, lo x hi
                        run_ts(tmem + TM_U, tmem + TM_RS + (i == 2 ? 32 : 0), w_k + (i == 1 ? LO_64 >> 4 : 0), 2, idesc, i);
                    mma_commit_e(&bars->u);
                }
                if (!wait(&bars->w_p3, ph)) break;  // U^T tile written
                {  // [dY hi; dO] U^T and (into TM_RS, rows 0-63 meant) dY lo U^T: B[t][j] = U^T[j][t] (MN-major)
                    const uint32_t idesc = idesc_bf16_f32(128, 64, 1, 1);
#pragma unroll 1
                    for (int i = 0; i < 4; i = opaque(i + 1))
                        mma4_ss(tmem + TM_P, rod_d + (i & 1) * 64, 16, ut_d + (i >> 1) * (LO_UT >> 4) + (i & 1) * 512, 128, idesc, i);
#pragma unroll 1
                    for (int i = 0; i < 2; i = opaque(i + 1)) mma4_ss(tmem + TM_RS, yl_d + i * 64, 16, ut_d + i * 512, 128, idesc, i);
                    mma_commit_e(&bars->b);
                }
                if (!wait(&bars->d_full, ph)) break;
                d_pending = -1;
                {  // dS' U^T: dS' read from the dS'^T tile as an MN-major A
                    const uint32_t idesc = idesc_bf16_f32(128, 64, 1, 1);
#pragma unroll 1
                    for (int i = 0; i < 6; i = opaque(i + 1)) {  // hi x hi, hi x lo, lo x hi
                        const int pr = i >> 1;
                        mma4_ss(tmem + TM_D2, s_mn + (pr == 2 ? LO_128 >> 4 : 0) + (i & 1) * 64, 16,
                                ut_d + (pr == 1 ? LO_UT >> 4 : 0) + (i & 1) * 512, 128, idesc, i);
                    }
                    mma_commit_e(&bars->d2);
                }
            }
            if (more) {  // Gram [K; Q] K^T of the next item into TM_U
                if (!wait(&bars->tma_kq[nx], ((n + 1) >> 1) & 1)) break;
                (nx ? kq1_pending : kq0_pending) = -1;
                run_gram(tmem + TM_U, smem_desc(kq1, 16, 1024), 16384, idesc_bf16_f32(128, 64, 0, 0));
                mma_commit_e(&bars->g);
            }
            if (n >= 0 && !wait(&bars->d2, ph)) break;
            if (more) {
                load_tile(&bars->s_full, OFF_SS, p.states + (size_t)N.w * 65536, 65536);
                s_pending = nx;
            }
            if (n >= 0) {
                if (!wait(&bars->w_p5, ph)) break;  // dP' and E written, the accumulators below read
                // (dP' K)^T = K^T dP'^T;  (dP'^T Q + E K)^T = Q^T dP' + K^T E
                const uint32_t id_kn = idesc_bf16_f32(128, 64, 1, 0), id_mn = idesc_bf16_f32(128, 64, 1, 1);
                const uint64_t kt = smem_desc(kq, 16384, 1024), qt = smem_desc(kq + 8192, 16384, 1024);
#pragma unroll 1
                for (int i = 0; i < 2; i = opaque(i + 1)) {
                    const uint32_t lo = i * (LO_64 >> 4);
                    mma4_ss(tmem + TM_P, kt, 128, w_k + lo, 2, id_kn, i);     // dP'[t][s]
                    mma4_ss(tmem + TM_E, qt, 128, w_mn + lo, 128, id_mn, i);  // dP'[s][t]
                    mma4_ss(tmem + TM_E, kt, 128, ut_k + lo, 2, id_kn, 1);    // E[t][s]
                }
                mma_commit_e(&bars->m2);
            }
            if (more) {  // X^T = S^T K^T of the next item (tile rows = d_v: a K-major A)
                if (!wait(&bars->s_full, nx)) break;
                s_pending = -1;
                const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 0);
#pragma unroll 1
                for (int i = 0; i < 4; i = opaque(i + 1))
                    mma4_ss(tmem + TM_X, s_k + (i >> 1) * (LO_128 >> 4) + (i & 1) * 1024, 256, smem_desc(kq1, 16, 1024) + (i & 1) * 1024, 2,
                            idesc, i);
                mma_commit_e(&bars->m1a);
            }
            if (n >= 0 && !wait(&bars->m2, ph)) break;
            if (more) {
                load_tile(&bars->t_full, OFF_W, p.tpp + (size_t)N.w * 16384, 16384);
                load_tile(&bars->rod_full, OFF_ROD, p.rod + (size_t)N.w * 49152, 49152);
                t_pending = rod_pending = nx;
            }
            if (n >= 0) {
                if (!wait(&bars->w_out, ph)) break;  // dq and dk staged (or written)
                if (leader && !p.part) {
                    for (int cb = 0; cb * 64 < p.dk; ++cb) {  // (rows past the sequence end are clipped)
                        tma_store_4d(&p.map_dq, sm + OFF_UT + cb * 8192, cb * 64, ih, ic * C, ib);
                        tma_store_4d(&p.map_dk, sm + OFF_UT + 16384 + cb * 8192, cb * 64, ih, ic * C, ib);
                    }
                    bulk_commit();
                    bulk_wait_read0();
                }
                __syncwarp();
            }
            if (!more) break;
            if (leader) {
                mbar_arrive_expect_tx(&bars->v_full, 2 * 8192);
                for (int cb = 0; cb < 2; ++cb) tma_load_4d(sm + OFF_V + cb * 8192, &p.map_v, &bars->v_full, cb * 64, N.h, N.c * C, N.b);
            }
            v_pending = nx;
            __syncwarp();
            iw = N.w, ib = N.b, ih = N.h, ic = N.c;
            N.next(grid, nc, p.H);
        }
        if (!ok) *abort_flag = 1;
        // every product, load and store issued has completed before TMEM and the CTA go (bounded)
        mma_commit_e(&bars->drain);
        if (leader) {
            const uint64_t ts = globaltimer_ns();
            auto settle = [&](uint64_t *bar, int parity) {
                while (parity >= 0 && !mbar_try_wait_sleep(bar, parity, 20000) && globaltimer_ns() - ts < DRAIN_NS) {
                }
            };
            settle(&bars->drain, 0);
            settle(&bars->tma_kq[0], kq0_pending);
            settle(&bars->tma_kq[1], kq1_pending);
            settle(&bars->rod_full, rod_pending);
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
        // sums by warp: part[0]: a (lanes 0-15, a token each) and w (lanes 16-31); part[1]: M's columns (lanes 0-15)
        float *part = reinterpret_cast<float *>(sm + OFF_PART);
        float *rsum = part + 2 * 16 * 32;  // [4 quarters][128]: row sums of M within a quarter of columns
        float *tok = rsum + 512;           // [64] each: a, w, the rows' sums over the quarters before quarter 1, 2, 3, dY . U
        // TMEM: this thread reads and writes lane `ln`, the columns of token quarter `qt`
        const int qt = warp >> 2, ln = (warp & 3) * 32 + lane, col0 = 16 * qt;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const bool gate_thr = ln < C && (ln >> 4) == qt;  // holds the diagonal of row t = ln
        const int tr = ln & (C - 1);                      // the row of this thread in the C x C matrices
        const bool above = (tr | 31) < col0;              // (whole warps) every entry above the diagonal
        volatile int *fast_flag = reinterpret_cast<volatile int *>(sm + OFF_MISC + 8);
        // element (token col0 + e, feature ln) of a [tokens][128] tile whose column blocks are `cb` bytes apart
        auto feat = [&](int e, uint32_t cb) { return (uint32_t)(ln >> 6) * cb + qt * 2048u + swz_offset(e, ln & 63, 0); };
        auto load16 = [&](const float *src, float (&x)[16]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = reinterpret_cast<const float4 *>(src + col0)[i];
                x[4 * i] = f.x;
                x[4 * i + 1] = f.y;
                x[4 * i + 2] = f.z;
                x[4 * i + 3] = f.w;
            }
        };
        // x[e] *= Gamma of row tr and column col0 + e (entries above the diagonal: anything)
        auto times_gamma = [&](float (&x)[16]) {
            const float4 gt = R.g[tr];
            if (*fast_flag) {
                const float4 gm = R.g[col0 + DECAY_MID];
                const float up = from_quarter(gt.x, gt.y, gm.x, gm.y);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] *= up * R.g[col0 + e].z;
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float4 gs = R.g[col0 + e];
                    x[e] *= pair_decay(gt.x, gt.y, gs.x, gs.y);
                }
            }
        };
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
        auto copy4 = [&](float *dst, const float *src, bool there) {  // (zero if not there)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 4 : 0) : "memory");
        };
        // gates and step sizes on their way into R.gate and R.beta (threads 0-63 and 64-127, tokens past the end as
        // zeros), an item ahead
        auto copy_gates = [&](const Items &X) {
            if (X.w < p.items && tid < 2 * C) {
                const int t = tid & (C - 1);
                const bool there = X.c * C + t < p.T;
                const float *src = (tid < C ? p.gate : p.beta) + X.row0(p.T, p.H) + (there ? (size_t)t * p.H : 0);
                copy4(tid < C ? &R.gate[t] : &R.beta[t], src, there);
            }
        };
        Items I(blockIdx.x, grid, nc, p.H);
        copy_gates(I);
        for (; I.w < p.items; I.next(grid, nc, p.H), ++it) {
            const int ph = it & 1;
            const int valid = min(C, p.T - I.c * C);
            const size_t row0 = I.row0(p.T, p.H);
            const uint8_t *KQ = sm + OFF_KQ + ph * 32768;
            // ------------------------------ P0: decays, <S, dS'>, gate terms, L and P ------------------------------
            asm volatile("cp.async.wait_all;" ::: "memory");
            named_bar(BAR_W, NW);  // every warp is done with the previous item's row data; this one's gates are in
            const float bt = gate_thr ? live_beta(R.beta[ln]) : 0.f;
            if (warp == 15) {
                float *gs = reinterpret_cast<float *>(R.g);
                const bool fast = chunk_decay(R.gate[2 * lane], R.gate[2 * lane + 1], lane, gs, gs + 1, gs + 2, 4, R.eg, R.ec);
                if (lane == 0) *fast_flag = fast;
            }
            {  // <S, dS'>, 32 elements a thread: S from its tile, dS' from HBM (the same layout)
                const uint4 *dh = reinterpret_cast<const uint4 *>(p.dse + (size_t)I.w * 65536) + tid;
                uint4 d[4];
                float2 s2 = make_float2(0.f, 0.f);
                auto both = [](uint32_t x, uint32_t y) {  // hi + lo of a pair
                    return __fadd2_rn(make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)),
                                      make_float2(__uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u)));
                };
#pragma unroll 1
                for (int x = 0; x < 4; x = opaque(x + 2)) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        d[2 * y] = __ldcg(dh + (x + y) * NW);
                        d[2 * y + 1] = __ldcg(dh + 2048 + (x + y) * NW);
                    }
                    if (x == 0) wait(&bars->s_full, ph);
                    const uint4 *sh = reinterpret_cast<const uint4 *>(sm + OFF_SS) + tid;
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint4 a = sh[(x + y) * NW], b = sh[2048 + (x + y) * NW];
                        s2 = __ffma2_rn(both(a.x, b.x), both(d[2 * y].x, d[2 * y + 1].x), s2);
                        s2 = __ffma2_rn(both(a.y, b.y), both(d[2 * y].y, d[2 * y + 1].y), s2);
                        s2 = __ffma2_rn(both(a.z, b.z), both(d[2 * y].z, d[2 * y + 1].z), s2);
                        s2 = __ffma2_rn(both(a.w, b.w), both(d[2 * y].w, d[2 * y + 1].w), s2);
                    }
                }
                float s = s2.x + s2.y;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
                if (lane == 0) R.sdot[warp] = s;
                if (ok) arrive(&bars->w_s);
            }
            named_bar(BAR_W, NW);
            {
                Items X = I;
                X.next(grid, nc, p.H);
                copy_gates(X);
            }
            wait(&bars->g, ph);
            if (ok) {  // Gamma o Gram of row tr, this quarter's columns: L (ln < 64) or P, strictly below the diagonal
                float m[16];
                tmem_ld16(lane_base + TM_U + col0, m);
                tmem_ld_wait();
                if (gate_thr) {
                    if (EULER) {
                        R.al[ln] = bt;
                    } else {
                        float lam = 0.f, db, dl;
#pragma unroll
                        for (int s = 0; s < 16; ++s) lam = (s == (ln & 15)) ? m[s] : lam;
                        gate_grad(bt, lam, 0, db, dl);
                        R.g[ln].w = db;
                        R.dadl[ln] = dl;
                        R.al[ln] = live_alpha(bt, lam, 0);
                    }
                }
                if (!above) {
                    times_gamma(m);
#pragma unroll
                    for (int s = 0; s < 16; ++s) m[s] = col0 + s < tr ? m[s] : 0.f;
                    tmem_st16(lane_base + TM_E + col0, m);  // until P4
                    tmem_st_wait();
                }
            }
            if (named_bar_any(BAR_W, NW, !ok)) break;  // every CUDA-core warp leaves together
            // ------------------------------ P2: R^T ------------------------------
            wait(&bars->v_full, ph);
            wait(&bars->m1a, ph);
            if (ok) {
                float r[16], f[16];
                tmem_ld16(lane_base + TM_X + col0, r);
                load16(R.eg, f);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) r[e] = fmaf(-f[e], r[e], bf16_at(sm + OFF_V + feat(e, 8192)));
                load16(R.al, f);
#pragma unroll
                for (int e = 0; e < 16; ++e) r[e] *= f[e];
                uint32_t hh[8], ll[8];
                split_pack_rn<8>(r, hh, ll);
                tmem_st8u(lane_base + TM_RS + 8 * qt, hh);
                tmem_st8u(lane_base + TM_RS + 32 + 8 * qt, ll);
                arrive(&bars->w_u);
            }
            // ------------------------------ P3: the U^T tile ------------------------------
            wait(&bars->u, ph);
            if (ok) {
                float x[16];
                tmem_ld16(lane_base + TM_U + col0, x);
                tmem_ld_wait();
                put16(sm + OFF_UT, LO_UT, ln, col0, x);
                arrive(&bars->w_p3);
            }
            // ------------------------------ P4: dalpha, dg, operands ------------------------------
            wait(&bars->b, ph);
            if (ok) {
                float mm[16], x[16];
                float total = 0.f;
                if (!above) {
                    tmem_ld16(lane_base + TM_P + col0, x);
                    if (ln < C) {  // (whole warps) dY lo U^T joins
                        tmem_ld16(lane_base + TM_RS + col0, mm);
                        tmem_ld_wait();
#pragma unroll
                        for (int s = 0; s < 16; ++s) x[s] += mm[s];
                    }
                    float m[16];
                    tmem_ld16(lane_base + TM_E + col0, m);
                    tmem_ld_wait();
                    // dalpha_t = (dY U^T)_tt / alpha_t: the diagonal by predicated stores (a branch that few threads take
                    // costs more than its instructions: its code is cold each time)
#pragma unroll
                    for (int s = 0; s < 16; ++s)
                        if (col0 + s == ln) tok[5 * C + ln] = x[s];
                    // dL = -diag(alpha) (dY U^T): M_ts = dP_ts P_ts and dL_ts L_ts (s < t; m is 0 elsewhere); exclusive prefix
                    // sums along the row, from this quarter's first column
                    const float fac = ln < C ? -R.al[tr] : 1.f;
#pragma unroll
                    for (int s = 0; s < 16; ++s) {
                        x[s] *= fac;
                        const float v = m[s] * x[s];
                        mm[s] = col0 + s <= tr ? total : 0.f;
                        total += v;
                    }
                    times_gamma(x);
                } else {
#pragma unroll
                    for (int s = 0; s < 16; ++s) mm[s] = 0.f;
                }
                rsum[qt * 128 + ln] = total;
                if (ln < C) {  // dL' = Gamma o dL, strictly below the diagonal, row t
#pragma unroll
                    for (int s = 0; s < 16; ++s) dLs[tr * DL_LD + col0 + s] = col0 + s < tr ? x[s] : 0.f;
                } else {       // dP' = Gamma o dP, row t
#pragma unroll
                    for (int s = 0; s < 16; ++s) x[s] = col0 + s <= tr ? x[s] : 0.f;
                    put16(sm + OFF_W, LO_64, tr, col0, x);
                }
                part[512 + warp * 32 + lane] = reduce_pair(mm, mm, lane);  // columns over this warp's rows
            }
            wait(&bars->d2, ph);
            if (ok) {  // a_t = e^{G_t} (q_t . (S dO_t) - alpha_t k_t . (S dY_t)) and w_t = c_t k_t . (dS' u_t)
                float x[16], v[16], y[16], f[16];
                tmem_ld16(lane_base + TM_DQ + col0, x);
                tmem_ld16(lane_base + TM_DK + col0, y);
                tmem_ld16(lane_base + TM_D2 + col0, v);
                load16(R.al, f);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint8_t *kp = KQ + feat(e, 16384);
                    const float k = bf16_at(kp);
                    x[e] = fmaf(bf16_at(kp + 8192), x[e], -f[e] * y[e] * k);
                    v[e] *= k;
                }
                const float s = reduce_pair(x, v, lane);
                part[warp * 32 + lane] = (lane < 16 ? R.eg : R.ec)[col0 + (lane & 15)] * s;
            }
            if (named_bar_any(BAR_W, NW, !ok)) break;
            {  // E = dL' + dL'^T + diag(2 dalpha dalpha/dlambda)
                const int t = tid >> 3, s0 = (tid & 7) * 8;
                float dg = 0.f;
                if (!EULER) dg = 2.f * __fdividef(tok[5 * C + t], R.al[t]) * R.dadl[t];
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = dLs[t * DL_LD + s0 + e] + dLs[(s0 + e) * DL_LD + t] + (s0 + e == t ? dg : 0.f);
                uint32_t hh[4], ll[4];
                split_pack_rn<4>(x, hh, ll);
                const uint32_t off = swz_offset(t, s0, 0);
                *reinterpret_cast<uint4 *>(sm + OFF_UT + off) = make_uint4(hh[0], hh[1], hh[2], hh[3]);
                *reinterpret_cast<uint4 *>(sm + OFF_UT + LO_64 + off) = make_uint4(ll[0], ll[1], ll[2], ll[3]);
            }
            if (tid < 2 * C) {  // tok: a and w over the warps
                const int t = tid & (C - 1);
                const float *x = part + (t >> 4) * 128 + (t & 15) + (tid < C ? 0 : 16);
                tok[tid] = (x[0] + x[32]) + (x[64] + x[96]);
            } else if (tid < 3 * C) {  // ... and each row's sums over the quarters before quarter 1, 2, 3
                const int r = tid & (C - 1);
                float s = 0.f;
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    s += rsum[q * 128 + r] + rsum[q * 128 + C + r];
                    tok[(2 + q) * C + r] = s;
                }
            }
            named_bar(BAR_W, NW);
            {  // dg_t: eight rows r a thread, a_r and what row r holds in the quarters before t's where r >= t, else w_r
                const int t = tid >> 3, q = t >> 4;
                const float *before = tok + (1 + q) * C;  // (used for q > 0)
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = (tid & 7) + 8 * e;
                    float v = tok[r >= t ? r : C + r];
                    if (q > 0 && r >= t) v += before[r];
                    s += v;
                }
                // ... and of M's columns, the through sum: two warps' entries a thread
                const int k = tid & 7;
                if (k < 4) s += part[512 + (4 * q + k) * 32 + (t & 15)];
                s = fmaf(R.eg[C - 1], R.sdot[2 * k] + R.sdot[2 * k + 1], s);
#pragma unroll
                for (int off = 1; off < 8; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
                if (k == 0 && t < valid) {
                    const float dal = __fdividef(tok[5 * C + t], R.al[t]);
                    p.dbeta[row0 + (size_t)t * p.H] = EULER ? dal : dal * R.g[t].w;
                    p.dg[row0 + (size_t)t * p.H] = s;
                }
            }
            arrive(&bars->w_p5);
            // ------------------------------ P6 ------------------------------
            wait(&bars->m2, ph);
            if (ok) {
                float dq[16], dk[16], x[16], f[16];
                tmem_ld16(lane_base + TM_DQ + col0, dq);
                tmem_ld16(lane_base + TM_P + col0, x);
                load16(R.eg, f);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) dq[e] = fmaf(f[e], dq[e], x[e]);
                tmem_ld16(lane_base + TM_DK + col0, x);
                tmem_ld16(lane_base + TM_E + col0, dk);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] *= -f[e];
                load16(R.al, f);
#pragma unroll
                for (int e = 0; e < 16; ++e) dk[e] = fmaf(f[e], x[e], dk[e]);
                tmem_ld16(lane_base + TM_D2 + col0, x);
                load16(R.ec, f);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->w_free);  // everything is in registers
#pragma unroll
                for (int e = 0; e < 16; ++e) dk[e] = fmaf(f[e], x[e], dk[e]);
                if (p.part) {
                    float *o = p.part + (row0 + (size_t)col0 * p.H) * p.dk + ln;
                    const size_t step = (size_t)p.H * p.dk;
#pragma unroll
                    for (int e = 0; e < 16; ++e, o += step)
                        if (col0 + e < valid && ln < p.dk) {
                            o[0] = dq[e];
                            o[p.plane] = dk[e];
                        }
                } else {  // staged as bf16 tiles; lanes ln and ln ^ 1 pair up, the even one writes dq, the odd one dk
                    const bool odd = (lane & 1) != 0;
                    uint8_t *dst = sm + OFF_UT + (odd ? 16384 : 0) + (ln >> 6) * 8192 + qt * 2048;
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
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
    const size_t n = (size_t)a.B * a.T * a.H * a.dk_dim;
    const bool euler = a.euler != 0;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) {
        *why = "querying the SM count";
        return e;
    }
    static bool done[4][64] = {};
    e = euler ? allow_smem(st::state_kernel<true>, st::SMEM_ALLOC, dev, done[0]) : allow_smem(st::state_kernel<false>, st::SMEM_ALLOC, dev, done[1]);
    if (e == cudaSuccess)
        e = euler ? allow_smem(gr::grad_kernel<true>, gr::SMEM_ALLOC, dev, done[2]) : allow_smem(gr::grad_kernel<false>, gr::SMEM_ALLOC, dev, done[3]);
    if (e != cudaSuccess) {
        *why = "setting the gated backward kernels' shared memory";
        return e;
    }
    st::Params s;
    gr::Params p;
    memset(&s, 0, sizeof s);
    memset(&p, 0, sizeof p);
    const int B = a.B, T = a.T, dk = a.dk_dim, dv = a.dv_dim;
    if (!bwd_row_map(&s.map_q, a.q, B, T, a.Hk, dk) || !bwd_row_map(&s.map_k, a.k, B, T, a.Hk, dk) ||
        !bwd_row_map(&s.map_do, a.dO, B, T, a.H, dv) || !bwd_row_map(&s.map_dv, a.dv, B, T, a.H, dv) ||
        !bwd_row_map(&p.map_v, a.v, B, T, a.H, dv) || !bwd_row_map(&p.map_dq, a.dq, B, T, a.Hk, dk) ||
        !bwd_row_map(&p.map_dk, a.dk, B, T, a.Hk, dk)) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    s.gate = a.g;
    s.beta = a.beta;
    s.dST = a.dST;
    s.dse = reinterpret_cast<uint8_t *>(ws + L.dse);
    s.rod = reinterpret_cast<uint8_t *>(ws + L.tok);
    s.tpp = reinterpret_cast<const uint8_t *>(ws + L.w);
    s.dS0 = a.dS0;
    s.status = a.status;
    s.T = a.T;
    s.H = a.H;
    s.rep = a.H / a.Hk;
    s.dk = dk;
    s.dv = dv;
    s.wait_ns = wait_limit_ns();
    s.debug_stall = (debug_stall() & STALL_BWD_STATE) ? 1 : 0;
    *why = "tcgen05 gated state-gradient kernel launch";
    (euler ? st::state_kernel<true> : st::state_kernel<false>)<<<(unsigned)units, st::THREADS, st::SMEM_ALLOC, a.stream>>>(s);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    p.map_q = s.map_q;
    p.map_k = s.map_k;
    p.gate = a.g;
    p.beta = a.beta;
    p.states = reinterpret_cast<const uint8_t *>(ws + L.states);
    p.dse = s.dse;
    p.rod = s.rod;
    p.tpp = s.tpp;
    p.part = a.Hk == a.H ? nullptr : reinterpret_cast<float *>(ws + L.part);
    p.plane = n;
    p.dbeta = a.dbeta;
    p.dg = a.dg;
    p.status = a.status;
    p.T = a.T;
    p.H = a.H;
    p.rep = s.rep;
    p.dk = dk;
    p.items = (int)items;
    p.wait_ns = s.wait_ns;
    p.debug_stall = (debug_stall() & STALL_BWD_GRAD) ? 1 : 0;
    *why = "tcgen05 gated gradient kernel launch";
    (euler ? gr::grad_kernel<true> : gr::grad_kernel<false>)<<<(unsigned)std::min<long>(items, sms), gr::NTH, gr::SMEM_ALLOC, a.stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess || !p.part) return e;
    *why = "gated head-sum kernel launch";
    return launch_gated_reduce_heads(a, p.part);
}

}  // namespace efla
