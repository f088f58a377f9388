// Helpers shared by the tcgen05 kernels: bounded mbarrier waits that also give up when
// another role of the CTA has aborted, a loop-counter barrier for the optimiser, and the
// bf16 hi/lo operand split.
#pragma once

#include "ptx.cuh"

namespace efla {
namespace tc {
namespace {  // internal to each kernel's translation unit
using namespace ptx;

// Bounded wait that also gives up when another role has aborted.  The slow
// path is out of line: it is reached rarely and the kernel's code must stay
// small enough for the instruction cache.
__device__ __noinline__ bool wait_bar_slow(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                           uint64_t limit_ns) {
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (mbar_try_wait_sleep(bar, parity, 20000)) return true;  // sleeps instead of spinning
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > limit_ns) {
            *abort_flag = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort_flag, uint64_t limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_bar_slow(bar, parity, abort_flag, limit_ns);
}
// The same for all 32 lanes of a warp, with one outcome for the whole warp: every lane
// waits, and the warp proceeds only if every lane's wait succeeded (the warp-collective
// TMEM loads and stores that follow need all lanes together).
__device__ __forceinline__ bool wait_bar_warp(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                              uint64_t limit_ns) {
    const bool ok = wait_bar(bar, parity, abort_flag, limit_ns);
    return __all_sync(0xffffffffu, ok);
}

// Hides a loop counter from the optimiser so that the loop stays rolled (the
// kernel's per-chunk code must fit the instruction cache).
__device__ __forceinline__ int opaque(int i) {
    asm volatile("" : "+r"(i));
    return i;
}

// Splits pairs x[2c], x[2c+1] into packed bf16 hi and lo words with
// x = hi + lo + e, |e| < 2^-15 |x|: hi is x truncated to bf16 (its upper 16
// bits), lo is the exact fp32 remainder x - hi truncated the same way.  Bit
// operations only (one byte permute per packed pair).
template <int NP>
__device__ __forceinline__ void split_pack(const float *x, uint32_t *hi, uint32_t *lo) {
#pragma unroll
    for (int c = 0; c < NP; ++c) {
        const uint32_t b0 = __float_as_uint(x[2 * c]), b1 = __float_as_uint(x[2 * c + 1]);
        hi[c] = __byte_perm(b0, b1, 0x7632);
        // the two remainders x - hi (exact) in one packed fp32x2 fma: hi * (-1) + x
        const float2 r = __ffma2_rn(make_float2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u)),
                                    make_float2(-1.f, -1.f), make_float2(x[2 * c], x[2 * c + 1]));
        lo[c] = __byte_perm(__float_as_uint(r.x), __float_as_uint(r.y), 0x7632);
    }
}

// The same with both parts rounded to nearest: |e| <= 2^-17 |x| (2^-18.7 in the mean square) and no bias,
// where the truncated split is up to 2^-15 off in one direction (the state it feeds is an fp32 output of
// the gated kernels).
template <int NP>
__device__ __forceinline__ void split_pack_rn(const float *x, uint32_t *hi, uint32_t *lo) {
#pragma unroll
    for (int c = 0; c < NP; ++c) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * c], x[2 * c + 1]);
        hi[c] = *reinterpret_cast<const uint32_t *>(&h);
        const float2 r = __ffma2_rn(make_float2(__uint_as_float(hi[c] << 16), __uint_as_float(hi[c] & 0xffff0000u)),
                                    make_float2(-1.f, -1.f), make_float2(x[2 * c], x[2 * c + 1]));
        const __nv_bfloat162 l = __floats2bfloat162_rn(r.x, r.y);
        lo[c] = *reinterpret_cast<const uint32_t *>(&l);
    }
}
template <bool RN, int NP>
__device__ __forceinline__ void split_as(const float *x, uint32_t *hi, uint32_t *lo) {
    if constexpr (RN)
        split_pack_rn<NP>(x, hi, lo);
    else
        split_pack<NP>(x, hi, lo);
}

// Rows row0 .. row0 + 31 of column j (this lane) of a 128 x 128 fp32 matrix, x[i] = M[row0 + i][j],
// into the operand-tile layout the backward kernels load whole: bf16 hi (truncated) in the first
// 32 KB and lo (the remainder, truncated) in the next, each as 2 column blocks of [128 rows][64]
// with the 128-byte swizzle.  Lanes j and j ^ 1 of a warp (consecutive columns) pair up: each
// shuffle hands one half to the partner, the even lane stores the hi word, the odd lane the lo
// word.  All 32 lanes take part.
__device__ __forceinline__ void put_col_split_tile(uint8_t *tile, int row0, int j, const float (&x)[32]) {
    const bool odd = (j & 1) != 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint32_t b = __float_as_uint(x[i]);
        const uint32_t h16 = b >> 16;
        const uint32_t l16 = __float_as_uint(x[i] - __uint_as_float(b & 0xffff0000u)) >> 16;
        const uint32_t recv = __shfl_xor_sync(0xffffffffu, odd ? h16 : l16, 1);
        const uint32_t word = odd ? (recv | (l16 << 16)) : (h16 | (recv << 16));
        *reinterpret_cast<uint32_t *>(tile + swz_offset(row0 + i, j & ~1, 16384) + (odd ? 32768u : 0u)) = word;
    }
}

// Tokens t0 .. t0 + 31 (x) of column j (this lane) of a [token][128] block, times `sign`, as
// bf16 hi and lo (the split above) into two arrays of that shape whose token rows are `stride`
// elements apart (hi and lo point at token 0, column 0); tokens at or past `valid` are not
// written.  Lanes j and j ^ 1 pair up as in put_col_split_tile: the even lane stores the hi
// word, the odd lane the lo word.
__device__ __forceinline__ void put_col_split_rows(__nv_bfloat16 *hi, __nv_bfloat16 *lo, size_t stride, int valid,
                                                   int t0, int j, float sign, const float (&x)[32]) {
    const bool odd = (j & 1) != 0;
    uint32_t *dst = reinterpret_cast<uint32_t *>(odd ? lo + (j - 1) : hi + j);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float v = sign * x[i];
        const uint32_t b = __float_as_uint(v);
        const uint32_t h16 = b >> 16;
        const uint32_t l16 = __float_as_uint(v - __uint_as_float(b & 0xffff0000u)) >> 16;
        const uint32_t recv = __shfl_xor_sync(0xffffffffu, odd ? h16 : l16, 1);
        if (t0 + i < valid) dst[(size_t)(t0 + i) * stride / 2] = odd ? (recv | (l16 << 16)) : (h16 | (recv << 16));
    }
}

// Four K = 16 steps of one product, issued together: one election and one block of code for the four.
// b and a (descriptors) advance by their steps in 16-byte units; the first step accumulates if `acc`.
// The kernels' roles run concurrently out of one instruction cache, so loops over these stay rolled; a
// loop over single steps took 118 cycles an MMA of 50 (election and descriptor arithmetic).
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint64_t b, uint32_t bs,
                                        uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t.reg .b32 r;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %10, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %5, %9, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %6, %9, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %7, %9, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], %8, %9, t;\n\t}" ::"r"(d),
        "r"(a0), "r"(a1), "r"(a2), "r"(a3), "l"(b), "l"(b + bs), "l"(b + 2 * bs), "l"(b + 3 * bs), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint32_t as, uint64_t b, uint32_t bs, uint32_t idesc,
                                        uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t.reg .b32 r;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %10, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %5, %9, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %6, %9, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %7, %9, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %8, %9, t;\n\t}" ::"r"(d),
        "l"(a), "l"(a + as), "l"(a + 2 * as), "l"(a + 3 * as), "l"(b), "l"(b + bs), "l"(b + 2 * bs), "l"(b + 3 * bs), "r"(idesc),
        "r"(acc)
        : "memory");
}
// D (+)= (hi + lo of A in TMEM, 64 columns each from a) B over K = 128; B K-major, column blocks `cb` bytes apart
__device__ __forceinline__ void run_ts_kmajor(uint32_t d, uint32_t a, uint64_t b, uint32_t cb, uint32_t idesc, uint32_t acc) {
#pragma unroll 1
    for (int i = 0; i < 4; i = opaque(i + 1)) {
        const uint32_t x = a + i * 32;
        mma4_ts(d, x, x + 8, x + 16, x + 24, b + (i & 1) * (cb >> 4), 2, idesc, acc | (uint32_t)i);
    }
}
// ... over K = 64: four steps of 8 TMEM columns
__device__ __forceinline__ void run_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t b_step, uint32_t idesc, uint32_t acc) {
    mma4_ts(d, a, a + 8, a + 16, a + 24, b, b_step, idesc, acc);
}
// ... with an operand of 64 tokens that was split in place, half by half: tokens 0-31 as hi in columns
// 0-15 and lo in 16-31, tokens 32-63 in columns 32-63 likewise (split_half).  a: its hi or lo.
__device__ __forceinline__ void run_ts_halves(uint32_t d, uint32_t a, uint64_t b, uint32_t b_step, uint32_t idesc, uint32_t acc) {
    mma4_ts(d, a, a + 8, a + 32, a + 40, b, b_step, idesc, acc);
}
// Gram product of a K-major tile with its first rows, K = 128
__device__ __forceinline__ void run_gram(uint32_t d, uint64_t kq, uint32_t cb, uint32_t idesc) {
#pragma unroll 1
    for (int i = 0; i < 2; i = opaque(i + 1)) mma4_ss(d, kq + i * (cb >> 4), 2, kq + i * (cb >> 4), 2, idesc, (uint32_t)i);
}
__device__ __forceinline__ void split_half(uint32_t base, int hf, const float (&x)[32]) {
    uint32_t hi[16], lo[16];
    split_pack_rn<16>(x, hi, lo);
    tmem_st16u(base + 32 * hf, hi);
    tmem_st16u(base + 32 * hf + 16, lo);
}
// Gated kernels: rows 32 g0 .. 32 g1 - 1 of the state (column j = this thread's TMEM lane, TMEM address
// ts of its transpose) times the chunk's decay el.  Out of line for the instruction cache.
__device__ __noinline__ void decay_state_rows(uint32_t ts, int g0, int g1, float el) {
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
        float sv[32];
        tmem_ld32(ts + g * 32, sv);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) sv[i] *= el;
        tmem_st32(ts + g * 32, sv);
    }
    tmem_st_wait();
}

// The gated backward's state tile: the transpose (rows j = d_v) of a 128 x 128 state as bf16 hi (32 KB),
// then lo, in core matrices without a swizzle: the 16 bytes of row j, columns 8 c .. 8 c + 7, lie at c *
// 2048 + j * 16.  A thread that owns a row then stores, and a bulk copy loads, whole lines.  As a K-major
// operand (rows j = M) its core matrices are 128 bytes apart along M and 2048 along K; as an MN-major one
// (rows j = K, columns = M) 2048 along M and 128 along K.
// Columns 32 g .. 32 g + 31 of row j, as split_pack gives them:
__device__ __forceinline__ void put_state_row(uint8_t *tile, int g, int j, const uint32_t (&hi)[16], const uint32_t (&lo)[16]) {
    uint8_t *row = tile + g * 8192 + j * 16;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        *reinterpret_cast<uint4 *>(row + q * 2048) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
        *reinterpret_cast<uint4 *>(row + 32768 + q * 2048) = make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
    }
}

// 32 values of shared memory (16-byte aligned) into registers, the same in every lane.
__device__ __forceinline__ void load32(const float *src, float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 f = reinterpret_cast<const float4 *>(src)[i];
        x[4 * i] = f.x;
        x[4 * i + 1] = f.y;
        x[4 * i + 2] = f.z;
        x[4 * i + 3] = f.w;
    }
}

}  // namespace
}  // namespace tc
}  // namespace efla
