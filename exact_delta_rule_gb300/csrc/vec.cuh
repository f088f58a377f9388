// 16-byte vectors of bf16 or fp32 as fp32 values, and sums over the lanes of a row.
#pragma once

#include "internal.cuh"

namespace efla {

template <typename T>
struct Vec;  // 16 bytes of T as fp32 values
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&x)[4]) {
        x[0] = __uint_as_float(r.x);
        x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z);
        x[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&x)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// 1 / (1 + e^{-x}) to 2 + 1.2 |x| ulp, as the output gate's; 0 for -infinity.
__device__ __forceinline__ float quick_sigmoid(float x) {
    float e, y;  // (flushing denormals is exact here and saves the scaling around both instructions)
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-x * 1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + e));
    return y;
}

// The same for two, packed.
__device__ __forceinline__ float2 quick_sigmoid(float2 x) {
    const float2 t = __fmul2_rn(x, make_float2(-1.44269504f, -1.44269504f));
    float2 e, y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    e = __fadd2_rn(e, make_float2(1.f, 1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(e.y));
    return y;
}

// Sum over the LPR lanes that hold a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// An asynchronous copy of 16 or 8 bytes into this thread's slot of shared memory; zeros where it is not live.
template <typename P>
__device__ __forceinline__ void fetch(P *dst, const P *src, bool live) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (sizeof(P) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(live ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(src), "r"(live ? 8 : 0) : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most `left` (0 to 3) of the latest groups are under way.
__device__ __forceinline__ void fetch_wait(int left) {
    if (left >= 3)
        asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (left == 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (left == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Lets a kernel have `bytes` of dynamic shared memory.  Without that the most is 48 KB together with what it declares
// itself (under 1 KB in every kernel launched so).
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
    return bytes > 47 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) : cudaSuccess;
}

}  // namespace efla
