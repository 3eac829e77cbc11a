// fp8z_elem.cuh -- 16-byte vectors of FP32, BF16 and FP16 elements, widened to
// and rounded from FP32 (round to nearest even), for the kernels around the
// optimizer step.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fp8z.h"

namespace fp8z {

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kCode = FP8Z_F32;
    static __device__ __forceinline__ float widen(float x) { return x; }
    static __device__ __forceinline__ float narrow(float x) { return x; }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kCode = FP8Z_BF16;
    static __device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 narrow(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<__half> {
    static constexpr int kCode = FP8Z_F16;
    static __device__ __forceinline__ float widen(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half narrow(float x) { return __float2half_rn(x); }
};

// N consecutive elements from a 16-byte-aligned address, through the
// non-coherent path.  Volatile, like every load here that the compiler might
// take for one of constant memory: a kernel may be set up before its inputs are
// written (fp8z_launch.cuh), and no load may move before its wait.
template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Pack {
    T v[N];
};

__device__ __forceinline__ uint4 ld_nc_16(const void* p) {
    uint4 u;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p)
                 : "memory");
    return u;
}

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> ld_nc(const T* p) {
    static_assert(sizeof(T) * N % 16 == 0, "whole 16-byte vectors");
    Pack<T, N> r;
    uint4* u = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < int(sizeof(T) * N / 16); ++i) u[i] = ld_nc_16(reinterpret_cast<const uint4*>(p) + i);
    return r;
}

// The same for memory that this kernel also writes (accumulation in place).
template <typename T, int N>
__device__ __forceinline__ Pack<T, N> ld_plain(const T* p) {
    Pack<T, N> r;
    uint4* u = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < int(sizeof(T) * N / 16); ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    return r;
}

template <typename T, int N>
__device__ __forceinline__ void st_vec(T* p, const Pack<T, N>& r) {
    const uint4* u = reinterpret_cast<const uint4*>(&r);
#pragma unroll
    for (int i = 0; i < int(sizeof(T) * N / 16); ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
}

// What is read for the last time, or written and not read again soon: loads that
// do not stay in L1 and bring a 256-byte line pair into L2, stores that leave L2 first.
__device__ __forceinline__ uint4 ld_stream_16(const void* p, int i) {      // the i-th 16 bytes from p
    uint4 u;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(static_cast<const uint4*>(p) + i)
                 : "memory");
    return u;
}

// Eight elements; `wide`: the address is a multiple of 32 bytes too, and FP32 goes
// out in one store, which writes whole 32-byte sectors.
template <typename T>
__device__ __forceinline__ void st_stream8(T* p, const Pack<T, 8>& r, bool wide) {
    const uint4* u = reinterpret_cast<const uint4*>(&r);
    if constexpr (sizeof(T) == 4) {
        if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0].x), "r"(u[0].y),
                         "r"(u[0].z), "r"(u[0].w), "r"(u[1].x), "r"(u[1].y), "r"(u[1].z), "r"(u[1].w)
                         : "memory");
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) __stcs(reinterpret_cast<uint4*>(p) + i, u[i]);
}

inline bool dtype_ok(int32_t d) { return d == FP8Z_F32 || d == FP8Z_BF16 || d == FP8Z_F16; }
inline int dtype_bytes(int32_t d) { return d == FP8Z_F32 ? 4 : 2; }

}  // namespace fp8z
