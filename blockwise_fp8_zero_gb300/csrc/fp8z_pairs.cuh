// fp8z_pairs.cuh -- two FP32 numbers in one register pair, and the packed instructions that
// take both at once.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fp8z_elem.cuh"

namespace fp8z {

__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_of(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void halves(uint64_t p, uint32_t& a, uint32_t& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(p));
}
__device__ __forceinline__ float2 halves(uint64_t p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 16 bytes (32 of FP32) as four pairs of neighbouring elements.
template <typename T>
struct Eight {
    static constexpr int kUnits = sizeof(T) / 2;
    uint4 u[kUnits];
    __device__ __forceinline__ uint64_t pair(int i) const {
        const uint4& v = u[sizeof(T) == 4 ? i / 2 : 0];
        if constexpr (sizeof(T) == 4) {
            return i % 2 ? pair_of(v.z, v.w) : pair_of(v.x, v.y);
        } else {
            const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
            if constexpr (sizeof(T) == 2 && Elem<T>::kCode == FP8Z_BF16) return pair_of(w << 16, w & 0xFFFF0000u);
            else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
                return pair_of(f.x, f.y);
            }
        }
    }
};

}  // namespace fp8z
