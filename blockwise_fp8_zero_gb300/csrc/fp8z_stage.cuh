// fp8z_stage.cuh -- how tiles of a product leave a warp (through shared memory and the
// TMA engine, or along their rows), and the tensor maps that tiles go in and out by.
#pragma once

#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "fp8z_device.cuh"
#include "fp8z_elem.cuh"
#include "fp8z_host.h"
#include "fp8z_tcgen05.cuh"

namespace fp8z {

constexpr int kSlab = 32 * 128;                        // staged results of a warp: 32 rows of 128 bytes

__device__ __forceinline__ uint32_t pack16(float a, float b, int bf16) {
    uint32_t r;
    if (bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// A warp's way out: 32 rows of 128 bytes go to a slab in the layout of a
// 128-byte-swizzled tensor map, and from there to global memory as one tile,
// clipped at the tensor's edges.  A row for each thread, stored by the threads,
// wrote 262 MB of dw at 3.4 TB/s with 32 bytes a store and less with 16; this
// way it takes 57 us.
struct Stager {
    uint32_t slab;
    int lane;
    __device__ __forceinline__ uint32_t begin() {
        if (lane == 0) bulk_wait_read<0>();                   // the slab's last tile has been read
        __syncwarp();
        return slab;
    }
    __device__ __forceinline__ void put(uint32_t s, int chunk, uint32_t a, uint32_t b, uint32_t c, uint32_t d) const {
        st_shared_v4(s + lane * 128 + ((chunk ^ (lane & 7)) << 4), a, b, c, d);
    }
    // store(address) is called by lane 0 alone, whose row is the slab's first
    template <typename F>
    __device__ __forceinline__ void end(F store) {
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            store(slab);
            bulk_commit();
        }
    }
};

__device__ __forceinline__ void stage32(Stager& sg, const uint32_t* r) {
    const uint32_t s = sg.begin();
#pragma unroll
    for (int j = 0; j < 8; ++j) sg.put(s, j, r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
}

// Results whose rows do not all start and end on 16-byte boundaries, or are not all a product's,
// and sums of 16-bit gradients (one rounding of the whole sum): 32 columns of the
// warp's rows pass through its slab, so that the threads write along the rows.
template <typename T>
__device__ __forceinline__ void weight_rows(T* p, int64_t ld, int rows, int n, const Stager& sg, bool accumulate) {
    if (sg.lane >= n) return;
    const int chunk = sg.lane >> 2, word = (sg.lane & 3) * 4;
#pragma unroll 8
    for (int r = 0; r < rows; ++r) {
        float v;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(sg.slab + r * 128 + ((chunk ^ (r & 7)) << 4) + word) : "memory");
        T* at = p + r * ld + sg.lane;
        *at = Elem<T>::narrow(accumulate ? Elem<T>::widen(__ldcg(at)) + v : v);
    }
}

// Tensor maps with the 128-byte swizzle: a box is 128 bytes wide.
inline bool make_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* p, const cuuint64_t* dims,
              const cuuint64_t* strides, const cuuint32_t* box) {
    const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(host::tensor_map_encoder());
    if (!enc) return false;
    std::memset(map, 0, sizeof(*map));
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, type, cuuint32_t(rank), const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace fp8z
