// fp8z_tiles.h -- how a tile's blocks of K are divided into sums.  Plain 32-bit
// arithmetic without CUDA, so that it is checked on the host at every size.
#pragma once

#ifdef __CUDACC__
#define FP8Z_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define FP8Z_HOST_DEVICE inline
#endif

namespace fp8z {

// Sums that blocks [k0, k1) take with at most `most` blocks each (0: one sum of all), at least one.
FP8Z_HOST_DEVICE int sums_of(int k0, int k1, int most) {
    if (most == 0) return 1;
    const int sums = (k1 - k0 + most - 1) / most;
    return sums > 1 ? sums : 1;
}

// First block of sum i of `sums`, k1 for i == sums; the first few are a block longer
// than the others.  Divided before it is multiplied: no product is larger than k1 - k0,
// whereas (k1 - k0) * i passes 2^31 from 131072 blocks in sums of eight on.
FP8Z_HOST_DEVICE int sum_start(int k0, int k1, int i, int sums) {
    if (sums == 1) return i == 0 ? k0 : k1;              // a short loop waits for no division
    const int each = (k1 - k0) / sums, longer = (k1 - k0) - each * sums;
    return k0 + each * i + (i < longer ? i : longer);
}

}  // namespace fp8z
