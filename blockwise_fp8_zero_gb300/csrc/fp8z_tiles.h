// fp8z_tiles.h -- how a tile's blocks of K are divided into sums, and the length of a
// run of equal things.  Plain 32-bit arithmetic without CUDA, so that it is checked on
// the host at every size.
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

// How many of 1 .. most belong to a run that starts at 0 and holds all of them up to some
// number.  count(first, step, end) tells how many of first, first + step, .. belong to it,
// of the 32 of them and of those below `end`.  The nearest 32 come first, then 32 spread
// over what is left: one look for a short run, six for one of 2^25.
template <typename F>
FP8Z_HOST_DEVICE int run_length(int most, F count) {
    int in = 0, out = most + 1;
    for (int step = 1; out - in > 1; step = (out - in + 31) / 32) {
        const int n = count(in + step, step, out);
        in += n * step;
        if (n < 32 && in + step < out) out = in + step;
    }
    return in;
}

}  // namespace fp8z
