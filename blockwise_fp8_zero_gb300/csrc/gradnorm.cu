// gradnorm.cu -- global gradient norm over a list of tensors, and clipping.
//
//   norm = |grad_scale| * sqrt(sum over all tensors of g^2)
//   coef = min(1, max_norm / (norm + eps)),  dst = (grad_scale * coef) * g
//
// Every element is read once for the norm and once more for the scaling (the
// coefficient is known only after the last element), and written once: the
// bound is HBM traffic, and the launches where the list is small.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "fp8z.h"
#include "fp8z_elem.cuh"
#include "fp8z_host.h"
#include "fp8z_launch.cuh"

namespace fp8z {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = FP8Z_TENSOR_CHUNK;        // elements of one block at a time
constexpr int kMaxGrid = 2048;
static_assert(kChunk % (kThreads * 8) == 0, "whole vectors per thread");

struct Workspace {
    uint32_t ticket, pad[3];
    double partial[kMaxGrid];
};
static_assert(sizeof(Workspace) <= FP8Z_GRAD_NORM_WORKSPACE, "workspace size in the header");

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// One thread's share of a chunk's squares: two sums of at most 17, added in FP32.
template <typename T>
__device__ __forceinline__ float chunk_squares(const T* g, int n) {
    constexpr int V = 16 / sizeof(T), R = kChunk / (kThreads * V);
    float a = 0.0f, b = 0.0f;
    if (n >= V && aligned16(g)) {
        const int done = n / V * V;                 // the last few elements of a tensor
        uint4 x[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = int(r * kThreads + threadIdx.x) * V;
            x[r] = ld_nc_16(g + (i + V <= n ? i : 0));       // loads without branches are all under way at once
            if (i + V > n) x[r] = make_uint4(0, 0, 0, 0);
        }
        if (int(threadIdx.x) < n - done) {
            const float p = Elem<T>::widen(g[done + threadIdx.x]);
            a = p * p;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const Pack<T, V> y = *reinterpret_cast<const Pack<T, V>*>(&x[r]);
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const float p = Elem<T>::widen(y.v[i]), q = Elem<T>::widen(y.v[i + 1]);
                a = fmaf(p, p, a);
                b = fmaf(q, q, b);
            }
        }
    } else {
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += 2 * kThreads) {
            const float p = Elem<T>::widen(g[i]), q = i + kThreads < n ? Elem<T>::widen(g[i + kThreads]) : 0.0f;
            a = fmaf(p, p, a);
            b = fmaf(q, q, b);
        }
    }
    return a + b;
}

__device__ __forceinline__ float squares(const fp8z_tensor_chunk& t) {
    if (t.src_dtype == FP8Z_F32) return chunk_squares(static_cast<const float*>(t.src), t.count);
    if (t.src_dtype == FP8Z_BF16) return chunk_squares(static_cast<const __nv_bfloat16*>(t.src), t.count);
    return chunk_squares(static_cast<const __half*>(t.src), t.count);
}

// Sum over the block in a fixed order: the result does not depend on timing.
// The sum is thread 0's.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double warp_sum[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    double r = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kThreads / 32; ++w) r += warp_sum[w];
    __syncthreads();
    return r;
}

__device__ __forceinline__ float2 norm_and_coef(double sum, float grad_scale, float max_norm, float eps) {
    const float nm = float(fabs(double(grad_scale)) * sqrt(sum));
    const float c = max_norm / (nm + eps);         // NaN stays NaN; an infinite limit never clips, whatever the norm
    return make_float2(nm, isinf(max_norm) || c >= 1.0f ? 1.0f : c);
}

// Each block takes neighbouring chunks and the sum goes on in FP64 from chunk to
// chunk: long lists lose nothing, and the FP64 pipe sees one addition per thread
// and 32 elements.  The block that finishes last adds the blocks' sums.
// 503 M FP32 elements: 285 us, 7.06 TB/s.
__global__ void __launch_bounds__(kThreads) norm_kernel(const fp8z_tensor_chunk* list, int64_t chunks, float grad_scale,
                                                        float max_norm, float eps, float* norm, Workspace* ws) {
    __shared__ bool last;
    dependent_wait();
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    double sum = 0.0;
    if (c0 < c1) {
        fp8z_tensor_chunk t = list[c0];
        for (int64_t c = c0; c < c1; ++c) {
            const fp8z_tensor_chunk next = list[c + 1 < c1 ? c + 1 : c];
            sum += double(squares(t));
            t = next;
        }
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        ws->partial[blockIdx.x] = sum;
        __threadfence();
        // wraps to 0 with the last block, so the workspace is ready for the next call
        last = atomicInc(&ws->ticket, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    sum = 0.0;
    for (int i = threadIdx.x; i < int(gridDim.x); i += kThreads) sum += __ldcg(&ws->partial[i]);
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        const float2 r = norm_and_coef(sum, grad_scale, max_norm, eps);
        norm[0] = r.x;
        norm[1] = r.y;
    }
}

// kFull: a whole chunk; the loads of a shorter one go on, to its first elements,
// where they would pass its end, so that all of them are under way at once.
template <bool kFull, typename S, typename D>
__device__ __forceinline__ void scale_vectors(const S* src, D* dst, int n, float f) {
    constexpr int V = 8, R = kChunk / (kThreads * V), W = V * sizeof(S) / 16;
    const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
    uint4 x[R][W];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = int(r * kThreads + threadIdx.x) * V;
#pragma unroll
        for (int w = 0; w < W; ++w) x[r][w] = ld_stream_16(src + (kFull || i + V <= n ? i : 0), w);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = int(r * kThreads + threadIdx.x) * V;
        const Pack<S, V> u = *reinterpret_cast<const Pack<S, V>*>(&x[r][0]);
        Pack<D, V> y;
#pragma unroll
        for (int j = 0; j < V; ++j) y.v[j] = Elem<D>::narrow(Elem<S>::widen(u.v[j]) * f);
        if (kFull || i + V <= n) st_stream8(dst + i, y, wide);
    }
}

template <typename S, typename D>
__device__ __forceinline__ void chunk_scale(const S* src, D* dst, int n, float f) {
    constexpr int V = 8;
    const bool aligned = aligned16(src) && aligned16(dst);
    if (n == kChunk && aligned) {
        scale_vectors<true>(src, dst, n, f);
        return;
    }
    int i = threadIdx.x;
    if (n >= V && aligned) {
        scale_vectors<false>(src, dst, n, f);
        i += n / V * V;                             // the last few elements of a tensor
    }
#pragma unroll 8
    for (; i < n; i += kThreads) dst[i] = Elem<D>::narrow(Elem<S>::widen(src[i]) * f);
}

template <typename S>
__device__ __forceinline__ void scale_from(const fp8z_tensor_chunk& t, float f) {
    const S* s = static_cast<const S*>(t.src);
    if (t.dst_dtype == FP8Z_F32) chunk_scale(s, static_cast<float*>(t.dst), t.count, f);
    else if (t.dst_dtype == FP8Z_BF16) chunk_scale(s, static_cast<__nv_bfloat16*>(t.dst), t.count, f);
    else chunk_scale(s, static_cast<__half*>(t.dst), t.count, f);
}

__device__ __forceinline__ void scale_chunk(const fp8z_tensor_chunk& t, float f) {
    if (t.dst == t.src && f == 1.0f) return;
    if (t.src_dtype == FP8Z_F32) scale_from<float>(t, f);
    else if (t.src_dtype == FP8Z_BF16) scale_from<__nv_bfloat16>(t, f);
    else scale_from<__half>(t, f);
}

// One block per chunk, last chunks first (they may still be in L2).  Blocks that
// come and go keep the memory system fuller than ones that stay and loop: 503 M
// FP32 elements copied with a factor ran at 7.1 TB/s this way, at 6.35 with 1216
// blocks over the same chunks.
__global__ void __launch_bounds__(kThreads) scale_kernel(const fp8z_tensor_chunk* list, int64_t chunks, float grad_scale,
                                                         const float* norm) {
    dependent_wait();
    const fp8z_tensor_chunk t = list[chunks - 1 - blockIdx.x];
    scale_chunk(t, grad_scale * norm[1]);
}

int launch(const fp8z_tensor_chunk* list, int64_t chunks, float grad_scale, float max_norm, float eps, float* norm,
           void* workspace, bool clip, void* stream) {
    if (chunks < 0 || chunks > 0x7FFFFFFF || (chunks > 0 && !list) || !norm || !workspace) return FP8Z_EINVAL;
    if (!std::isfinite(grad_scale) || !(max_norm >= 0.0f) || !(eps >= 0.0f) || !std::isfinite(eps)) return FP8Z_EINVAL;
    if (!host::aligned(list, 8) || !host::aligned(norm, 4) || !host::aligned(workspace, 16))
        return FP8Z_EALIGN;
    int sms = 0;
    if (int rc = host::device_sms(&sms)) return rc;
    const auto st = static_cast<cudaStream_t>(stream);
    auto* ws = static_cast<Workspace*>(workspace);
    const int64_t most = std::min<int64_t>(sms * 4, kMaxGrid);
    const dim3 grid(unsigned(std::min(std::max<int64_t>(chunks, 1), most)));
    if (int rc = launch_dependent(norm_kernel, grid, kThreads, 0, st, list, chunks, grad_scale, max_norm, eps, norm, ws))
        return rc;
    if (!clip || chunks == 0) return FP8Z_OK;
    return launch_dependent(scale_kernel, dim3(unsigned(chunks)), kThreads, 0, st, list, chunks, grad_scale, norm);
}

}  // namespace
}  // namespace fp8z

extern "C" int fp8z_encode_tensor_list(const void* const* srcs, void* const* dsts, const int64_t* numels,
                                       const int32_t* src_dtypes, const int32_t* dst_dtypes, int32_t n,
                                       fp8z_tensor_chunk* out, int64_t capacity, int64_t* chunks_out) {
    using namespace fp8z;
    if (n < 0 || !chunks_out || (n > 0 && (!srcs || !numels || !src_dtypes))) return FP8Z_EINVAL;
    if (n > 0 && (dsts == nullptr) != (dst_dtypes == nullptr)) return FP8Z_EINVAL;
    int64_t chunks = 0;
    for (int32_t i = 0; i < n; ++i) {
        const int32_t sd = src_dtypes[i], dd = dsts ? dst_dtypes[i] : sd;
        const void* s = srcs[i];
        const void* d = dsts ? dsts[i] : s;
        if (numels[i] < 0 || numels[i] > (1LL << 42) || !dtype_ok(sd) || !dtype_ok(dd)) return FP8Z_EINVAL;
        if (numels[i] > 0 && (!s || !d)) return FP8Z_EINVAL;
        // one tensor read and written with different element sizes would overwrite what is still to be read
        if (numels[i] > 0 && s == d && sd != dd) return FP8Z_EINVAL;
        if (!host::aligned(s, dtype_bytes(sd)) || !host::aligned(d, dtype_bytes(dd))) return FP8Z_EALIGN;
        chunks += (numels[i] + kChunk - 1) / kChunk;
        if (chunks > 0x7FFFFFFF) return FP8Z_EINVAL;
    }
    *chunks_out = chunks;
    if (!out) return FP8Z_OK;
    if (capacity < chunks) return FP8Z_ENOSPACE;
    for (int32_t i = 0; i < n; ++i) {
        const int32_t sd = src_dtypes[i], dd = dsts ? dst_dtypes[i] : sd;
        auto* s = static_cast<const uint8_t*>(srcs[i]);
        auto* d = dsts ? static_cast<uint8_t*>(dsts[i]) : const_cast<uint8_t*>(s);
        for (int64_t at = 0; at < numels[i]; at += kChunk)
            *out++ = {s + at * dtype_bytes(sd), d + at * dtype_bytes(dd), int32_t(std::min<int64_t>(kChunk, numels[i] - at)),
                      int16_t(sd), int16_t(dd)};
    }
    return FP8Z_OK;
}

extern "C" int fp8z_grad_norm(const fp8z_tensor_chunk* list, int64_t chunks, float grad_scale, float* norm,
                              void* workspace, void* stream) {
    const fp8z::host::NvtxRange nvtx_range("fp8z_grad_norm");
    return fp8z::launch(list, chunks, grad_scale, INFINITY, 0.0f, norm, workspace, false, stream);
}

extern "C" int fp8z_grad_clip(const fp8z_tensor_chunk* list, int64_t chunks, float grad_scale, float max_norm, float eps,
                              float* norm, void* workspace, void* stream) {
    const fp8z::host::NvtxRange nvtx_range("fp8z_grad_clip");
    return fp8z::launch(list, chunks, grad_scale, max_norm, eps, norm, workspace, true, stream);
}
