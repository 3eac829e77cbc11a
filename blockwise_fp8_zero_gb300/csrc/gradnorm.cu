// gradnorm.cu -- global gradient norm over a list of tensors, and clipping.
//
//   norm = |grad_scale| * sqrt(sum over all tensors of g^2)
//   coef = min(1, max_norm / (norm + eps)),  dst = (grad_scale * coef) * g
//
// Every element is read once for the norm and once more for the scaling (the
// coefficient is known only after the last element), and written once: the
// bound is HBM traffic, and the launches where the list is small.
#include <cfloat>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "fp8z.h"
#include "fp8z_elem.cuh"
#include "fp8z_host.h"

namespace fp8z {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = FP8Z_TENSOR_CHUNK;        // elements one block handles at a time
constexpr int kMaxGrid = 2048;
static_assert(kChunk % (kThreads * 8) == 0, "whole vectors per thread");

struct Workspace {
    uint32_t ticket, pad[3];
    double partial[kMaxGrid];
};
static_assert(sizeof(Workspace) <= FP8Z_GRAD_NORM_WORKSPACE, "workspace size in the header");

// The entry that chunk c belongs to: the last one whose first chunk is <= c
// and that has chunks at all (empty tensors share their successor's first).
__device__ __forceinline__ int find_entry(const fp8z_tensor_entry* __restrict__ list, int n, int64_t c) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (list[mid].first_chunk <= c) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Sum of squares of one thread's share of elements [0, n), n <= kChunk.
template <typename T>
__device__ __forceinline__ float chunk_squares(const T* __restrict__ g, int n) {
    constexpr int V = 16 / sizeof(T), R = kChunk / (kThreads * V);
    float a = 0.0f, b = 0.0f;
    if (n == kChunk && aligned16(g)) {
        Pack<T, V> x[R];
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = ld_nc<T, V>(g + (r * kThreads + threadIdx.x) * V);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const float p = Elem<T>::widen(x[r].v[i]), q = Elem<T>::widen(x[r].v[i + 1]);
                a = fmaf(p, p, a);
                b = fmaf(q, q, b);
            }
    } else {
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const float p = Elem<T>::widen(g[i]);
            a = fmaf(p, p, a);
        }
    }
    return a + b;
}

// Sixteen squares are added in FP32, then the running sum goes on in FP64:
// long lists lose nothing, and the FP64 pipe sees one addition per thread and chunk.
__global__ void __launch_bounds__(kThreads) norm_kernel(const fp8z_tensor_entry* __restrict__ list, int n,
                                                        int64_t chunks, float grad_scale, float max_norm,
                                                        float eps, float* __restrict__ norm,
                                                        Workspace* __restrict__ ws) {
    __shared__ double warp_sum[kThreads / 32];
    __shared__ bool last;
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    double sum = 0.0;
    if (c0 < c1) {
        int e = find_entry(list, n, c0);
        for (int64_t c = c0; c < c1; ++c) {
            while (e + 1 < n && list[e + 1].first_chunk <= c) ++e;
            const fp8z_tensor_entry t = list[e];
            const int64_t at = (c - t.first_chunk) * kChunk;
            const int m = int(min(int64_t(kChunk), t.numel - at));
            float s;
            if (t.src_dtype == FP8Z_F32) s = chunk_squares(static_cast<const float*>(t.src) + at, m);
            else if (t.src_dtype == FP8Z_BF16) s = chunk_squares(static_cast<const __nv_bfloat16*>(t.src) + at, m);
            else s = chunk_squares(static_cast<const __half*>(t.src) + at, m);
            sum += double(s);
        }
    }
    auto block_sum = [&](double v) {       // fixed order: the result does not depend on timing
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xFFFFFFFFu, v, o);
        if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
        __syncthreads();
        double r = 0.0;
        if (threadIdx.x == 0)
            for (int w = 0; w < kThreads / 32; ++w) r += warp_sum[w];
        __syncthreads();
        return r;
    };
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
    double v = 0.0;
    for (int i = threadIdx.x; i < int(gridDim.x); i += kThreads) v += __ldcg(&ws->partial[i]);
    v = block_sum(v);
    if (threadIdx.x == 0) {
        const float nm = float(fabs(double(grad_scale)) * sqrt(v));
        const float c = max_norm / (nm + eps);         // NaN stays NaN; an infinite limit never clips
        norm[0] = nm;
        norm[1] = isinf(max_norm) || c >= 1.0f ? 1.0f : c;
    }
}

template <typename S, typename D>
__device__ __forceinline__ void chunk_scale(const S* src, D* dst, int n, float f) {
    constexpr int V = 8, R = kChunk / (kThreads * V);
    if (n == kChunk && aligned16(src) && aligned16(dst)) {
        Pack<S, V> x[R];
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = ld_plain<S, V>(src + (r * kThreads + threadIdx.x) * V);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            Pack<D, V> y;
#pragma unroll
            for (int i = 0; i < V; ++i) y.v[i] = Elem<D>::narrow(Elem<S>::widen(x[r].v[i]) * f);
            st_vec<D, V>(dst + (r * kThreads + threadIdx.x) * V, y);
        }
    } else {
        for (int i = threadIdx.x; i < n; i += kThreads) dst[i] = Elem<D>::narrow(Elem<S>::widen(src[i]) * f);
    }
}

template <typename S>
__device__ __forceinline__ void chunk_scale_any(const fp8z_tensor_entry& t, int64_t at, int m, float f) {
    const S* s = static_cast<const S*>(t.src) + at;
    if (t.dst_dtype == FP8Z_F32) chunk_scale(s, static_cast<float*>(t.dst) + at, m, f);
    else if (t.dst_dtype == FP8Z_BF16) chunk_scale(s, static_cast<__nv_bfloat16*>(t.dst) + at, m, f);
    else chunk_scale(s, static_cast<__half*>(t.dst) + at, m, f);
}

__global__ void __launch_bounds__(kThreads) scale_kernel(const fp8z_tensor_entry* __restrict__ list, int n,
                                                         int64_t chunks, float grad_scale,
                                                         const float* __restrict__ norm) {
    const float f = grad_scale * norm[1];
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    if (c0 >= c1) return;
    int e = find_entry(list, n, c1 - 1);
    for (int64_t c = c1 - 1; c >= c0; --c) {     // what the norm read last may still be in L2
        while (list[e].first_chunk > c || list[e].numel == 0) --e;
        const fp8z_tensor_entry t = list[e];
        if (t.dst == t.src && t.dst_dtype == t.src_dtype && f == 1.0f) continue;
        const int64_t at = (c - t.first_chunk) * kChunk;
        const int m = int(min(int64_t(kChunk), t.numel - at));
        if (t.src_dtype == FP8Z_F32) chunk_scale_any<float>(t, at, m, f);
        else if (t.src_dtype == FP8Z_BF16) chunk_scale_any<__nv_bfloat16>(t, at, m, f);
        else chunk_scale_any<__half>(t, at, m, f);
    }
}

int launch(const fp8z_tensor_entry* list, int32_t n, int64_t chunks, float grad_scale, float max_norm, float eps,
           float* norm, void* workspace, bool clip, void* stream) {
    if (n < 0 || chunks < 0 || (chunks > 0 && !list) || !norm || !workspace) return FP8Z_EINVAL;
    if (!std::isfinite(grad_scale) || !(max_norm >= 0.0f) || !(eps >= 0.0f) || !std::isfinite(eps)) return FP8Z_EINVAL;
    if (!host::aligned(list, 8) || !host::aligned(norm, 4) || !host::aligned(workspace, 16)) return FP8Z_EALIGN;
    if (chunks > 0 && n == 0) return FP8Z_EINVAL;
    int sms = 0;
    if (int rc = host::device_sms(&sms)) return rc;
    const int64_t want = chunks < 1 ? 1 : chunks;
    const int grid = int(want < int64_t(sms) * 8 ? want : int64_t(sms) * 8);
    auto st = static_cast<cudaStream_t>(stream);
    norm_kernel<<<grid < kMaxGrid ? grid : kMaxGrid, kThreads, 0, st>>>(list, n, chunks, grad_scale, max_norm, eps,
                                                                      norm, static_cast<Workspace*>(workspace));
    if (clip && chunks > 0)
        scale_kernel<<<grid < kMaxGrid ? grid : kMaxGrid, kThreads, 0, st>>>(list, n, chunks, grad_scale, norm);
    return cudaGetLastError() == cudaSuccess ? FP8Z_OK : FP8Z_ECUDA;
}

}  // namespace
}  // namespace fp8z

extern "C" int fp8z_encode_tensor_list(const void* const* srcs, void* const* dsts, const int64_t* numels,
                                       const int32_t* src_dtypes, const int32_t* dst_dtypes, int32_t n,
                                       fp8z_tensor_entry* out, int64_t* chunks_out) {
    if (n < 0 || !chunks_out || (n > 0 && (!srcs || !numels || !src_dtypes || !out))) return FP8Z_EINVAL;
    if (n > 0 && (dsts == nullptr) != (dst_dtypes == nullptr)) return FP8Z_EINVAL;
    int64_t chunks = 0;
    for (int32_t i = 0; i < n; ++i) {
        const int32_t sd = src_dtypes[i], dd = dsts ? dst_dtypes[i] : sd;
        const void* s = srcs[i];
        void* d = dsts ? dsts[i] : const_cast<void*>(s);
        if (numels[i] < 0 || numels[i] > (1LL << 46) || !fp8z::dtype_ok(sd) || !fp8z::dtype_ok(dd)) return FP8Z_EINVAL;
        if (numels[i] > 0 && (!s || !d)) return FP8Z_EINVAL;
        // one tensor read and written with different element sizes would overwrite what is still to be read
        if (numels[i] > 0 && s == d && sd != dd) return FP8Z_EINVAL;
        if (!fp8z::host::aligned(s, fp8z::dtype_bytes(sd)) || !fp8z::host::aligned(d, fp8z::dtype_bytes(dd)))
            return FP8Z_EALIGN;
        out[i] = {s, d, numels[i], chunks, sd, dd};
        chunks += (numels[i] + FP8Z_TENSOR_CHUNK - 1) / FP8Z_TENSOR_CHUNK;
    }
    *chunks_out = chunks;
    return FP8Z_OK;
}

extern "C" int fp8z_grad_norm(const fp8z_tensor_entry* list, int32_t n, int64_t chunks, float grad_scale, float* norm,
                              void* workspace, void* stream) {
    const fp8z::host::NvtxRange nvtx_range("fp8z_grad_norm");
    return fp8z::launch(list, n, chunks, grad_scale, INFINITY, 0.0f, norm, workspace, false, stream);
}

extern "C" int fp8z_grad_clip(const fp8z_tensor_entry* list, int32_t n, int64_t chunks, float grad_scale,
                              float max_norm, float eps, float* norm, void* workspace, void* stream) {
    const fp8z::host::NvtxRange nvtx_range("fp8z_grad_clip");
    return fp8z::launch(list, n, chunks, grad_scale, max_norm, eps, norm, workspace, true, stream);
}
