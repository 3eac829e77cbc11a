// layernorm.cu -- layer norm, optionally into the row-wise E4M3 operand of a product, and
// its gradient.
//
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps),  xh = (x - mean) rstd
//   y  = xh w + b
//   dx = rstd (g - sum g / n - xh sum (g xh) / n),  g = dy w
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// A row is read once and waits in registers for its two sums, many rows together (queues,
// below) where there are many.  Rows longer than the registers hold are read again.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "fp8z.h"
#include "fp8z_device.cuh"
#include "fp8z_elem.cuh"
#include "fp8z_host.h"
#include "fp8z_launch.cuh"
#include "fp8z_pairs.cuh"

namespace fp8z {
namespace {

constexpr int kVec = 8;                       // columns a thread takes together

struct Norm {
    int rows, cols;
    const void* x;
    int64_t x_ld;
    const void* weight;       // nullptr: 1
    const void* bias;         // nullptr: 0
    int param_dtype;
    void* y;
    int64_t y_ld;
    float* mean;
    float* rstd;
    float eps;
    uint8_t* q;
    float* q_scale;
    int pow2;
};

struct NormGrad {
    int rows, cols;
    const void* dy;
    const void* x;
    int64_t dy_ld, x_ld, dx_ld;
    const void* weight;
    int param_dtype;
    const float* mean;
    const float* rstd;
    void* dx;
    float* part;              // [blocks][2][cols]
};

// Columns of a thread: kVec neighbours at a time where rows start on 16-byte boundaries
// (kWide), else single ones kThreads apart, so that a warp's loads stay together.
template <bool kWide, int kThreads>
__device__ __forceinline__ int column(int j, int e, int tid) {
    return kWide ? (j * kThreads + tid) * kVec + e : (j * kVec + e) * kThreads + tid;
}

template <typename T>
__device__ __forceinline__ float load_one(const T* p) {
    if constexpr (sizeof(T) == 4) {
        float v;
        asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
        return v;
    } else {
        uint16_t u;
        asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(u) : "l"(p) : "memory");
        return Elem<T>::widen(*reinterpret_cast<T*>(&u));
    }
}

// Vector j of a thread's columns; zeros past the row's end.  kStream: read once.
template <bool kWide, int kThreads, bool kStream, typename T>
__device__ __forceinline__ void load8(const T* row, int j, int tid, int cols, float (&x)[kVec]) {
    if constexpr (kWide) {
        const int c = (j * kThreads + tid) * kVec;
        if (c + kVec <= cols) {
            Pack<T, kVec> u;
            uint4* w = reinterpret_cast<uint4*>(&u);
#pragma unroll
            for (int i = 0; i < int(sizeof(T) / 2); ++i) w[i] = kStream ? ld_stream_16(row + c, i) : ld_nc_16(reinterpret_cast<const uint4*>(row + c) + i);
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[e] = Elem<T>::widen(u.v[e]);
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        const int c = column<kWide, kThreads>(j, e, tid);
        x[e] = c < cols ? load_one(row + c) : 0.0f;
    }
}

template <bool kWide, int kThreads>
__device__ __forceinline__ void load8_param(const void* p, int dtype, int j, int tid, int cols, float (&x)[kVec]) {
    if (dtype == FP8Z_F32) load8<kWide, kThreads, false>(static_cast<const float*>(p), j, tid, cols, x);
    else if (dtype == FP8Z_BF16) load8<kWide, kThreads, false>(static_cast<const __nv_bfloat16*>(p), j, tid, cols, x);
    else load8<kWide, kThreads, false>(static_cast<const __half*>(p), j, tid, cols, x);
}

template <bool kWide, int kThreads, typename T>
__device__ __forceinline__ void store8(T* row, int j, int tid, int cols, const float (&x)[kVec]) {
    if constexpr (kWide) {
        const int c = (j * kThreads + tid) * kVec;
        if (c + kVec <= cols) {
            Pack<T, kVec> u;
#pragma unroll
            for (int e = 0; e < kVec; ++e) u.v[e] = Elem<T>::narrow(x[e]);
            st_vec(row + c, u);
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        const int c = column<kWide, kThreads>(j, e, tid);
        if (c < cols) row[c] = Elem<T>::narrow(x[e]);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sums over a row's threads, the same in each, in a fixed order.  `slot` alternates, so
// that one barrier a sum is enough.
template <int kThreads>
__device__ __forceinline__ float2 row_sum(float a, float b, float2* shared, int slot) {
    constexpr int kWarps = kThreads / 32;
    a = warp_sum(a);
    b = warp_sum(b);
    if constexpr (kWarps == 1) return make_float2(a, b);
    float2* s = shared + slot * kWarps;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const int i = threadIdx.x & 31;
    const float2 v = i < kWarps ? s[i] : make_float2(0.0f, 0.0f);
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// The scale and codes of 128 columns, held by 16 lanes: the rule of fp8z_quantize_rowwise.
__device__ __forceinline__ float tile_scale(float amax, bool pow2) {
    if (amax == 0.0f) return 1.0f;
    if (!pow2) return fmaxf(__fdiv_rn(amax, 448.0f), FLT_MIN);
    if (amax > FLT_MAX) return __uint_as_float(254u << 23);                        // 2^127
    // the smallest power of two that is not below amax / 448, from amax = f 2^e, f in [1/2, 1):
    // 448 = 7/8 * 2^9
    int e;
    const float f = frexpf(amax, &e);
    const int k = max(e - 9 + (f > 0.875f ? 1 : 0), -126);
    return __uint_as_float(uint32_t(k + 127) << 23);
}

template <typename T, bool kWide, int kThreads, int kVecs>
__global__ void __launch_bounds__(kThreads == 32 ? 256 : kThreads) norm_kernel(const __grid_constant__ Norm A) {
    constexpr int kGroups = kThreads == 32 ? 8 : 1;                 // rows a block takes together
    __shared__ float2 shared[2 * (kThreads / 32)];
    dependent_wait();
    const int tid = threadIdx.x % kThreads;
    const float n = float(A.cols);
    for (int64_t row = int64_t(blockIdx.x) * kGroups + threadIdx.x / kThreads; row < A.rows; row += int64_t(gridDim.x) * kGroups) {
        const T* px = static_cast<const T*>(A.x) + row * A.x_ld;
        float x[kVecs][kVec];
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) load8<kWide, kThreads, true>(px, j, tid, A.cols, x[j]);
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int e = 0; e < kVec; ++e) sum += x[j][e];
        const float mean = row_sum<kThreads>(sum, 0.0f, shared, 0).x / n;
        float sq = 0.0f;
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                x[j][e] = column<kWide, kThreads>(j, e, tid) < A.cols ? x[j][e] - mean : 0.0f;
                sq = fmaf(x[j][e], x[j][e], sq);
            }
        const float rstd = __frcp_rn(__fsqrt_rn(row_sum<kThreads>(sq, 0.0f, shared, 1).x / n + A.eps));
        if (tid == 0) {
            if (A.mean) A.mean[row] = mean;
            if (A.rstd) A.rstd[row] = rstd;
        }
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            if (column<kWide, kThreads>(j, 0, tid & ~31) >= A.cols) break;              // the whole warp is past the end
            float w[kVec], b[kVec];
            if (A.weight) load8_param<kWide, kThreads>(A.weight, A.param_dtype, j, tid, A.cols, w);
            if (A.bias) load8_param<kWide, kThreads>(A.bias, A.param_dtype, j, tid, A.cols, b);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                float v = x[j][e] * rstd;
                if (A.weight) v *= w[e];
                if (A.bias) v += b[e];
                x[j][e] = v;
            }
            if (A.y) store8<kWide, kThreads>(static_cast<T*>(A.y) + row * A.y_ld, j, tid, A.cols, x[j]);
            if (kWide && A.q) {
                float amax = 0.0f;
#pragma unroll
                for (int e = 0; e < kVec; ++e) amax = fmaxf(amax, fabsf(x[j][e]));
                const int c = (j * kThreads + tid) * kVec;
                if (c >= A.cols) amax = 0.0f;
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
                const float s = tile_scale(amax, A.pow2);
                uint32_t q[2];
                if (A.pow2) {
                    const float r = 1.0f / s;                       // exact
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        q[i] = pack_e4m3x4(x[j][4 * i] * r, x[j][4 * i + 1] * r, x[j][4 * i + 2] * r, x[j][4 * i + 3] * r);
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        q[i] = pack_e4m3x4(__fdiv_rn(x[j][4 * i], s), __fdiv_rn(x[j][4 * i + 1], s),
                                           __fdiv_rn(x[j][4 * i + 2], s), __fdiv_rn(x[j][4 * i + 3], s));
                }
                if (c < A.cols) {
                    *reinterpret_cast<uint2*>(A.q + row * A.cols + c) = make_uint2(q[0], q[1]);
                    if ((threadIdx.x & 15) == 0) A.q_scale[row * (A.cols / FP8Z_BLOCK) + c / FP8Z_BLOCK] = s;
                }
            }
        }
    }
}

// Rows longer than 32768 columns: three passes, the later ones mostly from L2.
template <typename T>
__global__ void __launch_bounds__(1024) norm_long_kernel(const __grid_constant__ Norm A) {
    __shared__ float2 shared[2 * 32];
    dependent_wait();
    for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
        const T* px = static_cast<const T*>(A.x) + row * A.x_ld;
        float sum = 0.0f, sq = 0.0f;
        for (int c = threadIdx.x; c < A.cols; c += 1024) sum += load_one(px + c);
        const float mean = row_sum<1024>(sum, 0.0f, shared, 0).x / float(A.cols);
        for (int c = threadIdx.x; c < A.cols; c += 1024) {
            const float d = load_one(px + c) - mean;
            sq = fmaf(d, d, sq);
        }
        const float rstd = __frcp_rn(__fsqrt_rn(row_sum<1024>(sq, 0.0f, shared, 1).x / float(A.cols) + A.eps));
        if (threadIdx.x == 0) {
            if (A.mean) A.mean[row] = mean;
            if (A.rstd) A.rstd[row] = rstd;
        }
        const auto param = [&](const void* p, int c) {
            return A.param_dtype == FP8Z_F32 ? load_one(static_cast<const float*>(p) + c)
                   : A.param_dtype == FP8Z_BF16 ? load_one(static_cast<const __nv_bfloat16*>(p) + c)
                                                : load_one(static_cast<const __half*>(p) + c);
        };
        // four columns a lane, so that a warp has a tile of 128
        for (int c0 = threadIdx.x / 32 * 128; c0 < A.cols; c0 += 32 * 128) {
            float v[4], amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i * 32 + (threadIdx.x & 31);
                v[i] = 0.0f;
                if (c >= A.cols) continue;
                v[i] = (load_one(px + c) - mean) * rstd;
                if (A.weight) v[i] *= param(A.weight, c);
                if (A.bias) v[i] += param(A.bias, c);
                if (A.y) static_cast<T*>(A.y)[row * A.y_ld + c] = Elem<T>::narrow(v[i]);
                amax = fmaxf(amax, fabsf(v[i]));
            }
            if (!A.q) continue;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            const float s = tile_scale(amax, A.pow2);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                A.q[row * A.cols + c0 + i * 32 + (threadIdx.x & 31)] = uint8_t(cvt_e4m3x2(__fdiv_rn(v[i], s), 0.0f));
            if ((threadIdx.x & 31) == 0) A.q_scale[row * (A.cols / FP8Z_BLOCK) + c0 / FP8Z_BLOCK] = s;
        }
    }
}

// ------------------------------------------------------- rows through a queue
// 16 bytes into shared memory in the background; zeros where `in` is false.
__device__ __forceinline__ void copy_16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// kN sums over a block, the same in each thread, in a fixed order.  In a
// warp half of the sums change lanes at every step, so that four sums take six shuffles.
template <int kN, int kMaxWarps>
__device__ __forceinline__ void block_sums(float (&v)[kN], float* shared) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int which = 0, off = 16;
#pragma unroll
    for (int n = kN / 2; n > 0; n /= 2, off /= 2) {
        const bool high = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float mine = high ? v[i + n] : v[i], other = high ? v[i] : v[i + n];
            v[i] = mine + __shfl_xor_sync(0xFFFFFFFFu, other, off);
        }
        if (high) which += n;
    }
    const int last = off;                                // lanes that hold the same sum differ below it
#pragma unroll
    for (; off > 0; off /= 2) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], off);
    if ((lane & (2 * last - 1)) == 0) shared[warp * kN + which] = v[0];
    __syncthreads();
    // the warps' sums, 32 / kN lanes for each of the kN, in every warp alike
    constexpr int kEach = 32 / kN;
    float all = 0.0f;
#pragma unroll
    for (int w = 0; w < kMaxWarps; w += kEach) {
        const int mine = w + lane % kEach;
        if (mine < warps) all += shared[mine * kN + lane / kEach];
    }
#pragma unroll
    for (int o = kEach / 2; o > 0; o /= 2) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, all, i * kEach);
}

// A thread's own queue: its columns of the next batches of rows are on their way into
// shared memory while it works on one, and nobody else reads them, so that no barrier
// guards the queue.  No registers hold loads: up to 196 KB an SM are a batch in work and the
// others on their way.
template <typename T, int kVecs, int kRows, int kTensors>
struct Queue {
    static constexpr int kUnits = Eight<T>::kUnits, kPieces = kTensors * kRows * kVecs * kUnits;
    static constexpr int kQueue = 6 / (kTensors * kRows * kUnits / 2);
    static constexpr int bytes(int threads) { return kQueue * kPieces * threads * 16; }
    uint32_t base, step;                                 // of this thread; bytes from one piece to the next
    __device__ __forceinline__ uint32_t at(int slot, int tensor, int r, int j, int u) const {
        return base + (slot * kPieces + ((tensor * kRows + r) * kVecs + j) * kUnits + u) * step;
    }
    __device__ __forceinline__ void fetch(int slot, int tensor, const T* p, int64_t ld, int64_t row0, int rows,
                                          const bool (&in)[kVecs]) const {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const bool there = row0 + r < rows;
            const T* row = p + (there ? row0 + r : 0) * ld;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const bool mine = there && in[j];
                const uint4* from = reinterpret_cast<const uint4*>(row + (mine ? (j * blockDim.x + threadIdx.x) * kVec : 0));
#pragma unroll
                for (int u = 0; u < kUnits; ++u) copy_16(at(slot, tensor, r, j, u), from + u, mine);
            }
        }
    }
    __device__ __forceinline__ Eight<T> load(int slot, int tensor, int r, int j) const {
        Eight<T> x;
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x.u[u].x), "=r"(x.u[u].y), "=r"(x.u[u].z), "=r"(x.u[u].w)
                         : "r"(at(slot, tensor, r, j, u))
                         : "memory");
        return x;
    }
};

// The columns of a thread of the queued kernels, `j` of kVecs: those from eight(j) on.
__device__ __forceinline__ int eight(int j) { return (j * int(blockDim.x) + int(threadIdx.x)) * kVec; }

// Their weights, or `otherwise` where there are none.
__device__ __forceinline__ void params8(const void* p, int dtype, int j, bool in, float otherwise, uint64_t (&w)[4]) {
    float v[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = otherwise;
    if (p && in) {
        if (dtype == FP8Z_F32) load8<true, 0, false>(static_cast<const float*>(p) + eight(j), 0, 0, kVec, v);
        else if (dtype == FP8Z_BF16) load8<true, 0, false>(static_cast<const __nv_bfloat16*>(p) + eight(j), 0, 0, kVec, v);
        else load8<true, 0, false>(static_cast<const __half*>(p) + eight(j), 0, 0, kVec, v);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pair_of(v[2 * i], v[2 * i + 1]);
}

// Eight results as T, 16 bytes at a time.
template <typename T>
__device__ __forceinline__ void store_pairs(T* p, const uint64_t (&v)[4]) {
    Pack<T, kVec> y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = halves(v[i]);
        y.v[2 * i] = Elem<T>::narrow(f.x);
        y.v[2 * i + 1] = Elem<T>::narrow(f.y);
    }
    st_vec(p, y);
}

// The scale of a tile with the largest magnitude `amax`, and the codes E4M3(v / s) of eight of its
// columns, by the rule of fp8z_quantize_rowwise.  A quotient is formed as the numerator times
// a reciprocal and one correction by the remainder (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000", 1990), which rounds it as a division would wherever
// nothing overflows or goes below 2^-126 on the way; other tiles take the division.
__device__ __forceinline__ uint2 tile_codes(const uint64_t (&v)[4], float amax, bool pow2, float& s) {
    float t[kVec];
    if (!(amax > 0x1p-50f && amax < 0x1p100f)) {
        s = tile_scale(amax, pow2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = halves(v[i]);
            t[2 * i] = __fdiv_rn(f.x, s);
            t[2 * i + 1] = __fdiv_rn(f.y, s);
        }
    } else if (pow2) {
        // 448 = 7/8 * 2^9: the exponent of amax less 8, one more above 1.75 of its binade; 1 / s is exact
        const uint32_t bits = __float_as_uint(amax), k = (bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        s = __uint_as_float(k << 23);
        const float r = __uint_as_float((254 - k) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = halves(mul_pair(v[i], pair_of(r, r)));
            t[2 * i] = f.x;
            t[2 * i + 1] = f.y;
        }
    } else {
        constexpr float c = 1.0f / 448.0f;
        s = amax * c;
        s = fmaf(fmaf(-s, 448.0f, amax), c, s);
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
        r = fmaf(fmaf(-s, r, 1.0f), r, r);
        const uint64_t rr = pair_of(r, r), ss = pair_of(-s, -s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t q = mul_pair(v[i], rr);
            const float2 f = halves(fma_pair(fma_pair(q, ss, v[i]), rr, q));
            t[2 * i] = f.x;
            t[2 * i + 1] = f.y;
        }
    }
    return make_uint2(pack_e4m3x4(t[0], t[1], t[2], t[3]), pack_e4m3x4(t[4], t[5], t[6], t[7]));
}

// sum / n from per = 1 / n and one correction by the remainder: rounded as a division would be.  A
// mean that is off moves all codes of a row the same way: 8192 x 7168 rows of mean 5 had 654 codes beside
// those of 64 bits with this and inverse_root, where elementary operations in FP32 have 1110.
__device__ __forceinline__ float mean_of(float sum, float n, float per) {
    const float q = sum * per;
    return fabsf(sum) <= 0x1p120f ? fmaf(fmaf(-q, n, sum), per, q) : q;
}

// 1 / sqrt(x), off by little more than its rounding: the approximation and one Newton step, whose product
// x r counts with what its own rounding lost; infinite for 0, and 0 for a sum of squares that has
// overflowed.
__device__ __forceinline__ float inverse_root(float x) {
    const float r = rsqrtf(x), h = x * r, low = fmaf(x, r, -h);
    const float e = fmaf(-low, r, fmaf(-h, r, 1.0f));
    return x == 0.0f || x > FLT_MAX ? r : fmaf(r * 0.5f, e, r);
}

// Batches of two rows, one block a batch at a time: the sums of a batch share two barriers.
// A thread has eight neighbouring columns of every row; the block is as wide as the row.
// 16384 x 7168 BF16 into E4M3: 131 us at a floor of 52.  31 instructions an element (two passes over
// registers, largest magnitudes, a corrected quotient and a conversion) issue in 71 % of the cycles; in the
// others the SM's one block waits for its two barriers a batch, for shuffles and for the math pipes.
template <typename T, bool kCodes>
__global__ void __launch_bounds__(1024) norm_queue_kernel(const __grid_constant__ Norm A) {
    constexpr int kRows = 2, kVecs = 1;
    using Q = Queue<T, kVecs, kRows, 1>;
    constexpr int kQueue = Q::kQueue;
    extern __shared__ uint4 smem[];
    __shared__ float shared[2][32 * kRows];
    dependent_wait();
    const Q q{smem_addr(smem) + threadIdx.x * 16, blockDim.x * 16};
    const T* x = static_cast<const T*>(A.x);
    const int64_t batches = (int64_t(A.rows) + kRows - 1) / kRows;
    const float per = 1.0f / float(A.cols);
    uint64_t w[kVecs][4], b[kVecs][4];
    bool in[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        in[j] = eight(j) < A.cols;
        params8(A.weight, A.param_dtype, j, in[j], 1.0f, w[j]);
        params8(A.bias, A.param_dtype, j, in[j], 0.0f, b[j]);
    }
#pragma unroll
    for (int d = 0; d < kQueue - 1; ++d) {
        q.fetch(d, 0, x, A.x_ld, (blockIdx.x + int64_t(d) * gridDim.x) * kRows, A.rows, in);
        copy_commit();
    }
    int slot = 0;
    for (int64_t batch = blockIdx.x; batch < batches; batch += gridDim.x) {
        q.fetch(slot == 0 ? kQueue - 1 : slot - 1, 0, x, A.x_ld, (batch + int64_t(kQueue - 1) * gridDim.x) * kRows, A.rows, in);
        copy_commit();
        copy_wait<kQueue - 1>();
        uint64_t v[kRows][kVecs][4];
        float mean[kRows], rstd[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            uint64_t s = 0;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const Eight<T> raw = q.load(slot, 0, r, j);      // zeros past the row's end
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[r][j][i] = raw.pair(i);
                    s = add_pair(s, v[r][j][i]);
                }
            }
            const float2 f = halves(s);
            mean[r] = f.x + f.y;
        }
        block_sums<kRows, 32>(mean, shared[0]);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            mean[r] = mean_of(mean[r], float(A.cols), per);
            const uint64_t m = pair_of(-mean[r], -mean[r]);
            uint64_t s = 0;
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[r][j][i] = add_pair(v[r][j][i], m);
                    if (in[j]) s = fma_pair(v[r][j][i], v[r][j][i], s);
                }
            const float2 f = halves(s);
            rstd[r] = f.x + f.y;
        }
        block_sums<kRows, 32>(rstd, shared[1]);
        const int64_t row0 = batch * kRows;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            rstd[r] = inverse_root(mean_of(rstd[r], float(A.cols), per) + A.eps);
            if (threadIdx.x == 0 && row0 + r < A.rows) {
                if (A.mean) A.mean[row0 + r] = mean[r];
                if (A.rstd) A.rstd[row0 + r] = rstd[r];
            }
            const uint64_t f = pair_of(rstd[r], rstd[r]);
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[r][j][i] = fma_pair(mul_pair(v[r][j][i], f), w[j][i], b[j][i]);
        }
        if (A.y)
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int j = 0; j < kVecs; ++j)
                    if (in[j] && row0 + r < A.rows) store_pairs(static_cast<T*>(A.y) + (row0 + r) * A.y_ld + eight(j), v[r][j]);
        if constexpr (kCodes) {
            float amax[kRows][kVecs];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    amax[r][j] = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = halves(v[r][j][i]);
                        amax[r][j] = fmaxf(amax[r][j], fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int j = 0; j < kVecs; ++j) amax[r][j] = fmaxf(amax[r][j], __shfl_xor_sync(0xFFFFFFFFu, amax[r][j], o));
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    float s;
                    const uint2 codes = tile_codes(v[r][j], amax[r][j], A.pow2, s);
                    if (in[j] && row0 + r < A.rows) {
                        *reinterpret_cast<uint2*>(A.q + (row0 + r) * A.cols + eight(j)) = codes;
                        if ((threadIdx.x & 15) == 0) A.q_scale[(row0 + r) * (A.cols / FP8Z_BLOCK) + eight(j) / FP8Z_BLOCK] = s;
                    }
                }
        }
        slot = slot + 1 == kQueue ? 0 : slot + 1;
    }
    copy_wait<0>();
}

// ---------------------------------------------------------------- gradient
// A block walks over rows, keeps its columns' sums of dy xh and dy in registers, and
// leaves them in `part` at the end: dy and x are read once.
template <typename T, bool kWide, int kThreads, int kVecs>
__global__ void __launch_bounds__(kThreads == 32 ? 256 : kThreads) norm_grad_kernel(const __grid_constant__ NormGrad A) {
    constexpr int kGroups = kThreads == 32 ? 8 : 1;
    __shared__ float2 shared[2 * (kThreads / 32)];
    __shared__ float joined[kGroups == 1 ? 1 : kGroups][kGroups == 1 ? 1 : 2 * 32 * kVec * kVecs];
    dependent_wait();
    const int tid = threadIdx.x % kThreads, group = threadIdx.x / kThreads;
    const float n = float(A.cols);
    float dw[kVecs][kVec], db[kVecs][kVec], w[kVecs][kVec];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            dw[j][e] = db[j][e] = 0.0f;
            w[j][e] = 1.0f;
        }
        if (A.weight) load8_param<kWide, kThreads>(A.weight, A.param_dtype, j, tid, A.cols, w[j]);
    }
    int slot = 0;
    for (int64_t row = int64_t(blockIdx.x) * kGroups + group; row < A.rows; row += int64_t(gridDim.x) * kGroups) {
        const T* px = static_cast<const T*>(A.x) + row * A.x_ld;
        const T* pd = static_cast<const T*>(A.dy) + row * A.dy_ld;
        const float mean = load_one(A.mean + row), rstd = load_one(A.rstd + row);
        float x[kVecs][kVec], d[kVecs][kVec], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            load8<kWide, kThreads, true>(px, j, tid, A.cols, x[j]);
            load8<kWide, kThreads, true>(pd, j, tid, A.cols, d[j]);
        }
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                x[j][e] = column<kWide, kThreads>(j, e, tid) < A.cols ? (x[j][e] - mean) * rstd : 0.0f;
                dw[j][e] = fmaf(d[j][e], x[j][e], dw[j][e]);
                db[j][e] += d[j][e];
                d[j][e] *= w[j][e];
                s1 += d[j][e];
                s2 = fmaf(d[j][e], x[j][e], s2);
            }
        const float2 s = row_sum<kThreads>(s1, s2, shared, slot);
        slot ^= 1;
        const float c1 = s.x / n, c2 = s.y / n;
        if (A.dx)
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                float v[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) v[e] = rstd * (d[j][e] - c1 - x[j][e] * c2);
                store8<kWide, kThreads>(static_cast<T*>(A.dx) + row * A.dx_ld, j, tid, A.cols, v);
            }
    }
    float* out = A.part + int64_t(blockIdx.x) * 2 * A.cols;
    if constexpr (kGroups > 1) {
        // the eight rows' warps join their sums, in order
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                joined[group][(j * kVec + e) * 32 + tid] = dw[j][e];
                joined[group][(kVecs * kVec + j * kVec + e) * 32 + tid] = db[j][e];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * 32 * kVec * kVecs; i += 256) {
            const int je = i / 32, k = je % (kVecs * kVec), c = column<kWide, kThreads>(k / kVec, k % kVec, i % 32);
            float sum = 0.0f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) sum += joined[g][i];
            if (c < A.cols) out[(je >= kVecs * kVec ? A.cols : 0) + c] = sum;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const int c = column<kWide, kThreads>(j, e, tid);
                if (c < A.cols) {
                    out[c] = dw[j][e];
                    out[A.cols + c] = db[j][e];
                }
            }
    }
}

// The same with a queue of dy and x: both are read from shared memory again for dx, so that
// registers hold the sums of dw and db, and the weight, only.  16384 x 7168 BF16: 107 to 112 us with
// the join of the parts, 6.3 TB/s: memory traffic.
template <typename T, int kVecs>
__global__ void __launch_bounds__(512, 2 / kVecs) norm_grad_queue_kernel(const __grid_constant__ NormGrad A) {
    constexpr int kRows = sizeof(T) == 2 ? 2 : 1;
    using Q = Queue<T, kVecs, kRows, 2>;
    constexpr int kQueue = Q::kQueue;
    extern __shared__ uint4 smem[];
    __shared__ float shared[2][16 * 2 * kRows];
    dependent_wait();
    const Q q{smem_addr(smem) + threadIdx.x * 16, blockDim.x * 16};
    const T *x = static_cast<const T*>(A.x), *dy = static_cast<const T*>(A.dy);
    const int64_t batches = (int64_t(A.rows) + kRows - 1) / kRows;
    const float per = 1.0f / float(A.cols);
    uint64_t w[kVecs][4], dw[kVecs][4], db[kVecs][4];
    bool in[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        in[j] = eight(j) < A.cols;
        params8(A.weight, A.param_dtype, j, in[j], 1.0f, w[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[j][i] = db[j][i] = 0;
    }
    const auto fetch = [&](int slot, int64_t batch) {
        q.fetch(slot, 0, x, A.x_ld, batch * kRows, A.rows, in);
        q.fetch(slot, 1, dy, A.dy_ld, batch * kRows, A.rows, in);
        copy_commit();
    };
    float mean[kRows], rstd[kRows];                              // of the next batch
    const auto stats = [&](int64_t batch) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const bool there = batch * kRows + r < A.rows;
            mean[r] = there ? load_one(A.mean + batch * kRows + r) : 0.0f;
            rstd[r] = there ? load_one(A.rstd + batch * kRows + r) : 0.0f;
        }
    };
#pragma unroll
    for (int d = 0; d < kQueue - 1; ++d) fetch(d, blockIdx.x + int64_t(d) * gridDim.x);
    stats(blockIdx.x);
    int slot = 0, turn = 0;
    for (int64_t batch = blockIdx.x; batch < batches; batch += gridDim.x) {
        fetch(slot == 0 ? kQueue - 1 : slot - 1, batch + int64_t(kQueue - 1) * gridDim.x);
        copy_wait<kQueue - 1>();
        uint64_t m[kRows], f[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) m[r] = pair_of(-mean[r], -mean[r]), f[r] = pair_of(rstd[r], rstd[r]);
        stats(batch + gridDim.x);
        float sums[2 * kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            uint64_t s1 = 0, s2 = 0;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const Eight<T> xv = q.load(slot, 0, r, j), dv = q.load(slot, 1, r, j);   // zeros past the row's end
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t xh = mul_pair(add_pair(xv.pair(i), m[r]), f[r]), d = dv.pair(i), g = mul_pair(d, w[j][i]);
                    dw[j][i] = fma_pair(d, xh, dw[j][i]);
                    db[j][i] = add_pair(db[j][i], d);
                    s1 = add_pair(s1, g);
                    s2 = fma_pair(g, xh, s2);
                }
            }
            const float2 a = halves(s1), c = halves(s2);
            sums[r] = a.x + a.y;
            sums[kRows + r] = c.x + c.y;
        }
        block_sums<2 * kRows, 16>(sums, shared[turn]);
        turn ^= 1;
        if (A.dx)
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int64_t row = batch * kRows + r;
                if (row >= A.rows) break;
                const float c1 = sums[r] * per, c2 = sums[kRows + r] * per;
                const uint64_t n1 = pair_of(-c1, -c1), n2 = pair_of(-c2, -c2);
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    if (!in[j]) break;
                    const Eight<T> xv = q.load(slot, 0, r, j), dv = q.load(slot, 1, r, j);
                    uint64_t v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint64_t xh = mul_pair(add_pair(xv.pair(i), m[r]), f[r]), g = mul_pair(dv.pair(i), w[j][i]);
                        v[i] = mul_pair(fma_pair(xh, n2, add_pair(g, n1)), f[r]);
                    }
                    store_pairs(static_cast<T*>(A.dx) + row * A.dx_ld + eight(j), v);
                }
            }
        slot = slot + 1 == kQueue ? 0 : slot + 1;
    }
    copy_wait<0>();
    float* out = A.part + int64_t(blockIdx.x) * 2 * A.cols;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
        if (in[j]) {
            store_pairs(out + eight(j), dw[j]);
            store_pairs(out + A.cols + eight(j), db[j]);
        }
}

// ------------------------------------------------------ rows that start anywhere
// Rows that do not all start on 16-byte boundaries go through a block's queue in whole 16 bytes,
// from the boundary before a row on; a thread's eight columns are then shifted out of its own and
// the next 16 bytes (32 of FP32), and results shifted into whole 16 bytes the other way.
// 16384 x 2001 BF16: a column at a time 123 us, the gradient 117.
template <typename T>
struct Shifted {
    static constexpr int kUnits = Eight<T>::kUnits, kBytes = 16 * kUnits;      // of a thread's columns
    uint32_t base;                                       // of the row in shared memory

    // The row's bytes from the boundary before `row` on, 16 a copy.  The bytes before a tensor's
    // first row are not ours: its first 16 bytes come an element at a time.
    static __device__ __forceinline__ void fetch(uint32_t to, const T* row, int cols, bool there, bool first) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row);
        const int shift = int(at & 15), end = there ? shift + cols * int(sizeof(T)) : 0;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int c = (u * int(blockDim.x) + int(threadIdx.x)) * 16, n = min(max(end - c, 0), 16);
            if (first && there && c == 0) {
                for (int b = shift; b < n; b += int(sizeof(T))) {
                    if constexpr (sizeof(T) == 4)
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + b), "f"(load_one(reinterpret_cast<const float*>(at - shift + b))) : "memory");
                    else
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + b), "h"(*reinterpret_cast<const volatile uint16_t*>(at - shift + b)) : "memory");
                }
            } else {
                const uintptr_t from = n > 0 ? at - shift + c : at & ~uintptr_t(15);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + c), "l"(from), "r"(n) : "memory");
            }
        }
    }
    // The thread's columns of a row that starts `shift` bytes behind a boundary; `left` of them are the row's.
    __device__ __forceinline__ void load(int shift, int left, uint64_t (&v)[4]) const {
        uint32_t w[4 * kUnits + 4];
#pragma unroll
        for (int u = 0; u <= kUnits; ++u)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[4 * u]), "=r"(w[4 * u + 1]), "=r"(w[4 * u + 2]), "=r"(w[4 * u + 3])
                         : "r"(base + threadIdx.x * kBytes + u * 16)
                         : "memory");
        Eight<T> x;
        shift_down(w, shift, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = x.pair(i);
        if (left < kVec) clear(v, left);
    }
    static __device__ __forceinline__ void clear(uint64_t (&v)[4], int left) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = halves(v[i]);
            v[i] = pair_of(2 * i < left ? f.x : 0.0f, 2 * i + 1 < left ? f.y : 0.0f);
        }
    }
    // The words from byte `shift` (0 to 16) on; it is the same for all threads.
    static __device__ __forceinline__ void shift_down(const uint32_t (&w)[4 * kUnits + 4], int shift, Eight<T>& x) {
        uint32_t* o = reinterpret_cast<uint32_t*>(&x);
        const int bits = (shift & 2) * 8;
        const auto from = [&](auto first) {
            constexpr int k = decltype(first)::value;
#pragma unroll
            for (int i = 0; i < 4 * kUnits; ++i) o[i] = sizeof(T) == 2 && i + k < 4 * kUnits + 3 ? __funnelshift_r(w[i + k], w[i + k + 1], bits) : w[i + k];
        };
        switch (shift >> 2) {
            case 0: from(std::integral_constant<int, 0>()); break;
            case 1: from(std::integral_constant<int, 1>()); break;
            case 2: from(std::integral_constant<int, 2>()); break;
            case 3: from(std::integral_constant<int, 3>()); break;
            default: from(std::integral_constant<int, 4>());
        }
    }
    // The thread's results to its place, 16 bytes, from where they are shifted into `row` by store
    // after a barrier.
    __device__ __forceinline__ void put(const uint64_t (&v)[4], Eight<T>& own) const {
        Pack<T, kVec> y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = halves(v[i]);
            y.v[2 * i] = Elem<T>::narrow(f.x);
            y.v[2 * i + 1] = Elem<T>::narrow(f.y);
        }
        own = *reinterpret_cast<const Eight<T>*>(&y);
        const uint4 last = own.u[kUnits - 1];            // all that the thread after it needs
        st_shared_16(base + threadIdx.x * 16, last);
    }
    // A thread writes the 16 bytes (32) that end inside its own columns; what is before them is the
    // thread's before it.
    __device__ __forceinline__ void store(T* row, int cols, const Eight<T>& own) const {
        const int shift = int(reinterpret_cast<uintptr_t>(row) & 15), behind = shift / int(sizeof(T));
        uint32_t w[4 * kUnits + 4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(base + (threadIdx.x ? threadIdx.x - 1 : 0) * 16)
                     : "memory");
#pragma unroll
        for (int u = 0; u < kUnits; ++u) w[4 + 4 * u] = own.u[u].x, w[5 + 4 * u] = own.u[u].y, w[6 + 4 * u] = own.u[u].z, w[7 + 4 * u] = own.u[u].w;
        Eight<T> out;
        shift_down(w, 16 - shift, out);
        const int col = int(threadIdx.x) * kVec - behind, from = threadIdx.x ? 0 : behind, until = min(kVec, cols - col);
        if (from == 0 && until == kVec) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u) reinterpret_cast<uint4*>(row + col)[u] = out.u[u];
        } else {
            const T* e = reinterpret_cast<const T*>(&out);
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (i >= from && i < until) row[col + i] = e[i];
        }
    }
    static __device__ __forceinline__ void st_shared_16(uint32_t at, const uint4& v) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
    }
};

// Columns threadIdx.x * 8 on of a weight that may start anywhere.
__device__ __forceinline__ void params_any(const void* p, int dtype, int left, float otherwise, uint64_t (&w)[4]) {
    float v[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        const int c = int(threadIdx.x) * kVec + e;
        v[e] = otherwise;
        if (p && e < left)
            v[e] = dtype == FP8Z_F32 ? load_one(static_cast<const float*>(p) + c)
                   : dtype == FP8Z_BF16 ? load_one(static_cast<const __nv_bfloat16*>(p) + c)
                                        : load_one(static_cast<const __half*>(p) + c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pair_of(v[2 * i], v[2 * i + 1]);
}

template <typename T>
__global__ void __launch_bounds__(1024) norm_shift_kernel(const __grid_constant__ Norm A) {
    constexpr int kRows = 2, kQueue = 6 / Eight<T>::kUnits;
    using S = Shifted<T>;
    extern __shared__ uint4 smem[];
    __shared__ float shared[2][32 * kRows];
    dependent_wait();
    const uint32_t base = smem_addr(smem), row_bytes = blockDim.x * S::kBytes + 16;      // a thread also reads the 16 bytes after its own
    const T* x = static_cast<const T*>(A.x);
    const int64_t batches = (int64_t(A.rows) + kRows - 1) / kRows;
    const float per = 1.0f / float(A.cols);
    const int left = A.cols - int(threadIdx.x) * kVec;
    uint64_t w[4], b[4];
    params_any(A.weight, A.param_dtype, left, 1.0f, w);
    params_any(A.bias, A.param_dtype, left, 0.0f, b);
    const auto fetch = [&](int slot, int64_t batch) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int64_t row = batch * kRows + r;
            const bool there = row < A.rows;
            S::fetch(base + (slot * kRows + r) * row_bytes, x + (there ? row : 0) * A.x_ld, A.cols, there, row == 0);
        }
        copy_commit();
    };
#pragma unroll
    for (int d = 0; d < kQueue - 1; ++d) fetch(d, blockIdx.x + int64_t(d) * gridDim.x);
    int slot = 0;
    for (int64_t batch = blockIdx.x; batch < batches; batch += gridDim.x) {
        copy_wait<kQueue - 2>();
        __syncthreads();                                 // all copies of the batch are there, and all have read the one before
        fetch(slot == 0 ? kQueue - 1 : slot - 1, batch + int64_t(kQueue - 1) * gridDim.x);
        uint64_t v[kRows][4];
        float mean[kRows], rstd[kRows];
        const int64_t row0 = batch * kRows;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const T* row = x + (row0 + r < A.rows ? row0 + r : 0) * A.x_ld;
            S{base + (slot * kRows + r) * row_bytes}.load(int(reinterpret_cast<uintptr_t>(row) & 15), left, v[r]);
            const float2 f = halves(add_pair(add_pair(v[r][0], v[r][1]), add_pair(v[r][2], v[r][3])));
            mean[r] = f.x + f.y;
        }
        block_sums<kRows, 32>(mean, shared[0]);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            mean[r] = mean_of(mean[r], float(A.cols), per);
            uint64_t s = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[r][i] = add_pair(v[r][i], pair_of(-mean[r], -mean[r]));
            if (left < kVec) S::clear(v[r], left);
#pragma unroll
            for (int i = 0; i < 4; ++i) s = fma_pair(v[r][i], v[r][i], s);
            const float2 f = halves(s);
            rstd[r] = f.x + f.y;
        }
        block_sums<kRows, 32>(rstd, shared[1]);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (row0 + r >= A.rows) break;
            rstd[r] = inverse_root(mean_of(rstd[r], float(A.cols), per) + A.eps);
            if (threadIdx.x == 0) {
                if (A.mean) A.mean[row0 + r] = mean[r];
                if (A.rstd) A.rstd[row0 + r] = rstd[r];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v[r][i] = fma_pair(mul_pair(v[r][i], pair_of(rstd[r], rstd[r])), w[i], b[i]);
        }
        if (A.y) {
            Eight<T> own[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) S{base + (slot * kRows + r) * row_bytes}.put(v[r], own[r]);
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (row0 + r < A.rows)
                    S{base + (slot * kRows + r) * row_bytes}.store(static_cast<T*>(A.y) + (row0 + r) * A.y_ld, A.cols, own[r]);
        }
        slot = slot + 1 == kQueue ? 0 : slot + 1;
    }
    copy_wait<0>();
}

template <typename T>
__global__ void __launch_bounds__(1024) norm_grad_shift_kernel(const __grid_constant__ NormGrad A) {
    constexpr int kRows = sizeof(T) == 2 ? 2 : 1, kQueue = 3;
    using S = Shifted<T>;
    extern __shared__ uint4 smem[];
    __shared__ float shared[2][32 * 2 * kRows];
    dependent_wait();
    const uint32_t base = smem_addr(smem), row_bytes = blockDim.x * S::kBytes + 16;
    const T *x = static_cast<const T*>(A.x), *dy = static_cast<const T*>(A.dy);
    const int64_t batches = (int64_t(A.rows) + kRows - 1) / kRows;
    const float per = 1.0f / float(A.cols);
    const int left = A.cols - int(threadIdx.x) * kVec;
    uint64_t w[4], dw[4] = {}, db[4] = {};
    params_any(A.weight, A.param_dtype, left, 1.0f, w);
    const auto place = [&](int slot, int tensor, int r) { return base + ((slot * 2 + tensor) * kRows + r) * row_bytes; };
    const auto fetch = [&](int slot, int64_t batch) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int64_t row = batch * kRows + r, at = row < A.rows ? row : 0;
            S::fetch(place(slot, 0, r), x + at * A.x_ld, A.cols, row < A.rows, row == 0);
            S::fetch(place(slot, 1, r), dy + at * A.dy_ld, A.cols, row < A.rows, row == 0);
        }
        copy_commit();
    };
    float mean[kRows], rstd[kRows];                      // of the next batch
    const auto stats = [&](int64_t batch) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const bool there = batch * kRows + r < A.rows;
            mean[r] = there ? load_one(A.mean + batch * kRows + r) : 0.0f;
            rstd[r] = there ? load_one(A.rstd + batch * kRows + r) : 0.0f;
        }
    };
#pragma unroll
    for (int d = 0; d < kQueue - 1; ++d) fetch(d, blockIdx.x + int64_t(d) * gridDim.x);
    stats(blockIdx.x);
    int slot = 0, turn = 0;
    for (int64_t batch = blockIdx.x; batch < batches; batch += gridDim.x) {
        copy_wait<kQueue - 2>();
        __syncthreads();
        fetch(slot == 0 ? kQueue - 1 : slot - 1, batch + int64_t(kQueue - 1) * gridDim.x);
        uint64_t xh[kRows][4], g[kRows][4];
        float sums[2 * kRows], scale[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int64_t row = batch * kRows + r < A.rows ? batch * kRows + r : 0;
            S{place(slot, 0, r)}.load(int(reinterpret_cast<uintptr_t>(x + row * A.x_ld) & 15), left, xh[r]);
            S{place(slot, 1, r)}.load(int(reinterpret_cast<uintptr_t>(dy + row * A.dy_ld) & 15), left, g[r]);
            scale[r] = rstd[r];
            uint64_t s1 = 0, s2 = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xh[r][i] = mul_pair(add_pair(xh[r][i], pair_of(-mean[r], -mean[r])), pair_of(rstd[r], rstd[r]));
                dw[i] = fma_pair(g[r][i], xh[r][i], dw[i]);
                db[i] = add_pair(db[i], g[r][i]);
                g[r][i] = mul_pair(g[r][i], w[i]);
                s1 = add_pair(s1, g[r][i]);
                s2 = fma_pair(g[r][i], xh[r][i], s2);
            }
            const float2 a = halves(s1), c = halves(s2);
            sums[r] = a.x + a.y;
            sums[kRows + r] = c.x + c.y;
        }
        stats(batch + gridDim.x);
        block_sums<2 * kRows, 32>(sums, shared[turn]);
        turn ^= 1;
        if (A.dx) {
            Eight<T> own[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float c1 = sums[r] * per, c2 = sums[kRows + r] * per;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    g[r][i] = mul_pair(fma_pair(xh[r][i], pair_of(-c2, -c2), add_pair(g[r][i], pair_of(-c1, -c1))), pair_of(scale[r], scale[r]));
                S{place(slot, 0, r)}.put(g[r], own[r]);
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (batch * kRows + r < A.rows)
                    S{place(slot, 0, r)}.store(static_cast<T*>(A.dx) + (batch * kRows + r) * A.dx_ld, A.cols, own[r]);
        }
        slot = slot + 1 == kQueue ? 0 : slot + 1;
    }
    copy_wait<0>();
    float* out = A.part + int64_t(blockIdx.x) * 2 * A.cols + threadIdx.x * kVec;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = halves(dw[i]), c = halves(db[i]);
        if (2 * i < left) out[2 * i] = a.x, out[A.cols + 2 * i] = c.x;
        if (2 * i + 1 < left) out[2 * i + 1] = a.y, out[A.cols + 2 * i + 1] = c.y;
    }
}

// Rows longer than 32768 columns: the sums of dw and db are added to in `part`.
template <typename T>
__global__ void __launch_bounds__(1024) norm_grad_long_kernel(const __grid_constant__ NormGrad A) {
    __shared__ float2 shared[2 * 32];
    dependent_wait();
    float* out = A.part + int64_t(blockIdx.x) * 2 * A.cols;
    for (int c = threadIdx.x; c < 2 * A.cols; c += 1024) out[c] = 0.0f;
    __syncthreads();
    const auto weight = [&](int c) {
        return !A.weight ? 1.0f
               : A.param_dtype == FP8Z_F32 ? load_one(static_cast<const float*>(A.weight) + c)
               : A.param_dtype == FP8Z_BF16 ? load_one(static_cast<const __nv_bfloat16*>(A.weight) + c)
                                            : load_one(static_cast<const __half*>(A.weight) + c);
    };
    int slot = 0;
    for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
        const T* px = static_cast<const T*>(A.x) + row * A.x_ld;
        const T* pd = static_cast<const T*>(A.dy) + row * A.dy_ld;
        const float mean = load_one(A.mean + row), rstd = load_one(A.rstd + row);
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < A.cols; c += 1024) {
            const float xh = (load_one(px + c) - mean) * rstd, d = load_one(pd + c), g = d * weight(c);
            s1 += g;
            s2 = fmaf(g, xh, s2);
            out[c] = fmaf(d, xh, out[c]);
            out[A.cols + c] += d;
        }
        const float2 s = row_sum<1024>(s1, s2, shared, slot);
        slot ^= 1;
        const float c1 = s.x / float(A.cols), c2 = s.y / float(A.cols);
        if (A.dx)
            for (int c = threadIdx.x; c < A.cols; c += 1024) {
                const float xh = (load_one(px + c) - mean) * rstd, g = load_one(pd + c) * weight(c);
                static_cast<T*>(A.dx)[row * A.dx_ld + c] = Elem<T>::narrow(rstd * (g - c1 - xh * c2));
            }
    }
}

// dw and db from the blocks' parts: 32 columns a block, its 32 warps take every 32nd part
// and join in order.
template <typename P>
__global__ void __launch_bounds__(1024) norm_parts_kernel(const float* part, int parts, int cols, P* dweight, P* dbias,
                                                          int accumulate) {
    __shared__ float joined[32][33];
    dependent_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
    P* out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    float sum = 0.0f;
    if (c < cols)
#pragma unroll 8
        for (int i = warp; i < parts; i += 32) sum += __ldcg(part + (int64_t(i) * 2 + blockIdx.y) * cols + c);
    joined[warp][lane] = sum;
    __syncthreads();
    const int mine = blockIdx.x * 32 + warp;             // a warp joins one column
    sum = warp_sum(joined[lane][warp]);
    if (lane == 0 && mine < cols) out[mine] = Elem<P>::narrow(accumulate ? Elem<P>::widen(out[mine]) + sum : sum);
}

// ------------------------------------------------------------------- host
constexpr int kLongest = 32768;                        // columns a block's registers hold

// Parts of the weight's gradient, one for a block, at most.
int64_t most_parts(int64_t cols) { return cols <= 2048 ? 608 : 304; }

bool vectors(const void* p, int64_t ld, int64_t rows, int dtype) {
    return host::aligned(p, 16) && (rows <= 1 || ld * dtype_bytes(dtype) % 16 == 0);
}

template <typename T, bool kWide, int kThreads, int kVecs>
int start(const Norm& A, int sms, cudaStream_t st) {
    constexpr int kGroups = kThreads == 32 ? 8 : 1, kBlock = kThreads == 32 ? 256 : kThreads;
    const int64_t blocks = (int64_t(A.rows) + kGroups - 1) / kGroups, most = int64_t(sms) * (2048 / kBlock);
    return launch_dependent(&norm_kernel<T, kWide, kThreads, kVecs>, dim3(unsigned(std::min(blocks, most))), kBlock, 0, st, A);
}

template <typename T, bool kWide>
int start_width(const Norm& A, int sms, cudaStream_t st) {
    if (A.cols <= 32 * kVec) return start<T, kWide, 32, 1>(A, sms, st);
    if (A.cols <= 32 * kVec * 4) return start<T, kWide, 32, 4>(A, sms, st);
    // few rows: more threads a row
    if (A.cols <= 1024 * kVec && A.rows <= 2 * sms) return start<T, kWide, 1024, 1>(A, sms, st);
    if (A.cols <= 256 * kVec * 2) return start<T, kWide, 256, 2>(A, sms, st);
    if (A.cols <= 256 * kVec * 4) return start<T, kWide, 256, 4>(A, sms, st);
    return start<T, kWide, 1024, 4>(A, sms, st);
}

// Rows that the queues take: whole vectors, more columns than a warp's eight rows and no more
// than a block's registers, and enough rows to fill the SMs.
bool queued(bool wide, int64_t rows, int64_t cols, int sms) {
    return wide && cols % kVec == 0 && cols > 32 * kVec * 2 && cols <= 8192 && rows > 2 * sms;
}

// Other rows of as many columns: threads that hold a row and what may lie before and after it in whole 16 bytes.
template <typename T>
int shift_threads(int64_t cols) {
    return int((cols * int(sizeof(T)) + 29 + 16 * Eight<T>::kUnits * 32 - 1) / (16 * Eight<T>::kUnits * 32) * 32);
}
// The gradient's few rows are quicker a column at a time (1024 x 2001 BF16: 11 us, through the queue 20;
// 4096 x 2001: 34 and 34); the forward pass is not (1024 x 2001: 8.5 and 8.3, 4096: 28 and 15).
bool shifted(bool queue, int64_t rows, int64_t cols, bool grad, int sms) {
    return !queue && cols > 32 * kVec * 2 && cols <= 8176 && rows > (grad ? 24 : 4) * sms;
}

template <typename T>
int start_shift(const Norm& A, int slot, int sms, cudaStream_t st) {
    constexpr int kBatches = 6 / Eight<T>::kUnits, kMost = kBatches * 2 * (1024 * Shifted<T>::kBytes + 16);
    const auto k = &norm_shift_kernel<T>;
    if (int rc = host::set_smem_once(reinterpret_cast<const void*>(k), slot, kMost)) return rc;
    const int threads = shift_threads<T>(A.cols);
    const int64_t batches = (int64_t(A.rows) + 1) / 2, most = int64_t(sms) * (1024 / threads);
    return launch_dependent(k, dim3(unsigned(std::min(batches, most))), threads,
                            kBatches * 2 * (threads * Shifted<T>::kBytes + 16), st, A);
}

template <typename T>
int start_grad_shift(const NormGrad& A, int slot, int parts, cudaStream_t st) {
    constexpr int kRows = 3 * 2 * (sizeof(T) == 2 ? 2 : 1), kMost = kRows * (1024 * Shifted<T>::kBytes + 16);
    const auto k = &norm_grad_shift_kernel<T>;
    if (int rc = host::set_smem_once(reinterpret_cast<const void*>(k), slot, kMost)) return rc;
    const int threads = shift_threads<T>(A.cols);
    return launch_dependent(k, dim3(unsigned(parts)), threads, kRows * (threads * Shifted<T>::kBytes + 16), st, A);
}

// Threads of a queued row of the gradient, eight columns each (16 past 4096 columns), and blocks an SM.
int queue_threads(int64_t cols) { return int((cols + (cols > 4096 ? 511 : 255)) / (cols > 4096 ? 512 : 256) * 32); }
int queue_blocks(int64_t cols) { return cols > 4096 ? 1 : 1024 / queue_threads(cols); }

template <typename T, bool kCodes>
int start_queue(const Norm& A, int slot, int sms, cudaStream_t st) {
    using Q = Queue<T, 1, 2, 1>;
    const auto k = &norm_queue_kernel<T, kCodes>;
    if (int rc = host::set_smem_once(reinterpret_cast<const void*>(k), slot, Q::bytes(1024))) return rc;
    const int threads = int((A.cols + 255) / 256 * 32);
    const int64_t batches = (int64_t(A.rows) + 1) / 2, most = int64_t(sms) * (1024 / threads);
    return launch_dependent(k, dim3(unsigned(std::min(batches, most))), threads, Q::bytes(threads), st, A);
}

template <typename T, int kVecs>
int start_grad_queue(const NormGrad& A, int slot, int parts, cudaStream_t st) {
    using Q = Queue<T, kVecs, sizeof(T) == 2 ? 2 : 1, 2>;
    const auto k = &norm_grad_queue_kernel<T, kVecs>;
    if (int rc = host::set_smem_once(reinterpret_cast<const void*>(k), slot, Q::bytes(512))) return rc;
    const int threads = queue_threads(A.cols);
    return launch_dependent(k, dim3(unsigned(parts)), threads, Q::bytes(threads), st, A);
}

template <typename T>
int start_grad_queue(const NormGrad& A, int slot, int parts, cudaStream_t st) {
    return A.cols <= 4096 ? start_grad_queue<T, 1>(A, slot, parts, st) : start_grad_queue<T, 2>(A, slot + 1, parts, st);
}

template <typename T>
int start_type(const Norm& A, bool wide, int slot, int sms, cudaStream_t st) {
    const bool queue = queued(wide, A.rows, A.cols, sms);
    if (queue) return A.q ? start_queue<T, true>(A, slot, sms, st) : start_queue<T, false>(A, slot + 1, sms, st);
    if (!A.q && shifted(queue, A.rows, A.cols, false, sms)) return start_shift<T>(A, slot + 2, sms, st);
    if (A.cols > kLongest)
        return launch_dependent(&norm_long_kernel<T>, dim3(unsigned(std::min(A.rows, sms * 2))), 1024, 0, st, A);
    return wide ? start_width<T, true>(A, sms, st) : start_width<T, false>(A, sms, st);
}

// Blocks of the gradient, each of which leaves a part.
int parts_of(int64_t rows, int64_t cols, bool wide, int dtype, int sms) {
    const bool queue = queued(wide, rows, cols, sms);
    if (queue || shifted(queue, rows, cols, true, sms)) {
        const int per = dtype == FP8Z_F32 ? 1 : 2;
        const int blocks = queue ? queue_blocks(cols) : 1024 / (dtype == FP8Z_F32 ? shift_threads<float>(cols) : shift_threads<__half>(cols));
        // a part is written and read again: at least four batches a block, once every SM has one
        const int64_t batches = (rows + per - 1) / per;
        return int(std::min<int64_t>({batches, std::max<int64_t>(batches / 4, sms), int64_t(sms) * blocks, most_parts(cols)}));
    }
    const int64_t blocks = cols <= 32 * kVec * 2 ? (rows + 7) / 8 : rows;
    return int(std::min<int64_t>({std::max<int64_t>(blocks, 1), int64_t(sms) * (cols <= 256 * kVec ? 2 : 1), most_parts(cols)}));
}

template <typename T, bool kWide, int kThreads, int kVecs>
int start_grad(const NormGrad& A, int parts, cudaStream_t st) {
    return launch_dependent(&norm_grad_kernel<T, kWide, kThreads, kVecs>, dim3(unsigned(parts)), kThreads == 32 ? 256 : kThreads,
                            0, st, A);
}

template <typename T, bool kWide>
int start_grad_width(const NormGrad& A, int parts, cudaStream_t st) {
    if (A.cols <= 32 * kVec * 2) return start_grad<T, kWide, 32, 2>(A, parts, st);
    if (A.cols <= 256 * kVec) return start_grad<T, kWide, 256, 1>(A, parts, st);
    if (A.cols <= 512 * kVec) return start_grad<T, kWide, 512, 1>(A, parts, st);
    if (A.cols <= 1024 * kVec) return start_grad<T, kWide, 1024, 1>(A, parts, st);
    return start_grad<T, kWide, 1024, 4>(A, parts, st);
}

template <typename T>
int start_grad_type(const NormGrad& A, bool wide, int slot, int parts, int sms, cudaStream_t st) {
    const bool queue = queued(wide, A.rows, A.cols, sms);
    if (queue) return start_grad_queue<T>(A, slot, parts, st);
    if (shifted(queue, A.rows, A.cols, true, sms)) return start_grad_shift<T>(A, slot + 2, parts, st);
    if (A.cols > kLongest) return launch_dependent(&norm_grad_long_kernel<T>, dim3(unsigned(parts)), 1024, 0, st, A);
    return wide ? start_grad_width<T, true>(A, parts, st) : start_grad_width<T, false>(A, parts, st);
}

bool shape_ok(const fp8z_layer_norm_args& a) {
    const int64_t most = 1LL << 30;
    return a.rows >= 0 && a.cols >= 1 && a.rows <= most && a.cols <= (1LL << 24) && dtype_ok(a.dtype) &&
           (a.param_dtype == FP8Z_F32 || a.param_dtype == a.dtype) && a.x_ld >= a.cols && a.x_ld <= (1LL << 38);
}

}  // namespace
}  // namespace fp8z

extern "C" int fp8z_layer_norm(const void* x, const void* weight, const void* bias, const fp8z_layer_norm_args* args, void* y,
                               float* mean, float* rstd, uint8_t* q, float* q_scale, void* stream) {
    using namespace fp8z;
    const host::NvtxRange nvtx_range("fp8z_layer_norm");
    if (!args || !shape_ok(*args)) return FP8Z_EINVAL;
    const fp8z_layer_norm_args& a = *args;
    if (!std::isfinite(a.eps) || a.eps < 0.0f || (a.pow2 != 0 && a.pow2 != 1)) return FP8Z_EINVAL;
    if ((y && (a.y_ld < a.cols || a.y_ld > (1LL << 38))) || (q != nullptr) != (q_scale != nullptr)) return FP8Z_EINVAL;
    if (q && a.cols % FP8Z_BLOCK) return FP8Z_EINVAL;
    if (a.rows == 0) return FP8Z_OK;
    if (!x || (!y && !q && !mean && !rstd)) return FP8Z_EINVAL;
    const int size = dtype_bytes(a.dtype), psize = dtype_bytes(a.param_dtype);
    if (!host::aligned(x, size) || !host::aligned(y, size) || !host::aligned(weight, psize) || !host::aligned(bias, psize) ||
        !host::aligned(mean, 4) || !host::aligned(rstd, 4) || !host::aligned(q, 16) || !host::aligned(q_scale, 4))
        return FP8Z_EALIGN;
    const bool wide = vectors(x, a.x_ld, a.rows, a.dtype) && vectors(weight, 0, 1, 0) && vectors(bias, 0, 1, 0) &&
                      (!y || vectors(y, a.y_ld, a.rows, a.dtype));
    if (q && !wide && a.cols <= kLongest) return FP8Z_EALIGN;
    int sms = 0;
    if (int rc = host::device_sms(&sms)) return rc;
    const Norm A = {int(a.rows), int(a.cols), x, a.x_ld, weight, bias, a.param_dtype, y, a.y_ld, mean, rstd, a.eps,
                    q, q_scale, a.pow2};
    const auto st = static_cast<cudaStream_t>(stream);
    if (a.dtype == FP8Z_F32) return start_type<float>(A, wide, 27, sms, st);
    if (a.dtype == FP8Z_BF16) return start_type<__nv_bfloat16>(A, wide, 31, sms, st);
    return start_type<__half>(A, wide, 35, sms, st);
}

extern "C" int64_t fp8z_layer_norm_grad_workspace(int64_t rows, int64_t cols) {
    using namespace fp8z;
    if (rows < 0 || rows > (1LL << 30) || cols < 1 || cols > (1LL << 24)) return FP8Z_EINVAL;
    return std::min<int64_t>(std::max<int64_t>(rows, 1), most_parts(cols)) * 2 * cols * 4;
}

extern "C" int fp8z_layer_norm_grad(const void* dy, const void* x, const void* weight, const float* mean, const float* rstd,
                                    const fp8z_layer_norm_args* args, void* dx, void* dweight, void* dbias, void* workspace,
                                    int64_t workspace_bytes, void* stream) {
    using namespace fp8z;
    const host::NvtxRange nvtx_range("fp8z_layer_norm_grad");
    if (!args || !shape_ok(*args)) return FP8Z_EINVAL;
    const fp8z_layer_norm_args& a = *args;
    const int64_t far = 1LL << 38;
    if (a.dy_ld < a.cols || a.dy_ld > far || (dx && (a.dx_ld < a.cols || a.dx_ld > far))) return FP8Z_EINVAL;
    if ((a.accumulate != 0 && a.accumulate != 1) || !workspace) return FP8Z_EINVAL;
    if (a.rows > 0 && (!dy || !x || !mean || !rstd)) return FP8Z_EINVAL;
    const int size = dtype_bytes(a.dtype), psize = dtype_bytes(a.param_dtype);
    if (!host::aligned(dy, size) || !host::aligned(x, size) || !host::aligned(dx, size) || !host::aligned(weight, psize) ||
        !host::aligned(dweight, psize) || !host::aligned(dbias, psize) || !host::aligned(mean, 4) || !host::aligned(rstd, 4) ||
        !host::aligned(workspace, 16))
        return FP8Z_EALIGN;
    if (workspace_bytes < fp8z_layer_norm_grad_workspace(a.rows, a.cols)) return FP8Z_ENOSPACE;
    int sms = 0;
    if (int rc = host::device_sms(&sms)) return rc;
    const auto st = static_cast<cudaStream_t>(stream);
    auto* part = static_cast<float*>(workspace);
    int parts = 0;
    if (a.rows > 0) {
        const bool wide = vectors(x, a.x_ld, a.rows, a.dtype) && vectors(dy, a.dy_ld, a.rows, a.dtype) && vectors(weight, 0, 1, 0) &&
                          (!dx || vectors(dx, a.dx_ld, a.rows, a.dtype));
        parts = parts_of(a.rows, a.cols, wide, a.dtype, sms);
        const NormGrad A = {int(a.rows), int(a.cols), dy, x, a.dy_ld, a.x_ld, a.dx_ld, weight, a.param_dtype, mean, rstd, dx, part};
        const int rc = a.dtype == FP8Z_F32 ? start_grad_type<float>(A, wide, 39, parts, sms, st)
                       : a.dtype == FP8Z_BF16 ? start_grad_type<__nv_bfloat16>(A, wide, 42, parts, sms, st)
                                              : start_grad_type<__half>(A, wide, 45, parts, sms, st);
        if (rc) return rc;
    }
    if (!dweight && !dbias) return FP8Z_OK;
    const dim3 grid(unsigned((a.cols + 31) / 32), dbias ? 2 : 1);
    const auto join = [&](auto* dw, auto* db) {
        using P = std::remove_pointer_t<decltype(dw)>;
        return launch_dependent(&norm_parts_kernel<P>, grid, 1024, 0, st, part, parts, int(a.cols), dw, db, a.accumulate);
    };
    if (a.param_dtype == FP8Z_F32) return join(static_cast<float*>(dweight), static_cast<float*>(dbias));
    if (a.param_dtype == FP8Z_BF16) return join(static_cast<__nv_bfloat16*>(dweight), static_cast<__nv_bfloat16*>(dbias));
    return join(static_cast<__half*>(dweight), static_cast<__half*>(dbias));
}
