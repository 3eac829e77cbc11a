// xent.cu -- softmax cross entropy of a vocabulary projection, with its gradient,
// without keeping the logits.
//
//   l[t][v] = sum_h x[t][h] w[v][h]
//   lse[t]  = log sum_v exp l[t][v],   loss[t] = lse[t] - l[t][y_t]
//   P[t][v] = (exp(l[t][v] - lse[t]) - [v == y_t]) * keep[t]
//   dx = a * P w,   dw = a * P^T x,   a = grad_scale / (number of kept tokens, or 1)
//
// The loss needs one product whose epilogue turns each 256 columns of logits
// into a running maximum and a sum of exponentials per token.  The gradient
// goes through the vocabulary in pieces: the logits of a piece are computed
// again, turned into P in the epilogue and written in 16 bits; two products
// read it.  What is kept is one piece of P, never the logits.
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "fp8z.h"
#include "fp8z_device.cuh"
#include "fp8z_elem.cuh"
#include "fp8z_host.h"
#include "fp8z_tcgen05.cuh"

namespace fp8z {
namespace {

constexpr int kTM = 128, kTN = 256, kBK = 64;          // output tile, K per stage
constexpr int kStages = 4;
constexpr int kBytesA = kTM * kBK * 2, kBytesB = kTN * kBK * 2, kStageBytes = kBytesA + kBytesB;
constexpr int kThreads = 256;                          // warp 0 loads, warp 1 multiplies, warps 4-7 read the sums
constexpr int kTmemCols = 512;                         // two accumulators of 256 columns
constexpr int kNumBars = 2 * kStages + 5;
constexpr int kSmem = kStages * kStageBytes + kNumBars * 8 + 16 + 1024;
constexpr float kLog2e = 1.4426950408889634f;

enum Epilogue { kStats, kProb, kSum, kWeight };

struct MmaArgs {
    int m, n;                 // rows and columns of the result
    int mt, nt, splits;       // tiles, and parts of the K loop
    int kb;                   // K blocks of 64
    int b_wrap;               // B's K block returns to 0 here (the two parts of P share one x)
    int b_n0, b_k0;           // where B starts, in elements
    int bf16;
    int64_t timeout_ns;
    int32_t* dev_status;
    // kStats, kProb: rows are tokens, columns words v0 + n of this piece
    int v0;
    const int32_t* target;    // -1: takes no part in the loss
    float2* part;             // [tile][rows_pad] maximum and sum
    float* target_logit;
    const float* lse;
    void *p_hi, *p_lo;        // [rows_pad][p_ld]
    int64_t p_ld;
    int rows_pad;
    float p_scale;
    // kSum: FP32 [splits][rows_pad][out_ld];  kWeight: out + v0 rows
    void* out;
    int64_t out_ld;
    int out_dtype, accumulate, vec;
    const float* alpha;
};

struct TileAt {
    int m, n, k0, k1, split;
};

// Eight row tiles by all column tiles at a time, row tiles innermost: the
// blocks that run together share few rows and columns of operands.
__device__ __forceinline__ TileAt tile_at(const MmaArgs& A, int t) {
    const int per = A.mt * A.nt, split = t / per, r = t - split * per;
    const int group = r / (8 * A.nt), first = group * 8, rows = min(8, A.mt - first), in = r - group * 8 * A.nt;
    TileAt a;
    a.m = first + in % rows;
    a.n = in / rows;
    a.split = split;
    a.k0 = int(int64_t(A.kb) * split / A.splits);
    a.k1 = int(int64_t(A.kb) * (split + 1) / A.splits);
    return a;
}

__device__ __forceinline__ uint32_t pack16(float a, float b, int bf16) {
    uint32_t r;
    if (bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ float2 unpack16(uint32_t u, int bf16) {
    if (bf16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    const __half2 h = *reinterpret_cast<const __half2*>(&u);
    return __half22float2(h);
}

// Running maximum and sum of exponentials of one row over the tile's columns.
__device__ __forceinline__ void epilogue_stats(const MmaArgs& A, const TileAt& t, uint32_t acc, int row) {
    const int n_valid = min(kTN, A.n - t.n * kTN);
    const int target = row < A.m ? A.target[row] - (A.v0 + t.n * kTN) : -1;
    float mx = -INFINITY, sum = 0.0f;
    for (int c = 0; c < n_valid; c += 32) {
        uint32_t r[32];
        tmem_ld32(r, acc + c);
        tmem_wait_ld();
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (c + j >= n_valid) r[j] = __float_as_uint(-INFINITY);
            top = fmaxf(top, __uint_as_float(r[j]));
        }
        const float m2 = fmaxf(mx, top), ref = m2 == -INFINITY ? 0.0f : m2 * kLog2e;
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) s += ex2(fmaf(__uint_as_float(r[j]), kLog2e, -ref));
        sum = fmaf(sum, ex2(fmaf(mx, kLog2e, -ref)), s);
        mx = m2;
        if (target >= c && target < c + 32) {
            float x = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (target == c + j) x = __uint_as_float(r[j]);
            A.target_logit[row] = x;
        }
    }
    if (row < A.m) A.part[size_t(A.v0 / kTN + t.n) * A.rows_pad + row] = make_float2(mx, sum);
}

// P in 16 bits, and what the rounding left in another 16 where FP32 weight
// gradients are asked for.  Rows and columns past the end are written as zeros:
// the products read whole tiles.
__device__ __forceinline__ void epilogue_prob(const MmaArgs& A, const TileAt& t, uint32_t acc, int row) {
    const int n_valid = min(kTN, A.n - t.n * kTN);
    const int y = row < A.m ? A.target[row] : -1;
    const int target = y - (A.v0 + t.n * kTN);
    const float ref = y >= 0 ? A.lse[row] * kLog2e : 0.0f;
    const size_t at = size_t(row) * A.p_ld + size_t(t.n) * kTN;
    uint4* hi = reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.p_hi) + at);
    uint4* lo = A.p_lo ? reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.p_lo) + at) : nullptr;
    for (int c = 0; c < kTN; c += 32) {
        uint32_t r[32];
        tmem_ld32(r, acc + c);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t h[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float p[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int j = q * 8 + i * 2 + k;
                    float v = ex2(fmaf(__uint_as_float(r[j]), kLog2e, -ref));
                    if (target == c + j) v -= 1.0f;
                    p[k] = (y >= 0 && c + j < n_valid) ? v * A.p_scale : 0.0f;
                }
                h[i] = pack16(p[0], p[1], A.bf16);
                const float2 w = unpack16(h[i], A.bf16);
                l[i] = pack16(p[0] - w.x, p[1] - w.y, A.bf16);
            }
            hi[c / 8 + q] = make_uint4(h[0], h[1], h[2], h[3]);
            if (lo) lo[c / 8 + q] = make_uint4(l[0], l[1], l[2], l[3]);
        }
    }
}

__device__ __forceinline__ void epilogue_sum(const MmaArgs& A, const TileAt& t, uint32_t acc, int row) {
    float* out = static_cast<float*>(A.out) + (size_t(t.split) * A.rows_pad + row) * A.out_ld + size_t(t.n) * kTN;
    for (int c = 0; c < kTN && t.n * kTN + c < A.n; c += 32) {
        uint32_t r[32];
        tmem_ld32(r, acc + c);
        tmem_wait_ld();
        if (t.k0 == t.k1)
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = 0;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            if (t.n * kTN + c + j >= A.n) break;           // out_ld is a multiple of 4
            float4* p = reinterpret_cast<float4*>(out + c + j);
            float4 v = make_float4(__uint_as_float(r[j]), __uint_as_float(r[j + 1]), __uint_as_float(r[j + 2]),
                                   __uint_as_float(r[j + 3]));
            if (A.accumulate) {
                const float4 o = *p;
                v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
            }
            *p = v;
        }
    }
}

template <typename T>
__device__ __forceinline__ void weight_chunk(T* p, const uint32_t (&r)[32], int n, float a, const MmaArgs& A) {
    if (A.vec && n >= 32) {
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
            Pack<T, 8> y;
            if (A.accumulate) y = ld_plain<T, 8>(p + j);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = __uint_as_float(r[j + i]) * a;
                y.v[i] = Elem<T>::narrow(A.accumulate ? Elem<T>::widen(y.v[i]) + v : v);
            }
            st_vec<T, 8>(p + j, y);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j < n) {
                const float v = __uint_as_float(r[j]) * a;
                p[j] = Elem<T>::narrow(A.accumulate ? Elem<T>::widen(p[j]) + v : v);
            }
        }
    }
}

__device__ __forceinline__ void epilogue_weight(const MmaArgs& A, const TileAt& t, uint32_t acc, int row) {
    const float a = *A.alpha;
    for (int c = 0; c < kTN && t.n * kTN + c < A.n; c += 32) {
        uint32_t r[32];
        tmem_ld32(r, acc + c);
        tmem_wait_ld();
        if (t.k0 == t.k1)
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = 0;
        if (row >= A.m) continue;
        const int col = t.n * kTN + c;
        const size_t at = size_t(A.v0 + row) * A.out_ld + col;
        const int n = A.n - col;
        if (A.out_dtype == FP8Z_F32) weight_chunk(static_cast<float*>(A.out) + at, r, n, a, A);
        else if (A.out_dtype == FP8Z_BF16) weight_chunk(static_cast<__nv_bfloat16*>(A.out) + at, r, n, a, A);
        else weight_chunk(static_cast<__half*>(A.out) + at, r, n, a, A);
    }
}

// One block of 128 x 256 results at a time: a warp keeps kStages tiles of
// operands in flight, one thread issues the products into one of two
// accumulators in tensor memory while four warps read the other.
template <bool kAMn, bool kBMn, int kEpi>
__global__ void __launch_bounds__(kThreads, 1)
    mma_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
               const __grid_constant__ MmaArgs A) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_addr(smem_raw));
    const uint32_t bars = base + kStages * kStageBytes;
    auto full = [&](int s) { return bars + s * 8; };
    auto empty = [&](int s) { return bars + (kStages + s) * 8; };
    auto tfull = [&](int b) { return bars + (2 * kStages + b) * 8; };
    auto tempty = [&](int b) { return bars + (2 * kStages + 2 + b) * 8; };
    const uint32_t drain = bars + (2 * kStages + 4) * 8;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kStages * kStageBytes + kNumBars * 8);
    volatile uint32_t* tmem_at = reinterpret_cast<volatile uint32_t*>(smem + kStages * kStageBytes + kNumBars * 8 + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 2) tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_at)), kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;
    const Watchdog wd{abort_flag, A.dev_status, A.timeout_ns};
    const int tiles = A.mt * A.nt * A.splits;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, ph = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const TileAt at = tile_at(A, t);
                for (int k = at.k0; k < at.k1; ++k) {
                    if (!mbar_wait_bounded(empty(s), ph ^ 1, wd)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = base + s * kStageBytes, sb = sa + kBytesA;
                    mbar_arrive_expect_tx(full(s), kStageBytes);
                    const int ka = k * kBK, kb = (k >= A.b_wrap ? k - A.b_wrap : k) * kBK + A.b_k0;
                    if constexpr (kAMn) {
#pragma unroll
                        for (int j = 0; j < kTM / 64; ++j)
                            tma_load_2d(sa + j * (64 * kBK * 2), &ta, at.m * kTM + j * 64, ka, full(s));
                    } else {
                        tma_load_2d(sa, &ta, ka, at.m * kTM, full(s));
                    }
                    if constexpr (kBMn) {
#pragma unroll
                        for (int j = 0; j < kTN / 64; ++j)
                            tma_load_2d(sb + j * (64 * kBK * 2), &tb, A.b_n0 + at.n * kTN + j * 64, kb, full(s));
                    } else {
                        tma_load_2d(sb, &tb, kb, A.b_n0 + at.n * kTN, full(s));
                    }
                    ++issued;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // whatever a wait elsewhere gave up on: every copy lands before the block ends
            for (int i = 0; i < kStages && issued > i; ++i)
                mbar_wait_drain(full(i), uint32_t(((issued - i + kStages - 1) / kStages - 1) & 1), A.dev_status);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = umma_idesc(A.bf16 != 0, kAMn, kBMn, kTM, kTN);
            int s = 0, ph = 0, b = 0, bph = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const TileAt at = tile_at(A, t);
                if (!mbar_wait_bounded(tempty(b), bph ^ 1, wd)) break;
                tc_fence_after();
                for (int k = at.k0; k < at.k1; ++k) {
                    if (!mbar_wait_bounded(full(s), ph, wd)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = base + s * kStageBytes, sb = sa + kBytesA;
                    const uint64_t da = umma_desc(sa, kAMn ? 64 * kBK * 2 : 16, 1024);
                    const uint64_t db = umma_desc(sb, kBMn ? 64 * kBK * 2 : 16, 1024);
#pragma unroll
                    for (int i = 0; i < kBK / 16; ++i)      // 16 of K: 32 bytes of a row, or 16 rows of 128 bytes
                        umma_f16(tmem + b * kTN, da + i * (kAMn ? 128 : 2), db + i * (kBMn ? 128 : 2), idesc,
                                 k != at.k0 || i != 0);
                    umma_commit(empty(s));
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                if (!ok) break;
                umma_commit(tfull(b));
                if (b) bph ^= 1;
                b ^= 1;
            }
            umma_commit(drain);            // and every product is done before tensor memory is freed
            mbar_wait_drain(drain, 0, A.dev_status);
        }
    } else if (warp >= 4) {
        const int quarter = warp - 4;
        int b = 0, bph = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
            const TileAt at = tile_at(A, t);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(tfull(b), bph, wd))) break;
            tc_fence_after();
            const uint32_t acc = tmem + b * kTN + (uint32_t(quarter * 32) << 16);
            const int row = at.m * kTM + quarter * 32 + lane;
            if constexpr (kEpi == kStats) epilogue_stats(A, at, acc, row);
            else if constexpr (kEpi == kProb) epilogue_prob(A, at, acc, row);
            else if constexpr (kEpi == kSum) epilogue_sum(A, at, acc, row);
            else epilogue_weight(A, at, acc, row);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty(b));
            if (b) bph ^= 1;
            b ^= 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------ small kernels
// Targets as int32 (-1: ignored or out of range), once.
__global__ void target_kernel(const void* __restrict__ targets, int wide, int n, int64_t ignore, int64_t vocab,
                              int32_t* __restrict__ out, int32_t* dev_status) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int64_t y = wide ? static_cast<const int64_t*>(targets)[i] : static_cast<const int32_t*>(targets)[i];
    const bool ok = y != ignore && y >= 0 && y < vocab;
    if (y != ignore && !ok) report_status(dev_status, FP8Z_EINVAL);
    out[i] = ok ? int32_t(y) : -1;
}

// 16-bit rows copied to a stride the tensor maps can step over, zeros after the end.
__global__ void pad_rows_kernel(const uint16_t* __restrict__ src, int64_t ld, int64_t rows, int cols, int cols_pad,
                                uint16_t* __restrict__ dst) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int c = threadIdx.x; c < cols_pad; c += blockDim.x)
            dst[r * cols_pad + c] = c < cols ? src[r * ld + c] : uint16_t(0);
}

// lse and loss of 32 rows from the tiles' maxima and sums, eight threads a row.
__global__ void __launch_bounds__(256) rows_kernel(const float2* __restrict__ part, int tiles, int n, int rows_pad,
                                                   const int32_t* __restrict__ target,
                                                   const float* __restrict__ target_logit, float* __restrict__ lse_ws,
                                                   float* __restrict__ lse_out, float* __restrict__ loss) {
    __shared__ float2 sh[8][32];
    const int r = threadIdx.x & 31, g = threadIdx.x >> 5, row = blockIdx.x * 32 + r;
    float m = -INFINITY, s = 0.0f;
    auto add = [&](float2 p) {
        const float m2 = fmaxf(m, p.x), ref = m2 == -INFINITY ? 0.0f : m2;
        s = s * ex2((m - ref) * kLog2e) + p.y * ex2((p.x - ref) * kLog2e);
        m = m2;
    };
    if (row < n)
        for (int t = g; t < tiles; t += 8) add(part[size_t(t) * rows_pad + row]);
    sh[g][r] = make_float2(m, s);
    __syncthreads();
    if (g != 0 || row >= n) return;
    for (int k = 1; k < 8; ++k) add(sh[k][r]);
    const float lse = m + logf(s);
    lse_ws[row] = lse;
    if (lse_out) lse_out[row] = lse;
    loss[row] = target[row] >= 0 ? lse - target_logit[row] : 0.0f;
}

__global__ void __launch_bounds__(1024) total_kernel(const float* __restrict__ loss, const int32_t* __restrict__ target,
                                                     int n, int mean, float scale, float* __restrict__ total,
                                                     float* __restrict__ alpha) {
    __shared__ double sh[32];
    __shared__ int sc[32];
    double s = 0.0;
    int c = 0;
    for (int i = threadIdx.x; i < n; i += 1024) {
        s += double(loss[i]);
        c += target[i] >= 0;
    }
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_down_sync(0xFFFFFFFFu, s, o);
        c += __shfl_down_sync(0xFFFFFFFFu, c, o);
    }
    if ((threadIdx.x & 31) == 0) {
        sh[threadIdx.x >> 5] = s;
        sc[threadIdx.x >> 5] = c;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    s = 0.0;
    c = 0;
    for (int w = 0; w < 32; ++w) {
        s += sh[w];
        c += sc[w];
    }
    const double by = mean ? double(c > 0 ? c : 1) : 1.0;
    total[0] = float(s / by);
    total[1] = float(c);
    if (alpha) *alpha = float(double(scale) / by);
}

// dx = a * the sum of the K parts.
template <typename T>
__global__ void __launch_bounds__(256) finish_dx_kernel(const float* __restrict__ sum, int splits, int64_t part_stride,
                                                        int64_t sum_ld, int n, int hidden, const float* __restrict__ alpha,
                                                        T* __restrict__ dx, int64_t dx_ld) {
    const float a = *alpha;
    const int c = (blockIdx.y * 256 + threadIdx.x) * 4;
    const int64_t row = blockIdx.x;
    if (c >= hidden) return;
    float v[4] = {};
    for (int s = 0; s < splits; ++s) {
        const float4 q = *reinterpret_cast<const float4*>(sum + s * part_stride + row * sum_ld + c);
        v[0] += q.x;
        v[1] += q.y;
        v[2] += q.z;
        v[3] += q.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (c + i < hidden) dx[row * dx_ld + c + i] = Elem<T>::narrow(v[i] * a);
}

template <typename T>
__global__ void zero_rows_kernel(T* out, int64_t ld, int64_t rows, int cols) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int c = threadIdx.x; c < cols; c += blockDim.x) out[r * ld + c] = Elem<T>::narrow(0.0f);
}

// ------------------------------------------------------------------ launches
struct Layout {
    int64_t rows_pad, hidden_pad, vocab_tiles, piece, pieces, parts;
    int splits;
    bool copy_x, copy_w;
    size_t x, w, target, target_logit, lse, part, alpha, p, sum, total;
};

constexpr int64_t kPieceBytes = 1LL << 30;        // of P, unless the caller's workspace is smaller
constexpr int kSms = 152;                         // the layout's, the same for the size query and the call

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

bool args_ok(const fp8z_xent_args& a) {
    if (a.tokens < 0 || a.tokens > (1 << 24) || a.hidden < 1 || a.hidden > (1 << 20) || a.vocab < 1 ||
        a.vocab > (1 << 28))
        return false;
    if (a.dtype != FP8Z_BF16 && a.dtype != FP8Z_F16) return false;
    if (a.targets_dtype != FP8Z_I32 && a.targets_dtype != FP8Z_I64) return false;
    if (a.x_ld < a.hidden || a.w_ld < a.hidden) return false;
    if (a.reduction != FP8Z_MEAN && a.reduction != FP8Z_SUM) return false;
    return true;
}

bool grad_args_ok(const fp8z_xent_args& a) {
    return (a.dw_dtype == FP8Z_F32 || a.dw_dtype == a.dtype) && a.dx_ld >= a.hidden && a.dw_ld >= a.hidden &&
           (a.accumulate_dw == 0 || a.accumulate_dw == 1) && std::isfinite(a.grad_scale);
}

// Rows a tensor map can step over: base and stride multiples of 16 bytes.
bool map_ok(const void* p, int64_t ld, int64_t hidden) {
    return host::aligned(p, 16) && ld % 8 == 0 && hidden % 8 == 0;
}

Layout layout(const fp8z_xent_args& a, bool grad, bool copy_x, bool copy_w, int64_t have) {
    Layout L;
    std::memset(&L, 0, sizeof(L));
    L.copy_x = copy_x;
    L.copy_w = copy_w;
    L.rows_pad = up(a.tokens > 0 ? a.tokens : 1, kTM);
    L.hidden_pad = up(a.hidden, 8);
    L.vocab_tiles = (a.vocab + kTN - 1) / kTN;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t r = at;
        at += size_t(up(bytes, 256));
        return r;
    };
    L.x = take(copy_x ? a.tokens * L.hidden_pad * 2 : 0);
    L.w = take(copy_w ? a.vocab * L.hidden_pad * 2 : 0);
    L.target = take(L.rows_pad * 4);
    L.target_logit = take(L.rows_pad * 4);
    L.lse = take(L.rows_pad * 4);
    L.alpha = take(4);
    L.part = take(L.vocab_tiles * L.rows_pad * 8);
    if (grad) {
        L.parts = a.dw_dtype == FP8Z_F32 ? 2 : 1;
        const int64_t dx_tiles = L.rows_pad / kTM * ((L.hidden_pad + kTN - 1) / kTN);
        const int64_t row_bytes = L.rows_pad * 2 * L.parts;          // of one word in P
        // few rows: the dx product is cut along the vocabulary until every SM has a part
        int64_t splits = (kSms + dx_tiles - 1) / dx_tiles;
        const int64_t vocab_blocks = L.vocab_tiles * (kTN / kBK);
        if (splits > vocab_blocks / 4) splits = vocab_blocks / 4;
        L.splits = int(splits < 1 ? 1 : splits);
        L.sum = take(int64_t(L.splits) * L.rows_pad * up(L.hidden_pad, 4) * 4);
        int64_t room = kPieceBytes;
        if (have >= 0 && have - int64_t(at) < room) room = have - int64_t(at);
        int64_t tiles = room / (row_bytes * kTN);
        if (tiles < 1) tiles = 1;
        if (tiles > L.vocab_tiles) tiles = L.vocab_tiles;
        L.pieces = (L.vocab_tiles + tiles - 1) / tiles;
        L.piece = (L.vocab_tiles + L.pieces - 1) / L.pieces * kTN;       // equal pieces
        L.p = take(row_bytes * L.piece);
    }
    L.total = at;
    return L;
}

bool make_map(CUtensorMap* map, const void* p, int64_t inner, int64_t rows, int64_t ld, int box_inner, int box_rows) {
    const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(host::tensor_map_encoder());
    if (!enc) return false;
    std::memset(map, 0, sizeof(*map));
    const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(rows)}, strides[1] = {cuuint64_t(ld * 2)};
    const cuuint32_t box[2] = {cuuint32_t(box_inner), cuuint32_t(box_rows)}, estr[2] = {1, 1};
    // 16-bit elements move as they are, whichever type they hold
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kAMn, bool kBMn, int kEpi>
int launch_mma(const CUtensorMap& ta, const CUtensorMap& tb, const MmaArgs& A, int sms, cudaStream_t st) {
    const auto k = &mma_kernel<kAMn, kBMn, kEpi>;
    if (int rc = host::set_smem_once(reinterpret_cast<const void*>(k), 12 + kEpi, kSmem)) return rc;
    const int64_t tiles = int64_t(A.mt) * A.nt * A.splits;
    k<<<unsigned(tiles < sms ? tiles : sms), kThreads, kSmem, st>>>(ta, tb, A);
    return cudaGetLastError() == cudaSuccess ? FP8Z_OK : FP8Z_ECUDA;
}

int run(const void* x, const void* w, const void* targets, const fp8z_xent_args* args, float* loss, float* lse,
        float* total, void* dx, void* dw, bool grad, void* workspace, int64_t workspace_bytes, int32_t* dev_status,
        void* stream) {
    if (!args || !args_ok(*args) || (grad && !grad_args_ok(*args))) return FP8Z_EINVAL;
    const fp8z_xent_args& a = *args;
    if (!w || !total || !workspace || (a.tokens > 0 && (!x || !targets || !loss))) return FP8Z_EINVAL;
    if (grad && (!dw || (a.tokens > 0 && !dx))) return FP8Z_EINVAL;
    if (!host::aligned(x, 2) || !host::aligned(w, 2) || !host::aligned(targets, a.targets_dtype == FP8Z_I64 ? 8 : 4) ||
        !host::aligned(loss, 4) || !host::aligned(lse, 4) || !host::aligned(total, 4) ||
        !host::aligned(workspace, 256) || !host::aligned(dev_status, 4) ||
        (grad && (!host::aligned(dx, 2) || !host::aligned(dw, dtype_bytes(a.dw_dtype)))))
        return FP8Z_EALIGN;
    int sms = 0;
    if (int rc = host::device_sms(&sms)) return rc;
    const bool copy_x = !map_ok(x, a.x_ld, a.hidden), copy_w = !map_ok(w, a.w_ld, a.hidden);
    const Layout L = layout(a, grad, copy_x, copy_w, workspace_bytes);
    if (workspace_bytes < int64_t(L.total)) return FP8Z_ENOSPACE;
    const auto st = static_cast<cudaStream_t>(stream);
    auto* ws = static_cast<uint8_t*>(workspace);
    const int n = int(a.tokens), hidden = int(a.hidden), vocab = int(a.vocab);
    auto* target = reinterpret_cast<int32_t*>(ws + L.target);
    auto* target_logit = reinterpret_cast<float*>(ws + L.target_logit);
    auto* lse_ws = reinterpret_cast<float*>(ws + L.lse);
    auto* alpha = reinterpret_cast<float*>(ws + L.alpha);
    auto* part = reinterpret_cast<float2*>(ws + L.part);

    if (n == 0) {
        total_kernel<<<1, 1024, 0, st>>>(loss, target, 0, a.reduction == FP8Z_MEAN, 1.0f, total, nullptr);
        if (grad && !a.accumulate_dw) {
            if (a.dw_dtype == FP8Z_F32)
                zero_rows_kernel<<<sms * 8, 256, 0, st>>>(static_cast<float*>(dw), a.dw_ld, a.vocab, hidden);
            else
                zero_rows_kernel<<<sms * 8, 256, 0, st>>>(static_cast<__half*>(dw), a.dw_ld, a.vocab, hidden);
        }
        return cudaGetLastError() == cudaSuccess ? FP8Z_OK : FP8Z_ECUDA;
    }
    const void *xp = x, *wp = w;
    int64_t x_ld = a.x_ld, w_ld = a.w_ld;
    if (copy_x) {
        pad_rows_kernel<<<sms * 8, 256, 0, st>>>(static_cast<const uint16_t*>(x), a.x_ld, n, hidden, int(L.hidden_pad),
                                                 reinterpret_cast<uint16_t*>(ws + L.x));
        xp = ws + L.x;
        x_ld = L.hidden_pad;
    }
    if (copy_w) {
        pad_rows_kernel<<<sms * 8, 256, 0, st>>>(static_cast<const uint16_t*>(w), a.w_ld, vocab, hidden,
                                                 int(L.hidden_pad), reinterpret_cast<uint16_t*>(ws + L.w));
        wp = ws + L.w;
        w_ld = L.hidden_pad;
    }
    target_kernel<<<(n + 255) / 256, 256, 0, st>>>(targets, a.targets_dtype == FP8Z_I64, n, a.ignore_index, a.vocab,
                                                   target, dev_status);
    CUtensorMap x_k, w_k;
    if (!make_map(&x_k, xp, L.hidden_pad, n, x_ld, kBK, kTM) || !make_map(&w_k, wp, L.hidden_pad, vocab, w_ld, kBK, kTN))
        return FP8Z_ECUDA;
    MmaArgs A;
    std::memset(&A, 0, sizeof(A));
    A.bf16 = a.dtype == FP8Z_BF16;
    A.timeout_ns = host::wait_limit_ns();
    A.dev_status = dev_status;
    A.m = n;
    A.rows_pad = int(L.rows_pad);
    A.n = vocab;
    A.mt = int(L.rows_pad / kTM);
    A.nt = int(L.vocab_tiles);
    A.splits = 1;
    A.kb = A.b_wrap = int((L.hidden_pad + kBK - 1) / kBK);
    A.target = target;
    A.part = part;
    A.target_logit = target_logit;
    if (int rc = launch_mma<false, false, kStats>(x_k, w_k, A, sms, st)) return rc;
    rows_kernel<<<(n + 31) / 32, 256, 0, st>>>(part, A.nt, n, A.rows_pad, target, target_logit, lse_ws, lse, loss);
    // FP16 P is kept times 2^12: probabilities down to 2^-36 stay normal numbers or close
    const float p_scale = A.bf16 ? 1.0f : 4096.0f;
    total_kernel<<<1, 1024, 0, st>>>(loss, target, n, a.reduction == FP8Z_MEAN, grad ? a.grad_scale / p_scale : 1.0f,
                                     total, grad ? alpha : nullptr);
    if (!grad) return cudaGetLastError() == cudaSuccess ? FP8Z_OK : FP8Z_ECUDA;

    auto* p_hi = ws + L.p;
    auto* p_lo = L.parts == 2 ? p_hi + L.rows_pad * L.piece * 2 : nullptr;
    auto* sum = reinterpret_cast<float*>(ws + L.sum);
    CUtensorMap p_k, w_mn, p_mn, x_mn;
    if (!make_map(&p_k, p_hi, L.piece, L.rows_pad, L.piece, kBK, kTM) ||
        !make_map(&w_mn, wp, L.hidden_pad, vocab, w_ld, 64, kBK) ||
        !make_map(&p_mn, p_hi, L.piece, L.rows_pad * L.parts, L.piece, 64, kBK) ||
        !make_map(&x_mn, xp, L.hidden_pad, n, x_ld, 64, kBK))
        return FP8Z_ECUDA;
    for (int64_t i = 0; i < L.pieces; ++i) {
        const int v0 = int(i * L.piece);
        if (v0 >= vocab) break;
        const int words = int(a.vocab - v0 < L.piece ? a.vocab - v0 : L.piece), tiles = (words + kTN - 1) / kTN;
        MmaArgs Q = A;                                  // P of the piece
        Q.n = words;
        Q.nt = tiles;
        Q.v0 = v0;
        Q.b_n0 = v0;
        Q.lse = lse_ws;
        Q.p_hi = p_hi;
        Q.p_lo = p_lo;
        Q.p_ld = L.piece;
        Q.p_scale = p_scale;
        if (int rc = launch_mma<false, false, kProb>(x_k, w_k, Q, sms, st)) return rc;
        MmaArgs D = A;                                  // dx += P w
        D.n = int(L.hidden_pad);
        D.nt = int((L.hidden_pad + kTN - 1) / kTN);
        D.kb = D.b_wrap = tiles * (kTN / kBK);
        D.splits = L.splits;
        D.b_k0 = v0;
        D.out = sum;
        D.out_ld = up(L.hidden_pad, 4);
        D.accumulate = i > 0;
        if (int rc = launch_mma<false, true, kSum>(p_k, w_mn, D, sms, st)) return rc;
        MmaArgs W = A;                                  // dw of the piece's words = P^T x
        W.m = words;
        W.n = hidden;
        W.mt = (words + kTM - 1) / kTM;
        W.nt = D.nt;
        W.b_wrap = int(L.rows_pad / kBK);
        W.kb = W.b_wrap * int(L.parts);
        W.v0 = v0;
        W.out = dw;
        W.out_ld = a.dw_ld;
        W.out_dtype = a.dw_dtype;
        W.accumulate = a.accumulate_dw;
        W.vec = host::aligned(dw, 16) && (a.dw_ld * dtype_bytes(a.dw_dtype)) % 16 == 0;
        W.alpha = alpha;
        if (int rc = launch_mma<true, true, kWeight>(p_mn, x_mn, W, sms, st)) return rc;
    }
    const dim3 grid(unsigned(n), unsigned((hidden + 1023) / 1024));
    const int64_t sum_ld = up(L.hidden_pad, 4);
    if (A.bf16)
        finish_dx_kernel<<<grid, 256, 0, st>>>(sum, L.splits, L.rows_pad * sum_ld, sum_ld, n, hidden, alpha,
                                               static_cast<__nv_bfloat16*>(dx), a.dx_ld);
    else
        finish_dx_kernel<<<grid, 256, 0, st>>>(sum, L.splits, L.rows_pad * sum_ld, sum_ld, n, hidden, alpha,
                                               static_cast<__half*>(dx), a.dx_ld);
    return cudaGetLastError() == cudaSuccess ? FP8Z_OK : FP8Z_ECUDA;
}

}  // namespace
}  // namespace fp8z

extern "C" int64_t fp8z_linear_xent_workspace(const void* x, const void* w, const fp8z_xent_args* args,
                                              int32_t with_grad, int64_t piece_words) {
    using namespace fp8z;
    if (!args || !args_ok(*args) || (with_grad && !grad_args_ok(*args)) || piece_words < 0) return FP8Z_EINVAL;
    const bool cx = !map_ok(x, args->x_ld, args->hidden), cw = !map_ok(w, args->w_ld, args->hidden);
    Layout L = layout(*args, with_grad != 0, cx, cw, -1);
    if (with_grad && piece_words > 0) {
        const int64_t less = L.piece - up(piece_words, kTN);
        if (less > 0) return int64_t(L.total) - less * L.rows_pad * 2 * L.parts;
    }
    return int64_t(L.total);
}

extern "C" int fp8z_linear_xent(const void* x, const void* w, const void* targets, const fp8z_xent_args* args,
                                float* loss, float* lse, float* total, void* workspace, int64_t workspace_bytes,
                                int32_t* dev_status, void* stream) {
    const fp8z::host::NvtxRange nvtx_range("fp8z_linear_xent");
    return fp8z::run(x, w, targets, args, loss, lse, total, nullptr, nullptr, false, workspace, workspace_bytes,
                     dev_status, stream);
}

extern "C" int fp8z_linear_xent_grad(const void* x, const void* w, const void* targets, const fp8z_xent_args* args,
                                     float* loss, float* lse, float* total, void* dx, void* dw, void* workspace,
                                     int64_t workspace_bytes, int32_t* dev_status, void* stream) {
    const fp8z::host::NvtxRange nvtx_range("fp8z_linear_xent_grad");
    return fp8z::run(x, w, targets, args, loss, lse, total, dx, dw, true, workspace, workspace_bytes, dev_status,
                     stream);
}
