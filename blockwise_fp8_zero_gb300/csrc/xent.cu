// xent.cu -- softmax cross entropy of a vocabulary projection, with its gradient,
// without keeping the logits.
//
//   l[t][v] = sum_h x[t][h] w[v][h]
//   lse[t]  = log sum_v exp l[t][v],   loss[t] = lse[t] - l[t][y_t]
//   P[t][v] = (exp(l[t][v] - lse[t]) - [v == y_t]) * keep[t]
//   dx = a * P w,   dw = a * P^T x,   a = grad_scale / (number of kept tokens, or 1)
//
// The loss needs one product whose epilogue turns each 256 columns of logits
// into a maximum and a sum of exponentials per token.  Every exponential is taken
// of a difference to a maximum m that is formed first, and m and the sum s go on
// apart: the loss is log s + (m - l_y) and a probability exp(l - m) / s, so that
// neither loses what m holds beyond their own size (a loss of 1e-15 at logits of
// 4000 comes out as 0; from an FP32 lse it was 3e-4 off).  The gradient goes through
// the vocabulary in pieces: P of a piece, in 16 bits, is what the two other
// products read.  The buffer that holds one piece of P holds the logits of one
// piece just as well, so the first pass leaves the last piece's logits there
// and they become P in place; the pieces before it are multiplied again.  What
// is kept is one piece, never all the logits of a long batch.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "fp8z.h"
#include "fp8z_device.cuh"
#include "fp8z_elem.cuh"
#include "fp8z_host.h"
#include "fp8z_launch.cuh"
#include "fp8z_tcgen05.cuh"
#include "fp8z_tiles.h"

namespace fp8z {
namespace {

constexpr int kTM = 256, kTN = 256, kBK = 64;          // output tile of a pair of blocks, K per stage
constexpr int kHalf = 128;                             // a block's rows of A and of the result, and columns of B
constexpr int kTileBytes = kHalf * kBK * 2;            // of one operand's tile
constexpr int kRing = 6 * 2 * kTileBytes;              // six stages of A and B, or four of both parts of A and B
constexpr int kReaders = 8;                            // warps that read the sums: 32 rows and 128 columns each
constexpr int kThreads = 128 + 32 * kReaders;          // warps 0 and 3 load A and B, 1 multiplies, the readers follow
// The tensor cores cut a sum off where FP32 ends, toward zero, at every step of 16
// of K: logits of hidden 7168 (448 steps) came out so far off that the loss was 4e-6
// off (FP32 products: 8e-7), an FP32 dw of 4096 tokens (512 steps, two parts) 1e-5.
// So the sums of the logits and of an FP32 dw leave tensor memory after some blocks of
// K and are added up, rounded, in the readers' registers: loss 7e-7 off, dw 2.1e-6,
// of which the two parts of P make up 1.7e-6.  That takes 3 % of the loss's time (4 with
// 16 blocks of K for the logits, 2.5 with 32 and 9e-7) and 1 to 2 of the gradient's.
// A dx and a dw of 16 bits need less, but not nothing: 8192 steps (131072 words, or as many
// tokens) may cut off 1e-3 of what was added up, twice FP16's rounding, and what all rows of
// w have in common cancels in dx while its cut-off does not.  64 blocks, 256 steps, are 3e-5.
// 16384 steps of one sign took 1.1e-3 off a 16-bit dw.  It takes 0.7 % of a gradient's time at the most.
constexpr int kLogitBlocks = 24, kWeightBlocks = 8, kResultBlocks = 64;
constexpr int kTmemCols = 512;                         // two accumulators of 256 columns
constexpr int kSlab = 32 * 128;                        // staged results of a reader: 32 rows of 128 bytes
constexpr int kStaging = kReaders * kSlab;
constexpr int kNumBars = 2 * 6 + 5;
constexpr int kSmem = kRing + kStaging + kNumBars * 8 + 32 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory of one SM");
constexpr float kLog2e = 1.4426950408889634f;

enum Epilogue { kStats, kProb, kSum, kWeight, kWeightSplit };      // kWeightSplit: P in two parts

struct MmaArgs {
    int m, n;                 // rows and columns of the result
    int mt, nt, splits;       // tiles, and parts of the K loop
    int kb;                   // K blocks of 64
    int b_n0, b_k0;           // where B starts, in elements
    int b_blocks;             // B's map has its columns as blocks of 64
    int bf16;
    int64_t timeout_ns;
    int32_t* dev_status;
    // kStats, kProb: rows are tokens, columns words v0 + n of this launch
    int v0;
    const void* targets;      // as the caller gave them
    int targets_wide;
    int64_t ignore, vocab;
    const int32_t* target;    // -1: takes no part in the loss (written by rows_kernel)
    float2* part;             // [tile, or block of few_kernel][rows] maximum and sum
    float* target_logit;
    const float2* row_stats;  // maximum of a row, 1 / the sum of its exponentials
    int keep_from;            // words from here on leave their logits in the piece's buffer
    uint8_t* p;               // that buffer, p_bytes a row (few_kernel)
    int64_t p_bytes;
    uint32_t* ticket;         // of rows_kernel, set to zero here
    int split_p;              // P in two parts
    float p_scale;
    int rows;                 // tokens, rounded up to 32: stride of part
    // kSum: FP32 [splits][m];  kWeight: rows v0 + m of dw
    void* out;
    int64_t out_ld;
    int out_dtype, accumulate, staged;
    const float* alpha;
    int beside;               // kWeight: runs beside the kernel before it
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

// (a - m) * log2(e) of two logits by packed instructions: two for both, as many as fused
// multiplications and additions with a rounded m * log2(e).  4096 x 131072 x 576 takes 457 us
// this way and 475 with single ones.
__device__ __forceinline__ float2 exponents(uint32_t a, uint32_t b, float m) {
    float2 e;
    asm("{\n\t.reg .b64 L, M, K;\n\t"
        "mov.b64 L, {%2, %3};\n\t"
        "mov.b64 M, {%4, %4};\n\t"
        "mov.b64 K, {%5, %5};\n\t"
        "sub.rn.f32x2 L, L, M;\n\t"
        "mul.rn.f32x2 L, L, K;\n\t"
        "mov.b64 {%0, %1}, L;\n\t}"
        : "=f"(e.x), "=f"(e.y)
        : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)), "f"(m), "f"(kLog2e));
    return e;
}

__device__ __forceinline__ int load_target(const void* targets, int wide, int64_t ignore, int64_t vocab, int row) {
    const int64_t y = wide ? static_cast<const int64_t*>(targets)[row] : int64_t(static_cast<const int32_t*>(targets)[row]);
    return y == ignore || y < 0 || y >= vocab ? -1 : int(y);
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

// A reader's results: 128 columns, from c0 of the tile on, of the row of each lane.
constexpr int kOwn = 128;
using Sums = uint32_t[kOwn];

// Maximum and sum of exponentials of one row over the tile's columns.
__device__ __forceinline__ void epilogue_stats(const MmaArgs& A, const CUtensorMap& out, const TileAt& t, Sums& sums,
                                               int c0, int row, Stager& sg) {
    const int col0 = t.n * kTN, n_valid = min(kTN, A.n - col0);
    const int target = row < A.m ? load_target(A.targets, A.targets_wide, A.ignore, A.vocab, row) - col0 : -1;
    const bool keep = col0 >= A.keep_from;
    float mx = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kOwn; i += 32) {
        const int c = c0 + i;
        uint32_t* r = sums + i;
        if (c >= n_valid) break;
        if (keep) {
            stage32(sg, r);
            sg.end([&](uint32_t s) {
                if (row < A.m) tma_store_2d(&out, col0 - A.keep_from + c, row, s);
            });
        }
        if (c + 32 > n_valid) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c + j >= n_valid) r[j] = __float_as_uint(-INFINITY);
        }
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j) top = fmaxf(top, __uint_as_float(r[j]));
        const float m2 = fmaxf(mx, top), ref = m2 == -INFINITY ? 0.0f : m2;
        float s = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            const float2 e = exponents(r[j], r[j + 1], ref);
            s += ex2(e.x);
            s2 += ex2(e.y);
        }
        sum = fmaf(sum, ex2((mx - ref) * kLog2e), s + s2);
        mx = m2;
        if (target >= c && target < c + 32) {
            float x = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (target == c + j) x = __uint_as_float(r[j]);
            A.target_logit[row] = x;
        }
    }
    if (row < A.m) A.part[size_t(t.n * 2 + c0 / kOwn) * A.rows + row] = make_float2(mx, sum);
}

// P of eight neighbouring words of one row, times p_scale: in 16 bits, and what
// that rounding left in another 16.  stats: the row's maximum and 1 / its sum;
// target: the row's word relative to the first of the eight; valid: words before the
// vocabulary's end.
__device__ __forceinline__ void prob8(const uint32_t* r, float2 stats, int target, int valid, bool kept, float p_scale,
                                      int bf16, uint32_t (&h)[4], uint32_t (&l)[4]) {
    const float f = stats.y * p_scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 e = exponents(r[i * 2], r[i * 2 + 1], stats.x);
        float p[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j = i * 2 + k;
            const float v = ex2(k ? e.y : e.x);
            p[k] = kept && j < valid ? fmaf(v, f, target == j ? -p_scale : 0.0f) : 0.0f;
        }
        h[i] = pack16(p[0], p[1], bf16);
        const float2 w = unpack16(h[i], bf16);
        l[i] = pack16(p[0] - w.x, p[1] - w.y, bf16);
    }
}

// Words past the end become zeros: the products read whole tiles.  The buffer
// holds, for each row and tile of 256 words, 512 bytes of P and 512 bytes of its
// second part: the room of the tile's FP32 logits.
__device__ __forceinline__ void epilogue_prob(const MmaArgs& A, const CUtensorMap& out, const TileAt& t, Sums& sums,
                                              int c0, int row, Stager& sg) {
    const int n_valid = A.n - t.n * kTN;
    const int y = row < A.m ? A.target[row] : -1;
    const int target = y - (A.v0 + t.n * kTN);
    const float2 stats = y >= 0 ? A.row_stats[row] : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kOwn; i += 64) {
        uint32_t h[32], l[32];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int at = c0 + i + q * 8;
            uint32_t hq[4], lq[4];
            prob8(sums + i + q * 8, stats, target - at, n_valid - at, y >= 0, A.p_scale, A.bf16, hq, lq);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h[q * 4 + k] = hq[k];
                l[q * 4 + k] = lq[k];
            }
        }
        stage32(sg, h);
        sg.end([&](uint32_t s) { if (row < A.m) tma_store_3d(&out, c0 + i, 2 * t.n, row, s); });
        if (A.split_p) {
            stage32(sg, l);
            sg.end([&](uint32_t s) { if (row < A.m) tma_store_3d(&out, c0 + i, 2 * t.n + 1, row, s); });
        }
    }
}

__device__ __forceinline__ void epilogue_sum(const MmaArgs& A, const CUtensorMap& out, const TileAt& t, Sums& sums,
                                             int c0, int row, Stager& sg) {
    const int col0 = t.n * kTN + c0;
#pragma unroll
    for (int i = 0; i < kOwn; i += 32) {
        if (col0 + i >= A.n) break;
        stage32(sg, sums + i);
        sg.end([&](uint32_t s) {
            if (row >= A.m) return;
            if (A.accumulate) tma_add_3d(&out, col0 + i, row, t.split, s);
            else tma_store_3d(&out, col0 + i, row, t.split, s);
        });
    }
}

// A dw whose rows do not all start and end on 16-byte boundaries, and sums of 16-bit
// gradients (one rounding of the whole sum): 32 columns of the warp's 32 rows
// pass through its slab, so that the threads write along the rows.
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

__device__ __forceinline__ void epilogue_weight(const MmaArgs& A, const CUtensorMap& out, const TileAt& t, Sums& sums,
                                                int c0, int row, Stager& sg) {
    const float a = __ldcg(A.alpha);                 // not from an L1 that may be older than what wrote it
    const int y = A.v0 + row;                        // of lane 0, which issues the stores
    const int col0 = t.n * kTN + c0;
    if (A.staged && A.out_dtype != FP8Z_F32) {
#pragma unroll
        for (int i = 0; i < kOwn; i += 64) {
            if (col0 + i >= A.n) break;
            uint32_t h[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
                h[j] = pack16(__uint_as_float(sums[i + 2 * j]) * a, __uint_as_float(sums[i + 2 * j + 1]) * a, A.bf16);
            stage32(sg, h);
            sg.end([&](uint32_t s) { if (row < A.m) tma_store_2d(&out, col0 + i, y, s); });
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kOwn; i += 32) {
        const int col = col0 + i;
        uint32_t* r = sums + i;
        if (col >= A.n) break;
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * a);
        if (A.staged) {
            stage32(sg, r);
            sg.end([&](uint32_t s) {
                if (row >= A.m) return;
                if (A.accumulate) tma_add_2d(&out, col, y, s);
                else tma_store_2d(&out, col, y, s);
            });
        } else {
            __syncwarp();                            // the slab's last rows have been read
#pragma unroll
            for (int j = 0; j < 8; ++j) sg.put(sg.slab, j, r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
            __syncwarp();
            const int first = row - sg.lane, rows = min(32, A.m - first), n = A.n - col;
            const int64_t at = int64_t(A.v0 + first) * A.out_ld + col;
            if (A.out_dtype == FP8Z_F32) weight_rows(static_cast<float*>(A.out) + at, A.out_ld, rows, n, sg, A.accumulate);
            else if (A.out_dtype == FP8Z_BF16) weight_rows(static_cast<__nv_bfloat16*>(A.out) + at, A.out_ld, rows, n, sg, A.accumulate);
            else weight_rows(static_cast<__half*>(A.out) + at, A.out_ld, rows, n, sg, A.accumulate);
        }
    }
}

// A pair of blocks takes 256 x 256 results at a time.  Each block loads 128 rows
// of A and 128 columns of B into a ring of kStages tiles; one thread of the
// first block issues the products of both, into one of two accumulators in each
// block's tensor memory, while eight warps of each block read the other.  The
// copies of both blocks count on the first block's barriers, each block arriving
// for its own.
template <int kEpi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mma_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
               const __grid_constant__ CUtensorMap tc, const __grid_constant__ MmaArgs A) {
    constexpr bool kWeights = kEpi == kWeight || kEpi == kWeightSplit;
    constexpr bool kAMn = kWeights, kBMn = kEpi == kSum || kWeights;                 // operands along M or N
    constexpr int kSumBlocks = kEpi == kWeightSplit ? kWeightBlocks : kEpi == kSum || kEpi == kWeight ? kResultBlocks : kLogitBlocks;
    constexpr bool kAddAll = kEpi != kStats;                  // the first sum to zeros: fewer registers
    constexpr int kStep = kEpi == kSum || kEpi == kWeight ? 8 : 16;                  // columns added at a time: fewer registers, too
    constexpr int kParts = kEpi == kWeightSplit ? 2 : 1;      // of A: one B serves both, a third less to load
    constexpr int kBytesA = kParts * kTileBytes, kStageBytes = kBytesA + kTileBytes, kStages = kRing / kStageBytes;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_addr(smem_raw));
    constexpr int kBarsAt = kRing + kStaging;
    const uint32_t bars = base + kBarsAt;
    auto full = [&](int s) { return bars + s * 8; };                       // first block: both blocks' copies are there
    auto empty = [&](int s) { return bars + (kStages + s) * 8; };          // the products that read them are done
    auto tfull = [&](int b) { return bars + (2 * kStages + b) * 8; };
    auto tempty = [&](int b) { return bars + (2 * kStages + 2 + b) * 8; };  // first block: both blocks' warps have read it
    const uint32_t drain = bars + (2 * kStages + 4) * 8;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kBarsAt + kNumBars * 8);
    volatile uint32_t* tmem_at = reinterpret_cast<volatile uint32_t*>(smem + kBarsAt + kNumBars * 8 + 8);
    volatile uint32_t* issued_by = reinterpret_cast<volatile uint32_t*>(smem + kBarsAt + kNumBars * 8 + 16);   // [4]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = int(cluster_rank()), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 4);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), 2 * kReaders);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 32) {
        tensormap_prefetch(&ta);
        tensormap_prefetch(&tb);
    }
    if (warp == 2) tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_at)), kTmemCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    // dw needs nothing of dx's sum, which is launched just before it: a block may start as
    // soon as an SM is free.  dx's kernel lets it be launched after its own wait, so what
    // came before dx is done; dx itself is waited for at the end, for whoever comes next.
    const bool beside = kWeights && A.beside;
    if (!beside) dependent_wait();
    if (kEpi == kStats && blockIdx.x == 0 && threadIdx.x == 0) *A.ticket = 0;
    const uint32_t tmem = *tmem_at;
    const Watchdog wd{abort_flag, A.dev_status, A.timeout_ns};
    const int tiles = A.mt * A.nt * A.splits;

    if (warp == 0 || warp == 3) {          // one thread for A and one for B: an issue takes some 100 cycles of a stage's 512
        if (lane == 0) {
            int s = 0, ph = 0;
            uint32_t issued = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const TileAt at = tile_at(A, t);
                const int m = at.m * kTM + rank * kHalf, n = A.b_n0 + at.n * kTN + rank * kHalf;
                for (int k = at.k0; k < at.k1; ++k) {
                    if (!mbar_wait_bounded(empty(s), ph ^ 1, wd)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = base + s * kStageBytes, sb = sa + kBytesA, bar = cluster_addr(full(s), 0);
                    const int kb = k * kBK + A.b_k0;
                    if (warp == 0) {
                        mbar_arrive_expect_tx_cluster(bar, kBytesA);
                        if constexpr (kWeights)                  // P^T: 128 words, 64 tokens
#pragma unroll
                            for (int part = 0; part < kParts; ++part)
                                tma_load_4d_pair(sa + part * kTileBytes, &ta, 0, k * kBK, m % kTN / 64,
                                                 m / kTN * 2 + part, bar);
                        else if constexpr (kEpi == kSum)         // P: 128 tokens, 64 words of the first part
                            tma_load_3d_pair(sa, &ta, k * kBK % kTN, k * kBK / kTN * 2, m, bar);
                        else
                            tma_load_2d_pair(sa, &ta, k * kBK, m, bar);
                    } else {
                        mbar_arrive_expect_tx_cluster(bar, kTileBytes);
                        if constexpr (!kBMn) {
                            tma_load_2d_pair(sb, &tb, kb, n, bar);
                        } else if (A.b_blocks) {                 // 128 columns as two blocks of 64
                            tma_load_3d_pair(sb, &tb, 0, kb, n / 64, bar);
                        } else {
#pragma unroll
                            for (int j = 0; j < kHalf / 64; ++j)
                                tma_load_2d_pair(sb + j * (64 * kBK * 2), &tb, n + j * 64, kb, bar);
                        }
                    }
                    ++issued;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            st_cluster_u32(cluster_addr(smem_addr(const_cast<uint32_t*>(issued_by + 2 * rank + (warp == 3))), 0), issued);
        }
    } else if (warp == 1 && rank == 0) {
        if (lane == 0) {
            const uint32_t idesc = umma_idesc(A.bf16 != 0, kAMn, kBMn, kTM, kTN);
            int s = 0, ph = 0, b = 0, bph = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const TileAt at = tile_at(A, t);
                const int sums = sums_of(at.k0, at.k1, kSumBlocks);
                for (int i = 0; i < sums && ok; ++i) {
                    const int first = sum_start(at.k0, at.k1, i, sums), end = sum_start(at.k0, at.k1, i + 1, sums);
                    if (!mbar_wait_bounded(tempty(b), bph ^ 1, wd)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    for (int k = first; k < end; ++k) {
                        if (!mbar_wait_bounded(full(s), ph, wd)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = base + s * kStageBytes, sb = sa + kBytesA;
                        const uint64_t da = umma_desc(sa, kAMn ? 64 * kBK * 2 : 16, 1024);
                        const uint64_t db = umma_desc(sb, kBMn ? 64 * kBK * 2 : 16, 1024);
#pragma unroll
                        for (int j = 0; j < kBK / 16; ++j)  // 16 of K: 32 bytes of a row, or 16 rows of 128 bytes
#pragma unroll
                            for (int part = 0; part < kParts; ++part)
                                umma_f16(tmem + b * kTN, da + part * (kTileBytes / 16) + j * (kAMn ? 128 : 2),
                                         db + j * (kBMn ? 128 : 2), idesc, k != first || j != 0 || part != 0);
                        umma_commit_pair(empty(s));
                        if (++s == kStages) {
                            s = 0;
                            ph ^= 1;
                        }
                    }
                    if (!ok) break;
                    umma_commit_pair(tfull(b));
                    if (b) bph ^= 1;
                    b ^= 1;
                }
            }
            umma_commit_pair(drain);       // and every product is done before tensor memory is freed
            mbar_wait_drain(drain, 0, A.dev_status);
        }
    } else if (warp >= 4) {
        const int quarter = warp & 3, c0 = (warp - 4) / 4 * kOwn;    // a warp reaches its quarter of the lanes: 32 rows
        Stager sg{base + kRing + (warp - 4) * kSlab, lane};
        int b = 0, bph = 0;
        bool ok = true;
        for (int t = pair; t < tiles; t += pairs) {
            const TileAt at = tile_at(A, t);
            const int n_sums = sums_of(at.k0, at.k1, kSumBlocks);
            Sums sums;
            if constexpr (kAddAll)
#pragma unroll
                for (int j = 0; j < kOwn; ++j) sums[j] = 0;
            for (int i = 0; i < n_sums; ++i) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(tfull(b), bph, wd));
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + b * kTN + c0 + (uint32_t(quarter * 32) << 16);
                if (!kAddAll && i == 0) {
#pragma unroll
                    for (int c = 0; c < kOwn; c += 32) tmem_ld32(reinterpret_cast<uint32_t(&)[32]>(sums[c]), acc + c);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int c = 0; c < kOwn; c += kStep) {
                        uint32_t r[kStep];
                        if constexpr (kStep == 16) tmem_ld16(r, acc + c);
                        else tmem_ld8(r, acc + c);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < kStep; ++j)
                            sums[c + j] = __float_as_uint(__uint_as_float(sums[c + j]) + __uint_as_float(r[j]));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(tempty(b), 0);
                if (b) bph ^= 1;
                b ^= 1;
            }
            if (!ok) break;
            if (at.k0 == at.k1)                      // nothing was multiplied
#pragma unroll
                for (int j = 0; j < kOwn; ++j) sums[j] = 0;
            const int row = at.m * kTM + rank * kHalf + quarter * 32 + lane;
            if constexpr (kEpi == kStats) epilogue_stats(A, tc, at, sums, c0, row, sg);
            else if constexpr (kEpi == kProb) epilogue_prob(A, tc, at, sums, c0, row, sg);
            else if constexpr (kEpi == kSum) epilogue_sum(A, tc, at, sums, c0, row, sg);
            else epilogue_weight(A, tc, at, sums, c0, row, sg);
        }
        if (lane == 0) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    // Whatever a wait gave up on, every copy lands before either block ends.  A stage for which
    // some of the four threads never came to issue their copies lacks their arrivals: they are made here.
    if (rank == 0 && threadIdx.x == 0) {
        uint32_t most = 0;
        for (int j = 0; j < 4; ++j) most = max(most, issued_by[j]);
        for (int j = 0; j < 4; ++j)
            for (uint32_t i = issued_by[j]; i < most; ++i) mbar_arrive(full(i % kStages));
        for (uint32_t i = most > kStages ? most - kStages : 0; i < most; ++i)
            mbar_wait_drain(full(i % kStages), (i / kStages) & 1, A.dev_status);
    }
    if (rank == 1 && threadIdx.x == 0) mbar_wait_drain(drain, 0, A.dev_status);    // the last arrival from the first block
    cluster_sync();                        // neither block ends, nor frees, while the other may still reach it
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (beside) dependent_wait();
}

// ------------------------------------------------------------ small kernels
// Elements k .. k + 7 of a row of `cols` 16-bit elements that starts on any
// 2-byte boundary, zeros from `cols` on: five aligned words, shifted together.
__device__ __forceinline__ uint4 ld_row8(const uint16_t* row, int k, int cols) {
    uint32_t v[4] = {};
    if (k + 8 <= cols) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + k);
        const bool odd = (at & 2) != 0;
        const uint32_t* p = reinterpret_cast<const uint32_t*>(at & ~uintptr_t(3));
        uint32_t w[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = i < 4 || odd ? *reinterpret_cast<const volatile uint32_t*>(p + i) : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = odd ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < cols) v[i / 2] |= uint32_t(*reinterpret_cast<const volatile uint16_t*>(row + k + i)) << (i & 1) * 16;
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// The same where k may be negative, an element at a time.
__device__ __noinline__ uint4 part_row8(const uint16_t* row, int k, int cols) {
    uint4 v = make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        const uint32_t e = k + i >= 0 && k + i < cols ? *reinterpret_cast<const volatile uint16_t*>(row + k + i) : 0;
        v.x = __funnelshift_r(v.x, v.y, 16), v.y = __funnelshift_r(v.y, v.z, 16);
        v.z = __funnelshift_r(v.z, v.w, 16), v.w = __funnelshift_r(v.w, e, 16);
    }
    return v;
}

// 16-bit rows of x, then of w, copied to a stride the tensor maps can step over,
// zeros after the end: a warp a row, 16 bytes a thread.  Either may have no rows.
struct PadRows {
    const uint16_t* src;
    uint16_t* dst;
    int64_t ld;
    int rows;
};
__global__ void __launch_bounds__(256) pad_rows_kernel(const PadRows x, const PadRows w, int cols, int cols_pad) {
    dependent_wait();
    int r = int(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const bool of_x = r < x.rows;
    const PadRows& m = of_x ? x : w;
    if (!of_x) r -= x.rows;
    if (r >= m.rows) return;
    const uint16_t* from = m.src + r * m.ld;
    uint16_t* to = m.dst + int64_t(r) * cols_pad;
#pragma unroll 4
    for (int c = (threadIdx.x & 31) * 8; c < cols_pad; c += 256) *reinterpret_cast<uint4*>(to + c) = ld_row8(from, c, cols);
}

// x once for each way in which rows of w start between 16-byte boundaries: copy r
// begins with as many zeros as word r's row lies behind one, and is filled up with
// zeros to `cols_pad`.
__global__ void __launch_bounds__(256) shift_rows_kernel(const uint16_t* src, int64_t ld, int rows, int cols,
                                                         int cols_pad, const uint16_t* w, int64_t w_ld, uint16_t* dst) {
    dependent_wait();
    const int copy = blockIdx.y, row = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int behind = int(reinterpret_cast<uintptr_t>(w + copy * w_ld) >> 1 & 7);
    const uint16_t* p = src + row * ld;
    uint16_t* to = dst + (int64_t(copy) * rows + row) * cols_pad;
    for (int c = (threadIdx.x & 31) * 8; c < cols_pad; c += 256) {
        const int k = c - behind;
        *reinterpret_cast<uint4*>(to + c) = k >= 0 ? ld_row8(p, k, cols) : part_row8(p, k, cols);
    }
}

// ------------------------------------------------------------- few tokens
// The logits of up to 32 tokens are one pass over w at the memory's rate, and
// a tile of 256 rows would be multiplied mostly for nothing.  Here a warp takes
// 16 words and all of K: four lanes read 16 bytes each of a row and of the next
// row but seven, 32 elements of K a step, as the A fragments of two m16n8k16
// products (which lane holds which k does not matter as long as x is held the
// same way), and the tokens are the products' columns, eight a tile.  x waits in
// shared memory in the order of the lanes, up to 1024 elements of K at a time and
// the next ones on their way; each step's w is loaded four steps ahead.
// 8 tokens: 25 us over 32000 x 2048 and 276 us over 131072 x 7168 (6.8 TB/s), the
// row statistics included; 32 tokens 33 and 314; through tiles, 33 tokens take 37
// and 295, and eight took 40 and 340 (every pair of blocks then reads the same
// few lines of x at the same time).
constexpr int kFewTokens = 32, kFewWords = 128;        // most tokens; words of a block of eight warps

// 16 bytes into shared memory in the background; zeros where `in` is false.
__device__ __forceinline__ void copy_16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

__device__ __forceinline__ void mma_16n8k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1, bool bf16) {
    if (bf16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Blocks an SM that the registers allow.  8 tokens over 131072 x 7168: 277 us with four
// and 300 with three; 32 over 32000 x 2048: 32 with two, 35 with three.  Odd rows:
// 8 over 32000 x 2047 35 us with three and 40 with four, 32 over 43109 x 6354 151 and
// 165 with two.
template <int kTiles, bool kAligned>
constexpr int few_blocks_sm = !kAligned || kTiles == 2 ? 3 : kTiles == 1 ? 4 : 2;

// kAligned: the rows of w start on 16-byte boundaries (x's always do here).  Else
// every `period`th row is as far behind one as the first: a block takes words of one
// kind, reads their rows in whole 16 bytes from the boundary before them, the ends an
// element at a time, and multiplies them with the copy of x that is as far behind.
// 9 tokens over 43109 x 6354 take 110 us, 8 over 32000 x 2047 35; with five words of
// 4 bytes for each 16, shifted together, 330 and 101.
template <int kTiles, bool kBf16, bool kAligned>
__global__ void __launch_bounds__(256, few_blocks_sm<kTiles, kAligned>) few_kernel(const uint16_t* x, int64_t x_ld, const uint16_t* w, int64_t w_ld,
                                                  int hidden, int period, const __grid_constant__ MmaArgs A) {
    constexpr int kSteps = 32 / kTiles;                // of 32 elements, whose x is in shared memory
    __shared__ uint4 xs[2][kSteps][kTiles][32];        // [][step][tile][lane]: token lane / 4, elements 8 (lane % 4) on
    __shared__ float2 warp_part[8][kTiles * 8];
    dependent_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *A.ticket = 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int kind = kAligned ? 0 : int(blockIdx.x) % period, by = kAligned ? 1 : period;
    const int word = (int(blockIdx.x) / by * kFewWords + warp * 16 + g) * by + kind, word2 = word + 8 * by;
    const uint16_t* wa = w + int64_t(min(word, A.n - 1)) * w_ld;
    const uint16_t* wb = w + int64_t(min(word2, A.n - 1)) * w_ld;
    const int behind = kAligned ? 0 : int(reinterpret_cast<uintptr_t>(w + kind * w_ld) >> 1 & 7);
    const int ends = kAligned ? 0 : hidden + behind;                  // of the row, from its boundary
    const int width = kAligned ? hidden : int(x_ld);
    if constexpr (!kAligned) x += int64_t(kind) * A.m * x_ld;
    constexpr int U = 4;
    uint4 a[U], b[U];
    auto load = [&](int u, int k) {
        if constexpr (kAligned) {
            const bool in = k < hidden;                // a multiple of 8 here
            a[u] = in ? ld_stream_16(wa + k, 0) : make_uint4(0, 0, 0, 0);
            b[u] = in ? ld_stream_16(wb + k, 0) : make_uint4(0, 0, 0, 0);
        } else if (k >= behind && k + 8 <= ends) {
            a[u] = word < A.n ? ld_stream_16(wa + (k - behind), 0) : make_uint4(0, 0, 0, 0);
            b[u] = word2 < A.n ? ld_stream_16(wb + (k - behind), 0) : make_uint4(0, 0, 0, 0);
        } else {
            const bool in = k < ends;
            a[u] = in && word < A.n ? part_row8(wa, k - behind, hidden) : make_uint4(0, 0, 0, 0);
            b[u] = in && word2 < A.n ? part_row8(wb, k - behind, hidden) : make_uint4(0, 0, 0, 0);
        }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, q * 8 + 32 * u);
    auto fetch_x = [&](int c) {
        for (int i = threadIdx.x; i < kSteps * kTiles * 32; i += 256) {
            const int step = i / (kTiles * 32), token = i / 32 % kTiles * 8 + (i >> 2 & 7);
            const int k = (c * kSteps + step) * 32 + (i & 3) * 8;
            const bool in = token < A.m && k < width;
            copy_16(smem_addr(&xs[c & 1][0][0][0] + i), in ? x + token * x_ld + k : x, in);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int steps = (width + 31) / 32, chunks = (steps + kSteps - 1) / kSteps;
    float acc[kTiles][4] = {}, sum[kTiles][4] = {};    // of the x in shared memory, and of all before
    fetch_x(0);
    for (int c = 0; c < chunks; ++c) {
        if (c + 1 < chunks) {
            fetch_x(c + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const int here = min(kSteps, steps - c * kSteps);
        for (int step = 0; step < here; step += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (step + u < here) {
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) {
                        const uint4 v = xs[c & 1][step + u][t][lane];
                        mma_16n8k16(acc[t], a[u].x, b[u].x, a[u].y, b[u].y, v.x, v.y, kBf16);
                        mma_16n8k16(acc[t], a[u].z, b[u].z, a[u].w, b[u].w, v.z, v.w, kBf16);
                    }
                }
                load(u, (c * kSteps + step + u + U) * 32 + q * 8);
            }
        }
#pragma unroll
        for (int i = 0; i < 4 * kTiles; ++i) {         // as above: the products' sums are cut off, these are rounded
            sum[i / 4][i & 3] += acc[i / 4][i & 3];
            acc[i / 4][i & 3] = 0.0f;
        }
        __syncthreads();
    }
    // sum[t][i]: word, or word2 from i = 2 on;, token 8 t + 2 q + (i & 1)
#pragma unroll
    for (int i = 0; i < 2 * kTiles; ++i) {
        const int t = i / 2, c = i & 1, token = t * 8 + 2 * q + c;
        float v0 = sum[t][c], v1 = sum[t][2 + c];
        if (token < A.m) {
            const int y = load_target(A.targets, A.targets_wide, A.ignore, A.vocab, token);
            if (y == word) A.target_logit[token] = v0;
            if (y == word2) A.target_logit[token] = v1;
            float* keep = reinterpret_cast<float*>(A.p + token * A.p_bytes);
            if (word >= A.keep_from && word < A.n) keep[word - A.keep_from] = v0;
            if (word2 >= A.keep_from && word2 < A.n) keep[word2 - A.keep_from] = v1;
        }
        if (word >= A.n) v0 = -INFINITY;
        if (word2 >= A.n) v1 = -INFINITY;
        float m = fmaxf(v0, v1);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float ref = m == -INFINITY ? 0.0f : m;
        float s = ex2((v0 - ref) * kLog2e) + ex2((v1 - ref) * kLog2e);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (g == 0) warp_part[warp][token] = make_float2(m, s);
    }
    __syncthreads();
    if (int(threadIdx.x) < kTiles * 8 && int(threadIdx.x) < A.m) {
        float m = -INFINITY, s = 0.0f;
        for (int i = 0; i < 8; ++i) m = fmaxf(m, warp_part[i][threadIdx.x].x);
        const float ref = m == -INFINITY ? 0.0f : m;
        for (int i = 0; i < 8; ++i) {
            const float2 p = warp_part[i][threadIdx.x];
            s += p.y * ex2((p.x - ref) * kLog2e);
        }
        A.part[size_t(blockIdx.x) * A.rows + threadIdx.x] = make_float2(m, s);
    }
}

// lse and loss of 32 rows from the tiles' maxima and sums, 32 threads a row; the
// block that finishes last adds up the blocks' sums, in order.
struct BlockTotal {
    double loss;
    int64_t kept;
};

__global__ void __launch_bounds__(1024) rows_kernel(const float2* part, int tiles, int n, int rows,
                                                    const void* targets, int wide, int64_t ignore,
                                                    int64_t vocab, const float* target_logit,
                                                    int32_t* target, float2* row_stats,
                                                    float* lse_out, float* loss,
                                                    BlockTotal* totals, uint32_t* ticket,
                                                    int mean, float scale, float* total,
                                                    float* alpha, int32_t* dev_status) {
    __shared__ float2 sh[32][33];
    __shared__ bool last;
    dependent_wait();
    const int r = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int row = blockIdx.x * 32 + g;               // in the end a warp has a row, and lane 0 finishes it
    int y = -1;
    float own = 0.0f;
    if (r == 0 && row < n) {
        y = load_target(targets, wide, ignore, vocab, row);
        if (y < 0) {
            const int64_t raw = wide ? static_cast<const int64_t*>(targets)[row]
                                     : int64_t(static_cast<const int32_t*>(targets)[row]);
            if (raw != ignore) report_status(dev_status, FP8Z_EINVAL);
        } else {
            own = target_logit[row];
        }
    }
    float m = -INFINITY, s = 0.0f;
    auto add = [&](float2 p) {
        const float m2 = fmaxf(m, p.x), ref = m2 == -INFINITY ? 0.0f : m2;
        s = s * ex2((m - ref) * kLog2e) + p.y * ex2((p.x - ref) * kLog2e);
        m = m2;
    };
    const int col = blockIdx.x * 32 + r;               // the row of this thread's partial results
    if (col < n) {
        for (int t = g; t < tiles; t += 256) {
            float2 q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q[i] = t + 32 * i < tiles ? part[size_t(t + 32 * i) * rows + col] : make_float2(-INFINITY, 0.0f);
            float top = q[0].x;
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, q[i].x);
            const float ref = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += q[i].y * ex2((q[i].x - ref) * kLog2e);
            add(make_float2(top, sum));
        }
    }
    sh[r][g] = make_float2(m, s);
    __syncthreads();
    const float2 mine = sh[g][r];
    m = mine.x;
    s = mine.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        add(make_float2(__shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o)));
    __syncthreads();
    if (r == 0) {
        float out = 0.0f;
        if (row < n) {
            const float log_s = logf(s);
            out = y >= 0 ? log_s + (m - own) : 0.0f;
            target[row] = y;
            row_stats[row] = make_float2(m, 1.0f / s);
            if (lse_out) lse_out[row] = m + log_s;
            loss[row] = out;
        }
        sh[0][g] = make_float2(out, y >= 0 ? 1.0f : 0.0f);
    }
    __syncthreads();
    if (g != 0) return;
    BlockTotal b = {double(sh[0][r].x), int64_t(sh[0][r].y)};
    auto reduce = [&] {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            b.loss += __shfl_down_sync(0xFFFFFFFFu, b.loss, o);
            b.kept += __shfl_down_sync(0xFFFFFFFFu, b.kept, o);
        }
    };
    reduce();
    if (gridDim.x > 1) {
        if (r == 0) {
            totals[blockIdx.x] = b;
            __threadfence();
            last = atomicAdd(ticket, 1u) == gridDim.x - 1;
        }
        __syncwarp();
        if (!last) return;
        __threadfence();
        b = {0.0, 0};
        for (int i = r; i < int(gridDim.x); i += 32) {
            b.loss += __ldcg(&totals[i].loss);
            b.kept += __ldcg(reinterpret_cast<const long long*>(&totals[i].kept));
        }
        reduce();
    }
    if (r == 0) {
        const double by = mean ? double(b.kept > 0 ? b.kept : 1) : 1.0;
        total[0] = float(b.loss / by);
        total[1] = float(b.kept);
        if (alpha) *alpha = float(double(scale) / by);
    }
}

// The kept logits of a piece become P, in place: a warp takes a row's 256 words
// (1 KB), reads all of it, and writes the two parts over it.  The last block of a
// row copies the token's x for the product with P^T, with zeros in the place of a
// token that takes no part: its P is zero, but zero times an infinity or a NaN is
// not, and neither may reach dw.
constexpr int kProbTiles = 4;
__global__ void __launch_bounds__(256, 5) prob_kernel(uint8_t* p, int64_t row_bytes, int tiles, int words, int v0,
                                                   const int32_t* target, const float2* row_stats, float p_scale, int bf16,
                                                   int split_p, const uint16_t* x, int64_t x_ld, int hidden,
                                                   uint16_t* kept_x, int kept_ld) {
    dependent_wait();
    const int row = blockIdx.x, lane = threadIdx.x & 31;
    const int y = target[row];
    if (blockIdx.y == gridDim.y - 1) {
        const uint16_t* from = x + row * x_ld;
        uint16_t* to = kept_x + int64_t(row) * kept_ld;
        if (((reinterpret_cast<uintptr_t>(x) | uintptr_t(x_ld * 2) | uintptr_t(hidden * 2)) & 15) == 0) {
            for (int c = threadIdx.x * 8; c < kept_ld; c += 256 * 8)
                *reinterpret_cast<uint4*>(to + c) =
                    y >= 0 && c < hidden ? *reinterpret_cast<const uint4*>(from + c) : make_uint4(0, 0, 0, 0);
        } else {
            for (int c = threadIdx.x; c < kept_ld; c += 256) to[c] = y >= 0 && c < hidden ? from[c] : uint16_t(0);
        }
        return;
    }
    const float2 stats = y >= 0 ? row_stats[row] : make_float2(0.0f, 0.0f);
    // the last words first: L2 still holds their logits (1024 tokens x 32000 x 1024: 232 us for 241)
    const int t0 = (int(gridDim.y - 2 - blockIdx.y) * 8 + (threadIdx.x >> 5)) * kProbTiles;
    uint4 in[kProbTiles][2];
#pragma unroll
    for (int i = 0; i < kProbTiles; ++i) {
        if (t0 + i >= tiles) break;
        const uint4* q = reinterpret_cast<const uint4*>(p + row * row_bytes + int64_t(t0 + i) * 1024) + lane * 2;
        in[i][0] = q[0];
        in[i][1] = q[1];
    }
    __syncwarp();                                      // the whole warp has read what it now overwrites
#pragma unroll
    for (int i = 0; i < kProbTiles; ++i) {
        if (t0 + i >= tiles) break;
        const uint32_t r[8] = {in[i][0].x, in[i][0].y, in[i][0].z, in[i][0].w,
                               in[i][1].x, in[i][1].y, in[i][1].z, in[i][1].w};
        const int at = (t0 + i) * kTN + lane * 8;
        uint32_t h[4], l[4];
        prob8(r, stats, y - v0 - at, words - at, y >= 0, p_scale, bf16, h, l);
        uint4* q = reinterpret_cast<uint4*>(p + row * row_bytes + int64_t(t0 + i) * 1024);
        q[lane] = make_uint4(h[0], h[1], h[2], h[3]);
        if (split_p) q[32 + lane] = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

__global__ void empty_total_kernel(float* total) { total[threadIdx.x] = 0.0f; }

// dx = a * the sum of the K parts, zero for a token that takes no part.
template <typename T>
__global__ void __launch_bounds__(256) finish_dx_kernel(const float* sum, int splits, int64_t part_stride,
                                                        int64_t sum_ld, int hidden, const float* alpha,
                                                        const int32_t* target, T* dx, int64_t dx_ld) {
    dependent_wait();
    const float a = *alpha;
    const bool kept = target[blockIdx.x] >= 0;          // else zeros, whatever w holds
    const int c = (blockIdx.y * 256 + threadIdx.x) * 4;
    const int64_t row = blockIdx.x;
    if (c >= hidden) return;
    float v[4] = {};
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
        const float4 q = *reinterpret_cast<const float4*>(sum + s * part_stride + row * sum_ld + c);
        v[0] += q.x;
        v[1] += q.y;
        v[2] += q.z;
        v[3] += q.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (c + i < hidden) dx[row * dx_ld + c + i] = Elem<T>::narrow(kept ? v[i] * a : 0.0f);
}

template <typename T>
__global__ void zero_rows_kernel(T* out, int64_t ld, int64_t rows, int cols) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int c = threadIdx.x; c < cols; c += blockDim.x) out[r * ld + c] = Elem<T>::narrow(0.0f);
}

// ------------------------------------------------------------------ launches
struct Layout {
    int64_t rows, hidden_pad, kept_ld, vocab_tiles, piece, pieces, parts;
    int splits;
    bool copy_x, copy_w;
    size_t x, w, kept_x, target, target_logit, row_stats, part, totals, alpha, p, sum, total;
};

constexpr int64_t kPieceBytes = 1LL << 30;        // of one piece, see layout()
constexpr int kSms = 152;                         // the layout's, the same for the size query and the call

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

bool args_ok(const fp8z_xent_args& a) {
    if (a.tokens < 0 || a.tokens > (1 << 24) || a.hidden < 1 || a.hidden > (1 << 20) || a.vocab < 1 ||
        a.vocab > (1 << 28))
        return false;
    if (a.dtype != FP8Z_BF16 && a.dtype != FP8Z_F16) return false;
    if (a.targets_dtype != FP8Z_I32 && a.targets_dtype != FP8Z_I64) return false;
    if (a.x_ld < a.hidden || a.w_ld < a.hidden) return false;
    // tiles of the products are counted in 32 bits
    const int64_t tt = a.tokens / kTM + 1, vt = a.vocab / kTN + 1, ht = a.hidden / kTN + 1;
    if (tt * vt > (1 << 30) || vt * ht > (1 << 30) || tt * ht > (1 << 24)) return false;
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

// Parts of dx's sum over the vocabulary.  Too few tiles leave SMs idle, and a
// last wave that is not full leaves them idle too; every part is written and read
// again, and every wave starts and ends.  Times in ns: 270 for a tile's K block
// of 64 (the tensor cores' rate at 1.9 GHz), 2000 for a wave, 8 bytes of an
// element at 6.5 TB/s for a part.
int dx_splits(int64_t tiles, int64_t k_blocks, int64_t elems) {
    int best = 1;
    double least = 0.0;
    for (int s = 1; s <= 64 && s * 4 <= k_blocks; ++s) {
        const double waves = double((tiles * s + kSms / 2 - 1) / (kSms / 2));
        const double t = waves * double((k_blocks + s - 1) / s) * 270.0 + waves * 2000.0 +
                         double(s) * double(elems) * 8.0 / 6500.0;
        if (s == 1 || t < least) {
            least = t;
            best = s;
        }
    }
    return best;
}

// A w that no tensor map can step over: read as it is by the one pass of a few
// tokens' loss, else copied first.
bool reads_w_directly(const fp8z_xent_args& a, const void* w, bool grad) {
    return !grad && a.tokens <= kFewTokens && !map_ok(w, a.w_ld, a.hidden);
}

// Rows of w after which their distance from a 16-byte boundary repeats, and the
// elements of a row of x that is shifted by up to seven.
int period_of(int64_t w_ld) { return w_ld % 2 ? 8 : w_ld % 4 ? 4 : w_ld % 8 ? 2 : 1; }
int64_t shifted_width(int64_t hidden) { return up(hidden + 7, 8); }
int few_blocks(int64_t vocab, int period) {
    return period * int(((vocab + period - 1) / period + kFewWords - 1) / kFewWords);
}

Layout layout(const fp8z_xent_args& a, bool grad, bool copy_x, bool copy_w, bool direct, int64_t have) {
    Layout L;
    std::memset(&L, 0, sizeof(L));
    L.copy_x = copy_x;
    L.copy_w = copy_w;
    L.rows = up(a.tokens > 0 ? a.tokens : 1, 32);
    L.hidden_pad = up(a.hidden, 8);
    L.vocab_tiles = (a.vocab + kTN - 1) / kTN;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t r = at;
        at += size_t(up(bytes, 256));
        return r;
    };
    L.x = take(direct ? period_of(a.w_ld) * a.tokens * shifted_width(a.hidden) * 2 : copy_x ? a.tokens * L.hidden_pad * 2 : 0);
    L.w = take(copy_w ? a.vocab * L.hidden_pad * 2 : 0);
    L.target = take(L.rows * 4);
    L.target_logit = take(L.rows * 4);
    L.row_stats = take(L.rows * 8);
    L.alpha = take(8);
    L.part = take(std::max<int64_t>(L.vocab_tiles * (kTN / kOwn), few_blocks(a.vocab, direct ? period_of(a.w_ld) : 1)) * L.rows * 8);
    L.totals = take((L.rows / 32) * sizeof(BlockTotal));
    if (grad) {
        L.kept_ld = up(a.hidden, 64);
        L.kept_x = take(a.tokens * L.kept_ld * 2);
        L.parts = a.dw_dtype == FP8Z_F32 ? 2 : 1;
        L.splits = dx_splits((L.rows + kTM - 1) / kTM * ((L.hidden_pad + kTN - 1) / kTN), L.vocab_tiles * (kTN / kBK),
                             a.tokens * L.hidden_pad);
        L.sum = take(int64_t(L.splits) * a.tokens * L.hidden_pad * 4);
        // One piece takes 4 bytes a word and token.  By default it is at most 1 GiB, or the size of
        // the FP32 dw where that is more: what the call keeps stays below what the caller keeps.
        int64_t room = std::max(kPieceBytes, a.vocab * a.hidden * 4);
        if (have >= 0 && have - int64_t(at) < room) room = have - int64_t(at);
        const int64_t tile_bytes = std::max<int64_t>(a.tokens, 1) * kTN * 4;
        const int64_t tiles = std::min(std::max<int64_t>(room / tile_bytes, 1), L.vocab_tiles);
        L.pieces = (L.vocab_tiles + tiles - 1) / tiles;
        L.piece = (L.vocab_tiles + L.pieces - 1) / L.pieces * kTN;       // equal pieces
        L.pieces = (L.vocab_tiles * kTN + L.piece - 1) / L.piece;
        L.p = take(a.tokens * L.piece * 4);
    }
    L.total = at;
    return L;
}

// Tensor maps with the 128-byte swizzle: a box is 128 bytes wide.
bool make_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* p, const cuuint64_t* dims,
              const cuuint64_t* strides, const cuuint32_t* box) {
    const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(host::tensor_map_encoder());
    if (!enc) return false;
    std::memset(map, 0, sizeof(*map));
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, type, cuuint32_t(rank), const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 16-bit elements move as they are, whichever of the two types they hold.
bool map_16(CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)}, strides[1] = {cuuint64_t(ld * 2)};
    const cuuint32_t box[2] = {64, cuuint32_t(box_rows)};
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, box);
}

bool map_f32(CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t ld) {
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)}, strides[1] = {cuuint64_t(ld * 4)};
    const cuuint32_t box[2] = {32, 32};
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p, dims, strides, box);
}

// B along its columns, two blocks of 64 in one copy, where its rows are whole blocks; else one block.
bool map_columns(CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t ld, bool blocks) {
    if (!blocks) return map_16(map, p, cols, rows, ld, kBK);
    const cuuint64_t dims[3] = {64, cuuint64_t(rows), cuuint64_t(cols / 64)};
    const cuuint64_t strides[2] = {cuuint64_t(ld * 2), 128};
    const cuuint32_t box[3] = {64, kBK, kHalf / 64};
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, strides, box);
}

// The piece's buffer as P^T: 64 words, tokens, the four blocks of a tile, the two parts of each tile in turn.
bool map_p_columns(CUtensorMap* map, const void* p, int64_t piece, int64_t rows) {
    const cuuint64_t dims[4] = {64, cuuint64_t(rows), kTN / 64, cuuint64_t(piece / kTN * 2)};
    const cuuint64_t strides[3] = {cuuint64_t(piece * 4), 128, kTN * 2};
    const cuuint32_t box[4] = {64, kBK, kHalf / 64, 1};
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p, dims, strides, box);
}

// The piece's buffer as P: 256 words, the two parts of each tile in turn, rows.
bool map_p(CUtensorMap* map, const void* p, int64_t piece, int64_t rows, int box_rows) {
    const cuuint64_t dims[3] = {cuuint64_t(kTN), cuuint64_t(piece / kTN * 2), cuuint64_t(rows)};
    const cuuint64_t strides[2] = {kTN * 2, cuuint64_t(piece * 4)};
    const cuuint32_t box[3] = {64, 1, cuuint32_t(box_rows)};
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, strides, box);
}

// dx's parts: hidden, tokens, parts.
bool map_sum(CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t parts) {
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(parts)};
    const cuuint64_t strides[2] = {cuuint64_t(cols * 4), cuuint64_t(cols * rows * 4)};
    const cuuint32_t box[3] = {32, 32, 1};
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p, dims, strides, box);
}

template <int kEpi>
int launch_mma(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, const MmaArgs& A, int sms,
               cudaStream_t st) {
    const auto k = &mma_kernel<kEpi>;
    if (int rc = host::set_smem_once(reinterpret_cast<const void*>(k), 12 + kEpi, kSmem)) return rc;
    const int64_t tiles = int64_t(A.mt) * A.nt * A.splits;
    return launch_dependent(k, dim3(2 * unsigned(tiles < sms / 2 ? tiles : sms / 2)), kThreads, kSmem, st, ta, tb, tc, A);
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
    const bool direct = reads_w_directly(a, w, grad);
    const bool copy_x = !map_ok(x, a.x_ld, a.hidden) && !direct, copy_w = !map_ok(w, a.w_ld, a.hidden) && !direct;
    const Layout L = layout(a, grad, copy_x, copy_w, direct, workspace_bytes);
    if (workspace_bytes < int64_t(L.total)) return FP8Z_ENOSPACE;
    const auto st = static_cast<cudaStream_t>(stream);
    auto* ws = static_cast<uint8_t*>(workspace);
    const int n = int(a.tokens), hidden = int(a.hidden), vocab = int(a.vocab);
    auto* target = reinterpret_cast<int32_t*>(ws + L.target);
    auto* target_logit = reinterpret_cast<float*>(ws + L.target_logit);
    auto* row_stats = reinterpret_cast<float2*>(ws + L.row_stats);
    auto* alpha = reinterpret_cast<float*>(ws + L.alpha);
    auto* part = reinterpret_cast<float2*>(ws + L.part);
    const auto done = [] { return cudaGetLastError() == cudaSuccess ? FP8Z_OK : FP8Z_ECUDA; };

    if (n == 0) {
        empty_total_kernel<<<1, 2, 0, st>>>(total);
        if (grad && !a.accumulate_dw) {
            if (a.dw_dtype == FP8Z_F32)
                zero_rows_kernel<<<sms * 8, 256, 0, st>>>(static_cast<float*>(dw), a.dw_ld, a.vocab, hidden);
            else
                zero_rows_kernel<<<sms * 8, 256, 0, st>>>(static_cast<__half*>(dw), a.dw_ld, a.vocab, hidden);
        }
        return done();
    }
    const void *xp = x, *wp = w;
    int64_t x_ld = a.x_ld, w_ld = a.w_ld;
    if (copy_x || copy_w) {
        const PadRows px = {static_cast<const uint16_t*>(x), reinterpret_cast<uint16_t*>(ws + L.x), a.x_ld, copy_x ? n : 0};
        const PadRows pw = {static_cast<const uint16_t*>(w), reinterpret_cast<uint16_t*>(ws + L.w), a.w_ld, copy_w ? vocab : 0};
        if (int rc = launch_dependent(pad_rows_kernel, dim3(unsigned((px.rows + pw.rows + 7) / 8)), 256, 0, st, px, pw, hidden,
                                      int(L.hidden_pad)))
            return rc;
        if (copy_x) {
            xp = ws + L.x;
            x_ld = L.hidden_pad;
        }
        if (copy_w) {
            wp = ws + L.w;
            w_ld = L.hidden_pad;
        }
    }
    const int period = period_of(a.w_ld);
    if (direct) {
        x_ld = shifted_width(hidden);
        if (int rc = launch_dependent(shift_rows_kernel, dim3(unsigned((n + 7) / 8), unsigned(period)), 256, 0, st,
                                      static_cast<const uint16_t*>(x), a.x_ld, n, hidden, int(x_ld),
                                      static_cast<const uint16_t*>(w), a.w_ld, reinterpret_cast<uint16_t*>(ws + L.x)))
            return rc;
        xp = ws + L.x;
    }
    uint8_t* p = ws + L.p;
    CUtensorMap x_k, w_k, logits;
    if (!direct && (!map_16(&x_k, xp, L.hidden_pad, n, x_ld, kHalf) ||
                    !map_16(&w_k, wp, L.hidden_pad, vocab, w_ld, kHalf)))
        return FP8Z_ECUDA;
    if (!grad) logits = w_k;                        // not used
    else if (!map_f32(&logits, p, L.piece, n, L.piece)) return FP8Z_ECUDA;
    const int last = grad ? int((L.pieces - 1) * L.piece) : vocab;      // the piece whose logits stay
    MmaArgs A;
    std::memset(&A, 0, sizeof(A));
    A.bf16 = a.dtype == FP8Z_BF16;
    A.timeout_ns = host::wait_limit_ns();
    A.dev_status = dev_status;
    A.m = n;
    A.rows = int(L.rows);
    A.n = vocab;
    A.mt = (n + kTM - 1) / kTM;
    A.nt = int(L.vocab_tiles);
    A.splits = 1;
    A.kb = int((L.hidden_pad + kBK - 1) / kBK);
    A.targets = targets;
    A.targets_wide = a.targets_dtype == FP8Z_I64;
    A.ignore = a.ignore_index;
    A.vocab = a.vocab;
    A.target = target;
    A.part = part;
    A.target_logit = target_logit;
    A.keep_from = last;
    A.ticket = reinterpret_cast<uint32_t*>(alpha + 1);
    A.p = p;
    A.p_bytes = L.piece * 4;
    int parts = A.nt * (kTN / kOwn);
    if (n <= kFewTokens) {
        parts = few_blocks(vocab, direct ? period : 1);
        const auto launch_few = [&](auto kernel) {
            return launch_dependent(kernel, dim3(unsigned(parts)), 256, 0, st, static_cast<const uint16_t*>(xp), x_ld,
                                    static_cast<const uint16_t*>(wp), w_ld, direct ? hidden : int(L.hidden_pad), period, A);
        };
        const auto by_type = [&](auto tiles) {
            constexpr int T = decltype(tiles)::value;
            if (direct) return A.bf16 ? launch_few(&few_kernel<T, true, false>) : launch_few(&few_kernel<T, false, false>);
            return A.bf16 ? launch_few(&few_kernel<T, true, true>) : launch_few(&few_kernel<T, false, true>);
        };
        if (int rc = n <= 8    ? by_type(std::integral_constant<int, 1>())
                     : n <= 16 ? by_type(std::integral_constant<int, 2>())
                               : by_type(std::integral_constant<int, 4>()))
            return rc;
    } else if (int rc = launch_mma<kStats>(x_k, w_k, logits, A, sms, st)) {
        return rc;
    }
    // FP16 P is kept times 2^15, at which 1 is still finite: normal numbers down to 2^-29, and
    // the smallest that counts is 2^-39 (with two parts: 16 bits or more from 2^-23 on)
    const float p_scale = A.bf16 ? 1.0f : 32768.0f;
    if (int rc = launch_dependent(rows_kernel, dim3(unsigned((n + 31) / 32)), 1024, 0, st, part, parts, n, A.rows, targets,
                                  A.targets_wide, A.ignore, A.vocab, target_logit, target, row_stats, lse, loss,
                                  reinterpret_cast<BlockTotal*>(ws + L.totals), A.ticket, a.reduction == FP8Z_MEAN,
                                  grad ? a.grad_scale / p_scale : 1.0f, total, grad ? alpha : nullptr, dev_status))
        return rc;
    if (!grad) return FP8Z_OK;

    auto* sum = reinterpret_cast<float*>(ws + L.sum);
    // dw leaves in tiles where its rows start and end on 16-byte boundaries: a tile's store writes
    // whole 16 bytes, and what lies behind a row that ends between two is not ours
    const int64_t dw_bytes = dtype_bytes(a.dw_dtype);
    const bool dw_tiles = host::aligned(dw, 16) && a.dw_ld * dw_bytes % 16 == 0 && a.hidden * dw_bytes % 16 == 0;
    const bool blocks = L.hidden_pad % 64 == 0;
    CUtensorMap p_k, w_mn, p_mn, x_mn, p_out, sum_out, dw_out = x_k;
    if (!map_p(&p_k, p, L.piece, n, kHalf) || !map_columns(&w_mn, wp, L.hidden_pad, vocab, w_ld, blocks) ||
        !map_p_columns(&p_mn, p, L.piece, n) || !map_columns(&x_mn, ws + L.kept_x, L.kept_ld, n, L.kept_ld, true) ||
        !map_p(&p_out, p, L.piece, n, 32) || !map_sum(&sum_out, sum, L.hidden_pad, n, L.splits))
        return FP8Z_ECUDA;
    if (dw_tiles && !(a.dw_dtype == FP8Z_F32 ? map_f32(&dw_out, dw, hidden, vocab, a.dw_ld)
                                            : map_16(&dw_out, dw, hidden, vocab, a.dw_ld, 32)))
        return FP8Z_ECUDA;
    for (int64_t i = L.pieces - 1; i >= 0; --i) {
        const int v0 = int(i * L.piece);
        const int words = int(a.vocab - v0 < L.piece ? a.vocab - v0 : L.piece), tiles = (words + kTN - 1) / kTN;
        if (v0 == last) {
            const dim3 grid(unsigned(n), unsigned((tiles + 8 * kProbTiles - 1) / (8 * kProbTiles) + 1));
            if (int rc = launch_dependent(prob_kernel, grid, 256, 0, st, p, L.piece * 4, tiles, words, v0, target, row_stats,
                                          p_scale, A.bf16, L.parts == 2, static_cast<const uint16_t*>(x), a.x_ld, hidden,
                                          reinterpret_cast<uint16_t*>(ws + L.kept_x), int(L.kept_ld)))
                return rc;
        } else {
            MmaArgs Q = A;                              // the piece's logits again, as P
            Q.n = words;
            Q.nt = tiles;
            Q.v0 = v0;
            Q.b_n0 = v0;
            Q.row_stats = row_stats;
            Q.split_p = L.parts == 2;
            Q.p_scale = p_scale;
            if (int rc = launch_mma<kProb>(x_k, w_k, p_out, Q, sms, st)) return rc;
        }
        MmaArgs D = A;                                  // dx += P w
        D.n = int(L.hidden_pad);
        D.nt = int((L.hidden_pad + kTN - 1) / kTN);
        D.kb = tiles * (kTN / kBK);
        D.splits = L.splits;
        D.b_k0 = v0;
        D.accumulate = v0 != last;
        D.b_blocks = blocks;
        if (int rc = launch_mma<kSum>(p_k, w_mn, sum_out, D, sms, st)) return rc;
        MmaArgs W = A;                                  // dw of the piece's words = P^T x
        W.m = words;
        W.n = hidden;
        W.mt = (words + kTM - 1) / kTM;
        W.nt = D.nt;
        W.v0 = v0;
        W.out = dw;
        W.out_ld = a.dw_ld;
        W.out_dtype = a.dw_dtype;
        W.accumulate = a.accumulate_dw;
        W.staged = dw_tiles && (a.dw_dtype == FP8Z_F32 || !a.accumulate_dw);
        W.alpha = alpha;
        W.b_blocks = 1;
        W.kb = (n + kBK - 1) / kBK;
        // Where a pair of blocks has few tiles of dw, an early start counts: 729 tokens x 2541 x 240
        // take 33 us for 40, 256 x 32000 x 1024 107 for 116.  Where it has many, the pairs drift apart
        // and share less of what they load: 517 x 100666 x 6376 would take 2060 us for 2007.
        W.beside = int64_t(W.mt) * W.nt <= 16 * (kSms / 2);
        if (int rc = L.parts == 2 ? launch_mma<kWeightSplit>(p_mn, x_mn, dw_out, W, sms, st)
                                  : launch_mma<kWeight>(p_mn, x_mn, dw_out, W, sms, st))
            return rc;
    }
    const dim3 grid(unsigned(n), unsigned((hidden + 1023) / 1024));
    if (A.bf16)
        return launch_dependent(finish_dx_kernel<__nv_bfloat16>, grid, 256, 0, st, sum, L.splits, n * L.hidden_pad,
                                L.hidden_pad, hidden, alpha, target, static_cast<__nv_bfloat16*>(dx), a.dx_ld);
    return launch_dependent(finish_dx_kernel<__half>, grid, 256, 0, st, sum, L.splits, n * L.hidden_pad, L.hidden_pad, hidden,
                            alpha, target, static_cast<__half*>(dx), a.dx_ld);
}

}  // namespace
}  // namespace fp8z

extern "C" int64_t fp8z_linear_xent_workspace(const void* x, const void* w, const fp8z_xent_args* args,
                                              int32_t with_grad, int64_t piece_words) {
    using namespace fp8z;
    if (!args || !args_ok(*args) || (with_grad && !grad_args_ok(*args)) || piece_words < 0) return FP8Z_EINVAL;
    const bool direct = reads_w_directly(*args, w, with_grad != 0);
    const bool cx = !map_ok(x, args->x_ld, args->hidden) && !direct, cw = !map_ok(w, args->w_ld, args->hidden) && !direct;
    Layout L = layout(*args, with_grad != 0, cx, cw, direct, -1);
    if (with_grad && piece_words > 0) {
        const int64_t less = L.piece - up(piece_words, kTN);
        if (less > 0) return int64_t(L.total) - less * args->tokens * 4;
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
