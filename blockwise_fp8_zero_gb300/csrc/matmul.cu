// matmul.cu -- products of E4M3 matrices with a scale for every 128 elements of K.
//
//   out[i][j] (+)= sum over blocks c of 128 of K:
//                  a_scale[i][c] * b_scale[j / R][c] * sum_{k in c} a[i][k] * b[j][k]
//
// R = 128: b is a weight in 128 x 128 blocks (a layer's forward pass, and its input
// gradient from the column-major copy).  R = 1: b is row-wise quantized like a (a
// weight gradient from two column-wise layouts).  The tensor cores multiply codes;
// scales differ from one block of K to the next, so a block's sum leaves tensor
// memory, is multiplied by its two scales and added up in FP32 registers.
//
// A bank of experts is one call, too: rows sorted by expert against [experts, n, k]
// weights, or K cut into the experts' tokens against [experts, m, n] gradients.
#include <algorithm>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "fp8z.h"
#include "fp8z_device.cuh"
#include "fp8z_elem.cuh"
#include "fp8z_host.h"
#include "fp8z_launch.cuh"
#include "fp8z_pairs.cuh"
#include "fp8z_stage.cuh"
#include "fp8z_tcgen05.cuh"

namespace fp8z {
namespace {

constexpr int kBK = 128;                       // K of a stage: 128 bytes of a row, and one scale
constexpr int kMaxGroups = 256;
enum { kByRows = 1, kByK = 2 };

struct Args {
    int m, n, kb;             // rows of a, rows of b, blocks of K (of all groups)
    int mt, nt;               // tiles of a product
    int groups, by;           // 1 and 0 without groups
    const void* offsets;
    int wide, total;          // offsets are 64-bit; what the last one may be
    const float* a_scale;
    const float* b_scale;
    int64_t a_scale_ld, b_scale_ld, b_scale_group;
    int b_scale_last;         // the last row of b's scales
    void* out;
    int64_t out_ld, out_group;
    int out_dtype, accumulate, staged;
    int64_t timeout_ns;
    int32_t* dev_status;
};

// Where the groups start, checked: not falling, inside the tensor, and, where they cut
// K, on whole blocks.  False (and nothing is computed) if one is not.  All threads.
__device__ __forceinline__ bool load_offsets(const Args& A, int* starts) {
    if (A.by == 0) return true;
    int bad = 0;
    for (int i = threadIdx.x; i <= A.groups; i += blockDim.x) {
        const auto at = [&](int j) {
            return A.wide ? static_cast<const volatile int64_t*>(A.offsets)[j]
                          : int64_t(static_cast<const volatile int32_t*>(A.offsets)[j]);
        };
        const int64_t o = at(i), before = i > 0 ? at(i - 1) : 0;
        bad |= o < before || o > A.total || (A.by == kByK && o % kBK != 0 && o != A.total);
        starts[i] = int(o);
    }
    if (!__syncthreads_or(bad)) return true;
    if (blockIdx.x == 0 && threadIdx.x == 0) report_status(A.dev_status, FP8Z_EINVAL);
    return false;
}

__device__ __forceinline__ float ld_scale(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}

// True in one lane of a warp that is together, by the instruction from which the compiler knows that
// there is one: what needs uniform registers (products, commits, tiled copies) then takes its
// operands straight, where behind a comparison of lane numbers it goes through a loop over lanes.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(one));
    return one != 0;
}

// Registers a thread of this warpgroup has from here on.
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// The registers of a tmem_ld16 or tmem_ld32 hold their values from here on.
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
// tmem_ld8, tmem_ld16 and tmem_ld32 for a warp that is together already.
__device__ __forceinline__ void tmem_load(uint32_t (&r)[8], uint32_t taddr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_load(uint32_t (&r)[16], uint32_t taddr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_load(uint32_t (&r)[32], uint32_t taddr) { tmem_ld32(r, taddr); }

__device__ __forceinline__ void ld_shared_pairs(uint32_t addr, uint64_t& a, uint64_t& b) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint64_t ld_shared_pair(uint32_t addr) {
    uint64_t a;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(a) : "r"(addr) : "memory");
    return a;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// A block's sums times their scales, added up: kCols columns of tensor memory from
// `acc` on, of the row of each lane, kStep at a time, the next ones on their way.
// kColScales: the columns' scales are the FP32 numbers at `scales` in shared memory and
// `f` is the row's; otherwise `f` is both.
template <int kCols, bool kColScales, int kStep>
__device__ __forceinline__ void add_block(uint64_t (&sums)[kCols / 2], uint32_t acc, float f, uint32_t scales) {
    const uint64_t ff = pair_of(f, f);
    uint32_t r[2][kStep];
    uint64_t col[kColScales ? kStep / 2 : 1];
    tmem_load(r[0], acc);
#pragma unroll
    for (int c = 0; c < kCols / kStep; ++c) {
        if constexpr (kColScales)
#pragma unroll
            for (int j = 0; j < kStep / 4; ++j) ld_shared_pairs(scales + (c * kStep + j * 4) * 4, col[2 * j], col[2 * j + 1]);
        tmem_arrived(r[c & 1]);
        if (c + 1 < kCols / kStep) tmem_load(r[(c + 1) & 1], acc + kStep * (c + 1));
#pragma unroll
        for (int j = 0; j < kStep / 2; ++j) {
            uint64_t x = ff;
            if constexpr (kColScales) x = mul_pair(col[j], ff);
            uint64_t& s = sums[c * (kStep / 2) + j];
            s = fma_pair(pair_of(r[c & 1][2 * j], r[c & 1][2 * j + 1]), x, s);
        }
    }
}

// 16 rows and 32 columns: lane t holds rows t / 4 and t / 4 + 8 and, of every 8 columns, the
// two from 2 (t % 4) on.
__device__ __forceinline__ void tmem_load_16x256b(uint32_t (&r)[16], uint32_t taddr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// The same for 128 columns that each have a scale.  A lane that has one row and all columns
// would load 128 scales a block, 16 bytes a lane each time: 1024 cycles of the SM's loads,
// twice what the products take.  With four rows and 32 columns a lane it is a quarter.
// Pair (h, g, e) of `sums`: row 16 h + 8 e + t / 4, columns from 8 g + 2 (t % 4) on.  `rows`
// and `cols`: where the scales of the lane's first row and of its first columns are.
__device__ __forceinline__ void add_block_rows(uint64_t (&sums)[64], uint32_t acc, uint32_t rows, uint32_t cols) {
    uint32_t r[2][16];
    tmem_load_16x256b(r[0], acc);
    uint64_t f[4], col[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = ld_shared_f32(rows + i * 32);
        f[i] = pair_of(x, x);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {                      // 32 columns of 16 rows, then of the other 16
        const int h = c & 1, q = c >> 1;
        if (h == 0)
#pragma unroll
            for (int j = 0; j < 4; ++j) col[j] = ld_shared_pair(cols + (q * 4 + j) * 32);
        tmem_arrived(r[c & 1]);
        if (c < 7) tmem_load_16x256b(r[(c + 1) & 1], acc + ((c + 1) >> 1) * 32 + (uint32_t((c + 1) & 1) << 20));
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint64_t& s = sums[(h * 16 + q * 4 + j) * 2 + e];
                s = fma_pair(pair_of(r[c & 1][j * 4 + e * 2], r[c & 1][j * 4 + e * 2 + 1]), mul_pair(col[j], f[h * 2 + e]), s);
            }
    }
}

// ------------------------------------------------------------- large products
constexpr int kTM = 256, kTN = 256, kHalf = 128;       // tile of a pair of blocks; a block's rows of a and of b
constexpr int kTileBytes = kHalf * kBK;
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kReaders = 8, kOwn = 128;                // warps that read the sums: 32 rows and 128 columns each
constexpr int kAccumulators = 2;
// The readers' sums and the loads on their way take more registers than an even share of
// the block's 384 x 168: 128 x 64 + 256 x 216 is a little less.
constexpr int kOtherRegs = 64, kReaderRegs = 216;
constexpr int kScaleSlots = 2, kScaleBlocks = 4;       // of scales: slots of four blocks of K

template <bool kRows>
struct Large {
    static constexpr int kStages = 5;
    // a block's scales: its rows' and all columns', or the products of rows' and each 128 columns' one
    static constexpr int kScaleWords = kRows ? kHalf + kTN : 2 * kHalf, kScaleBytes = kScaleBlocks * kScaleWords * 4;
    static constexpr int kThreads = 128 + 32 * kReaders;       // loads, products, b's scales, none; readers
    static constexpr int kStaging = kStages * kStageBytes;
    static constexpr int kScales = kStaging + kReaders * kSlab;
    static constexpr int kBars = kScales + kScaleSlots * kScaleBytes;
    static constexpr int kNumBars = 2 * kStages + 2 * kAccumulators + 1 + 2 * kScaleSlots;
    static constexpr int kStarts = kBars + kNumBars * 8 + 32;
    static constexpr int kSmem = kStarts + (kMaxGroups + 1) * 4 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory of one SM");
};

struct Tile {
    int group, row, row_end, n, k0, k1;        // rows [row, row_end) are this product's; n: column tile
};

// The t-th tile of all products; t must not fall from call to call.  Eight row tiles by
// all column tiles at a time, row tiles innermost: the blocks that run together share
// few rows of operands.
struct TileWalk {
    int group = 0, before = 0;
    __device__ __forceinline__ bool at(const Args& A, const int* starts, int t, Tile& out) {
        int first = 0, rows = A.m, mt = A.mt;
        out.k0 = 0;
        out.k1 = A.kb;
        if (A.by == kByRows) {
            while (true) {
                if (group == A.groups) return false;
                first = starts[group];
                rows = starts[group + 1] - first;
                mt = (rows + kTM - 1) / kTM;
                if (t < before + mt * A.nt) break;
                before += mt * A.nt;
                ++group;
            }
            t -= before;
        } else {
            group = t / (A.mt * A.nt);
            if (group >= A.groups) return false;
            t -= group * A.mt * A.nt;
            if (A.by == kByK) {
                // both up: a group that starts at a ragged end of K is empty
                out.k0 = (starts[group] + kBK - 1) / kBK;
                out.k1 = (starts[group + 1] + kBK - 1) / kBK;
            }
        }
        const int strip = t / (8 * A.nt), in = t - strip * 8 * A.nt, high = min(8, mt - strip * 8);
        out.group = group;
        out.row = first + (strip * 8 + in % high) * kTM;
        out.row_end = first + rows;
        out.n = in / high;
        return true;
    }
};

// 32 FP32 columns, or 64 of 16 bits (k16), from column i of the warp's sums on into its slab,
// whichever way the sums lie (add_block, or kRows: add_block_rows).
template <bool kRows, bool k16>
__device__ __forceinline__ void stage(Stager& sg, uint64_t (&sums)[kOwn / 2], int i, bool bf16) {
    const auto packed = [&](uint64_t p) {
        uint32_t a, b;
        halves(p, a, b);
        return pack16(__uint_as_float(a), __uint_as_float(b), bf16);
    };
    if constexpr (!kRows) {
        uint32_t r[32];
#pragma unroll
        for (int j = 0; j < (k16 ? 32 : 16); ++j) {
            if constexpr (k16) r[j] = packed(sums[i / 2 + j]);
            else halves(sums[i / 2 + j], r[2 * j], r[2 * j + 1]);
        }
        stage32(sg, r);
    } else {
        const uint32_t slab = sg.begin();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = h * 16 + e * 8 + sg.lane / 4;
#pragma unroll
                for (int g = 0; g < (k16 ? 8 : 4); ++g) {
                    const uint64_t p = sums[(h * 16 + i / 8 + g) * 2 + e];
                    const int byte = (g * 8 + sg.lane % 4 * 2) * (k16 ? 2 : 4);
                    const uint32_t to = slab + swz128(row, byte);
                    if constexpr (k16) asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(packed(p)) : "memory");
                    else asm volatile("st.shared.b64 [%0], %1;" ::"r"(to), "l"(p) : "memory");
                }
            }
    }
}

// The tile's results of one warp: 128 columns from c0 on, of the row of each lane.  A
// tile of 32 rows leaves at once where its rows are all this product's (or the tensor
// ends with them) and all rows start and end on 16-byte boundaries.
template <bool kRows>
__device__ __forceinline__ void store_large(const Args& A, const CUtensorMap& out, const Tile& t, uint64_t (&sums)[kOwn / 2],
                                            int c0, int row, Stager& sg) {
    const int first = row - sg.lane, rows = min(32, t.row_end - first), col0 = t.n * kTN + c0;
    if (rows <= 0) return;
    const bool tiles = A.staged && (A.by != kByRows || rows == 32);
    const int z = A.by == kByK ? t.group : 0;
    if (tiles && A.out_dtype != FP8Z_F32) {
#pragma unroll
        for (int i = 0; i < kOwn; i += 64) {
            if (col0 + i >= A.n) break;
            stage<kRows, true>(sg, sums, i, A.out_dtype == FP8Z_BF16);
            sg.end([&](uint32_t s) { tma_store_3d(&out, col0 + i, row, z, s); });
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kOwn; i += 32) {
        const int col = col0 + i;
        if (col >= A.n) break;
        stage<kRows, false>(sg, sums, i, false);
        if (tiles) {
            sg.end([&](uint32_t s) {
                if (A.accumulate) tma_add_3d(&out, col, row, z, s);
                else tma_store_3d(&out, col, row, z, s);
            });
        } else {
            __syncwarp();
            const int64_t at = z * A.out_group + int64_t(first) * A.out_ld + col;
            const int n = A.n - col;
            if (A.out_dtype == FP8Z_F32) weight_rows(static_cast<float*>(A.out) + at, A.out_ld, rows, n, sg, A.accumulate);
            else if (A.out_dtype == FP8Z_BF16) weight_rows(static_cast<__nv_bfloat16*>(A.out) + at, A.out_ld, rows, n, sg, false);
            else weight_rows(static_cast<__half*>(A.out) + at, A.out_ld, rows, n, sg, false);
            __syncwarp();
        }
    }
}

// A pair of blocks takes 256 x 256 results at a time.  Each block loads 128 rows of a
// and 128 of b into a ring of stages; one thread of the first block issues the products
// of both, each block of K into the other of two accumulators, while eight warps of
// each block read the one before, scale it and add it up.
//
// 4096 x 18432 x 7168: 448 to 485 us by the box, 2.2 to 2.4 PFLOP/s.  The copies alone (64 KB a pair and block
// of K from L2) take 343; the rest is the way of an accumulator to its readers and back with
// two of them, all that tensor memory holds at 256 columns.  Stages (3 to 5) do not matter;
// sixteen readers of 64 columns take 512 us, halves of 128 columns with four accumulators 619.
// With a scale for every column, 2048 x 7168 x 8192 added to FP32 takes 171 us (1.4 PFLOP/s):
// the readers' second scale is one packed product more for every sum.
template <bool kRows>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Large<kRows>::kThreads, 1)
    large_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                 const __grid_constant__ CUtensorMap tc, const __grid_constant__ Args A) {
    using L = Large<kRows>;
    constexpr int kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_addr(smem_raw));
    const uint32_t bars = base + L::kBars;
    auto full = [&](int s) { return bars + s * 8; };                       // first block: both blocks' copies are there
    auto empty = [&](int s) { return bars + (kStages + s) * 8; };          // the products that read them are done
    auto tfull = [&](int b) { return bars + (2 * kStages + b) * 8; };
    auto tempty = [&](int b) { return bars + (2 * kStages + 2 + b) * 8; };  // first block: both blocks' warps have read it
    const uint32_t drain = bars + (2 * kStages + 4) * 8;
    auto sfull = [&](int i) { return bars + (2 * kStages + 5 + i) * 8; };
    auto sempty = [&](int i) { return bars + (2 * kStages + 5 + kScaleSlots + i) * 8; };
    uint8_t* words = smem + L::kBars + L::kNumBars * 8;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(words);
    volatile uint32_t* tmem_at = reinterpret_cast<volatile uint32_t*>(words + 8);
    volatile uint32_t* issued_by = reinterpret_cast<volatile uint32_t*>(words + 16);   // [2]
    int* starts = reinterpret_cast<int*>(smem + L::kStarts);
    const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int rank = int(cluster_rank()), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 2);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < kAccumulators; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), 2 * kReaders);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(sfull(i), 1);
            mbar_init(sempty(i), kReaders);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        issued_by[0] = issued_by[1] = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 32) {
        tensormap_prefetch(&ta);
        tensormap_prefetch(&tb);
    }
    if (warp == 1) tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_at)), kAccumulators * kTN);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    dependent_wait();
    const uint32_t tmem = *tmem_at;
    const Watchdog wd{abort_flag, A.dev_status, A.timeout_ns};
    const bool run = load_offsets(A, starts);          // the same in both blocks
    TileWalk walk;
    Tile at;

    if (warp < 4) fewer_registers<kOtherRegs>();
    if (!run) {
    } else if (warp == 0) {
        if (elect_one()) {
            int s = 0, ph = 0;
            uint32_t issued = 0;
            bool ok = true;
            for (int t = pair; ok && walk.at(A, starts, t, at); t += pairs) {
                const int am = at.row + rank * kHalf, bn = at.n * kTN + rank * kHalf, z = A.by == kByRows ? at.group : 0;
                for (int k = at.k0; k < at.k1; ++k) {
                    if (!mbar_wait_bounded(empty(s), ph ^ 1, wd)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = base + s * kStageBytes, bar = cluster_addr(full(s), 0);
                    mbar_arrive_expect_tx_cluster(bar, kStageBytes);
                    tma_load_2d_pair(sa, &ta, k * kBK, am, bar);
                    tma_load_3d_pair(sa + kTileBytes, &tb, k * kBK, bn, z, bar);
                    ++issued;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            st_cluster_u32(cluster_addr(smem_addr(const_cast<uint32_t*>(issued_by + rank)), 0), issued);
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = umma_idesc_e4m3(kTM, kTN);
            int s = 0, ph = 0, b = 0, bph = 0;
            bool ok = true;
            for (int t = pair; ok && walk.at(A, starts, t, at); t += pairs) {
                for (int k = at.k0; k < at.k1; ++k) {
                    if (!mbar_wait_bounded(full(s), ph, wd) || !mbar_wait_bounded(tempty(b), bph ^ 1, wd)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = base + s * kStageBytes;
                    const uint64_t da = umma_desc(sa, 16, 1024), db = umma_desc(sa + kTileBytes, 16, 1024);
#pragma unroll
                    for (int j = 0; j < kBK / 32; ++j)      // 32 of K: 32 bytes of a row
                        umma_e4m3_pair(tmem + b * kTN, da + j * 2, db + j * 2, idesc, j != 0);
                    umma_commit_pair(empty(s));
                    umma_commit_pair(tfull(b));
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                    if (b) bph ^= 1;
                    b ^= 1;
                }
            }
            umma_commit_pair(drain);       // of this thread's products: another's commit would say nothing of them
        }
    } else if (warp >= 4) {
        more_registers<kReaderRegs>();
        const int quarter = warp & 3, c0 = (warp - 4) / 4 * kOwn;    // a warp reaches its quarter of the lanes: 32 rows
        Stager sg{base + L::kStaging + (warp - 4) * kSlab, lane};
        int b = 0, bph = 0, slot = 0, sph = 0;
        bool ok = true;
        for (int t = pair; ok && walk.at(A, starts, t, at); t += pairs) {
            const int row = at.row + rank * kHalf + quarter * 32 + lane;
            uint64_t sums[kOwn / 2];
#pragma unroll
            for (int j = 0; j < kOwn / 2; ++j) sums[j] = 0;
            for (int k = at.k0; k < at.k1; ++k) {
                const int of = (k - at.k0) % kScaleBlocks;
                if (of == 0) ok = mbar_wait_bounded(sfull(slot), sph, wd);
                const uint32_t scales = base + L::kScales + slot * L::kScaleBytes + of * L::kScaleWords * 4;
                ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait_bounded(tfull(b), bph, wd));
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + b * kTN + c0 + (uint32_t(quarter * 32) << 16);
                if constexpr (kRows) add_block_rows(sums, acc, scales + (quarter * 32 + lane / 4) * 4, scales + (kHalf + c0 + lane % 4 * 2) * 4);
                else add_block<kOwn, false, 16>(sums, acc, ld_shared_f32(scales + (c0 + quarter * 32 + lane) * 4), 0);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_relaxed(tempty(b), 0);
                if (b) bph ^= 1;
                b ^= 1;
                if (of == kScaleBlocks - 1 || k + 1 == at.k1) {
                    if (lane == 0) mbar_arrive(sempty(slot));
                    if (slot) sph ^= 1;
                    slot ^= 1;
                }
            }
            if (ok) store_large<kRows>(A, tc, at, sums, c0, row, sg);
        }
        if (lane == 0) bulk_wait_all();
    } else if (warp == 2) {
        // Scales, two blocks of K at a time: 12 to 24 loads a lane are under way at once.
        constexpr int kB = kRows ? kTN / 32 : 2;       // of b that a lane brings
        int slot = 0, sph = 0;
        bool ok = true;
        for (int t = pair; ok && walk.at(A, starts, t, at); t += pairs) {
            const float* pa = A.a_scale + int64_t(at.row + rank * kHalf + lane) * A.a_scale_ld;
            const float* pb = A.b_scale + at.group * A.b_scale_group;
            const int rows = A.m - (at.row + rank * kHalf + lane), b0 = kRows ? at.n * kTN + lane : at.n * 2;
            for (int k = at.k0; ok && k < at.k1; k += kScaleBlocks) {
#pragma unroll 1
                for (int i = 0; i < kScaleBlocks; i += 2) {
                    float v[2][kHalf / 32], w[2][kB];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bool in = k + i + h < at.k1;
#pragma unroll
                        for (int j = 0; j < kHalf / 32; ++j) v[h][j] = in && j * 32 < rows ? ld_scale(pa + j * 32 * A.a_scale_ld + k + i + h) : 0.0f;
#pragma unroll
                        for (int j = 0; j < kB; ++j)
                            w[h][j] = in ? ld_scale(pb + min(b0 + j * (kRows ? 32 : 1), A.b_scale_last) * A.b_scale_ld + k + i + h) : 0.0f;
                    }
                    if (i == 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(sempty(slot), sph ^ 1, wd));
                    if (!ok) break;
                    const uint32_t to = base + L::kScales + slot * L::kScaleBytes + i * L::kScaleWords * 4 + lane * 4;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int j = 0; j < kHalf / 32; ++j) {
                            st_shared_f32(to + (h * L::kScaleWords + j * 32) * 4, kRows ? v[h][j] : v[h][j] * w[h][0]);
                            if (!kRows) st_shared_f32(to + (h * L::kScaleWords + kHalf + j * 32) * 4, v[h][j] * w[h][1]);
                        }
                        if (kRows)
#pragma unroll
                            for (int j = 0; j < kB; ++j) st_shared_f32(to + (h * L::kScaleWords + kHalf + j * 32) * 4, w[h][j]);
                    }
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(sfull(slot));
                if (slot) sph ^= 1;
                slot ^= 1;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    // Whatever a wait gave up on, every copy lands before either block ends.  A stage for which
    // one of the two threads never came to issue its copies lacks its arrival: it is made here.
    if (rank == 0 && threadIdx.x == 0) {
        if (run) mbar_wait_drain(drain, 0, A.dev_status);      // every product is done before tensor memory is freed
        const uint32_t most = max(issued_by[0], issued_by[1]);
        for (int j = 0; j < 2; ++j)
            for (uint32_t i = issued_by[j]; i < most; ++i) mbar_arrive(full(i % kStages));
        for (uint32_t i = most > kStages ? most - kStages : 0; i < most; ++i)
            mbar_wait_drain(full(i % kStages), (i / kStages) & 1, A.dev_status);
    }
    if (run && rank == 1 && threadIdx.x == 0) mbar_wait_drain(drain, 0, A.dev_status);    // the last arrival from the first block
    cluster_sync();                        // neither block ends, nor frees, while the other may still reach it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kAccumulators * kTN);
    }
}

// ------------------------------------------------------- few rows, small products
// One block takes 128 rows of b by kT rows of a, b's rows in the tensor memory's lanes:
// a weight of few tokens is read once, at the memory's rate, and no tile is mostly empty.
// Where that leaves SMs without work, the blocks of a cluster share a tile: each takes
// a part of K, and then adds up the parts of some of a's rows, which it reads from the
// others' shared memory in a fixed order.
// 8 x 18432 x 7168: 25 us, of which the weights' 132 MB are 19.5 at the copy's rate.
constexpr int kRowsB = 128;
constexpr int kSmallThreads = 192;             // loads, products, four readers
constexpr int kMaxSplits = 8;

template <int kT>
struct Small {
    static constexpr int kTileA = kT * kBK, kTileB = kRowsB * kBK, kStageBytes = kTileA + kTileB;
    static constexpr int kStages = kT <= 32 ? 5 : 4;                           // two blocks an SM
    static constexpr int kAcc = kT >= 32 ? 256 / kT : 8;                       // accumulators
    static constexpr int kTmem = kAcc * kT;
    static constexpr int kScales = kStages * kStageBytes;                      // two blocks' scales for each reader
    static constexpr int kBars = kScales + 4 * 2 * kT * 4;
    static constexpr int kNumBars = 2 * kStages + 2 * kAcc + 1;
    static constexpr int kStarts = kBars + kNumBars * 8 + 32;
    static constexpr int kSmem = kStarts + (kMaxGroups + 1) * 4 + 1024;
    static_assert(kSmem <= 113 * 1024, "two blocks an SM");
    static_assert(kT * kRowsB * 4 <= kScales, "the parts of a tile fit the ring");
};

template <typename T>
__device__ __forceinline__ void put_out(T* p, float v, bool add) {
    *p = Elem<T>::narrow(add ? Elem<T>::widen(*p) + v : v);
}

__device__ __forceinline__ void put_out(const Args& A, int row, int col, float v) {
    const int64_t at = int64_t(row) * A.out_ld + col;
    if (A.out_dtype == FP8Z_F32) put_out(static_cast<float*>(A.out) + at, v, A.accumulate);
    else if (A.out_dtype == FP8Z_BF16) put_out(static_cast<__nv_bfloat16*>(A.out) + at, v, false);
    else put_out(static_cast<__half*>(A.out) + at, v, false);
}

template <int kT, bool kRows>
__global__ void __launch_bounds__(kSmallThreads, 2)
    small_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                 const __grid_constant__ Args A, const int splits) {
    using L = Small<kT>;
    constexpr int kStages = L::kStages, kAcc = L::kAcc;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_addr(smem_raw));
    const uint32_t bars = base + L::kBars;
    auto full = [&](int s) { return bars + s * 8; };
    auto empty = [&](int s) { return bars + (kStages + s) * 8; };
    auto tfull = [&](int b) { return bars + (2 * kStages + b) * 8; };
    auto tempty = [&](int b) { return bars + (2 * kStages + kAcc + b) * 8; };
    const uint32_t drain = bars + (2 * kStages + 2 * kAcc) * 8;
    uint8_t* words = smem + L::kBars + L::kNumBars * 8;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(words);
    volatile uint32_t* tmem_at = reinterpret_cast<volatile uint32_t*>(words + 8);
    volatile uint32_t* issued_by = reinterpret_cast<volatile uint32_t*>(words + 16);
    int* starts = reinterpret_cast<int*>(smem + L::kStarts);
    const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int part = int(blockIdx.x % unsigned(splits)), tile = int(blockIdx.x / unsigned(splits));

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < kAcc; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        *issued_by = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 32) {
        tensormap_prefetch(&ta);
        tensormap_prefetch(&tb);
    }
    if (warp == 1) tmem_alloc_one(smem_addr(const_cast<uint32_t*>(tmem_at)), L::kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    dependent_wait();
    const uint32_t tmem = *tmem_at;
    const Watchdog wd{abort_flag, A.dev_status, A.timeout_ns};

    // Row tiles innermost: blocks next to each other read the same rows of b.
    const int n0 = tile / A.mt * kRowsB;
    int mt = tile % A.mt, group = 0, row0 = mt * kT, row_end = A.m;
    bool run = load_offsets(A, starts);
    if (run && A.by == kByRows) {
        // mt counts the row tiles of all groups; the last few of the launch may not be there
        int first = 0, last = 0;
        for (; group < A.groups; ++group) {
            first = starts[group];
            last = starts[group + 1];
            const int tiles = (last - first + kT - 1) / kT;
            if (mt < tiles) break;
            mt -= tiles;
        }
        run = group < A.groups;
        row0 = first + mt * kT;
        row_end = last;
    }
    const int k0 = int(int64_t(A.kb) * part / splits), k1 = int(int64_t(A.kb) * (part + 1) / splits);
    const int rows = min(kT, row_end - row0);
    uint64_t sums[kT / 2];
#pragma unroll
    for (int j = 0; j < kT / 2; ++j) sums[j] = 0;
    bool ok = true;

    if (!run) {
    } else if (warp == 0) {
        if (elect_one()) {
            int s = 0, ph = 0;
            uint32_t issued = 0;
            for (int k = k0; k < k1; ++k) {
                if (!mbar_wait_bounded(empty(s), ph ^ 1, wd)) break;
                const uint32_t sb = base + s * L::kStageBytes;
                mbar_arrive_expect_tx(full(s), L::kStageBytes);
                tma_load_3d(sb, &tb, k * kBK, n0, group, full(s));
                tma_load_2d(sb + L::kTileB, &ta, k * kBK, row0, full(s));
                ++issued;
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            *issued_by = issued;
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t idesc = umma_idesc_e4m3(kRowsB, kT);
            int s = 0, ph = 0, b = 0, bph = 0;
            for (int k = k0; k < k1; ++k) {
                if (!mbar_wait_bounded(tempty(b), bph ^ 1, wd) || !mbar_wait_bounded(full(s), ph, wd)) break;
                tc_fence_after();
                const uint32_t sb = base + s * L::kStageBytes;
                const uint64_t db = umma_desc(sb, 16, 1024), da = umma_desc(sb + L::kTileB, 16, 1024);
#pragma unroll
                for (int j = 0; j < kBK / 32; ++j) umma_e4m3(tmem + b * kT, db + j * 2, da + j * 2, idesc, j != 0);
                umma_commit_one(empty(s));
                umma_commit_one(tfull(b));
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1;
                }
                if (++b == kAcc) {
                    b = 0;
                    bph ^= 1;
                }
            }
            umma_commit_one(drain);        // of this thread's products: another's commit would say nothing of them
        }
    } else {
        const int quarter = warp & 3, col = n0 + quarter * 32 + lane;
        constexpr int kEach = (kT + 31) / 32;          // rows of a whose scales a lane brings
        const float* pa[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) pa[j] = A.a_scale + min(row0 + j * 32 + lane, A.m - 1) * A.a_scale_ld;
        const float* pb = A.b_scale + group * A.b_scale_group + min(kRows ? col : n0 / kBK, A.b_scale_last) * A.b_scale_ld;
        const uint32_t scales = base + L::kScales + (warp - 2) * 2 * kT * 4;
        float fa[kEach], fb = 0.0f;
        if (k0 < k1) {
#pragma unroll
            for (int j = 0; j < kEach; ++j) fa[j] = ld_scale(pa[j] + k0);
            fb = ld_scale(pb + k0);
        }
        int b = 0, bph = 0;
        for (int k = k0; k < k1; ++k) {
            const float f = kRows ? fb : 1.0f;
            const uint32_t to = scales + (k & 1) * kT * 4;
#pragma unroll
            for (int j = 0; j < kEach; ++j)
                if (j * 32 + lane < kT) st_shared_f32(to + (j * 32 + lane) * 4, kRows ? fa[j] : fa[j] * fb);
            if (k + 1 < k1) {
#pragma unroll
                for (int j = 0; j < kEach; ++j) fa[j] = ld_scale(pa[j] + k + 1);
                fb = ld_scale(pb + k + 1);
            }
            __syncwarp();
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(tfull(b), bph, wd));
            if (!ok) break;
            tc_fence_after();
            add_block<kT, true, 16>(sums, tmem + b * kT + (uint32_t(quarter * 32) << 16), f, to);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty(b));
            if (++b == kAcc) {
                b = 0;
                bph ^= 1;
            }
        }
        if (splits == 1) {
            if (ok && col < A.n) {
#pragma unroll
                for (int j = 0; j < kT; ++j) {
                    uint32_t v[2];
                    halves(sums[j / 2], v[0], v[1]);
                    if (j < rows) put_out(A, row0 + j, col, __uint_as_float(v[j & 1]));
                }
            }
        } else {
            // every product that reads the ring is done: its last sums have been read
#pragma unroll
            for (int j = 0; j < kT; j += 2) {
                uint32_t v0, v1;
                halves(sums[j / 2], v0, v1);
                st_shared_f32(base + (j * kRowsB + quarter * 32 + lane) * 4, __uint_as_float(v0));
                st_shared_f32(base + ((j + 1) * kRowsB + quarter * 32 + lane) * 4, __uint_as_float(v1));
            }
        }
    }
    if (splits > 1) {
        cluster_sync();
        if (run && warp >= 2) {
            const int at = threadIdx.x - 64, col = n0 + at;
            uint32_t from[kMaxSplits];
#pragma unroll
            for (int i = 0; i < kMaxSplits; ++i) from[i] = i < splits ? cluster_addr(base + at * 4, i) : 0;
            if (ok && col < A.n)
                for (int j = part; j < rows; j += splits) {
                    float v[kMaxSplits];
#pragma unroll
                    for (int i = 0; i < kMaxSplits; ++i) v[i] = i < splits ? ld_cluster_f32(from[i] + j * kRowsB * 4) : 0.0f;
                    float sum = v[0];
#pragma unroll
                    for (int i = 1; i < kMaxSplits; ++i) sum += v[i];
                    put_out(A, row0 + j, col, sum);
                }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t issued = *issued_by;
        for (uint32_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
            mbar_wait_drain(full(i % kStages), (i / kStages) & 1, A.dev_status);
    }
    if (splits > 1) cluster_sync();        // the others may still read this block's sums
    if (warp == 1) {
        if (run) mbar_wait_drain(drain, 0, A.dev_status);      // every product is done before tensor memory is freed
        tc_fence_after();
        tmem_dealloc_one(tmem, L::kTmem);
    }
}

// ------------------------------------------------------------ small kernels
// Rows of bytes copied to a stride the tensor maps can step over: 16 bytes a thread, zeros
// after the end.  Words that hold only bytes of the row are loaded whole.
__global__ void __launch_bounds__(256) pad_bytes_kernel(const uint8_t* src, int64_t ld, int64_t group_ld, int rows,
                                                        int cols, uint8_t* dst, int cols_pad, int64_t pieces) {
    dependent_wait();
    const int per = cols_pad / 16;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < pieces; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t r = i / per;
        const int c = int(i - r * per) * 16;
        const uint8_t* p = src + r / rows * group_ld + r % rows * ld + c;
        uint32_t v[4] = {};
        const uint32_t shift = uint32_t(reinterpret_cast<uintptr_t>(p) & 3) * 8;
        if (c >= 4 && c + 20 <= cols) {
            const volatile uint32_t* w = reinterpret_cast<const volatile uint32_t*>(p - shift / 8);
            uint32_t x[5];
#pragma unroll
            for (int j = 0; j < 5; ++j) x[j] = w[j];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __funnelshift_r(x[j], x[j + 1], shift);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j < cols) v[j / 4] |= uint32_t(*reinterpret_cast<const volatile uint8_t*>(p + j)) << (j & 3) * 8;
        }
        *reinterpret_cast<uint4*>(dst + r * cols_pad + c) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// The result where K is empty.
template <typename T>
__global__ void __launch_bounds__(256) zero_kernel(T* out, int64_t ld, int64_t group_ld, int rows, int cols) {
    dependent_wait();
    T* p = out + blockIdx.z * group_ld;
    for (int r = blockIdx.x; r < rows; r += gridDim.x)
        for (int c = threadIdx.x; c < cols; c += blockDim.x) p[int64_t(r) * ld + c] = Elem<T>::narrow(0.0f);
}

// ------------------------------------------------------------------- host
bool bytes_map(CUtensorMap* map, int rank, const void* p, int64_t cols, int64_t rows, int64_t groups, int64_t ld,
               int64_t group_ld, int box_rows) {
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(groups)};
    const cuuint64_t strides[2] = {cuuint64_t(ld), cuuint64_t(group_ld)};
    const cuuint32_t box[3] = {kBK, cuuint32_t(box_rows), 1};
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, p, dims, strides, box);
}

bool out_map(CUtensorMap* map, const fp8z_matmul_args& a, void* p) {
    const bool bank = a.group_by == FP8Z_GROUP_K && a.groups > 1;
    const int64_t size = dtype_bytes(a.out_dtype);
    const cuuint64_t dims[3] = {cuuint64_t(a.n), cuuint64_t(a.m), cuuint64_t(bank ? a.groups : 1)};
    const cuuint64_t strides[2] = {cuuint64_t(a.out_ld * size), cuuint64_t((bank ? a.out_group : a.out_ld * a.m) * size)};
    const cuuint32_t box[3] = {cuuint32_t(128 / size), 32, 1};
    const auto type = a.out_dtype == FP8Z_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return make_map(map, type, 3, p, dims, strides, box);
}

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

constexpr int64_t kMost = 1LL << 30;

bool args_ok(const fp8z_matmul_args& a) {
    if (a.m < 0 || a.n < 0 || a.k < 0 || a.m > kMost || a.n > kMost || a.k > kMost) return false;
    if (a.groups < 0 || a.groups > kMaxGroups) return false;
    if (a.groups > 0 && a.group_by != FP8Z_GROUP_ROWS && a.group_by != FP8Z_GROUP_K) return false;
    if (a.groups > 0 && a.offsets_dtype != FP8Z_I32 && a.offsets_dtype != FP8Z_I64) return false;
    if (a.b_scale_rows != 1 && a.b_scale_rows != FP8Z_BLOCK) return false;
    if (a.groups > 0 && (a.b_scale_rows == 1) != (a.group_by == FP8Z_GROUP_K)) return false;
    if (!dtype_ok(a.out_dtype) || (a.accumulate != 0 && a.accumulate != 1)) return false;
    if (a.accumulate && a.out_dtype != FP8Z_F32) return false;
    const int64_t kb = (a.k + kBK - 1) / kBK, most = 1LL << 38;
    if (a.a_ld < a.k || a.b_ld < a.k || a.out_ld < a.n || a.a_scale_ld < kb || a.b_scale_ld < kb) return false;
    if (a.a_ld > most || a.b_ld > most || a.out_ld > most || a.a_scale_ld > most || a.b_scale_ld > most) return false;
    const int64_t scale_rows = a.b_scale_rows == 1 ? a.n : (a.n + kBK - 1) / kBK;
    if (a.groups > 1 && a.group_by == FP8Z_GROUP_ROWS &&
        (a.b_group < a.b_ld * (a.n - 1) + a.k || a.b_scale_group < a.b_scale_ld * (scale_rows - 1) + kb ||
         a.b_group > most || a.b_scale_group > most))
        return false;
    if (a.groups > 1 && a.group_by == FP8Z_GROUP_K && (a.out_group < a.out_ld * (a.m - 1) + a.n || a.out_group > most))
        return false;
    // tiles are counted in 32 bits
    const int64_t products = a.groups > 0 && a.group_by == FP8Z_GROUP_K ? a.groups : 1;
    return ((a.m + 15) / 16 + a.groups) * ((a.n + 127) / 128) * products <= (1LL << 26);
}

// A tensor map steps over rows of whole 16 bytes.
bool map_ok(const void* p, int64_t rows, int64_t ld, int64_t groups, int64_t group_ld) {
    return host::aligned(p, 16) && (rows <= 1 || ld % 16 == 0) && (groups <= 1 || group_ld % 16 == 0);
}

struct Plan {
    bool copy_a, copy_b;
    int64_t k_pad, a_at, b_at, bytes;
};
Plan plan(const void* a, const void* b, const fp8z_matmul_args& g) {
    Plan p;
    const bool bank = g.groups > 0 && g.group_by == FP8Z_GROUP_ROWS;
    p.copy_a = !map_ok(a, g.m, g.a_ld, 1, 0);
    p.copy_b = !map_ok(b, g.n, g.b_ld, bank ? g.groups : 1, g.b_group);
    p.k_pad = up(g.k, 16);
    p.a_at = 0;
    p.b_at = p.copy_a ? up(g.m * p.k_pad, 256) : 0;
    p.bytes = p.b_at + (p.copy_b ? up((bank ? g.groups : 1) * g.n * p.k_pad, 256) : 0);
    return p;
}

// Whether tiles of 128 rows of b, how many rows of a they take, and into how many parts K
// is cut; 0 rows: pairs of blocks and tiles of 256 x 256.
struct Choice {
    int rows, splits;
};
// By time: a block of K takes a pair 0.5 us (0.85 where every column has a scale), and a small block
// 0.45 us, or 0.6 where two share an SM; a launch takes 4 us, a large tile's results 1.5, joining the
// parts of K 1.5; nothing is quicker than its bytes.  Measured: 512 x 2048 x 7168 33 us by pairs and 25
// with tiles of 64 rows and K in two, 1000 x 2048 x 2048 14.6 and 15.4, 4096 x 2048 x 2048 25 and 66.
Choice choose(const fp8z_matmul_args& g, int sms) {
    if (g.groups > 0 && g.group_by == FP8Z_GROUP_K) return {0, 1};
    const int64_t kb = (g.k + kBK - 1) / kBK, groups = std::max<int64_t>(g.groups, 1);
    const int64_t each = (g.m + groups - 1) / groups;         // rows of a product, on average
    const auto tiles = [&](int64_t rows_a, int64_t rows_b) { return (each + rows_a - 1) / rows_a * groups * ((g.n + rows_b - 1) / rows_b); };
    const auto waves = [](int64_t t, int64_t at_once) { return double((t + at_once - 1) / at_once); };
    const double block = g.b_scale_rows == 1 ? 0.85 : 0.5, bytes = 5.0 + double(std::min<int64_t>(groups, std::max<int64_t>(g.m, 1))) * double(g.n) * double(g.k) / 6.5e6;
    Choice best = {0, 1};
    double least = std::max(bytes, 4.0 + waves(tiles(kTM, kTN), sms / 2) * (double(kb) * block + 1.5));
    for (int rows = 16; rows <= 64; rows *= 2) {
        if (rows > 16 && rows / 2 >= each) break;
        const int64_t t = tiles(rows, kRowsB);
        for (int splits = 1; splits <= kMaxSplits && splits <= kb; ++splits) {
            const double cost = 4.0 + waves(t * splits, 2 * sms) * double((kb + splits - 1) / splits) * (t * splits > sms ? 0.6 : 0.45) + (splits > 1 ? 1.5 : 0.0);
            // the fewer parts and rows among equals
            if (std::max(cost, bytes) < least - 0.01) {
                least = std::max(cost, bytes);
                best = {rows, splits};
            }
        }
    }
    return best;
}

template <bool kRows>
int launch_large(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, const Args& A, int64_t tiles, int sms,
                 cudaStream_t st) {
    const auto k = &large_kernel<kRows>;
    if (int rc = host::set_smem_once(reinterpret_cast<const void*>(k), 17 + kRows, Large<kRows>::kSmem)) return rc;
    return launch_dependent(k, dim3(2 * unsigned(std::min<int64_t>(tiles, sms / 2))), Large<kRows>::kThreads,
                            Large<kRows>::kSmem, st, ta, tb, tc, A);
}

template <int kT>
int launch_small(const CUtensorMap& ta, const CUtensorMap& tb, const Args& A, bool rows, int splits, int64_t blocks, int slot,
                 cudaStream_t st) {
    const auto k = rows ? &small_kernel<kT, true> : &small_kernel<kT, false>;
    if (int rc = host::set_smem_once(reinterpret_cast<const void*>(k), slot + rows, Small<kT>::kSmem)) return rc;
    return launch_dependent_clusters(k, splits, dim3(unsigned(blocks)), kSmallThreads, Small<kT>::kSmem, st, ta, tb, A, splits);
}

int run(const void* a, const float* a_scale, const void* b, const float* b_scale, const fp8z_matmul_args* args,
        const void* offsets, void* out, void* workspace, int64_t workspace_bytes, int32_t* dev_status, void* stream) {
    if (!args || !args_ok(*args)) return FP8Z_EINVAL;
    const fp8z_matmul_args& g = *args;
    const bool grouped = g.groups > 0, by_rows = grouped && g.group_by == FP8Z_GROUP_ROWS, by_k = grouped && !by_rows;
    if (g.m == 0 || g.n == 0) return FP8Z_OK;
    if (!out || (g.k > 0 && (!a || !a_scale || !b || !b_scale)) || (grouped && !offsets)) return FP8Z_EINVAL;
    if (!host::aligned(a_scale, 4) || !host::aligned(b_scale, 4) || !host::aligned(out, dtype_bytes(g.out_dtype)) ||
        (grouped && !host::aligned(offsets, g.offsets_dtype == FP8Z_I64 ? 8 : 4)) || !host::aligned(dev_status, 4) ||
        !host::aligned(workspace, 256))
        return FP8Z_EALIGN;
    const Plan p = plan(a, b, g);
    if (g.k > 0 && p.bytes > 0 && !workspace) return FP8Z_EINVAL;
    if (g.k > 0 && workspace_bytes < p.bytes) return FP8Z_ENOSPACE;
    int sms = 0;
    if (int rc = host::device_sms(&sms)) return rc;
    const auto st = static_cast<cudaStream_t>(stream);
    if (g.k == 0) {
        if (by_rows) return FP8Z_EINVAL;               // a weight without columns
        if (g.accumulate) return FP8Z_OK;
        const dim3 grid(unsigned(std::min<int64_t>(g.m, sms * 8)), 1, unsigned(by_k ? g.groups : 1));
        const auto zero = [&](auto* t) {
            using T = std::remove_pointer_t<decltype(t)>;
            return launch_dependent(&zero_kernel<T>, grid, 256, 0, st, static_cast<T*>(out), g.out_ld, g.out_group, int(g.m), int(g.n));
        };
        if (g.out_dtype == FP8Z_F32) return zero(static_cast<float*>(nullptr));
        if (g.out_dtype == FP8Z_BF16) return zero(static_cast<__nv_bfloat16*>(nullptr));
        return zero(static_cast<__half*>(nullptr));
    }
    const auto copy = [&](const void* src, int64_t ld, int64_t group_ld, int64_t groups, int64_t rows, int64_t to) {
        const int64_t pieces = groups * rows * (p.k_pad / 16);
        return launch_dependent(pad_bytes_kernel, dim3(unsigned(std::min<int64_t>((pieces + 255) / 256, sms * 16))), 256, 0, st,
                                static_cast<const uint8_t*>(src), ld, group_ld, int(rows), int(g.k),
                                static_cast<uint8_t*>(workspace) + to, int(p.k_pad), pieces);
    };
    const int64_t banks = by_rows ? g.groups : 1;
    int64_t a_ld = up(g.a_ld, 16), b_ld = up(g.b_ld, 16), b_group = banks > 1 ? g.b_group : b_ld * g.n;
    if (p.copy_a) {
        if (int rc = copy(a, g.a_ld, 0, 1, g.m, p.a_at)) return rc;
        a = static_cast<uint8_t*>(workspace) + p.a_at;
        a_ld = p.k_pad;
    }
    if (p.copy_b) {
        if (int rc = copy(b, g.b_ld, g.b_group, banks, g.n, p.b_at)) return rc;
        b = static_cast<uint8_t*>(workspace) + p.b_at;
        b_ld = p.k_pad;
        b_group = b_ld * g.n;
    }
    const bool rows_scaled = g.b_scale_rows == 1;
    Args A;
    std::memset(&A, 0, sizeof(A));
    A.m = int(g.m);
    A.n = int(g.n);
    A.kb = int((g.k + kBK - 1) / kBK);
    A.groups = grouped ? g.groups : 1;
    A.by = by_rows ? kByRows : by_k ? kByK : 0;
    A.offsets = offsets;
    A.wide = g.offsets_dtype == FP8Z_I64;
    A.total = int(by_rows ? g.m : g.k);
    A.a_scale = a_scale;
    A.b_scale = b_scale;
    A.a_scale_ld = g.a_scale_ld;
    A.b_scale_ld = g.b_scale_ld;
    A.b_scale_group = by_rows ? g.b_scale_group : 0;
    A.b_scale_last = int(rows_scaled ? g.n - 1 : (g.n - 1) / FP8Z_BLOCK);
    A.out = out;
    A.out_ld = g.out_ld;
    A.out_group = by_k ? g.out_group : 0;
    A.out_dtype = g.out_dtype;
    A.accumulate = g.accumulate;
    A.timeout_ns = host::wait_limit_ns();
    A.dev_status = dev_status;

    const Choice c = choose(g, sms);
    CUtensorMap ta, tb, tc;
    if (!bytes_map(&ta, 2, a, g.k, g.m, 1, a_ld, 0, c.rows ? c.rows : kHalf) ||
        !bytes_map(&tb, 3, b, g.k, g.n, banks, b_ld, b_group, kHalf))
        return FP8Z_ECUDA;
    if (c.rows == 0) {
        A.mt = int((g.m + kTM - 1) / kTM);
        A.nt = int((g.n + kTN - 1) / kTN);
        const int64_t size = dtype_bytes(g.out_dtype);
        // a tile's store writes whole 16 bytes, and what lies behind a row that ends between two is not ours
        A.staged = host::aligned(out, 16) && g.out_ld * size % 16 == 0 && g.n * size % 16 == 0 &&
                   (!by_k || g.groups == 1 || g.out_group * size % 16 == 0);
        if (!A.staged) tc = ta;                        // not used
        else if (!out_map(&tc, g, out)) return FP8Z_ECUDA;
        const int64_t tiles = by_rows ? (g.m / kTM + g.groups) * A.nt : int64_t(A.mt) * A.nt * A.groups;
        return rows_scaled ? launch_large<true>(ta, tb, tc, A, tiles, sms, st) : launch_large<false>(ta, tb, tc, A, tiles, sms, st);
    }
    // groups end inside row tiles: at most one more a group
    A.mt = int(by_rows ? g.m / c.rows + std::min<int64_t>(g.groups, g.m) : (g.m + c.rows - 1) / c.rows);
    const int64_t blocks = int64_t(A.mt) * ((g.n + kRowsB - 1) / kRowsB) * c.splits;
    switch (c.rows) {
        case 16: return launch_small<16>(ta, tb, A, rows_scaled, c.splits, blocks, 19, st);
        case 32: return launch_small<32>(ta, tb, A, rows_scaled, c.splits, blocks, 21, st);
        default: return launch_small<64>(ta, tb, A, rows_scaled, c.splits, blocks, 23, st);
    }
}

}  // namespace
}  // namespace fp8z

extern "C" int64_t fp8z_matmul_workspace(const void* a, const void* b, const fp8z_matmul_args* args) {
    using namespace fp8z;
    if (!args || !args_ok(*args)) return FP8Z_EINVAL;
    return plan(a, b, *args).bytes;
}

extern "C" int fp8z_matmul(const void* a, const float* a_scale, const void* b, const float* b_scale,
                           const fp8z_matmul_args* args, const void* offsets, void* out, void* workspace,
                           int64_t workspace_bytes, int32_t* dev_status, void* stream) {
    const fp8z::host::NvtxRange nvtx_range("fp8z_matmul");
    return fp8z::run(a, a_scale, b, b_scale, args, offsets, out, workspace, workspace_bytes, dev_status, stream);
}
