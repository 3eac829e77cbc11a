// embed.cu -- embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[t] = scale * table[id_t]
//   d_table[v] (+)= scale * sum over {t : id_t = v} of d_out[t],  nothing for padding_idx
//
// The gradient sorts the tokens by id (stable, so equal ids keep token order),
// cuts the sorted list into pieces of equal length, sums each run of equal ids
// inside a piece in registers, and joins the runs that cross pieces.  Every sum
// runs in FP32 in an order that the ids alone give, whatever the schedule, and a
// word that makes up half of a batch costs no more than many rare ones.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "fp8z.h"
#include "fp8z_device.cuh"
#include "fp8z_elem.cuh"
#include "fp8z_host.h"
#include "fp8z_launch.cuh"
#include "fp8z_tiles.h"

namespace fp8z {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t load_id(const void* ids, int wide, int64_t i) {
    return wide ? static_cast<const int64_t*>(ids)[i] : int64_t(static_cast<const int32_t*>(ids)[i]);
}

// ------------------------------------------------------------------ lookup
// One block writes one piece of one row.  VEC: rows of both sides start on
// 16-byte boundaries, eight elements a thread and step; else one element.
template <typename S, typename D, bool VEC>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const void* ids, int wide,
                                                          const S* table, int64_t table_ld,
                                                          int64_t vocab, D* out, int64_t out_ld,
                                                          int hidden, float scale, int32_t* dev_status) {
    constexpr int V = VEC ? 8 : 1, R = 4;
    dependent_wait();
    const int64_t t = blockIdx.x;
    const int64_t id = load_id(ids, wide, t);
    const bool ok = id >= 0 && id < vocab;
    if (!ok && threadIdx.x == 0 && blockIdx.y == 0) report_status(dev_status, FP8Z_EINVAL);
    const S* src = table + (ok ? id : 0) * table_ld;
    D* dst = out + t * out_ld;
    const int c0 = blockIdx.y * (kThreads * V * R) + threadIdx.x * V;
    Pack<S, V> x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = c0 + r * kThreads * V;
        if (c < hidden && ok) {
            if constexpr (VEC) x[r] = ld_nc<S, V>(src + c);
            else x[r].v[0] = src[c];
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = c0 + r * kThreads * V;
        if (c >= hidden) break;
        Pack<D, V> y;
#pragma unroll
        for (int i = 0; i < V; ++i) y.v[i] = Elem<D>::narrow(ok ? Elem<S>::widen(x[r].v[i]) * scale : 0.0f);
        if constexpr (VEC) st_vec<D, V>(dst + c, y);
        else dst[c] = y.v[0];
    }
}

// ------------------------------------------------------------------- sort
// Stable radix sort of (id, token) by digits of up to kMaxDigit bits, one
// block per tile of kTile tokens, or per several neighbouring tiles of a list of more
// than kMostBlocks: count the digits of each block's tokens, then place every token at
// (tokens of smaller digits) + (equal digits of earlier blocks and tiles) + (its rank
// among equal digits of its own tile).  Ids that take no gradient (padding, out of
// range) get the key `vocab`, which sorts last.  Every block walks over the counts of
// all blocks, work that would grow with the square of the tokens (2^24: 275 GB a pass),
// so their number is bounded: 4194304 tokens x 8 take 4.05 ms, with 512 or 128 blocks
// 0.07 more, with 1024 0.66 and with a block for each tile 2.27.
constexpr int kItems = 8;
constexpr int kTile = kThreads * kItems;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDigit = 10;
constexpr int kBins = 1 << kMaxDigit;
constexpr int kMostBlocks = 256;

struct SortShape {
    int bits;        // key bits
    int passes;
    int digit;       // bits per pass
    int tiles;       // of one block
    int blocks;
};

SortShape sort_shape(int64_t tokens, int64_t vocab) {
    SortShape s;
    s.bits = 1;
    while ((int64_t(1) << s.bits) <= vocab) ++s.bits;       // keys 0 .. vocab
    s.passes = (s.bits + kMaxDigit - 1) / kMaxDigit;
    s.digit = (s.bits + s.passes - 1) / s.passes;
    const int64_t tiles = (tokens + kTile - 1) / kTile;
    s.tiles = tiles > kMostBlocks ? int((tiles + kMostBlocks - 1) / kMostBlocks) : 1;
    s.blocks = int((tiles + s.tiles - 1) / s.tiles);
    return s;
}

struct Ids {
    const void* ids;
    int64_t vocab, padding;
    int wide;
    int32_t* dev_status;
    __device__ __forceinline__ uint32_t key(int64_t i, bool report) const {
        const int64_t id = load_id(ids, wide, i);
        if (id == padding && padding >= 0) return uint32_t(vocab);
        if (id < 0 || id >= vocab) {
            if (report) report_status(dev_status, FP8Z_EINVAL);
            return uint32_t(vocab);
        }
        return uint32_t(id);
    }
};

// Rows that no token names are written as zeros, by blocks that run beside the
// sort's and the sums' in the same launches: a launch of the sort takes some 8 us
// on a few SMs, and the rest of the machine writes about kFillBesideSort bytes in
// that time.  Which rows occur is known from `used`, or, where one block sorts
// the whole list, from the ids themselves.
constexpr int kFillRows = 64;           // most rows of one block
constexpr int64_t kFillBytes = 128 << 10;
constexpr int64_t kFillBesideSort = 48 << 20;
struct Fill {
    void* table;
    const uint8_t* used;                         // [vocab], or null
    int64_t ld_bytes, row_bytes, begin, end;     // rows [begin, end) are this launch's
    int rows, blocks;                            // rows of one block
};

__device__ __forceinline__ void fill_rows(const Fill& f, const Ids& ids, int n, int64_t block) {
    __shared__ uint32_t named[kFillRows / 32];
    const int64_t r0 = f.begin + block * f.rows;
    const int rows = int(min(int64_t(f.rows), f.end - r0));
    if (threadIdx.x < kFillRows / 32) named[threadIdx.x] = 0;
    __syncthreads();
    if (f.used) {
        if (int(threadIdx.x) < rows && f.used[r0 + threadIdx.x])
            atomicOr(&named[threadIdx.x >> 5], 1u << (threadIdx.x & 31));
    } else {
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const int64_t r = int64_t(ids.key(i, false)) - r0;
            if (r >= 0 && r < rows) atomicOr(&named[r >> 5], 1u << (r & 31));
        }
    }
    __syncthreads();
    const bool wide = ((reinterpret_cast<uintptr_t>(f.table) | f.ld_bytes | f.row_bytes) & 15) == 0;
    for (int r = 0; r < rows; ++r) {
        if (named[r >> 5] >> (r & 31) & 1) continue;
        uint8_t* p = static_cast<uint8_t*>(f.table) + (r0 + r) * f.ld_bytes;
        if (wide)
            for (int64_t c = threadIdx.x; c < f.row_bytes / 16; c += blockDim.x)
                reinterpret_cast<uint4*>(p)[c] = make_uint4(0, 0, 0, 0);
        else
            for (int64_t c = threadIdx.x; c < f.row_bytes / 2; c += blockDim.x) reinterpret_cast<uint16_t*>(p)[c] = 0;
    }
}

// counts[block * kBins + digit]; the first pass marks the rows that occur
__global__ void __launch_bounds__(kThreads) count_kernel(Ids ids, const uint32_t* keys, int n, int tiles, int shift,
                                                         int digit, uint32_t* counts, Fill fill,
                                                         uint32_t* tickets, int ntickets, uint8_t* used) {
    __shared__ uint32_t bins[kBins];
    dependent_wait();
    const int blocks = gridDim.x - fill.blocks;
    if (int(blockIdx.x) >= blocks) {
        fill_rows(fill, ids, n, blockIdx.x - blocks);
        return;
    }
    if (tickets)
        for (int i = blockIdx.x * kThreads + threadIdx.x; i < ntickets; i += blocks * kThreads) tickets[i] = 0;
    const uint32_t mask = (1u << digit) - 1;
    for (int b = threadIdx.x; b <= int(mask); b += kThreads) bins[b] = 0;
    __syncthreads();
    for (int tile = 0; tile < tiles; ++tile) {
        const int t0 = (blockIdx.x * tiles + tile) * kTile;
#pragma unroll
        for (int r = 0; r < kItems; ++r) {
            const int i = t0 + r * kThreads + threadIdx.x;
            if (i < n) {
                const uint32_t k = keys ? keys[i] : ids.key(i, true);
                atomicAdd(&bins[(k >> shift) & mask], 1u);
                if (used && k < uint32_t(ids.vocab)) used[k] = 1;
            }
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b <= int(mask); b += kThreads) counts[size_t(blockIdx.x) * kBins + b] = bins[b];
}

struct SortShared {
    uint16_t warp_count[kWarps][kBins];      // equal digits in earlier rounds, then in earlier warps
    uint32_t base[kBins];
    uint32_t warp_total[kWarps];
};

// base[b] = tokens of smaller digits anywhere + tokens of digit b in earlier
// blocks, from the block's own sums of (earlier blocks, all blocks) for each bin.
template <typename F>
__device__ __forceinline__ void digit_bases(SortShared& sh, int nb, F sums) {
    constexpr int B = kBins / kThreads;                 // neighbouring bins of one thread
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t mine[B], total[B], sum = 0;
#pragma unroll
    for (int j = 0; j < B; ++j) {
        const int b = threadIdx.x * B + j;
        mine[j] = total[j] = 0;
        if (b < nb) sums(b, mine[j], total[j]);
        sum += total[j];
    }
    uint32_t scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += y;
    }
    if (lane == 31) sh.warp_total[warp] = scan;
    __syncthreads();
    uint32_t before = scan - sum;
    for (int w = 0; w < warp; ++w) before += sh.warp_total[w];
#pragma unroll
    for (int j = 0; j < B; ++j) {
        const int b = threadIdx.x * B + j;
        if (b < nb) sh.base[b] = before + mine[j];
        before += total[j];
    }
}

// Rank of each of the warp's tokens (32 * kItems of them in order, 32 at a time)
// among equal digits of the tile's earlier tokens.  k: keys; rounds < n in use.
__device__ __forceinline__ void tile_ranks(SortShared& sh, const uint32_t (&k)[kItems], uint32_t (&rank)[kItems],
                                           int count, int shift, int nb) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t mask = nb - 1;
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        const bool in = r * 32 + lane < count;
        const uint32_t d = (k[r] >> shift) & mask;
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, in ? d : 0xFFFFFFFFu);
        const int before_me = __popc(peers & ((1u << lane) - 1));
        uint32_t seen = 0;
        if (in) seen = sh.warp_count[warp][d];
        __syncwarp();
        if (in && before_me == 0) sh.warp_count[warp][d] = uint16_t(seen + __popc(peers));
        __syncwarp();
        rank[r] = seen + before_me;
    }
}

// Counts of the tile's warps become the counts of the warps before each; of_tile gets the
// tile's for the digits of this thread, kThreads apart.
__device__ __forceinline__ void warp_bases(SortShared& sh, int nb, uint32_t (&of_tile)[kBins / kThreads]) {
#pragma unroll
    for (int j = 0; j < kBins / kThreads; ++j) {
        const int b = threadIdx.x + j * kThreads;
        uint32_t s = 0;
        if (b < nb)
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const uint32_t c = sh.warp_count[w][b];
                sh.warp_count[w][b] = uint16_t(s);
                s += c;
            }
        of_tile[j] = s;
    }
}

__device__ __forceinline__ void clear_counts(SortShared& sh, int nb) {
    for (int i = threadIdx.x; i < nb * kWarps / 2; i += kThreads) {
        const int w = i / (nb / 2), b = i % (nb / 2);
        reinterpret_cast<uint32_t*>(sh.warp_count[w])[b] = 0;
    }
}

__global__ void __launch_bounds__(kThreads) place_kernel(Ids ids, const uint32_t* keys,
                                                         const uint32_t* vals, int n, int tiles, int shift,
                                                         int digit, const uint32_t* counts, int blocks,
                                                         uint32_t* keys_out,
                                                         uint32_t* vals_out, Fill fill) {
    __shared__ SortShared sh;
    dependent_wait();
    if (int(blockIdx.x) >= blocks) {
        fill_rows(fill, ids, n, blockIdx.x - blocks);
        return;
    }
    const int nb = 1 << digit, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int begin = blockIdx.x * tiles * kTile, first = begin + warp * (32 * kItems) + lane;
    uint32_t k[kItems], v[kItems];
    auto load = [&](int tile) {                        // the first tile's come in while the counts are read
#pragma unroll
        for (int r = 0; r < kItems; ++r) {
            const int i = first + tile * kTile + r * 32;
            const bool in = i < n;
            k[r] = in ? (keys ? keys[i] : ids.key(i, false)) : 0;
            v[r] = in ? (vals ? vals[i] : uint32_t(i)) : 0;
        }
    };
    load(0);
    clear_counts(sh, nb);
    digit_bases(sh, nb, [&](int b, uint32_t& mine, uint32_t& total) {
#pragma unroll 4
        for (int t = 0; t < blocks; ++t) {
            const uint32_t c = counts[size_t(t) * kBins + b];
            if (t < int(blockIdx.x)) mine += c;
            total += c;
        }
    });
    for (int tile = 0; tile < tiles; ++tile) {
        const int start = begin + tile * kTile, t0 = start + warp * (32 * kItems);
        uint32_t rank[kItems];
        tile_ranks(sh, k, rank, n - t0, shift, nb);
        __syncthreads();
        uint32_t of_tile[kBins / kThreads];            // tokens of this thread's digits
        warp_bases(sh, nb, of_tile);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kItems; ++r) {
            if (t0 + r * 32 + lane < n) {
                const uint32_t d = (k[r] >> shift) & (nb - 1);
                const uint32_t at = sh.base[d] + sh.warp_count[warp][d] + rank[r];
                keys_out[at] = k[r];
                vals_out[at] = v[r];
            }
        }
        if (tile + 1 == tiles || start + kTile >= n) break;
        load(tile + 1);
        __syncthreads();                               // the bases and counts have been read
#pragma unroll
        for (int j = 0; j < kBins / kThreads; ++j)
            if (int(threadIdx.x) + j * kThreads < nb) sh.base[threadIdx.x + j * kThreads] += of_tile[j];
        clear_counts(sh, nb);
        __syncthreads();
    }
}

// Up to kRankMost tokens: a token's place is the number of keys before its own,
// all of them compared from shared memory, a warp a token.  One launch instead of
// four or six, but tokens squared comparisons: the whole gradient of 4000 tokens
// x 1024 takes 22 us this way and about 35 by digits, of 8000 59 and 37.
constexpr int kRankTokens = 32;                        // of one block
constexpr int kRankMost = 4096, kRankScan = 512;       // up to kRankScan all fills look the rows up in the ids
__global__ void __launch_bounds__(kThreads) rank_kernel(Ids ids, int n, uint32_t* keys_out, uint32_t* vals_out, Fill fill,
                                                        uint32_t* tickets, int ntickets, uint8_t* used) {
    __shared__ uint32_t keys[kRankMost];
    dependent_wait();
    const int blocks = gridDim.x - fill.blocks;
    if (int(blockIdx.x) >= blocks) {
        fill_rows(fill, ids, n, blockIdx.x - blocks);
        return;
    }
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < ntickets; i += blocks * kThreads) tickets[i] = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        keys[i] = ids.key(i, blockIdx.x == 0);
        if (used && blockIdx.x == 0 && keys[i] < uint32_t(ids.vocab)) used[keys[i]] = 1;
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int T = kRankTokens / kWarps;
    const int i0 = blockIdx.x * kRankTokens + warp * T;
    uint32_t k[T];
    int before[T] = {};
#pragma unroll
    for (int t = 0; t < T; ++t) k[t] = i0 + t < n ? keys[i0 + t] : 0;
    for (int j = lane; j < n; j += 32) {
        const uint32_t q = keys[j];
#pragma unroll
        for (int t = 0; t < T; ++t) before[t] += q < k[t] || (q == k[t] && j < i0 + t);
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int at = __reduce_add_sync(0xFFFFFFFFu, before[t]);
        if (lane == 0 && i0 + t < n) {
            keys_out[at] = k[t];
            vals_out[at] = uint32_t(i0 + t);
        }
    }
}

// -------------------------------------------------------------------- sums
constexpr int kMaxPiece = 32, kGroup = 32;
// Columns one block takes: eight neighbours a thread, or, where rows start between
// 16-byte boundaries, four single ones a block apart (with one, 16384 x 1001 took 55 us
// for 47 and 5719 x 3031 67 for 46; one and 16 rows under way 60 and 88).
template <bool VEC>
constexpr int kCols = kThreads * (VEC ? 8 : 4);

// Adds to or writes V neighbouring elements.  FP32 sums are added by the memory
// system: one addition for each element of the call, in no race with another, and no
// thread waits for the old value (added up by the threads, 65536 x 1024 takes 156 us for
// 101, 16384 x 7168 177 for 143).  It takes subnormal numbers for zero.
template <typename D, int V>
__device__ __forceinline__ void write_row(D* p, const float (&acc)[V], float scale, bool accumulate) {
    if constexpr (std::is_same_v<D, float>) {
        if (accumulate) {
            if constexpr (V > 1) {
#pragma unroll
                for (int i = 0; i < V; i += 4)
                    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p + i), "f"(acc[i] * scale),
                                 "f"(acc[i + 1] * scale), "f"(acc[i + 2] * scale), "f"(acc[i + 3] * scale)
                                 : "memory");
            } else {
                asm volatile("red.global.add.f32 [%0], %1;" ::"l"(p), "f"(acc[0] * scale) : "memory");
            }
            return;
        }
    }
    Pack<D, V> y;
    if (accumulate) {
        if constexpr (V > 1) y = ld_plain<D, V>(p);
        else y.v[0] = *p;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float s = acc[i] * scale;
        y.v[i] = Elem<D>::narrow(accumulate ? Elem<D>::widen(y.v[i]) + s : s);
    }
    if constexpr (V > 1) st_vec<D, V>(p, y);
    else *p = y.v[0];
}

// One block sums the runs of one piece of the sorted list, in its columns.  A run
// inside its piece is finished there.  A longer one leaves a partial sum for each
// of its pieces (partial[2 * piece] for one that came in from the piece before,
// partial[2 * piece + 1] for one that starts there), and the last of its blocks to
// arrive adds them up.  Over more than kGroup pieces the last block of each kGroup
// neighbours adds theirs up, and the last of these the groups' sums.  Both go in the
// list's order, and which way is taken depends on the ids alone.  65536 tokens x 1024
// over 4096 words take 114 us, with one word for half of them 109, for all 117 (a block
// that adds up all of a run alone made the half 272); at three blocks an SM, which four
// would spill registers for (16384 x 7168: 358 us for 340).
template <typename S, typename D, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) runs_kernel(const uint32_t* keys,
                                                        const uint32_t* vals, int n, uint32_t vocab,
                                                        int piece_len, const S* d_out, int64_t d_ld,
                                                        D* d_table, int64_t t_ld, int hidden, float scale,
                                                        bool accumulate, float* partial, uint32_t* tickets,
                                                        int slabs, Ids ids, Fill fill) {
    constexpr int V = VEC ? 8 : 4, kStep = VEC ? 1 : kThreads;       // columns of a thread, and from one to the next
    __shared__ bool finish;
    __shared__ uint32_t skeys[kMaxPiece], svals[kMaxPiece];
    dependent_wait();
    // sums and fills take turns, so that the machine always has some of both
    const int64_t sums = int64_t(gridDim.x) - fill.blocks, b = blockIdx.x;
    const int64_t sum = b * sums / gridDim.x;
    if ((b + 1) * sums / gridDim.x == sum) {
        fill_rows(fill, ids, n, b - sum);
        return;
    }
    const int piece = int(sum / slabs), slab = int(sum % slabs);
    const int col = slab * kCols<VEC> + threadIdx.x * (VEC ? V : 1);
    const bool mine = col < hidden;
    auto has = [&](int j) { return col + j * kStep < hidden; };
    auto write = [&](uint32_t to, const float (&v)[V]) {
        D* p = d_table + int64_t(to) * t_ld + col;
        if constexpr (VEC) {
            if (mine) write_row<D, V>(p, v, scale, accumulate);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float one[1] = {v[j]};
                if (has(j)) write_row<D, 1>(p + j * kStep, one, scale, accumulate);
            }
        }
    };
    const int i0 = piece * piece_len, i1 = min(n, i0 + piece_len);
    if (i0 + int(threadIdx.x) < i1) {
        skeys[threadIdx.x] = keys[i0 + threadIdx.x];
        svals[threadIdx.x] = vals[i0 + threadIdx.x];
    }
    const uint32_t key_before = i0 > 0 ? keys[i0 - 1] : vocab, key_after = i1 < n ? keys[i1] : vocab;
    __syncthreads();
    uint32_t key = skeys[0];
    if (key >= vocab) return;                       // the ids without a gradient come last
    float acc[V] = {};

    // Leaves this piece's part of a run over several pieces.
    auto part_of_run = [&](bool from_before) {
        if (mine) {
            float* p = partial + size_t(2 * piece + (from_before ? 0 : 1)) * hidden + col;
            if constexpr (VEC) {
                __stcg(reinterpret_cast<float4*>(p), make_float4(acc[0], acc[1], acc[2], acc[3]));
                __stcg(reinterpret_cast<float4*>(p) + 1, make_float4(acc[4], acc[5], acc[6], acc[7]));
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (has(j)) __stcg(p + j * kStep, acc[j]);
            }
        }
        // the run's first and last piece: the keys are sorted, so a border of pieces inside the
        // run is one with its key on the other side
        const int lane = threadIdx.x & 31;
        const int last = piece + run_length((n - 1) / piece_len - piece, [&](int from, int step, int end) {
            const int q = from + step * lane;
            return __popc(__ballot_sync(0xFFFFFFFFu, q < end && keys[(piece + q) * piece_len] == key));
        });
        const int first = piece - run_length(piece, [&](int from, int step, int end) {
            const int q = from + step * lane;
            return __popc(__ballot_sync(0xFFFFFFFFu, q < end && keys[(piece - q + 1) * piece_len - 1] == key));
        });
        // whether this block is the last of `others` + 1 to arrive at a ticket
        auto arrive = [&](uint32_t* ticket, int others) {
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) finish = atomicAdd(ticket, 1u) == uint32_t(others);
            __syncthreads();
            const bool last_one = finish;
            __syncthreads();                        // `finish` is free again
            __threadfence();
            return last_one;
        };
        auto slot = [&](int q) { return partial + size_t(2 * q + (q == first ? 1 : 0)) * hidden + col; };
        auto add = [&](const float* p) {
            if constexpr (VEC) {
                const float4 a = __ldcg(reinterpret_cast<const float4*>(p));
                const float4 b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
                acc[0] += a.x, acc[1] += a.y, acc[2] += a.z, acc[3] += a.w;
                acc[4] += b.x, acc[5] += b.y, acc[6] += b.z, acc[7] += b.w;
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (has(j)) acc[j] += __ldcg(p + j * kStep);
            }
        };
        const int group = piece / kGroup;
        const bool one_level = last - first < kGroup;
        const int q0 = one_level ? first : max(first, group * kGroup);
        const int q1 = one_level ? last : min(last, group * kGroup + kGroup - 1);
        // (a piece may end one run and start the next: as for the sums, each has its own ticket)
        if (!arrive(&tickets[size_t(3 * q0 + (q0 == first ? 1 : 0)) * slabs + slab], q1 - q0)) return;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = 0.0f;
        if (mine)
#pragma unroll 4
            for (int q = q0; q <= q1; ++q) add(slot(q));
        if (!one_level) {
            if (mine)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (has(j)) __stcg(slot(q0) + j * kStep, acc[j]);
            const int g0 = first / kGroup, g1 = last / kGroup;
            if (!arrive(&tickets[size_t(3 * first + 2) * slabs + slab], g1 - g0)) return;
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = 0.0f;
            if (mine)
#pragma unroll 4
                for (int g = g0; g <= g1; ++g) add(slot(max(first, g * kGroup)));
        }
        write(key, acc);
    };

    // Adds rows [i, end) to acc; where the key changes, finishes the run before.
    auto add_rows = [&](int i, int end) {
        constexpr int U = 4;                          // eight rows under way take 128 registers: 381 us for 345
        for (; i < end; i += U) {
            Pack<S, V> x[U];
            uint32_t k[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                k[u] = i + u < end ? skeys[i + u - i0] : vocab;
                if (k[u] < vocab && mine) {
                    const S* p = d_out + int64_t(svals[i + u - i0]) * d_ld + col;
                    if constexpr (VEC) x[u] = ld_nc<S, V>(p);
                    else
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            if (has(j)) x[u].v[j] = p[j * kStep];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i + u >= end) break;
                if (k[u] != key) {
                    write(key, acc);
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[j] = 0.0f;
                    key = k[u];
                    if (key >= vocab) return;
                }
                if (mine) {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (VEC || has(j)) acc[j] += Elem<S>::widen(x[u].v[j]);
                }
            }
        }
    };

    // first the run that comes in from the piece before, if one does, then the rest
    // (one copy of the code for both: with two, 65536 x 1024 took 125 us for 115)
    bool from_before = key_before == key;
    for (int i = i0, end; i < i1; i = end, from_before = false) {
        end = i1;
        if (from_before)
            for (end = i + 1; end < i1 && skeys[end - i0] == key;) ++end;
        if (i > i0) {
            key = skeys[i - i0];
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = 0.0f;
        }
        if (key < vocab) add_rows(i, end);
        if (key >= vocab) return;
        if (from_before || key_after == key) part_of_run(from_before);
        else write(key, acc);
    }
}

// ----------------------------------------------------------------- launches
struct GradLayout {
    SortShape sort;
    int piece_len, pieces;
    size_t keys, vals, counts, partial, tickets, used, total;      // byte offsets (two key and two value buffers)
};

// Pieces of 32 tokens, shorter while there are too few for the machine: a
// piece's partial rows cost 2 * hidden * 4 bytes against 32 rows read.
GradLayout grad_layout(int64_t tokens, int64_t vocab, int64_t hidden) {
    GradLayout g;
    g.sort = sort_shape(tokens, vocab);
    g.piece_len = tokens >= 8192 ? kMaxPiece : tokens >= 2048 ? 16 : 8;
    g.pieces = int((tokens + g.piece_len - 1) / g.piece_len);
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    size_t at = 0;
    g.keys = at;
    at += 2 * up(size_t(tokens) * 4);
    g.vals = at;
    at += 2 * up(size_t(tokens) * 4);
    g.counts = at;
    at += up(size_t(g.sort.blocks) * kBins * 4);
    g.partial = at;
    at += up(size_t(g.pieces) * 2 * size_t(hidden) * 4);
    g.tickets = at;                 // three for each piece and block of columns, of four elements a thread at least
    at += up(3 * size_t(g.pieces) * size_t((hidden + kCols<false> - 1) / kCols<false>) * 4);
    g.used = at;
    at += tokens > kRankScan ? up(size_t(vocab)) : 0;
    g.total = at > 0 ? at : 256;    // never an empty buffer, which has no address
    return g;
}

template <typename S, typename D>
int run_lookup(const void* ids, int wide, int64_t tokens, const S* table, int64_t table_ld, int64_t vocab, D* out,
               int64_t out_ld, int64_t hidden, float scale, int32_t* dev_status, cudaStream_t st) {
    const bool vec = hidden % 8 == 0 && (table_ld * sizeof(S)) % 16 == 0 && (out_ld * sizeof(D)) % 16 == 0 &&
                     host::aligned(table, 16) && host::aligned(out, 16);
    const int per = kThreads * 4 * (vec ? 8 : 1);
    const dim3 grid(unsigned(tokens), unsigned((hidden + per - 1) / per));
    const auto kernel = vec ? &lookup_kernel<S, D, true> : &lookup_kernel<S, D, false>;
    return launch_dependent(kernel, grid, kThreads, 0, st, ids, wide, table, table_ld, vocab, out, out_ld, int(hidden),
                            scale, dev_status);
}

template <typename S, typename D>
int run_grad(const Ids& ids, int64_t tokens, const S* d_out, int64_t d_ld, D* d_table, int64_t t_ld, int64_t hidden,
             float scale, bool accumulate, uint8_t* ws, cudaStream_t st) {
    const GradLayout g = grad_layout(tokens, ids.vocab, hidden);
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(ws + g.keys),
                         reinterpret_cast<uint32_t*>(ws + g.keys + up(size_t(tokens) * 4))};
    uint32_t* vals[2] = {reinterpret_cast<uint32_t*>(ws + g.vals),
                         reinterpret_cast<uint32_t*>(ws + g.vals + up(size_t(tokens) * 4))};
    auto* counts = reinterpret_cast<uint32_t*>(ws + g.counts);
    auto* partial = reinterpret_cast<float*>(ws + g.partial);
    auto* tickets = reinterpret_cast<uint32_t*>(ws + g.tickets);
    const int n = int(tokens);
    const bool vec = hidden % 8 == 0 && (d_ld * sizeof(S)) % 16 == 0 && (t_ld * sizeof(D)) % 16 == 0 &&
                     host::aligned(d_out, 16) && host::aligned(d_table, 16);
    const int cols = vec ? kCols<true> : kCols<false>, slabs = int((hidden + cols - 1) / cols);
    const bool one = n <= kRankMost;
    uint8_t* used = accumulate || n <= kRankScan ? nullptr : ws + g.used;
    const int64_t row_bytes = hidden * int64_t(sizeof(D));
    int64_t filled = accumulate ? ids.vocab : 0;
    auto next_fill = [&](int64_t bytes) {               // the next rows, about so many bytes of them
        Fill f = {};
        f.table = d_table;
        f.used = used;
        f.ld_bytes = t_ld * int64_t(sizeof(D));
        f.row_bytes = row_bytes;
        f.begin = filled;
        f.end = filled = std::min<int64_t>(ids.vocab, filled + (bytes + row_bytes - 1) / row_bytes);
        f.rows = int(std::min<int64_t>(kFillRows, std::max<int64_t>(1, kFillBytes / row_bytes)));
        f.blocks = int((f.end - f.begin + f.rows - 1) / f.rows);
        return f;
    };
    const int64_t all = ids.vocab * row_bytes;
    const uint32_t *k = keys[0], *v = vals[0];
    if (used && cudaMemsetAsync(used, 0, size_t(ids.vocab), st) != cudaSuccess) return FP8Z_ECUDA;
    if (n > 0 && one) {
        Fill f = next_fill(kFillBesideSort);
        f.used = nullptr;                               // not known yet: the ids tell which rows occur
        const int blocks = (n + kRankTokens - 1) / kRankTokens;
        if (int rc = launch_dependent(rank_kernel, dim3(unsigned(blocks + f.blocks)), kThreads, 0, st, ids, n, keys[0],
                                      vals[0], f, tickets, 3 * g.pieces * slabs, used))
            return rc;
    } else if (n > 0) {
        for (int p = 0; p < g.sort.passes; ++p) {
            const uint32_t* kin = p ? keys[(p - 1) & 1] : nullptr;
            const uint32_t* vin = p ? vals[(p - 1) & 1] : nullptr;
            Fill f = next_fill(p ? kFillBesideSort : 0);         // the first launch finds out which rows occur
            if (int rc = launch_dependent(count_kernel, dim3(unsigned(g.sort.blocks + f.blocks)), kThreads, 0, st, ids,
                                          kin, n, g.sort.tiles, p * g.sort.digit, g.sort.digit, counts, f, p ? nullptr : tickets,
                                          3 * g.pieces * slabs, p ? nullptr : used))
                return rc;
            f = next_fill(kFillBesideSort);
            if (int rc = launch_dependent(place_kernel, dim3(unsigned(g.sort.blocks + f.blocks)), kThreads, 0, st, ids,
                                          kin, vin, n, g.sort.tiles, p * g.sort.digit, g.sort.digit, counts, g.sort.blocks,
                                          keys[p & 1], vals[p & 1], f))
                return rc;
        }
        k = keys[(g.sort.passes - 1) & 1];
        v = vals[(g.sort.passes - 1) & 1];
    }
    const Fill f = next_fill(all);
    const int64_t blocks = int64_t(g.pieces) * slabs + f.blocks;
    if (blocks == 0) return FP8Z_OK;
    const auto kernel = vec ? &runs_kernel<S, D, true> : &runs_kernel<S, D, false>;
    return launch_dependent(kernel, dim3(unsigned(blocks)), kThreads, 0, st, k, v, n, uint32_t(ids.vocab), g.piece_len,
                            d_out, d_ld, d_table, t_ld, int(hidden), scale, accumulate, partial, tickets, slabs, ids, f);
}

bool shape_ok(int64_t tokens, int64_t vocab, int64_t hidden) {
    return tokens >= 0 && tokens <= (1LL << 30) && vocab >= 1 && vocab <= (1LL << 30) && hidden >= 1 &&
           hidden <= (1LL << 23);
}

// Calls f(S*, D*) with null pointers of the two element types.
template <typename F>
int by_dtypes(int32_t s, int32_t d, F f) {
    auto inner = [&](auto* sp) {
        if (d == FP8Z_F32) return f(sp, static_cast<float*>(nullptr));
        if (d == FP8Z_BF16) return f(sp, static_cast<__nv_bfloat16*>(nullptr));
        return f(sp, static_cast<__half*>(nullptr));
    };
    if (s == FP8Z_F32) return inner(static_cast<float*>(nullptr));
    if (s == FP8Z_BF16) return inner(static_cast<__nv_bfloat16*>(nullptr));
    return inner(static_cast<__half*>(nullptr));
}

}  // namespace
}  // namespace fp8z

extern "C" int fp8z_embedding(const void* ids, int32_t ids_dtype, int64_t tokens, const void* table, int32_t table_dtype,
                              int64_t vocab, int64_t hidden, int64_t table_ld, void* out, int32_t out_dtype,
                              int64_t out_ld, float scale, int32_t* dev_status, void* stream) {
    using namespace fp8z;
    const host::NvtxRange nvtx_range("fp8z_embedding");
    if (!shape_ok(tokens, vocab, hidden) || !dtype_ok(table_dtype) || !dtype_ok(out_dtype) ||
        (ids_dtype != FP8Z_I32 && ids_dtype != FP8Z_I64) || table_ld < hidden || out_ld < hidden || !std::isfinite(scale))
        return FP8Z_EINVAL;
    if (tokens == 0) return FP8Z_OK;
    if (!ids || !table || !out) return FP8Z_EINVAL;
    if (!host::aligned(ids, ids_dtype == FP8Z_I64 ? 8 : 4) || !host::aligned(table, dtype_bytes(table_dtype)) ||
        !host::aligned(out, dtype_bytes(out_dtype)) || !host::aligned(dev_status, 4))
        return FP8Z_EALIGN;
    int sms = 0;
    if (int rc = host::device_sms(&sms)) return rc;
    return by_dtypes(table_dtype, out_dtype, [&](auto* s, auto* d) {
        using S = std::remove_pointer_t<decltype(s)>;
        using D = std::remove_pointer_t<decltype(d)>;
        return run_lookup<S, D>(ids, ids_dtype == FP8Z_I64, tokens, static_cast<const S*>(table), table_ld, vocab,
                                static_cast<D*>(out), out_ld, hidden, scale, dev_status,
                                static_cast<cudaStream_t>(stream));
    });
}

extern "C" int64_t fp8z_embedding_grad_workspace(int64_t tokens, int64_t vocab, int64_t hidden) {
    if (!fp8z::shape_ok(tokens, vocab, hidden)) return FP8Z_EINVAL;
    return int64_t(fp8z::grad_layout(tokens, vocab, hidden).total);
}

extern "C" int fp8z_embedding_grad(const void* ids, int32_t ids_dtype, int64_t tokens, const void* d_out,
                                   int32_t d_dtype, int64_t d_ld, void* d_table, int32_t table_dtype, int64_t vocab,
                                   int64_t hidden, int64_t table_ld, float scale, int64_t padding_idx,
                                   int32_t accumulate, void* workspace, int64_t workspace_bytes, int32_t* dev_status,
                                   void* stream) {
    using namespace fp8z;
    const host::NvtxRange nvtx_range("fp8z_embedding_grad");
    if (!shape_ok(tokens, vocab, hidden) || !dtype_ok(d_dtype) || !dtype_ok(table_dtype) ||
        (ids_dtype != FP8Z_I32 && ids_dtype != FP8Z_I64) || d_ld < hidden || table_ld < hidden || !std::isfinite(scale) ||
        (accumulate != 0 && accumulate != 1))
        return FP8Z_EINVAL;
    if (!d_table || !workspace || (tokens > 0 && (!ids || !d_out))) return FP8Z_EINVAL;
    if (!host::aligned(ids, ids_dtype == FP8Z_I64 ? 8 : 4) || !host::aligned(d_out, dtype_bytes(d_dtype)) ||
        !host::aligned(d_table, dtype_bytes(table_dtype)) || !host::aligned(workspace, 16) ||
        !host::aligned(dev_status, 4))
        return FP8Z_EALIGN;
    if (workspace_bytes < fp8z_embedding_grad_workspace(tokens, vocab, hidden)) return FP8Z_ENOSPACE;
    // a block for each piece and slab of columns, four columns a thread at the least
    if (int64_t(grad_layout(tokens, vocab, hidden).pieces) * ((hidden + kCols<false> - 1) / kCols<false>) > (1 << 29))
        return FP8Z_EINVAL;
    if (tokens == 0 && accumulate) return FP8Z_OK;
    int sms = 0;
    if (int rc = host::device_sms(&sms)) return rc;
    const Ids id = {ids, vocab, padding_idx, ids_dtype == FP8Z_I64 ? 1 : 0, dev_status};
    return by_dtypes(d_dtype, table_dtype, [&](auto* s, auto* d) {
        using S = std::remove_pointer_t<decltype(s)>;
        using D = std::remove_pointer_t<decltype(d)>;
        return run_grad<S, D>(id, tokens, static_cast<const S*>(d_out), d_ld, static_cast<D*>(d_table), table_ld,
                              hidden, scale, accumulate != 0, static_cast<uint8_t*>(workspace),
                              static_cast<cudaStream_t>(stream));
    });
}
