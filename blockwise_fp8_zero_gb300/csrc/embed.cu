// embed.cu -- embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[t] = scale * table[id_t]
//   d_table[v] (+)= scale * sum over {t : id_t = v} of d_out[t],  nothing for padding_idx
//
// The gradient sorts the tokens by id (stable, so equal ids keep token order),
// cuts the sorted list into pieces of equal length, sums each run of equal ids
// inside a piece in registers, and joins the runs that cross pieces in a second
// pass.  Every sum runs in FP32 in token order, whatever the schedule, and a
// word that makes up most of a batch costs no more than many rare ones.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "fp8z.h"
#include "fp8z_device.cuh"
#include "fp8z_elem.cuh"
#include "fp8z_host.h"

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
__global__ void __launch_bounds__(kThreads) lookup_kernel(const void* __restrict__ ids, int wide,
                                                          const S* __restrict__ table, int64_t table_ld,
                                                          int64_t vocab, D* __restrict__ out, int64_t out_ld,
                                                          int hidden, float scale, int32_t* dev_status) {
    constexpr int V = VEC ? 8 : 1, R = 4;
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
// block per tile of kTile tokens: count the digits of each tile, then place
// every token at (tokens of smaller digits) + (equal digits of earlier tiles)
// + (its rank among equal digits of its own tile).  Ids that take no gradient
// (padding, out of range) get the key `vocab`, which sorts last.
constexpr int kItems = 8;
constexpr int kTile = kThreads * kItems;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDigit = 10;
constexpr int kBins = 1 << kMaxDigit;

struct SortShape {
    int bits;        // key bits
    int passes;
    int digit;       // bits per pass
    int tiles;
};

SortShape sort_shape(int64_t tokens, int64_t vocab) {
    SortShape s;
    s.bits = 1;
    while ((int64_t(1) << s.bits) <= vocab) ++s.bits;       // keys 0 .. vocab
    s.passes = (s.bits + kMaxDigit - 1) / kMaxDigit;
    s.digit = (s.bits + s.passes - 1) / s.passes;
    s.tiles = int((tokens + kTile - 1) / kTile);
    return s;
}

struct Ids {
    const void* ids;
    int64_t vocab, padding;
    int wide;
    int32_t* dev_status;
    __device__ __forceinline__ uint32_t key(int64_t i, bool report) const {
        const int64_t id = load_id(ids, wide, i);
        if (id == padding) return uint32_t(vocab);
        if (id < 0 || id >= vocab) {
            if (report) report_status(dev_status, FP8Z_EINVAL);
            return uint32_t(vocab);
        }
        return uint32_t(id);
    }
};

// counts[tile * kBins + digit]; the first pass also marks the rows that occur.
__global__ void __launch_bounds__(kThreads) count_kernel(Ids ids, const uint32_t* __restrict__ keys, int n, int shift,
                                                         int digit, uint32_t* __restrict__ counts,
                                                         uint8_t* __restrict__ used) {
    __shared__ uint32_t bins[kBins];
    const uint32_t mask = (1u << digit) - 1;
    for (int b = threadIdx.x; b <= int(mask); b += kThreads) bins[b] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * kTile;
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        const int i = t0 + r * kThreads + threadIdx.x;
        if (i < n) {
            const uint32_t k = keys ? keys[i] : ids.key(i, true);
            atomicAdd(&bins[(k >> shift) & mask], 1u);
            if (used && k < uint32_t(ids.vocab)) used[k] = 1;
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b <= int(mask); b += kThreads) counts[size_t(blockIdx.x) * kBins + b] = bins[b];
}

__global__ void __launch_bounds__(kThreads) place_kernel(Ids ids, const uint32_t* __restrict__ keys,
                                                         const uint32_t* __restrict__ vals, int n, int shift,
                                                         int digit, const uint32_t* __restrict__ counts, int tiles,
                                                         uint32_t* __restrict__ keys_out,
                                                         uint32_t* __restrict__ vals_out) {
    __shared__ uint16_t warp_count[kWarps][kBins];      // equal digits in earlier rounds, then in earlier warps
    __shared__ uint32_t base[kBins];
    __shared__ uint32_t warp_total[kWarps];
    const int nb = 1 << digit, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t mask = nb - 1;
    for (int b = threadIdx.x; b < nb; b += kThreads)
#pragma unroll
        for (int w = 0; w < kWarps; ++w) warp_count[w][b] = 0;
    // base[b] = tokens of smaller digits anywhere + tokens of digit b in earlier tiles
    constexpr int B = kBins / kThreads;                 // neighbouring bins of one thread
    uint32_t mine[B], total[B], sum = 0;
#pragma unroll
    for (int j = 0; j < B; ++j) {
        const int b = threadIdx.x * B + j;
        mine[j] = total[j] = 0;
        if (b < nb)
            for (int t = 0; t < tiles; ++t) {
                const uint32_t c = counts[size_t(t) * kBins + b];
                if (t < int(blockIdx.x)) mine[j] += c;
                total[j] += c;
            }
        sum += total[j];
    }
    uint32_t scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += y;
    }
    if (lane == 31) warp_total[warp] = scan;
    __syncthreads();
    uint32_t before = scan - sum;
    for (int w = 0; w < warp; ++w) before += warp_total[w];
#pragma unroll
    for (int j = 0; j < B; ++j) {
        const int b = threadIdx.x * B + j;
        if (b < nb) base[b] = before + mine[j];
        before += total[j];
    }
    // rank inside the tile: a warp owns 256 consecutive tokens, 32 at a time in order
    const int t0 = blockIdx.x * kTile + warp * (32 * kItems);
    uint32_t k[kItems], v[kItems], rank[kItems];
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        const int i = t0 + r * 32 + lane;
        const bool in = i < n;
        k[r] = in ? (keys ? keys[i] : ids.key(i, false)) : 0;
        v[r] = in ? (vals ? vals[i] : uint32_t(i)) : 0;
    }
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        const bool in = t0 + r * 32 + lane < n;
        const uint32_t d = (k[r] >> shift) & mask;
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, in ? d : 0xFFFFFFFFu);
        const int before_me = __popc(peers & ((1u << lane) - 1));
        uint32_t seen = 0;
        if (in) seen = warp_count[warp][d];
        __syncwarp();
        if (in && before_me == 0) warp_count[warp][d] = uint16_t(seen + __popc(peers));
        __syncwarp();
        rank[r] = seen + before_me;
    }
    __syncthreads();
    for (int b = threadIdx.x; b < nb; b += kThreads) {
        uint32_t s = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t c = warp_count[w][b];
            warp_count[w][b] = uint16_t(s);
            s += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        if (t0 + r * 32 + lane < n) {
            const uint32_t d = (k[r] >> shift) & mask;
            const uint32_t at = base[d] + warp_count[warp][d] + rank[r];
            keys_out[at] = k[r];
            vals_out[at] = v[r];
        }
    }
}

// -------------------------------------------------------------------- sums
// Columns one block takes: V per thread.
template <bool VEC>
constexpr int kCols = kThreads * (VEC ? 8 : 1);

template <typename D, int V>
__device__ __forceinline__ void write_row(D* p, const float (&acc)[V], float scale, bool accumulate) {
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

// Blocks [0, pieces) x slabs sum the runs of one piece of the sorted list;
// blocks beyond write zeros to the rows that do not occur.  A run inside its
// piece is finished here.  One that came in from the piece before leaves its
// part in partial[2 * piece], one that starts here and goes on in
// partial[2 * piece + 1]; join_kernel adds them.
template <typename S, typename D, bool VEC>
__global__ void __launch_bounds__(kThreads) runs_kernel(const uint32_t* __restrict__ keys,
                                                        const uint32_t* __restrict__ vals, int n, uint32_t vocab,
                                                        int piece_len, int pieces, const S* __restrict__ d_out,
                                                        int64_t d_ld, D* __restrict__ d_table, int64_t t_ld, int hidden,
                                                        float scale, bool accumulate, float* __restrict__ partial,
                                                        const uint8_t* __restrict__ used, int fill_rows) {
    constexpr int V = VEC ? 8 : 1;
    const int col = blockIdx.y * kCols<VEC> + threadIdx.x * V;
    if (col >= hidden) return;
    if (int(blockIdx.x) >= pieces) {
        const int64_t r0 = int64_t(blockIdx.x - pieces) * fill_rows;
        const float zero[V] = {};
        for (int r = 0; r < fill_rows; ++r)
            if (r0 + r < vocab && !used[r0 + r]) write_row<D, V>(d_table + (r0 + r) * t_ld + col, zero, 0.0f, false);
        return;
    }
    const int i0 = blockIdx.x * piece_len, i1 = min(n, i0 + piece_len);
    uint32_t key = keys[i0];
    if (key >= vocab) return;                       // the ids without a gradient come last
    bool from_before = i0 > 0 && keys[i0 - 1] == key;
    float acc[V] = {};
    constexpr int U = 4;
    for (int i = i0; i < i1; i += U) {
        Pack<S, V> x[U];
        uint32_t k[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            k[u] = i + u < i1 ? keys[i + u] : vocab;
            if (k[u] < vocab) {
                const S* p = d_out + int64_t(vals[i + u]) * d_ld + col;
                if constexpr (VEC) x[u] = ld_nc<S, V>(p);
                else x[u].v[0] = *p;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u >= i1) break;
            if (k[u] != key) {                      // the run ends inside the piece
                if (from_before) {
#pragma unroll
                    for (int j = 0; j < V; ++j) partial[size_t(2 * blockIdx.x) * hidden + col + j] = acc[j];
                } else {
                    write_row<D, V>(d_table + int64_t(key) * t_ld + col, acc, scale, accumulate);
                }
                from_before = false;
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] = 0.0f;
                key = k[u];
                if (key >= vocab) return;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] += Elem<S>::widen(x[u].v[j]);
        }
    }
    const bool goes_on = i1 < n && keys[i1] == key;
    if (from_before || goes_on) {
        float* p = partial + size_t(2 * blockIdx.x + (from_before ? 0 : 1)) * hidden + col;
#pragma unroll
        for (int j = 0; j < V; ++j) p[j] = acc[j];
    } else {
        write_row<D, V>(d_table + int64_t(key) * t_ld + col, acc, scale, accumulate);
    }
}

template <typename D>
__global__ void __launch_bounds__(kThreads) join_kernel(const uint32_t* __restrict__ keys, int n, uint32_t vocab,
                                                        int piece_len, const float* __restrict__ partial,
                                                        D* __restrict__ d_table, int64_t t_ld, int hidden, float scale,
                                                        bool accumulate) {
    const int p = blockIdx.x, i0 = p * piece_len, i1 = min(n, i0 + piece_len);
    const uint32_t key = keys[i1 - 1];
    if (key >= vocab || i1 >= n || keys[i1] != key) return;     // no run goes on
    if (i0 > 0 && keys[i0 - 1] == key && keys[i0] == key) return;   // it began in an earlier piece
    // the run's end: doubling steps from i1, then halving
    int lo = i1, step = 1;
    while (lo + step < n && keys[lo + step] == key) {
        lo += step;
        step *= 2;
    }
    int hi = min(n, lo + step);                                 // keys[lo] == key, keys[hi] != key or hi == n
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (keys[mid] == key) lo = mid; else hi = mid;
    }
    const int last = lo / piece_len;
    const int col = blockIdx.y * kThreads + threadIdx.x;
    if (col >= hidden) return;
    float acc[1] = {partial[size_t(2 * p + 1) * hidden + col]};
#pragma unroll 8
    for (int q = p + 1; q <= last; ++q) acc[0] += partial[size_t(2 * q) * hidden + col];
    write_row<D, 1>(d_table + int64_t(key) * t_ld + col, acc, scale, accumulate);
}

// ----------------------------------------------------------------- launches
struct GradLayout {
    SortShape sort;
    int piece_len, pieces;
    size_t keys, vals, counts, partial, used, total;      // byte offsets (two key and two value buffers)
};

// Pieces of 32 tokens, shorter while there are too few for the machine: a
// piece's partial rows cost 2 * hidden * 4 bytes against 32 rows read.
GradLayout grad_layout(int64_t tokens, int64_t vocab, int64_t hidden) {
    GradLayout g;
    g.sort = sort_shape(tokens, vocab);
    g.piece_len = tokens >= 8192 ? 32 : tokens >= 2048 ? 16 : 8;
    g.pieces = int((tokens + g.piece_len - 1) / g.piece_len);
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    size_t at = 0;
    g.keys = at;
    at += 2 * up(size_t(tokens) * 4);
    g.vals = at;
    at += 2 * up(size_t(tokens) * 4);
    g.counts = at;
    at += up(size_t(g.sort.tiles) * kBins * 4);
    g.partial = at;
    at += up(size_t(g.pieces) * 2 * size_t(hidden) * 4);
    g.used = at;
    at += up(size_t(vocab));
    g.total = at;
    return g;
}

template <typename S, typename D>
int run_lookup(const void* ids, int wide, int64_t tokens, const S* table, int64_t table_ld, int64_t vocab, D* out,
               int64_t out_ld, int64_t hidden, float scale, int32_t* dev_status, cudaStream_t st) {
    const bool vec = hidden % 8 == 0 && (table_ld * sizeof(S)) % 16 == 0 && (out_ld * sizeof(D)) % 16 == 0 &&
                     host::aligned(table, 16) && host::aligned(out, 16);
    const int per = kThreads * 4 * (vec ? 8 : 1);
    const dim3 grid(unsigned(tokens), unsigned((hidden + per - 1) / per));
    if (vec)
        lookup_kernel<S, D, true><<<grid, kThreads, 0, st>>>(ids, wide, table, table_ld, vocab, out, out_ld,
                                                             int(hidden), scale, dev_status);
    else
        lookup_kernel<S, D, false><<<grid, kThreads, 0, st>>>(ids, wide, table, table_ld, vocab, out, out_ld,
                                                              int(hidden), scale, dev_status);
    return cudaGetLastError() == cudaSuccess ? FP8Z_OK : FP8Z_ECUDA;
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
    uint8_t* used = accumulate ? nullptr : ws + g.used;
    const int n = int(tokens);
    if (used && cudaMemsetAsync(used, 0, size_t(ids.vocab), st) != cudaSuccess) return FP8Z_ECUDA;
    for (int p = 0; p < g.sort.passes && n > 0; ++p) {
        const uint32_t* kin = p ? keys[(p - 1) & 1] : nullptr;
        const uint32_t* vin = p ? vals[(p - 1) & 1] : nullptr;
        count_kernel<<<g.sort.tiles, kThreads, 0, st>>>(ids, kin, n, p * g.sort.digit, g.sort.digit, counts,
                                                        p ? nullptr : used);
        place_kernel<<<g.sort.tiles, kThreads, 0, st>>>(ids, kin, vin, n, p * g.sort.digit, g.sort.digit, counts,
                                                        g.sort.tiles, keys[p & 1], vals[p & 1]);
    }
    const uint32_t* k = keys[(g.sort.passes - 1) & 1];
    const uint32_t* v = vals[(g.sort.passes - 1) & 1];
    const bool vec = hidden % 8 == 0 && (d_ld * sizeof(S)) % 16 == 0 && (t_ld * sizeof(D)) % 16 == 0 &&
                     host::aligned(d_out, 16) && host::aligned(d_table, 16);
    const int fill_rows = 8;
    const int64_t fill = accumulate ? 0 : (ids.vocab + fill_rows - 1) / fill_rows;
    const int cols = vec ? kCols<true> : kCols<false>;
    const dim3 grid(unsigned(g.pieces + fill), unsigned((hidden + cols - 1) / cols));
    if (grid.x > 0) {
        if (vec)
            runs_kernel<S, D, true><<<grid, kThreads, 0, st>>>(k, v, n, uint32_t(ids.vocab), g.piece_len, g.pieces, d_out,
                                                               d_ld, d_table, t_ld, int(hidden), scale, accumulate,
                                                               partial, used, fill_rows);
        else
            runs_kernel<S, D, false><<<grid, kThreads, 0, st>>>(k, v, n, uint32_t(ids.vocab), g.piece_len, g.pieces,
                                                                d_out, d_ld, d_table, t_ld, int(hidden), scale,
                                                                accumulate, partial, used, fill_rows);
    }
    if (g.pieces > 1) {
        const dim3 jgrid(unsigned(g.pieces - 1), unsigned((hidden + kThreads - 1) / kThreads));
        join_kernel<D><<<jgrid, kThreads, 0, st>>>(k, n, uint32_t(ids.vocab), g.piece_len, partial, d_table, t_ld,
                                                   int(hidden), scale, accumulate);
    }
    return cudaGetLastError() == cudaSuccess ? FP8Z_OK : FP8Z_ECUDA;
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
