// adamw.cu -- AdamW over a list of tensors that are not kept in FP8 blocks, with
// moments in 32 or in 8 bits.
//
//   g' = factor * g
//   m' = beta1 m + (1 - beta1) g',   v' = beta2 v + (1 - beta2) g'^2
//   p' = p decay - step_size m' / (sqrt(v') / sqrt(1 - beta2^t) + eps)
//
// lpnh.cn "Model-Optimizer" article, §4.3, with each operation rounded on its own and in
// the order of the FP8 step, so that the same scalars move a parameter the same way in either.  They are
// formed from 64-bit hyper-parameters here, from 32-bit ones there: the same where FP32 holds those
// numbers, else 1 - beta is up to 2^-25 beta apart.
//
// In 8 bits a moment is E4M3 with one FP32 scale for every 128 elements, v as its square root (what
// the update divides by, and half the range of exponents).  Codes are the nearest: a root that a step moves by
// less than half a code stays, so that one among larger ones follows its gradients only within the factors
// that fp8z.h gives (1.9 at beta2 = 0.95, 11.4 at 0.999).
//
// Everything is read and written once: 28 bytes an element with FP32 moments and gradients,
// 16.1 with BF16 gradients, 8-bit moments and a BF16 copy.  200 M elements: 806 to 856 us with
// FP32 moments (0.97 of a copy's rate), 617 with 8-bit ones (5.2 TB/s; 75 instructions an element issue
// in 61 % of the cycles, most waits are for loads).
#include <cfloat>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "fp8z.h"
#include "fp8z_device.cuh"
#include "fp8z_elem.cuh"
#include "fp8z_host.h"
#include "fp8z_launch.cuh"

namespace fp8z {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRun = FP8Z_BLOCK;                 // elements of a scale: four a lane
constexpr int kChunk = FP8Z_ADAMW_CHUNK;
static_assert(kChunk % kRun == 0, "chunks are whole runs");

struct Step {
    host::AdamwScalars s;
    int post;                                    // FP8Z_DECAY_POST
};

// The multiplier of a run whose largest magnitude is amax: 448 times 1 / amax, 1 for a run of zeros.
__device__ __forceinline__ float run_scale(float amax) {
    return amax == 0.0f ? 1.0f : fminf(__fmul_rn(448.0f, __frcp_rn(amax)), FLT_MAX);
}

// Largest of the lanes' magnitudes; as whole numbers, non-negative floats keep their order.
__device__ __forceinline__ float warp_max(float a) {
    return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(a)));
}

// Root and quotient as an approximation and one correction by its remainder (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000", 1990).  The root is rounded as __fsqrt_rn rounds it
// (all fractions of two binades compared), the quotient is a unit off in a few of 2^32 pairs: the
// reciprocal behind it is itself an approximation.  At 16 bytes an element instructions
// count (200 M elements with 8-bit moments and IEEE roots and quotients: 856 us).  Values where that might
// overflow or lose its remainder, and zero, take the IEEE operation.
__device__ __forceinline__ float root_near(float v) {
    float y;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(v));
    const float r = v * y;
    return v > 0x1p-100f && v < 0x1p120f ? fmaf(fmaf(-r, r, v), 0.5f * y, r) : __fsqrt_rn(v);
}
__device__ __forceinline__ float quotient_near(float m, float d) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d));
    const float q = m * y;
    return d > 0x1p-100f && d < 0x1p100f && fabsf(m) < 0x1p20f * d ? fmaf(fmaf(-q, d, m), y, q) : __fdiv_rn(m, d);
}

// One element; r = sqrt(v').  k8: with 8-bit moments, wherever they lie, the near operations.
template <bool k8>
__device__ __forceinline__ void adamw1(const Step& A, float g, float& p, float& m, float& v, float& r) {
    m = __fadd_rn(__fmul_rn(A.s.beta1, m), __fmul_rn(A.s.omb1, g));
    v = __fadd_rn(__fmul_rn(A.s.beta2, v), __fmul_rn(A.s.omb2, __fmul_rn(g, g)));
    r = k8 ? root_near(v) : __fsqrt_rn(v);
    const float d = __fadd_rn(__fmul_rn(r, A.s.rs_bc2), A.s.eps);
    const float su = __fmul_rn(A.s.step_size, k8 ? quotient_near(m, d) : __fdiv_rn(m, d));
    if (!A.post) {
        p = __fsub_rn(__fmul_rn(p, A.s.decay), su);
    } else {
        const float pu = __fsub_rn(p, su);
        p = __fsub_rn(pu, __fmul_rn(A.s.lr_wd, pu));
    }
}

// E4M3 of four roots times their run's scale.  A v that is not zero does not become zero (m / sqrt(0) would be a
// step without bound): what is above 0 is coded as 2^-9, the smallest code, at least.
__device__ __forceinline__ uint32_t root_codes(const float (&r)[4], float s) {
    const auto code = [&](int j) { return r[j] > 0.0f ? fmaxf(r[j] * s, 0x1p-9f) : r[j]; };
    return pack_e4m3x4(code(0), code(1), code(2), code(3));
}

// Four elements of a lane: neighbours from 4 * lane on where the tensors allow 16-byte
// loads (kVec), else every 32nd from lane on; `n` elements of the run are there.
template <bool kVec>
struct Four {
    int lane, n;
    __device__ __forceinline__ int at(int j) const { return kVec ? lane * 4 + j : lane + 32 * j; }
    __device__ __forceinline__ bool whole() const { return kVec && lane * 4 + 4 <= n; }

    template <typename T>
    __device__ __forceinline__ void load(const T* p, float (&x)[4]) const {
        if (whole()) {
            if constexpr (sizeof(T) == 4) {
                const uint4 u = ld_nc_16(p + lane * 4);
                x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
            } else {
                uint2 u;
                asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(u.x), "=r"(u.y) : "l"(p + lane * 4) : "memory");
                const Pack<T, 4> y = *reinterpret_cast<const Pack<T, 4>*>(&u);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = Elem<T>::widen(y.v[j]);
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = at(j) < n ? Elem<T>::widen(p[at(j)]) : 0.0f;
    }
    // p, m and v are this kernel's own to write: loaded as they are now
    __device__ __forceinline__ void load_state(const float* p, float (&x)[4]) const {
        if (whole()) {
            const float4 u = *reinterpret_cast<const float4*>(p + lane * 4);
            x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = at(j) < n ? p[at(j)] : 0.0f;
    }
    __device__ __forceinline__ uint32_t load_codes(const uint8_t* p) const {
        if (whole()) return *reinterpret_cast<const uint32_t*>(p + lane * 4);
        uint32_t q = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at(j) < n) q |= uint32_t(p[at(j)]) << 8 * j;
        return q;
    }
    template <typename T>
    __device__ __forceinline__ void store(T* p, const float (&x)[4]) const {
        if (whole()) {
            Pack<T, 4> y;
#pragma unroll
            for (int j = 0; j < 4; ++j) y.v[j] = Elem<T>::narrow(x[j]);
            if constexpr (sizeof(T) == 4) __stcs(reinterpret_cast<uint4*>(p + lane * 4), *reinterpret_cast<const uint4*>(&y));
            else __stcs(reinterpret_cast<uint2*>(p + lane * 4), *reinterpret_cast<const uint2*>(&y));
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at(j) < n) p[at(j)] = Elem<T>::narrow(x[j]);
    }
    __device__ __forceinline__ void store_codes(uint8_t* p, uint32_t q) const {
        if (whole()) {
            __stcs(reinterpret_cast<uint32_t*>(p + lane * 4), q);
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at(j) < n) p[at(j)] = uint8_t(q >> 8 * j);
    }
};

__device__ __forceinline__ void decode4(uint32_t q, float s, float (&x)[4]) {
    const float2 a = e4m3x2_to_float2(q), b = e4m3x2_to_float2(q >> 16);
    x[0] = a.x * s, x[1] = a.y * s, x[2] = b.x * s, x[3] = b.y * s;
}

__device__ __forceinline__ float absmax4(const float (&x)[4]) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) a = fmaxf(a, fabsf(x[j]));
    return a;
}

template <bool kVec>
__device__ __forceinline__ void load_grad(const fp8z_adamw_chunk& t, int at, const Four<kVec>& f, float (&g)[4]) {
    if (t.g_dtype == FP8Z_F32) f.load(static_cast<const float*>(t.g) + at, g);
    else if (t.g_dtype == FP8Z_BF16) f.load(static_cast<const __nv_bfloat16*>(t.g) + at, g);
    else f.load(static_cast<const __half*>(t.g) + at, g);
}

// The step of a lane's four elements, and their way back.
template <bool kVec, bool k8>
__device__ __forceinline__ void update(const fp8z_adamw_chunk& t, const Step& A, float factor, int at, const Four<kVec>& f,
                                       float (&p)[4], const float (&g)[4], float (&m)[4], float (&v)[4]) {
    float r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        adamw1<k8>(A, __fmul_rn(g[j], factor), p[j], m[j], v[j], r[j]);
        if (f.at(j) >= f.n) m[j] = r[j] = 0.0f;
    }
    f.store(t.p + at, p);
    if (t.copy_dtype == FP8Z_BF16) f.store(static_cast<__nv_bfloat16*>(t.copy) + at, p);
    else if (t.copy_dtype == FP8Z_F16) f.store(static_cast<__half*>(t.copy) + at, p);
    if constexpr (k8) {
        const float sm = run_scale(warp_max(absmax4(m))), sv = run_scale(warp_max(absmax4(r)));
        f.store_codes(static_cast<uint8_t*>(t.m) + at, pack_e4m3x4(m[0] * sm, m[1] * sm, m[2] * sm, m[3] * sm));
        f.store_codes(static_cast<uint8_t*>(t.v) + at, root_codes(r, sv));
        if (f.lane == 0) {
            t.m_scale[at / kRun] = __frcp_rn(sm);
            t.v_scale[at / kRun] = __frcp_rn(sv);
        }
    } else {
        f.store(static_cast<float*>(t.m) + at, m);
        f.store(static_cast<float*>(t.v) + at, v);
    }
}

// One run of a tensor's end, or of tensors that are not aligned for vectors.
template <bool kVec, bool k8>
__device__ __forceinline__ void run_step(const fp8z_adamw_chunk& t, const Step& A, float factor, int at, const Four<kVec>& f) {
    float p[4], g[4], m[4], v[4];
    f.load_state(t.p + at, p);
    load_grad(t, at, f, g);
    if constexpr (k8) {
        decode4(f.load_codes(static_cast<const uint8_t*>(t.m) + at), t.m_scale[at / kRun], m);
        decode4(f.load_codes(static_cast<const uint8_t*>(t.v) + at), t.v_scale[at / kRun], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = v[j] * v[j];
    } else {
        f.load_state(static_cast<const float*>(t.m) + at, m);
        f.load_state(static_cast<const float*>(t.v) + at, v);
    }
    update<kVec, k8>(t, A, factor, at, f, p, g, m, v);
}

// 16 bytes of the widest tensor a lane, for every tensor of the chunk.
__device__ __forceinline__ bool vectors(const fp8z_adamw_chunk& t) {
    const uintptr_t g = reinterpret_cast<uintptr_t>(t.g) & (t.g_dtype == FP8Z_F32 ? 15 : 7);
    const uintptr_t mv = (reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v)) & (t.state_bits == 8 ? 3 : 15);
    return ((reinterpret_cast<uintptr_t>(t.p) & 15) | g | mv | (reinterpret_cast<uintptr_t>(t.copy) & 7)) == 0;
}

// Four neighbouring elements of a whole run, as they lie in memory.
template <typename G, bool k8>
struct Loaded {
    uint4 p, m4, v4;
    uint4 g4;
    uint2 g2;
    uint32_t m, v;
    float ms, vs;

    __device__ __forceinline__ void load(const fp8z_adamw_chunk& t, int at, int lane) {
        const int i = at + lane * 4;
        p = ld_stream_16(t.p + i, 0);
        if constexpr (sizeof(G) == 4) g4 = ld_stream_16(static_cast<const float*>(t.g) + i, 0);
        else asm volatile("ld.global.L1::no_allocate.L2::256B.v2.u32 {%0, %1}, [%2];" : "=r"(g2.x), "=r"(g2.y) : "l"(static_cast<const G*>(t.g) + i) : "memory");
        if constexpr (k8) {
            asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(m) : "l"(static_cast<const uint8_t*>(t.m) + i) : "memory");
            asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(static_cast<const uint8_t*>(t.v) + i) : "memory");
            ms = t.m_scale[at / kRun];
            vs = t.v_scale[at / kRun];
        } else {
            m4 = ld_stream_16(static_cast<const float*>(t.m) + i, 0);
            v4 = ld_stream_16(static_cast<const float*>(t.v) + i, 0);
        }
    }
    static __device__ __forceinline__ void floats(const uint4& u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    }
    __device__ __forceinline__ void unpack(float (&pp)[4], float (&g)[4], float (&mm)[4], float (&vv)[4]) const {
        floats(p, pp);
        if constexpr (sizeof(G) == 4) {
            floats(g4, g);
        } else {
            const Pack<G, 4> y = *reinterpret_cast<const Pack<G, 4>*>(&g2);
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = Elem<G>::widen(y.v[j]);
        }
        if constexpr (k8) {
            decode4(m, ms, mm);
            decode4(v, vs, vv);
#pragma unroll
            for (int j = 0; j < 4; ++j) vv[j] = vv[j] * vv[j];
        } else {
            floats(m4, mm);
            floats(v4, vv);
        }
    }
};

// kRuns whole runs with 8-bit moments, every eighth from `at` on.  The runs' scales, two for
// each, are formed by a few lanes for all.
template <int kRuns, typename G>
__device__ __forceinline__ void update8(const fp8z_adamw_chunk& t, const Step& A, float factor, int at, int lane,
                                        const Loaded<G, true> (&l)[kRuns]) {
    const Four<true> f{lane, kRun};
    float m[kRuns][4], r[kRuns][4];
    float top = 0.0f;                              // of this lane's moment of this lane's run
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
        float p[4], g[4], v[4];
        l[i].unpack(p, g, m[i], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) adamw1<true>(A, __fmul_rn(g[j], factor), p[j], m[i][j], v[j], r[i][j]);
        const int to = at + i * kWarps * kRun;
        f.store(t.p + to, p);
        if (t.copy_dtype == FP8Z_BF16) f.store(static_cast<__nv_bfloat16*>(t.copy) + to, p);
        else if (t.copy_dtype == FP8Z_F16) f.store(static_cast<__half*>(t.copy) + to, p);
        const float am = warp_max(absmax4(m[i])), ar = warp_max(absmax4(r[i]));
        if (lane == 2 * i) top = am;
        if (lane == 2 * i + 1) top = ar;
    }
    const float scale = run_scale(top), kept = __frcp_rn(scale);
    if (lane < 2 * kRuns) ((lane & 1) ? t.v_scale : t.m_scale)[at / kRun + (lane >> 1) * kWarps] = kept;
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
        const float sm = __shfl_sync(0xFFFFFFFFu, scale, 2 * i), sv = __shfl_sync(0xFFFFFFFFu, scale, 2 * i + 1);
        const int to = at + i * kWarps * kRun;
        f.store_codes(static_cast<uint8_t*>(t.m) + to, pack_e4m3x4(m[i][0] * sm, m[i][1] * sm, m[i][2] * sm, m[i][3] * sm));
        f.store_codes(static_cast<uint8_t*>(t.v) + to, root_codes(r[i], sv));
    }
}

// A chunk: each warp takes every eighth run, several at a time, so that the loads of all of them
// are under way together.  200 M elements with 8-bit moments: one at a time 918 us.
template <typename G, bool k8>
__device__ __forceinline__ void chunk_step(const fp8z_adamw_chunk& t, const Step& A, float factor) {
    constexpr int kRuns = k8 ? 4 : 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int at = warp * kRun;
    for (; at + ((kRuns - 1) * kWarps + 1) * kRun <= t.count; at += kRuns * kWarps * kRun) {
        Loaded<G, k8> l[kRuns];
#pragma unroll
        for (int i = 0; i < kRuns; ++i) l[i].load(t, at + i * kWarps * kRun, lane);
        if constexpr (k8) {
            update8<kRuns>(t, A, factor, at, lane, l);
        } else {
#pragma unroll
            for (int i = 0; i < kRuns; ++i) {
                float p[4], g[4], m[4], v[4];
                l[i].unpack(p, g, m, v);
                update<true, false>(t, A, factor, at + i * kWarps * kRun, Four<true>{lane, kRun}, p, g, m, v);
            }
        }
    }
    for (; at < t.count; at += kWarps * kRun) run_step<true, k8>(t, A, factor, at, Four<true>{lane, t.count - at});
}

template <bool k8>
__device__ __forceinline__ void chunk_step(const fp8z_adamw_chunk& t, const Step& A, float factor) {
    if (!vectors(t)) {
        for (int at = threadIdx.x / 32 * kRun; at < t.count; at += kWarps * kRun)
            run_step<false, k8>(t, A, factor, at, Four<false>{int(threadIdx.x & 31), t.count - at});
    } else if (t.g_dtype == FP8Z_F32) {
        chunk_step<float, k8>(t, A, factor);
    } else if (t.g_dtype == FP8Z_BF16) {
        chunk_step<__nv_bfloat16, k8>(t, A, factor);
    } else {
        chunk_step<__half, k8>(t, A, factor);
    }
}

__global__ void __launch_bounds__(kThreads) adamw_kernel(const fp8z_adamw_chunk* list, const __grid_constant__ Step A,
                                                         const float* factor) {
    dependent_wait();
    const fp8z_adamw_chunk t = list[blockIdx.x];
    const float f = factor ? *factor : 1.0f;
    if (t.state_bits == 8) chunk_step<true>(t, A, f);
    else chunk_step<false>(t, A, f);
}

// ------------------------------------------------------------------- host
bool params_ok(const fp8z_adamw_params& p) {
    const auto in = [](double x, double low, double high) { return x >= low && x < high; };       // false for NaN
    return in(p.lr, 0.0, FLT_MAX) && in(p.beta1, 0.0, 1.0) && in(p.beta2, 0.0, 1.0) && float(p.beta1) < 1.0f &&
           float(p.beta2) < 1.0f && in(p.eps, 0.0, FLT_MAX) && float(p.eps) > 0.0f && in(p.weight_decay, 0.0, FLT_MAX) &&
           p.step >= 1 && (p.decay_mode == FP8Z_DECAY_PRE || p.decay_mode == FP8Z_DECAY_POST);
}

// As host::adamw_scalars, from numbers that are not rounded to 32 bits first.
host::AdamwScalars scalars(const fp8z_adamw_params& p) {
    const double t = double(p.step), c1 = 1.0 - std::pow(p.beta1, t), c2 = 1.0 - std::pow(p.beta2, t);
    return {float(p.beta1), float(p.beta2), float(1.0 - p.beta1), float(1.0 - p.beta2), float(p.eps), float(p.lr / c1),
            float(1.0 / std::sqrt(c2)), float(1.0 - p.lr * p.weight_decay), float(p.lr * p.weight_decay)};
}

}  // namespace
}  // namespace fp8z

extern "C" int fp8z_encode_adamw_list(const fp8z_adamw_tensor* tensors, int32_t n, fp8z_adamw_chunk* out, int64_t capacity,
                                      int64_t* chunks_out) {
    using namespace fp8z;
    if (n < 0 || !chunks_out || (n > 0 && !tensors)) return FP8Z_EINVAL;
    int64_t chunks = 0;
    for (int32_t i = 0; i < n; ++i) {
        const fp8z_adamw_tensor& t = tensors[i];
        if (t.count < 0 || t.count > (1LL << 42) || !dtype_ok(t.g_dtype)) return FP8Z_EINVAL;
        if (t.state_bits != 8 && t.state_bits != 32) return FP8Z_EINVAL;
        if (t.copy && t.copy_dtype != FP8Z_BF16 && t.copy_dtype != FP8Z_F16) return FP8Z_EINVAL;
        const bool scales = t.state_bits == 8;
        if (t.count > 0 && (!t.p || !t.g || !t.m || !t.v || (scales && (!t.m_scale || !t.v_scale)))) return FP8Z_EINVAL;
        if (!host::aligned(t.p, 4) || !host::aligned(t.g, dtype_bytes(t.g_dtype)) || !host::aligned(t.m, scales ? 1 : 4) ||
            !host::aligned(t.v, scales ? 1 : 4) || !host::aligned(t.m_scale, 4) || !host::aligned(t.v_scale, 4) ||
            !host::aligned(t.copy, 2))
            return FP8Z_EALIGN;
        chunks += (t.count + kChunk - 1) / kChunk;
        if (chunks > 0x7FFFFFFF) return FP8Z_EINVAL;
    }
    *chunks_out = chunks;
    if (!out) return FP8Z_OK;
    if (capacity < chunks) return FP8Z_ENOSPACE;
    for (int32_t i = 0; i < n; ++i) {
        const fp8z_adamw_tensor& t = tensors[i];
        const int bytes = t.state_bits / 8;
        for (int64_t at = 0; at < t.count; at += kChunk) {
            fp8z_adamw_chunk c = {};
            c.p = t.p + at;
            c.g = static_cast<const uint8_t*>(t.g) + at * dtype_bytes(t.g_dtype);
            c.m = static_cast<uint8_t*>(t.m) + at * bytes;
            c.v = static_cast<uint8_t*>(t.v) + at * bytes;
            if (t.state_bits == 8) {
                c.m_scale = t.m_scale + at / kRun;
                c.v_scale = t.v_scale + at / kRun;
            }
            c.copy = t.copy ? static_cast<uint8_t*>(t.copy) + at * 2 : nullptr;
            c.count = int32_t(t.count - at < kChunk ? t.count - at : kChunk);
            c.g_dtype = int16_t(t.g_dtype);
            c.copy_dtype = int8_t(t.copy ? t.copy_dtype : -1);
            c.state_bits = int8_t(t.state_bits);
            *out++ = c;
        }
    }
    return FP8Z_OK;
}

extern "C" int fp8z_adamw(const fp8z_adamw_chunk* list, int64_t chunks, const fp8z_adamw_params* hp,
                          const float* grad_factor, void* stream) {
    using namespace fp8z;
    const host::NvtxRange nvtx_range("fp8z_adamw");
    if (chunks < 0 || chunks > 0x7FFFFFFF || (chunks > 0 && !list) || !hp || !params_ok(*hp)) return FP8Z_EINVAL;
    if (!host::aligned(list, 8) || !host::aligned(grad_factor, 4)) return FP8Z_EALIGN;
    if (chunks == 0) return FP8Z_OK;
    int sms = 0;
    if (int rc = host::device_sms(&sms)) return rc;
    const Step A = {scalars(*hp), hp->decay_mode == FP8Z_DECAY_POST};
    return launch_dependent(adamw_kernel, dim3(unsigned(chunks)), kThreads, 0, static_cast<cudaStream_t>(stream), list, A,
                            grad_factor);
}
