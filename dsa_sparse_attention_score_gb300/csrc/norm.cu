// norm.cu -- root-mean-square norm of rows, with the residual's addition in
// front and, in place of plain outputs, e4m3 codes with one scale per group:
//     h = x + residual (rounded to the rows' type, as it is stored),
//     y = h / sqrt(mean(h^2) + eps) * weight,
//     scale = max(max |y| / 448, 2^-40),  code = e4m3(y / scale)  per group.
//
// Bound by HBM, and with codes by instructions (8191 rows of 4096 fp16 values: 70% of what
// an SM issues, DRAM at 51%): a row's values are read once, kept in registers over the
// one reduction that the row needs, and written once.  A row belongs to a run of
// threads of one CTA (several short rows share a CTA), each of which holds V
// units of W values; a unit is 16 bytes where the rows allow it.  Measured on
// GB300, 16,384 rows of 7168 bf16 values with residual and sum (939 MB): two units
// a thread 158 us (5.9 TB/s), one 182, four 244 (fewer threads an SM); taking rows
// in turn with the next one's loads ahead 216 (registers).  8191 rows of 4096 fp16
// values to codes (236 MB): 48 us with 40 registers a thread and the weights loaded
// behind the reduction (54 with 60 registers: fewer threads an SM; plain outputs
// lose by it, 158 -> 167 us).  At 40 the forms of two units and more spill (fp16 40
// bytes a thread, bf16 56, float32 132, rows that are not aligned 20 to 124): bf16 takes 55 us for
// the same rows, float32 83.  Without a residual, at 3 bytes a value instead of 7, fp16
// takes 40 us, bf16 44.
#include <algorithm>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "quant8.cuh"

namespace dsa {

namespace {

constexpr float kLeastScale = 9.094947017729282e-13f;   // 2^-40, as in the 8-bit cache
constexpr float kTop = 448.f;                           // the largest e4m3 value

struct NormParams {
    const void *x, *residual;      // residual null: none
    void *sum;                     // null: not stored
    const void *weight;            // null: 1
    int weight_f32;
    void *out;
    uint8_t *codes;                // [n, dim]
    float *scale;                  // [n, groups]
    int64_t xs, rs, ss, os;        // values between rows
    int n, dim, group;
    int groups, group_log2;        // of a row; of one group's values where a row has several
    float eps;
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int W> struct alignas(W * sizeof(T) >= 16 ? 16 : sizeof(T)) Unit { T v[W]; };

template <typename T, int W, bool kAligned> __device__ __forceinline__ Unit<T, W> load_unit(const T *p) {
    Unit<T, W> u;
    if constexpr (kAligned || W == 1) {
        u = *reinterpret_cast<const Unit<T, W> *>(p);
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e) u.v[e] = p[e];
    }
    return u;
}
template <typename T, int W, bool kAligned> __device__ __forceinline__ void store_unit(T *p, const Unit<T, W> &u) {
    if constexpr (kAligned || W == 1) {
        *reinterpret_cast<Unit<T, W> *>(p) = u;
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e) p[e] = u.v[e];
    }
}

// v / 448 for v >= 0, the float32 quotient: a product with the rounded reciprocal, off by
// up to 1.5 steps, and its remainder, which a fused multiply-add gives exactly, times
// the reciprocal again (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  Divisions proper here and for the codes made 8191 x 4096
// fp16 15% slower, this nothing that is measured; without the remainders codes next to a
// border between two fall on the wrong side.
__device__ __forceinline__ float over_top(float v) {
    const float q = v * (1.f / kTop);
    return fmaf(fmaf(-q, kTop, v), 1.f / kTop, q);
}

// Reduction over the threads of a row (blockDim.x of them, whole warps).
template <typename Op, typename V> __device__ __forceinline__ V row_reduce(V v, Op op, V *sh) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, d));
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    V *row = sh + threadIdx.y * warps;
    __syncthreads();                                     // an earlier reduction has been read
    if ((threadIdx.x & 31) == 0) row[threadIdx.x >> 5] = v;
    __syncthreads();
    v = row[0];
    for (int w = 1; w < warps; ++w) v = op(v, row[w]);   // the same order in every thread
    return v;
}

}  // namespace

template <typename T, int W, int V, bool kAligned, bool kCodes>
__global__ void __maxnreg__(kCodes ? 40 : 64) rms_norm_kernel(const NormParams p) {
    __shared__ uint32_t sh[32];
    const uint32_t row = blockIdx.x * blockDim.y + threadIdx.y;   // up to 3 behind 2^31 - 1 rows
    const bool live = row < (uint32_t)p.n;
    const int tx = threadIdx.x, step = blockDim.x;
    const T *x = static_cast<const T *>(p.x) + row * p.xs;
    pdl_wait();
    // h stays in its own type (half the registers of float32 for 16-bit rows)
    Unit<T, W> h[V], w[V];
    {
        Unit<T, W> r[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int at = (tx + k * step) * W;
            if (live && at < p.dim) {
                h[k] = load_unit<T, W, kAligned>(x + at);
                if (p.residual) r[k] = load_unit<T, W, kAligned>(static_cast<const T *>(p.residual) + row * p.rs + at);
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) h[k].v[e] = from_f<T>(0.f);
            }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int at = (tx + k * step) * W;
            if (!(live && at < p.dim)) continue;
            if (p.residual) {
#pragma unroll
                for (int e = 0; e < W; ++e) h[k].v[e] = from_f<T>(to_f(h[k].v[e]) + to_f(r[k].v[e]));
            }
            if (p.sum) store_unit<T, W, kAligned>(static_cast<T *>(p.sum) + row * p.ss + at, h[k]);
        }
    }
    const bool own_weight = p.weight && !p.weight_f32;
    auto load_weight = [&] {
        if (!own_weight) return;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int at = (tx + k * step) * W;
            if (at < p.dim) w[k] = load_unit<T, W, kAligned>(static_cast<const T *>(p.weight) + at);
        }
    };
    constexpr bool late = kCodes && V > 1;               // registers before latency
    if (!late) load_weight();
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int e = 0; e < W; ++e) ss = fmaf(to_f(h[k].v[e]), to_f(h[k].v[e]), ss);
    ss = row_reduce(ss, [](float a, float b) { return a + b; }, reinterpret_cast<float *>(sh));
    if (late) load_weight();
    const float rstd = 1.f / sqrtf(ss / (float)p.dim + p.eps);
    // the W values of unit k
    auto values = [&](int k, float (&y)[W]) {
        const int at = (tx + k * step) * W;
#pragma unroll
        for (int e = 0; e < W; ++e) {
            y[e] = to_f(h[k].v[e]) * rstd;
            if (own_weight) y[e] *= to_f(w[k].v[e]);
            else if (p.weight) y[e] *= __ldg(static_cast<const float *>(p.weight) + at + e);
        }
    };
    if constexpr (!kCodes) {
        if (!live) return;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int at = (tx + k * step) * W;
            if (at < p.dim) {
                float y[W];
                values(k, y);
                Unit<T, W> u;
#pragma unroll
                for (int e = 0; e < W; ++e) u.v[e] = from_f<T>(y[e]);
                store_unit<T, W, kAligned>(static_cast<T *>(p.out) + row * p.os + at, u);
            }
        }
    } else {
        // Magnitudes compare as their bits do, NaN above infinity above all numbers.
        auto top_of = [&](const float (&y)[W]) {
            uint32_t t = 0;
#pragma unroll
            for (int e = 0; e < W; ++e) t = max(t, __float_as_uint(y[e]) & 0x7fffffffu);
            return t;
        };
        const bool whole = p.group == p.dim;             // one scale a row
        uint32_t all = 0;
        if (whole) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float y[W];
                if ((tx + k * step) * W < p.dim) {
                    values(k, y);
                    all = max(all, top_of(y));
                }
            }
            all = row_reduce(all, [](uint32_t a, uint32_t b) { return max(a, b); }, sh);
        }
        const int lanes = p.group / W;                   // of one group (a power of two up to 32 otherwise)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int at = (tx + k * step) * W;
            float y[W];
#pragma unroll
            for (int e = 0; e < W; ++e) y[e] = 0.f;
            if (at < p.dim) values(k, y);
            uint32_t t = all;
            if (!whole) {
                t = top_of(y);
                for (int d = 1; d < lanes; d <<= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, d));
            }
            if (live && at < p.dim) {
                const bool bad = t >= 0x7f800000u;
                const float scale = bad ? __int_as_float(0x7fffffff) : fmaxf(over_top(__uint_as_float(t)), kLeastScale);
                const float inv = __frcp_rn(scale);
                // y / scale in the same way, two at a time (signs as they are here keep that of a 0)
                const uint64_t inv2 = f2(inv, inv), less2 = f2(-inv, -inv), scale2 = f2(scale, scale);
                auto coded = [&](float a, float b) {
                    const uint64_t q = f2_mul(f2(a, b), inv2);
                    const float2 r = f2_get(f2_fma(f2_fma(q, scale2, f2(-a, -b)), less2, q));
                    return e4m3x2(r.x, r.y);
                };
                uint32_t c[W / 4];
#pragma unroll
                for (int e = 0; e < W; e += 4)
                    c[e / 4] = bad ? 0u : coded(y[e], y[e + 1]) | coded(y[e + 2], y[e + 3]) << 16;
                uint8_t *dst = p.codes + (int64_t)row * p.dim + at;
                if constexpr (W == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(c[0], c[1]);
                else *reinterpret_cast<uint32_t *>(dst) = c[0];
                if (whole ? at == 0 : (at & (p.group - 1)) == 0) p.scale[(int64_t)row * p.groups + (whole ? 0 : at >> p.group_log2)] = scale;
            }
        }
    }
}

namespace {

template <typename T, int W, int V, bool kAligned, bool kCodes>
cudaError_t launch_norm_as(const NormParams &p, cudaStream_t stream) {
    const int units = (p.dim + W - 1) / W;
    const int threads = std::max(32, ((units + V - 1) / V + 31) / 32 * 32), rows = std::max(1, 128 / threads);
    return launch_k(rms_norm_kernel<T, W, V, kAligned, kCodes>, dim3((unsigned)(((int64_t)p.n + rows - 1) / rows)),
                    dim3((unsigned)threads, (unsigned)rows), 0, stream, true, p);
}

// Units a thread: one where that leaves no more than a wave of CTAs (two of
// 1024 threads an SM) -- the row's latency is then its one load's --, else two;
// more only where a CTA has no more threads.
template <typename T, int W, bool kAligned, bool kCodes>
cudaError_t launch_norm_units(const NormParams &p, cudaStream_t stream) {
    const int units = (p.dim + W - 1) / W;
    if constexpr (W == 1) {
        if (units <= 4096) return launch_norm_as<T, W, 4, kAligned, kCodes>(p, stream);
        return launch_norm_as<T, W, 16, kAligned, kCodes>(p, stream);
    } else {
        if (units <= 1024 && (int64_t)p.n * units <= 2048 * kSMs) return launch_norm_as<T, W, 1, kAligned, kCodes>(p, stream);
        if (units <= 2048) return launch_norm_as<T, W, 2, kAligned, kCodes>(p, stream);
        if constexpr (sizeof(T) == 4) return launch_norm_as<T, W, 4, kAligned, kCodes>(p, stream);
        return cudaErrorInvalidValue;                    // (16,384 values of 16 bits are 2048 units)
    }
}

template <typename T> cudaError_t launch_norm_t(const NormParams &p, cudaStream_t stream) {
    constexpr int W = 16 / sizeof(T);
    const auto bits = [](const void *q) { return reinterpret_cast<uintptr_t>(q); };
    const bool aligned = ((bits(p.x) | bits(p.residual) | bits(p.sum) | bits(p.out) | (p.weight_f32 ? 0 : bits(p.weight))) & 15) == 0 &&
                         (p.xs | p.rs | p.ss | p.os) % W == 0;
    if (p.codes) return aligned ? launch_norm_units<T, W, true, true>(p, stream) : launch_norm_units<T, W, false, true>(p, stream);
    if (p.dim % W == 0) return aligned ? launch_norm_units<T, W, true, false>(p, stream) : launch_norm_units<T, W, false, false>(p, stream);
    return launch_norm_units<T, 1, true, false>(p, stream);
}

}  // namespace

cudaError_t launch_rms_norm(const NormLaunch &a, cudaStream_t stream) {
    NormParams p{};
    p.x = a.x;
    p.residual = a.residual;
    p.sum = a.sum;
    p.weight = a.weight;
    p.weight_f32 = a.weight_f32;
    p.out = a.out;
    p.codes = a.codes;
    p.scale = a.scale;
    p.xs = a.x_stride;
    p.rs = a.residual ? a.residual_stride : 0;
    p.ss = a.sum ? a.sum_stride : 0;
    p.os = a.out ? a.out_stride : 0;
    p.n = a.n;
    p.dim = a.dim;
    p.group = a.group;
    p.groups = a.group ? a.dim / a.group : 0;
    while ((1 << p.group_log2) < a.group) ++p.group_log2;
    p.eps = a.eps;
    switch (a.dtype) {
        case DSA_DT_F32: return launch_norm_t<float>(p, stream);
        case DSA_DT_F16: return launch_norm_t<__half>(p, stream);
        default: return launch_norm_t<__nv_bfloat16>(p, stream);
    }
}

}  // namespace dsa
