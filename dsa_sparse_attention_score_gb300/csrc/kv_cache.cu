// kv_cache.cu -- writing latent rows into the cache, 8-bit or bf16, and
// reading 8-bit rows back.
//
// The cached row of a token is its kv latent (512) and, with a tail, the 64
// rotary values turned at the token's position (quant8.cuh and rope.cuh have
// the formulas).  Both directions move each byte once and compute a few flops
// per value: bound by HBM for many rows, by launch latency for a few.  One
// warp per row: lane l holds latent values 16 l .. 16 l + 15, so that its
// codes are one 16-byte word and the row's largest magnitude is one warp
// reduction; and tail pair l, so that a lane forms one angle.  Nothing is
// staged in shared memory.  The chain position -> sequence -> block table ->
// row is three dependent loads long, so with many tokens a warp takes two at a
// time, their lookups side by side in two lanes and their rows in flight
// together.
// Device times: appending 32 tokens, 8-bit and paged, 2.6 us (launch latency);
// 16384 tokens 8.2 us (3.6 TB/s: under two rows per warp that can be resident, so half
// the time is the chain of lookups); reading back 2048 tokens 2.6 us, 128k
// tokens 37.5 us (6.1 TB/s, 90% of a plain copy's rate).
#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "quant8.cuh"
#include "rope.cuh"

namespace dsa {

namespace {

constexpr int kWarps = 4;               // rows per CTA

template <typename T> __device__ __forceinline__ float as_f(T v);
template <> __device__ __forceinline__ float as_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float as_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float as_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// 16 consecutive values; 16-byte loads when the rows allow it.
template <typename T>
__device__ __forceinline__ void load16(const T *src, bool vec, float (&v)[16]) {
    if (vec) {
        constexpr int N = 16 / sizeof(T);          // values per load
#pragma unroll
        for (int i = 0; i < 16 / N; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(src) + i);
            T e[N];
            *reinterpret_cast<uint4 *>(e) = u;
#pragma unroll
            for (int j = 0; j < N; ++j) v[i * N + j] = as_f(e[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = as_f(src[i]);
    }
}

struct AppendParams {
    const void *c_new, *r_new;          // r_new null: no tail
    int64_t c_stride, r_stride;         // values between rows
    int vec;                            // latent rows are 16-byte aligned
    int rotate;
    DevRope rope;
    uint16_t *kv;                       // bf16 rows (null: 8-bit)
    uint8_t *codes;
    float *scale;
};

// Cache rows of tokens t0 .. t0 + R - 1: lane i < R gets token t0 + i's position
// and row, -1 past the last token (not flagged) or out of bounds (flagged).
template <int R>
__device__ __forceinline__ int64_t token_rows(const DevBatch &b, int t0, int lane, int32_t *pos_out, uint32_t *status) {
    const int t = t0 + lane;
    const bool mine = lane < R && t < b.T;
    const int32_t pos = mine ? __ldg(b.q_pos + t) : -1;
    int seq = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int s = seq_of_warp(b.cu_q, b.B, min(t0 + i, b.T - 1), lane);
        seq = lane == i ? s : seq;
    }
    int64_t row = -1;
    if (mine) {
        const int64_t kv0 = seq_base(b, seq);
        if (pos >= 0 && pos < b.max_kv && kv0 >= 0) row = cache_row(b, seq, kv0, pos);
        if (row >= b.cache_rows) row = -1;
        if (row < 0) flag(status, DSA_DEV_BAD_POSITION);
    }
    *pos_out = pos;
    return row;
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

}  // namespace

// The row of one token, held by the warp: its latent values v and tail pair.
template <bool kQ8>
__device__ __forceinline__ void store_row(const AppendParams &p, const float (&v)[16], float ra, float rb, int32_t pos,
                                          int64_t row, int lane) {
    const bool tail = p.r_new != nullptr;
    // tail pair of this lane: values i0 and i1 of the 64
    const bool inter = p.rope.interleaved;
    const int i0 = inter ? 2 * lane : lane, i1 = inter ? 2 * lane + 1 : lane + 32;
    if (tail && p.rotate) {
        const float2 w = rope_cos_sin(pos, __ldg(p.rope.inv_freq + lane), p.rope.scale, p.rope.inverse);
        const float x = ra * w.x - rb * w.y;
        rb = ra * w.y + rb * w.x;
        ra = x;
    }
    if (!kQ8) {
        const int width = tail ? D_ROW : D_L;
        uint16_t *dst = p.kv + row * width;
        uint4 o[2];
        uint32_t *w = reinterpret_cast<uint32_t *>(o);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = bf16x2(v[2 * i], v[2 * i + 1]);
        reinterpret_cast<uint4 *>(dst)[2 * lane] = o[0];
        reinterpret_cast<uint4 *>(dst)[2 * lane + 1] = o[1];
        if (tail) {
            dst[D_L + i0] = __bfloat16_as_ushort(__float2bfloat16_rn(ra));
            dst[D_L + i1] = __bfloat16_as_ushort(__float2bfloat16_rn(rb));
        }
        return;
    }
    // the largest magnitude by its bits, which order like the values and put
    // infinity and NaN above every finite one
    uint32_t top = max(__float_as_uint(ra) & 0x7FFFFFFFu, __float_as_uint(rb) & 0x7FFFFFFFu);
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xffffffffu, top);
    const bool finite = top < 0x7F800000u;
    const int e = finite ? q8_exponent(__uint_as_float(top)) : 0;
    const float inv = exp2_int(-e);
    const int width = tail ? kQ8Row : D_L;
    uint8_t *dst = p.codes + row * width;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = finite ? e4m3x2(v[4 * i] * inv, v[4 * i + 1] * inv) | e4m3x2(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16 : 0u;
    reinterpret_cast<uint4 *>(dst)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
    if (tail) {
        ra *= inv;
        rb *= inv;
        uint32_t hi = e4m3x2(ra, rb);
        const float2 h = e4m3x2_to_float2(hi);
        uint32_t lo = e4m3x2(ra - h.x, rb - h.y);
        if (!finite) hi = lo = 0u;
        if (inter) {
            reinterpret_cast<uint16_t *>(dst + D_L)[lane] = (uint16_t)hi;
            reinterpret_cast<uint16_t *>(dst + D_L + D_R)[lane] = (uint16_t)lo;
        } else {
            dst[D_L + i0] = (uint8_t)hi;
            dst[D_L + i1] = (uint8_t)(hi >> 8);
            dst[D_L + D_R + i0] = (uint8_t)lo;
            dst[D_L + D_R + i1] = (uint8_t)(lo >> 8);
        }
    }
    if (lane == 0) p.scale[row] = finite ? exp2_int(e) : __int_as_float(0x7FC00000);
}

template <typename T, bool kQ8, int R>
__global__ void __launch_bounds__(32 * kWarps) kv_append_kernel(const AppendParams p, const DevBatch b, uint32_t *status) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int t0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * R;
    if (t0 >= b.T) return;
    float v[R][16], ra[R], rb[R];
    const int i0 = p.rope.interleaved ? 2 * lane : lane, i1 = p.rope.interleaved ? 2 * lane + 1 : lane + 32;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t t = min(t0 + i, b.T - 1);
        load16(static_cast<const T *>(p.c_new) + t * p.c_stride + lane * 16, p.vec, v[i]);
        ra[i] = rb[i] = 0.f;
        if (p.r_new) {
            const T *r = static_cast<const T *>(p.r_new) + t * p.r_stride;
            ra[i] = as_f(r[i0]);
            rb[i] = as_f(r[i1]);
        }
    }
    int32_t pos;
    const int64_t row = token_rows<R>(b, t0, lane, &pos, status);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t row_i = __shfl_sync(0xffffffffu, row, i);
        const int32_t pos_i = __shfl_sync(0xffffffffu, pos, i);
        if (row_i >= 0) store_row<kQ8>(p, v[i], ra[i], rb[i], pos_i, row_i, lane);
    }
}

struct ReadParams {
    const uint8_t *codes;
    const float *scale;
    int tail;
    void *out;
    int64_t stride;                     // values between output rows
    int vec;                            // output rows are 16-byte aligned
};

// A code times a power of two is exact in bf16, so only the tail's sum rounds.
// A token out of bounds gets a row of zeros.
template <bool kBf16, int R>
__global__ void __launch_bounds__(32 * kWarps) kv_read_kernel(const ReadParams p, const DevBatch b, uint32_t *status) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int t0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * R;
    if (t0 >= b.T) return;
    int32_t pos;
    const int64_t row = token_rows<R>(b, t0, lane, &pos, status);
    uint4 c[R];
    uint32_t hi[R], lo[R];
    float s[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t row_i = __shfl_sync(0xffffffffu, row, i);
        c[i] = make_uint4(0u, 0u, 0u, 0u);
        hi[i] = lo[i] = 0;
        s[i] = 0.f;
        if (row_i >= 0) {
            const uint8_t *src = p.codes + row_i * (p.tail ? kQ8Row : D_L);
            c[i] = __ldg(reinterpret_cast<const uint4 *>(src) + lane);
            if (p.tail) {
                hi[i] = __ldg(reinterpret_cast<const uint16_t *>(src + D_L) + lane);
                lo[i] = __ldg(reinterpret_cast<const uint16_t *>(src + D_L + D_R) + lane);
            }
            s[i] = __ldg(p.scale + row_i);
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (t0 + i >= b.T) break;
        const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
        float v[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 x = e4m3x2_to_float2(w[j] & 0xFFFFu), y = e4m3x2_to_float2(w[j] >> 16);
            v[4 * j] = x.x * s[i]; v[4 * j + 1] = x.y * s[i]; v[4 * j + 2] = y.x * s[i]; v[4 * j + 3] = y.y * s[i];
        }
        const float2 h = e4m3x2_to_float2(hi[i]), l = e4m3x2_to_float2(lo[i]);
        const float ta = (h.x + l.x) * s[i], tb = (h.y + l.y) * s[i];
        if (kBf16) {
            uint16_t *dst = static_cast<uint16_t *>(p.out) + (int64_t)(t0 + i) * p.stride;
            uint32_t u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = bf16x2(v[2 * j], v[2 * j + 1]);
            const uint32_t o2 = bf16x2(ta, tb);
            if (p.vec) {
                reinterpret_cast<uint4 *>(dst)[2 * lane] = make_uint4(u[0], u[1], u[2], u[3]);
                reinterpret_cast<uint4 *>(dst)[2 * lane + 1] = make_uint4(u[4], u[5], u[6], u[7]);
                if (p.tail) reinterpret_cast<uint32_t *>(dst + D_L)[lane] = o2;
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) dst[16 * lane + j] = (uint16_t)(u[j >> 1] >> (16 * (j & 1)));
                if (p.tail) {
                    dst[D_L + 2 * lane] = (uint16_t)o2;
                    dst[D_L + 2 * lane + 1] = (uint16_t)(o2 >> 16);
                }
            }
        } else {
            float *dst = static_cast<float *>(p.out) + (int64_t)(t0 + i) * p.stride;
            if (p.vec) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    reinterpret_cast<float4 *>(dst)[4 * lane + j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) dst[16 * lane + j] = v[j];
            }
            if (p.tail) {
                dst[D_L + 2 * lane] = ta;
                dst[D_L + 2 * lane + 1] = tb;
            }
        }
    }
}

namespace {

// Several tokens per warp once there are enough to give every SM several warps;
// one below that, where the latency of a single row counts.
constexpr int kBatchTokens = 2;
inline bool batched(const DevBatch &b) { return b.T >= 16 * kSMs * kBatchTokens; }
inline unsigned grid_of(const DevBatch &b, int per_warp) {
    return (unsigned)(((int64_t)b.T + kWarps * per_warp - 1) / (kWarps * per_warp));
}

template <typename T, bool kQ8>
cudaError_t launch_append_as(const AppendParams &p, const DevBatch &b, uint32_t *status, cudaStream_t stream) {
    if (batched(b))
        return launch_k(kv_append_kernel<T, kQ8, kBatchTokens>, dim3(grid_of(b, kBatchTokens)), dim3(32 * kWarps), 0, stream, true,
                        p, b, status);
    return launch_k(kv_append_kernel<T, kQ8, 1>, dim3(grid_of(b, 1)), dim3(32 * kWarps), 0, stream, true, p, b, status);
}
template <typename T>
cudaError_t launch_append_t(const AppendParams &p, const DevBatch &b, uint32_t *status, cudaStream_t stream) {
    return p.kv ? launch_append_as<T, false>(p, b, status, stream) : launch_append_as<T, true>(p, b, status, stream);
}
template <bool kBf16>
cudaError_t launch_read_as(const ReadParams &p, const DevBatch &b, uint32_t *status, cudaStream_t stream) {
    if (batched(b))
        return launch_k(kv_read_kernel<kBf16, kBatchTokens>, dim3(grid_of(b, kBatchTokens)), dim3(32 * kWarps), 0, stream, true, p, b,
                        status);
    return launch_k(kv_read_kernel<kBf16, 1>, dim3(grid_of(b, 1)), dim3(32 * kWarps), 0, stream, true, p, b, status);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendLaunch &a, const DevBatch &b, uint32_t *status, cudaStream_t stream) {
    const int64_t size = a.dtype == DSA_DT_F32 ? 4 : 2;
    AppendParams p;
    p.c_new = a.c_new;
    p.r_new = a.r_new;
    p.c_stride = a.c_stride;
    p.r_stride = a.r_stride;
    p.vec = ((reinterpret_cast<uintptr_t>(a.c_new) | (uintptr_t)(a.c_stride * size)) & 15) == 0;
    p.rotate = a.inv_freq != nullptr;
    p.rope = DevRope{a.inv_freq, D_R, a.interleaved, a.rope_scale, 0};
    p.kv = a.kv;
    p.codes = a.codes;
    p.scale = a.scale;
    switch (a.dtype) {
        case DSA_DT_F32: return launch_append_t<float>(p, b, status, stream);
        case DSA_DT_F16: return launch_append_t<__half>(p, b, status, stream);
        default: return launch_append_t<__nv_bfloat16>(p, b, status, stream);
    }
}

cudaError_t launch_kv_read(const uint8_t *codes, const float *scale, int tail, void *out, int out_dtype, int64_t stride,
                           const DevBatch &b, uint32_t *status, cudaStream_t stream) {
    const int64_t size = out_dtype == DSA_DT_F32 ? 4 : 2;
    ReadParams p{codes, scale, tail, out, stride,
                 ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(stride * size)) & 15) == 0};
    return out_dtype == DSA_DT_F32 ? launch_read_as<false>(p, b, status, stream) : launch_read_as<true>(p, b, status, stream);
}

}  // namespace dsa
