// rope.cu -- rotary positions on (part of) the heads of a token's rows.
//
// Value pair (a, b) of a token at position p turns by the angle p * f_j:
//     (a, b) -> s (a cos - b sin, a sin + b cos),
// pairs being neighbours (interleaved) or the two halves of the rotated part;
// the other values of a head are copied.  The transpose (gradient) is the
// same with the angle negated.
//
// One pass over memory and three flops a value: bound by HBM, or by launch
// latency for a few tokens.  A CTA takes one token and up to 256 * kUnits
// 16-byte units of its heads; the units are loaded before the angles are
// formed (rot_dim / 2 of them, once per CTA, in 64 bits), so that the trig
// hides behind the loads.  Rows whose addresses or extents are not multiples of 16
// bytes take the same kernel with units of one value.
#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "rope.cuh"

namespace dsa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kUnits = 4;              // units in flight per thread
constexpr int kMaxPairs = 256;         // rot_dim <= 512

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T v[V]; };

struct RopeParams {
    const void *x;
    void *y;
    int64_t xt, xh, yt, yh;    // token and head strides, in values
    const int32_t *pos;
    DevRope r;
    int heads, dim, off;       // values per head; first rotated one
    int copy;                  // write the values that do not turn
};

}  // namespace

// V values per unit.  Interleaved: a unit is V neighbouring values, pairs
// inside it (V = 1 stands for one pair, or one copied value).  Halves: a unit
// is V values of the first half and their V partners.
template <typename T, bool kInter, int V>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    __shared__ float2 cs[kMaxPairs];
    using VT = Vec<T, V>;
    constexpr int S = kInter && V == 1 ? 2 : V;          // values a rotated unit spans (per part)
    constexpr int kParts = (!kInter || V == 1) ? 2 : 1;  // loads of a rotated unit
    const int t = blockIdx.x, tid = threadIdx.x;
    const int half = p.r.rot_dim >> 1;
    const int rot_units = (kInter ? p.r.rot_dim : half) / S;
    const int copy_units = p.copy ? (p.dim - p.r.rot_dim) / V : 0;
    const int per_head = rot_units + copy_units;
    const int total = p.heads * per_head;
    const int first = blockIdx.y * (kRopeThreads * kUnits) + tid;
    const T *x = static_cast<const T *>(p.x) + (int64_t)t * p.xt;
    T *y = static_cast<T *>(p.y) + (int64_t)t * p.yt;
    VT a[kUnits], b[kUnits];
    int head[kUnits], at[kUnits], part2[kUnits], pair[kUnits];   // pair < 0: copied
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int i = first + u * kRopeThreads;
        head[u] = -1;
        if (i >= total) continue;
        const int h = i / per_head, r = i - h * per_head;
        head[u] = h;
        if (r < rot_units) {
            at[u] = p.off + r * S;
            part2[u] = at[u] + (kInter ? 1 : half);
            pair[u] = kInter ? r * S / 2 : r * S;
        } else {
            const int c = (r - rot_units) * V;
            at[u] = c < p.off ? c : c + p.r.rot_dim;
            pair[u] = -1;
        }
        const T *src = x + (int64_t)h * p.xh;
        a[u] = *reinterpret_cast<const VT *>(src + at[u]);
        if (kParts == 2 && pair[u] >= 0) b[u] = *reinterpret_cast<const VT *>(src + part2[u]);
    }
    const int32_t pos = __ldg(p.pos + t);
    for (int j = tid; j < half; j += kRopeThreads) cs[j] = rope_cos_sin(pos, __ldg(p.r.inv_freq + j), p.r.scale, p.r.inverse);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        if (head[u] < 0) continue;
        T *dst = y + (int64_t)head[u] * p.yh;
        if (pair[u] >= 0) {
            if (kParts == 1) {
#pragma unroll
                for (int e = 0; e + 1 < V; e += 2) {
                    const float2 w = cs[pair[u] + e / 2];
                    const float va = to_f(a[u].v[e]), vb = to_f(a[u].v[e + 1]);
                    a[u].v[e] = from_f<T>(va * w.x - vb * w.y);
                    a[u].v[e + 1] = from_f<T>(va * w.y + vb * w.x);
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 w = cs[pair[u] + e];
                    const float va = to_f(a[u].v[e]), vb = to_f(b[u].v[e]);
                    a[u].v[e] = from_f<T>(va * w.x - vb * w.y);
                    b[u].v[e] = from_f<T>(va * w.y + vb * w.x);
                }
                *reinterpret_cast<VT *>(dst + part2[u]) = b[u];
            }
        }
        *reinterpret_cast<VT *>(dst + at[u]) = a[u];
    }
}

namespace {

template <typename T, bool kInter, int V>
cudaError_t launch_rope_as(const RopeParams &p, int n_tokens, cudaStream_t stream) {
    const int units = (kInter && V > 1 ? p.r.rot_dim / V : p.r.rot_dim / 2 / V) + (p.copy ? (p.dim - p.r.rot_dim) / V : 0);
    const int64_t total = (int64_t)units * p.heads;
    const int64_t ny = (total + kRopeThreads * kUnits - 1) / (kRopeThreads * kUnits);
    if (ny > 65535) return cudaErrorInvalidConfiguration;
    if (ny == 0) return cudaSuccess;
    rope_kernel<T, kInter, V><<<dim3((unsigned)n_tokens, (unsigned)ny), kRopeThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rope_t(const RopeParams &p, int n_tokens, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    // 16-byte units: every address and every extent a multiple of 16 bytes
    const int64_t any = p.xt | p.xh | p.yt | p.yh | p.dim | p.off | (p.r.interleaved ? p.r.rot_dim : p.r.rot_dim / 2);
    const bool vec = any % V == 0 && p.r.rot_dim % V == 0 &&
                     ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.y)) & 15) == 0;
    if (p.r.interleaved)
        return vec ? launch_rope_as<T, true, V>(p, n_tokens, stream) : launch_rope_as<T, true, 1>(p, n_tokens, stream);
    return vec ? launch_rope_as<T, false, V>(p, n_tokens, stream) : launch_rope_as<T, false, 1>(p, n_tokens, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch &a, cudaStream_t stream) {
    RopeParams p;
    p.x = a.x;
    p.y = a.y;
    p.xt = a.x_token_stride;
    p.xh = a.x_head_stride;
    p.yt = a.y_token_stride;
    p.yh = a.y_head_stride;
    p.pos = a.pos;
    p.r = DevRope{a.inv_freq, a.rot_dim, a.interleaved, a.scale, a.inverse};
    p.heads = a.heads;
    p.dim = a.head_dim;
    p.off = a.rot_off;
    p.copy = a.copy_rest;
    switch (a.dtype) {
        case DSA_DT_F32: return launch_rope_t<float>(p, a.n_tokens, stream);
        case DSA_DT_F16: return launch_rope_t<__half>(p, a.n_tokens, stream);
        default: return launch_rope_t<__nv_bfloat16>(p, a.n_tokens, stream);
    }
}

}  // namespace dsa
