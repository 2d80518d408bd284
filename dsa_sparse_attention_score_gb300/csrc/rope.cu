// rope.cu -- rotary positions on (part of) the heads of a token's rows.
//
// Value pair (a, b) of a token at position p turns by the angle p * f_j:
//     (a, b) -> s (a cos - b sin, a sin + b cos),
// pairs being neighbours (interleaved) or the two halves of the rotated part;
// the other values of a head are copied.  The transpose (gradient) is the
// same with the angle negated.
//
// One pass over memory and three flops a value: bound by HBM, or by launch
// latency for a few tokens.  A CTA takes one token; a thread takes the same
// unit of 16 bytes of kUnits heads, so that its place in a head and its angles
// are found once, and its loads are out before the angles are formed (rot_dim
// / 2 of them, once per CTA).  Rows whose addresses or extents are not
// multiples of 16 bytes take the same kernel with units of one value.
#include <algorithm>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "rope.cuh"

namespace dsa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kUnits = 4;              // heads per thread
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
    int per_head, lanes;       // units of a head; those a CTA takes of each head
    int rows;                  // heads a CTA takes at a time
};

}  // namespace

// V values per unit.  Interleaved: a unit is V neighbouring values, pairs
// inside it (V = 1 stands for one pair, or one copied value).  Halves: a unit
// is V values of the first half and their V partners.  grid: token, block of
// heads, block of a head's units.
template <typename T, bool kInter, int V>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    __shared__ float2 cs[kMaxPairs];
    using VT = Vec<T, V>;
    constexpr int S = kInter && V == 1 ? 2 : V;          // values a rotated unit spans (per part)
    constexpr int kParts = (!kInter || V == 1) ? 2 : 1;  // loads of a rotated unit
    constexpr int kPairs = V > 1 && kInter ? V / 2 : V;  // angles of a rotated unit
    const int t = blockIdx.x, tid = threadIdx.x;
    const int half = p.r.rot_dim >> 1;
    const int rot_units = (kInter ? p.r.rot_dim : half) / S;
    const int row = tid / p.lanes, r = blockIdx.z * p.lanes + tid - row * p.lanes;
    const int h0 = blockIdx.y * (p.rows * kUnits) + row;
    const bool live = row < p.rows && r < p.per_head, turns = r < rot_units;
    const int c = (r - rot_units) * V;                   // a copied unit's place among the copied values
    const int v = turns ? p.off + r * S : c < p.off ? c : c + p.r.rot_dim;
    const int partner = kInter ? 1 : half;
    const T *x = static_cast<const T *>(p.x) + (int64_t)t * p.xt + v;
    T *y = static_cast<T *>(p.y) + (int64_t)t * p.yt + v;
    VT a[kUnits], b[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int h = h0 + u * p.rows;
        if (live && h < p.heads) {
            a[u] = *reinterpret_cast<const VT *>(x + (int64_t)h * p.xh);
            if (kParts == 2 && turns) b[u] = *reinterpret_cast<const VT *>(x + (int64_t)h * p.xh + partner);
        }
    }
    const int32_t pos = __ldg(p.pos + t);
    for (int j = tid; j < half; j += blockDim.x) cs[j] = rope_cos_sin(pos, __ldg(p.r.inv_freq + j), p.r.scale, p.r.inverse);
    __syncthreads();
    if (!live) return;
    float2 w[kPairs];
    if (turns) {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) w[e] = cs[r * kPairs + e];
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int h = h0 + u * p.rows;
        if (h >= p.heads) break;
        T *dst = y + (int64_t)h * p.yh;
        if (turns) {
            if (kParts == 1) {
#pragma unroll
                for (int e = 0; e + 1 < V; e += 2) {
                    const float2 f = w[e / 2];
                    const float va = to_f(a[u].v[e]), vb = to_f(a[u].v[e + 1]);
                    a[u].v[e] = from_f<T>(va * f.x - vb * f.y);
                    a[u].v[e + 1] = from_f<T>(va * f.y + vb * f.x);
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 f = w[e];
                    const float va = to_f(a[u].v[e]), vb = to_f(b[u].v[e]);
                    a[u].v[e] = from_f<T>(va * f.x - vb * f.y);
                    b[u].v[e] = from_f<T>(va * f.y + vb * f.x);
                }
                *reinterpret_cast<VT *>(dst + partner) = b[u];
            }
        }
        *reinterpret_cast<VT *>(dst) = a[u];
    }
}

namespace {

template <typename T, bool kInter, int V>
cudaError_t launch_rope_as(RopeParams p, int n_tokens, cudaStream_t stream) {
    p.per_head = (kInter && V > 1 ? p.r.rot_dim / V : p.r.rot_dim / 2 / V) + (p.copy ? (p.dim - p.r.rot_dim) / V : 0);
    p.lanes = std::min(p.per_head, kRopeThreads);
    // as many heads at a time as threads allow, fewer when the token is short
    p.rows = std::max(1, std::min(kRopeThreads / p.lanes, (p.heads + kUnits - 1) / kUnits));
    const int threads = (p.rows * p.lanes + 31) / 32 * 32;
    const int ny = (p.heads + p.rows * kUnits - 1) / (p.rows * kUnits), nz = (p.per_head + p.lanes - 1) / p.lanes;
    if (ny > 65535 || nz > 65535) return cudaErrorInvalidConfiguration;
    rope_kernel<T, kInter, V><<<dim3((unsigned)n_tokens, (unsigned)ny, (unsigned)nz), threads, 0, stream>>>(p);
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
