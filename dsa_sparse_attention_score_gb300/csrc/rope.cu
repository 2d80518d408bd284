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
// unit of kUnits heads, so that its place in a head and its angles
// are found once, and its loads are out before the angles are formed (rot_dim
// / 2 of them, once per CTA).  Rows whose addresses or extents are not
// multiples of 16 bytes take the same kernel with units of one value.
// In and out of HBM, on the device: 4096 tokens x 128 heads x 64 values, pairs of
// neighbours, 22.3 us (6.0 TB/s); 4093 x 64 heads of 128, halves of the first 64
// turned and the rest copied, 25.2 us (5.3 TB/s).
#include <algorithm>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "rope.cuh"

namespace dsa {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kUnits = 4;              // heads per thread
constexpr int kMaxPairs = 256;         // rot_dim <= 512

// Two neighbouring values at a time: packed conversions run at twice to four
// times the rate of single ones.
template <typename T> struct Two;
template <> struct Two<float> {
    using P = float2;
    static __device__ __forceinline__ float2 get(P v) { return v; }
    static __device__ __forceinline__ P put(float a, float b) { return make_float2(a, b); }
    static __device__ __forceinline__ float one(float v) { return v; }
    static __device__ __forceinline__ float back(float v) { return v; }
};
template <> struct Two<__half> {
    using P = __half2;
    static __device__ __forceinline__ float2 get(P v) { return __half22float2(v); }
    static __device__ __forceinline__ P put(float a, float b) { return __floats2half2_rn(a, b); }
    static __device__ __forceinline__ float one(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half back(float v) { return __float2half_rn(v); }
};
template <> struct Two<__nv_bfloat16> {
    using P = __nv_bfloat162;
    static __device__ __forceinline__ float2 get(P v) { return __bfloat1622float2(v); }
    static __device__ __forceinline__ P put(float a, float b) { return __floats2bfloat162_rn(a, b); }
    static __device__ __forceinline__ float one(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 back(float v) { return __float2bfloat16_rn(v); }
};

// V values as V / 2 pairs, or a single one.
template <typename T, int V> struct alignas(sizeof(T) * V) Vec { typename Two<T>::P v[V / 2]; };
template <typename T> struct Vec<T, 1> { T v[1]; };

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

// Place of angle j: one entry free after every eight, so that threads reading
// runs of four or eight angles each do so without bank conflicts.
constexpr __host__ __device__ int padded(int j) { return j + (j >> 3); }

// V values per unit.  Interleaved: a unit is V neighbouring values, pairs
// inside it.  Halves: a unit is V values of either half, and its partner's
// values are read a second time (from L1), so that a head's loads and stores
// stay whole lines; with units of both halves, whose loads are half lines for
// 64 16-bit values, the same tokens took a quarter longer (37 us against 30,
// both before later steps).  V = 1: a pair, or one copied value.  grid: token,
// block of heads, block of a head's units.
template <typename T, bool kInter, int V>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const RopeParams p) {
    __shared__ float2 cs[padded(kMaxPairs)];
    using VT = Vec<T, V>;
    using W = Two<T>;
    constexpr bool kBoth = !kInter || V == 1;            // a rotated unit needs two loads
    constexpr int kPairs = kInter && V > 1 ? V / 2 : V;  // angles of a rotated unit
    pdl_wait();
    const int t = blockIdx.x, tid = threadIdx.x;
    const int half = p.r.rot_dim >> 1;
    const int rot_units = V > 1 ? p.r.rot_dim / V : half;
    const int row = tid / p.lanes, r = blockIdx.z * p.lanes + tid - row * p.lanes;
    const int h0 = blockIdx.y * (p.rows * kUnits) + row;
    const bool live = row < p.rows && r < p.per_head, turns = r < rot_units;
    const bool second = !kInter && V > 1 && r * V >= half;       // a unit of the second half
    const int c = (r - rot_units) * V;                   // a copied unit's place among the copied values
    const int v = turns ? p.off + r * (kInter && V == 1 ? 2 : V) : c < p.off ? c : c + p.r.rot_dim;
    const int partner = kInter ? 1 : second ? -half : half;
    const T *x = static_cast<const T *>(p.x) + (int64_t)t * p.xt + v;
    T *y = static_cast<T *>(p.y) + (int64_t)t * p.yt + v;
    VT a[kUnits], b[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int h = h0 + u * p.rows;
        if (live && h < p.heads) {
            a[u] = *reinterpret_cast<const VT *>(x + (int64_t)h * p.xh);
            if (kBoth && turns) b[u] = *reinterpret_cast<const VT *>(x + (int64_t)h * p.xh + partner);
        }
    }
    const int32_t pos = __ldg(p.pos + t);
    for (int j = tid; j < half; j += blockDim.x) cs[padded(j)] = rope_cos_sin(pos, __ldg(p.r.inv_freq + j), p.r.scale, p.r.inverse);
    __syncthreads();                                     // also: every load of the heads is done (x may be y)
    if (!live) return;
    float2 w[kPairs];
    if (turns) {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            w[e] = cs[padded(r * kPairs + e - (second ? half : 0))];
            if (second) w[e].y = -w[e].y;
        }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int h = h0 + u * p.rows;
        if (h >= p.heads) break;
        T *dst = y + (int64_t)h * p.yh;
        if (turns) {
            if constexpr (V == 1) {
                const float va = W::one(a[u].v[0]), vb = W::one(b[u].v[0]);
                a[u].v[0] = W::back(va * w[0].x - vb * w[0].y);
                dst[partner] = W::back(va * w[0].y + vb * w[0].x);
            } else {
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const float2 z = W::get(a[u].v[e]);
                    if constexpr (kInter) {
                        a[u].v[e] = W::put(z.x * w[e].x - z.y * w[e].y, z.x * w[e].y + z.y * w[e].x);
                    } else {
                        const float2 q = W::get(b[u].v[e]);
                        a[u].v[e] = W::put(z.x * w[2 * e].x - q.x * w[2 * e].y, z.y * w[2 * e + 1].x - q.y * w[2 * e + 1].y);
                    }
                }
            }
        }
        *reinterpret_cast<VT *>(dst) = a[u];
    }
}

namespace {

template <typename T, bool kInter, int V>
cudaError_t launch_rope_as(RopeParams p, int n_tokens, cudaStream_t stream) {
    p.per_head = (V > 1 ? p.r.rot_dim / V : p.r.rot_dim / 2) + (p.copy ? (p.dim - p.r.rot_dim) / V : 0);
    p.lanes = std::min(p.per_head, kRopeThreads);
    // as many heads at a time as threads allow, fewer when the token is short
    p.rows = std::max(1, std::min(kRopeThreads / p.lanes, (p.heads + kUnits - 1) / kUnits));
    const int threads = (p.rows * p.lanes + 31) / 32 * 32;
    const int ny = (p.heads + p.rows * kUnits - 1) / (p.rows * kUnits), nz = (p.per_head + p.lanes - 1) / p.lanes;
    if (ny > 65535 || nz > 65535) return cudaErrorInvalidConfiguration;
    return launch_k(rope_kernel<T, kInter, V>, dim3((unsigned)n_tokens, (unsigned)ny, (unsigned)nz), dim3((unsigned)threads), 0,
                    stream, true, p);
}

template <typename T>
cudaError_t launch_rope_t(const RopeParams &p, int n_tokens, cudaStream_t stream) {
    // Units of 16 bytes: every address and every extent a multiple of that.
    constexpr int V = 16 / sizeof(T);
    const int64_t any = p.xt | p.xh | p.yt | p.yh | p.dim | p.off | p.r.rot_dim | (p.r.interleaved ? 0 : p.r.rot_dim / 2);
    const bool vec = any % V == 0 && ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.y)) & 15) == 0;
    if (p.r.interleaved)
        return vec ? launch_rope_as<T, true, V>(p, n_tokens, stream) : launch_rope_as<T, true, 1>(p, n_tokens, stream);
    // (halves: a head's units stay in one CTA, see rope_kernel)
    return vec && p.dim / V <= kRopeThreads ? launch_rope_as<T, false, V>(p, n_tokens, stream) : launch_rope_as<T, false, 1>(p, n_tokens, stream);
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
