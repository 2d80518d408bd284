// sparse_attn_q8.cu -- sparse MLA attention over selected rows of the 8-bit
// latent cache (quant8.cuh has the row's format):
//     z_j = sm_scale * (q_lat . c_j + q_rope . r_j),  o = sum_j softmax(z)_j c_j,
// c_j = 2^E_j codes_j[0:512], r_j = 2^E_j (hi_j + lo_j).
//
// The plain kernel: a CTA takes one token and eight heads, one warp per head;
// rows are decoded sixteen at a time into shared memory, and each warp keeps
// its head's query, running maximum, sum and output in registers.
#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "quant8.cuh"

namespace dsa {

namespace {

constexpr int kHeadsPerCta = 8;
constexpr int kChunk = 16;              // rows decoded at a time

}  // namespace

__global__ void __launch_bounds__(32 * kHeadsPerCta) sparse_attn_q8_kernel(const AttnQ8Launch p, const DevBatch b, uint32_t *status) {
    __shared__ float rows[kChunk][D_ROW];
    __shared__ int64_t at[kChunk];
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y * kHeadsPerCta + warp;
    const bool tail = p.q_rope != nullptr;
    const int pos = __ldg(b.q_pos + t);
    const int seq = seq_of_warp(b.cu_q, b.B, t, lane);
    const int64_t kv0 = seq_base(b, seq);
    int64_t own = -1;
    if (pos >= 0 && pos < b.max_kv && kv0 >= 0) own = cache_row(b, seq, kv0, pos);
    const bool ok = own >= 0 && own < b.cache_rows;
    if (!ok && threadIdx.x == 0 && blockIdx.y == 0) flag(status, DSA_DEV_BAD_POSITION);
    float q[18], acc[16], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    const int64_t qrow = (int64_t)t * p.H + h;
    if (h < p.H) {
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = __bfloat162float(__ushort_as_bfloat16(p.q_lat[qrow * D_L + lane + 32 * i]));
#pragma unroll
        for (int i = 0; i < 2; ++i) q[16 + i] = tail ? __bfloat162float(__ushort_as_bfloat16(p.q_rope[qrow * D_R + lane + 32 * i])) : 0.f;
    }
    const int width = tail ? kQ8Row : D_L;
    for (int j0 = 0; ok && j0 < p.k; j0 += kChunk) {
        const int n = min(kChunk, p.k - j0);
        if (threadIdx.x < kChunk) {
            int64_t row = -1;
            const int v = (int)threadIdx.x < n ? __ldg(p.idx + (int64_t)t * p.k + j0 + threadIdx.x) : -1;
            if (v >= 0 && v <= pos) row = cache_row(b, seq, kv0, v);
            if (row >= b.cache_rows) row = -1;
            if (row < 0 && v != -1 && blockIdx.y == 0) flag(status, DSA_DEV_BAD_INDEX);
            at[threadIdx.x] = row;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n * D_ROW; i += 32 * kHeadsPerCta) {
            const int r = i / D_ROW, d = i - r * D_ROW;
            const int64_t row = at[r];
            float v = 0.f;
            if (row >= 0 && (tail || d < D_L)) {
                const uint8_t *src = p.codes + row * width;
                v = e4m3x2_to_float2(src[d]).x;
                if (d >= D_L) v += e4m3x2_to_float2(src[d + D_R]).x;
                v *= p.scale[row];
            }
            rows[r][d] = v;
        }
        __syncthreads();
        if (h < p.H) {
            for (int r = 0; r < n; ++r) {
                if (at[r] < 0) continue;
                float z = 0.f, c[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) { c[i] = rows[r][lane + 32 * i]; z += c[i] * q[i]; }
                z += rows[r][D_L + lane] * q[16] + rows[r][D_L + lane + 32] * q[17];
#pragma unroll
                for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
                z *= p.sm_scale;
                const float mn = fmaxf(m, z), al = __expf(m - mn), w = __expf(z - mn);
                l = l * al + w;
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = acc[i] * al + w * c[i];
                m = mn;
            }
        }
        __syncthreads();
    }
    if (h >= p.H) return;
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t o = qrow * D_L + lane + 32 * i;
        if (p.out_bf16) static_cast<uint16_t *>(p.out)[o] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i] * inv));
        else static_cast<float *>(p.out)[o] = acc[i] * inv;
    }
    if (p.lse && lane == 0) p.lse[qrow] = l > 0.f ? m + logf(l) : -INFINITY;
}

cudaError_t launch_sparse_attn_q8(const AttnQ8Launch &a, const DevBatch &b, uint32_t *status, cudaStream_t stream, bool pdl) {
    (void)pdl;
    dim3 grid((unsigned)b.T, (unsigned)((a.H + kHeadsPerCta - 1) / kHeadsPerCta));
    sparse_attn_q8_kernel<<<grid, 32 * kHeadsPerCta, 0, stream>>>(a, b, status);
    return cudaGetLastError();
}

}  // namespace dsa
