// sparse_attn_q8.cu -- sparse MLA attention over selected rows of the 8-bit
// latent cache (quant8.cuh has the row's format):
//     z_j = sm_scale * (q_lat . c_j + q_rope . r_j),  o = sum_j softmax(z)_j c_j,
// c_j = 2^E_j codes_j[0:512], r_j = 2^E_j (hi_j + lo_j).
//
// The tensor cores read the codes as they lie in the cache; no row is ever
// decoded.  What makes that possible:
//  - The row's scale leaves both contractions.  z_j = 2^E_j (codes_j . q), and
//    with u_j = z_j log2(e) + E_j the output is sum_j 2^(u_j - M) codes_j over
//    l = sum_j 2^(z_j log2(e) - M): the scale is folded into the weights (E_j = log2 of the scale: a power of two is not
//    needed here).
//  - A bf16 query is the sum of two e4m3 pieces: q 2^-e = hi + lo with
//    hi = e4m3(q 2^-e), lo = e4m3(q 2^-e - hi).  Four significant bits each,
//    the remainder signed, hold bf16's eight: the split is exact for values
//    above 2^-10 of the head's largest, and off by 2^-19 of it below.
//  - A weight is split the same way, in units where the largest lies in
//    [2^3.5, 2^8]: each is off by at most 2^-8 of itself (half a bf16 step) or
//    2^-13.5 of the largest.
// So every product is 8-bit by 8-bit with float32 sums, at twice the rate of
// bf16 products and half the bytes: the two pieces cost what one bf16 product
// would, and the rows come in at 644 bytes instead of 1152.
//
// One CTA per (token, head group of 64, split) walks tiles of 128 selected
// rows.  A tile is five 16 KB blocks of 128 rows x 128 bytes (SWIZZLE_128B):
// four of latent codes, one of the tail (64 hi | 64 lo).
//     S^T[row, piece*head]  = C[row, :] . Q[piece*head, :]^T   M=128, N=128, K=512 + 128
//     O^T[dim, head]       += C[row, dim]^T . P^T[row, head]   4 x M=128, N=64, K=128, both pieces
// The same bytes are the K-major A operand of S^T and the MN-major A operand
// of O^T.  The tail's two halves multiply the same 64 query values, so its
// four K steps read the two of q_rope twice.  S^T accumulates a head's two
// pieces in columns h and 64 + h, which the softmax adds; O^T adds both pieces of
// P^T in place.  The tail block is dead once S^T is computed and holds P^T.
//
// Shared memory: queries 72 KB and a ring of nine blocks (144 KB), one short
// of two tiles: a tile's tail block goes in when the first value product of
// the tile before has freed its slot.  One producer warp per latent block
// gathers it with 16-byte cp.async copies (a row's 128 bytes are one cache
// line; masked rows are filled with zeros and read nothing); four more hold
// the tail block in registers until its slot is free.  The MMA thread issues score blocks and value
// products as their inputs arrive; sixteen softmax warps (four per TMEM lane
// quarter, 16 heads each) turn a tile's S^T into P^T.  The reference M of a
// head's weights is set 2^3.5 below its first tile's maximum and moves only
// when a weight would exceed 2^8, so most tiles need no maxima, only the
// question whether any weight does.
#include <cstddef>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "quant8.cuh"

namespace dsa {

namespace {

constexpr int kHeads = 64;                    // heads per CTA (padded)
constexpr int kRows = 128;                    // selected rows per tile
constexpr int kBlockBytes = kRows * 128;      // 16 KB
constexpr int kTileBlocks = 5;                // 4 latent + the tail (P^T)
constexpr int kSlots = 9;
constexpr int kQBlockBytes = 2 * kHeads * 128;        // hi and lo rows of 128 codes
constexpr int kQTailBytes = 2 * kHeads * 64;          // hi and lo rows of 64 codes (SWIZZLE_64B)
constexpr int kQBytes = 4 * kQBlockBytes + kQTailBytes;
constexpr int kPieceBytes = kRows * 64;       // one piece of P^T (SWIZZLE_64B)
constexpr int kParts = 4;                     // groups of 16 heads
constexpr int kPartHeads = kHeads / kParts;
constexpr int kSoftmaxWarps = 4 * kParts;     // one per (TMEM lane quarter, part)
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kMmaWarp = kSoftmaxWarps;
constexpr int kTailWarps = 4;                 // 32 rows of the tail block each
constexpr int kProducerWarps = 4 + kTailWarps;   // warps 17..20: a latent block each; 21..24: the tail
constexpr int kThreads = 32 * (kSoftmaxWarps + 1 + kProducerWarps);
constexpr float kTopLog2 = 3.5f;              // a new maximum's weight is 2^3.5 ...
constexpr float kRaiseLog2 = 8.0f;            // ... and none exceeds 2^8
constexpr int kFewMoved = 4;                  // heads of 16 rescaled one by one
constexpr float kMinScale = 0x1p-40f;
constexpr uint32_t kTmemCols = 512;           // S^T: 2 x 128 columns, O^T: 4 x 64
constexpr uint32_t kColS = 0;
constexpr uint32_t kColO = 256;

struct Params {
    const uint16_t *q_lat, *q_rope;
    const uint8_t *codes;
    const float *scale;
    const int32_t *idx;
    void *out;
    float *lse;
    uint16_t *part_o;        // [T, n_split, groups, 64, 512] bf16, unnormalised
    float *part_ml;          // [T, n_split, groups, 64, 2]
    DevBatch b;
    uint32_t *status;
    int H, k, groups, out_bf16;
    float scale_log2;        // sm_scale * log2(e)
    int tiles_per_cta, n_split, n_tiles;
};

struct Ctl {
    uint64_t q_full;
    uint64_t full[kSlots];
    uint64_t empty[kSlots];
    uint64_t s_full[2];
    uint64_t p_full[2];
    uint64_t o_full[2];      // by tile parity: tile i's completes after tile i - 2's has been waited for
    uint32_t tmem_base;
    int32_t abort_flag;
    alignas(16) float qs[kHeads];   // 2^e of the head's query times scale_log2
    float red[4][kHeads];    // a tile's maxima by lane quarter; the row sums at the end
    alignas(16) float ma[kSoftmaxWarps][2 * kPartHeads];   // each warp's -m, and how far m moved
    int32_t warp_alive[kSoftmaxWarps];
};

// qs and ma are read four at a time
static_assert(offsetof(Ctl, qs) % 16 == 0 && offsetof(Ctl, ma) % 16 == 0 && (2 * kPartHeads * 4) % 16 == 0 &&
                  (kSlots * kBlockBytes + kQBytes) % 16 == 0, "16-byte reads of shared memory");

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, Ctl &c, uint32_t *status, uint64_t limit_ns) {
    if (*(volatile int32_t *)&c.abort_flag) return false;
    if (mbar_wait(bar, parity, limit_ns)) return true;
    *(volatile int32_t *)&c.abort_flag = 1;
    flag(status, DSA_DEV_TIMEOUT);
    return false;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));   // volatile: stays where the warp is whole
    return r;
}

// Transposing butterfly: each lane holds 16 values, lane L ends up with the
// sum of value L mod 16 over the warp.
__device__ __forceinline__ float warp_sum_16(const float (&x)[16], int lane) {
    float a[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i] = x[i];
#pragma unroll
    for (int half = 8; half >= 1; half >>= 1) {
        const bool up = lane & half;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < half) {
                const float keep = up ? a[half + i] : a[i];
                const float send = up ? a[i] : a[half + i];
                a[i] = keep + __shfl_xor_sync(0xffffffffu, send, half);
            }
        }
    }
    return a[0] + __shfl_xor_sync(0xffffffffu, a[0], 16);
}

// 16 bf16 values in two words of four.
__device__ __forceinline__ void bf16x16(const uint4 &a, const uint4 &b, float (&v)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// The two e4m3 pieces of sixteen values.
__device__ __forceinline__ void split16(const float (&v)[16], float inv, uint4 &hi, uint4 &lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = v[4 * i] * inv, b = v[4 * i + 1] * inv, c = v[4 * i + 2] * inv, d = v[4 * i + 3] * inv;
        const uint32_t h0 = e4m3x2(a, b), h1 = e4m3x2(c, d);
        const float2 f0 = e4m3x2_to_float2(h0), f1 = e4m3x2_to_float2(h1);
        h[i] = h0 | h1 << 16;
        l[i] = e4m3x2(a - f0.x, b - f0.y) | e4m3x2(c - f1.x, d - f1.y) << 16;
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1) sparse_attn_q8_kernel(const Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *ring = base;
    uint8_t *q_s = base + kSlots * kBlockBytes;          // four latent blocks, then the tail's
    Ctl &ctl = *reinterpret_cast<Ctl *>(q_s + kQBytes);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const DevBatch &b = p.b;
    const int t = blockIdx.x / p.groups;
    const int hg = blockIdx.x - t * p.groups;
    const int h0 = hg * kHeads, nh = min(kHeads, p.H - h0);
    const int split = blockIdx.y;
    const bool tail = p.q_rope != nullptr;
    const int width = tail ? kQ8Row : D_L;               // bytes per cached row
    const int64_t part_idx = ((int64_t)t * p.n_split + split) * p.groups + hg;
    tl_start(b.timeline, kTlAttn);
    const int pos = __ldg(b.q_pos + t);
    const int seq = seq_of_warp(b.cu_q, b.B, t, lane);
    const int64_t kv0 = seq_base(b, seq);
    const int tile_lo = split * p.tiles_per_cta;
    const int tile_hi = min(p.n_tiles, tile_lo + p.tiles_per_cta);
    int64_t own_row = -1;
    if (pos >= 0 && pos < b.max_kv && kv0 >= 0) own_row = cache_row(b, seq, kv0, pos);
    const bool pos_ok = own_row >= 0 && own_row < b.cache_rows;
    if (!pos_ok || tile_lo >= tile_hi) {
        if (!pos_ok && threadIdx.x == 0 && split == 0) flag(p.status, DSA_DEV_BAD_POSITION);
        if (p.n_split > 1) {
            for (int i = threadIdx.x; i < kHeads * D_L / 2; i += kThreads)
                reinterpret_cast<uint32_t *>(p.part_o + part_idx * kHeads * D_L)[i] = 0u;
            if (threadIdx.x < kHeads) {
                float *ml = p.part_ml + (part_idx * kHeads + threadIdx.x) * 2;
                ml[0] = -INFINITY;
                ml[1] = 0.f;
            }
        } else {
            const int64_t o = ((int64_t)t * p.H + h0) * D_L;
            for (int i = threadIdx.x; i < nh * D_L; i += kThreads) {
                if (p.out_bf16) static_cast<uint16_t *>(p.out)[o + i] = 0;
                else static_cast<float *>(p.out)[o + i] = 0.f;
            }
            if (p.lse && threadIdx.x < nh) p.lse[(int64_t)t * p.H + h0 + threadIdx.x] = -INFINITY;
        }
        return;
    }
    const int n_my = tile_hi - tile_lo;

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&ctl.q_full), kSoftmaxWarps);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_u32(&ctl.full[i]), 32);
            mbar_init(smem_u32(&ctl.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl.s_full[i]), 1);
            mbar_init(smem_u32(&ctl.p_full[i]), kSoftmaxWarps);
        }
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&ctl.o_full[i]), 1);
        ctl.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&ctl.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;
    const int32_t *idx_row = p.idx + (int64_t)t * p.k;
    // Cache row of entry e of the token's selection: -1 for padding and for
    // entries out of range (flagged by one thread per entry).
    auto row_of = [&](int e, bool report) -> int32_t {
        const int32_t v = e < p.k ? __ldg(idx_row + e) : -1;
        int64_t row = -1;
        if (v >= 0 && v <= pos) row = cache_row(b, seq, kv0, v);
        if (row >= b.cache_rows) row = -1;
        if (row < 0 && v != -1 && report) flag(p.status, DSA_DEV_BAD_INDEX);
        return (int32_t)row;
    };

    if (warp > kMmaWarp) {
        // ---------------- producers
        const int pw = warp - kMmaWarp - 1;
        const int j = min(pw, 4);                    // the warp's block of the tile
        const uint8_t *src = p.codes + j * 128 + (lane & 7) * 16;
        // lane's chunk of rows 4 g + lane / 8; g odd flips bit 2 of the swizzled chunk
        const uint32_t d0 = sw128_offset((uint32_t)(lane >> 3), (uint32_t)(lane & 7));
        pdl_wait();                                  // the indices come from the preceding kernel
        if (pw < 4) {
            // a latent block: asynchronous copies into its slot
            for (int it = 0; it < n_my; ++it) {
                const uint32_t n = (uint32_t)(kTileBlocks * it + j), slot = n % kSlots, use = n / kSlots;
                int32_t my_row[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) my_row[q] = row_of((tile_lo + it) * kRows + 32 * q + lane, j == 0);
                if (!wait_bar(smem_u32(&ctl.empty[slot]), (use & 1u) ^ 1u, ctl, p.status, b.wait_ns)) break;
                if (b.skip_copies) continue;
                const uint32_t dst = smem_u32(ring + slot * kBlockBytes) + d0;
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int g = 0; g < 8; ++g) {
                        const int32_t row = __shfl_sync(0xffffffffu, my_row[q], 4 * g + (lane >> 3));
                        cp_async16_or_zero((dst + (uint32_t)(8 * q + g) * 512u) ^ ((uint32_t)(g & 1) << 6),
                                           src + (int64_t)max(row, 0) * width, row < 0 ? 0u : 16u);
                    }
                cp_async_commit();
                cp_async_wait_all();
                fence_proxy_async_smem();
                mbar_arrive(smem_u32(&ctl.full[slot]));
            }
        } else {
            // The tail block, whose slot frees last: its rows wait in
            // registers, so that only the stores lie between the free slot
            // and the score product.  Rows without a tail have nothing to
            // gather: the warps only pass the free slot on to the softmax,
            // which puts P^T there.
            const int r0 = 32 * (pw - 4);
            for (int it = 0; it < n_my; ++it) {
                const uint32_t n = (uint32_t)(kTileBlocks * it + 4), slot = n % kSlots, use = n / kSlots;
                uint4 v[8];
                if (tail) {
                    const int32_t my_row = row_of((tile_lo + it) * kRows + r0 + lane, false);
#pragma unroll
                    for (int g = 0; g < 8; ++g) {
                        const int32_t row = __shfl_sync(0xffffffffu, my_row, 4 * g + (lane >> 3));
                        v[g] = make_uint4(0u, 0u, 0u, 0u);
                        if (row >= 0) v[g] = __ldg(reinterpret_cast<const uint4 *>(src + (int64_t)row * width));
                    }
                }
                if (!wait_bar(smem_u32(&ctl.empty[slot]), (use & 1u) ^ 1u, ctl, p.status, b.wait_ns)) break;
                if (b.skip_copies) continue;
                if (tail) {
                    uint8_t *dst = ring + slot * kBlockBytes + r0 * 128;
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                        *reinterpret_cast<uint4 *>(dst + ((d0 + (uint32_t)g * 512u) ^ ((uint32_t)(g & 1) << 6))) = v[g];
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane < 32 / kTailWarps) mbar_arrive(smem_u32(&ctl.full[slot]));
            }
        }
    } else if (warp == kMmaWarp) {
        // ---------------- MMA issuer, in a fixed order per tile:
        //   S(i + 1) latent blocks | P^T(i) | O(i) block 0 | S(i + 1) tail | O(i) blocks 1..3
        // The first value-product block frees the slot that the next tile's
        // tail needs; the rest of the value product runs beside the next
        // softmax.  Polling for whichever input came first instead cost 360 to
        // 600 cycles of bookkeeping per block against 300 to 460 of products.
        // The whole warp runs the loop (uniform descriptors); one elected
        // lane issues.
        const uint32_t id_s = idesc_e4m3(kRows, 2 * kHeads, false, false);
        const uint32_t id_o = idesc_e4m3(128, kHeads, true, true);
        const uint32_t ra = smem_u32(ring), qa = smem_u32(q_s), full0 = smem_u32(&ctl.full[0]), empty0 = smem_u32(&ctl.empty[0]);
        const uint64_t s_a0 = sdesc_sw128(ra, 16, 1024), s_b0 = sdesc_sw128(qa, 16, 1024);
        const uint64_t s_bt = sdesc_sw64(qa + 4 * kQBlockBytes, 16, 512);
        const uint64_t o_b0 = sdesc_sw64(ra, 16, 512);
        auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
            const bool ok = __all_sync(0xffffffffu, wait_bar(bar, parity, ctl, p.status, b.wait_ns));
            tc_fence_after();
            return ok;
        };
        // Block j of tile i has number 5 i + j: slot and use follow from those
        // of the tile's first block (base, use0).
        auto score_block = [&](int j, uint32_t base, uint32_t use0, uint32_t d_s, uint64_t bd, uint32_t b2) -> bool {
            const uint32_t wrap = base + j >= kSlots ? 1u : 0u, slot = base + j - (wrap ? kSlots : 0u);
            if (!wait(full0 + 8 * slot, (use0 + wrap) & 1u)) return false;
            const uint64_t ad = s_a0 + (uint64_t)(slot * (kBlockBytes >> 4));
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    umma_f8(d_s, ad + (uint64_t)(ks * 2), bd + (uint64_t)((ks & 1) * 2) + (ks & 2 ? b2 : 0u), id_s, (j || ks) ? 1u : 0u);
            }
            __syncwarp();
            return true;
        };
        auto score_latent = [&](int it, uint32_t base, uint32_t use0) -> bool {
            const uint32_t d_s = tmem + kColS + (it & 1) * 2 * kHeads;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (!score_block(j, base, use0, d_s, s_b0 + (uint64_t)(j * (kQBlockBytes >> 4)), 4)) return false;
            if (!tail && elect_one()) umma_commit(smem_u32(&ctl.s_full[it & 1]));
            __syncwarp();
            return true;
        };
        auto score_tail = [&](int it, uint32_t base, uint32_t use0) -> bool {
            if (!tail) return true;
            // K steps 2 and 3, the remainders, read the query again
            if (!score_block(4, base, use0, tmem + kColS + (it & 1) * 2 * kHeads, s_bt, 0)) return false;
            if (elect_one()) umma_commit(smem_u32(&ctl.s_full[it & 1]));
            __syncwarp();
            return true;
        };
        bool go = wait(smem_u32(&ctl.q_full), 0) && score_latent(0, 0, 0) && score_tail(0, 0, 0);
        uint32_t base = 0, use0 = 0;
        for (int it = 0; go && it < n_my; ++it) {
            const uint32_t wrap = base + kTileBlocks >= kSlots ? 1u : 0u;
            const uint32_t next = base + kTileBlocks - (wrap ? kSlots : 0u), next_use = use0 + wrap;
            const bool more = it + 1 < n_my;
            if (more) go = score_latent(it + 1, next, next_use);
            go = go && wait(smem_u32(&ctl.p_full[it & 1]), (uint32_t)(it >> 1) & 1u);
            if (!go) break;
            const uint32_t pslot = base + 4 - (base + 4 >= kSlots ? kSlots : 0u);
            const uint64_t bd = o_b0 + (uint64_t)(pslot * (kBlockBytes >> 4));
            const uint32_t acc0 = it > 0 ? 1u : 0u;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t slot = base + c - (base + c >= kSlots ? kSlots : 0u);
                const uint64_t ad = s_a0 + (uint64_t)(slot * (kBlockBytes >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int piece = 0; piece < 2; ++piece)
#pragma unroll
                        for (int ks = 0; ks < kRows / 32; ++ks)
                            umma_f8(tmem + kColO + c * kHeads, ad + (uint64_t)(ks * (32 * 128 >> 4)),
                                    bd + (uint64_t)(piece * (kPieceBytes >> 4) + ks * (32 * 64 >> 4)), id_o, (piece || ks) ? 1u : acc0);
                    umma_commit(empty0 + 8 * slot);
                    if (c == 3) {
                        umma_commit(empty0 + 8 * pslot);
                        umma_commit(smem_u32(&ctl.o_full[it & 1]));
                    }
                }
                __syncwarp();
                if (c == 0 && more) go = score_tail(it + 1, next, next_use);
            }
            base = next;
            use0 = next_use;
        }
    } else {
        // ---------------- queries, softmax and epilogue (warps 0..15)
        const int quarter = warp & 3;                      // TMEM lanes 32*quarter ..
        const int part = warp >> 2;                        // heads 16*part ..
        const int hb = kPartHeads * part;
        const int r = quarter * 32 + lane;                 // row within the tile
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        float *ma = ctl.ma[warp];
        // each warp splits four heads' queries: lane l the values 16 l .. 16 l + 15
#pragma unroll 2
        for (int i = 0; i < kHeads / kSoftmaxWarps; ++i) {
            const int h = warp * (kHeads / kSoftmaxWarps) + i;
            uint4 a = make_uint4(0u, 0u, 0u, 0u), c = a, ra = a, rc = a;
            if (h < nh) {
                const int64_t row = (int64_t)t * p.H + h0 + h;
                const uint4 *src = reinterpret_cast<const uint4 *>(p.q_lat + row * D_L) + 2 * lane;
                a = __ldg(src);
                c = __ldg(src + 1);
                if (tail && lane < 4) {
                    const uint4 *rs = reinterpret_cast<const uint4 *>(p.q_rope + row * D_R) + 2 * lane;
                    ra = __ldg(rs);
                    rc = __ldg(rs + 1);
                }
            }
            float v[16], w[16];
            bf16x16(a, c, v);
            bf16x16(ra, rc, w);
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 16; ++k) top = max(top, max(__float_as_uint(v[k]) & 0x7FFFFFFFu, __float_as_uint(w[k]) & 0x7FFFFFFFu));
            top = __reduce_max_sync(0xffffffffu, top);
            const int e = q8_exponent(__uint_as_float(top));
            const float inv = exp2_int(-e);
            uint4 hi, lo;
            split16(v, inv, hi, lo);
            uint8_t *blk = q_s + (lane >> 3) * kQBlockBytes;
            *reinterpret_cast<uint4 *>(blk + sw128_offset((uint32_t)h, (uint32_t)(lane & 7))) = hi;
            *reinterpret_cast<uint4 *>(blk + sw128_offset((uint32_t)(kHeads + h), (uint32_t)(lane & 7))) = lo;
            if (lane < 4) {
                split16(w, inv, hi, lo);
                uint8_t *tb = q_s + 4 * kQBlockBytes;
                *reinterpret_cast<uint4 *>(tb + sw64_offset((uint32_t)h, (uint32_t)lane)) = hi;
                *reinterpret_cast<uint4 *>(tb + sw64_offset((uint32_t)(kHeads + h), (uint32_t)lane)) = lo;
            }
            if (lane == 0) ctl.qs[h] = h < nh ? exp2_int(e) * p.scale_log2 : 0.f;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.q_full));
        pdl_wait();
        bool alive = true;
        named_barrier(1, kSoftmaxThreads);
        uint64_t lpart[8];                                 // row sums of l, two heads each
#pragma unroll
        for (int h = 0; h < 8; ++h) lpart[h] = f2(0.f, 0.f);
        // lane h < 16: the reference m of head hb + h, 3.5 to 8 below its
        // largest u so far (the same in the four warps of the part); 0 as long
        // as every row was masked (fresh)
        float m = 0.f;
        bool fresh = true;
        if (lane < 16) ma[lane] = 0.f;
        __syncwarp();
        // Scale of this thread's row of a tile (0: masked), looked up a tile
        // ahead.  Any positive scale will do; a row never written (scale 0)
        // counts as zeros at the smallest one.
        auto scale_of = [&](int it) -> float {
            const int32_t row = row_of((tile_lo + it) * kRows + r, false);
            if (row < 0) return 0.f;
            const float s = __ldg(p.scale + row);
            return s < kMinScale ? kMinScale : s;
        };
        float next_scale = scale_of(0);
        // Every softmax thread runs the same sequence of named barriers whatever
        // happens; `alive` (warp-uniform) only gates tensor-memory and shared
        // memory work after a bounded wait gave up.
        for (int it = 0; it < n_my; ++it) {
            const int buf = it & 1;
            const float rs = next_scale;
            if (it + 1 < n_my) next_scale = scale_of(it + 1);
            const bool valid = rs != 0.f;                  // a masked row's products are 0: u = -inf
            const float ef = valid ? log2f(rs) : -INFINITY;
            const float irs = valid ? 1.f / rs : 0.f;
            const uint64_t rs2 = f2(rs, rs), ef2 = f2(ef, ef), irs2 = f2(irs, irs);
            if (alive) alive = wait_bar(smem_u32(&ctl.s_full[buf]), (uint32_t)(it >> 1) & 1u, ctl, p.status, b.wait_ns);
            alive = __all_sync(0xffffffffu, alive);
            float x[16], top = -INFINITY;                  // u, then u - m
            if (alive) {
                tc_fence_after();
                uint32_t u[16], w[16];
                const uint32_t a = tmem + lane_addr + kColS + buf * 2 * kHeads + hb;
                tmem_ld16(a, u);
                tmem_ld16(a + kHeads, w);
                tmem_wait_ld(u, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 q4 = *reinterpret_cast<const float4 *>(ctl.qs + hb + 4 * i);
                    const float4 n4 = *reinterpret_cast<const float4 *>(ma + 4 * i);
                    const uint64_t qs[2] = {f2(q4.x, q4.y), f2(q4.z, q4.w)}, nm[2] = {f2(n4.x, n4.y), f2(n4.z, n4.w)};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int h = 4 * i + 2 * j;
                        const uint64_t a2 = f2(__uint_as_float(u[h]), __uint_as_float(u[h + 1]));
                        const uint64_t b2 = f2(__uint_as_float(w[h]), __uint_as_float(w[h + 1]));
                        const float2 v = f2_get(f2_add(f2_fma(f2_mul(f2_add(a2, b2), rs2), qs[j], nm[j]), ef2));
                        x[h] = v.x;
                        x[h + 1] = v.y;
                        top = fmaxf(top, fmaxf(v.x, v.y));
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < 16; ++h) x[h] = -INFINITY;
            }
            // Does any weight of the part exceed 2^8?  Then the heads' maxima
            // are found and m moves where it has to; few tiles but a token's
            // first come here.
            uint32_t moved = 0;                            // heads of the part whose m moves
            if (named_barrier_or(2 + part, 128, fresh || top > kRaiseLog2)) {
                float wmax[16];
#pragma unroll
                for (int h = 0; h < 16; ++h) wmax[h] = warp_max(x[h]);
                float over = wmax[0];
#pragma unroll
                for (int h = 1; h < 16; ++h) over = (lane & 15) == h ? wmax[h] : over;
                if (lane < 16) ctl.red[quarter][hb + lane] = over;
                named_barrier(2 + part, 128);
                const int hl = hb + (lane & 15);
                over = fmaxf(fmaxf(ctl.red[0][hl], ctl.red[1][hl]), fmaxf(ctl.red[2][hl], ctl.red[3][hl]));
                const float up = (fresh ? over != -INFINITY : over > kRaiseLog2) ? over - kTopLog2 : 0.f;
                m += up;
                if (lane < 16) {
                    ma[lane] = -m;
                    ma[kPartHeads + lane] = up;
                }
                moved = fresh ? 0u : __ballot_sync(0xffffffffu, lane < 16 && up != 0.f);
                fresh = __all_sync(0xffffffffu, over == -INFINITY) && fresh;
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 16; ++h) x[h] -= ma[kPartHeads + h];
                if (moved) {
#pragma unroll
                    for (int h = 0; h < 8; ++h)
                        lpart[h] = f2_mul(lpart[h], f2(ex2(-ma[kPartHeads + 2 * h]), ex2(-ma[kPartHeads + 2 * h + 1])));
                }
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w[4] = {ex2(x[4 * i]), ex2(x[4 * i + 1]), ex2(x[4 * i + 2]), ex2(x[4 * i + 3])};
                lpart[2 * i] = f2_fma(f2(w[0], w[1]), irs2, lpart[2 * i]);
                lpart[2 * i + 1] = f2_fma(f2(w[2], w[3]), irs2, lpart[2 * i + 1]);
                // through fp16, whose 11 bits the two pieces cannot tell from 24
                const __half2 a = __floats2half2_rn(w[0], w[1]), c = __floats2half2_rn(w[2], w[3]);
                const uint32_t ha = e4m3x2(a), hc = e4m3x2(c);
                hi[i] = ha | hc << 16;
                lo[i] = e4m3x2(__hsub2(a, e4m3x2_to_half2(ha))) | e4m3x2(__hsub2(c, e4m3x2_to_half2(hc))) << 16;
            }
            const uint32_t pn = (uint32_t)(kTileBlocks * it + 4), pslot = pn % kSlots;
            if (!tail && alive) {
                // no score product has waited for this slot
                alive = wait_bar(smem_u32(&ctl.full[pslot]), (pn / kSlots) & 1u, ctl, p.status, b.wait_ns);
                alive = __all_sync(0xffffffffu, alive);
            }
            if (alive) {
                uint8_t *pb = ring + pslot * kBlockBytes + sw64_offset((uint32_t)r, (uint32_t)part);
                *reinterpret_cast<uint4 *>(pb) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(pb + kPieceBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            if (moved && it > 0) {
                // Columns of O^T whose maximum moved, once the previous tile's
                // value product has landed: one by one while they are few
                // (the usual tile moves one or two of 64 heads), else all.
                if (alive) alive = wait_bar(smem_u32(&ctl.o_full[(it - 1) & 1]), (uint32_t)((it - 1) >> 1) & 1u, ctl, p.status, b.wait_ns);
                alive = __all_sync(0xffffffffu, alive);
                if (alive) {
                    tc_fence_after();
                    const uint32_t o = tmem + lane_addr + kColO + hb;
                    if (__popc(moved) <= kFewMoved) {
                        while (moved) {
                            const int h = __ffs(moved) - 1;
                            moved &= moved - 1;
                            const float al = ex2(-ma[kPartHeads + h]);
                            uint32_t u[4];
#pragma unroll
                            for (int c = 0; c < 4; ++c) tmem_ld1(o + c * kHeads + h, u[c]);
                            tmem_wait_ld(u);
#pragma unroll
                            for (int c = 0; c < 4; ++c) tmem_st1(o + c * kHeads + h, __float_as_uint(__uint_as_float(u[c]) * al));
                        }
                    } else {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t u[16];
                            tmem_ld16(o + c * kHeads, u);
                            tmem_wait_ld(u);
#pragma unroll
                            for (int h = 0; h < 16; ++h) u[h] = __float_as_uint(__uint_as_float(u[h]) * ex2(-ma[kPartHeads + h]));
                            tmem_st16(o + c * kHeads, u);
                        }
                    }
                    tmem_wait_st();
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl.p_full[buf]));
        }
        // ---- final: O^T of the last tile, row sums, outputs
        if (alive) alive = wait_bar(smem_u32(&ctl.o_full[(n_my - 1) & 1]), (uint32_t)((n_my - 1) >> 1) & 1u, ctl, p.status, b.wait_ns);
        alive = __all_sync(0xffffffffu, alive);
        float lrow[16];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            const float2 v = f2_get(lpart[h]);
            lrow[2 * h] = v.x;
            lrow[2 * h + 1] = v.y;
        }
        const float lsum = warp_sum_16(lrow, lane);
        named_barrier(2 + part, 128);                      // red may still be read
        if (lane < 16) ctl.red[quarter][hb + lane] = lsum;
        if (lane == 0) ctl.warp_alive[warp] = alive ? 1 : 0;
        named_barrier(1, kSoftmaxThreads);
        const int hl = hb + (lane & 15);
        const float l = ctl.red[0][hl] + ctl.red[1][hl] + ctl.red[2][hl] + ctl.red[3][hl];
        if (lane < 16) ma[lane] = fresh ? 0.f : 1.f / l;
        __syncwarp();
        bool all_alive = true;
#pragma unroll
        for (int w = 0; w < kSoftmaxWarps; ++w) all_alive = all_alive && ctl.warp_alive[w];
        if (all_alive) {
            // thread (quarter, lane) holds output dim 128 c + 32 quarter + lane
            // of the part's heads
            tc_fence_after();
            const int rd = quarter * 32 + lane;
            const int64_t o = ((int64_t)t * p.H + h0) * D_L;
            uint16_t *po = p.n_split > 1 ? p.part_o + part_idx * kHeads * D_L : nullptr;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                const int d = c * 128 + rd;
                uint32_t u[16];
                tmem_ld16(tmem + lane_addr + kColO + c * kHeads + hb, u);
                tmem_wait_ld(u);
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int h = hb + q;
                    const float v = __uint_as_float(u[q]);
                    if (po) {
                        po[h * D_L + d] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                    } else if (h < nh) {
                        if (p.out_bf16) static_cast<uint16_t *>(p.out)[o + h * D_L + d] = __bfloat16_as_ushort(__float2bfloat16_rn(v * ma[q]));
                        else static_cast<float *>(p.out)[o + h * D_L + d] = v * ma[q];
                    }
                }
            }
            if (quarter == 0 && lane < 16) {
                const int h = hb + lane;
                if (po) {
                    float *ml = p.part_ml + (part_idx * kHeads + h) * 2;
                    ml[0] = fresh ? -INFINITY : m;
                    ml[1] = l;
                } else if (p.lse && h < nh) {
                    p.lse[(int64_t)t * p.H + h0 + h] = fresh ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                }
            }
        }
    }

    tc_fence_before();
    __syncwarp();
    __syncthreads();
    pdl_trigger();
    tl_end(b.timeline, kTlAttn);
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

int attn_q8_tile_rows() { return kRows; }

cudaError_t launch_sparse_attn_q8(const AttnQ8Launch &a, const DevBatch &b, uint32_t *status, cudaStream_t stream, bool pdl) {
    Params p{};
    p.q_lat = a.q_lat;
    p.q_rope = a.q_rope;
    p.codes = a.codes;
    p.scale = a.scale;
    p.idx = a.idx;
    p.out = a.out;
    p.lse = a.lse;
    p.part_o = a.part_o;
    p.part_ml = a.part_ml;
    p.b = b;
    p.status = status;
    p.H = a.H;
    p.k = a.k;
    p.groups = (a.H + kHeads - 1) / kHeads;
    p.out_bf16 = a.out_bf16;
    p.scale_log2 = a.sm_scale * 1.4426950408889634f;
    p.tiles_per_cta = a.tiles_per_cta;
    p.n_split = a.n_split;
    p.n_tiles = (a.k + kRows - 1) / kRows;
    const size_t smem = 1024 + kSlots * kBlockBytes + kQBytes + sizeof(Ctl);
    static_assert(1024 + kSlots * kBlockBytes + kQBytes + sizeof(Ctl) <= 232448, "one CTA's shared memory");
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(sparse_attn_q8_kernel), 11, smem);
    if (e != cudaSuccess) return e;
    if (a.n_split > 65535 || p.groups < 1 || p.groups > 2 || (int64_t)b.T * p.groups > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    return launch_k(sparse_attn_q8_kernel, dim3((unsigned)(b.T * p.groups), (unsigned)a.n_split), dim3(kThreads), smem, stream,
                    pdl, p);
}

}  // namespace dsa
