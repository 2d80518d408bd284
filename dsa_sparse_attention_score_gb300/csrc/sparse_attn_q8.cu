// sparse_attn_q8.cu -- sparse MLA attention over selected rows of the 8-bit
// latent cache (quant8.cuh has the row's format):
//     z_j = sm_scale * (q_lat . c_j + q_rope . r_j),  o = sum_j softmax(z)_j c_j,
// c_j = 2^E_j codes_j[0:512], r_j = 2^E_j (hi_j + lo_j).
//
// The tensor cores read the codes as they lie in the cache; no row is ever
// decoded.  What makes that possible:
//  - The row's scale leaves both contractions.  z_j = 2^E_j (codes_j . q), and
//    with u_j = z_j log2(e) + E_j the output is sum_j 2^(u_j - M) codes_j over
//    l = sum_j 2^(z_j log2(e) - M): the scale is folded into the weights (E_j =
//    log2 of the scale: a power of two is not needed here).
//  - A bf16 query is the sum of two e4m3 pieces: q 2^-e = hi + lo with
//    hi = e4m3(q 2^-e), lo = e4m3(q 2^-e - hi).  Four significant bits each,
//    the remainder signed, hold bf16's eight: the split is exact for values
//    above 2^-9.8 of the head's largest, and off by at most 2^-17.8 of it below.
//  - A weight is an e4m3 piece and an e5m2 remainder, in units where the
//    largest lies in [2^2, 2^8]: off by at most 2^-7 of itself (rms 2^-9.7, as
//    for a rounding to bf16) or 2^-15 of the largest.  e5m2 keeps three
//    significant bits of the remainder but reaches down to 2^-16, which buys
//    six octaves of headroom before the units have to move; with e4m3
//    remainders and 4.5 octaves 40% of the tiles moved some head's.
//  - A split's partial output is fp16 times a power of two that keeps its
//    largest sum in range (attn_q8_part_unit).
// So every product is 8-bit by 8-bit with float32 sums, at twice the rate of
// bf16 products and half the bytes: the two pieces cost what one bf16 product
// would, and the rows come in at 644 bytes instead of 1152.
//
// A unit of work is a (token, head group of 64, split), one per CTA of the
// grid; the CTAs that run take over those that have not started and walk
// their tiles of 128 selected rows.  A tile's latent codes are four 16 KB
// blocks of 128 rows x 128 bytes (SWIZZLE_128B) in shared memory, its tails
// (64 hi | 64 lo) 32 columns of tensor memory, a row a lane.
//     S^T[row, piece*head]  = C[row, :] . Q[piece*head, :]^T   M=128, N=128, K=512 + 128
//     O^T[dim, head]       += C[row, dim]^T . P^T[row, head]   4 x M=128, N=64, K=128, both pieces
// The same bytes are the K-major A operand of S^T and the MN-major A operand
// of O^T.  The tail's two halves multiply the same 64 query values, so its
// four K steps read the two of q_rope twice.  S^T accumulates a head's two
// pieces in columns h and 64 + h, which the softmax adds; O^T adds both pieces
// of P^T in place.
//
// Shared memory: queries 72 KB, a ring of two tiles' latent blocks 128 KB, P^T
// 16 KB.  Tensor memory: S^T 128 columns, two tiles' tails 64, O^T 256.  Four
// warps bring in 32 rows of every tile each, the latent codes with 16-byte
// cp.async copies, the tails through registers; two issue the score and the
// value products as their inputs arrive; eight softmax warps (two per TMEM lane
// quarter, 32 heads each) turn a tile's S^T into P^T, and write a unit's
// outputs; they and two more split the next unit's queries meanwhile.  The
// reference M of a head's weights is set 2^2 below its first tile's maximum and
// moves only when a weight would exceed 2^8, so most tiles need no maxima, only
// the question whether any weight does.
//
// Measured, one call after the other over three sets of inputs, 64 heads: a
// prefill chunk of 2048 tokens over 2048 rows each 638 us (915 TFLOP/s counted as
// for bf16, 48% of what the tensor cores do on one large bf16 product); a decode
// step of 8 sequences over 2048 rows 16.7 us and of 32 sequences 29.6 us, the join
// of the splits included (3.5 us).  What bounds it:
//  - A tile takes about 4600 cycles, and a unit 16 of them and some 11000 for
//    its outputs and the next one's queries.  The products read their operands
//    from shared memory at its full rate, S^T 144 KB and O^T 192 KB a tile, and
//    with the gather's 64 KB and P^T's 16 KB that is 3300 cycles at 128 bytes
//    each.  The rest is the chain of every other tile: value product (1900
//    cycles, which frees the ring's blocks), gather (1500), scores (1300),
//    softmax (2700); the two chains take turns on the tensor core.
//  - With the tail as a fifth block, whose slot P^T took over, the next tile's
//    scores waited for the value product: 5000 cycles, a ragged decode of 32 in
//    33.2 us where the other form took 30.3.
//  - A decode step's CTA runs one or two tiles: 4000 cycles to the queries' two
//    pieces, 1000 to the first scores, 3000 of softmax, 2000 of value products,
//    4000 of outputs, each once, with the code coming in from L2.
#include <algorithm>
#include <cstddef>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "quant8.cuh"

namespace dsa {

namespace {

constexpr int kHeads = 64;                    // heads per CTA (padded)
constexpr int kRows = 128;                    // selected rows per tile
constexpr int kBlockBytes = kRows * 128;      // 16 KB
constexpr int kTileBlocks = 4;                // of latent codes
constexpr int kSlots = 2 * kTileBlocks;
constexpr int kQBlockBytes = 2 * kHeads * 128;        // hi and lo rows of 128 codes
constexpr int kQTailBytes = 2 * kHeads * 64;          // hi and lo rows of 64 codes (SWIZZLE_64B)
constexpr int kQBytes = 4 * kQBlockBytes + kQTailBytes;
constexpr int kPieceBytes = kRows * 64;       // one piece of P^T (SWIZZLE_64B)
constexpr int kParts = 2;                     // groups of 32 heads
constexpr int kPartHeads = kHeads / kParts;
constexpr int kSoftmaxWarps = 4 * kParts;     // one per (TMEM lane quarter, part)
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
// Warps 0..3 bring in 32 rows of a tile each, 4..11 do the softmax, 12 issues
// the score products, 13 the value products, 14 and 15 split half of the
// queries of the CTA's second and later units.
constexpr int kRowWarps = 4;                  // one per TMEM lane quarter
constexpr int kFirstSoftmax = kRowWarps;      // a multiple of 4: warp mod 4 is the lane quarter
constexpr int kFirstIssuer = kFirstSoftmax + kSoftmaxWarps;
constexpr int kFirstSplit = kFirstIssuer + 2;
constexpr int kSplitWarps = 2;
// heads of a later unit's queries that a softmax and a split warp take
constexpr int kSoftmaxSplit = 4, kOwnSplit = (kHeads - kSoftmaxWarps * kSoftmaxSplit) / kSplitWarps;
constexpr int kThreads = 32 * (kFirstSplit + kSplitWarps);
constexpr float kTopLog2 = 2.0f;              // a new maximum's weight is 2^2 ...
constexpr float kRaiseLog2 = 8.0f;            // ... and none exceeds 2^8
constexpr int kFewMoved = 6;                  // heads of 32 rescaled one by one
constexpr float kMinScale = 0x1p-40f;
// Least e of a head's queries: under it split8 would add to their exponents,
// zeros' among them.
constexpr int kQueryMinExp = -112;
constexpr uint32_t kTmemCols = 512;           // S^T: 128 columns, the tails of two tiles: 2 x 32, O^T: 4 x 64
constexpr uint32_t kColS = 0;
constexpr uint32_t kColT = 2 * kHeads;
constexpr uint32_t kColO = 256;
constexpr int kRingBytes = kSlots * kBlockBytes + kBlockBytes;    // latent blocks of two tiles, P^T

struct Params {
    const uint16_t *q_lat, *q_rope;
    const uint8_t *codes;
    const float *scale;
    const int32_t *idx;
    void *out;
    float *lse;
    uint16_t *part_o;        // [T, n_split, groups, 64, 512] fp16, unnormalised, times part_unit
    float *part_ml;          // [T, n_split, groups, 64, 2]
    DevBatch b;
    uint32_t *status;
    int H, k, groups, out_bf16;
    float scale_log2;        // sm_scale * log2(e)
    float part_unit;
    int tiles_per_cta, n_split, n_tiles;
};

// One unit of work: a head group of a token, a run of its tiles.
struct Unit {
    int t, h0, nh, split;
    int pos, seq;
    int64_t kv0;
    int tile_lo, n;          // first tile and tiles; none when the position is out of bounds
    bool bad;
};

struct Ctl {
    uint64_t q_full;
    uint64_t q_empty;        // the unit's scores have read its queries
    uint64_t full[kSlots];
    uint64_t empty[kSlots];
    uint64_t t_full[2];      // by tile parity: the tile's tails are in tensor memory
    uint64_t t_empty[2];     // ... and have been read
    uint64_t s_full;
    uint64_t s_empty;        // S^T has been read
    uint64_t p_full;
    uint64_t next_full[2];   // the answer to a request for another unit, in turn
    uint64_t next_empty[2];
    uint64_t row_full[3];    // by tile mod 3: the tile's row scales are there
    uint64_t o_empty;        // the unit's accumulator has been read out
    uint64_t o_full[2];      // by tile parity: tile i's completes after tile i - 2's has been waited for
    uint32_t tmem_base;
    int32_t abort_flag;
    alignas(16) uint4 next[2];          // the answers
    alignas(16) float qs[2][kHeads];   // by unit parity: 2^e of the head's query times scale_log2
    float2 row[3][kRows];    // by tile mod 3: a row's scale (0: masked) and its log2
    float red[4][kHeads];    // a tile's maxima by lane quarter
    float sum[4][kHeads];    // a unit's row sums
    alignas(16) float ma[kSoftmaxWarps][2 * kPartHeads];   // each warp's -m, and how far m moved
    Unit unit[kSoftmaxWarps][2];        // each warp's current and next unit, by unit parity
};

// qs and ma are read four at a time
static_assert(offsetof(Ctl, qs) % 16 == 0 && offsetof(Ctl, ma) % 16 == 0 && offsetof(Ctl, row) % 8 == 0 &&
                  offsetof(Ctl, next) % 16 == 0 && (2 * kPartHeads * 4) % 16 == 0 &&
                  (kRingBytes + kQBytes) % 16 == 0, "16-byte reads of shared memory");

// What lies off the usual path is called, not inlined: the kernel's code has to
// stay in the SM's instruction cache (inlined everywhere it was 175 KB, and
// warps of a decode grid spent half their time waiting for instructions).
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, int32_t *abort_flag, uint32_t *status, uint64_t limit_ns) {
    if (*(volatile int32_t *)abort_flag) return false;
    if (mbar_wait(bar, parity, limit_ns)) return true;
    *(volatile int32_t *)abort_flag = 1;
    flag(status, DSA_DEV_TIMEOUT);
    return false;
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, Ctl &c, uint32_t *status, uint64_t limit_ns) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, &c.abort_flag, status, limit_ns);
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

// Transposing butterfly: each lane holds 32 values, lane L ends up with the
// sum of value L over the warp.
__device__ __forceinline__ float warp_sum_32(float (&a)[32], int lane) {
#pragma unroll
    for (int half = 16; half >= 1; half >>= 1) {
        const bool up = lane & half;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < half) {
                const float keep = up ? a[half + i] : a[i];
                const float send = up ? a[i] : a[half + i];
                a[i] = keep + __shfl_xor_sync(0xffffffffu, send, half);
            }
        }
    }
    return a[0];
}

// The largest magnitudes of eight bf16 values' upper and lower halves, as 15 bits each.
__device__ __forceinline__ uint32_t max_bf16(const uint4 &v) {
    constexpr uint32_t M = 0x7FFF7FFFu;
    return __vmaxu2(__vmaxu2(v.x & M, v.y & M), __vmaxu2(v.z & M, v.w & M));
}

// The two e4m3 pieces of eight bf16 values times 2^-e, none above 448.  fp16
// holds the products to 2^-24, far below the last piece's 2^-10, and they get
// there in integers, two at a time: bf16's exponent field less 112 + e is
// fp16's (drop: that times 2^7, negated, in both halves); what falls below
// 2^-14 goes to a value below it or to 0.
__device__ __forceinline__ void split8(const uint4 &v, uint32_t drop, uint2 &hi, uint2 &lo) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = __viaddmax_s16x2_relu(w[i] & 0x7FFF7FFFu, drop, 0u);
        const uint32_t bits = u << 3 | (w[i] & 0x80008000u);
        const __half2 x = *reinterpret_cast<const __half2 *>(&bits);
        h[i] = e4m3x2(x);
        l[i] = e4m3x2(__hsub2(x, e4m3x2_to_half2(h[i])));
    }
    hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

// Answer c to the CTA's requests for units (see the kernel).
__device__ __noinline__ int read_answer(Ctl &ctl, int c, uint32_t *status, uint64_t limit_ns, int lane) {
    const int i = c & 1;
    int u = -1;
    if (__all_sync(0xffffffffu, wait_bar(smem_u32(&ctl.next_full[i]), (uint32_t)(c >> 1) & 1u, ctl, status, limit_ns)))
        u = clc_answer(smem_u32(&ctl.next[i]));
    fence_proxy_async_smem();                            // read before the next answer is written
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&ctl.next_empty[i]));
    return __shfl_sync(0xffffffffu, u, 0);
}

// Heads first .. end - 1 (a multiple of four) of a unit as two e4m3 pieces in
// shared memory, and their scales in qs; q_lat and q_rope at the unit's first
// of nh heads (zeros beyond).  Four heads at a time: of the latent values lane l takes 16 l ..
// 16 l + 15 of every head, of the tails eight values of head l / 8.
__device__ __noinline__ void split_queries(const uint16_t *q_lat, const uint16_t *q_rope, int nh, int first, int end,
                                           float scale_log2, uint8_t *q_s, float *qs, int lane) {
#pragma unroll 1
    for (int h0 = first; h0 < end; h0 += 4) {
        uint4 a[4], c[4], tv = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = c[i] = make_uint4(0u, 0u, 0u, 0u);
            if (h0 + i < nh) {
                const uint4 *src = reinterpret_cast<const uint4 *>(q_lat + (int64_t)(h0 + i) * D_L) + 2 * lane;
                a[i] = __ldg(src);
                c[i] = __ldg(src + 1);
            }
        }
        const int ht = lane >> 3;                        // the lane's head of the tails
        if (q_rope && h0 + ht < nh) tv = __ldg(reinterpret_cast<const uint4 *>(q_rope + (int64_t)(h0 + ht) * D_R) + (lane & 7));
        uint32_t drop_t = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // the largest magnitude by its bf16 bits
            const uint32_t both = __vmaxu2(ht == i ? max_bf16(tv) : 0u, __vmaxu2(max_bf16(a[i]), max_bf16(c[i])));
            const uint32_t top = __reduce_max_sync(0xffffffffu, max(both & 0xFFFFu, both >> 16));
            const int e = q8_exponent(__uint_as_float(top << 16), kQueryMinExp);
            const uint32_t drop = (uint32_t)(-(112 + e) * 128 & 0xFFFF) * 0x10001u;
            if (ht == i) drop_t = drop;
            if (lane == i) qs[h0 + i] = h0 + i >= nh ? 0.f : top < 0x7F80u ? exp2_int(e) * scale_log2 : __int_as_float(0x7FC00000);
            uint2 h2[2], l2[2];
            split8(a[i], drop, h2[0], l2[0]);
            split8(c[i], drop, h2[1], l2[1]);
            uint8_t *blk = q_s + (lane >> 3) * kQBlockBytes;
            *reinterpret_cast<uint4 *>(blk + sw128_offset((uint32_t)(h0 + i), (uint32_t)(lane & 7))) =
                make_uint4(h2[0].x, h2[0].y, h2[1].x, h2[1].y);
            *reinterpret_cast<uint4 *>(blk + sw128_offset((uint32_t)(kHeads + h0 + i), (uint32_t)(lane & 7))) =
                make_uint4(l2[0].x, l2[0].y, l2[1].x, l2[1].y);
        }
        uint2 h2, l2;
        split8(tv, drop_t, h2, l2);
        uint8_t *tb = q_s + 4 * kQBlockBytes + (lane & 1) * 8;
        *reinterpret_cast<uint2 *>(tb + sw64_offset((uint32_t)(h0 + ht), (uint32_t)(lane & 7) >> 1)) = h2;
        *reinterpret_cast<uint2 *>(tb + sw64_offset((uint32_t)(kHeads + h0 + ht), (uint32_t)(lane & 7) >> 1)) = l2;
    }
}

__device__ __noinline__ Unit load_unit(const Params &p, int u, int lane) {
    const DevBatch &b = p.b;
    Unit w;
    const int g = u / p.n_split;
    w.split = u - g * p.n_split;
    w.t = g / p.groups;
    w.h0 = (g - w.t * p.groups) * kHeads;
    w.nh = min(kHeads, p.H - w.h0);
    w.pos = __ldg(b.q_pos + w.t);
    w.seq = seq_of_warp(b.cu_q, b.B, w.t, lane);
    w.kv0 = seq_base(b, w.seq);
    w.tile_lo = w.split * p.tiles_per_cta;
    int64_t own = -1;
    if (w.pos >= 0 && w.pos < b.max_kv && w.kv0 >= 0) own = cache_row(b, w.seq, w.kv0, w.pos);
    w.bad = own < 0 || own >= b.cache_rows;
    w.n = w.bad ? 0 : max(0, min(p.n_tiles, w.tile_lo + p.tiles_per_cta) - w.tile_lo);
    return w;
}

// A unit without tiles or without a selected row: zeros (an empty partial of a
// split).
__device__ __noinline__ void write_empty(const Params &p, const Unit &w, int tx) {
    if (w.bad && tx == 0 && w.split == 0) flag(p.status, DSA_DEV_BAD_POSITION);
    if (p.n_split > 1) {
        const int64_t part_row = (((int64_t)w.t * p.n_split + w.split) * p.groups + w.h0 / kHeads) * kHeads;
        for (int i = tx; i < kHeads * D_L / 2; i += kSoftmaxThreads)
            reinterpret_cast<uint32_t *>(p.part_o + part_row * D_L)[i] = 0u;
        if (tx < kHeads) {
            p.part_ml[(part_row + tx) * 2] = -INFINITY;
            p.part_ml[(part_row + tx) * 2 + 1] = 0.f;
        }
    } else {
        const int64_t row = (int64_t)w.t * p.H + w.h0;
        for (int i = tx; i < w.nh * D_L; i += kSoftmaxThreads) {
            if (p.out_bf16) static_cast<uint16_t *>(p.out)[row * D_L + i] = 0;
            else static_cast<float *>(p.out)[row * D_L + i] = 0.f;
        }
        if (p.lse && tx < w.nh) p.lse[row + tx] = -INFINITY;
    }
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1) sparse_attn_q8_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *ring = base;
    uint8_t *p_s = base + kSlots * kBlockBytes;          // P^T
    uint8_t *q_s = base + kRingBytes;                    // four latent blocks, then the tail's
    Ctl &ctl = *reinterpret_cast<Ctl *>(q_s + kQBytes);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const DevBatch &b = p.b;
    const bool tail = p.q_rope != nullptr;
    const int width = tail ? kQ8Row : D_L;               // bytes per cached row
    tl_start(b.timeline, kTlAttn);

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&ctl.q_full), kSoftmaxWarps + kSplitWarps);
        mbar_init(smem_u32(&ctl.q_empty), 1);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_u32(&ctl.full[i]), kRowWarps);
            mbar_init(smem_u32(&ctl.empty[i]), 1);
        }
        mbar_init(smem_u32(&ctl.s_full), 1);
        mbar_init(smem_u32(&ctl.s_empty), kSoftmaxWarps);
        mbar_init(smem_u32(&ctl.p_full), kSoftmaxWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl.t_full[i]), kRowWarps);
            mbar_init(smem_u32(&ctl.t_empty[i]), 1);
            mbar_init(smem_u32(&ctl.o_full[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl.next_full[i]), 1);
            mbar_init(smem_u32(&ctl.next_empty[i]), kThreads / 32);
        }
        for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&ctl.row_full[i]), kRowWarps);
        mbar_init(smem_u32(&ctl.o_empty), kSoftmaxWarps);
        ctl.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&ctl.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;
    pdl_wait();                                          // no input is read before this
    // The CTA's units: its own, then those of CTAs that have not started, taken
    // over one at a time (SMs differ by 20% in speed here: 13 or 14 equal
    // units per CTA left the slowest 793 us against a mean of 685).  The first
    // row warp asks shortly before its last tile of a unit; every warp reads
    // answer c when it is through with its unit c: a unit, or -1 for the end.
    // A grid of one wave has nothing to take over (asking would cost it 2 us).
    const bool one_wave = gridDim.x <= kSMs;
    auto next_unit_id = [&](int c) -> int { return one_wave ? -1 : read_answer(ctl, c, p.status, b.wait_ns, lane); };
    // Every role walks the CTA's units and their tiles in the same order.  g
    // counts tiles over all units: tile g has slots 4 (g & 1) .. of the ring, tail
    // columns g & 1, and the phase (g >> 1) & 1 of their barriers.  v counts the
    // units that have tiles.

    if (warp < kRowWarps) {
        // ---------------- rows.  Lane l looks up the cache row of position l of
        // its warp's quarter, one tile ahead.  The latent codes of the quarter's
        // rows go to the ring with asynchronous copies (a row's 128 bytes of a
        // block are one cache line; masked rows are filled with zeros and read
        // nothing); the tail codes go through registers to the rows' lanes of
        // tensor memory, where the score products take them as their first
        // operand; the scales go to the softmax.
        const int r0 = 32 * warp;
        const uint32_t tails = tmem + ((uint32_t)r0 << 16) + kColT;
        const uint32_t d0 = smem_u32(ring) + r0 * 128 + sw128_offset((uint32_t)(lane >> 3), (uint32_t)(lane & 7));
        bool go = true;
        int g = 0;
        int asked = 0;                                   // answers requested
        auto request = [&](int c) {                      // answer c
            const int i = c & 1;
            if (one_wave || warp != 0 || lane != 0) return;
            if (wait_bar(smem_u32(&ctl.next_empty[i]), ((uint32_t)(c >> 1) & 1u) ^ 1u, ctl, p.status, b.wait_ns)) {
                clc_request(smem_u32(&ctl.next[i]), smem_u32(&ctl.next_full[i]));
                asked = c + 1;
            }
        };
        for (int u = blockIdx.x, c = 0; u >= 0; u = next_unit_id(c++)) {
            const Unit w = load_unit(p, u, lane);
            if (w.n <= 2) request(c);
            __syncwarp();
            auto index = [&](int it) -> int32_t {            // the lane's entry of a tile
                const int e = (w.tile_lo + it) * kRows + r0 + lane;
                return it < w.n && e < p.k ? __ldg(p.idx + (int64_t)w.t * p.k + e) : -1;
            };
            auto row_at = [&](int32_t v) -> int32_t {        // its cache row: -1 for padding and out of range (flagged)
                int64_t row = -1;
                if (v >= 0 && v <= w.pos) row = cache_row(b, w.seq, w.kv0, v);
                if (row >= b.cache_rows) row = -1;
                if (row < 0 && v != -1) flag(p.status, DSA_DEV_BAD_INDEX);
                return (int32_t)row;
            };
            int32_t row = -1;
            float s = 0.f;
            uint32_t v[32];
            auto load = [&]() {                              // the row's scale and tail
                s = row < 0 ? 0.f : __ldg(p.scale + row);
                if (tail) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(p.codes + (int64_t)row * width + 4 * 128);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 x = row < 0 ? make_uint4(0u, 0u, 0u, 0u) : __ldg(src + i);
                        v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
                    }
                }
            };
            if (w.n > 0) {
                row = row_at(index(0));
                load();
            }
#pragma unroll 1
            for (int it = 0; go && it < w.n; ++it, ++g) {
                const int buf = g & 1, i3 = g % 3;
                const uint32_t phase = (uint32_t)(g >> 1) & 1u;
                if (it == w.n - 2 && w.n > 2) request(c);
                __syncwarp();
                const int32_t ahead = index(it + 1);
                const bool whole = __all_sync(0xffffffffu, row >= 0);
                const uint8_t *src[8];                       // lane's chunk of rows 4 i + lane / 8
                uint32_t live = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int32_t x = __shfl_sync(0xffffffffu, row, 4 * i + (lane >> 3));
                    live |= (x >= 0 ? 1u : 0u) << i;
                    src[i] = p.codes + (int64_t)max(x, 0) * width + (lane & 7) * 16;
                }
#pragma unroll
                for (int j = 0; j < kTileBlocks; ++j) {
                    const int slot = kTileBlocks * buf + j;
                    go = go && __all_sync(0xffffffffu, wait_bar(smem_u32(&ctl.empty[slot]), phase ^ 1u, ctl, p.status, b.wait_ns));
                    if (go && !b.skip_copies) {
                        const uint32_t dst = d0 + slot * kBlockBytes;
                        if (whole) {                         // (few instructions a copy: they compete with the softmax)
#pragma unroll
                            for (int i = 0; i < 8; ++i) cp_async16((i & 1 ? dst ^ 64u : dst) + i * 512u, src[i] + j * 128);
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                cp_async16_or_zero((i & 1 ? dst ^ 64u : dst) + i * 512u, src[i] + j * 128, live >> i & 1u ? 16u : 0u);
                        }
                    }
                    cp_async_commit();
                }
                // Tile g - 2's tails have been read, so its scores had begun and
                // tile g - 3's scales have served.
                go = go && __all_sync(0xffffffffu, wait_bar(smem_u32(&ctl.t_empty[buf]), phase ^ 1u, ctl, p.status, b.wait_ns));
                if (!go || b.skip_copies) continue;
                // The row's scale.  Any positive one will do; a row never
                // written (scale 0) counts as zeros at the smallest.
                if (row >= 0 && s < kMinScale) s = kMinScale;
                ctl.row[i3][r0 + lane] = row < 0 ? make_float2(0.f, -INFINITY) : make_float2(s, log2f(s));
                if (tail) {
                    tc_fence_after();                    // behind the products that read tile g - 2's tails
                    tmem_st32(tails + 32 * buf, v);
                    tmem_wait_st();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&ctl.row_full[i3]));
                    if (tail) mbar_arrive(smem_u32(&ctl.t_full[buf]));
                }
                auto landed = [&](int j) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&ctl.full[kTileBlocks * buf + j]));
                };
                cp_async_wait<3>(); landed(0);
                cp_async_wait<2>(); landed(1);
                cp_async_wait<1>(); landed(2);
                cp_async_wait<0>(); landed(3);
                if (it + 1 < w.n) {
                    row = row_at(ahead);
                    load();
                }
            }
        }
        cp_async_wait<0>();                                // (a wait may have given up behind copies)
        // (after a wait that gave up the last answer may still be on its way)
        if (asked) mbar_wait(smem_u32(&ctl.next_full[(asked - 1) & 1]), (uint32_t)((asked - 1) >> 1) & 1u, b.wait_ns);
        __syncwarp();
    } else if (warp >= kFirstSplit) {
        // ---------------- half of the queries of every unit but the first, while
        // the softmax warps finish the unit before
        const int first = kSoftmaxWarps * kSoftmaxSplit + kOwnSplit * (warp - kFirstSplit);
        bool go = true;
        int v = 0;
        for (int u = blockIdx.x, c = 0; u >= 0; u = next_unit_id(c++)) {
            const Unit w = load_unit(p, u, lane);
            if (!go || w.n == 0) continue;
            if (v > 0) {
                const int64_t row0 = (int64_t)w.t * p.H + w.h0;
                for (int h = lane + 32 * (warp - kFirstSplit); h < w.nh; h += 32 * kSplitWarps) {
                    prefetch_l2_bulk(p.q_lat + (row0 + h) * D_L, 2 * D_L);
                    if (tail) prefetch_l2_bulk(p.q_rope + (row0 + h) * D_R, 2 * D_R);
                }
                go = __all_sync(0xffffffffu, wait_bar(smem_u32(&ctl.q_empty), (uint32_t)(v - 1) & 1u, ctl, p.status, b.wait_ns));
                if (!go) continue;
                split_queries(p.q_lat + row0 * D_L, tail ? p.q_rope + row0 * D_R : nullptr, w.nh, first, first + kOwnSplit,
                              p.scale_log2, q_s, ctl.qs[v & 1], lane);
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(smem_u32(&ctl.q_full));
            ++v;
        }
    } else if (warp >= kFirstIssuer) {
        // ---------------- MMA issuers: warp 12 the score products, warp 13 the
        // value products, each block as its inputs arrive.  With one warp for
        // both, its waits for one stream held up the other and their
        // bookkeeping (200 to 400 cycles per block) lay between the products.
        // The tensor core takes the two streams' products as they come; they meet in no
        // accumulator and every reuse of memory goes through a barrier:
        //  - scores of tile g overwrite those of tile g - 1 once its softmax has
        //    read them;
        //  - the value product of tile g reads blocks its scores have read.
        // The whole warp runs the loop (uniform descriptors); one elected
        // lane issues.
        const uint32_t ra = smem_u32(ring);
        const uint64_t a0 = sdesc_sw128(ra, 16, 1024);
        auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
                   __all_sync(0xffffffffu, wait_bar(bar, parity, ctl, p.status, b.wait_ns));
        };
        int g = 0, v = 0;
        bool go = true;
        for (int u = blockIdx.x, c = 0; u >= 0; u = next_unit_id(c++)) {
            const int n = load_unit(p, u, lane).n;
            if (!go || n == 0) continue;
            if (warp == kFirstIssuer) {
                const uint32_t id_s = idesc_f8(kRows, 2 * kHeads, false, false);
                const uint32_t qa = smem_u32(q_s);
                const uint64_t q0 = sdesc_sw128(qa, 16, 1024), qt = sdesc_sw64(qa + 4 * kQBlockBytes, 16, 512);
                const uint32_t full0 = smem_u32(&ctl.full[0]);
                go = wait(smem_u32(&ctl.q_full), (uint32_t)v & 1u);
                for (int it = 0; go && it < n; ++it, ++g) {
                    const uint32_t buf = g & 1, phase = (uint32_t)(g >> 1) & 1u, d_s = tmem + kColS;
                    go = wait(smem_u32(&ctl.s_empty), buf ^ 1u);
                    tc_fence_after();
                    if (tail) {                          // K steps 2 and 3 (remainders) read the query again
                        go = go && wait(smem_u32(&ctl.t_full[buf]), phase);
                        tc_fence_after();
                    }
                    if (go && tail && elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            umma_f8_ts(d_s, tmem + kColT + 32 * buf + 8 * ks, qt + (uint64_t)((ks & 1) * 2), id_s, ks ? 1u : 0u);
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < kTileBlocks; ++j) {
                        const uint32_t slot = kTileBlocks * buf + j;
                        go = go && wait(full0 + 8 * slot, phase);
                        if (go && elect_one()) {
                            const uint64_t ad = a0 + (uint64_t)(slot * (kBlockBytes >> 4));
                            const uint64_t bd = q0 + (uint64_t)(j * (kQBlockBytes >> 4));
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                umma_f8(d_s, ad + (uint64_t)(ks * 2), bd + (uint64_t)(ks * 2), id_s, (tail || j || ks) ? 1u : 0u);
                            // (with the first block, which every row warp lands after its wait
                            // for tile g - 2's: no phase goes by unseen)
                            if (j == 0) umma_commit(smem_u32(&ctl.t_empty[buf]));
                            if (j == kTileBlocks - 1) {
                                umma_commit(smem_u32(&ctl.s_full));
                                if (it + 1 == n) umma_commit(smem_u32(&ctl.q_empty));
                            }
                        }
                        __syncwarp();
                    }
                }
            } else {
                const uint32_t id_hi = idesc_f8(128, kHeads, true, true), id_lo = idesc_f8(128, kHeads, true, true, true);
                const uint64_t bd = sdesc_sw64(smem_u32(p_s), 16, 512);
                const uint32_t empty0 = smem_u32(&ctl.empty[0]);
                // the accumulator of the unit before has been read
                if (v > 0) go = wait(smem_u32(&ctl.o_empty), (uint32_t)(v - 1) & 1u);
                for (int it = 0; go && it < n; ++it, ++g) {
                    const uint32_t acc0 = it > 0 ? 1u : 0u;
                    go = wait(smem_u32(&ctl.p_full), (uint32_t)g & 1u);
                    tc_fence_after();
                    if (go && elect_one()) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t slot = kTileBlocks * (g & 1) + c;
                            const uint64_t ad = a0 + (uint64_t)(slot * (kBlockBytes >> 4));
#pragma unroll
                            for (int piece = 0; piece < 2; ++piece)
#pragma unroll
                                for (int ks = 0; ks < kRows / 32; ++ks)
                                    umma_f8(tmem + kColO + c * kHeads, ad + (uint64_t)(ks * (32 * 128 >> 4)),
                                            bd + (uint64_t)(piece * (kPieceBytes >> 4) + ks * (32 * 64 >> 4)), piece ? id_lo : id_hi,
                                            (piece || ks) ? 1u : acc0);
                            umma_commit(empty0 + 8 * slot);
                        }
                        umma_commit(smem_u32(&ctl.o_full[g & 1]));
                    }
                    __syncwarp();
                }
            }
            ++v;
        }
    } else {
        // ---------------- queries, softmax and epilogue
        const int sw = warp - kFirstSoftmax, tx = (int)threadIdx.x - 32 * kFirstSoftmax;
        const int quarter = sw & 3;                        // TMEM lanes 32*quarter ..
        const int part = sw >> 2;                          // heads 32*part ..
        const int hb = kPartHeads * part;
        const int r = quarter * 32 + lane;                 // row within the tile
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        float *ma = ctl.ma[sw];
        bool alive = true;
        int g = 0, v = 0;

        // `heads` heads per warp of the unit's queries as two pieces.
        auto stage_queries = [&](const Unit &w, int parity, int heads) {
            const int64_t row0 = (int64_t)w.t * p.H + w.h0;
            split_queries(p.q_lat + row0 * D_L, tail ? p.q_rope + row0 * D_R : nullptr, w.nh, sw * heads,
                          (sw + 1) * heads, p.scale_log2, q_s, ctl.qs[parity], lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl.q_full));
        };
        int claims = 0;
        // Puts unit u into the warp's slot (n = -1: there is none).
        auto set_unit = [&](int u, int parity) {
            Unit w;
            w.n = -1;
            if (u >= 0) w = load_unit(p, u, lane);
            if (lane == 0) ctl.unit[sw][parity] = w;
            __syncwarp();
        };
        // Gives empty units their outputs until one with tiles, or the end, is
        // in the slot.  Only between units: the answers asked for here need
        // every warp to be through with the unit before.
        auto skip_empty = [&](int parity, int heads) {
            while (ctl.unit[sw][parity].n == 0) {
                write_empty(p, ctl.unit[sw][parity], tx);
                __syncwarp();
                set_unit(next_unit_id(claims++), parity);
            }
            if (ctl.unit[sw][parity].n > 0) stage_queries(ctl.unit[sw][parity], parity, heads);
        };
        set_unit(blockIdx.x, 0);
        skip_empty(0, kHeads / kSoftmaxWarps);
        // Every softmax thread runs the same sequence of named barriers whatever
        // happens; `alive` (warp-uniform) only gates tensor-memory and shared
        // memory work after a bounded wait gave up.
        while (ctl.unit[sw][v & 1].n > 0) {
            const Unit &w = ctl.unit[sw][v & 1];
            const int n_tiles = w.n;
            uint64_t lpart[kPartHeads / 2];                // row sums of l, two heads each
#pragma unroll
            for (int h = 0; h < kPartHeads / 2; ++h) lpart[h] = f2(0.f, 0.f);
            // lane h: the reference m of head hb + h, 2 to 8 below its largest
            // u so far (the same in the four warps of the part); 0 as long as
            // every row was masked or NaN (fresh)
            float m = 0.f;
            bool fresh = true;
            bool seen = false;                             // this thread had a row that is not masked
            ma[lane] = 0.f;
            __syncwarp();
            const float *qs_u = ctl.qs[v & 1] + hb;
            if (alive) alive = wait_bar(smem_u32(&ctl.q_full), (uint32_t)v & 1u, ctl, p.status, b.wait_ns);   // everyone's qs
            for (int it = 0; it < n_tiles; ++it, ++g) {
                if (it + 1 == n_tiles) set_unit(next_unit_id(claims++), (v + 1) & 1);
                if (alive) alive = wait_bar(smem_u32(&ctl.row_full[g % 3]), (uint32_t)(g / 3) & 1u, ctl, p.status, b.wait_ns);
                const float2 rv = ctl.row[g % 3][r];       // a masked row's products are 0: u = -inf
                seen = seen || rv.x != 0.f;
                const float irs = rv.x == 0.f ? 0.f : 1.f / rv.x;
                const uint64_t rs2 = f2(rv.x, rv.x), ef2 = f2(rv.y, rv.y), irs2 = f2(irs, irs);
                if (alive) alive = wait_bar(smem_u32(&ctl.s_full), (uint32_t)g & 1u, ctl, p.status, b.wait_ns);
                alive = __all_sync(0xffffffffu, alive);
                float x[kPartHeads], top = -INFINITY;      // u - m
                if (alive) {
                    tc_fence_after();
                    const uint32_t a = tmem + lane_addr + kColS + hb;
                    uint32_t a16[2][16], b16[2][16];
                    tmem_ld16(a, a16[0]);
                    tmem_ld16(a + kHeads, b16[0]);
                    tmem_wait_ld(a16[0], b16[0]);
                    tmem_ld16(a + 16, a16[1]);             // lands behind the first half's arithmetic
                    tmem_ld16(a + kHeads + 16, b16[1]);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (half) {
                            tmem_wait_ld(a16[1], b16[1]);
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(smem_u32(&ctl.s_empty));
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {        // (the two scales first: one of them alone could overflow)
                            const float4 q4 = *reinterpret_cast<const float4 *>(qs_u + 16 * half + 4 * i);
                            const float4 n4 = *reinterpret_cast<const float4 *>(ma + 16 * half + 4 * i);
                            const uint64_t qs[2] = {f2(q4.x, q4.y), f2(q4.z, q4.w)}, nm[2] = {f2(n4.x, n4.y), f2(n4.z, n4.w)};
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int h = 4 * i + 2 * j;
                                const uint64_t a2 = f2(__uint_as_float(a16[half][h]), __uint_as_float(a16[half][h + 1]));
                                const uint64_t b2 = f2(__uint_as_float(b16[half][h]), __uint_as_float(b16[half][h + 1]));
                                const float2 d = f2_get(f2_add(f2_fma(f2_add(a2, b2), f2_mul(qs[j], rs2), nm[j]), ef2));
                                x[16 * half + h] = d.x;
                                x[16 * half + h + 1] = d.y;
                                top = fmaxf(top, fmaxf(d.x, d.y));
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < kPartHeads; ++h) x[h] = -INFINITY;
                }
                // Does any weight of the part exceed 2^8?  Then the heads'
                // maxima are found and m moves where it has to; few tiles but a
                // unit's first come here.
                uint32_t moved = 0;                        // heads of the part whose m moves
                if (named_barrier_or(2 + part, 128, fresh || top > kRaiseLog2)) {
                    float over = 0.f;
#pragma unroll
                    for (int h = 0; h < kPartHeads; ++h) {
                        const float v32 = warp_max(x[h]);
                        over = lane == h ? v32 : over;
                    }
                    ctl.red[quarter][hb + lane] = over;
                    named_barrier(2 + part, 128);
                    const int hl = hb + lane;
                    over = fmaxf(fmaxf(ctl.red[0][hl], ctl.red[1][hl]), fmaxf(ctl.red[2][hl], ctl.red[3][hl]));
                    // (NaN moves nothing: it gets through to l and the products by itself)
                    const float up = over > (fresh ? -INFINITY : kRaiseLog2) ? over - kTopLog2 : 0.f;
                    m += up;
                    ma[lane] = -m;
                    ma[kPartHeads + lane] = up;
                    moved = fresh ? 0u : __ballot_sync(0xffffffffu, up != 0.f);
                    fresh = __all_sync(0xffffffffu, !(over > -INFINITY)) && fresh;
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < kPartHeads; h += 4) {
                        const float4 up4 = *reinterpret_cast<const float4 *>(ma + kPartHeads + h);
                        x[h] -= up4.x; x[h + 1] -= up4.y; x[h + 2] -= up4.z; x[h + 3] -= up4.w;
                        if (moved) {
                            lpart[h / 2] = f2_mul(lpart[h / 2], f2(ex2(-up4.x), ex2(-up4.y)));
                            lpart[h / 2 + 1] = f2_mul(lpart[h / 2 + 1], f2(ex2(-up4.z), ex2(-up4.w)));
                        }
                    }
                }
                // the weights' two pieces, 16 heads (16 bytes) at a time
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int h = 16 * half + 4 * i;
                        const float e[4] = {ex2(x[h]), ex2(x[h + 1]), ex2(x[h + 2]), ex2(x[h + 3])};
                        lpart[h / 2] = f2_fma(f2(e[0], e[1]), irs2, lpart[h / 2]);
                        lpart[h / 2 + 1] = f2_fma(f2(e[2], e[3]), irs2, lpart[h / 2 + 1]);
                        // through fp16, whose 11 bits the two pieces cannot tell from 24
                        const __half2 a = __floats2half2_rn(e[0], e[1]), c = __floats2half2_rn(e[2], e[3]);
                        const uint32_t ha = e4m3x2(a), hc = e4m3x2(c);
                        hi[i] = ha | hc << 16;
                        lo[i] = e5m2x2(__hsub2(a, e4m3x2_to_half2(ha))) | e5m2x2(__hsub2(c, e4m3x2_to_half2(hc))) << 16;
                    }
                    if (half == 0 && g > 0) {              // P^T of tile g - 1 has been read
                        if (alive) alive = wait_bar(smem_u32(&ctl.o_full[(g - 1) & 1]), (uint32_t)((g - 1) >> 1) & 1u, ctl, p.status, b.wait_ns);
                        alive = __all_sync(0xffffffffu, alive);
                    }
                    if (alive) {
                        const uint32_t o = sw64_offset((uint32_t)r, (uint32_t)(2 * part + half));
                        *reinterpret_cast<uint4 *>(p_s + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4 *>(p_s + kPieceBytes + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                if (moved && it > 0) {
                    // Columns of O^T whose reference moved: one by one while
                    // they are few, else all.
                    if (alive) {
                        tc_fence_after();
                        const uint32_t o = tmem + lane_addr + kColO + hb;
                        if (__popc(moved) <= kFewMoved) {
                            while (moved) {
                                const int h = __ffs(moved) - 1;
                                moved &= moved - 1;
                                const float al = ex2(-ma[kPartHeads + h]);
                                uint32_t c4[4];
#pragma unroll
                                for (int c = 0; c < 4; ++c) tmem_ld1(o + c * kHeads + h, c4[c]);
                                tmem_wait_ld(c4);
#pragma unroll
                                for (int c = 0; c < 4; ++c) tmem_st1(o + c * kHeads + h, __float_as_uint(__uint_as_float(c4[c]) * al));
                            }
                        } else {
#pragma unroll 1
                            for (int c = 0; c < 8; ++c) {
                                uint32_t c16[16];
                                const uint32_t at = o + (c >> 1) * kHeads + (c & 1) * 16;
                                const float *up = ma + kPartHeads + (c & 1) * 16;
                                tmem_ld16(at, c16);
                                tmem_wait_ld(c16);
#pragma unroll
                                for (int h = 0; h < 16; ++h) c16[h] = __float_as_uint(__uint_as_float(c16[h]) * ex2(-up[h]));
                                tmem_st16(at, c16);
                            }
                        }
                        tmem_wait_st();
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl.p_full));
            }
            // ---- outputs: the row sums behind the last value product as well
            const int gl = g - 1;                          // the unit's last tile
            float lrow[kPartHeads];
#pragma unroll
            for (int h = 0; h < kPartHeads / 2; ++h) {
                const float2 d = f2_get(lpart[h]);
                lrow[2 * h] = d.x;
                lrow[2 * h + 1] = d.y;
            }
            const float lsum = warp_sum_32(lrow, lane);
            ctl.sum[quarter][hb + lane] = lsum;
            const bool none = !named_barrier_or(2 + part, 128, seen);      // every row of the unit was masked
            const int hl = hb + lane;
            const float l = ctl.sum[0][hl] + ctl.sum[1][hl] + ctl.sum[2][hl] + ctl.sum[3][hl];
            ma[lane] = p.n_split > 1 ? p.part_unit : l == 0.f ? 0.f : 1.f / l;
            __syncwarp();
            // ---- While the last value product runs: its share of the next unit's
            // queries (the score products have read this one's).
            const bool staged = ctl.unit[sw][(v + 1) & 1].n > 0;
            if (staged) stage_queries(ctl.unit[sw][(v + 1) & 1], (v + 1) & 1, kSoftmaxSplit);
            if (alive) alive = wait_bar(smem_u32(&ctl.o_full[gl & 1]), (uint32_t)(gl >> 1) & 1u, ctl, p.status, b.wait_ns);
            alive = __all_sync(0xffffffffu, alive);
            const int64_t row0 = (int64_t)w.t * p.H + w.h0;
            const int64_t part0 = (((int64_t)w.t * p.n_split + w.split) * p.groups + w.h0 / kHeads) * kHeads;
            if (alive && none) {
                write_empty(p, w, tx);                     // whatever the queries are, NaN among them
            } else if (alive) {
                // Thread (quarter, lane) holds output dim 128 c + 32 quarter +
                // lane of the part's heads.  Of 16-bit results neighbouring lanes
                // swap halves, so that the even one stores two dims of head 2 i
                // and the odd one of head 2 i + 1.
                tc_fence_after();
                const int live = (p.n_split > 1 ? kHeads : w.nh) - hb;     // heads of the part that are stored
                const uint32_t o_t = tmem + lane_addr + kColO + hb;
                // (the factors in registers first: between shared stores their
                // loads would wait for one another)
                float f[kPartHeads];
#pragma unroll
                for (int h = 0; h < kPartHeads; h += 4) {
                    const float4 f4 = *reinterpret_cast<const float4 *>(ma + h);
                    f[h] = f4.x; f[h + 1] = f4.y; f[h + 2] = f4.z; f[h + 3] = f4.w;
                }
                if (p.n_split > 1 || p.out_bf16) {
                    uint16_t *dst = (p.n_split > 1 ? p.part_o + part0 * D_L : static_cast<uint16_t *>(p.out) + row0 * D_L) +
                                    (int64_t)(hb + (lane & 1)) * D_L + quarter * 32 + (lane & 30);
                    const uint32_t take = lane & 1 ? 0x3276u : 0x5410u;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t c32[32];
                        tmem_ld32(o_t + c * kHeads, c32);
                        tmem_wait_ld(c32);
                        uint32_t o16[kPartHeads / 2];
                        if (p.n_split > 1) {
#pragma unroll
                            for (int i = 0; i < kPartHeads / 2; ++i) {
                                const __half2 o2 = __floats2half2_rn(__uint_as_float(c32[2 * i]) * f[2 * i],
                                                                     __uint_as_float(c32[2 * i + 1]) * f[2 * i + 1]);
                                o16[i] = *reinterpret_cast<const uint32_t *>(&o2);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < kPartHeads / 2; ++i) {
                                const __nv_bfloat162 o2 = __floats2bfloat162_rn(__uint_as_float(c32[2 * i]) * f[2 * i],
                                                                                __uint_as_float(c32[2 * i + 1]) * f[2 * i + 1]);
                                o16[i] = *reinterpret_cast<const uint32_t *>(&o2);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < kPartHeads / 2; ++i) {
                            const uint32_t both = __byte_perm(o16[i], __shfl_xor_sync(0xffffffffu, o16[i], 1), take);
                            if (2 * i + (lane & 1) < live) *reinterpret_cast<uint32_t *>(dst + (int64_t)(2 * i) * D_L + c * 128) = both;
                        }
                    }
                } else {
                    float *of = static_cast<float *>(p.out) + (row0 + hb) * D_L + quarter * 32 + lane;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t c32[32];
                        tmem_ld32(o_t + c * kHeads, c32);
                        tmem_wait_ld(c32);
#pragma unroll
                        for (int h = 0; h < kPartHeads; ++h)
                            if (h < live) of[(int64_t)h * D_L + c * 128] = __uint_as_float(c32[h]) * f[h];
                    }
                }
                if (quarter == 0) {
                    const int h = hb + lane;
                    if (p.n_split > 1) {
                        p.part_ml[(part0 + h) * 2] = l == 0.f ? -INFINITY : m;
                        p.part_ml[(part0 + h) * 2 + 1] = l;
                    } else if (p.lse && h < w.nh) {
                        p.lse[row0 + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl.o_empty));
            if (!staged) skip_empty((v + 1) & 1, kSoftmaxSplit);
            ++v;
        }
    }

    tc_fence_before();
    __syncwarp();
    __syncthreads();
    // Dependents launch only now: CTAs of the next grid waiting on this one
    // would share the SMs and slow it down.
    pdl_trigger();
    tl_end(b.timeline, kTlAttn);
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

int attn_q8_tile_rows() { return kRows; }

// The partial outputs of splits are sums of up to tiles * 128 weights of at
// most 2^8 times codes of at most 448: times 2^-8 / tiles (rounded down to a
// power of two) they stay under 57344, inside fp16.  Its eleven bits reach down to
// 2^-14, a product of the unit weight and the smallest code at one tile, so a
// partial is rounded to 2^-11 of itself; in bf16, with the same bytes, to 2^-8,
// which was most of a split decode's error (1.6e-3 of its size).
float attn_q8_part_unit(int tiles_per_cta) {
    float unit = 0x1p-8f;
    for (int t = 1; t < tiles_per_cta; t *= 2) unit *= 0.5f;
    return unit;
}

cudaError_t launch_sparse_attn_q8(const AttnQ8Launch &a, const DevBatch &b, uint32_t *status, cudaStream_t stream) {
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
    p.part_unit = attn_q8_part_unit(a.tiles_per_cta);
    p.scale_log2 = a.sm_scale * 1.4426950408889634f;
    p.tiles_per_cta = a.tiles_per_cta;
    p.n_split = a.n_split;
    p.n_tiles = (a.k + kRows - 1) / kRows;
    const size_t smem = 1024 + kRingBytes + kQBytes + sizeof(Ctl);
    static_assert(1024 + kRingBytes + kQBytes + sizeof(Ctl) <= 232448, "one CTA's shared memory");
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(sparse_attn_q8_kernel), 11, smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)b.T * p.groups * a.n_split;
    if (p.groups < 1 || p.groups > 2 || units > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_k(sparse_attn_q8_kernel, dim3((unsigned)units), dim3(kThreads), smem, stream, true, p);
}

}  // namespace dsa
