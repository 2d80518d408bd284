// mla_attn.cu -- attention of every query head over all the cached latent
// rows that its token sees (or those in a sliding window and the first ones):
//     z_s = sm_scale * (q_lat . c_s[0:512] + q_rope . c_s[512:576]),
//     o   = sum_s softmax(z)_s c_s[0:512],   lse = log(sum_s exp(z_s)).
//
// The query rows (token, head) of a sequence are taken 128 at a time, whatever
// the head count; such an item meets its visible rows in tiles of 128
// positions.  A cluster of two CTAs works on an item with cta_group::2 MMAs:
//     S[row, s]   = Q[row, 0:576] . C[s, 0:576]^T     (M=128, N=128, K=576)
//     O[row, dim] += P[row, s] . C[s, dim]             (M=128, N=2x256, K=128)
// An O of 128 rows and 512 dims would fill the tensor memory of one SM.  With
// M=128 over a pair of SMs each holds 64 rows, a row's first N / 2 columns in
// lane r and the rest in lane r + 64: O takes 256 columns, two S buffers take 128,
// and the other 128 hold the first 256 dims of the queries (as A in tensor memory).
// Measured on GB300, this form runs at 4093 multiply-adds a clock and SM (all
// the tensor core has), also while 64 bytes a clock come in through TMA.
// Each CTA's shared memory holds
//   the other dims of its 64 query rows                 40 KB
//   its 64 of the tile's keys, nine 64-column blocks    72 KB   (B of S)
//   three halves of 64 keys for its 256 output dims     96 KB   (B of O)
//   P of its 64 rows                                    16 KB
// The value rows are read a second time from L2 because a pair's B operand lies
// at one address in both CTAs: S wants a CTA's own keys there, O all keys.
//
// Per tile S takes 1152 clocks and O 1024, and 136 KB come into an SM.  S(i+1),
// O(i), S(i+2), O(i+1)... follow each other on the tensor core, and the softmax of a
// tile has the time of one O and one S.  Keys are refilled in three groups of blocks
// and values in halves of a tile, each as soon as the product that read it is done.
// Warps 0-7 are softmax and output, in two groups that take the tiles in turn; one
// warp each issues S's and O's products and copies keys and values.
// Measured: 2048 tokens of 64 heads after 6144 positions 1.23 to 1.29 ms in a row of
// calls (1.58 to 1.66 PFLOP/s, 92 to 97% of the sustained rate of the card's library
// products; the power cap holds the clock at 1.6 GHz.  One launch under a profiler took
// 1.09 to 1.15 ms at 1.9 to 1.8 GHz): 2.06 million clocks, 2710 a tile with changes of
// pieces, begin and end, 2450 between two tiles of an item; the tensor pipe 85% busy.
// 32 sequences of 4k-64k positions, 128 heads, one token each 0.25 to 0.27 ms (4.8 to
// 5.2 TB/s: 3700 clocks a tile; HBM delivers one in 2800).  8 of 8192, 64 heads 31 us
// (HBM's share is 11: the first S comes 6 us after the launch, the output of the last
// piece takes 2.5 and the join 5).  What bounds calls of many short items is the change
// of pieces, 7000 clocks in which the tensor core waits for an output.
//
// The work is cut by tiles, not by items: the tiles of all items in a row are
// divided evenly among the clusters.  An item that several clusters share gets
// its parts (unnormalised O, running maximum, sum) into the workspace, and
// mla_combine_kernel joins them.
//
// Code that only some calls or tiles reach is kept out of the loops: an instruction
// that is not in the SM's cache takes a round trip to L2, and what every warp runs
// in a tile has to stay there (tiles fell from 7500 misses an SM to 790, a prefill
// from 1.55 to 1.27 ms).
#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {

namespace {

constexpr int kClusters = kSMs / 2;           // pairs of CTAs in the grid
constexpr int kRows = 128;                    // query rows of an item
constexpr int kHalf = 64;                     // rows and keys of one CTA
constexpr int kKeys = 128;                    // positions of a tile
constexpr int kGroup = 16;                    // keys of one MMA step of O
constexpr int kBlock = kHalf * 128;           // 64 rows x 64 bf16: 8 KB
constexpr int kQTmem = 4;                     // blocks of the queries in tensor memory
constexpr int kQOff = 0;                      // the other five
constexpr int kKOff = 5 * kBlock;             // nine blocks
constexpr int kVOff = 14 * kBlock;            // three halves of a tile's keys: [64-dim block][64 keys]
constexpr int kPOff = 26 * kBlock;            // two blocks
constexpr int kCtlOff = 28 * kBlock;
constexpr int kVHalf = 4 * kBlock;
constexpr int kSoftmaxWarps = 8;
constexpr int kSWarp = 8, kOWarp = 9, kKWarp = 10, kVWarp = 11;
constexpr int kThreads = 384;
constexpr int kSBufs = 2, kVBufs = 3;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColQ = 256, kColS = 384;
constexpr float kRescaleLog2 = 20.0f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kItemCost = 1;                  // what an item costs beside its tiles, in tiles

// ---------------------------------------------------------------- pairs of CTAs
__device__ __forceinline__ void tmem_alloc2(uint32_t dst, uint32_t n) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(n) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t n) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(n) : "memory");
}
__device__ __forceinline__ void umma2_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// The same with A in tensor memory: row r of the CTA's 64 in lanes r and r + 64, two
// values a column.
__device__ __forceinline__ void umma2_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// 64 columns of 16 lanes: thread t holds columns 8 j + 2 (t % 4) and the next one of
// lane t / 4 in u[4 j], u[4 j + 1] and of lane t / 4 + 8 in u[4 j + 2], u[4 j + 3].
__device__ __forceinline__ void tmem_st_16x256_x8(uint32_t taddr, const uint32_t (&u)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
        "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]),
        "r"(u[16]), "r"(u[17]), "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]),
        "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
        : "memory");
}
// One arrival at the same barrier of both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void commit2(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// TMA copies into this CTA that complete on a barrier of either CTA.
__device__ __forceinline__ void tma2_load(uint32_t dst, const CUtensorMap *m, uint32_t bar, int32_t col, int32_t row) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(col), "r"(row), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma2_gather4(uint32_t dst, const CUtensorMap *m, uint32_t bar, int32_t col, int4 r) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(col), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
        : "memory");
}
// Arrivals at a barrier of either CTA.  What they publish is read by the tensor
// core alone, behind a proxy fence of the writer, or is a byte count: a release
// over the cluster, which waits out every store of the thread, is not needed
// (it cost 2700 clocks a tile).
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_expect_remote(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void named_barrier_arrive(int id, int nthreads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---------------------------------------------------------------- work

// What a call attends over, in device terms.
struct Problem {
    DevBatch b;
    int H;
    int window;                   // INT32_MAX: every position
    int n_sink;
    const int32_t *sink_pos0;     // null: 0
    int align;                    // of a tile's first position
};

// Up to 128 query rows of one sequence and the positions some of them see:
// [lo, hi] and the first ones [s_lo, s_hi), as tiles of the grid of 128.  The plan
// writes them into the workspace.
struct __align__(16) Item {
    int32_t seq, row0, nrows;         // flat rows (token * H + head)
    int32_t cost0;                    // costs of the items before
    int32_t lo, hi, s_lo, s_hi;       // hi < 0: nothing
    int32_t min_pos;                  // the least position of its tokens (those that see anything)
    int32_t first_pos, n_first;       // tiles of the first positions before pos0, from first_pos on
    int32_t pos0, n;                  // first position of the tiles of [lo, hi]; all tiles
    int32_t wrap;                     // the last tile's keys from here on are positions from first_pos on (128: none)
    int64_t kv0;
};

__device__ __forceinline__ int item_cost(int n) { return n + kItemCost; }

__device__ __forceinline__ void item_tiles(const Problem &p, Item &it) {
    it.n = it.n_first = 0;
    it.s_lo = it.s_hi = 0;
    it.lo = 0;
    it.pos0 = it.first_pos = 0;
    it.wrap = kKeys;
    if (it.hi < 0) return;
    // 64 bits: a window near 2^31 must not wrap
    it.lo = (int)max((int64_t)0, (int64_t)it.min_pos - p.window + 1);
    // Tiles begin where the rows of a box may: a window of 1000 takes 8 of them, from a
    // grid of 128 on mostly 9 (a prefill through it 270 -> 259 us).  (The last tile of positions
    // close to 2^31 must not wrap.)
    const int align = it.hi > INT32_MAX - 2 * kKeys ? kKeys : p.align;
    it.pos0 = it.lo / align * align;
    it.n = (it.hi - it.pos0) / kKeys + 1;
    if (p.n_sink > 0) {
        const int a = p.sink_pos0 ? max(0, __ldg(p.sink_pos0 + it.seq)) : 0;
        const int e = (int)min((int64_t)a + p.n_sink, (int64_t)it.hi + 1);
        if (a < e) {
            it.s_lo = a;
            it.s_hi = e;
            it.first_pos = a / align * align;
            // Those before pos0 behind the last tile's own keys, if there is room (259 -> 241 us),
            // else in tiles of their own.
            const int more = a < it.pos0 ? min(e, it.pos0) - it.first_pos : 0;
            const int used = ((it.hi - it.pos0) % kKeys / kGroup + 1) * kGroup;
            if (more > 0 && used + more <= kKeys) it.wrap = used;
            else it.n_first = (more + kKeys - 1) / kKeys;
            it.n += it.n_first;
        }
    }
}
// The plan of a call, in the workspace.
struct PlanHead {
    int32_t total;                // costs of all items
    int32_t clusters;             // clusters with work: every one has some
};
// floor(total * c / n), the costs before cluster c of n, in 32 bits.
__device__ __forceinline__ int share(int total, int c, int n) {
    const int each = total / n;
    return each * c + (total - each * n) * c / n;
}
struct Start { int32_t item, off; };                 // a cluster's first item and the costs of it done before
struct Split { int32_t row0, nrows, first, parts; }; // an item that begins in a cluster and ends in a later one

// Where an item's tiles are: n_first of the first positions, from first_pos on, then
// those of the others, from pos0 on; the last one's keys from `wrap` on are first
// positions again (128: none).
struct Grid {
    int32_t n_first, first_pos, pos0, last, wrap;
    // position of tile i's first key, and of one of its keys
    __device__ __forceinline__ int tile(int i) const { return i < n_first ? first_pos + i * kKeys : pos0 + (i - n_first) * kKeys; }
    __device__ __forceinline__ int key(int i, int k) const {
        int pos = tile(i) + k;
        if (i == last && k >= wrap) pos = first_pos + k - wrap;
        return pos;
    }
};

// A piece of an item, for every warp of the CTA (Ctl::piece).
struct Piece {
    int32_t t0, t1;               // tiles of the item to do; t0 == t1: an item that sees nothing
    Grid grid;
    int32_t lo, hi, s_lo, s_hi, min_pos;   // as in Item
    int32_t row0, nrows, seq;
    int32_t whole;                // all tiles of the item
    int32_t rest;                 // tiles of the item behind t1
    int32_t end;                  // no piece: there are no more
    int64_t kv0;
};
constexpr int kPieces = 3;        // read ahead

struct Ctl {
    uint64_t k_full[3], k_empty[2];
    uint64_t v_full[kVBufs];
    uint64_t o_done[2][2];        // by tile and half of the keys: a group of softmax warps waits for every other tile
    uint64_t q_full, q_empty, q_tmem;
    uint64_t s_full[kSBufs], s_empty[kSBufs], p_full[2];
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    uint32_t tmem_base;
    int32_t abort_flag;
    float red[2][2][2][kHalf];    // a group's maxima by tile and half of the keys
    alignas(16) float m[2][kHalf];   // running maxima by tile
    PlanHead head;                // the plan, and what is left of it behind the first piece:
    int32_t todo[5];              // a Todo
    Piece piece[kPieces];
};
constexpr size_t kSmem = kCtlOff + sizeof(Ctl);
static_assert(kSmem <= 232448, "shared memory of one CTA");

// The tile's groups of 16 keys with a position between the first and the last that some
// row sees, one bit each.
__device__ __forceinline__ uint32_t groups_of(int lo, int hi) {   // from the tile's first key on, both included
    const int g0 = max(lo, 0) / kGroup, g1 = min(hi, kKeys - 1) / kGroup;
    return hi < 0 || g0 > g1 ? 0u : (0xffu << g0) & (0xffu >> (kKeys / kGroup - 1 - g1));
}
__device__ __forceinline__ uint32_t tile_groups(const Piece &it, const Grid &grid, int i) {
    const int p0 = grid.tile(i);
    if (p0 >= it.lo && p0 + kKeys - 1 <= it.hi) return 0xffu;
    uint32_t m = groups_of(it.lo - p0, it.hi - p0) | groups_of(it.s_lo - p0, it.s_hi - 1 - p0);
    if (i == grid.last && grid.wrap < kKeys) {
        const int p1 = grid.first_pos - grid.wrap;
        m |= groups_of(it.s_lo - p1, min(it.s_hi, grid.pos0) - 1 - p1);
    }
    return m;
}

struct MlaParams {
    Problem pr;
    uint32_t *status;
    const PlanHead *head;
    const Item *items;
    const Start *start;
    const uint16_t *q_lat;        // bf16 [T * H, 512]
    Split *split;                 // [clusters]
    // Parts of items, unnormalised: float32 [2 * clusters, 128, 512] with float32 outputs;
    // with bf16 ones fp16, 32 dims of a row times a power of two (part_unit holds
    // 1 over it): 11 bits, which the output's own 8 hide, at half the bytes, for dims
    // down to 2^-29 of the largest of the 32.
    void *part_o;
    float *part_unit;             // [2 * clusters, 128, 16]
    float *part_ml;               // [2 * clusters, 128, 2]
    void *out;
    int out_bf16;
    float *lse;
    float scale_log2;
    int tail;                     // rows of 576 (1) or 512 (0)
    bool one;                     // without a plan ahead (items null): at most one item a sequence
    int rows_per_box;             // 64, 16 or 0: rows that lie together for certain (pages)
};

// Bits [lo, hi) of 64.
__device__ __forceinline__ uint64_t key_bits(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 64);
    return lo < hi ? (~0ull >> (64 - (hi - lo))) << lo : 0ull;
}

// Token position if the token is in order, else -1 (flagged unless it is padding).
__device__ __forceinline__ int token_pos(const DevBatch &b, int t, uint32_t *status) {
    const int p = __ldg(b.q_pos + t);
    if (p >= 0 && p < b.max_kv) return p;
    if (p != -1) flag(status, DSA_DEV_BAD_POSITION);
    return -1;
}
// Bounded wait of a whole warp; the same answer in every lane.  (Reading the
// clock takes long: only every few tries, each of which waits for a while.)
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, int32_t *abort_flag, uint32_t *status, uint64_t limit_ns) {
    bool ok = false;
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1; !ok; ++n) {
        ok = mbar_try_wait(bar, parity);
        if (ok || n % 8 != 0) continue;
        if (*(volatile int32_t *)abort_flag) break;
        const uint64_t t = global_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > limit_ns) {
            *(volatile int32_t *)abort_flag = 1;
            flag(status, DSA_DEV_TIMEOUT);
        }
    }
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, Ctl &c, uint32_t *status, uint64_t limit_ns) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return wait_long(bar, parity, &c.abort_flag, status, limit_ns);
}

// The ring of pieces, as one warp reads it.
struct Reader {
    uint32_t n = 0;
    __device__ __forceinline__ const Piece *next(Ctl &c, uint32_t *status, uint64_t limit) {
        if (!wait_bar(smem_u32(&c.piece_full[n % kPieces]), (n / kPieces) & 1u, c, status, limit)) return nullptr;
        return &c.piece[n % kPieces];
    }
    __device__ __forceinline__ void done(Ctl &c, int lane) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.piece_empty[n % kPieces]));
        ++n;
    }
};

// Cache row of a position, whoever sees it: negative where there is none.
__device__ __forceinline__ int32_t any_row(const DevBatch &b, int seq, int64_t kv0, int pos) {
    int64_t r = kv0 + pos;
    if (b.block_table) {
        const int blk = pos / b.block_size;
        const int e = blk < b.max_blocks ? __ldg(b.block_table + (int64_t)seq * b.max_blocks + blk) : -1;
        r = e < 0 ? -1 : (int64_t)e * b.block_size + (pos - blk * b.block_size);
    }
    return r >= 0 && r < b.cache_rows ? (int32_t)r : -1;
}
// The rest of an item whose sequence and rows are set.
__device__ __forceinline__ void item_fill(const Problem &p, Item &it) {
    const DevBatch &b = p.b;
    it.kv0 = seq_base(b, it.seq);
    it.min_pos = INT32_MAX;
    it.hi = -1;
    for (int t = it.row0 / p.H; t <= (it.row0 + it.nrows - 1) / p.H; ++t) {
        const int pos = __ldg(b.q_pos + t);
        if (pos >= 0 && pos < b.max_kv) {
            it.min_pos = min(it.min_pos, pos);
            it.hi = max(it.hi, pos);
        }
    }
    item_tiles(p, it);
}
// Item `part` of a sequence (false: it has no such rows).  Where every sequence has
// one token (decode) its position is loaded beside the offsets, not behind them.
__device__ __forceinline__ bool item_of(const Problem &p, int seq, int part, bool one, uint32_t *status, Item &it) {
    const DevBatch &b = p.b;
    const int guess = __ldg(b.q_pos + min(seq, b.T - 1));
    const int t0 = __ldg(b.cu_q + seq), t1 = __ldg(b.cu_q + seq + 1);
    it.kv0 = seq_base(b, seq);
    if (t0 < 0 || t1 < t0 || t1 > b.T || (one && (t1 - t0) * p.H > kRows)) {
        flag(status, DSA_DEV_BAD_POSITION);
        return false;
    }
    it.seq = seq;
    it.row0 = t0 * p.H + part * kRows;
    it.nrows = min(kRows, t1 * p.H - it.row0);
    if (it.nrows <= 0) return false;
    it.min_pos = INT32_MAX;
    it.hi = -1;
    const int last = (it.row0 + it.nrows - 1) / p.H;
#pragma unroll 4
    for (int t = it.row0 / p.H; t <= last; ++t) {
        const int pos = t == seq ? guess : __ldg(b.q_pos + t);
        if (pos >= 0 && pos < b.max_kv) {
            it.min_pos = min(it.min_pos, pos);
            it.hi = max(it.hi, pos);
        }
    }
    item_tiles(p, it);
    return true;
}

// What a cluster has still to do.
struct Todo {
    int32_t seq, item;            // next item (of the sequence; of all with a plan ahead)
    int32_t off, left;            // costs of it done, costs left to this cluster
    int32_t written;              // pieces in the ring
    // The next piece, of item `it`; false: costs that stand for no tile.
    __device__ __forceinline__ bool take(const Item &it, Piece &pc, bool by_seq) {
        const int cost = item_cost(it.n), n = min(left, cost - off);
        pc.t0 = min(off, it.n);
        pc.t1 = min(off + n, it.n);
        const bool first = off == 0;
        left -= n;
        off += n;
        if (off == cost) {
            ++(by_seq ? seq : item);
            off = 0;
        }
        pc.grid = Grid{it.n_first, it.first_pos, it.pos0, it.n - 1, it.wrap};
        pc.lo = it.lo;
        pc.hi = it.hi;
        pc.s_lo = it.s_lo;
        pc.s_hi = it.s_hi;
        pc.min_pos = it.min_pos;
        pc.row0 = it.row0;
        pc.nrows = it.nrows;
        pc.seq = it.seq;
        pc.whole = pc.t0 == 0 && pc.t1 == it.n;
        pc.rest = it.n - pc.t1;
        pc.kv0 = it.kv0;
        pc.end = 0;
        return pc.t1 > pc.t0 || (it.n == 0 && first);
    }
};
static_assert(sizeof(Todo) == sizeof(Ctl::todo), "a Todo's place");
// This CTA's query rows of a piece into L2, long before they are wanted.
__device__ __forceinline__ void ask_for_queries(const MlaParams &p, const Piece &pc) {
    if (pc.t1 == pc.t0) return;
    const int64_t row = (int64_t)pc.row0 + kHalf * (int)cluster_rank(), rows = (int64_t)p.pr.b.T * p.pr.H - row;
    if (rows > 0) prefetch_l2_bulk(p.q_lat + row * D_L, (uint32_t)min(rows, (int64_t)kHalf) * (D_L * 2));
}

// Writes the cluster's pieces into the ring, one a call, with a whole warp.
struct Scheduler {
    Todo todo;
    bool end = false;
    __device__ __forceinline__ bool write(const MlaParams &p, Ctl &ctl, int lane);
};

// Of rows that no token sees not even 0 times a value may come into a product, and their
// blocks need not be there.  The tokens of a piece see all positions between its first
// and its last one, unless some are not in order or their windows do not meet.  Those
// rare pieces are looked at token by token, out of the usual path, over all tiles between
// their first and last position.  That this is looked up costs chunks over pages of 16
// rows 3% (247 -> 254 us), other calls nothing that is measured.  (Parameters by value:
// behind a reference they are loaded through generic addresses.)
struct Tokens {
    const int32_t *q_pos, *table;   // of the piece's first token; the sequence's blocks (null: contiguous)
    int64_t kv0, cache_rows;
    int32_t n, max_kv, block_size, max_blocks, window;
};
__device__ __forceinline__ Tokens tokens_of(const Problem &p, const Piece *pc) {
    const DevBatch &b = p.b;
    const int first = pc->row0 / p.H;
    return Tokens{b.q_pos + first, b.block_table ? b.block_table + (int64_t)pc->seq * b.max_blocks : nullptr, pc->kv0, b.cache_rows,
                  (pc->row0 + pc->nrows - 1) / p.H - first + 1, b.max_kv, b.block_size, b.max_blocks, p.window};
}
// The position of token t of them if it is in order, else -1.
__device__ __forceinline__ int position_in_order(const Tokens &k, int t) {
    const int pos = t < k.n ? __ldg(k.q_pos + t) : -1;
    if (pos < 0 || pos >= k.max_kv || k.kv0 < 0) return -1;
    int64_t r = k.kv0 + pos;
    if (k.table) {
        const int blk = pos / k.block_size, e = blk < k.max_blocks ? __ldg(k.table + blk) : -1;
        r = e < 0 ? -1 : (int64_t)e * k.block_size + (pos - blk * k.block_size);
    }
    return r >= 0 && r < k.cache_rows ? pos : -1;
}
// x: do tokens in order see all positions between the first that a window from `least`
// reaches back to, and `hi`?  y: the largest position in order (-1: none).
__device__ __noinline__ int2 all_between_seen(const Tokens k, int least, int hi) {
    const int lane = threadIdx.x & 31;
    int lo = INT32_MAX, last = -1, before = -1;               // before: the last token's in order so far
    bool gaps = false;
#pragma unroll 1
    for (int t = 0; t < k.n; t += 32) {
        const int pos = position_in_order(k, t + lane);
        if (pos >= 0) lo = min(lo, pos), last = max(last, pos);
        // windows that meet from token to token leave no gap, whatever the order
        const uint32_t there = __ballot_sync(0xffffffffu, pos >= 0), ahead = there & ((1u << lane) - 1);
        const int x = __shfl_sync(0xffffffffu, pos, ahead ? 31 - __clz(ahead) : 0), to = ahead ? x : before;
        gaps |= pos >= 0 && to >= 0 && abs(pos - to) > k.window;
        const int y = __shfl_sync(0xffffffffu, pos, there ? 31 - __clz(there) : 0);
        if (there) before = y;
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    last = __reduce_max_sync(0xffffffffu, last);
    return make_int2(!__any_sync(0xffffffffu, gaps) && lo == least && last == hi, last);
}
// Which of the four positions from `a` on (its own of each lane) some token in order sees,
// as bits; [s_lo, s_hi) are the first ones.
__device__ __noinline__ uint32_t seen_token_by_token(const Tokens k, int s_lo, int s_hi, int a) {
    const int lane = threadIdx.x & 31;
    uint32_t m = 0;
#pragma unroll 1
    for (int t = 0; t < k.n; t += 32) {
        const int pos = position_in_order(k, t + lane);
#pragma unroll 1
        for (int j = 0; j < min(32, k.n - t); ++j) {
            const int last = __shfl_sync(0xffffffffu, pos, j), before = last - k.window;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int x = a + e;
                m |= (uint32_t)(x <= last && (x > before || (x >= s_lo && x < s_hi))) << e;
            }
        }
    }
    return m;
}

__device__ __forceinline__ bool Scheduler::write(const MlaParams &p, Ctl &ctl, int lane) {
    while (!end) {
        end = todo.left <= 0;
        Piece pc{};
        pc.end = end;
        if (!end) {
            Item it;
            if (p.items) {
                it = p.items[todo.item];
            } else if (!item_of(p.pr, todo.seq, todo.item, p.one, p.status, it)) {
                end = ++todo.seq >= p.pr.b.B;                 // the next sequence's first
                todo.item = 0;
                if (!end) continue;
                pc.end = true;
            }
            if (!end && !todo.take(it, pc, p.one && !p.items)) continue;
        }
        const uint32_t n = (uint32_t)todo.written, slot = n % kPieces;
        if (!wait_bar(smem_u32(&ctl.piece_empty[slot]), ((n / kPieces) & 1u) ^ 1u, ctl, p.status, p.pr.b.wait_ns)) {
            end = true;
            return false;
        }
        if (lane == 0) {
            ctl.piece[slot] = pc;
            mbar_arrive(smem_u32(&ctl.piece_full[slot]));
            ask_for_queries(p, pc);
        }
        __syncwarp();
        ++todo.written;
        break;
    }
    return true;
}

// Copies of rows that do not lie together, out of the usual path: four keys a lane
// of n blocks (lanes 0..15 and 16..31 of alternate ones), and four rows of values.
__device__ __noinline__ void copy_keys(uint32_t dst, const CUtensorMap *kv1, uint32_t full, int kb0, int n, int4 r, int lane) {
#pragma unroll 1
    for (int c = lane; c < n * 16; c += 32) tma2_gather4(dst + (kb0 + c / 16) * kBlock, kv1, full, (kb0 + c / 16) * 64, r);
    __syncwarp();
}
// A group's 16 rows of values, four of them in each of the lanes from `lane0` on; one
// lane issues the copies from uniform registers (a lane's own take 130 clocks each, not 12).
__device__ __noinline__ void copy_values(uint32_t dst, const CUtensorMap *kv1, uint32_t full, int col, int4 r, int lane0) {
#pragma unroll 1
    for (int m = 0; m < 4; ++m) {
        int4 u;
        u.x = __reduce_max_sync(0xffffffffu, __shfl_sync(0xffffffffu, r.x, lane0 + m));
        u.y = __reduce_max_sync(0xffffffffu, __shfl_sync(0xffffffffu, r.y, lane0 + m));
        u.z = __reduce_max_sync(0xffffffffu, __shfl_sync(0xffffffffu, r.z, lane0 + m));
        u.w = __reduce_max_sync(0xffffffffu, __shfl_sync(0xffffffffu, r.w, lane0 + m));
        if (elect_one()) {
#pragma unroll
            for (int d = 0; d < 4; ++d) tma2_gather4(dst + m * 512 + d * kBlock, kv1, full, col + 64 * d, u);
        }
        __syncwarp();
    }
}
// That of a position, the spare one where nobody sees it.
__device__ __forceinline__ int32_t row_or_spare(const DevBatch &b, uint32_t *status, const Piece *pc, bool seen, int pos, int32_t spare) {
    if (!seen) return spare;
    const int32_t r = any_row(b, pc->seq, pc->kv0, pos);
    if (r >= 0) return r;
    flag(status, DSA_DEV_BAD_INDEX);
    return spare;
}
// The rows of the four keys from `pos` on, of which those in the bits `see` are seen.
__device__ __forceinline__ int4 four_rows(const DevBatch &b, uint32_t *status, const Piece *pc, uint32_t see, int pos, int32_t spare) {
    return make_int4(row_or_spare(b, status, pc, see & 1u, pos, spare), row_or_spare(b, status, pc, see & 2u, pos + 1, spare),
                     row_or_spare(b, status, pc, see & 4u, pos + 2, spare), row_or_spare(b, status, pc, see & 8u, pos + 3, spare));
}
__device__ __forceinline__ int4 four_any_rows(const DevBatch &b, const Piece *pc, int pos) {
    return make_int4(max(0, any_row(b, pc->seq, pc->kv0, pos)), max(0, any_row(b, pc->seq, pc->kv0, pos + 1)),
                     max(0, any_row(b, pc->seq, pc->kv0, pos + 2)), max(0, any_row(b, pc->seq, pc->kv0, pos + 3)));
}

// Exclusive prefix over a CTA of N threads, and the sum; sh: 64 words.
template <int N>
__device__ __forceinline__ int plan_scan(int v, int &sum, int *sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = lane < N / 32 ? sh[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += z;
        }
        sh[32 + lane] = y;
    }
    __syncthreads();
    sum = sh[63];
    const int before = (warp ? sh[32 + warp - 1] : 0) + x - v;
    __syncthreads();
    return before;
}

// A cluster's first piece into the ring, by the one thread that knows its first
// item: the other warps begin with it right away.
__device__ __forceinline__ void begin(const MlaParams &p, Ctl &ctl, int cluster, PlanHead head, int seq, int item, int off, const Item &it) {
    const int left = share(head.total, cluster + 1, head.clusters) - share(head.total, cluster, head.clusters);
    Todo todo{seq, item, off, left, 0};
    Piece pc;
    if (todo.take(it, pc, p.one && !p.items)) {
        ctl.piece[0] = pc;
        mbar_arrive(smem_u32(&ctl.piece_full[0]));
        ask_for_queries(p, pc);
        todo.written = 1;
    }
    *reinterpret_cast<Todo *>(ctl.todo) = todo;
}
// The plan of a call with no more sequences and items than threads, made by every CTA
// for itself: 8 us less than with a plan kernel ahead (decode 42.6 -> 34.5 us).
__device__ __forceinline__ void plan_here(const MlaParams &p, Ctl &ctl, int cluster) {
    const DevBatch &b = p.pr.b;
    int *const sh = reinterpret_cast<int *>(&ctl.red[0][0][0][0]);
    int seq = (int)threadIdx.x, item = 0;                     // of this thread
    bool there = seq < b.B;
    if (!p.one) {
        // items of the sequences before each, and from there this thread's
        int n = 0, items;
        if (there) {
            const int t0 = __ldg(b.cu_q + seq), t1 = __ldg(b.cu_q + seq + 1);
            if (t0 >= 0 && t1 >= t0 && t1 <= b.T) n = ((t1 - t0) * p.pr.H + kRows - 1) / kRows;
            else flag(p.status, DSA_DEV_BAD_POSITION);
        }
        const int before = plan_scan<kThreads>(n, items, sh);
        int *const first = sh + 64;
        if (there) first[seq] = before;
        __syncthreads();
        if (items > kThreads && threadIdx.x == 0) flag(p.status, DSA_DEV_BAD_POSITION);   // only where cu_q falls somewhere
        there = (int)threadIdx.x < items;
        int hi = b.B;
        for (seq = 0; hi - seq > 1;) {                        // first[seq] <= threadIdx.x < first[hi]
            const int mid = (seq + hi) >> 1;
            if (first[mid] <= (int)threadIdx.x) seq = mid; else hi = mid;
        }
        item = (int)threadIdx.x - first[seq];
    }
    Item it;
    int cost = 0;
    if (there && item_of(p.pr, seq, item, p.one, p.status, it)) cost = item_cost(it.n);
    int total;
    const int before = plan_scan<kThreads>(cost, total, sh);
    const PlanHead head{total, min((int)gridDim.x / 2, total)};
    if (threadIdx.x == 0) ctl.head = head;
    if (cluster < head.clusters) {
        const int at = share(total, cluster, head.clusters);
        if (at >= before && at < before + cost) begin(p, ctl, cluster, head, seq, item, at - before, it);
    }
}
// The same from the plan kernel's, by one thread.
__device__ __forceinline__ void plan_read(const MlaParams &p, Ctl &ctl, int cluster) {
    const PlanHead head = *p.head;
    ctl.head = head;
    if (cluster >= head.clusters) return;
    const Start st = p.start[cluster];
    begin(p, ctl, cluster, head, 0, st.item, st.off, p.items[st.item]);
}

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_attn_kernel(const __grid_constant__ MlaParams p, const __grid_constant__ CUtensorMap q_lat_map,
                    const __grid_constant__ CUtensorMap q_rope_map, const __grid_constant__ CUtensorMap kv64_map,
                    const __grid_constant__ CUtensorMap kv16_map, const __grid_constant__ CUtensorMap kv1_map) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctl &ctl = *reinterpret_cast<Ctl *>(smem + kCtlOff);
    const uint32_t s0 = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int cluster = blockIdx.x >> 1;
    const DevBatch &b = p.pr.b;
    if (s0 & 1023u) {             // the same in every CTA of the grid
        if (threadIdx.x == 0) flag(p.status, DSA_DEV_SMEM_LAYOUT);
        return;
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&ctl.k_full[i]), 2);   // both CTAs' producers, and their bytes
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl.k_empty[i]), 1);
            mbar_init(smem_u32(&ctl.o_done[i][0]), 1);
            mbar_init(smem_u32(&ctl.o_done[i][1]), 1);
        }
        for (int i = 0; i < kSBufs; ++i) {
            mbar_init(smem_u32(&ctl.s_full[i]), 1);
            mbar_init(smem_u32(&ctl.s_empty[i]), kSoftmaxWarps);          // a group's in both CTAs
        }
        for (int32_t &x : ctl.todo) x = 0;                    // what a cluster without work has to do
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(smem_u32(&ctl.piece_full[i]), 1);
            mbar_init(smem_u32(&ctl.piece_empty[i]), kSoftmaxWarps + 2 + (rank == 0 ? 2 : 0));
        }
        for (int i = 0; i < kVBufs; ++i) mbar_init(smem_u32(&ctl.v_full[i]), 2);
        mbar_init(smem_u32(&ctl.q_tmem), kSoftmaxWarps);                      // a group's in both CTAs
        mbar_init(smem_u32(&ctl.q_full), 2);
        mbar_init(smem_u32(&ctl.q_empty), 1);
        mbar_init(smem_u32(&ctl.p_full[0]), kSoftmaxWarps);
        mbar_init(smem_u32(&ctl.p_full[1]), kSoftmaxWarps / 2);
        ctl.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kSWarp) tmem_alloc2(smem_u32(&ctl.tmem_base), kTmemCols);
    if (warp == kKWarp && lane == 0) {
        tma_prefetch_desc(&kv64_map);
        tma_prefetch_desc(&q_lat_map);
        tma_prefetch_desc(&q_rope_map);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;
    pdl_wait();
    if (!p.items) plan_here(p, ctl, cluster);
    else if (threadIdx.x == 0) plan_read(p, ctl, cluster);
    __syncthreads();
    const uint64_t limit = b.wait_ns;
    const int n_blocks = p.tail ? 9 : 8;
    // waits for the value product of half h of tile t's keys
    auto wait_o = [&](int h, uint32_t t) {
        return wait_bar(smem_u32(&ctl.o_done[t & 1u][h]), (t >> 1) & 1u, ctl, p.status, limit);
    };

    if (warp == kKWarp) {
        // ---------------- keys: this CTA's 64 of each tile, in three groups of blocks.
        // Keys that nobody sees may be anything: their scores are masked.
        uint32_t g = 0, nq = 0;                               // tiles and pieces so far
        const uint32_t q_bar = dsmem_map(smem_u32(&ctl.q_full), 0);
        const int step = p.rows_per_box ? p.rows_per_box : 4; // keys of one copy
        const int copies = kHalf / step;                      // of one block
        const int mine = lane % copies;
        const uint32_t k_bar = dsmem_map(smem_u32(&ctl.k_full[0]), 0);
        bool alive = true;
        Reader rd;
        while (alive) {
            const Piece *pc = rd.next(ctl, p.status, limit);
            if (!pc || pc->end) break;
            const int t0 = pc->t0, t1 = pc->t1, seq = pc->seq;
            const int64_t kv0 = pc->kv0;
            const Grid grid = pc->grid;
            for (int i = t0; alive && i < t1; ++i, ++g) {
                // (a half with keys of two places: boxes of 16)
                const bool mixed = i == grid.last && grid.wrap < kHalf * ((int)rank + 1) && p.rows_per_box == 64;
                const int a = grid.key(i, kHalf * (int)rank + (mixed ? (lane & 3) * kGroup : mine * step));
                int4 r = make_int4(0, 0, 0, 0);
                if (p.rows_per_box) r.x = max(0, any_row(b, seq, kv0, a));
                else r = four_any_rows(b, pc, a);
                const uint32_t dst = s0 + kKOff + mine * step * 128;
                // the boxes' rows in uniform registers: issued by one lane from there a copy takes
                // 12 clocks, by several lanes from their own registers 130 each
                int row[4];
                if (copies <= 4) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) row[j] = __reduce_max_sync(0xffffffffu, __shfl_sync(0xffffffffu, r.x, j));
                }
#pragma unroll 1
                for (int q = 0; q < 3; ++q) {
                    const int nb = min(3, n_blocks - 3 * q);
                    const uint32_t full = k_bar + q * 8;
                    // the last group is free once the tile before is scored
                    if (q < 2) alive = wait_bar(smem_u32(&ctl.k_empty[q]), (g & 1u) ^ 1u, ctl, p.status, limit);
                    else if (g > 0) alive = wait_bar(smem_u32(&ctl.s_full[(g - 1) & 1u]), ((g - 1) >> 1) & 1u, ctl, p.status, limit);
                    if (!alive) break;
                    if (q == 2 && i == t0) {
                        // the queries of this CTA's 64 rows.  Rows past the sequence's are some
                        // other token's (or zero past the tensor): they only feed accumulator
                        // rows that are never stored.
                        alive = wait_bar(smem_u32(&ctl.q_empty), (nq & 1u) ^ 1u, ctl, p.status, limit);
                        if (!alive) break;
                        ++nq;
                        const int q_row = __reduce_max_sync(0xffffffffu, pc->row0) + kHalf * (int)rank;
                        if (!b.skip_copies && elect_one()) {
                            arrive_expect_remote(q_bar, (uint32_t)((n_blocks - kQTmem) * kBlock));
#pragma unroll 1
                            for (int c = kQTmem; c < 8; ++c) tma2_load(s0 + kQOff + (c - kQTmem) * kBlock, &q_lat_map, q_bar, c * 64, q_row);
                            if (p.tail) tma2_load(s0 + kQOff + (8 - kQTmem) * kBlock, &q_rope_map, q_bar, 0, q_row);
                        }
                        __syncwarp();
                    }
                    if (b.skip_copies) continue;
                    if (p.rows_per_box == 64 && !mixed) {
                        if (elect_one()) {
                            arrive_expect_remote(full, (uint32_t)(nb * kBlock));
#pragma unroll
                            for (int c = 0; c < 3; ++c)
                                if (c < nb) tma2_load(s0 + kKOff + (3 * q + c) * kBlock, &kv64_map, full, (3 * q + c) * 64, row[0]);
                        }
                        __syncwarp();
                        continue;
                    }
                    if (p.rows_per_box) {
                        if (elect_one()) {
                            arrive_expect_remote(full, (uint32_t)(nb * kBlock));
#pragma unroll 1
                            for (int c = 3 * q; c < 3 * q + nb; ++c)
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    tma2_load(s0 + kKOff + c * kBlock + j * 2048, &kv16_map, full, c * 64, row[j]);
                        }
                        __syncwarp();
                        continue;
                    }
                    if (lane == 0) arrive_expect_remote(full, (uint32_t)(nb * kBlock));
                    __syncwarp();
                    copy_keys(dst, &kv1_map, full, 3 * q, nb, r, lane);
                }
            }
            rd.done(ctl, lane);
        }
        // the last arrivals at this CTA's barriers, before it ends
        if (alive && g > 0) {
            for (int q = 0; q < 2; ++q) wait_bar(smem_u32(&ctl.k_empty[q]), (g - 1) & 1u, ctl, p.status, limit);
            wait_bar(smem_u32(&ctl.q_empty), (nq - 1) & 1u, ctl, p.status, limit);
        }
    } else if (warp == kVWarp) {
        // ---------------- values: all keys of a tile in two halves, this CTA's 256 dims.
        // Groups of 16 keys before the first position that some token sees, or behind the
        // last one, are neither read nor multiplied; in the others a row that nobody sees
        // is a copy of one that somebody does (P is 0 there, and 0 times what an unused
        // row may hold is not).
        uint32_t g = 0, buf = 0;                              // tiles so far, the next half's place
        bool alive = true;
        const uint32_t v_bar = dsmem_map(smem_u32(&ctl.v_full[0]), 0);
        Reader rd;
        while (alive) {
            const Piece *pc = rd.next(ctl, p.status, limit);
            if (!pc || pc->end) break;
            const int t1 = pc->t1, lo = pc->lo, hi = pc->hi, s_lo = pc->s_lo, s_hi = pc->s_hi;
            const Grid grid = pc->grid;
            // If the last position has a row, its token is in order and sees all back to its
            // window's begin; that of the least one, as far back as the piece goes.
            bool odd = false;                                 // otherwise: look at each token
            const int32_t row_of_end = hi < 0 || pc->kv0 < 0 ? -1 : any_row(b, pc->seq, pc->kv0, lane & 1 ? pc->min_pos : hi);
            const uint32_t ends = __ballot_sync(0xffffffffu, row_of_end >= 0);
            int32_t spare = __shfl_sync(0xffffffffu, row_of_end, 0);
            if (!(ends & 1u) || (lo < (int64_t)hi - p.pr.window + 1 && (!(ends & 2u) || hi - pc->min_pos > p.pr.window))) {
                const int2 x = all_between_seen(tokens_of(p.pr, pc), pc->min_pos, hi);
                odd = !x.x;
                spare = x.y < 0 ? 0 : max(0, any_row(b, pc->seq, pc->kv0, x.y));
            }
            for (int i = pc->t0; alive && i < t1; ++i, ++g) {
                const uint32_t groups = tile_groups(*pc, grid, i);
                // where a group's 16 rows lie together, lane j looks group j up; one that is
                // seen in full is a box
                int32_t first = -1;
                uint32_t ones = 0, see = 0;
                if (odd) see = seen_token_by_token(tokens_of(p.pr, pc), s_lo, s_hi, grid.key(i, 4 * lane));
                if (p.rows_per_box) {
                    const int a = grid.key(i, kGroup * (lane & 7)), e = a + kGroup - 1;
                    bool some = groups >> (lane & 7) & 1u, all = (a >= lo && e <= hi) || (a >= s_lo && e < s_hi);
                    if (odd) {
                        const uint32_t some4 = __ballot_sync(0xffffffffu, see != 0), all4 = __ballot_sync(0xffffffffu, see == 0xfu);
                        some &= (some4 >> (4 * (lane & 7)) & 0xfu) != 0;
                        all = (all4 >> (4 * (lane & 7)) & 0xfu) == 0xfu;
                    }
                    if (some) {
                        first = any_row(b, pc->seq, pc->kv0, a);
                        if (first < 0) flag(p.status, DSA_DEV_BAD_INDEX);
                    }
                    ones = __ballot_sync(0xffffffffu, first >= 0 && all) & 0xffu;
                }
                // the other groups' rows, four a lane
                int4 r = make_int4(0, 0, 0, 0);
                if (groups & ~ones) {
                    const int a = grid.key(i, 4 * lane);
                    if (!odd) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            see |= (uint32_t)((a + e >= lo && a + e <= hi) || (a + e >= s_lo && a + e < s_hi)) << e;
                    }
                    if (p.rows_per_box) {
                        const int32_t row = __shfl_sync(0xffffffffu, first, lane >> 2), at = row + 4 * (lane & 3);
                        r.x = row >= 0 && see & 1u ? at : spare;
                        r.y = row >= 0 && see & 2u ? at + 1 : spare;
                        r.z = row >= 0 && see & 4u ? at + 2 : spare;
                        r.w = row >= 0 && see & 8u ? at + 3 : spare;
                    } else {
                        r = four_rows(b, p.status, pc, see, a, spare);
                    }
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const uint32_t n = 2 * g + h;                           // halves so far
                    if (n >= kVBufs) alive = wait_o((n - kVBufs) & 1u, (n - kVBufs) >> 1);
                    if (!alive) break;
                    const uint32_t at = s0 + kVOff + buf * kVHalf, full = v_bar + buf * 8;
                    buf = buf + 1 == kVBufs ? 0 : buf + 1;
                    if (b.skip_copies) continue;
                    const uint32_t mine = __reduce_or_sync(0xffffffffu, ones >> (4 * h) & 0xfu);
                    int row[4];
                    row[0] = __reduce_max_sync(0xffffffffu, __shfl_sync(0xffffffffu, first, 4 * h));
                    if (p.rows_per_box == 64 && mine == 0xfu && (i < grid.last || grid.wrap >= 64 * (h + 1))) {
                        // the half's four blocks of this CTA's dims
                        if (elect_one()) {
                            arrive_expect_remote(full, kVHalf);
#pragma unroll
                            for (int d = 0; d < 4; ++d)
                                tma2_load(at + d * kBlock, &kv64_map, full, 256 * (int)rank + 64 * d, row[0]);
                        }
                        __syncwarp();
                        continue;
                    }
#pragma unroll
                    for (int j = 1; j < 4; ++j) row[j] = __reduce_max_sync(0xffffffffu, __shfl_sync(0xffffffffu, first, 4 * h + j));
                    if (elect_one()) {
                        arrive_expect_remote(full, (uint32_t)__popc((groups >> (4 * h)) & 0xfu) * (kGroup * 128u) * 4u);
#pragma unroll 1
                        for (int d = 0; d < 4; ++d)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (mine >> j & 1u)
                                    tma2_load(at + d * kBlock + j * 2048, &kv16_map, full, 256 * (int)rank + 64 * d, row[j]);
                    }
                    __syncwarp();
                    for (uint32_t rest = (groups & ~ones) >> (4 * h) & 0xfu; rest; rest &= rest - 1)
                        copy_values(at + (__ffs(rest) - 1) * 2048, &kv1_map, full, 256 * (int)rank, r, 16 * h + 4 * (__ffs(rest) - 1));
                }
            }
            rd.done(ctl, lane);
        }
    } else if (warp == kSWarp || warp == kOWarp) {
        // ---------------- MMA issuers, the even CTA's for both: one for S, one for O.
        // The tensor core's queue is short, a wait or a commit takes the issuer 50 to
        // 150 clocks: while one issuer is at them the other's products run.
        // O's issuers, which wait for the first P of a piece, also write the pieces
        // down for all warps of their CTA, one ahead.
        Scheduler sched;
        sched.todo = *reinterpret_cast<const Todo *>(ctl.todo);
        bool alive = true;
        if (rank == 1) {
            while (warp == kOWarp && alive && !sched.end) alive = sched.write(p, ctl, lane);
        } else {
            uint32_t g = 0, n = 0;                            // tiles and pieces so far
            uint32_t buf = 0, v_parity = 0;                   // the next half of a tile's values
            Reader rd;
            while (alive) {
                while (warp == kOWarp && alive && !sched.end && sched.todo.written < (int)rd.n + 2) alive = sched.write(p, ctl, lane);
                if (!alive) break;
                const Piece *pc = rd.next(ctl, p.status, limit);
                if (!pc) break;
                // (reductions put what is the same in every lane into uniform
                // registers, where the products take their descriptors from)
                const int t0 = __reduce_max_sync(0xffffffffu, pc->t0), t1 = __reduce_max_sync(0xffffffffu, pc->t1);
                if (__any_sync(0xffffffffu, pc->end)) break;
                if (warp == kSWarp) {
                    constexpr uint32_t id_s = idesc_f16(kRows, kKeys, true, false, false);
                    const uint64_t qd = sdesc_sw128(s0 + kQOff, 16, 1024), kd = sdesc_sw128(s0 + kKOff, 16, 1024);
                    if (t1 > t0) {
                        alive = wait_bar(smem_u32(&ctl.q_tmem), n & 1u, ctl, p.status, limit);
                        if (alive) alive = wait_bar(smem_u32(&ctl.q_full), n & 1u, ctl, p.status, limit);
                        ++n;
                    }
#pragma unroll 1
                    for (int i = t0; alive && i < t1; ++i, ++g) {
                        const uint32_t d_s = tmem + kColS + (g & 1u) * (kKeys / 2);
                        alive = wait_bar(smem_u32(&ctl.s_empty[g & 1u]), ((g >> 1) & 1u) ^ 1u, ctl, p.status, limit);
#pragma unroll 1
                        for (int q = 0; q < 3; ++q) {
                            if (alive) alive = wait_bar(smem_u32(&ctl.k_full[q]), g & 1u, ctl, p.status, limit);
                            if (!alive) break;
                            tc_fence_after();
                            if (elect_one()) {
                                const int kb1 = min(3 * q + 3, n_blocks);
#pragma unroll 1
                                for (int kb = 3 * q; kb < kb1; ++kb) {
                                    const uint64_t kk = kd + (uint64_t)(kb * (kBlock >> 4));
                                    if (kb < kQTmem) {
#pragma unroll
                                        for (int ks = 0; ks < 4; ++ks)
                                            umma2_f16_ts(d_s, tmem + kColQ + kb * 32 + ks * 8, kk + 2 * ks, id_s, (kb | ks) != 0);
                                    } else {
                                        const uint64_t qq = qd + (uint64_t)((kb - kQTmem) * (kBlock >> 4));
#pragma unroll
                                        for (int ks = 0; ks < 4; ++ks) umma2_f16(d_s, qq + 2 * ks, kk + 2 * ks, id_s, 1u);
                                    }
                                }
                                commit2(q < 2 ? smem_u32(&ctl.k_empty[q]) : smem_u32(&ctl.s_full[g & 1u]));
                                if (q == 2 && i == t1 - 1) commit2(smem_u32(&ctl.q_empty));
                            }
                            __syncwarp();
                        }
                    }
                } else {
                    constexpr uint32_t id_o = idesc_f16(kRows, 256, true, false, true);
                    const uint64_t pd = sdesc_sw128(s0 + kPOff, 16, 1024), vd = sdesc_sw128(s0 + kVOff, kBlock, 1024);
#pragma unroll 1
                    for (int i = t0; alive && i < t1; ++i, ++g) {
                        const uint32_t groups = __reduce_or_sync(0xffffffffu, tile_groups(*pc, pc->grid, i));
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            alive = wait_bar(smem_u32(&ctl.v_full[buf]), v_parity, ctl, p.status, limit);
                            if (alive) alive = wait_bar(smem_u32(&ctl.p_full[h]), g & 1u, ctl, p.status, limit);
                            if (!alive) break;
                            tc_fence_after();
                            const uint64_t vb = vd + (uint64_t)(buf * (kVHalf >> 4)), pb = pd + (uint64_t)(h * (kBlock >> 4));
                            const uint32_t on = groups >> (4 * h);
                            const bool begun = i > t0 || (h && (groups & 0xfu));
                            if (elect_one()) {
#pragma unroll 1
                                for (int j = 0; j < 2; ++j) {
                                    const uint64_t vj = vb + (uint64_t)((j * 2 * kBlock) >> 4);
#pragma unroll
                                    for (int ks = 0; ks < 4; ++ks)
                                        if (on >> ks & 1u)
                                            umma2_f16(tmem + kColO + j * 128, pb + 2 * ks, vj + (uint64_t)(ks * kGroup * 128 >> 4), id_o,
                                                      begun || (on & ((1u << ks) - 1)) != 0);
                                }
                                commit2(smem_u32(&ctl.o_done[g & 1u][h]));
                            }
                            __syncwarp();
                            if (++buf == kVBufs) {
                                buf = 0;
                                v_parity ^= 1u;
                            }
                        }
                    }
                }
                rd.done(ctl, lane);
            }
        }
    } else {
        // ---------------- softmax and output.  TMEM lane L holds row L % 64 of this
        // CTA's rows, keys (of S) or dims (of O) of half L / 64.  Two groups of four
        // warps take the tiles in turn, so that one's loads, maxima and barriers run
        // beside the other's exponentials; the running maximum of a row goes from
        // group to group.  (All eight warps on one tile took 3300 clocks a tile.)
        const int tx = (int)threadIdx.x;
        const int quarter = warp & 3, group = warp >> 2, half = quarter >> 1;
        const int r = (warp & 1) * 32 + lane;
        const uint32_t lane_tmem = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t p_bar0 = dsmem_map(smem_u32(&ctl.p_full[0]), 0), p_bar1 = dsmem_map(smem_u32(&ctl.p_full[1]), 0);
        const uint32_t s_bar = dsmem_map(smem_u32(&ctl.s_empty[0]), 0);
        // Named barriers: 1..4 the two warps of a group that share rows, 5 and 6 from
        // one group to the other, 7 all.
        const int rows_bar = 1 + 2 * group + (warp & 1);
        uint8_t *prow = smem + kPOff + half * kBlock + r * 128;
        const uint32_t swz = (uint32_t)(r & 7);
        if (rank == 0 && tx == 0) p.split[cluster] = Split{0, 0, 0, 0};
        // A scale that is not positive is multiplied in where scores are masked.
        const bool plain = p.scale_log2 > 0.f;
        const float scale = plain ? p.scale_log2 : 1.f;
        uint32_t g = 0;                                       // tiles so far
        // The softmax warps run the same sequence of named barriers whatever happens;
        // `alive` (the same in a warp) only gates work on tensor memory and shared
        // memory after a bounded wait gave up.
        bool alive = true;
        Reader rd;
        // The first 256 dims of the queries of piece n, by one group: row r into lanes r
        // and r + 64.  The products that read the piece before's are done.
        const uint32_t q_bar = dsmem_map(smem_u32(&ctl.q_tmem), 0);
        auto load_queries = [&](uint32_t n, bool empty) {
            if (!wait_bar(smem_u32(&ctl.piece_full[n % kPieces]), (n / kPieces) & 1u, ctl, p.status, limit)) return;
            const Piece *pc = &ctl.piece[n % kPieces];
            if (pc->end || pc->t0 == pc->t1) return;
            // four threads a row: 32 bytes of eight rows a load (with a row a thread, 16 bytes
            // each, a windowed prefill took 283 us instead of 271)
            const int64_t row = (int64_t)pc->row0 + kHalf * (int)rank + (warp & 1) * 32 + (lane >> 2);
            const int64_t rows = (int64_t)b.T * p.pr.H;
            const uint2 *src = reinterpret_cast<const uint2 *>(p.q_lat + row * D_L) + (lane & 3);
#pragma unroll 1
            for (int c = 0; c < 128; c += 64) {
                uint32_t u[2][32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const int of = 8 * (e >> 3);              // rows of lane, lane + 8, + 16 and + 24
                    const uint2 x = row + of < rows ? __ldg(src + of * (D_L / 4) + c / 2 + 4 * (e & 7)) : make_uint2(0, 0);
                    const int at = 4 * (e & 7) + 2 * (e >> 3 & 1);
                    u[e >> 4][at] = x.x, u[e >> 4][at + 1] = x.y;
                }
                if (c == 0) {
                    // the loads are under way: now the scores of the last tile have to be there
                    if (!empty && !wait_bar(smem_u32(&ctl.s_full[(g - 1) & 1u]), ((g - 1) >> 1) & 1u, ctl, p.status, limit)) return;
                    tc_fence_after();
                }
                tmem_st_16x256_x8(lane_tmem + kColQ + c, u[0]);
                tmem_st_16x256_x8(lane_tmem + (16u << 16) + kColQ + c, u[1]);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_remote(q_bar);
        };
        // The position of this thread's row in piece n, -1 without one.
        auto row_pos = [&](const Piece *pc) {
            const int row = kHalf * (int)rank + r;
            if (row >= pc->nrows) return -1;
            const int pos = token_pos(b, (pc->row0 + row) / p.pr.H, p.status);
            if (pos >= 0 && (pc->kv0 < 0 || any_row(b, pc->seq, pc->kv0, pos) < 0)) {
                flag(p.status, DSA_DEV_BAD_POSITION);
                return -1;
            }
            return pos;
        };
        if (group == 1) load_queries(0, true);
        int pos = -1, next_pos = -1;
        bool known = false;                                   // next_pos is the next piece's
        // A piece's output waits for its last products: until those are done it is
        // owed, and the next piece is looked up.
        const Piece *owed = nullptr;
        float m_owed = 0.f, l_owed = 0.f;                     // as m and l below
        int pos_owed = -1;
        while (true) {
            const Piece *pc = rd.next(ctl, p.status, limit);
            if (named_barrier_or(7, kSoftmaxWarps * 32, !pc)) break;
            if (pc->end && !owed) break;
            const int t0 = pc->t0, t1 = pc->t1, n_first = pc->grid.n_first;
            if (!pc->end) pos = known ? next_pos : row_pos(pc);
            // Every row of the item sees every key of the tiles [clear0, clear1).
            const int64_t open = (int64_t)pc->hi - p.pr.window + 1;      // the last token's window begins here
            const int clear0 = n_first + (open <= pc->grid.pos0 ? 0 : (int)((open - pc->grid.pos0 + kKeys - 1) / kKeys));
            const int clear1 = plain ? n_first + (pc->min_pos + 1 - pc->grid.pos0) / kKeys : 0;
            float m = -INFINITY, l = 0.f;                     // m: as of this group's last tile
            const uint32_t g0 = g;                            // of the piece's first tile
            if (owed) {
                // ---- the output of the piece before
                const bool empty = owed->t1 == owed->t0;
                const int row = kHalf * (int)rank + r;
                const bool mine = row < owed->nrows;
                if (!empty) {
                    // its last tile was g0 - 1.  That tile's group has not been at another
                    // since, and the maxima of its tile before are not wanted any more.
                    const int last = (int)((g0 - 1) & 1u);
                    if (alive) alive = wait_o(1, g0 - 1);
                    tc_fence_after();
                    float *const m_last = ctl.red[last][(((g0 - 1) >> 1) & 1u) ^ 1u][0];
                    if (last == group && half == 0) m_last[r] = m_owed;
                    named_barrier(7, kSoftmaxWarps * 32);
                    const float mn = m_last[r];
                    auto &sums = ctl.red[last ^ 1];               // read by all of its group
                    // (not by the maximum: scores of NaN leave it at -infinity, but not the sum at 0)
                    sums[group][half][r] = l_owed == 0.f ? 0.f : l_owed * ex2(m_owed - mn);
                    m_owed = mn;
                    named_barrier(7, kSoftmaxWarps * 32);
                    l_owed = (sums[0][0][r] + sums[0][1][r]) + (sums[1][0][r] + sums[1][1][r]);
                }
                const bool none = pos_owed < 0 || l_owed == 0.f;  // a sum of NaN is not none
                if (alive && row - lane < owed->nrows) {
                    // 64 bytes of each of the warp's 32 rows at a time, turned in the warp's
                    // share of P's buffer so that stores write whole sectors (a row a lane
                    // straight from the accumulator took 13,000 clocks).
                    // A part goes to slot 2c where the item began in an earlier cluster, else to 2c + 1.
                    const bool whole = owed->whole, narrow = p.out_bf16;
                    const int64_t out_row = (int64_t)owed->row0 + row;
                    const int64_t part_row = ((int64_t)2 * cluster + (owed->t0 == 0 ? 1 : 0)) * kRows + row;
                    const float factor = whole ? 1.f / l_owed : 1.f;
                    const int col0 = 256 * half + 128 * group, bytes = narrow ? 2 : 4;
                    const int rows_left = owed->nrows - (row - lane);            // of the warp's 32
                    uint8_t *stage = smem + kPOff + warp * 2048;
                    uint8_t *dst = static_cast<uint8_t *>(whole ? p.out : p.part_o) +
                                   (((whole ? out_row : part_row) - lane + (lane >> 2)) * D_L + col0) * bytes + 16 * (lane & 3);
                    const uint32_t o_tmem = lane_tmem + kColO + 128 * group;
                    const int step = 64 / bytes;
#pragma unroll 1
                    for (int c = 0; c < 128; c += step) {
                        uint32_t w[16];
                        if (narrow && !empty) {
                            uint32_t o[32];
                            tmem_ld32(o_tmem + c, o);
                            tmem_wait_ld(o);
                            if (whole) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(o[2 * e]) * factor, __uint_as_float(o[2 * e + 1]) * factor);
                                    w[e] = *reinterpret_cast<const uint32_t *>(&h);
                                }
                            } else {
                                float top = 0.f;
#pragma unroll
                                for (int e = 0; e < 32; ++e) top = fmaxf(top, fabsf(__uint_as_float(o[e])));
                                // values below 2^15 after it: those down to 2^-29 of the largest keep 11 bits
                                const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127, -112), 127) - 14;
                                const float unit = __int_as_float((127 - ex) << 23);
                                if (mine) p.part_unit[part_row * 16 + ((col0 + c) >> 5)] = __int_as_float((127 + ex) << 23);
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const __half2 h = __floats2half2_rn(__uint_as_float(o[2 * e]) * unit, __uint_as_float(o[2 * e + 1]) * unit);
                                    w[e] = *reinterpret_cast<const uint32_t *>(&h);
                                }
                            }
                        } else if (!empty) {
                            tmem_ld16(o_tmem + c, w);
                            tmem_wait_ld(w);
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * factor);
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<uint4 *>(stage + sw64_offset((uint32_t)lane, (uint32_t)q)) =
                                none ? make_uint4(0, 0, 0, 0) : make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
                        __syncwarp();
                        uint4 v[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            v[q] = *reinterpret_cast<const uint4 *>(stage + sw64_offset((uint32_t)(8 * q + (lane >> 2)), (uint32_t)(lane & 3)));
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (8 * q + (lane >> 2) < rows_left) *reinterpret_cast<uint4 *>(dst + (int64_t)(8 * q) * D_L * bytes + c * bytes) = v[q];
                        __syncwarp();
                    }
                    if (mine && half == 0 && group == 0) {
                        if (!whole) *reinterpret_cast<float2 *>(p.part_ml + part_row * 2) = none ? make_float2(-INFINITY, 0.f) : make_float2(m_owed, l_owed);
                        else if (p.lse) p.lse[out_row] = none ? -INFINITY : (m_owed + log2f(l_owed)) * kLn2;
                    }
                    if (!whole && owed->t0 == 0 && rank == 0 && tx == 0) {
                        // the clusters that the item's tiles reach into
                        const int total = ctl.head.total, n = ctl.head.clusters;
                        int rest = owed->rest, parts = 1;
                        for (int k = cluster + 1; rest > 0 && k < n; ++k, ++parts) rest -= share(total, k + 1, n) - share(total, k, n);
                        p.split[cluster] = Split{owed->row0, owed->nrows, cluster, parts};
                    }
                }
                tc_fence_before();                                // O may be overwritten after the next P
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl.piece_empty[(rd.n - 1) % kPieces]));
                owed = nullptr;
                named_barrier(7, kSoftmaxWarps * 32);             // all have read O, and their staging ends, before any stores a P
            }
            if (pc->end) break;
            for (int i = t0 + ((int)(g0 & 1u) ^ group); i < t1; i += 2) {
                g = g0 + (uint32_t)(i - t0);
                const uint32_t s_tmem = lane_tmem + kColS + (g & 1u) * (kKeys / 2);
                if (alive) alive = wait_bar(smem_u32(&ctl.s_full[g & 1u]), (g >> 1) & 1u, ctl, p.status, limit);
                tc_fence_after();
                if ((i < clear0 || i >= clear1) && alive) {
                    // one bit a key of this half: the window's and the first ones'
                    const int kp = pc->grid.tile(i) + kHalf * half;
                    const int from = (int)max((int64_t)0, (int64_t)pos - p.pr.window + 1);
                    // (keys of the first tiles from pos0 on are those of the others)
                    uint64_t see = (key_bits(from - kp, pos + 1 - kp) | key_bits(pc->s_lo - kp, min(pc->s_hi, pos + 1) - kp)) &
                                   key_bits(0, i < n_first ? pc->grid.pos0 - kp : kHalf);
                    if (i == pc->grid.last && pc->grid.wrap < kKeys) {
                        const int cut = pc->grid.wrap - kHalf * half, ks = pc->grid.first_pos - cut;
                        see = (see & key_bits(0, cut)) | key_bits(pc->s_lo - ks, min(min(pc->s_hi, pc->grid.pos0), pos + 1) - ks);
                    }
                    const float factor = plain ? 1.f : p.scale_log2;
#pragma unroll 1
                    for (int c = 0; c < 64; c += 16) {
                        const uint32_t bits = (uint32_t)(see >> c);
                        uint32_t u[16];
                        tmem_ld16(s_tmem + c, u);
                        tmem_wait_ld(u);
#pragma unroll
                        for (int e = 0; e < 16; ++e) u[e] = bits & (1u << e) ? __float_as_uint(__uint_as_float(u[e]) * factor) : 0xff800000u;
                        tmem_st16(s_tmem + c, u);
                    }
                    tmem_wait_st();
                }
                float top = -INFINITY;
                if (alive) {
#pragma unroll 1
                    for (int c = 0; c < 64; c += 32) {
                        uint32_t u[32];
                        tmem_ld32(s_tmem + c, u);
                        tmem_wait_ld(u);
                        float a0 = top, a1 = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            a0 = fmaxf(fmaxf(a0, __uint_as_float(u[e])), __uint_as_float(u[e + 1]));
                            a1 = fmaxf(fmaxf(a1, __uint_as_float(u[e + 2])), __uint_as_float(u[e + 3]));
                        }
                        top = fmaxf(a0, a1);
                    }
                }
                auto &red = ctl.red[group][(g >> 1) & 1u];
                red[half][r] = top;
                named_barrier(rows_bar, 64);
                const float mx = fmaxf(top, red[half ^ 1][r]) * scale;
                float mo = -INFINITY;                         // as of the tile before
                if (i > t0) {
                    named_barrier(5 + (group ^ 1), kSoftmaxWarps * 32);
                    mo = ctl.m[(g - 1) & 1u][r];
                }
                // The maximum is only raised by more than 2^20 at a time: the result is
                // the same either way, P's and O's exponents have room, and O is
                // rescaled seldom (with 2^8, rows whose first tile shows them a few keys
                // made every other tile of a windowed prefill wait for it).
                const bool raise = mx > mo + kRescaleLog2 || (mo == -INFINITY && mx != -INFINITY);
                const float mn = raise ? mx : mo;
                if (i + 1 < t1) {
                    if (half == 0) ctl.m[g & 1u][r] = mn;
                    named_barrier_arrive(5 + group, kSoftmaxWarps * 32);
                }
                const float al = raise && mo != -INFINITY ? ex2(mo - mn) : raise ? 0.f : 1.f;
                l *= m == -INFINITY ? 0.f : ex2(m - mn);      // (1 where the maximum stayed)
                m = mn;
                const float mm = mn == -INFINITY ? 0.f : -mn;
                uint64_t sum = f2(0.f, 0.f);
                if (alive) {
                    // P in pairs of bf16 over the first half of S's own columns, until
                    // its place in shared memory is free.  bf16, the values' type, is what
                    // one product takes: P is off by up to 2^-8 of itself, outputs by 0.001
                    // of their size (the sum is of P before it).  A second product of the
                    // remainders would take O's clocks again, and their place in shared
                    // memory is not there.
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        uint32_t u[32], w[16];
                        tmem_ld32(s_tmem + 32 * c, u);
                        tmem_wait_ld(u);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float x = ex2(fmaf(__uint_as_float(u[2 * e]), scale, mm));
                            const float y = ex2(fmaf(__uint_as_float(u[2 * e + 1]), scale, mm));
                            sum = f2_add(sum, f2(x, y));
                            const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
                            w[e] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                        tmem_st16(s_tmem + 16 * c, w);
                    }
                    tmem_wait_st();
                }
                const float2 s2 = f2_get(sum);
                l += s2.x + s2.y;
                // O may be rescaled once the product of the tile before is done
                if (i > t0 && __any_sync(0xffffffffu, al != 1.f)) {
                    if (alive) alive = wait_o(1, g - 1);
                    if (alive) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 256; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(lane_tmem + kColO + c, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                            tmem_st32(lane_tmem + kColO + c, o);
                        }
                        tmem_wait_st();
                    }
                }
                // The product begins with the first half of the keys: of the second
                // half's warps it only needs that O is as it should be (said once the
                // product before has begun, or its own count would be taken for this one's).
                // P's half is free once the same half of the product before is done.
                if (i > t0 && alive) alive = wait_o(0, g - 1);
                if (half == 1 && alive) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_remote(p_bar0);
                }
                if (i > t0 && half == 1 && alive) alive = wait_o(1, g - 1);
                if (alive) {
                    uint32_t w[32];
                    tmem_ld32(s_tmem, w);
                    tmem_wait_ld(w);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<uint4 *>(prow + ((c ^ swz) << 4)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        arrive_remote(half ? p_bar1 : p_bar0);
                        arrive_remote(s_bar + (g & 1u) * 8);  // the next S but one may come
                    }
                }
            }
            g = g0 + (uint32_t)(t1 - t0);
            // ---- the next piece's queries, by the group that is done first, once the
            // last tile is scored
            const bool empty = t1 == t0;
            if (empty ? group == 0 : (int)((g - 1) & 1u) != group) {
                if (alive) load_queries(rd.n + 1, empty);
            }
            // its positions, asked for before they are wanted
            known = mbar_test(smem_u32(&ctl.piece_full[(rd.n + 1) % kPieces]), ((rd.n + 1) / kPieces) & 1u);
            if (known) {
                const Piece *nx = &ctl.piece[(rd.n + 1) % kPieces];
                next_pos = nx->end ? -1 : row_pos(nx);
            }
            owed = pc;
            m_owed = m, l_owed = l, pos_owed = pos;
            ++rd.n;
        }
    }

    __syncwarp();
    if (*(volatile int32_t *)&ctl.abort_flag) {
        // let copies in flight land before the shared memory goes
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 1000000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    pdl_trigger();
    cluster_sync_all();
    if (warp == kSWarp) {
        tc_fence_after();
        tmem_dealloc2(tmem, kTmemCols);
    }
}

// One CTA: the items of the call, their costs, and where each cluster begins.
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) mla_plan_kernel(const Problem p, uint32_t *status, int max_items, int clusters,
                                                                PlanHead *head, Item *items, Start *start, int32_t *item0) {
    __shared__ int sh[64];
    pdl_wait();
    const DevBatch &b = p.b;
    int base = 0;                                             // items of the sequences before
    for (int s0 = 0; s0 < b.B; s0 += kPlanThreads) {
        const int s = s0 + (int)threadIdx.x;
        int n = 0;
        if (s < b.B) {
            const int t0 = __ldg(b.cu_q + s), t1 = __ldg(b.cu_q + s + 1);
            if (t0 < 0 || t1 < t0 || t1 > b.T) flag(status, DSA_DEV_BAD_POSITION);
            else n = ((t1 - t0) * p.H + kRows - 1) / kRows;
        }
        int sum;
        const int before = plan_scan<kPlanThreads>(n, sum, sh);
        if (s < b.B) item0[s] = base + before;
        base += sum;
    }
    __syncthreads();
    if (base > max_items) {                                   // only where cu_q falls somewhere
        if (threadIdx.x == 0) flag(status, DSA_DEV_BAD_POSITION);
        base = max_items;
    }
    int total = 0;
    for (int i0 = 0; i0 < base; i0 += kPlanThreads) {
        const int i = i0 + (int)threadIdx.x;
        int cost = 0;
        Item it{};
        if (i < base) {
            int lo = 0, hi = b.B;                             // item0[lo] <= i < item0[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (item0[mid] <= i) lo = mid; else hi = mid;
            }
            const int t0 = __ldg(b.cu_q + lo), t1 = __ldg(b.cu_q + lo + 1);
            it.seq = lo;
            it.row0 = t0 * p.H + (i - item0[lo]) * kRows;
            it.nrows = min(kRows, t1 * p.H - it.row0);
            item_fill(p, it);
            cost = item_cost(it.n);
        }
        int sum;
        const int before = plan_scan<kPlanThreads>(cost, sum, sh);
        if (i < base) {
            it.cost0 = total + before;
            items[i] = it;
        }
        total += sum;
    }
    __syncthreads();
    const int n = min(clusters, total);
    if (threadIdx.x == 0) *head = PlanHead{total, n};
    for (int c = (int)threadIdx.x; c < n; c += kPlanThreads) {
        const int at = share(total, c, n);
        int lo = 0, hi = base;                                // items[lo].cost0 <= at < items[hi].cost0
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (items[mid].cost0 <= at) lo = mid; else hi = mid;
        }
        start[c] = Start{lo, at - items[lo].cost0};
    }
    pdl_trigger();
}

// Joins the parts of an item that several clusters share: a row's 512 dims over as
// many threads as there are 16-byte pieces, as many parts at a time as there are
// loads in flight.
constexpr int kJoinThreads = 256;
constexpr int kJoinLoads = 8;
template <bool kBf16> constexpr int kJoinRows = kBf16 ? kJoinThreads / 64 : kJoinThreads / 128;

template <bool kBf16>
__global__ void __launch_bounds__(kJoinThreads) mla_combine_kernel(const Split *split, const void *part_o, const float *part_unit,
                                                                   const float *part_ml, void *out, float *lse) {
    constexpr int kPer = kBf16 ? 8 : 4;                       // dims a thread
    constexpr int kRowThreads = D_L / kPer;
    __shared__ float wgt[kJoinRows<kBf16>][kClusters];
    pdl_wait();
    const Split s = split[blockIdx.x];
    const int mine = threadIdx.x / kRowThreads, tx = threadIdx.x % kRowThreads, lane = threadIdx.x & 31;
    const int row = blockIdx.y * kJoinRows<kBf16> + mine;
    if (blockIdx.y * kJoinRows<kBf16> >= s.nrows) return;     // 0 rows without a shared item
    const bool there = row < s.nrows;
    auto slot = [&](int k) { return ((int64_t)2 * (s.first + k) + (k == 0 ? 1 : 0)) * kRows + (there ? row : 0); };
    uint4 v[kJoinLoads];
    float unit[kJoinLoads];
    auto load = [&](int k0) {
#pragma unroll
        for (int q = 0; q < kJoinLoads; ++q)
            if (k0 + q < s.parts) unit[q] = kBf16 ? part_unit[slot(k0 + q) * 16 + tx / 4] : 1.f;
#pragma unroll
        for (int q = 0; q < kJoinLoads; ++q)
            if (k0 + q < s.parts)
                v[q] = *(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(part_o) + slot(k0 + q) * (D_L * (kBf16 ? 2 : 4))) + tx);
    };
    load(0);                                                  // beside the statistics, not behind them
    // every warp of the row has all maxima and sums; one lets the others have the weights
    float M = -INFINITY, L = 0.f;
    float2 ml[(kClusters + 31) / 32];
#pragma unroll
    for (int i = 0; i < (kClusters + 31) / 32; ++i) {
        const int k = lane + 32 * i;
        ml[i] = k < s.parts ? *reinterpret_cast<const float2 *>(part_ml + slot(k) * 2) : make_float2(-INFINITY, 0.f);
        M = fmaxf(M, ml[i].x);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
#pragma unroll
    for (int i = 0; i < (kClusters + 31) / 32; ++i) {
        const float w = ml[i].x == -INFINITY ? 0.f : ex2(ml[i].x - M);
        L += w * ml[i].y;
        if (tx < 32 && lane + 32 * i < s.parts) wgt[mine][lane + 32 * i] = w;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
    __syncthreads();
    float acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < s.parts; k0 += kJoinLoads) {
        if (k0) load(k0);
#pragma unroll
        for (int q = 0; q < kJoinLoads; ++q) {
            if (k0 + q < s.parts) {
                const float w = wgt[mine][k0 + q] * unit[q];
                const uint32_t u[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (kBf16) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[e]));
                        acc[2 * e] += w * f.x;
                        acc[2 * e + 1] += w * f.y;
                    } else {
                        acc[e] += w * __uint_as_float(u[e]);
                    }
                }
            }
        }
    }
    if (!there) return;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int64_t at = ((int64_t)s.row0 + row) * D_L + kPer * tx;
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (kBf16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
            u[e] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            u[e] = __float_as_uint(acc[e] * inv);
        }
    }
    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(out) + at * (kBf16 ? 2 : 4)) = make_uint4(u[0], u[1], u[2], u[3]);
    if (lse && tx == 0) lse[(int64_t)s.row0 + row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// ---------------------------------------------------------------- host
namespace {

struct MlaLayout {
    size_t head, start, split, ml, part, unit, item0, items, total;
    int64_t max_items;
};
MlaLayout mla_layout(int64_t T, int64_t B, int64_t H, size_t off) {
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) / 256 * 256;
        return at;
    };
    MlaLayout L;
    L.max_items = T * H / kRows + B;
    L.head = take(sizeof(PlanHead));
    L.start = take(kClusters * sizeof(Start));
    L.split = take(kClusters * sizeof(Split));
    L.ml = take((size_t)2 * kClusters * kRows * 2 * sizeof(float));
    L.part = take((size_t)2 * kClusters * kRows * D_L * sizeof(float));
    L.unit = take((size_t)2 * kClusters * kRows * 16 * sizeof(float));
    L.item0 = take((size_t)B * sizeof(int32_t));
    L.items = take((size_t)L.max_items * sizeof(Item));
    L.total = off;
    return L;
}

}  // namespace

size_t mla_attn_workspace(int T, int B, int H) { return mla_layout(T, B, H, kStatusBytes).total; }

bool mla_attn_countable(int T, int B, int H, int max_kv) {
    // costs are 32-bit numbers
    return mla_layout(T, B, H, kStatusBytes).max_items * ((int64_t)max_kv / kKeys + 3 + kItemCost) < INT32_MAX;
}

cudaError_t launch_mla_attn(const MlaLaunch &a, const MlaMaps &maps, const DevBatch &b, void *ws, cudaStream_t stream) {
    const MlaLayout L = mla_layout(b.T, b.B, a.H, kStatusBytes);
    uint8_t *w = static_cast<uint8_t *>(ws);
    uint32_t *status = reinterpret_cast<uint32_t *>(w);
    MlaParams p{};
    p.status = status;
    p.q_lat = a.q_lat;
    PlanHead *head = reinterpret_cast<PlanHead *>(w + L.head);
    Item *items = reinterpret_cast<Item *>(w + L.items);
    Start *start = reinterpret_cast<Start *>(w + L.start);
    p.head = head;
    // No more sequences and items than threads: the kernel plans for itself.  Each
    // thread goes through its item's tokens; with fewer than 8 heads there are many.
    p.one = (int64_t)b.max_q * a.H <= kRows;
    const bool here = b.B <= kThreads && (p.one || (L.max_items <= kThreads && a.H >= 8));
    p.items = here ? nullptr : items;
    p.start = start;
    p.split = reinterpret_cast<Split *>(w + L.split);
    p.part_o = w + L.part;
    p.part_unit = reinterpret_cast<float *>(w + L.unit);
    p.part_ml = reinterpret_cast<float *>(w + L.ml);
    p.out = a.out;
    p.out_bf16 = a.out_bf16;
    p.lse = a.lse;
    p.scale_log2 = a.sm_scale * 1.4426950408889634f;
    p.tail = a.tail;
    p.rows_per_box = !b.block_table || b.block_size % 64 == 0 ? 64 : b.block_size % 16 == 0 ? 16 : 0;
    // (a box must not pass the end of a page)
    p.pr = Problem{b, a.H, a.window, a.n_sink, a.sink_pos0, b.block_table && p.rows_per_box ? p.rows_per_box : 1};
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(mla_attn_kernel), 12, kSmem);
    if (e != cudaSuccess) return e;
    if (!here) {
        e = launch_k(mla_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, true, p.pr, status, (int)L.max_items, kClusters, head,
                     items, start, reinterpret_cast<int32_t *>(w + L.item0));
        if (e != cudaSuccess) return e;
    }
    e = launch_k(mla_attn_kernel, dim3(2 * kClusters), dim3(kThreads), kSmem, stream, true, p, maps.q_lat, maps.q_rope, maps.kv64,
                 maps.kv16, maps.kv1);
    if (e != cudaSuccess) return e;
    const int rows = a.out_bf16 ? kJoinRows<true> : kJoinRows<false>;
    return launch_k(a.out_bf16 ? mla_combine_kernel<true> : mla_combine_kernel<false>, dim3(kClusters, kRows / rows),
                    dim3(kJoinThreads), 0, stream, true, (const Split *)p.split, (const void *)p.part_o, (const float *)p.part_unit,
                    (const float *)p.part_ml, a.out, a.lse);
}

}  // namespace dsa
