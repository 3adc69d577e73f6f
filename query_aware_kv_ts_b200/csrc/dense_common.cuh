// What the dense attention kernels share: their arguments, and the division
// of the work over the blocks.
//
// An item is a group of up to TT query tokens of one sequence with the G
// query heads of one kv head, against the tokens that the last of them sees.
// The items of the whole call stand in one line, sequence by sequence, kv
// head by kv head, each as long as its tokens plus a constant, and block c
// takes the c-th of as many equal parts of that line as there are blocks (of
// fewer, where parts would be shorter than a tile).  Parts end inside items,
// at a multiple of kDenseTile tokens; the pieces of such an item are joined in
// their order.  So blocks are equally loaded at any mixture of lengths, and
// one long sequence spreads over the whole GPU.  Everything follows from the
// device's offsets in closed form, and no result depends on which block comes
// first.
#pragma once

#include "ts_device.cuh"
#include "ts_internal.h"

namespace ts {

constexpr int kDenseTile = 128;         // tokens per K / V tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2f = 0.693147180559945309f;

// A block's ends inside items, for dense_merge.
struct __align__(16) DensePiece {
    int32_t b, g, t;     // the item that the block begins and does not end
    int32_t flags;
};
enum : int32_t {
    kPieceHead = 1,      // the block begins an item that it does not end
    kPieceThrough = 2,   // the block lies wholly inside an item: neither begins nor ends it
};

struct DenseArgs {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_st, st, sh;
    const int64_t *seq_off, *q_off;
    __nv_bfloat16 *out;
    float *lse;
    uint32_t *ctrl;
    DensePiece *pieces;   // [grid]
    float *part;          // [2 * grid][rows of an item][D + 4]: weighted V sums, then (max in base 2, sum)
    int B, Hq, Hkv, G;
    int TT;               // query tokens per item
    int single;           // 1: the sequences with one query token, 0: those with more
    int split;            // 0: parts end between items only
    int item_cost;        // what an item's beginning and end take, in tokens of its tiles
    double inv_grid;      // 1 / blocks
    int slot_rows;        // rows of one partial result
    uint32_t *counts;     // [grid][8], zero between calls: of the item that a block begins and does not end
    float scale_log2;
    // paged cache (page_table != null): token i of sequence b is pool row
    // page_table[b * pt_stride + (i >> page_shift)] << page_shift | (i & (page - 1))
    const int32_t *page_table;
    int pt_stride, page_shift;
    int64_t pool_pages;
    int64_t kv_rows;      // token rows of the cache (of the pool)
    // K and V tiles in shared memory: rows of 64 channels (128 bytes, 128-byte
    // swizzle), 8 tokens together; bytes from 8 tokens to the next 8, and from
    // the first 64 channels to the others.  A paged cache's boxes hold whole
    // rows of some tokens, a packed one's 64 channels of all 128.
    int group_stride, half_stride;
    int box_shift;        // log2 of the tokens of one box
};

struct DenseItem {
    int32_t b, g, t;           // sequence, kv head, group of query tokens
    int32_t kt0, kt1;          // tiles of this piece, kt0 < kt1 (one empty tile for an item that sees nothing)
    int32_t tiles;             // of the whole item
    int32_t tokens;            // query tokens of the item
    int32_t slot;              // -1: the whole item; else its piece's place in the partial results
    int64_t q_row;             // its first query row
    int64_t off, n, first_pos; // the sequence's first row and length; position of its first query token
    int64_t line;              // the sequence's beginning on the line, and its query tokens
    int32_t f;
    int32_t head;              // of a shared item, the block that begins it
};

__device__ __forceinline__ int64_t seq_items(const DenseArgs &a, int64_t f)
{
    // (f stays below 2^25: a 32-bit division)
    return a.single ? f == 1 : (f > 1 ? ((uint32_t)f + (uint32_t)a.TT - 1u) / (uint32_t)a.TT : 0u);
}
// Length of the first t items of one kv head of a sequence on the line:
// item s counts base + (s + 1) TT + a.item_cost.
__device__ __forceinline__ int64_t items_cost(const DenseArgs &a, int64_t base, int64_t t)
{
    return t * (base + a.item_cost) + (int64_t)a.TT * (t * (t + 1) / 2);
}

// The first sequence from b on that has items, B if none has.  Whole warp, 32
// sequences a round trip.
__device__ __forceinline__ int dense_next_seq(const DenseArgs &a, int b)
{
    for (; b < a.B; b += 32) {
        const int i = b + (threadIdx.x & 31);
        const bool has = i < a.B && seq_items(a, __ldcg(a.q_off + i + 1) - __ldcg(a.q_off + i)) > 0;
        const uint32_t vote = __ballot_sync(0xffffffffu, has);
        if (vote)
            return b + __ffs(vote) - 1;
    }
    return a.B;
}

// A place on the line, at a tile boundary of an item (b == B: its end).
struct DensePlace {
    int32_t b, g, t, cut;
    int32_t tiles;            // of the item
    int64_t f, n, off, q0;    // of the sequence: query tokens, tokens, first token row, first query row
    int64_t line;             // the sequence's beginning on the line
};

__device__ __forceinline__ void dense_item_at(const DenseArgs &a, DensePlace &p)
{
    const int64_t last = p.n - p.f + min((int64_t)(p.t + 1) * a.TT, p.f);   // tokens that its last query sees
    p.tiles = last > 0 ? (int32_t)((last + kDenseTile - 1) / kDenseTile) : 1;
}

__device__ __forceinline__ void dense_load_seq(const DenseArgs &a, DensePlace &p)
{
    p.off = __ldcg(a.seq_off + p.b);
    p.n = __ldcg(a.seq_off + p.b + 1) - p.off;
    p.q0 = __ldcg(a.q_off + p.b);
    p.f = __ldcg(a.q_off + p.b + 1) - p.q0;
}

__device__ __forceinline__ int64_t dense_head_cost(const DenseArgs &a, const DensePlace &p)
{
    return items_cost(a, p.n > p.f ? p.n - p.f : 0, seq_items(a, p.f));
}

__device__ __forceinline__ void dense_next_item(const DenseArgs &a, DensePlace &p)
{
    p.cut = 0;
    if (++p.t >= seq_items(a, p.f)) {
        p.t = 0;
        if (++p.g == a.Hkv) {
            p.g = 0;
            p.line += a.Hkv * dense_head_cost(a, p);   // (sequences without items take no room on it)
            p.b = dense_next_seq(a, p.b + 1);
            if (p.b < a.B)
                dense_load_seq(a, p);
        }
    }
    if (p.b < a.B)
        dense_item_at(a, p);
}

// The offsets and the line's sequence boundaries, [B + 1] each, as
// dense_locate reads them.
struct DenseTables {
    int64_t *start, *seq_off, *q_off;
};

// The line cut into parts, none shorter than a tile: so a part inside an item
// holds a tile of it.
struct DenseParts {
    int64_t total;
    int32_t count;
    double inverse;

    __device__ __forceinline__ void cut(const DenseArgs &a, int64_t length)
    {
        total = length;
        const int64_t most = length / (kDenseTile + 1);   // (1 for at()'s rounding)
        count = most < (int64_t)gridDim.x ? (most > 1 ? (int32_t)most : 1) : (int32_t)gridDim.x;
        inverse = count == (int32_t)gridDim.x ? a.inv_grid : 1.0 / count;
    }
    // Where part c begins.
    __device__ __forceinline__ int64_t at(int c) const
    {
        return c >= count ? total : (int64_t)((double)total * c * inverse);
    }
};

// The tile of an item of `cost` at which a part that ends rem after the item's
// beginning is cut (its number of tiles: behind it).  Items of 8 tiles or more
// have no piece of a single one, whose start and join cost more than its tile;
// over prompts, mixed steps and decode batches that is within 3 % of cutting
// anywhere, in both directions.
__device__ __forceinline__ int32_t dense_cut(const DenseArgs &a, int64_t rem, int64_t cost, int32_t tiles)
{
    if (!a.split)
        return 2 * rem < cost ? 0 : tiles;
    const int64_t c = rem < a.item_cost - kDenseTile / 2 ? 0 : (rem - a.item_cost + kDenseTile / 2) / kDenseTile;
    if (c >= tiles || (tiles >= 8 && c > tiles - 2))
        return tiles;
    return tiles >= 8 && c < 2 ? 0 : (int32_t)c;
}

__device__ __forceinline__ void dense_table_seq(const DenseTables &tab, DensePlace &p)
{
    p.off = tab.seq_off[p.b];
    p.n = tab.seq_off[p.b + 1] - p.off;
    p.q0 = tab.q_off[p.b];
    p.f = tab.q_off[p.b + 1] - p.q0;
    p.line = tab.start[p.b];
}

__device__ __forceinline__ DensePlace dense_locate(const DenseArgs &a, const DenseTables &tab, int64_t x)
{
    const int64_t *start = tab.start;
    DensePlace p;
    p.b = a.B;
    p.g = p.t = p.cut = p.tiles = 0;
    p.f = p.n = p.off = p.q0 = p.line = 0;
    if (x >= start[a.B])
        return p;
    int lo = 0, hi = a.B;                      // start[lo] <= x < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    p.b = lo;
    dense_table_seq(tab, p);
    const int64_t base = p.n > p.f ? p.n - p.f : 0, items = seq_items(a, p.f);
    const int64_t head = items_cost(a, base, items);
    int64_t rem = x - start[lo];
    while (rem >= head) {                      // at most 7 times
        rem -= head;
        ++p.g;
    }
    int64_t t0 = 0, t1 = items;                // items_cost(t0) <= rem < items_cost(t1)
    while (t1 - t0 > 1) {
        const int64_t mid = (t0 + t1) >> 1;
        if (items_cost(a, base, mid) <= rem)
            t0 = mid;
        else
            t1 = mid;
    }
    p.t = (int32_t)t0;
    rem -= items_cost(a, base, t0);
    dense_item_at(a, p);
    p.cut = dense_cut(a, rem, base + (t0 + 1) * a.TT + a.item_cost, p.tiles);
    if (p.cut == p.tiles) {                    // the next item's beginning
        p.cut = 0;
        if (++p.t == items) {
            p.t = 0;
            if (++p.g == a.Hkv) {
                p.g = 0;
                do {
                    ++p.b;
                } while (p.b < a.B && start[p.b + 1] == start[p.b]);
                if (p.b < a.B)
                    dense_table_seq(tab, p);
            }
        }
        if (p.b < a.B)
            dense_item_at(a, p);
    }
    return p;
}

// The pieces of a block's part from at to end, one after another: next() is
// false at the end.  All lanes of a warp walk alike.
struct DenseWalk {
    DensePlace at, end;
    DenseParts parts;

    __device__ __forceinline__ bool same_item() const { return at.b == end.b && at.g == end.g && at.t == end.t; }
    // For dense_merge; call it before next().
    __device__ __forceinline__ DensePiece piece(const DenseArgs &a) const
    {
        DensePiece p;
        p.b = end.b;
        p.g = end.g;
        p.t = end.t;
        const bool inside = end.b < a.B && end.cut > 0;     // the part ends inside an item
        p.flags = inside ? (same_item() && at.cut > 0 ? kPieceThrough : kPieceHead) : 0;
        return p;
    }
    __device__ __forceinline__ bool next(const DenseArgs &a, DenseItem &it)
    {
        if (at.b >= a.B)
            return false;
        const bool last = same_item();
        if (last && at.cut >= end.cut)
            return false;
        it.b = at.b;
        it.g = at.g;
        it.t = at.t;
        it.kt0 = at.cut;
        it.kt1 = last ? end.cut : at.tiles;
        it.tiles = at.tiles;
        it.tokens = (int32_t)min((int64_t)a.TT, at.f - (int64_t)at.t * a.TT);
        it.slot = it.kt0 == 0 && it.kt1 == at.tiles ? -1 : 2 * (int32_t)blockIdx.x + (it.kt0 == 0 ? 1 : 0);
        it.off = at.off;
        it.q_row = at.q0 + (int64_t)at.t * a.TT;
        it.n = at.n;
        it.line = at.line;
        it.f = (int32_t)at.f;
        it.first_pos = at.n - at.f + (int64_t)at.t * a.TT;
        if (last)
            at.cut = end.cut;                                // next() ends here
        else
            dense_next_item(a, at);
        return true;
    }
};

// The block that begins a shared item.
__device__ __forceinline__ int32_t dense_head(const DenseArgs &a, const DenseItem &it, const DenseParts &parts)
{
    if (it.kt0 == 0)
        return (int32_t)blockIdx.x;
    const int64_t base = it.n > it.f ? it.n - it.f : 0;
    const int64_t x = it.line + it.g * items_cost(a, base, seq_items(a, it.f)) + items_cost(a, base, it.t);
    int c = min((int)((float)x * (float)parts.count / (float)parts.total), parts.count - 1);
    while (parts.at(c) > x)
        --c;
    while (parts.at(c + 1) <= x)
        ++c;
    // a part that ends too near the item's beginning ends there
    while (dense_cut(a, parts.at(c + 1) - x, base + (it.t + 1) * (int64_t)a.TT + a.item_cost, it.tiles) == 0)
        ++c;
    return c;
}

// The block's part, found by one warp: the tables (in shared memory, where the
// tiles will be) after one round trip to the offsets, 32 sequences at a time,
// then both ends at once, one in lane 0 and one in lane 1.
constexpr size_t kDenseTableBytes = 3 * sizeof(int64_t) * (kMaxBatch + 1) + 2 * sizeof(DensePlace);
__device__ __forceinline__ void dense_begin(const DenseArgs &a, void *smem, int lane, DenseWalk &w)
{
    int64_t *t = static_cast<int64_t *>(smem);
    const DenseTables tab = {t, t + kMaxBatch + 1, t + 2 * (kMaxBatch + 1)};
    DensePlace *place = reinterpret_cast<DensePlace *>(t + 3 * (kMaxBatch + 1));
    int64_t run = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        int64_t s0 = 0, s1 = 0, q0 = 0, q1 = 0;
        if (b < a.B) {
            s0 = __ldcg(a.seq_off + b);
            s1 = __ldcg(a.seq_off + b + 1);
            q0 = __ldcg(a.q_off + b);
            q1 = __ldcg(a.q_off + b + 1);
        }
        const int64_t n = s1 - s0, f = q1 - q0;
        int64_t cost = a.Hkv * items_cost(a, n > f ? n - f : 0, seq_items(a, f));
        if (a.B > 1) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, cost, o);
                if (lane >= o)
                    cost += y;
            }
        }
        if (b < a.B) {
            tab.seq_off[b] = s0;
            tab.q_off[b] = q0;
            tab.seq_off[b + 1] = s1;
            tab.q_off[b + 1] = q1;
            tab.start[b + 1] = run + cost;
        }
        run += __shfl_sync(0xffffffffu, cost, 31);
    }
    if (lane == 0)
        tab.start[0] = 0;
    __syncwarp();
    w.parts.cut(a, tab.start[a.B]);
    if (lane < 2)
        place[lane] = dense_locate(a, tab, w.parts.at((int)blockIdx.x + lane));
    __syncwarp();
    w.at = place[0];
    w.end = place[1];
    __syncwarp();
}

// The pool's page with token i of sequence b; -1 for an entry outside the pool,
// and behind the table's row (device lengths may pass what the host's said).
__device__ __forceinline__ int32_t dense_page(const DenseArgs &a, int b, int64_t i)
{
    const int64_t j = i >> a.page_shift;
    const int32_t pg = j < a.pt_stride ? __ldcg(a.page_table + (int64_t)b * a.pt_stride + j) : -1;
    return pg < a.pool_pages ? pg : -1;
}

// The K / V row of token i of a sequence that begins at row off (packed); -1
// where the cache has none.
__device__ __forceinline__ int64_t dense_row(const DenseArgs &a, int b, int64_t off, int64_t i)
{
    if (a.page_table == nullptr)
        return off + i < a.kv_rows ? off + i : -1;
    const int32_t pg = dense_page(a, b, i);
    return pg < 0 ? -1 : ((int64_t)pg << a.page_shift) + (i & (((int64_t)1 << a.page_shift) - 1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&x);
}

// The two bf16 of w with infinities and NaN replaced by zero.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w)
{
    if ((w & 0x7f80u) == 0x7f80u)
        w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u)
        w &= 0x0000ffffu;
    return w;
}

// First tile of an item in which some token is not seen by all its queries:
// there V may hold what no weight of zero takes away (inf, NaN), and rows
// that no token owns.
__device__ __forceinline__ int64_t dense_masked_from(int64_t first_pos)
{
    return first_pos + 1 > 0 ? (first_pos + 1) / kDenseTile : 0;
}

constexpr int kStreamRows = 128;            // packed rows of one accumulator: floor(128 / G) tokens x G heads
constexpr int kItemSlots = 4;
template <int D>
constexpr int kTileBytes = kDenseTile * D * 2;

// What the loading warp and the others of a block share: a ring of K and V
// tiles and a ring of items.
template <int NS>
struct DenseRing {
    uint64_t full[NS], empty[NS];
    uint64_t item_full[kItemSlots], item_empty[kItemSlots];
    DenseItem item[kItemSlots];

    __device__ void init(int stages, int tile_readers, int item_readers)
    {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], tile_readers);
        }
        for (int s = 0; s < kItemSlots; ++s) {
            mbar_init(&item_full[s], 1);
            mbar_init(&item_empty[s], item_readers);
        }
    }
};

template <int D>
struct QueryLoad {
    const CUtensorMap *map;
    uint8_t *sq;                             // two streams of 128 rows
    uint64_t *full, *empty;
    int32_t *bad;                            // per item slot, cleared when an item begins
};

__device__ __forceinline__ void tma_load_tile(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y,
                                              int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
// Whole rows of a page's tokens: {64 channels, 8 tokens, 2 halves, groups of 8, 1 head}.
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t group,
                                              int32_t head)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %3, %3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(group), "r"(head)
        : "memory");
}

// One lane of the warp, the same each time.  What one lane issues from code
// that the whole warp walks keeps its operands in uniform registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}

__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Whole warp: wait for a barrier's phase, bounded (a try that fails has
// suspended the warp for some 4 us: 17 s in all); false when it gave up.  The loop is one asm block: a wait on a
// phase that is there already costs one try and one branch, on which the
// tensor cores wait between products.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint32_t *ctrl, int lane)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, %3;\n\t"
        "WAIT_%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE_%=;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 q, n, 0;\n\t"
        "@q bra WAIT_%=;\n\t"
        "DONE_%=:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "n"(kSpinLimit)
        : "memory");
    if (!ok && lane == 0)
        report_timeout(ctrl, kSiteDense);
    return ok != 0;
}

// The loading warp: walks the block's items, publishes each, and streams its
// K and V tiles (K and V of a tile in turn) into the ring, and with QL its
// queries.  A packed cache's tile is a box of all 128 tokens per 64 channels;
// a paged one's a box per page, or per 128 tokens of one (a box costs its
// issue, so with 16-token pages one box for both halves of the channels
// counts).  An item with b < 0 ends the line.
template <int D, int NS, bool QL, int MAXNS>
__device__ __forceinline__ void load_items(const DenseArgs &a, DenseRing<MAXNS> &r, uint8_t *ring,
                                           const CUtensorMap *kmap, const CUtensorMap *vmap, int lane,
                                           const QueryLoad<D> &q)
{
    const int T = kStreamRows / a.G;
    const int log_pages = 7 - a.box_shift;           // boxes along a tile's 128 tokens
    const int ahead = 31 >> log_pages;               // tiles, less one, whose pages one round trip finds
    const int32_t oob = (int32_t)(a.pool_pages << a.page_shift);   // past the pool: reads zeros
    const uint32_t ring0 = smem_u32(ring), full0 = smem_u32(r.full);
    DenseWalk w;
    dense_begin(a, ring, lane, w);
    fence_proxy_async_smem();                        // the tables are read: tiles may go over them
    fence_proxy_async_global();                      // and what the kernel before wrote is loaded
    if (lane == 0)
        a.pieces[blockIdx.x] = w.piece(a);
    uint32_t n = 0;                                  // tiles loaded (K and V count one each)
    DenseItem it;
    bool ok = true;
    uint32_t k = 0;
    for (; ok; ++k) {
        const bool more = w.next(a, it);
        const int slot = k % kItemSlots;
        if (k >= kItemSlots && !warp_wait(&r.item_empty[slot], ((k / kItemSlots) - 1) & 1, a.ctrl, lane)) {
            ok = false;
            break;
        }
        if (lane == 0) {
            if (!more)
                it.b = -1;
            r.item[slot] = it;
            if (QL)
                q.bad[slot] = 0;
            mbar_arrive(&r.item_full[slot]);
        }
        if (!more)
            break;
        if (QL) {
            if (k > 0 && !warp_wait(q.empty, (k - 1) & 1, a.ctrl, lane)) {
                ok = false;
                break;
            }
            if (elect_one()) {
                const int streams = it.tokens > T ? 2 : 1;
                mbar_arrive_expect_tx(q.full, (uint32_t)(streams * T * a.G * D * 2));
                for (int s = 0; s < streams; ++s)
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tma_load_tile(smem_u32(q.sq) + (s * (D / 64) + x) * (kStreamRows * 128), q.map,
                                      smem_u32(q.full), x * 64, it.g * a.G, (int32_t)(it.q_row + s * T));
            }
            __syncwarp();
        }
        const int kt0 = uniform(it.kt0), kt1 = uniform(it.kt1), g = uniform(it.g);
        int32_t row = uniform((int32_t)(it.off + (int64_t)kt0 * kDenseTile));
        for (int kt = kt0; kt < kt1 && ok; ++kt) {
            const int done = (kt - kt0) & ahead;
            if (a.page_table != nullptr && done == 0) {
                // one round trip to the block table finds the pages of the
                // next tiles, one page a lane
                const int64_t i = ((int64_t)kt << 7) + ((int64_t)lane << a.box_shift);
                row = oob;
                if (i < it.n) {
                    const int32_t pg = dense_page(a, it.b, i);
                    if (pg >= 0)
                        row = (pg << a.page_shift) + (int32_t)(i & ((1 << a.page_shift) - 1));
                }
            }
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                // (wanted at the item's end only; written before the arrival
                // for its first V tile, it is there by then)
                if (kv == 1 && kt == kt0 && it.slot >= 0 && !QL) {
                    const int32_t c = dense_head(a, it, w.parts);
                    if (elect_one())
                        r.item[slot].head = c;
                    __syncwarp();
                }
                const int st = n % NS;
                if (n >= (uint32_t)NS && !warp_wait(&r.empty[st], ((n / NS) - 1) & 1, a.ctrl, lane)) {
                    ok = false;
                    break;
                }
                const CUtensorMap *map = kv ? vmap : kmap;
                const uint32_t dst = ring0 + st * kTileBytes<D>, bar = full0 + st * 8;
                if (elect_one())
                    mbar_arrive_expect_tx(&r.full[st], (uint32_t)kTileBytes<D>);
                __syncwarp();
                if (a.page_table == nullptr) {
                    if (elect_one()) {
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_load_tile(dst + x * (kDenseTile * 128), map, bar, x * 64, row, g);
                    }
                    __syncwarp();
                } else {
#pragma unroll 1
                    for (int p0 = 0; p0 < 1 << log_pages; p0 += 8) {
                        int32_t y[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            y[i] = __shfl_sync(0xffffffffu, row, (done << log_pages) + p0 + i);
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                if (i > 0 && p0 + i >= 1 << log_pages)
                                    break;
                                const uint32_t to = dst + (((p0 + i) * D * 2) << a.box_shift);
                                if (D == 128)
                                    tma_load_page(to, map, bar, y[i] >> 3, g);
                                else
                                    tma_load_tile(to, map, bar, 0, y[i], g);
                            }
                        }
                        __syncwarp();
                    }
                }
                ++n;
            }
            if (a.page_table == nullptr)
                row += kDenseTile;
        }
    }
    // a wait gave up: no more loads are issued; wait (bounded) for those in
    // flight, the last NS tiles and the queries, before the block may end
    if (!ok) {
        for (uint32_t j = n > (uint32_t)NS ? n - NS : 0u; j < n; ++j)
            (void)mbar_wait_bounded(&r.full[j % NS], (j / NS) & 1, kSpinLimit);
        if (QL && k > 0)
            (void)mbar_wait_bounded(q.full, (k - 1) & 1, kSpinLimit);
    }
}

// Whole warp: one row of an item that the blocks head to last share: head has
// its first piece (slot 2 c + 1), each further block the next (slot 2 q).
// With (m_p, l_p, O_p) a piece's maximum in base 2, sum and weighted sum, and
// M = max m_p:
//   O = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p
// in piece order, to row `at` (query row x head) of the output.  32 pieces a
// round trip, F pieces' rows in flight.  A piece whose factor is 0 counts too:
// a NaN or infinity that the row sees there has to stay.
template <int D, int F>
__device__ __forceinline__ void dense_join_row(const DenseArgs &a, int head, int last, int row, int64_t at, int lane)
{
    constexpr int PS = D + 4, C = D / 32;
    auto piece = [&](int q) {
        return a.part + ((int64_t)(q == head ? 2 * q + 1 : 2 * q) * a.slot_rows + row) * PS;
    };
    float M = -INFINITY, L = 0.0f, acc[C];
#pragma unroll
    for (int e = 0; e < C; ++e)
        acc[e] = 0.0f;
    for (int q0 = head; q0 <= last; q0 += 32) {
        const int count = min(32, last - q0 + 1);
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (lane < count)
            ml = __ldcg(reinterpret_cast<const float2 *>(piece(q0 + lane) + D));
        float top = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (top > M) {                               // the sums so far, relative to the new maximum
            const float f = ex2(M - top);
            M = top;
            L *= f;
#pragma unroll
            for (int e = 0; e < C; ++e)
                acc[e] *= f;
        }
        // (a maximum of -inf with a sum: every score seen was NaN)
        const float w = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : ex2(ml.x - M);
        const float l = ml.y * w;
        for (int j0 = 0; j0 < count; j0 += F) {
            float2 x[F][C / 2];
            float wj[F];
#pragma unroll
            for (int j = 0; j < F; ++j) {
                wj[j] = __shfl_sync(0xffffffffu, w, j0 + j);
                L += __shfl_sync(0xffffffffu, l, j0 + j);
#pragma unroll
                for (int e = 0; e < C / 2; ++e)
                    x[j][e] = j0 + j < count
                                  ? __ldcg(reinterpret_cast<const float2 *>(piece(q0 + j0 + j) + lane * C) + e)
                                  : make_float2(0.0f, 0.0f);
            }
#pragma unroll
            for (int j = 0; j < F; ++j)
#pragma unroll
                for (int e = 0; e < C / 2; ++e) {
                    acc[2 * e] += wj[j] * x[j][e].x;
                    acc[2 * e + 1] += wj[j] * x[j][e].y;
                }
        }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int e = 0; e < C; e += 2)
        *reinterpret_cast<uint32_t *>(a.out + at * D + lane * C + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    if (a.lse != nullptr && lane == 0)
        a.lse[at] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2f;
}

}  // namespace ts
