// Dense attention (ts_dense_attn): which kernels a call takes, over how many
// blocks, and the join of items that several blocks shared.
//   row i of sequence b (f_b rows, n_b cached tokens) sits at p = n_b - f_b + i
//   out[i, h, :] = sum_{j <= p} softmax_j(scale * q[i, h, :] . K[j, g]) * V[j, g]
//   lse[i, h]    = log sum_{j <= p} exp(scale * q[i, h, :] . K[j, g])
// Sequences with one query row go to dense_one.cu (bound by reading K and V),
// those with more to dense_tc.cu (bound by the products); a batch that holds
// both takes both.
#include "dense_common.cuh"

namespace ts {
namespace {

constexpr int kMergeWarps = 8;

// What an item costs beside its tokens, in tokens (half a tile for the last
// one's rest included).  Chosen at head_dim 128: with 200 / 400 / 650 for
// prompts, 8192 tokens of 28/4 heads take 466 / 427 / 435 us and a mixed step
// 517 / 458 / 460 (calls back to back); at head_dim 64 an item's end weighs
// less (8192 tokens of 32/8: 482 / 503 / 510 us).  For single tokens
// 96 / 192 / 400 are within 5 % of one another, except 4 requests of 1000 at
// head_dim 64, 13.7 / 10.4 / 11.3 us.
constexpr int kOneItemCost = 192, kTcItemCost = 400;

// The shared items of dense_tc: a block of this kernel for each block of that
// one and group of rows; those whose block begins no shared item return.  One
// warp a row.  (dense_one's blocks join theirs themselves, a few rows an item;
// up to 256 rows of many pieces want more warps than the last block has.)
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
dense_merge(const DenseArgs a, int blocks)
{
    pdl_wait();
    pdl_launch_dependents();
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 piece = __ldcg(reinterpret_cast<const int4 *>(a.pieces + c));
    const DensePiece p = {piece.x, piece.y, piece.z, piece.w};
    if (!(p.flags & kPieceHead))
        return;
    int last = c + 1;                                // the first block behind c that is not wholly inside the item
    for (;; last += 32) {
        const uint32_t vote = __ballot_sync(
            0xffffffffu, last + lane >= blocks - 1 || !(__ldcg(&a.pieces[last + lane].flags) & kPieceThrough));
        if (vote) {
            last += __ffs(vote) - 1;
            break;
        }
    }
    const int T = kStreamRows / a.G;
    const int64_t q0 = __ldcg(a.q_off + p.b), f = __ldcg(a.q_off + p.b + 1) - q0, q_row = q0 + (int64_t)p.t * a.TT;
    const int tokens = (int)min((int64_t)a.TT, f - (int64_t)p.t * a.TT);
    for (int i = blockIdx.y * kMergeWarps + warp; i < tokens * a.G; i += gridDim.y * kMergeWarps) {
        const int token = i / a.G, head = i - token * a.G;
        dense_join_row<D, 4>(a, c, last, token / T * kStreamRows + (token % T) * a.G + head,
                          (q_row + token) * a.Hq + p.g * a.G + head, lane);
    }
}

}  // namespace

cudaError_t launch_dense_tc(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                            const DenseArgs &a, int D, int grid, cudaStream_t st);
cudaError_t launch_dense_one(const CUtensorMap &kmap, const CUtensorMap &vmap, const DenseArgs &a, int D, int grid,
                             cudaStream_t st);

void plan_dense(const ts_kv_t *kv, const int64_t *q_off, DensePlan *dp)
{
    const Plan &p = dp->p;
    // the control block, then the counters of the shared items (in one place
    // for every shape, so that a workspace may serve several)
    size_t o = 256;
    dp->off_counts = o;
    o = align_up(o + sizeof(uint32_t) * 8 * (size_t)p.sms, 256);
    for (int one = 0; one < 2; ++one) {
        DenseLaunch &w = dp->launch[one];
        w.TT = one ? 1 : 2 * (kStreamRows / p.G);
        int64_t items = 0, tiles = 0, most = 0;
        for (int b = 0; b < p.B; ++b) {
            const int64_t f = q_off[b + 1] - q_off[b];
            if (one ? f != 1 : f < 2)
                continue;
            const int64_t n = kv->capacity > 0 ? kv->capacity : kv->seq_offsets_host[b + 1] - kv->seq_offsets_host[b];
            const int64_t t = n > 0 ? (n + kDenseTile - 1) / kDenseTile : 1;
            const int64_t i = (f + w.TT - 1) / w.TT;
            items += i;
            tiles += i * ((n > f ? (n - f) / kDenseTile : 0) + t + 1) / 2;   // of the mean item: half its queries' span
            most = t > most ? t : most;
        }
        items *= p.Hkv;
        tiles *= p.Hkv;
        // One query token: what a block reads, it reads at some 27 bytes a
        // clock, so a tile to a block where there are few.  Several: where no
        // item has more than 4 tiles none is cut, its pieces' start and their
        // join cost more than they save (prompts of 200 and 500 tokens, 28/4
        // heads: 13.1 and 17.1 us whole, 20.6 and 31.6 cut; 700 and 1000
        // tokens, 6 and 8 tiles, which are cut: 32.8 and 37.7 us, against 21.1
        // and 27.0 whole, so the border could lie higher).  Pieces have 3
        // tiles or more.
        w.split = one ? most > 1 : most > 4;
        const int64_t parts = !w.split ? items : (one ? tiles : (tiles + 2) / 3);
        w.grid = (int)(parts < p.sms ? (parts > 1 ? parts : items > 0) : p.sms);
        w.slot_rows = one ? 16 : 2 * kStreamRows;
        w.off_pieces = o;
        o = align_up(o + sizeof(DensePiece) * (size_t)w.grid, 256);
        w.off_part = o;
        if (w.split)
            o = align_up(o + sizeof(float) * 2 * (size_t)w.grid * w.slot_rows * (p.D + 4), 256);
    }
    dp->total_bytes = o;
}

ts_status_t launch_dense(const DensePlan &dp, const ts_kv_t *kv, const void *q, int64_t q_stride_tok,
                         const int64_t *q_off, void *out, float *lse, uint8_t *ws, cudaStream_t st)
{
    const Plan &p = dp.p;
    DenseArgs a;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(kv->k);
    a.v = static_cast<const __nv_bfloat16 *>(kv->v);
    a.q_st = q_stride_tok;
    a.st = kv->stride_tok;
    a.sh = kv->stride_head;
    a.seq_off = kv->seq_offsets_dev;
    a.q_off = q_off;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.ctrl = reinterpret_cast<uint32_t *>(ws);
    a.B = p.B;
    a.Hq = p.Hq;
    a.Hkv = p.Hkv;
    a.G = p.G;
    a.scale_log2 = p.scale * kLog2e;
    a.page_table = p.paged ? kv->page_table_dev : nullptr;
    a.pt_stride = kv->page_table_stride;
    a.page_shift = p.page_shift;
    a.pool_pages = kv->pool_pages;
    a.kv_rows = p.kv_rows;

    // K and V boxes: 64 channels x 128 tokens of one kv head; of a paged cache
    // the rows of a page (128 tokens of it at most), with head_dim 128 as
    // {64 channels, 8 tokens, both halves of the channels, groups of 8 tokens}.
    // Q boxes: one kv head's query heads x the tokens of a stream.  A cache
    // without a row is never read from: its maps cover query rows instead, and
    // every token is masked.
    a.box_shift = p.paged && p.page_shift < 7 ? p.page_shift : 7;
    const int box = 1 << a.box_shift;
    const bool none = p.kv_rows < 1, pages = p.paged && p.D == 128;
    a.group_stride = pages ? 2048 : 1024;
    a.half_stride = pages ? 1024 : kDenseTile * 128;
    const int64_t rows = none ? 1 : p.kv_rows, st_tok = none ? q_stride_tok : kv->stride_tok,
                  st_head = none ? p.D : kv->stride_head;
    const TmaDim by_page[4] = {{8, st_tok, 8}, {2, 64, 2}, {rows / 8, 8 * st_tok, box / 8}, {p.Hkv, st_head, 1}};
    const TmaDim by_tile[2] = {{rows, st_tok, box}, {p.Hkv, st_head, 1}};
    const TmaDim by_query[2] = {{p.Hq, p.D, p.G}, {dp.rows, q_stride_tok, kStreamRows / p.G}};
    CUtensorMap kmap, vmap, qmap;
    ts_status_t s = TS_OK;
    for (int kv_ = 0; kv_ < 2 && s == TS_OK; ++kv_) {
        const void *base = none ? q : (kv_ ? kv->v : kv->k);
        s = pages ? encode_tiles(kv_ ? &vmap : &kmap, base, 64, by_page, 4)
                  : encode_tiles(kv_ ? &vmap : &kmap, base, p.D, by_tile, 2);
    }
    if (s == TS_OK && dp.launch[0].grid > 0)
        s = encode_tiles(&qmap, q, p.D, by_query, 2);
    if (s != TS_OK)
        return s;
    for (int one = 1; one >= 0; --one) {
        const DenseLaunch &w = dp.launch[one];
        if (w.grid == 0)
            continue;
        a.TT = w.TT;
        a.single = one;
        a.split = w.split;
        a.item_cost = one ? kOneItemCost : kTcItemCost;
        a.inv_grid = 1.0 / w.grid;
        a.slot_rows = w.slot_rows;
        a.counts = reinterpret_cast<uint32_t *>(ws + dp.off_counts);
        a.pieces = reinterpret_cast<DensePiece *>(ws + w.off_pieces);
        a.part = reinterpret_cast<float *>(ws + w.off_part);
        cudaError_t e = one ? launch_dense_one(kmap, vmap, a, p.D, w.grid, st)
                            : launch_dense_tc(qmap, kmap, vmap, a, p.D, w.grid, st);
        if (e == cudaSuccess && !one && w.split && w.grid > 1) {
            const dim3 grid(w.grid - 1, 8);
            e = p.D == 128 ? launch_ex(dense_merge<128>, grid, dim3(kMergeWarps * 32), 0, st, 1, a, w.grid)
                           : launch_ex(dense_merge<64>, grid, dim3(kMergeWarps * 32), 0, st, 1, a, w.grid);
        }
        if (e != cudaSuccess) {
            set_error("dense attention launch: %s", cudaGetErrorString(e));
            return TS_ERR_CUDA;
        }
    }
    return TS_OK;
}

}  // namespace ts
