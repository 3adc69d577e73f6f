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

// An item that blocks c, c+1, ... shared: block c holds its beginning (slot
// 2c + 1), each further one the rest of its part (slot 2q), up to the first
// that is not wholly inside the item.  With (m_p, l_p, O_p) a piece's maximum
// in base 2, sum and weighted sum, M = max m_p:
//   O = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p
// in piece order.  One warp a row, grid (blocks of the main kernel - 1, row
// groups); blocks whose c ends at an item's end return.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
dense_merge(const DenseArgs a, int blocks, int slot_rows)
{
    pdl_wait();
    pdl_launch_dependents();
    constexpr int PS = D + 4, C = D / 32;
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const DensePiece p = a.pieces[c];
    if (!(p.flags & kPieceHead))
        return;
    int last = c + 1;
    for (;; last += 32) {
        const bool ends = last + lane >= blocks || !(a.pieces[last + lane].flags & kPieceThrough);
        const uint32_t vote = __ballot_sync(0xffffffffu, ends);
        if (vote) {
            last = min(last + __ffs(vote) - 1, blocks - 1);
            break;
        }
    }
    const int count = last - c + 1, T = kStreamRows / a.G;
    const int64_t f = a.q_off[p.b + 1] - a.q_off[p.b], q_row = a.q_off[p.b] + (int64_t)p.t * a.TT;
    const int tokens = (int)min((int64_t)a.TT, f - (int64_t)p.t * a.TT);
    for (int i = blockIdx.y * kMergeWarps + warp; i < tokens * a.G; i += gridDim.y * kMergeWarps) {
        const int token = i / a.G, head = i - token * a.G;
        const int row = token / T * kStreamRows + (token % T) * a.G + head;
        auto piece = [&](int u) {
            return a.part + ((int64_t)(u == 0 ? 2 * c + 1 : 2 * (c + u)) * slot_rows + row) * PS;
        };
        auto holds = [&](int u) { return u == 0 || !(a.pieces[c + u].flags & kPieceEmpty); };
        float M = -INFINITY;
        for (int u = lane; u < count; u += 32)
            if (holds(u))
                M = fmaxf(M, piece(u)[D]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float L = 0.0f, acc[C];
#pragma unroll
        for (int e = 0; e < C; ++e)
            acc[e] = 0.0f;
        for (int u0 = 0; u0 < count; u0 += 32) {
            float w = 0.0f, l = 0.0f;
            if (u0 + lane < count && holds(u0 + lane)) {
                const float2 ml = *reinterpret_cast<const float2 *>(piece(u0 + lane) + D);
                // (a maximum of -inf with a sum: every score seen was NaN)
                w = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : ex2(ml.x - M);
                l = ml.y * w;
            }
#pragma unroll 4
            for (int j = 0; j < min(32, count - u0); ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, j);
                L += __shfl_sync(0xffffffffu, l, j);
                if (wj != 0.0f) {
                    const float *src = piece(u0 + j) + lane * C;
#pragma unroll
                    for (int e = 0; e < C; e += 2) {
                        const float2 x = *reinterpret_cast<const float2 *>(src + e);
                        acc[e] += wj * x.x;
                        acc[e + 1] += wj * x.y;
                    }
                }
            }
        }
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        const int64_t at = (q_row + token) * a.Hq + p.g * a.G + head;
#pragma unroll
        for (int e = 0; e < C; e += 2)
            *reinterpret_cast<uint32_t *>(a.out + at * D + lane * C + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
        if (a.lse != nullptr && lane == 0)
            a.lse[at] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2f;
    }
}

}  // namespace

cudaError_t launch_dense_tc(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                            const DenseArgs &a, int D, int box, int grid, cudaStream_t st);
cudaError_t launch_dense_one(const CUtensorMap &kmap, const CUtensorMap &vmap, const DenseArgs &a, int D, int box,
                             int grid, cudaStream_t st);

void plan_dense(const ts_kv_t *kv, const int64_t *q_off, DensePlan *dp)
{
    const Plan &p = dp->p;
    size_t o = 256;                            // the control block
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
        // Up to 4 tiles an item is not worth cutting: its pieces' start and
        // their join cost more than they save.
        w.split = most > 4;
        const int64_t parts = w.split ? (tiles + 2) / 3 : items;
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
    a.scale = p.scale;
    a.scale_log2 = p.scale * kLog2e;
    a.page_table = p.paged ? kv->page_table_dev : nullptr;
    a.pt_stride = kv->page_table_stride;
    a.page_shift = p.page_shift;
    a.pool_pages = kv->pool_pages;

    // K and V in boxes of one kv head's 64 channels x up to 128 tokens (a
    // page, where pages are shorter); Q in boxes of one kv head's query heads
    // x the tokens of a stream.  A cache without a row is never read from:
    // its map covers a query row instead, and every token is masked.
    const int box = p.paged && (1 << p.page_shift) < kDenseTile ? 1 << p.page_shift : kDenseTile;
    const bool none = p.kv_rows < 1;
    CUtensorMap kmap, vmap, qmap;
    ts_status_t s = encode_map3(&kmap, none ? q : kv->k, p.D, none ? 1 : p.kv_rows, p.Hkv,
                                none ? q_stride_tok : kv->stride_tok, none ? p.D : kv->stride_head, box, 1);
    if (s == TS_OK)
        s = encode_map3(&vmap, none ? q : kv->v, p.D, none ? 1 : p.kv_rows, p.Hkv,
                        none ? q_stride_tok : kv->stride_tok, none ? p.D : kv->stride_head, box, 1);
    if (s == TS_OK && dp.launch[0].grid > 0)
        s = encode_map3(&qmap, q, p.D, p.Hq, dp.rows, p.D, q_stride_tok, p.G, kStreamRows / p.G);
    if (s != TS_OK)
        return s;
    for (int one = 1; one >= 0; --one) {
        const DenseLaunch &w = dp.launch[one];
        if (w.grid == 0)
            continue;
        a.TT = w.TT;
        a.single = one;
        a.split = w.split;
        a.pieces = reinterpret_cast<DensePiece *>(ws + w.off_pieces);
        a.part = reinterpret_cast<float *>(ws + w.off_part);
        cudaError_t e = one ? launch_dense_one(kmap, vmap, a, p.D, box, w.grid, st)
                            : launch_dense_tc(qmap, kmap, vmap, a, p.D, box, w.grid, st);
        if (e == cudaSuccess && w.split && w.grid > 1) {
            const dim3 grid(w.grid - 1, one ? (p.G + kMergeWarps - 1) / kMergeWarps : 8);
            e = p.D == 128 ? launch_ex(dense_merge<128>, grid, dim3(kMergeWarps * 32), 0, st, 1, a, w.grid, w.slot_rows)
                           : launch_ex(dense_merge<64>, grid, dim3(kMergeWarps * 32), 0, st, 1, a, w.grid, w.slot_rows);
        }
        if (e != cudaSuccess) {
            set_error("dense attention launch: %s", cudaGetErrorString(e));
            return TS_ERR_CUDA;
        }
    }
    return TS_OK;
}

}  // namespace ts
