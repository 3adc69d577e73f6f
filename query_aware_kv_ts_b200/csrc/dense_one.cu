// Dense attention of one query token (decode): sequences with a single query
// row, its G <= 16 heads of a kv head against all of the sequence's tokens.
// Bound by reading K and V once, so what counts is bytes in flight: one
// persistent block per SM, a loading warp that keeps a ring of 32 KB tiles
// filled by TMA (K and V in turn), and eight warps that take 16 tokens of
// every tile each.  Measured: one token over 1,048,576 of 4 x 128, 2.1 GB,
// 324-335 us (98-101 % of the copy rate); 32 requests of 8192 to 65536 tokens
// of 8 x 128 on 16-token pages, 3.0 GB, 489-502 us on several cards (90-92 %).
// With calls back to back on few inputs, part of them in L2: 445 us, and 431
// packed, 433 with 32-token pages, 625 with 8-token ones, whose boxes of 2 KB
// cost their issue; the same batch with head_dim 64: 346 packed, 337, 397 and
// 584 with 32-, 16- and 8-token pages (boxes of 4, 2 and 1 KB).  A block alone
// reads about 27 bytes a clock (clock64 in a copy with counters), so a small
// batch goes to as many as it has tiles (4 requests of about 1000 tokens:
// 12.5 us, 3 us of them the kernel's start to its first load).  A warp keeps its own running maximum, sum and weighted
// sums, and the eight are joined at the end of the item, so nothing in the
// loop waits for another warp.
//
// The products run on mma.sync (m16n8k16): the 16 rows are the heads, and a
// tensor-core tile of 128 rows would hold at most 16 of them.  A weight goes
// into the second product as a bf16 and a bf16 remainder (about 16 bits):
// up to 8 heads the remainders are the rows 8-15, which costs nothing; above
// that a second product.
#include "dense_common.cuh"

namespace ts {
namespace {

constexpr int kOneWarps = 8;
constexpr int kOneThreads = (kOneWarps + 1) * 32;
constexpr float kRaise = 8.0f;           // log2 of how far weights may grow before the sums are rescaled
constexpr int kOneMaxStages = 10;
constexpr int kCountTiles = 20;          // bits of the joins' counters that count tiles (4M tokens: 32768)

template <int D, bool WIDE>
constexpr int kJoinBytes = kOneWarps * (WIDE ? 16 : 8) * (D + 4) * 4;
template <int D, bool WIDE>
constexpr int kOneStages = (WIDE ? 128 : 160) * 1024 / kTileBytes<D>;

struct OneShared {
    DenseRing<kOneMaxStages> ring;
    uint64_t joined, join_free;
};

// WIDE: more than 8 heads.
template <int D, bool WIDE>
__device__ __forceinline__ void attend_items(const DenseArgs &a, OneShared &sh, uint32_t ring, float *join, int warp,
                                             int lane)
{
    constexpr int NS = kOneStages<D, WIDE>;
    constexpr int ROWS = WIDE ? 16 : 8;
    constexpr int PS = D + 4;
    const int r0 = lane >> 2, c0 = (lane & 3) * 2;
    const float c = fabsf(a.scale_log2), sign = a.scale_log2 < 0.0f ? -1.0f : 1.0f;
    // this lane's rows of the ldmatrix loads: K rows are tokens (keys by
    // channels), V's are transposed on the way
    const int k_tok = warp * 16 + (lane & 7) + (lane >> 4) * 8, k_chunk = (lane >> 3) & 1;
    const int v_tok = warp * 16 + (lane & 15), v_chunk = lane >> 4;
    const int k_row = (k_tok >> 3) * a.group_stride + (k_tok & 7) * 128;
    const int v_row = (v_tok >> 3) * a.group_stride + (v_tok & 7) * 128;
    uint32_t n = 0;
    for (uint32_t k = 0;; ++k) {
        const int slot = k % kItemSlots;
        if (!warp_wait(&sh.ring.item_full[slot], (k / kItemSlots) & 1, a.ctrl, lane))
            return;
        const int b = sh.ring.item[slot].b;
        if (b < 0)
            return;
        const int g = sh.ring.item[slot].g, kt0 = sh.ring.item[slot].kt0, kt1 = sh.ring.item[slot].kt1;
        const int part_slot = sh.ring.item[slot].slot;
        const int tiles = sh.ring.item[slot].tiles;
        const int64_t q_row = sh.ring.item[slot].q_row, len = sh.ring.item[slot].n;
        uint32_t qa[D / 16][4];
        const __nv_bfloat16 *q = a.q + q_row * a.q_st + (int64_t)g * a.G * D;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = r0 + (e & 1) * 8;
                qa[ks][e] = 0u;
                if ((WIDE || !(e & 1)) && row < a.G)
                    qa[ks][e] = __ldcg(reinterpret_cast<const uint32_t *>(q + (int64_t)row * D + ks * 16 + c0 +
                                                                          (e >> 1) * 8));
            }
        // weighted sums: rows r0 and r0 + 8 (up to 8 heads, the remainders')
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[i][e] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        for (int kt = kt0; kt < kt1; ++kt, n += 2) {
            const int left = (int)min(len - (int64_t)kt * kDenseTile - warp * 16, (int64_t)16);   // tokens of the slab
            // ---- S = Q K^T for this warp's 16 tokens ----
            const int sk = n % NS, sv = (n + 1) % NS;
            if (!warp_wait(&sh.ring.full[sk], (n / NS) & 1, a.ctrl, lane))
                return;
            float s[2][4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[0][e] = s[1][e] = 0.0f;
            const uint32_t kb = ring + sk * kTileBytes<D> + k_row;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t b0, b1, b2, b3;
                ldmatrix_x4(b0, b1, b2, b3,
                            kb + (ks >> 2) * a.half_stride + (((((ks & 3) * 2 + k_chunk) ^ (k_tok & 7))) << 4));
                mma_16816(s[0], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b0, b1);
                mma_16816(s[1], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b2, b3);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.ring.empty[sk]);
            if (left < 16 || sign < 0.0f) {
#pragma unroll
                for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[nb][e] = nb * 8 + c0 + (e & 1) < left ? s[nb][e] * sign : -INFINITY;
            }
            // ---- running maximum (raised only when far exceeded), weights, sum ----
            float top[2];
            top[0] = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
            top[1] = WIDE ? fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3])) : -INFINITY;
            bool raise = (top[0] - m[0]) * c > kRaise;
            if (WIDE)
                raise |= (top[1] - m[1]) * c > kRaise;
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int e = 0; e < (WIDE ? 2 : 1); ++e) {
                    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
                    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
                    top[e] = fmaxf(top[e], m[e]);
                    const float f = top[e] == -INFINITY ? 1.0f : ex2((m[e] - top[e]) * c);
                    m[e] = top[e];
                    l[e] *= f;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        o[i][2 * e] *= f;
                        o[i][2 * e + 1] *= f;
                        if (!WIDE) {
                            o[i][2] *= f;
                            o[i][3] *= f;
                        }
                    }
                }
            }
            uint32_t hi[2][2], lo[2][2];             // [8 tokens][row]
#pragma unroll
            for (int e = 0; e < (WIDE ? 2 : 1); ++e) {
                const float mc = m[e] == -INFINITY ? 0.0f : m[e] * c;
#pragma unroll
                for (int nb = 0; nb < 2; ++nb) {
                    const float p0 = ex2(fmaf(s[nb][2 * e], c, -mc)), p1 = ex2(fmaf(s[nb][2 * e + 1], c, -mc));
                    l[e] += p0 + p1;
                    if (WIDE) {
                        // both parts go into one sum: cut off, not rounded,
                        // the remainder has the weight's sign, and at least
                        // the smallest normal number keeps 0 times an
                        // infinity of V out of it
                        hi[nb][e] = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
                        lo[nb][e] = pack_bf16(fmaxf(p0 - bf16_lo(hi[nb][e]), fminf(p0, 1.1754944e-38f)),
                                              fmaxf(p1 - bf16_hi(hi[nb][e]), fminf(p1, 1.1754944e-38f)));
                    } else {
                        hi[nb][e] = pack_bf16(p0, p1);
                        lo[nb][e] = pack_bf16(p0 - bf16_lo(hi[nb][e]), p1 - bf16_hi(hi[nb][e]));
                    }
                }
            }
            // ---- O += P V ----
            if (!warp_wait(&sh.ring.full[sv], ((n + 1) / NS) & 1, a.ctrl, lane))
                return;
            const uint32_t vb = ring + sv * kTileBytes<D> + v_row;
            // rows behind the sequence's end hold anything: no weight of zero
            // takes a NaN away, so they go in as zeros
            uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
            if (left < 16) {
                keep0 = (c0 < left ? 0xffffu : 0u) | (c0 + 1 < left ? 0xffff0000u : 0u);
                keep1 = (c0 + 8 < left ? 0xffffu : 0u) | (c0 + 9 < left ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int i = 0; i < D / 8; i += 2) {
                uint32_t b0, b1, b2, b3;
                ldmatrix_x4_trans(b0, b1, b2, b3,
                                  vb + (i >> 3) * a.half_stride + ((((i & 7) + v_chunk) ^ (v_tok & 7)) << 4));
                b0 &= keep0;
                b1 &= keep1;
                b2 &= keep0;
                b3 &= keep1;
                if (WIDE) {
                    mma_16816(o[i], hi[0][0], hi[0][1], hi[1][0], hi[1][1], b0, b1);
                    mma_16816(o[i], lo[0][0], lo[0][1], lo[1][0], lo[1][1], b0, b1);
                    mma_16816(o[i + 1], hi[0][0], hi[0][1], hi[1][0], hi[1][1], b2, b3);
                    mma_16816(o[i + 1], lo[0][0], lo[0][1], lo[1][0], lo[1][1], b2, b3);
                } else {
                    mma_16816(o[i], hi[0][0], lo[0][0], hi[1][0], lo[1][0], b0, b1);
                    mma_16816(o[i + 1], hi[0][0], lo[0][0], hi[1][0], lo[1][0], b2, b3);
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.ring.empty[sv]);
        }
        const int head = sh.ring.item[slot].head;
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.ring.item_empty[slot]);
        // ---- the eight warps' sums joined, in a fixed order ----
        if (k > 0 && !warp_wait(&sh.join_free, (k - 1) & 1, a.ctrl, lane))
            return;
#pragma unroll
        for (int e = 0; e < (WIDE ? 2 : 1); ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            float *row = join + (warp * ROWS + r0 + e * 8) * PS;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                // a remainder (of either sign, or 0) times an infinity of V
                // is no correction: an infinite sum stays what it is
                float x[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float y = o[i][2 * e + u];
                    x[u] = WIDE || isinf(y) ? y : y + o[i][2 + u];
                }
                *reinterpret_cast<float2 *>(row + i * 8 + c0) = make_float2(x[0], x[1]);
            }
            if ((lane & 3) == 0)
                *reinterpret_cast<float2 *>(row + D) = make_float2(m[e] * c, l[e]);
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.joined);
        if (!warp_wait(&sh.joined, k & 1, a.ctrl, lane))
            return;
        for (int row = warp; row < a.G; row += kOneWarps) {
            float mw[kOneWarps], M = -INFINITY, L = 0.0f;
            float acc[D / 32];
#pragma unroll
            for (int w = 0; w < kOneWarps; ++w) {
                mw[w] = join[(w * ROWS + row) * PS + D];
                M = fmaxf(M, mw[w]);
            }
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                acc[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < kOneWarps; ++w) {
                const float *src = join + (w * ROWS + row) * PS;
                // (a maximum of -inf with a sum: every score seen was NaN)
                const float f = mw[w] == -INFINITY ? (src[D + 1] == 0.0f ? 0.0f : 1.0f) : ex2(mw[w] - M);
                // (also where f is 0: times a NaN or infinity of what the row
                // sees it is NaN, which has to stay)
                L += f * src[D + 1];
#pragma unroll
                for (int i = 0; i < D / 32; i += 2) {
                    const float2 x = *reinterpret_cast<const float2 *>(src + lane * (D / 32) + i);
                    acc[i] += f * x.x;
                    acc[i + 1] += f * x.y;
                }
            }
            if (part_slot < 0) {
                const float inv = L == 0.0f ? 0.0f : 1.0f / L;
                const int64_t at = q_row * a.Hq + g * a.G + row;
#pragma unroll
                for (int i = 0; i < D / 32; i += 2)
                    *reinterpret_cast<uint32_t *>(a.out + at * D + lane * (D / 32) + i) =
                        pack_bf16(acc[i] * inv, acc[i + 1] * inv);
                if (a.lse != nullptr && lane == 0)
                    a.lse[at] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2f;
            } else {
                float *dst = a.part + ((int64_t)part_slot * a.slot_rows + row) * PS;
#pragma unroll
                for (int i = 0; i < D / 32; i += 2)
                    *reinterpret_cast<float2 *>(dst + lane * (D / 32) + i) = make_float2(acc[i], acc[i + 1]);
                if (lane == 0)
                    *reinterpret_cast<float2 *>(dst + D) = make_float2(M, L);
            }
        }
        // A shared item's rows are joined by whichever block's warp comes last
        // (the sum is taken in piece order, whoever that is): each adds its
        // tiles to the rows' counter and goes on, the block that ends the item
        // also its own number, so that the last one knows the blocks between.
        if (part_slot >= 0 && warp < a.G) {
            uint32_t *count = a.counts + head * 8 + warp;
            const uint32_t mine = (uint32_t)(kt1 - kt0) + (kt1 == tiles ? (blockIdx.x + 1u) << kCountTiles : 0u);
            __threadfence();
            __syncwarp();
            uint32_t sum = 0;
            if (lane == 0)
                sum = atomicAdd(count, mine) + mine;
            sum = __shfl_sync(0xffffffffu, sum, 0);
            if ((sum & ((1u << kCountTiles) - 1u)) == (uint32_t)tiles) {
                __threadfence();
#pragma unroll 1
                for (int row = warp; row < a.G; row += kOneWarps)
                    dense_join_row<D, 8>(a, head, (int)(sum >> kCountTiles) - 1, row, q_row * a.Hq + g * a.G + row, lane);
                if (lane == 0)
                    *count = 0u;                     // as the next call finds it
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.join_free);
    }
}

template <int D, bool WIDE>
__global__ void __launch_bounds__(kOneThreads, 1)
dense_one(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
          const __grid_constant__ DenseArgs a)
{
    extern __shared__ uint8_t dyn_smem[];
    __shared__ OneShared sh;
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
    float *join = reinterpret_cast<float *>(ring + kOneStages<D, WIDE> * kTileBytes<D>);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        sh.ring.init(kOneStages<D, WIDE>, kOneWarps, kOneWarps);
        mbar_init(&sh.joined, kOneWarps);
        mbar_init(&sh.join_free, kOneWarps);
        mbar_fence_init();
    }
    if (warp == kOneWarps && lane < 2)
        tma_prefetch_desc(lane ? &vmap : &kmap);
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    if (warp == kOneWarps) {
        const QueryLoad<D> none = {};
        load_items<D, kOneStages<D, WIDE>, false>(a, sh.ring, ring, &kmap, &vmap, lane, none);
    } else {
        attend_items<D, WIDE>(a, sh, smem_u32(ring), join, warp, lane);
    }
}

template <int D, bool WIDE>
cudaError_t launch_one(const CUtensorMap &kmap, const CUtensorMap &vmap, const DenseArgs &a, int grid, cudaStream_t st)
{
    const size_t smem = 1024 + (size_t)kOneStages<D, WIDE> * kTileBytes<D> + kJoinBytes<D, WIDE>;
    const cudaError_t e = ensure_dyn_smem((const void *)dense_one<D, WIDE>, (int)smem);
    if (e != cudaSuccess)
        return e;
    return launch_ex(dense_one<D, WIDE>, dim3(grid), dim3(kOneThreads), smem, st, 1, kmap, vmap, a);
}

}  // namespace

cudaError_t launch_dense_one(const CUtensorMap &kmap, const CUtensorMap &vmap, const DenseArgs &a, int D, int grid,
                             cudaStream_t st)
{
    if (D == 128)
        return a.G > 8 ? launch_one<128, true>(kmap, vmap, a, grid, st)
                       : launch_one<128, false>(kmap, vmap, a, grid, st);
    return a.G > 8 ? launch_one<64, true>(kmap, vmap, a, grid, st)
                   : launch_one<64, false>(kmap, vmap, a, grid, st);
}

}  // namespace ts
