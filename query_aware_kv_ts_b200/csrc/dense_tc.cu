// Dense attention on the 5th-generation tensor cores: sequences with two or
// more query tokens (whole prompts, chunks).  For an item (see
// dense_common.cuh) of query tokens x the G heads of a kv head:
//   S = Q K^T            [128 x 128] per tile of 128 tokens, fp32 in TMEM
//   m, l                 running maximum and sum of each row
//   P = 2^((S - m) c)    rounded to bf16, written over S in TMEM (c = scale log2 e)
//   O += P V             [128 x d], fp32 in TMEM
//
// One persistent block per SM.  Two streams of 128 packed rows each (T =
// floor(128 / G) tokens x G heads, token-major: one row of the accumulator is
// one thread) share every K and V tile.  Warps 0-3 and 4-7 are the streams'
// softmax, one thread a row, so that no reduction crosses threads; warp 8
// walks the items and loads Q, K and V with TMA (128-byte swizzle) into a
// ring of tiles; warp 9 issues the MMAs; warp 10 clears what a masked token
// must not leak out of V.  While one stream's softmax runs, the tensor cores
// do the other's products.
//
// Measured, head_dim 128: a prompt of 8192 tokens, 28/4 heads, 488-493 us (976
// TFLOP/s of the causal half); 2048 new tokens over 129,025 on 16-token pages,
// 3.95-4.06 ms (926-951).  A tile takes both streams 3300 cycles (clock64 in a
// copy with counters), of which the products are 2048.  What bounds it is the
// chain inside a stream: the next S is issued behind P V and both behind P, so
// a tile costs a stream its softmax (1750 cycles, two streams sharing the
// exponential unit's 2048), the two products (512 each) and the hand-over;
// runs longer than some 100 us are at the board's power limit (1.4-1.5 GHz of
// 1.965).  Tried and
// slower: half rows on four softmax groups with a barrier for their common
// reference (857 against 906 TFLOP/s then), P handed over in halves to a
// polling issuer (770 against 920), every other tile of a narrow item on the
// idle stream (a block's loads, 27 bytes a clock, do not feed it).
#include "dense_common.cuh"

namespace ts {
namespace {

constexpr int kSoftmaxWarps = 8;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kGuardWarp = 10;   // and an idle one
constexpr int kTcThreads = 12 * 32;
// Registers: 384 threads x 168 at launch; the loading, issuing and guarding
// warps' group gives some to the two softmax groups
// (128 x 96 + 256 x 200 <= 384 x 168).
constexpr int kAuxRegs = 96, kSoftmaxRegs = 200;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;            // S (and P over it) at 0 and 128, O at 256 and 256 + d
constexpr float kRaise = 4096.0f;           // sum of a tile's weights above which the reference is raised

constexpr int kTcMaxStages = 8;

struct TcShared {
    DenseRing<kTcMaxStages> ring;
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_ready[2], o_full[2];
    uint64_t clean[kTcMaxStages];                       // the masked V tile in this stage has been cleared
    uint64_t done;
    int32_t bad[kItemSlots];                 // the item's masked tiles held infinities or NaN in V
    uint32_t tmem;
};

// D[tmem] (+)= A[tmem] * B[smem], B stored with its N index contiguous.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// Shared-memory descriptor of an operand whose M / N index is contiguous:
// 64-channel blocks of 128-byte rows (one row a token), 128-byte swizzle.
// 8 tokens are group bytes apart (stride), 64-channel blocks half bytes
// (leading dimension).
__device__ __forceinline__ uint64_t umma_desc_sw128_mn(uint32_t smem_addr, uint32_t group, uint32_t half)
{
    return (uint64_t)((smem_addr >> 4) & 0x3fffu) | ((uint64_t)(half >> 4) << 16) | ((uint64_t)(group >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// The same for K, whose channels are the sum's index: 64 channels a row, 8
// tokens group bytes apart.
__device__ __forceinline__ uint64_t umma_desc_sw128_k(uint32_t smem_addr, uint32_t group)
{
    return (uint64_t)((smem_addr >> 4) & 0x3fffu) | ((uint64_t)1 << 16) | ((uint64_t)(group >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]),
        "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
        "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(
            v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations of one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 32 weights 2^(s c - mc): their sum added to sum, as bf16 in p.  The tensor
// cores take P in V's type; a second product with the remainders would be 512
// cycles more a stream and tile.  Rounding is off by 2^-8 of a weight at most,
// in either direction, as the output's own rounding is: the error against 64
// bits is 2.0-2.3e-3 of the norm where that alone leaves 1.6e-3.  The sum takes
// the weights before rounding, so it has no part in it.  (A share of
// them by a polynomial on the FMA units, beside the exponential unit, was
// 2-5 % slower in long runs: those run at the power limit, where what counts
// is the number of operations.)
__device__ __forceinline__ void weights32(const float *s, uint64_t c2, uint64_t mc2, uint64_t *sum, uint32_t *p)
{
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float y0, y1;
        unpair(fma2(pair(s[2 * e], s[2 * e + 1]), c2, mc2), y0, y1);
        y0 = ex2(y0);
        y1 = ex2(y1);
        sum[e & 1] = add2(sum[e & 1], pair(y0, y1));
        p[e] = pack_bf16(y0, y1);
    }
}

// 4 x 4 pieces of 16 bytes across 4 lanes: lane i's piece j becomes lane j's
// piece i.
__device__ __forceinline__ void transpose4(uint4 (&w)[4], int lane)
{
    auto swap = [&](uint4 &x, uint4 &y, int bit) {      // lanes with the bit give x and get y, the others the reverse
        const bool up = lane & bit;
        uint4 g = up ? x : y;
        g.x = __shfl_xor_sync(0xffffffffu, g.x, bit);
        g.y = __shfl_xor_sync(0xffffffffu, g.y, bit);
        g.z = __shfl_xor_sync(0xffffffffu, g.z, bit);
        g.w = __shfl_xor_sync(0xffffffffu, g.w, bit);
        if (up)
            x = g;
        else
            y = g;
    };
    swap(w[0], w[1], 1);
    swap(w[2], w[3], 1);
    swap(w[0], w[2], 2);
    swap(w[1], w[3], 2);
}

// Where the rows of a lane's quad go, apart from the item: token and head of
// each in the stream, and its row of the output behind the stream's first.
struct QuadRows {
    int32_t token[4], row[4];
};

// The item's end for this thread's row: O / l to the output, or O, m and l to
// the partial results.  mb: the row's reference in base 2.  Four lanes
// exchange 16-byte pieces first, so that a store covers 8 rows of 64 bytes
// and not 32 of 16.
template <int D>
__device__ __forceinline__ void finish_row(const DenseArgs &a, const DenseItem &it, bool bad, int stream, int r,
                                           int lane, const QuadRows &rows, uint32_t to, float mb, float l)
{
    const int T = kStreamRows / a.G, me = lane & 3;
    const int tokens = min(T, it.tokens - stream * T), slot = it.slot;
    const bool whole = slot < 0;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t row0 = (it.q_row + stream * T) * a.Hq + it.g * a.G;
    const int my_token = me < 2 ? (me ? rows.token[1] : rows.token[0]) : (me == 2 ? rows.token[2] : rows.token[3]);
    const int my_row = me < 2 ? (me ? rows.row[1] : rows.row[0]) : (me == 2 ? rows.row[2] : rows.row[3]);
    __nv_bfloat16 *out = a.out + row0 * D + me * 8;
    float *part = a.part + ((int64_t)slot * a.slot_rows + stream * kStreamRows + (r & ~3)) * (D + 4) + me * 4;
#pragma unroll 1
    for (int x = 0; x < D; x += 32) {
        uint32_t o[32];
        tmem_ld32(to + x, o);
        tmem_wait_ld();
        if (bad && my_token < tokens) {
            // infinities and NaN of the masked tiles that this row sees
            const int64_t pos = it.first_pos + stream * T + my_token;
            const int64_t t0 = max(it.first_pos + 1, (int64_t)it.kt0 * kDenseTile);
            const int64_t t1 = min(pos + 1, (int64_t)it.kt1 * kDenseTile);
            const unsigned short *values = reinterpret_cast<const unsigned short *>(a.v);
            for (int64_t t = t0; t < t1; ++t) {
                const int64_t vr = dense_row(a, it.b, it.off, t);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float y = vr < 0 ? 0.0f : bf16_lo(__ldcg(values + vr * a.st + it.g * a.sh + x + e));
                    if (!isfinite(y))
                        o[e] = __float_as_uint(__uint_as_float(o[e]) + y);
                }
            }
        }
        __syncwarp();
        uint4 w[4];
        if (whole) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t *y = o + 8 * j;
                w[j].x = pack_bf16(__uint_as_float(y[0]) * inv, __uint_as_float(y[1]) * inv);
                w[j].y = pack_bf16(__uint_as_float(y[2]) * inv, __uint_as_float(y[3]) * inv);
                w[j].z = pack_bf16(__uint_as_float(y[4]) * inv, __uint_as_float(y[5]) * inv);
                w[j].w = pack_bf16(__uint_as_float(y[6]) * inv, __uint_as_float(y[7]) * inv);
            }
            transpose4(w, lane);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (rows.token[u] < tokens)
                    *reinterpret_cast<uint4 *>(out + rows.row[u] * D + x) = w[u];
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = make_uint4(o[16 * h + 4 * j], o[16 * h + 4 * j + 1], o[16 * h + 4 * j + 2],
                                      o[16 * h + 4 * j + 3]);
                transpose4(w, lane);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (rows.token[u] < tokens)
                        *reinterpret_cast<uint4 *>(part + u * (D + 4) + x + h * 16) = w[u];
            }
        }
    }
    if (my_token < tokens) {
        if (!whole)
            *reinterpret_cast<float2 *>(part + me * D + D) = make_float2(mb, l);   // of row `me` of the quad
        else if (a.lse != nullptr)
            a.lse[row0 + my_row] = l == 0.0f ? -INFINITY : (mb + log2f(l)) * kLn2f;
    }
}

__device__ __forceinline__ void load_scores(uint32_t ts, bool negative, float (&s)[32])
{
    uint32_t *y = reinterpret_cast<uint32_t *>(s);
    tmem_ld32(ts, y);
    tmem_wait_ld();
    // (nothing that uses them moves above the wait)
#pragma unroll
    for (int e = 0; e < 32; e += 8)
        asm volatile("" : "+r"(y[e]), "+r"(y[e + 1]), "+r"(y[e + 2]), "+r"(y[e + 3]), "+r"(y[e + 4]), "+r"(y[e + 5]),
                          "+r"(y[e + 6]), "+r"(y[e + 7]));
    if (negative) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
            s[e] = -s[e];
    }
}

// One tile's weights 2^((S - m) c) of this thread's row: as bf16 in p, and
// their sum.  limit: the tokens that the row sees.
template <bool MASKED>
__device__ __forceinline__ float tile_weights(uint32_t ts, float m, float c, bool negative, int limit, uint32_t *p)
{
    const float mc = m == -INFINITY ? 0.0f : m * c;
    const uint64_t c2 = pair(c, c), mc2 = pair(-mc, -mc);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int x = 0; x < kDenseTile / 32; ++x) {
        float s[32];
        load_scores(ts + x * 32, negative, s);
        // (the 32 rows of a warp have few tokens: most of a masked tile's
        // scores are seen by all or none)
        if (MASKED && !__all_sync(0xffffffffu, limit >= (x + 1) * 32)) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
                s[e] = x * 32 + e < limit ? s[e] : -INFINITY;
        }
        weights32(s, c2, mc2, sum, p + x * 16);
    }
    float y0, y1;
    unpair(add2(sum[0], sum[1]), y0, y1);
    return y0 + y1;
}

// The largest score that the row sees among the tile's first `chunks` x 32.
__device__ __forceinline__ float tile_top(uint32_t ts, bool negative, int limit, int chunks)
{
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
    for (int x = 0; x < chunks; ++x, limit -= 32) {
        float s[32];
        load_scores(ts + x * 32, negative, s);
        if (limit >= 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
                top[e & 1] = fmaxf(top[e & 1], s[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e)
                top[e & 1] = fmaxf(top[e & 1], e < limit ? s[e] : -INFINITY);
        }
        __syncwarp();
    }
    return fmaxf(top[0], top[1]);
}

// O of this thread's row times f.  Stores to TMEM are asynchronous: a tile that
// is done again may come here a second time, so they are waited for.
template <int D>
__device__ __forceinline__ void rescale_row(uint32_t to, float f)
{
#pragma unroll 1
    for (int x = 0; x < D; x += 16) {
        uint32_t o[16];
        tmem_ld_32x32b<16>(to + x, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tmem_st16(to + x, o);
    }
    tmem_wait_st();
}

// ---- the softmax of one stream: 128 threads, one row each -------------------
// A row's reference m is the largest of the first scores that it sees.  A tile's
// weights are taken with m as it stands: they may grow above 1, and their sum
// tells when they do.  Only when a row's sum passes kRaise is its maximum
// found, m raised, O rescaled and the tile done again: fp32 and bf16 keep
// their relative precision at any m, and the result is divided by a sum with
// the same reference.  (The maximum of every tile, first, would be 300 cycles
// more between S and P, which the tensor cores wait for.)
template <int D>
__device__ __forceinline__ void softmax_stream(const DenseArgs &a, TcShared &sh, int stream, int quarter, int lane)
{
    const int r = quarter * 32 + lane;               // the row in the stream
    const uint32_t lanes = sh.tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t ts = lanes + stream * 128, to = lanes + kTmemO + stream * D;
    const bool negative = a.scale_log2 < 0.0f;
    const float c = fabsf(a.scale_log2);
    QuadRows rows;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        rows.token[u] = ((r & ~3) + u) / a.G;
        rows.row[u] = rows.token[u] * a.Hq + ((r & ~3) + u) - rows.token[u] * a.G;
    }
    const int my_token = r / a.G;
    uint32_t phase = 0, done = 0;                    // of s_full and o_full
    for (uint32_t k = 0;; ++k) {
        const int slot = k % kItemSlots;
        if (!warp_wait(&sh.ring.item_full[slot], (k / kItemSlots) & 1, a.ctrl, lane))
            return;
        if (sh.ring.item[slot].b < 0)
            return;
        const int first = stream * (kStreamRows / a.G);   // of the stream's tokens in the item
        if (first >= sh.ring.item[slot].tokens) {    // the item fills the first stream only
            if (lane == 0)
                mbar_arrive(&sh.ring.item_empty[slot]);
            continue;
        }
        const int kt0 = sh.ring.item[slot].kt0, kt1 = sh.ring.item[slot].kt1;
        const int masked_from = (int)dense_masked_from(sh.ring.item[slot].first_pos);
        // tokens that the row sees from tile kt0 on
        int64_t left = sh.ring.item[slot].first_pos + first + my_token + 1 - (int64_t)kt0 * kDenseTile;
        float m = -INFINITY, l = 0.0f;               // m in units of S
        for (int kt = kt0; kt < kt1; ++kt, left -= kDenseTile) {
            if (!warp_wait(&sh.s_full[stream], phase & 1, a.ctrl, lane))
                return;
            ++phase;
            tmem_fence_after();
            const int limit = left < 0 ? 0 : (left < kDenseTile ? (int)left : kDenseTile);
            bool raise = m == -INFINITY;             // no reference yet
            uint32_t p[kDenseTile / 2];
            float sum = 0.0f;
#pragma unroll 1
            for (int again = 0; again < 2; ++again) {
                if (__any_sync(0xffffffffu, raise)) {
                    // (to begin with, 32 scores that the row sees are enough,
                    // unless they are all -inf)
                    float top;
#pragma unroll 1
                    for (int chunks = kt == kt0 && !again ? 1 : 4;; chunks = 4) {
                        top = tile_top(ts, negative, limit, chunks);
                        if (chunks == 4 || !__any_sync(0xffffffffu, raise && limit > 32 && top == -INFINITY))
                            break;
                    }
                    float f = 1.0f;
                    if (raise && top > m) {
                        f = ex2((m - top) * c);
                        m = top;
                    }
                    l *= f;
                    if (kt > kt0)
                        rescale_row<D>(to, f);
                }
                sum = kt >= masked_from ? tile_weights<true>(ts, m, c, negative, limit, p)
                                        : tile_weights<false>(ts, m, c, negative, limit, p);
                raise = sum > kRaise;
                if (!__any_sync(0xffffffffu, raise))
                    break;
            }
            l += sum;
            tmem_st32(ts, p);
            tmem_st32(ts + 32, p + 32);
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.p_ready[stream]);
        }
        if (!warp_wait(&sh.o_full[stream], done & 1, a.ctrl, lane))
            return;
        ++done;
        tmem_fence_after();
        finish_row<D>(a, sh.ring.item[slot], sh.bad[slot] != 0, stream, r, lane, rows, to, m * c, l);
        tmem_fence_before();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.ring.item_empty[slot]);
    }
}

// ---- the products -----------------------------------------------------------
// One lane issues them, but the whole warp walks: what addresses and counts
// depend on is the same in every lane and stays in uniform registers, where
// the instruction wants it (a walk of one lane spent 100 cycles an MMA on
// bringing its operands there, more than the 64 that the product takes).
template <int D, int NS>
__device__ __forceinline__ void issue_products(const DenseArgs &a, TcShared &sh, uint32_t sq, uint32_t ring, int lane)
{
    constexpr uint32_t idesc_s = umma_idesc_bf16_f32(128, kDenseTile);
    constexpr uint32_t idesc_o = umma_idesc_bf16_f32(128, D) | (1u << 16);   // B's N index is contiguous
    const int T = kStreamRows / a.G;
    const uint32_t tmem = (uint32_t)uniform((int)sh.tmem);
    const uint32_t group = a.group_stride, half = a.half_stride;
    uint32_t n = 0;                                  // tiles consumed
    uint32_t p_phase[2] = {0, 0}, clean = 0;
    // one lane: S of stream s = Q K^T with K in stage st
    auto scores = [&](int s, int st) {
        const uint64_t q = umma_desc_sw128(sq + s * (kStreamRows * D * 2));
        const uint64_t k = umma_desc_sw128_k(ring + st * kTileBytes<D>, group);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t in = (ks & 3) * 2;        // 32 bytes a step inside the 128-byte row
            umma_bf16(tmem + s * 128, q + (uint64_t)((ks >> 2) * (128 * 128 >> 4) + in),
                      k + (uint64_t)((ks >> 2) * (half >> 4) + in), idesc_s, ks > 0);
        }
        umma_commit(&sh.s_full[s]);
    };
    // one lane: O of stream s (+)= P V with V in stage st
    auto values = [&](int s, int st, bool more) {
        const uint64_t v = umma_desc_sw128_mn(ring + st * kTileBytes<D>, group, half);
#pragma unroll
        for (int ks = 0; ks < kDenseTile / 16; ++ks)
            umma_bf16_ts(tmem + kTmemO + s * D, tmem + s * 128 + ks * 8, v + (uint64_t)(ks * (2 * group >> 4)), idesc_o,
                         more || ks > 0);
    };
    for (uint32_t k = 0;; ++k) {
        const int slot = k % kItemSlots;
        if (!warp_wait(&sh.ring.item_full[slot], (k / kItemSlots) & 1, a.ctrl, lane))
            return;
        if (uniform(sh.ring.item[slot].b) < 0)
            return;
        const int kt0 = uniform(sh.ring.item[slot].kt0), kt1 = uniform(sh.ring.item[slot].kt1);
        const bool two = uniform(sh.ring.item[slot].tokens) > T;
        const int masked_from = uniform((int)dense_masked_from(sh.ring.item[slot].first_pos));
        if (!warp_wait(&sh.q_full, k & 1, a.ctrl, lane))
            return;
        {
            const int st = n % NS;
            if (!warp_wait(&sh.ring.full[st], (n / NS) & 1, a.ctrl, lane))
                return;
            tmem_fence_after();
            if (elect_one()) {
                scores(0, st);
                if (two)
                    scores(1, st);
                umma_commit(&sh.ring.empty[st]);
                if (kt0 + 1 == kt1)
                    umma_commit(&sh.q_empty);
            }
            __syncwarp();
            ++n;
        }
        for (int kt = kt0; kt < kt1; ++kt) {
            const int sv = n % NS, sk = (n + 1) % NS;
            const bool more = kt + 1 < kt1;
            if (kt >= masked_from) {
                if (!warp_wait(&sh.clean[sv], (clean >> sv) & 1, a.ctrl, lane))
                    return;
                clean ^= 1u << sv;
            } else if (!warp_wait(&sh.ring.full[sv], (n / NS) & 1, a.ctrl, lane)) {
                return;
            }
            // (the next K before P: it is there long before, and a wait between
            // two products would leave the tensor cores idle)
            if (more && !warp_wait(&sh.ring.full[sk], ((n + 1) / NS) & 1, a.ctrl, lane))
                return;
            if (!warp_wait(&sh.p_ready[0], p_phase[0]++ & 1, a.ctrl, lane))
                return;
            tmem_fence_after();
            if (elect_one()) {
                values(0, sv, kt > kt0);
                if (!two)
                    umma_commit(&sh.ring.empty[sv]);
                if (more) {
                    scores(0, sk);
                    if (!two) {
                        umma_commit(&sh.ring.empty[sk]);
                        if (kt + 2 == kt1)
                            umma_commit(&sh.q_empty);
                    }
                } else {
                    umma_commit(&sh.o_full[0]);
                }
            }
            __syncwarp();
            if (two) {
                if (!warp_wait(&sh.p_ready[1], p_phase[1]++ & 1, a.ctrl, lane))
                    return;
                tmem_fence_after();
                if (elect_one()) {
                    values(1, sv, kt > kt0);
                    umma_commit(&sh.ring.empty[sv]);
                    if (more) {
                        scores(1, sk);
                        umma_commit(&sh.ring.empty[sk]);
                        if (kt + 2 == kt1)
                            umma_commit(&sh.q_empty);
                    } else {
                        umma_commit(&sh.o_full[1]);
                    }
                }
                __syncwarp();
            }
            n += more ? 2 : 1;
        }
        if (lane == 0)
            mbar_arrive(&sh.ring.item_empty[slot]);
    }
}

// ---- V of the masked tiles ---------------------------------------------------
// A masked token's weight is 0, but 0 times an infinity or NaN is NaN in the
// product, and rows behind the sequence's end hold anything.  So tokens that
// no row of the item sees become zero, and of those that some rows see the
// infinite and NaN elements, which the softmax threads add to the rows that do.
template <int D, int NS>
__device__ __forceinline__ void guard_values(const DenseArgs &a, TcShared &sh, uint8_t *ring, int lane)
{
    uint32_t n = 0;
    for (uint32_t k = 0;; ++k) {
        const int slot = k % kItemSlots;
        if (!warp_wait(&sh.ring.item_full[slot], (k / kItemSlots) & 1, a.ctrl, lane))
            return;
        if (sh.ring.item[slot].b < 0)
            return;
        const int kt0 = sh.ring.item[slot].kt0, kt1 = sh.ring.item[slot].kt1;
        // positions of the item's first and last query token
        const int64_t first = sh.ring.item[slot].first_pos, last = first + sh.ring.item[slot].tokens - 1;
        const int64_t masked_from = dense_masked_from(first);
        for (int kt = kt0; kt < kt1; ++kt, n += 2) {
            // it waits for and releases every tile, K's too, so that it never
            // falls a turn of the ring behind or ahead of the barriers' phases
            if (!warp_wait(&sh.ring.full[n % NS], (n / NS) & 1, a.ctrl, lane))
                return;
            if (lane == 0)
                mbar_arrive(&sh.ring.empty[n % NS]);
            const int st = (n + 1) % NS;
            if (!warp_wait(&sh.ring.full[st], ((n + 1) / NS) & 1, a.ctrl, lane))
                return;
            if (kt < masked_from) {
                if (lane == 0)
                    mbar_arrive(&sh.ring.empty[st]);
                continue;
            }
            // tokens seen by all rows, by some, by none (of the tile's 128)
            const int64_t t0 = (int64_t)kt * kDenseTile;
            const int all = (int)max(min(first + 1 - t0, (int64_t)kDenseTile), (int64_t)0);
            const int some = (int)max(min(last + 1 - t0, (int64_t)kDenseTile), (int64_t)all);
            bool bad = false;
            for (int half = 0; half < D / 64; ++half) {
                uint8_t *rows = ring + st * kTileBytes<D> + half * a.half_stride + (lane & 7) * 16;
                // 8 pieces of 16 bytes a token, 4 tokens at a time
                auto piece = [&](int t) {
                    return reinterpret_cast<uint4 *>(rows + (t >> 3) * a.group_stride + (t & 7) * 128);
                };
#pragma unroll 4
                for (int t = some + (lane >> 3); t < kDenseTile; t += 4)
                    *piece(t) = make_uint4(0u, 0u, 0u, 0u);
                for (int t = all + (lane >> 3); t < some; t += 4) {
                    const uint4 x = *piece(t);
                    const uint4 w = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z),
                                               finite_or_zero(x.w));
                    if (w.x != x.x || w.y != x.y || w.z != x.z || w.w != x.w) {
                        *piece(t) = w;
                        bad = true;
                    }
                }
            }
            if (bad)
                sh.bad[slot] = 1;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.clean[st]);
                mbar_arrive(&sh.ring.empty[st]);
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.ring.item_empty[slot]);
    }
}

template <int D, int NS>
__global__ void __launch_bounds__(kTcThreads, 1)
dense_tc(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
         const __grid_constant__ CUtensorMap vmap, const __grid_constant__ DenseArgs a)
{
    // all of it dynamic, without padding: five 32 KB tiles and Q leave 3 KB
    extern __shared__ __align__(1024) uint8_t dyn_smem[];
    uint8_t *sq = dyn_smem, *ring = sq + 2 * kStreamRows * D * 2;
    TcShared &sh = *reinterpret_cast<TcShared *>(ring + NS * kTileBytes<D>);
    if (smem_u32(dyn_smem) & 1023u) {                // (the swizzle's atoms are 1024 bytes)
        if (threadIdx.x == 0)
            report_timeout(a.ctrl, kSiteDense);
        return;
    }
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    if (tid == 0) {
        sh.ring.init(NS, 2, kSoftmaxWarps + 2);      // a tile is freed by the MMAs and the guard
        for (int s = 0; s < NS; ++s)
            mbar_init(&sh.clean[s], 1);
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.p_ready[s], 4);
            mbar_init(&sh.o_full[s], 1);
        }
        mbar_init(&sh.done, 1);
        mbar_fence_init();
    }
    if (warp == kMmaWarp)
        tmem_alloc(&sh.tmem, kTmemCols);
    // the query rows that no load fills (126 of 128 have a token with 7 heads a
    // group): what lay there would make scores of any size, and a reference
    // raised at every tile
    if (warp < 4) {
        const int pad = kStreamRows / a.G * a.G;
        for (int i = tid; i < 2 * (D / 64) * (kStreamRows - pad) * 8; i += 128) {
            const int row = i >> 3, block = row / (kStreamRows - pad);
            *reinterpret_cast<uint4 *>(sq + block * (kStreamRows * 128) + (pad + row % (kStreamRows - pad)) * 128 +
                                       (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
    }
    if (warp == kLoadWarp && lane < 3)
        tma_prefetch_desc(lane == 0 ? &qmap : (lane == 1 ? &kmap : &vmap));
    pdl_wait();
    pdl_launch_dependents();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();

    if (warp < kSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        softmax_stream<D>(a, sh, warp >> 2, warp & 3, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAuxRegs));
        if (warp == kLoadWarp) {
            const QueryLoad<D> q = {&qmap, sq, &sh.q_full, &sh.q_empty, sh.bad};
            load_items<D, NS, true>(a, sh.ring, ring, &kmap, &vmap, lane, q);
        } else if (warp == kMmaWarp) {
            issue_products<D, NS>(a, sh, smem_u32(sq), smem_u32(ring), lane);
            // every MMA issued has completed before TMEM is released
            if (elect_one())
                umma_commit(&sh.done);
            __syncwarp();
            if (!warp_wait(&sh.done, 0, a.ctrl, lane))
                (void)warp_wait(&sh.done, 0, a.ctrl, lane);
        } else if (warp == kGuardWarp) {
            guard_values<D, NS>(a, sh, ring, lane);
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == kMmaWarp)
        tmem_dealloc(sh.tmem, kTmemCols);
}

}  // namespace

template <int D, int NS>
static cudaError_t launch_tc(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                             const DenseArgs &a, int grid, cudaStream_t st)
{
    constexpr size_t smem = (size_t)2 * kStreamRows * D * 2 + (size_t)NS * kTileBytes<D> + sizeof(TcShared);
    static_assert(smem <= 227 * 1024 && kDenseTableBytes <= NS * kTileBytes<D>, "shared memory");
    const cudaError_t e = ensure_dyn_smem((const void *)dense_tc<D, NS>, (int)smem);
    if (e != cudaSuccess)
        return e;
    return launch_ex(dense_tc<D, NS>, dim3(grid), dim3(kTcThreads), smem, st, 1, qmap, kmap, vmap, a);
}

cudaError_t launch_dense_tc(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                            const DenseArgs &a, int D, int grid, cudaStream_t st)
{
    return D == 128 ? launch_tc<128, 5>(qmap, kmap, vmap, a, grid, st)
                    : launch_tc<64, 8>(qmap, kmap, vmap, a, grid, st);
}

}  // namespace ts
