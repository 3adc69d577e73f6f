// Causal attention of each sequence's newest tokens over all of its cached
// tokens (ts_dense_attn): whole prompts, chunks of prompts, single tokens.
//   row i of sequence b (f_b rows, n_b cached tokens) sits at p = n_b - f_b + i
//   out[i, h, :] = sum_{j <= p} softmax_j(scale * q[i, h, :] . K[j, g]) * V[j, g]
//   lse[i, h]    = log sum_{j <= p} exp(scale * q[i, h, :] . K[j, g])
//
// One block takes 64 packed rows (token-major, the G query heads of kv head g
// side by side) and walks the sequence's tokens 64 at a time with a running
// maximum and sum per row: S = Q K^T and O += P V on tensor cores (m16n8k16,
// fp32 accumulators), P rounded to bf16 for the second product (as V is).
#include "ts_device.cuh"
#include "ts_internal.h"

namespace ts {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2f = 0.693147180559945309f;
constexpr int kRows = 64;      // packed rows per block, 16 per warp
constexpr int kTok = 64;       // tokens per tile
constexpr int kDenseThreads = 128;

struct DenseArgs {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_st, st, sh;
    const int64_t *seq_off, *q_off;
    __nv_bfloat16 *out;
    float *lse;
    int Hq, Hkv, G;
    float scale_log2;
    const int32_t *page_table;
    int pt_stride, page_shift;
    int64_t pool_pages;
};

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

// The K / V row of token i of the sequence, -1 where it has none.
__device__ __forceinline__ int64_t token_row(const DenseArgs &a, int b, int64_t off, int64_t n, int64_t i)
{
    if (i >= n)
        return -1;
    if (a.page_table == nullptr)
        return off + i;
    const int32_t pg = __ldcg(a.page_table + (int64_t)b * a.pt_stride + (i >> a.page_shift));
    if (pg < 0 || pg >= a.pool_pages)
        return -1;
    return ((int64_t)pg << a.page_shift) + (i & (((int64_t)1 << a.page_shift) - 1));
}

template <int D>
__global__ void __launch_bounds__(kDenseThreads)
dense_simple(const DenseArgs a)
{
    constexpr int RS = D * 2 + 16;
    __shared__ __align__(128) uint8_t sK[kTok * RS];
    __shared__ __align__(128) uint8_t sV[kTok * RS];
    __shared__ int s_bad;
    __shared__ uint8_t s_valid[kTok];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = blockIdx.y, b = blockIdx.z, G = a.G;
    const int64_t off = a.seq_off[b], n = a.seq_off[b + 1] - off;
    const int64_t q0 = a.q_off[b], f = a.q_off[b + 1] - q0;
    const int64_t row0 = (int64_t)blockIdx.x * kRows;
    if (row0 >= f * G)
        return;
    if (tid == 0)
        s_bad = 0;
    const int64_t first_pos = n - f + row0 / G;                       // of the block's first row
    const int64_t last_pos = n - f + min(f * G - 1, row0 + kRows - 1) / G;
    const int r0 = lane >> 2, c0 = (lane & 3) * 2;

    int64_t rows[2], pos[2];
    bool live[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        rows[e] = row0 + warp * 16 + r0 + e * 8;
        live[e] = rows[e] < f * G;
        pos[e] = live[e] ? n - f + rows[e] / G : -1;
    }
    uint32_t qa[D / 16][4];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int rr = e & 1;
            qa[ks][e] = 0u;
            if (live[rr])
                qa[ks][e] = __ldg(reinterpret_cast<const uint32_t *>(
                    a.q + (q0 + rows[rr] / G) * a.q_st + (int64_t)(g * G + rows[rr] % G) * D + ks * 16 + c0 +
                    (e >> 1) * 8));
        }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[i][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const int64_t clean_from = first_pos + 1 > 0 ? (first_pos + 1) / kTok * kTok : 0;   // first tile with a masked token

    for (int64_t t0 = 0; t0 <= last_pos; t0 += kTok) {
        __syncthreads();
        if (tid < kTok)
            s_valid[tid] = token_row(a, b, off, n, t0 + tid) >= 0;
        constexpr int CPR = D / 8;
        for (int i = tid; i < kTok * CPR; i += kDenseThreads) {
            const int r = i / CPR, c = i - r * CPR;
            const int64_t row = token_row(a, b, off, n, t0 + r);
            uint4 kx = make_uint4(0u, 0u, 0u, 0u), vx = kx;
            if (row >= 0) {
                kx = __ldg(reinterpret_cast<const uint4 *>(a.k + row * a.st + g * a.sh) + c);
                vx = __ldg(reinterpret_cast<const uint4 *>(a.v + row * a.st + g * a.sh) + c);
            }
            if (t0 >= clean_from) {
                // a masked token's weight is 0, and 0 * inf would be NaN in the
                // product: such elements go in as zero and are added at the end
                const uint4 w = make_uint4(finite_or_zero(vx.x), finite_or_zero(vx.y), finite_or_zero(vx.z),
                                           finite_or_zero(vx.w));
                if (w.x != vx.x || w.y != vx.y || w.z != vx.z || w.w != vx.w)
                    s_bad = 1;
                vx = w;
            }
            *reinterpret_cast<uint4 *>(sK + r * RS + c * 16) = kx;
            *reinterpret_cast<uint4 *>(sV + r * RS + c * 16) = vx;
        }
        __syncthreads();
        float s[kTok / 8][4];
#pragma unroll
        for (int nb = 0; nb < kTok / 8; nb += 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[nb][e] = s[nb + 1][e] = 0.0f;
            const uint32_t base = smem_u32(sK + (nb * 8 + (lane & 7) + (lane >> 4) * 8) * RS) + ((lane >> 3) & 1) * 16;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t b0, b1, b2, b3;
                ldmatrix_x4(b0, b1, b2, b3, base + ks * 32);
                mma_16816(s[nb], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b0, b1);
                mma_16816(s[nb + 1], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b2, b3);
            }
        }
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int nb = 0; nb < kTok / 8; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = nb * 8 + c0 + (e & 1);
                s[nb][e] = (t0 + t <= pos[e >> 1] && s_valid[t]) ? s[nb][e] * a.scale_log2 : -INFINITY;
                mx[e >> 1] = fmaxf(mx[e >> 1], s[nb][e]);
            }
        float base[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
            base[e] = mx[e] == -INFINITY ? 0.0f : mx[e];
            const float c = exp2f(m[e] - base[e]);
            m[e] = mx[e];
            l[e] *= c;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                o[i][2 * e] *= c;
                o[i][2 * e + 1] *= c;
            }
        }
#pragma unroll
        for (int nb = 0; nb < kTok / 8; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[nb][e] = exp2f(s[nb][e] - base[e >> 1]);
                l[e >> 1] += s[nb][e];
            }
#pragma unroll
        for (int kt = 0; kt < kTok / 16; ++kt) {
            const uint32_t p0 = pack_bf16(s[2 * kt][0], s[2 * kt][1]), p1 = pack_bf16(s[2 * kt][2], s[2 * kt][3]);
            const uint32_t p2 = pack_bf16(s[2 * kt + 1][0], s[2 * kt + 1][1]),
                           p3 = pack_bf16(s[2 * kt + 1][2], s[2 * kt + 1][3]);
            const uint32_t base_v = smem_u32(sV + (kt * 16 + (lane & 15)) * RS) + (lane >> 4) * 16;
#pragma unroll
            for (int i = 0; i < D / 8; i += 2) {
                uint32_t b0, b1, b2, b3;
                ldmatrix_x4_trans(b0, b1, b2, b3, base_v + i * 16);
                mma_16816(o[i], p0, p1, p2, p3, b0, b1);
                mma_16816(o[i + 1], p0, p1, p2, p3, b2, b3);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        if (s_bad)
            for (int64_t t = clean_from; t <= pos[e]; ++t) {
                const int64_t row = token_row(a, b, off, n, t);
                for (int i = 0; row >= 0 && i < D / 8; ++i)
                    for (int x = 0; x < 2; ++x) {
                        const float y = __bfloat162float(a.v[row * a.st + g * a.sh + i * 8 + c0 + x]);
                        if (!isfinite(y))
                            o[i][2 * e + x] += y;
                    }
            }
        if (!live[e])
            continue;
        const float inv = l[e] == 0.0f ? 0.0f : 1.0f / l[e];
        const int64_t at = (q0 + rows[e] / G) * a.Hq + g * G + rows[e] % G;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<uint32_t *>(a.out + at * D + i * 8 + c0) =
                pack_bf16(o[i][2 * e] * inv, o[i][2 * e + 1] * inv);
        if (a.lse != nullptr && (lane & 3) == 0)
            a.lse[at] = l[e] == 0.0f ? -INFINITY : m[e] * kLn2f + logf(l[e]);
    }
}

}  // namespace

cudaError_t launch_dense(const DensePlan &dp, const ts_kv_t *kv, const void *q, int64_t q_stride_tok,
                         const int64_t *q_off, void *out, float *lse, uint8_t *ws, cudaStream_t st)
{
    (void)ws;
    const Plan &p = dp.p;
    if (dp.rows == 0)
        return cudaSuccess;
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
    a.Hq = p.Hq;
    a.Hkv = p.Hkv;
    a.G = p.G;
    a.scale_log2 = p.scale * kLog2e;
    a.page_table = p.paged ? kv->page_table_dev : nullptr;
    a.pt_stride = kv->page_table_stride;
    a.page_shift = p.page_shift;
    a.pool_pages = kv->pool_pages;
    const dim3 grid((unsigned)((dp.max_rows * p.G + kRows - 1) / kRows), p.Hkv, p.B);
    return p.D == 128 ? launch_ex(dense_simple<128>, grid, dim3(kDenseThreads), 0, st, 1, a)
                      : launch_ex(dense_simple<64>, grid, dim3(kDenseThreads), 0, st, 1, a);
}

}  // namespace ts
