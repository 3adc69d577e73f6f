// Bringing new tokens into a KV cache, many requests at once: the block table,
// slot map and offsets of a paged cache from the requests' lengths
// (ts_extend_pages), and the tokens' K and V rows to their slots (ts_write_kv).
#include "ts_device.cuh"
#include "ts_internal.h"

namespace ts {
namespace {

constexpr int kExtendThreads = 256;
constexpr int kPerThread = kMaxBatch / kExtendThreads;   // sequences per thread of the scans

struct ExtendArgs {
    const int64_t *cached, *fresh;
    int B;
    int page_shift;
    const int32_t *free_pages;
    int64_t n_free, pool_pages;
    int32_t *page_table;
    int stride;
    int64_t *seq_offsets, *q_offsets;   // [B + 1]
    int64_t *slots;
    int64_t n_slots;
    int64_t *pages_used;
};

__device__ __forceinline__ int64_t clamp_length(int64_t n)
{
    return n < 0 ? 0 : (n > 0x7fffffff ? 0x7fffffff : n);
}

// Exclusive prefix sum over the block of one value per thread; the total in
// *total.  s_warp: one entry per warp.
__device__ __forceinline__ int64_t block_exclusive(int64_t x, int64_t *s_warp, int64_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += y;
    }
    if (lane == 31)
        s_warp[warp] = incl;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kExtendThreads / 32; ++w) {
        const int64_t y = s_warp[w];
        before += w < warp ? y : 0;
        all += y;
    }
    __syncthreads();   // s_warp is free again
    *total = all;
    return before + incl - x;
}

// Sequence b holds c cached tokens and gains f: its pages ceil(c / P) ..
// ceil((c + f) / P) - 1 come from the free list, in sequence order, and token
// c + j of it sits in slot table[b][(c + j) / P] * P + (c + j) % P.
//
// Everything a token needs follows from three prefix sums over the sequences
// (tokens, lengths, pages), which every block takes for itself (at most 1024
// sequences, 4 per thread): no pass waits for another and one launch does it.
// A thread then takes one new token at a time.  The one that opens a page
// also enters it in the block table; slots read the free list, never an entry
// that this launch writes.  Bound by three dependent round trips to memory
// (lengths, free list, store): 3.3 us a launch in a graph, at 256 requests of
// one new token as at 48 with 177,000.
__global__ void __launch_bounds__(kExtendThreads)
extend_pages_kernel(const ExtendArgs a)
{
    __shared__ int64_t s_q[kMaxBatch + 1];     // first new token of each sequence
    __shared__ int32_t s_cached[kMaxBatch];
    __shared__ int32_t s_have[kMaxBatch];      // pages before this call
    __shared__ int64_t s_first[kMaxBatch];     // first new page, as an index into the free list
    __shared__ int64_t s_warp[kExtendThreads / 32];
    pdl_wait();
    pdl_launch_dependents();

    const int tid = threadIdx.x;
    const int64_t P = (int64_t)1 << a.page_shift;
    int64_t c[kPerThread], f[kPerThread], pg[kPerThread], have[kPerThread];
    int64_t sum_f = 0, sum_n = 0, sum_p = 0;
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const int b = tid * kPerThread + u;
        c[u] = b < a.B ? clamp_length(__ldcg(a.cached + b)) : 0;
        f[u] = b < a.B ? clamp_length(__ldcg(a.fresh + b)) : 0;
    }
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        have[u] = min((c[u] + P - 1) >> a.page_shift, (int64_t)a.stride);
        pg[u] = min((c[u] + f[u] + P - 1) >> a.page_shift, (int64_t)a.stride) - have[u];
        sum_f += f[u];
        sum_n += c[u] + f[u];
        sum_p += pg[u];
    }
    int64_t total_f, total_n, total_p;
    int64_t ex_f = block_exclusive(sum_f, s_warp, &total_f);
    int64_t ex_n = block_exclusive(sum_n, s_warp, &total_n);
    int64_t ex_p = block_exclusive(sum_p, s_warp, &total_p);
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const int b = tid * kPerThread + u;
        if (b < a.B) {
            s_q[b] = ex_f;
            s_cached[b] = (int32_t)c[u];
            s_have[b] = (int32_t)have[u];
            s_first[b] = ex_p;
            if (blockIdx.x == 0) {
                a.q_offsets[b] = ex_f;
                a.seq_offsets[b] = ex_n;
            }
        }
        ex_f += f[u];
        ex_n += c[u] + f[u];
        ex_p += pg[u];
    }
    if (tid == 0) {
        s_q[a.B] = total_f;
        if (blockIdx.x == 0) {
            a.q_offsets[a.B] = total_f;
            a.seq_offsets[a.B] = total_n;
            *a.pages_used = total_p;
        }
    }
    __syncthreads();

    for (int64_t i = (int64_t)blockIdx.x * kExtendThreads + tid; i < a.n_slots;
         i += (int64_t)gridDim.x * kExtendThreads) {
        int64_t slot = -1;
        if (i < total_f) {
            int lo = 0, hi = a.B;              // s_q[lo] <= i < s_q[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_q[mid] <= i)
                    lo = mid;
                else
                    hi = mid;
            }
            const int64_t pos = s_cached[lo] + (i - s_q[lo]);
            const int64_t j = pos >> a.page_shift;
            if (j < a.stride) {
                int32_t *entry = a.page_table + (int64_t)lo * a.stride + j;
                int32_t page = -1;
                if (j < s_have[lo]) {
                    page = __ldcg(entry);       // the last page from before, partly filled
                } else {
                    const int64_t at = s_first[lo] + (j - s_have[lo]);
                    if (at < a.n_free)
                        page = __ldcg(a.free_pages + at);
                    if (page < 0 || page >= a.pool_pages)
                        page = -1;              // the list ran out, or holds no page of the pool
                    if ((pos & (P - 1)) == 0)
                        *entry = page;          // this token opens the page
                }
                if (page >= 0 && page < a.pool_pages)
                    slot = ((int64_t)page << a.page_shift) + (pos & (P - 1));
            }
        }
        a.slots[i] = slot;
    }
}

struct WriteArgs {
    uint4 *k, *v;
    const uint4 *k_new, *v_new;
    const int64_t *slots;
    int64_t n_new, kv_rows;
    int64_t st, sh;             // cache strides in 16-byte pieces
    int64_t new_st;             // token stride of the new rows in 16-byte pieces
    int log_d8, log_hkv;        // log2 of the pieces of one head's row, of the kv heads
};

constexpr int kWriteThreads = 256;
constexpr int kWriteUnroll = 4;

// One thread moves 16-byte pieces; consecutive threads move consecutive
// pieces of a token's rows, K's tokens first and V's behind them, four
// independent loads in flight.  A copy: bound by HBM at large sizes (16384
// tokens of 4 x 128, 67 MB moved: 12.2 us, 5.5 TB/s; two or eight loads in
// flight, or fewer blocks, measured 12.4-12.9), by the launch and two dependent
// round trips (slot, store) at small ones (64 tokens: 1.8 us in a graph).
__global__ void __launch_bounds__(kWriteThreads)
write_kv_kernel(const WriteArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int log_row = a.log_d8 + a.log_hkv;
    const int64_t per = a.n_new << log_row;              // pieces of K
    const int64_t step = (int64_t)gridDim.x * kWriteThreads;
    for (int64_t i0 = (int64_t)blockIdx.x * kWriteThreads + threadIdx.x; i0 < 2 * per; i0 += kWriteUnroll * step) {
        uint4 x[kWriteUnroll];
        int64_t slot[kWriteUnroll];
#pragma unroll
        for (int u = 0; u < kWriteUnroll; ++u) {
            const int64_t i = i0 + u * step;
            slot[u] = -1;
            if (i < 2 * per) {
                const int64_t j = i >= per ? i - per : i;
                slot[u] = __ldcg(a.slots + (j >> log_row));
                x[u] = __ldcg((i >= per ? a.v_new : a.k_new) + (j >> log_row) * a.new_st +
                             (j & (((int64_t)1 << log_row) - 1)));
            }
        }
#pragma unroll
        for (int u = 0; u < kWriteUnroll; ++u) {
            const int64_t i = i0 + u * step;
            if (slot[u] >= 0 && slot[u] < a.kv_rows) {
                const int64_t j = i >= per ? i - per : i;
                const int g = (int)((j >> a.log_d8) & (((int64_t)1 << a.log_hkv) - 1));
                const int c = (int)(j & (((int64_t)1 << a.log_d8) - 1));
                (i >= per ? a.v : a.k)[slot[u] * a.st + g * a.sh + c] = x[u];
            }
        }
    }
}

int log2_of(int x)
{
    int s = 0;
    while ((1 << s) < x)
        ++s;
    return s;
}

}  // namespace

cudaError_t launch_extend_pages(const int64_t *cached, const int64_t *fresh, int B, int page_size,
                                const int32_t *free_pages, int64_t n_free, int64_t pool_pages, int32_t *page_table,
                                int stride, int64_t *seq_offsets, int64_t *q_offsets, int64_t *slots,
                                int64_t n_slots, int64_t *pages_used, int sms, cudaStream_t st)
{
    const ExtendArgs a = {cached, fresh, B, log2_of(page_size), free_pages, n_free, pool_pages, page_table, stride,
                          seq_offsets, q_offsets, slots, n_slots, pages_used};
    const int64_t want = (n_slots + kExtendThreads - 1) / kExtendThreads;
    const int grid = (int)(want < 1 ? 1 : (want < 2 * sms ? want : 2 * sms));
    return launch_ex(extend_pages_kernel, dim3(grid), dim3(kExtendThreads), 0, st, 1, a);
}

cudaError_t launch_write_kv(const Plan &p, const ts_kv_t *kv, void *k_cache, void *v_cache, const void *k_new,
                            const void *v_new, int64_t new_stride_tok, const int64_t *slots, int64_t n_new,
                            cudaStream_t st)
{
    WriteArgs a;
    a.k = static_cast<uint4 *>(k_cache);
    a.v = static_cast<uint4 *>(v_cache);
    a.k_new = static_cast<const uint4 *>(k_new);
    a.v_new = static_cast<const uint4 *>(v_new);
    a.slots = slots;
    a.n_new = n_new;
    a.kv_rows = p.kv_rows;
    a.st = kv->stride_tok / 8;
    a.sh = kv->stride_head / 8;
    a.new_st = new_stride_tok / 8;
    a.log_d8 = log2_of(p.D / 8);
    a.log_hkv = log2_of(p.Hkv);
    const int64_t pieces = 2 * n_new * p.Hkv * (p.D / 8);
    const int64_t per_block = (int64_t)kWriteThreads * kWriteUnroll;
    const int64_t want = (pieces + per_block - 1) / per_block;
    const int64_t most = (int64_t)p.sms * 32;
    return launch_ex(write_kv_kernel, dim3((unsigned)(want < most ? want : most)), dim3(kWriteThreads), 0, st, 1, a);
}

}  // namespace ts
