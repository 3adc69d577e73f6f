// Where dense attention finds a token's row (dense_common.cuh: dense_page and
// dense_row) on the CPU, for tests/test_dense_rows_cpu.py: every read of the
// block table is checked against its bounds, for lengths that pass the table's
// row and the cache too.  Prints "<tokens> tokens, <failures> failures".
#include <cstdint>
#include <cstdio>
#include <vector>

#define __device__
#define __forceinline__ inline

struct DenseArgs {
    const int32_t *page_table;
    int pt_stride, page_shift;
    int64_t pool_pages, kv_rows;
};
static const int32_t *table_begin, *table_end;
static int failures;
static int32_t __ldcg(const int32_t *p)
{
    if (p >= table_begin && p < table_end)
        return *p;
    ++failures;
    return 0;
}

#include "rows.inc"

int main()
{
    int64_t tokens = 0;
    for (int shift : {3, 4, 7, 12})
        for (int stride : {1, 3, 40}) {
            const int B = 3, pool = 11;
            std::vector<int32_t> table(B * stride);
            for (int i = 0; i < B * stride; ++i)
                table[i] = i % 5 == 4 ? (i % 2 ? -1 - i : pool + i) : (7 * i + 2) % pool;      // some outside the pool
            table_begin = table.data();
            table_end = table_begin + table.size();
            const DenseArgs a = {table.data(), stride, shift, pool, (int64_t)pool << shift};
            for (int b = 0; b < B; ++b)
                for (int64_t i = 0; i < ((int64_t)stride + 2) << shift; ++i, ++tokens) {
                    const int64_t j = i >> shift;
                    const int32_t pg = j < stride ? table[b * stride + j] : -1;
                    const int64_t want = pg < 0 || pg >= pool ? -1 : ((int64_t)pg << shift) + i % ((int64_t)1 << shift);
                    failures += dense_row(a, b, 0, i) != want;
                }
        }
    const DenseArgs packed = {nullptr, 0, 0, 0, 100};
    for (int64_t off : {0, 40, 99, 100})
        for (int64_t i = 0; i < 200; ++i, ++tokens)
            failures += dense_row(packed, 0, off, i) != (off + i < 100 ? off + i : -1);
    std::printf("%lld tokens, %d failures\n", (long long)tokens, failures);
    return failures != 0;
}
