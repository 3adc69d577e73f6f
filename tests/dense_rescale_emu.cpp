// The rescaling of one row of the accumulator (dense_tc.cu, rescale_row) on the
// CPU, for tests/test_dense_rescale_cpu.py.
//
// Tensor memory is modelled as asynchronous: a store becomes visible to loads
// at the next wait for stores only, and a load's registers hold its values
// after the wait for loads only.  Two rescales in turn must give the product
// of both factors.  Prints "<values> values, <failures> failures".
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <utility>
#include <vector>

#define __device__
#define __forceinline__ inline

constexpr int kColumns = 512;
static uint32_t tmem[kColumns];
static std::vector<std::pair<uint32_t, uint32_t>> stores;     // column, value: not visible yet
struct Load {
    uint32_t column;
    uint32_t *to;
    int count;
};
static std::vector<Load> loads;

static float __uint_as_float(uint32_t x)
{
    float y;
    std::memcpy(&y, &x, 4);
    return y;
}
static uint32_t __float_as_uint(float x)
{
    uint32_t y;
    std::memcpy(&y, &x, 4);
    return y;
}
template <int N>
static void tmem_ld_32x32b(uint32_t column, uint32_t *v)
{
    loads.push_back({column, v, N});
}
static void tmem_wait_ld()
{
    for (const Load &l : loads)
        std::memcpy(l.to, tmem + l.column, sizeof(uint32_t) * l.count);
    loads.clear();
}
static void tmem_st16(uint32_t column, const uint32_t *v)
{
    for (uint32_t e = 0; e < 16; ++e)
        stores.emplace_back(column + e, v[e]);
}
static void tmem_wait_st()
{
    for (const auto &s : stores)
        tmem[s.first] = s.second;
    stores.clear();
}

#include "rescale.inc"

template <int D>
static void run(int &values, int &failures)
{
    const uint32_t to = 256;
    for (uint32_t c = 0; c < kColumns; ++c)
        tmem[c] = __float_as_uint(1.0f + c);
    rescale_row<D>(to, 0.5f);
    rescale_row<D>(to, 0.25f);
    tmem_wait_st();
    for (uint32_t c = 0; c < kColumns; ++c, ++values) {
        const float f = c >= to && c < to + D ? 0.125f : 1.0f;
        failures += __uint_as_float(tmem[c]) != (1.0f + c) * f;
    }
}

int main()
{
    int values = 0, failures = 0;
    run<64>(values, failures);
    run<128>(values, failures);
    std::printf("%d values, %d failures\n", values, failures);
    return failures != 0;
}
