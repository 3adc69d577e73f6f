// The division of dense attention's work over blocks (dense_common.cuh) on
// the CPU, for tests/test_dense_walk_cpu.py.
//
// The source between the header's piece and row definitions (walk.inc) is
// compiled for the host.  For random batches, head counts and grids every
// block's pieces are walked; together they must cover every tile of every
// item once, and the pieces that dense_merge would join for an item (the
// block that begins it, then each further block up to the first that is not
// wholly inside it) must be the ones that were walked.  Prints
// "<cases> cases, <failures> failures".
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <map>
#include <random>
#include <tuple>
#include <vector>

struct dim3 {
    unsigned x = 1, y = 1, z = 1;
};
static dim3 blockIdx, gridDim;
#define __device__
#define __forceinline__ inline
#define __align__(x) alignas(x)
constexpr int kMaxBatch = 1024;
template <typename T>
static T __ldcg(const T *p) { return *p; }
using std::max;
using std::min;
typedef uint16_t __nv_bfloat16;

struct DenseArgs;
static int dense_next_seq(const DenseArgs &a, int b);
#include "walk.inc"

// (the device's takes 32 sequences a round trip)
static int dense_next_seq(const DenseArgs &a, int b)
{
    while (b < a.B && seq_items(a, a.q_off[b + 1] - a.q_off[b]) == 0)
        ++b;
    return b;
}

int main()
{
    std::mt19937_64 rng(7);
    auto pick = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
    int cases = 0, failures = 0;
    for (int trial = 0; trial < 12000; ++trial) {
        const int B = (int)pick(1, trial % 7 == 0 ? 40 : 6);
        std::vector<int64_t> so(B + 1, 0), qo(B + 1, 0);
        const int64_t n_hi = trial % 3 == 0 ? 200 : (trial % 3 == 1 ? 5000 : 200000);
        const int64_t f_hi = trial % 4 == 0 ? 1 : (trial % 4 == 1 ? 20 : (trial % 4 == 2 ? 700 : 6000));
        for (int b = 0; b < B; ++b) {
            const int64_t n = pick(0, n_hi), f = pick(0, 5) == 0 ? 1 : pick(0, f_hi);
            so[b + 1] = so[b] + n;
            qo[b + 1] = qo[b] + (pick(0, 30) ? min(f, n) : f);      // now and then more queries than tokens
        }
        DenseArgs a = {};
        a.seq_off = so.data();
        a.q_off = qo.data();
        a.B = B;
        a.Hkv = 1 << pick(0, 3);
        a.G = (int)pick(1, 16);
        a.single = (int)pick(0, 1);
        a.TT = a.single ? 1 : 2 * (128 / a.G);
        a.split = pick(0, 3) != 0;
        a.item_cost = (int)pick(64, 600);
        gridDim.x = (unsigned)(pick(0, 4) ? (pick(0, 3) ? pick(1, 148) : 148) : 1);
        std::vector<int64_t> start(B + 1, 0);
        for (int b = 0; b < B; ++b) {
            const int64_t n = so[b + 1] - so[b], f = qo[b + 1] - qo[b];
            start[b + 1] = start[b] + a.Hkv * items_cost(a, n > f ? n - f : 0, seq_items(a, f));
        }
        a.inv_grid = 1.0 / gridDim.x;
        const DenseTables tab = {start.data(), so.data(), qo.data()};
        using Key = std::tuple<int, int, int>;
        struct Part {
            int kt0, kt1, slot, tiles, tokens, head;
        };
        std::map<Key, std::vector<Part>> got;
        std::vector<DensePiece> pieces(gridDim.x);
        bool ok = true;
        for (unsigned c = 0; c < gridDim.x; ++c) {
            blockIdx.x = c;
            DenseWalk w;
            w.parts.cut(a, start[B]);
            w.at = dense_locate(a, tab, w.parts.at((int)c));
            w.end = dense_locate(a, tab, w.parts.at((int)c + 1));
            pieces[c] = w.piece(a);
            DenseItem it;
            while (w.next(a, it)) {
                ok &= it.kt0 < it.kt1 && it.off == so[it.b] && it.q_row == qo[it.b] + (int64_t)it.t * a.TT;
                ok &= it.n == so[it.b + 1] - so[it.b];
                ok &= it.first_pos == it.n - (qo[it.b + 1] - qo[it.b]) + (int64_t)it.t * a.TT;
                got[Key(it.b, it.g, it.t)].push_back({it.kt0, it.kt1, it.slot, it.tiles, it.tokens,
                                                          it.slot >= 0 ? dense_head(a, it, w.parts) : -1});
            }
        }
        size_t items = 0;
        for (int b = 0; b < B; ++b) {
            const int64_t n = so[b + 1] - so[b], f = qo[b + 1] - qo[b];
            if (a.single ? f != 1 : f < 2)
                continue;
            for (int g = 0; g < a.Hkv; ++g)
                for (int64_t t = 0; t * a.TT < f; ++t) {
                    ++items;
                    const int64_t seen = n - f + min((t + 1) * a.TT, f);
                    const int tiles = seen > 0 ? (int)((seen + 127) / 128) : 1;
                    auto &parts = got[Key(b, g, (int)t)];
                    int at = 0;
                    for (const Part &p : parts) {
                        ok &= p.kt0 == at && p.tiles == tiles && p.tokens == (int)min((int64_t)a.TT, f - t * a.TT);
                        ok &= (p.slot < 0) == (p.kt0 == 0 && p.kt1 == tiles);
                        at = p.kt1;
                    }
                    ok &= at == tiles && (a.split || parts.size() == 1);
                }
        }
        ok &= got.size() == items;
        // the joins: slots in order, one chain per item in parts
        std::map<Key, std::vector<int>> joined;
        for (unsigned c = 0; c + 1 < gridDim.x; ++c) {
            if (!(pieces[c].flags & kPieceHead))
                continue;
            std::vector<int> slots{2 * (int)c + 1};
            for (unsigned q = c + 1; q < gridDim.x; ++q) {
                slots.push_back(2 * (int)q);
                if (!(pieces[q].flags & kPieceThrough))
                    break;
            }
            joined[Key(pieces[c].b, pieces[c].g, pieces[c].t)] = slots;
        }
        ok &= !(pieces[gridDim.x - 1].flags);
        for (auto &e : got) {
            std::vector<int> slots;
            for (const Part &p : e.second)
                if (p.slot >= 0)
                    slots.push_back(p.slot);
            ok &= slots.empty() ? !joined.count(e.first) : joined.count(e.first) && joined[e.first] == slots;
            joined.erase(e.first);
        }
        ok &= joined.empty();
        // every piece knows the block that begins its item, which begins no other shared one
        std::map<int, Key> heads;
        for (auto &e : got)
            for (const Part &p : e.second)
                if (p.slot >= 0)
                    ok &= 2 * p.head + 1 == e.second[0].slot && heads.emplace(p.head, e.first).first->second == e.first;
        ++cases;
        if (!ok && failures++ < 5)
            std::printf("failed: trial %d B %d Hkv %d G %d single %d split %d grid %u\n", trial, B, a.Hkv, a.G, a.single,
                        a.split, gridDim.x);
    }
    std::printf("%d cases, %d failures\n", cases, failures);
    return failures != 0;
}
