// Host-side check of the prompt attention's units, using the very functions the
// kernel calls (awq_prompt_units.cuh): for random batches, head groups and grids
// it replays every block's walk and checks that each unit's key tiles are taken
// exactly once, that a unit that nothing is seen of is taken once, that a block
// has at most one unit that is cut at its begin and one cut at its end, and that
// the blocks which share a cut unit are those that the kernel counts. Prints "ok
// <batches>" and exits 0, or prints the first disagreement and exits 1.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "../awq_int4_moe_gb300/csrc/awq_prompt_units.cuh"

using namespace awq;

namespace {

struct Taken {
    std::vector<int> tiles;
    int empty = 0;
    std::vector<int> blocks;
    Unit u;
};

[[noreturn]] void fail(const char *what, int batch, int block)
{
    std::printf("FAIL %s: batch %d, block %d\n", what, batch, block);
    std::exit(1);
}

template <bool TWO>
void check(int id, const ChunkArgs &a, int grid)
{
    int64_t total = 0;
    for (int b = 0; b < a.batch; ++b) total += Costs(sequence_at(a, b), a, TWO).head * a.cache.num_heads;
    const int64_t per = share_of(total, grid);
    std::map<std::tuple<int, int, int>, Taken> seen;
    for (int c = 0; c < grid; ++c) {
        const int64_t x0 = std::min(total, per * c), x1 = std::min(total, x0 + per);
        int first = 0;
        int64_t before = 0;
        if (x0 < x1)
            for (;; ++first) {
                const int64_t cost = Costs(sequence_at(a, first), a, TWO).head * a.cache.num_heads;
                if (x0 < before + cost) break;
                before += cost;
            }
        UnitWalk<TWO> walk(a, x0, x1, first, before);
        Unit u;
        int begins = 0, ends = 0, last = 0;
        while (walk.next(a, u)) {
            if (u.b < 0 || u.b >= a.batch || u.h < 0 || u.h >= a.cache.num_heads) fail("unit out of range", id, c);
            const Sequence s = sequence_at(a, u.b);
            const int want = std::max(0, s.len - s.n + (u.row0 + u.rows - 1) / a.group + 1);
            if (u.rows < 1 || u.row0 + u.rows > s.n * a.group || u.keys != want) fail("unit's rows", id, c);
            if (u.k0 < 0 || u.k1 > u.tiles() || (u.tiles() > 0 && u.k0 >= u.k1)) fail("unit's tiles", id, c);
            if (u.n0 < 0 || u.n0 > u.k1 - u.k0) fail("first slot's tiles", id, c);
            Taken &t = seen[{u.b, u.h, u.row0}];
            t.u = u;
            t.tiles.resize(u.tiles(), 0);
            for (int k = u.k0; k < u.k1; ++k) ++t.tiles[k];
            if (u.tiles() == 0) ++t.empty;
            if (u.cut()) {
                if (begins && u.k0 > 0) fail("a second cut at the begin", id, c);
                if (ends) fail("a unit behind one that is cut at its end", id, c);
                begins += u.k0 > 0;
                ends += u.k0 == 0;
                if (u.k0 > 0 && last) fail("a cut begin behind another unit", id, c);
                t.blocks.push_back(c);
            }
            ++last;
        }
    }
    // every unit, whole
    for (int b = 0; b < a.batch; ++b) {
        const Sequence s = sequence_at(a, b);
        for (int h = 0; h < a.cache.num_heads; ++h)
            for (int row0 = 0; row0 < s.n * a.group; row0 += a.unit_rows) {
                const auto it = seen.find({b, h, row0});
                if (it == seen.end()) fail("a unit that no block has", id, b);
                const Taken &t = it->second;
                for (int n : t.tiles)
                    if (n != 1) fail("a tile not taken once", id, b);
                if (t.tiles.empty() && t.empty != 1) fail("an empty unit not taken once", id, b);
                if (t.blocks.empty()) continue;
                std::vector<int> want;
                for (int c = first_block(t.u, per); c <= last_block(t.u, per); ++c)
                    if (shares(t.u, per, c)) want.push_back(c);
                if (want != t.blocks) fail("blocks of a cut unit", id, b);
                seen.erase(it);
            }
    }
    for (const auto &e : seen)
        if (e.second.blocks.size()) fail("a unit that is none", id, -1);
}

}  // namespace

int main()
{
    std::mt19937 g(7);
    auto between = [&](int lo, int hi) { return lo + static_cast<int>(g() % static_cast<uint32_t>(hi - lo + 1)); };
    const int batches = 3000;
    for (int id = 0; id < batches; ++id) {
        ChunkArgs a{};
        a.batch = between(1, id % 10 == 0 ? 60 : 6);
        a.cache.num_heads = between(1, 8);
        a.group = between(1, 20);
        const bool two = id % 3;
        a.unit_rows = (two ? 256 : 128) / a.group * a.group;
        const int longest = id % 4 == 0 ? 40000 : 900;
        std::vector<int32_t> cu{0}, lens;
        for (int b = 0; b < a.batch; ++b) {
            const int len = between(0, 5) ? between(0, longest) : 0;
            int n = between(0, 3) ? between(0, std::min(len, 700)) : between(0, 40);      // more new ones than there are, too
            lens.push_back(len);
            cu.push_back(cu.back() + n);
        }
        a.tokens = cu.back();
        a.max_len = longest;
        a.narrow_cost = id % 2 ? kChunkNarrowCost : 0;
        if (id % 50 == 7) {                      // bounds and lengths that are not what they may be
            cu[a.batch / 2] = between(-5, a.tokens + 5);
            lens[0] = between(0, 1) ? -3 : longest + 9;
        }
        a.cu_seqlens = cu.data();
        a.seq_lens = id % 5 ? lens.data() : nullptr;
        const int grid = id % 7 ? 152 : between(1, 160);
        if (two) check<true>(id, a, grid);
        else check<false>(id, a, grid);
    }
    std::printf("ok %d\n", batches);
    return 0;
}
