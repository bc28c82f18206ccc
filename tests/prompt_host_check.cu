// Host-side checks of the prompt attention's sizes, using the very functions the
// kernel calls. One check a run, by its name; prints "ok" and exits 0, or prints
// the first disagreement and exits 1.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "../awq_int4_moe_gb300/csrc/awq_prompt_units.cuh"

using namespace awq;

namespace {

[[noreturn]] void fail(const char *what, long a, long b)
{
    std::printf("FAIL %s: %ld, %ld\n", what, a, b);
    std::exit(1);
}

// Boxes of e4m3 codes begin on 128-byte boundaries of their stage, do not reach
// into one another, and two stages or more fit.
void copies()
{
    for (int columns : {64, 128})
        for (int box = 1; box <= kChunkKeys; box *= 2) {
            const int row = code_row_bytes(columns, box), apart = box * row;
            if (apart % 128) fail("a box that begins between boundaries", columns, box);
            if (row < columns || (box > 1 && row != columns)) fail("rows of a box apart from one another", columns, box);
            if (kChunkCodeBytes / (kChunkKeys * row) < 2) fail("stages", columns, box);
        }
}

// Each sequence of a batch is one thread's, up to the largest batch.
void sequences()
{
    for (int threads : {384, 512})
        for (int batch : {1, 2, 383, 384, 385, 511, 512, 513, 100000, 0x7fffffff - 1000, 0x7fffffff - 383, 0x7fffffff - 1, 0x7fffffff}) {
            int at = 0;
            for (int t = 0; t < threads; ++t) {
                const Span s = sequences_of(batch, t, threads);
                if (s.lo != at || s.hi < s.lo || s.hi > batch) fail("a thread's sequences", batch, t);
                at = s.hi;
            }
            if (at != batch) fail("sequences of no thread", batch, at);
        }
}

// The units of a batch as the blocks of a grid take them: nothing but the batch's own
// units, and of a cut one a first and a last piece of kPiece key tiles or more,
// pieces between them of kCutStep or more.
template <bool TWO>
void pieces_of(int id, const ChunkArgs &a, int grid, long &inner)
{
    int64_t total = 0;
    for (int b = 0; b < a.batch; ++b) total += Costs(sequence_at(a, b), a, TWO).head * a.cache.num_heads;
    const int64_t per = share_of(total, grid);
    std::map<std::tuple<int, int, int>, std::vector<Unit>> taken;
    for (int c = 0; c < grid; ++c) {
        const int64_t x0 = per * c < total ? per * c : total, x1 = x0 + per < total ? x0 + per : total;
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
        while (walk.next(a, u)) taken[{u.b, u.h, u.row0}].push_back(u);
    }
    for (int b = 0; b < a.batch; ++b) {
        const Sequence s = sequence_at(a, b);
        for (int h = 0; h < a.cache.num_heads; ++h)
            for (int row0 = 0; row0 < s.n * a.group; row0 += a.unit_rows) {
                const auto it = taken.find({b, h, row0});
                if (it == taken.end()) fail("a unit that no block has", id, b);
                const std::vector<Unit> &p = it->second;
                for (size_t i = 0; i < p.size() && p.size() > 1; ++i) {
                    const bool end = i == 0 || i + 1 == p.size();
                    if (p[i].k1 - p[i].k0 < (end ? kPiece : kCutStep)) fail("a piece of too few tiles", id, p[i].k1 - p[i].k0);
                    inner += !end;
                }
                taken.erase(it);
            }
    }
    if (!taken.empty()) fail("a unit that is not the batch's", id, static_cast<long>(taken.size()));
}

void pieces()
{
    std::mt19937 g(11);
    auto between = [&](int lo, int hi) { return lo + static_cast<int>(g() % static_cast<uint32_t>(hi - lo + 1)); };
    long inner = 0;
    for (int id = 0; id < 1000; ++id) {
        ChunkArgs a{};
        a.batch = between(1, id % 5 ? 5 : 50);
        a.cache.num_heads = between(1, 8);
        a.group = between(1, 20);
        const bool two = id % 3;
        a.unit_rows = (two ? 256 : 128) / a.group * a.group;
        std::vector<int32_t> cu{0}, lens;
        for (int b = 0; b < a.batch; ++b) {
            lens.push_back(between(0, 4) ? between(0, id % 2 ? 30000 : 900) : 0);
            cu.push_back(cu.back() + (between(0, 2) ? between(0, 8) : between(0, 600)));
        }
        a.tokens = cu.back();
        a.max_len = 30000;
        a.narrow_cost = id % 4 ? kChunkNarrowCost : 0;
        a.cu_seqlens = cu.data();
        a.seq_lens = lens.data();
        const int grid = id % 7 ? 152 : between(1, 160);
        if (two) pieces_of<true>(id, a, grid, inner);
        else pieces_of<false>(id, a, grid, inner);
    }
    if (inner < 1000) fail("hardly a piece between two others", inner, 0);
}

}  // namespace

int main(int argc, char **argv)
{
    const char *const name = argc > 1 ? argv[1] : "";
    if (!std::strcmp(name, "copies")) copies();
    else if (!std::strcmp(name, "sequences")) sequences();
    else if (!std::strcmp(name, "pieces")) pieces();
    else fail("no such check", 0, 0);
    std::puts("ok");
    return 0;
}
