// Host-side checks of the prompt attention's sizes, using the very functions the
// kernel calls. One check a run, by its name; prints "ok" and exits 0, or prints
// the first disagreement and exits 1.
#include <cstdio>
#include <cstdlib>
#include <cstring>

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

}  // namespace

int main(int argc, char **argv)
{
    const char *const name = argc > 1 ? argv[1] : "";
    if (!std::strcmp(name, "copies")) copies();
    else if (!std::strcmp(name, "sequences")) sequences();
    else fail("no such check", 0, 0);
    std::puts("ok");
    return 0;
}
