// The units of the prompt's attention and how the blocks share them: plain
// functions of the batch's lengths, for the kernel and for checks on the host.
#pragma once

#include "awq_prompt_kernels.cuh"

namespace awq {

// No cut lies within this many key tiles of a unit's ends, for a piece costs its turnaround,
// its bytes in the workspace and a join: a share that would begin or end there has
// the whole or nothing of it. Pieces between two cuts are what the blocks' shares make them, two
// tiles or more (5 new tokens over 2000, 20 heads over 4: pieces of 6, 2, 2 and 6). With 4 / 6 / 8,
// 13 ragged prompts take 179 / 171 / 171 us, 16 sequences that decode beside three
// chunks 110 / 107 / 108, 64 of up to 3000 that decode with heads of 64 83 / 85 / 90 over fp16 and 76 / 79 / 80 over
// e4m3, 8 of 8 new tokens over 4000 with heads of 256 37 / 42 / 46. Pairs of tiles, so that two slots have
// the same number (in eights, 4 prompts with heads of 256 take 153 us, not 143).
constexpr int kPiece = 6, kCutStep = 2;

__host__ __device__ __forceinline__ int least(int a, int b) { return a < b ? a : b; }
__host__ __device__ __forceinline__ int most(int a, int b) { return a > b ? a : b; }
// x / y for 0 <= x, 0 < y, short where both fit 32 bits (nearly always).
__host__ __device__ __forceinline__ int64_t short_div(int64_t x, int64_t y)
{
    if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return x / y;
}

// What a block has of a unit: key tiles k0 .. k1 - 1. 16 words, made by one warp
// and read by the others from shared memory.
struct Unit {
    int64_t at, cost;      // its place in the sum of costs
    int b, h;              // sequence, KV head; b < 0: no more units
    int q0, ctx;           // the sequence's first row of q, its tokens before the new ones
    int row0, rows;        // packed rows
    int keys;              // keys that its last row sees
    int k0, k1, n0;        // n0: tiles from k0 on that its first 128 rows see something of
    int all0, all1;        // keys that every row of the unit and every row of its second tile sees
    __host__ __device__ __forceinline__ int tiles() const { return (keys + kChunkKeys - 1) / kChunkKeys; }
    __host__ __device__ __forceinline__ bool cut() const { return k0 > 0 || k1 < tiles(); }
};
static_assert(sizeof(Unit) == 64, "16 words");

// Keys that packed row `row` sees, `ctx` tokens before the sequence's new ones.
__host__ __device__ __forceinline__ int row_limit(int ctx, int row, int group)
{
    return most(0, ctx + static_cast<int>(static_cast<uint32_t>(row) / static_cast<uint32_t>(group)) + 1);
}

// Key tiles of a unit before a cut at `y` of its cost.
__host__ __device__ __forceinline__ int cut_at(int64_t y, int64_t cost, int tiles)
{
    if (y <= 0) return 0;
    if (y >= cost) return tiles;          // (most units are not cut)
    const int k = static_cast<int>(short_div(y * tiles, cost)) / kCutStep * kCutStep;
    if (k < kPiece || tiles - k < kPiece) return 2 * k < tiles ? 0 : tiles;
    return k;
}

struct Sequence {
    int q0, n, len;
    bool bad;                // its bounds or its length are not what they may be
};
__host__ __device__ __forceinline__ Sequence sequence_at(const ChunkArgs &a, int b)
{
    const int c0 = a.cu_seqlens[b], c1 = a.cu_seqlens[b + 1], len = a.seq_lens ? a.seq_lens[b] : 0;
    Sequence s;
    s.q0 = least(most(c0, 0), a.tokens);
    s.n = least(most(c1, s.q0), a.tokens) - s.q0;
    s.len = a.seq_lens ? least(most(len, 0), a.max_len) : s.n;
    s.bad = c0 != s.q0 || c1 != s.q0 + s.n || len < 0 || len > a.max_len;
    return s;
}

// The sequences whose costs one of `threads` threads adds up: lo .. hi - 1 (in 32 bits
// for every batch that has 32).
struct Span {
    int lo, hi;
};
__host__ __device__ __forceinline__ Span sequences_of(int batch, int thread, int threads)
{
    const int64_t per = batch / threads + (batch % threads != 0), lo = thread * per;
    Span s;
    s.lo = static_cast<int>(lo < batch ? lo : batch);
    s.hi = batch - s.lo > per ? static_cast<int>(s.lo + per) : batch;
    return s;
}

// Costs of a sequence's units for one KV head: unit i costs lin + R (i + 1), in
// keys times G (so that all sequences count alike). A narrow one by itself costs 7/8 of
// that (half the products, but as many bytes: 16 sequences that decode beside three
// chunks 107 us, with a factor of 1 113; nothing else measured changes by more than 1 %), over e4m3 with a larger fixed
// part, as its first tiles wait for their expansion. With none / 384 / 768 keys' time more, 4 new tokens of 32
// sequences take 172 / 150 / 143 us, 16 beside chunks 106 / 107 / 110, 64 that decode with heads of 64
// 74 / 79 / 81; over 16 bits 384 cost those 85 -> 90 us.
struct Costs {
    int64_t lin, head;
    int T, R;
    bool narrow;
    __host__ __device__ __forceinline__ Costs() {}
    __host__ __device__ __forceinline__ Costs(const Sequence &s, const ChunkArgs &a, bool two_slots) : R(a.unit_rows)
    {
        const uint32_t rows = static_cast<uint32_t>(s.n) * static_cast<uint32_t>(a.group);     // (below 2^31: the host has checked)
        T = static_cast<int>((rows + static_cast<uint32_t>(R) - 1) / static_cast<uint32_t>(R));
        narrow = two_slots && rows <= 128;
        lin = a.group * (static_cast<int64_t>(most(s.len - s.n, 0)) + kChunkUnitCost + (narrow ? a.narrow_cost : 0));
        head = before(T);
    }
    __host__ __device__ __forceinline__ int64_t before(int i) const
    {
        const int64_t c = i * lin + static_cast<int64_t>(i) * (i + 1) / 2 * R;
        return narrow ? c * 7 / 8 : c;
    }
};

// Walks through the units of a block's share [x0, x1) of the costs. Only its place
// is kept; the sequence is looked at again for each unit.
template <bool TWO_SLOTS>
struct UnitWalk {
    int64_t x0, x1, at;      // the share; where the next unit begins
    int b, h, t;

    __host__ __device__ __forceinline__ UnitWalk(const ChunkArgs &a, int64_t from, int64_t to, int first, int64_t first_at)
        : x0(from), x1(to), at(first_at), b(first), h(0), t(0)
    {
        if (x0 >= x1) {
            at = x1;                                    // no share: no units
            return;
        }
        const Costs c(sequence_at(a, b), a, TWO_SLOTS);
        h = static_cast<int>(short_div(x0 - at, c.head));
        at += h * c.head;
        // the last unit that begins at or before x0
        int lo = 0, hi = c.T - 1;
#pragma unroll 1
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (at + c.before(mid) <= x0) lo = mid;
            else hi = mid - 1;
        }
        t = lo;
        at += c.before(t);
    }
    // The block's next unit.
    __host__ __device__ __forceinline__ bool next(const ChunkArgs &a, Unit &u)
    {
#pragma unroll 1
        while (at < x1) {
            const Sequence s = sequence_at(a, b);
            const Costs c(s, a, TWO_SLOTS);
            if (t == c.T) {                             // (units remain, as costs do)
                t = 0;
                if (++h == a.cache.num_heads || c.T == 0) {
                    h = 0;
                    ++b;
                }
                continue;
            }
            const int row0 = t * a.unit_rows, rows = least(a.unit_rows, s.n * a.group - row0), ctx = s.len - s.n;
            u.at = at;
            u.cost = c.before(t + 1) - c.before(t);
            u.b = b;
            u.h = h;
            u.q0 = s.q0;
            u.ctx = ctx;
            u.row0 = row0;
            u.rows = rows;
            u.keys = row_limit(ctx, row0 + rows - 1, a.group);
            const int tiles = u.tiles();
            u.k0 = cut_at(x0 - at, u.cost, tiles);
            u.k1 = cut_at(x1 - at, u.cost, tiles);
            const int seen0 = row_limit(ctx, row0 + least(rows, 128) - 1, a.group);
            u.n0 = least(u.k1 - u.k0, most(0, (seen0 + kChunkKeys - 1) / kChunkKeys - u.k0));
            u.all0 = row_limit(ctx, row0, a.group);
            u.all1 = row_limit(ctx, row0 + 128, a.group);
            const bool mine = tiles ? u.k1 > u.k0 : x0 <= at;
            at += u.cost;
            ++t;
            if (mine) return true;
        }
        return false;
    }
};

// The blocks' equal share of the sum of all costs, and those that share a cut
// unit: block c has [c per, (c + 1) per).
__host__ __device__ __forceinline__ int64_t share_of(int64_t total, int blocks) { return short_div(total + blocks - 1, blocks); }
__host__ __device__ __forceinline__ int first_block(const Unit &u, int64_t per) { return static_cast<int>(short_div(u.at, per)); }
__host__ __device__ __forceinline__ int last_block(const Unit &u, int64_t per) { return static_cast<int>(short_div(u.at + u.cost - 1, per)); }
__host__ __device__ __forceinline__ bool shares(const Unit &u, int64_t per, int c)
{
    return cut_at((c + 1) * per - u.at, u.cost, u.tiles()) > cut_at(c * per - u.at, u.cost, u.tiles());
}

}  // namespace awq
