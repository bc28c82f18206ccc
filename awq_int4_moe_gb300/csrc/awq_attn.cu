// awq_paged_attention: one new token per sequence over the paged cache.
//
// Work is counted in units of KT cached tokens (8 KB of K and V where a row
// is at most 256 bytes) of one segment: a (sequence, KV head, tile of query
// heads). Units are numbered segment by segment, and every warp of the grid
// takes the same number of consecutive ones, whatever segments they belong
// to, so that all read the same number of cache bytes however ragged the
// batch is. A segment that lies inside a warp's range is finished there; what
// is cut leaves parts (running maximum, sum, unnormalised output, all fp32):
// the block's warps join theirs in shared memory at the end, and a
// segment that is cut between blocks leaves a piece per block in the
// workspace, joined in block order by the block that finishes last (so the
// result does not depend on which one that is). No warp waits for another
// before that.
//
// A warp copies its units' rows with cp.async (16 bytes a lane, several units
// deep, running on into the next segment). With up to 8 query heads as the
// columns of the tensor-core tile (mma.m16n8k16, fp32 accumulators; 9 to 16
// heads are two tiles):
//   S'[16 tokens x 8] = K Q', K's rows read with ldmatrix as the A operand
//   m' = max(m, S), P = exp2(S - m'), l = l * 2^(m - m') + sum P
//   O'[16 of D x 8]   = O' * 2^(m - m') + V' P', V read with ldmatrix.trans
// so no row of the tile is padding at 8 heads, a head's statistics and its
// output are in the same lanes, and P moves from the accumulator's layout to
// the B operand's with movmatrix. m is raised only where a score passes it by
// more than 2^8 (P stays below 2^8 times the maximum's own weight, the sums are
// fp32), which drops both the search for the maximum and the scaling of O' from
// nearly every unit. P
// enters the tensor core as two 16-bit terms, P = hi + lo (2^-23 of a weight is
// lost with fp16, 2^-17 with bf16), so that the numerator takes the weights
// that the fp32 sum takes and their rounding does not reach the output.
//
// e4m3 planes are expanded to fp16 in registers (exact): a 4-byte lane of an
// ldmatrix row holds 4 neighbouring elements of the head, so Q's elements are
// dealt to the fragments in the same order (the dot product does not care),
// and V's rows of O' come in an order that the store undoes. bf16 Q becomes
// fp16 with its head's power of two taken out (exact to 2^-24 of the head's
// largest element).
//
// Bound: 4 * group operations per cached element of 1 or 2 bytes, so the
// bytes decide; the tensor-core tiles have a few times the rate they need. 1
// sequence of 131071 tokens, 32 / 4 heads of 128, bf16: 51.5 us, 5.2 TB/s; 64 of
// up to 16000, 64 / 8 heads, e4m3: 173 us, 5.9 TB/s; the fixed part (lengths,
// table, first copies, merge, join) is about 9 us of each.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "awq_decoder_kernels.cuh"
#include "awq_launch.cuh"

namespace awq {

namespace {

constexpr int kLens = 128;              // sequence lengths kept in shared memory
constexpr float kLazy = 8.f;           // a score raises the maximum when it passes it by this (base 2)
// fp16 weights are taken against 2^-7 of the maximum: they stay below 2^15 and
// keep 31 bits below the maximum's own before they vanish (with 24, thousands
// of tokens of a weight of 2^-25 would vanish beside a single large one).
constexpr float kRaiseF16 = 7.f;
// Least factor that turns a score into a base-2 logarithm: with 0 (a scale of 0) a
// masked score of -infinity would be NaN. The smallest fp32 makes 2^-21 of the
// largest score.
constexpr float kMinFactor = 1.40129846e-45f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The cache's rows are read once per call and are first to leave L2, so that
// they do not push out what the next call needs again (its code, q, the page
// table, the workspace).
__device__ __forceinline__ uint64_t evict_first_policy()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void *src, uint32_t bytes, uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes), "l"(policy)
                 : "memory");
}

__device__ __forceinline__ float4 lds_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ int atom_add_acq_rel(int32_t *p, int v)
{
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                        uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes as two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t four, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}

// 8x8 16-bit matrix across the warp, transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A pair of fp32 values as 16-bit terms hi + lo.
template <typename C>
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = pack2<C>(a, b);
    const float2 h = unpack2<C>(hi);
    lo = pack2<C>(a - h.x, b - h.y);
}

// Reductions over the eight lanes that hold a head's column.
__device__ __forceinline__ float col_max(float v)
{
    v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
    v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
    return fmaxf(v, __shfl_xor_sync(~0u, v, 16));
}
__device__ __forceinline__ float col_sum(float v)
{
    v += __shfl_xor_sync(~0u, v, 4);
    v += __shfl_xor_sync(~0u, v, 8);
    return v + __shfl_xor_sync(~0u, v, 16);
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

struct BatchView {
    const int32_t *seq_lens;
    const int32_t *s_len;     // lengths of sequences b0 .. b0 + kLens - 1
    int b0, max_len;
    int per_seq;              // segments of a sequence: KV heads x head tiles

    __device__ __forceinline__ int clamp(int n) const { return n < 0 ? 0 : n > max_len ? max_len : n; }
    __device__ __forceinline__ int len(int b) const
    {
        const int i = b - b0;
        return clamp(i < kLens ? s_len[i] : seq_lens[b]);
    }
};

// A position in the flat order of units: segment s of sequence b (n tokens),
// unit u.
template <int KT>
struct Cursor {
    int b, s, n, u;
    int left;                 // units from u to the end of the warp's range

    __device__ __forceinline__ int units() const { return (n + KT - 1) / KT; }
    // the segment's units that belong to the warp: [u, end())
    __device__ __forceinline__ int end() const
    {
        const int e = units();
        return left < e - u ? u + left : e;
    }
    // to the first unit of the next segment that has any
    __device__ __forceinline__ void next_segment(const BatchView &v)
    {
        left -= end() - u;
        u = 0;
        if (left <= 0) return;
        if (++s == v.per_seq) {
            s = 0;
            do {
                ++b;
                n = v.len(b);
            } while (n == 0);
        }
    }
};

// Warps of a block. An e4m3 unit costs about 2,800 cycles of a warp's time
// and is due every 350 cycles of a multiprocessor, so that 8 warps only just
// keep up with the memory; 16-bit units take half of that. 12 for 16-bit rows
// of 64 as well (128 sequences of up to 1500, 8 heads: 38.3 us, 42.8 with 8;
// 64 / 8 heads: 42.6, 47.4; 256 of 512, 20 / 4 heads: 31.0, 29.2), but not for
// those of 128 (1 of 131071, 32 / 4 heads: 54.1 us, 51.6 with 8). Two tiles of
// heads need the registers of 8 warps (64 of up to 4000, 64 / 4 heads, e4m3:
// 49.7 us, 55.1 with 12; with heads of 256 the compiler spills 36 to 84 bytes:
// 55.6 us, bf16 84.2, floors 20 and 40), 16-bit rows of 256 elements the shared
// memory of 4 (16 KB a unit).
constexpr int attn_warps(bool fp8, int dp, int nt)
{
    return !fp8 && dp == 256 ? 4 : nt == 1 && dp <= (fp8 ? 128 : 64) ? 12 : 8;
}

// NT: tiles of 8 query heads.
template <bool FP8, int DP, int NT>
struct Geo {
    static constexpr int kElem = FP8 ? 1 : 2;
    static constexpr int kRow = DP * kElem;             // bytes of a token's row in shared memory
    static constexpr int kChunks = kRow / 16;
    static constexpr int KT = kRow >= 256 ? 16 : 4096 / kRow;    // tokens of a unit
    static constexpr int kPlane = KT * kRow;
    static constexpr int kStage = 2 * kPlane;           // K rows, then V rows
    static constexpr int kPitch = attn_part_pitch(DP);  // floats of a part's row: output, maximum, sum
    // Warps of a block, and units of each in shared memory (one in use, the
    // others in flight; 64 to 128 KB in flight cover the latency, more only
    // lengthens it).
    static constexpr int kWarps = attn_warps(FP8, DP, NT);
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStages = kWarps * kStage > 64 * 1024 ? 2 : 3;
    static constexpr int kQPitch = 2 * DP + 16;         // bytes of a q row on its way to the fragments: no bank twice
    static constexpr int kSmem = kWarps * (kStages * kStage + 8 * kQPitch);
    static constexpr int kJoinRows = kStages * kStage / (4 * kPitch) >= 32 ? 32 : 16;   // pieces' rows over a warp's ring
    static constexpr bool kPartsFit = kStages * kStage >= 2 * 8 * NT * kPitch * 4;     // two parts over a warp's ring
    static_assert(kSmem <= 226 * 1024 && kStages * kStage >= 8 * NT * kPitch * 4 && kStages * kStage >= kJoinRows * kPitch * 4, "a part fits over a warp's ring");

    // 16-byte chunk c of row r, placed so that 8 rows of one chunk fall into
    // different banks. Planes are aligned to a row, so chunk c ^ x of the row
    // is at(r, c) ^ (x << 4).
    static __device__ __forceinline__ uint32_t at(int r, int c)
    {
        const int sw = kRow >= 128 ? (r & 7) : ((r >> 1) & 3);
        return static_cast<uint32_t>(r * kRow + ((c ^ sw) << 4));
    }
};

// A part of a segment, left by a warp.
struct PartMeta {
    int32_t seg_begin;        // flat number of the segment's first unit; -1: none
    int32_t b, s;
};

template <typename T, bool FP8, int DP, int NT>
__global__ void __launch_bounds__(Geo<FP8, DP, NT>::kThreads, 1) attn_kernel(const AttnArgs a)
{
    using G = Geo<FP8, DP, NT>;
    using C = typename std::conditional<FP8, __half, T>::type;   // the tensor core's type
    constexpr float kRaise = std::is_same<C, __half>::value ? kRaiseF16 : 0.f;
    constexpr int KS = DP / 16, KT = G::KT, SUB = KT / 16;
    constexpr int kWarps = G::kWarps, kAttnThreads = G::kThreads;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int32_t s_len[kLens];
    __shared__ int32_t s_scan[kWarps];
    __shared__ int32_t s_first[2];                                // first sequence of the block, units before it
    __shared__ PartMeta s_meta[2 * kWarps];
    __shared__ uint32_t s_joins;                                  // cut segments that this block joins

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    const awq_kv_cache &c = a.cache;
    const int D = c.head_dim;
    uint8_t *const ring = smem + warp * G::kStages * G::kStage;
    const uint32_t ring_addr = smem_u32(ring);
    uint8_t *const q_space = smem + kWarps * G::kStages * G::kStage + warp * 8 * G::kQPitch;
    // the workspace: two pieces per block, then the first part of every warp
    constexpr int kPiece = kAttnRows * G::kPitch;
    float *const block_parts = a.parts + (2 * kAttnMaxCtas + static_cast<int64_t>(blockIdx.x) * kWarps) * kPiece;

    // chunks past the head's end are never copied: they stay zero
    if (D != DP)
        for (int i = lane; i < G::kStages * G::kStage / 16; i += 32)
            reinterpret_cast<uint4 *>(ring)[i] = make_uint4(0, 0, 0, 0);

    BatchView view;
    view.seq_lens = a.seq_lens;
    view.s_len = s_len;
    view.b0 = 0;
    {
        const int64_t most = static_cast<int64_t>(a.max_pages) * c.page_size;
        view.max_len = most > 0x7fffffc0 ? 0x7fffffc0 : static_cast<int>(most);
    }
    view.per_seq = c.num_heads * a.row_tiles;

    grid_dependency_wait();
    grid_launch_dependents();

    // ---- total units, and the block's range
    const int per_thread = (a.batch + kAttnThreads - 1) / kAttnThreads;
    const int b_lo = tid * per_thread, b_hi = min(a.batch, b_lo + per_thread);
    int mine = 0;                        // units (the host has checked that they number below 2^31)
    for (int b = b_lo; b < b_hi; ++b) {
        const int raw = a.seq_lens[b], n = view.clamp(raw);
        if (n != raw && blockIdx.x == 0) set_status(a.status, AWQ_ERR_BAD_INDEX);
        if (b < kLens) s_len[b] = n;
        mine += (n + KT - 1) / KT;
    }
    mine *= view.per_seq;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_scan[warp] = incl;
    if (tid < 2 * kWarps) s_meta[tid].seg_begin = -1;
    __syncthreads();
    int total = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    // sequences without tokens: zeros, sequence b by block b mod the grid
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
        if (view.clamp(b < kLens ? s_len[b] : a.seq_lens[b]) > 0) continue;
        const int chunks = D / 8;
        for (int i = tid; i < a.q_heads * chunks; i += kAttnThreads) {
            const int h = i / chunks;
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.out.data) + b * a.out.token_stride + h * a.out.head_stride +
                                       8 * (i - h * chunks)) = make_uint4(0, 0, 0, 0);
        }
        if (a.lse)
            for (int h = tid; h < a.q_heads; h += kAttnThreads) a.lse[static_cast<int64_t>(b) * a.q_heads + h] = -INFINITY;
    }
    const int per_warp = (total - 1) / (static_cast<int>(gridDim.x) * kWarps) + 1;
    const int per = per_warp * kWarps;
    const int begin = min(total, static_cast<int>(min(static_cast<int64_t>(blockIdx.x) * per, static_cast<int64_t>(total))));
    const int block_end = total - begin < per ? total : begin + per;
    if (begin >= total) return;
    if (begin >= before && begin - before < mine) {
        int b = b_lo, at = before;
        for (; b < b_hi - 1; ++b) {
            const int u = (view.clamp(a.seq_lens[b]) + KT - 1) / KT * view.per_seq;
            if (begin - at < u) break;
            at += u;
        }
        s_first[0] = b;
        s_first[1] = at;
    }
    __syncthreads();
    Cursor<KT> seg;                      // the segment being computed
    seg.b = s_first[0];
    int local = begin - s_first[1] + warp * per_warp;
    if (a.batch > kLens) {
        view.b0 = seg.b;
        if (tid < kLens) s_len[tid] = view.b0 + tid < a.batch ? a.seq_lens[view.b0 + tid] : 0;
        __syncthreads();
    }
    seg.left = max(0, min(per_warp, block_end - begin - warp * per_warp));
    seg.n = view.len(seg.b);
    seg.s = seg.u = 0;
    if (seg.left > 0) {
        while (true) {
            const int u = seg.units() * view.per_seq;
            if (local < u) break;
            local -= u;
            ++seg.b;
            seg.n = view.len(seg.b);
        }
        seg.s = local / seg.units();
        seg.u = local - seg.s * seg.units();
    }

    // ---- the copies run ahead of the computation
    Cursor<KT> pre = seg;
    int pre_u = pre.u;                   // the next unit to copy
    int pre_end = pre.left > 0 ? pre.end() : 0;
    constexpr int kRowsPer = 32 / G::kChunks;        // rows of one copy instruction of the warp
    const int ch = lane % G::kChunks, sub_row = lane / G::kChunks;
    const bool in_row = ch * 16 < D * G::kElem;
    const uint32_t dst0 = ring_addr + G::at(sub_row, ch);
    const char *const k_data = static_cast<const char *>(c.k.data), *const v_data = static_cast<const char *>(c.v.data);
    int64_t k_head = 0, v_head = 0;      // bytes to the segment's KV head
    // Pages of whole multiples of 16 tokens (paged16): every 16 rows of a unit
    // are neighbours in one page, found by lane i for rows 16 i ..; else every
    // row is looked up, by lane i for row i (and i + 32).
    constexpr int TL = KT > 32 ? KT / 32 : 1;
    const bool paged16 = c.page_size % 16 == 0;
    int32_t pre_page[TL], pre_place[TL];

    // a segment's q rows, 16 bytes a lane: 8 heads of DP elements per tile
    uint4 q_raw[NT][DP / 32];
    auto load_q = [&]() {
        const int kv_head = a.row_tiles == 1 ? seg.s : seg.s / a.row_tiles, tile = seg.s - kv_head * a.row_tiles;
        const int rows_here = min(kAttnRows, a.group - tile * kAttnRows);
        const T *q = static_cast<const T *>(a.q.data) + seg.b * a.q.token_stride + (kv_head * a.group + tile * kAttnRows) * a.q.head_stride;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                const int r = 8 * nt + (32 * i + lane) / (DP / 8), d = 8 * ((32 * i + lane) % (DP / 8));
                q_raw[nt][i] = r < rows_here && d < D ? *reinterpret_cast<const uint4 *>(q + r * a.q.head_stride + d)
                                                      : make_uint4(0, 0, 0, 0);
            }
    };
    // ahead of the copies, behind which it would wait for all of them (where the
    // registers last that long)
    constexpr bool kEarlyQ = NT * DP <= 256;
    if (kEarlyQ && seg.left > 0) load_q();

    // the copies' new segment: its KV head, and its q rows into L1 for when the
    // computation gets there
    auto new_segment = [&]() {
        const int kv_head = a.row_tiles == 1 ? pre.s : pre.s / a.row_tiles, tile = pre.s - kv_head * a.row_tiles;
        k_head = kv_head * c.k.head_stride * G::kElem;
        v_head = kv_head * c.v.head_stride * G::kElem;
        const int rows_here = pre.left > 0 ? min(kAttnRows, a.group - tile * kAttnRows) : 0;
        const char *q = reinterpret_cast<const char *>(static_cast<const T *>(a.q.data) + pre.b * a.q.token_stride +
                                                       (kv_head * a.group + tile * kAttnRows) * a.q.head_stride);
        const int lines = (2 * D + 127) / 128;
        for (int i = lane; i < rows_here * lines; i += 32) {
            const int r = i / lines;
            uint32_t unused;
            asm volatile("ld.global.u32 %0, [%1];" : "=r"(unused) : "l"(q + r * a.q.head_stride * 2 + (i - r * lines) * 128));
        }
    };
    auto find = [&]() {
        if (pre.left > 0 && pre_u >= pre_end) {
            pre.next_segment(view);
            pre_u = pre.u;
            pre_end = pre.left > 0 ? pre.end() : 0;
            new_segment();
        }
        if (pre.left > 0) {
#pragma unroll
            for (int i = 0; i < TL; ++i) {
                const int row = paged16 ? 16 * (lane % SUB) : KT < 32 ? lane % KT : lane + 32 * i;
                const int tok = min(pre_u * KT + row, paged16 ? (pre.n - 1) & ~15 : pre.n - 1);
                const int page = a.page_shift ? static_cast<int>(__umulhi(tok, a.page_magic) >> (a.page_shift - 1)) : tok;
                pre_place[i] = tok - page * c.page_size;
                pre_page[i] = a.page_table[pre.b * a.table_stride + page];
            }
        }
    };
    const uint64_t policy = evict_first_policy();
    int put = 0;                         // ring slot of the next copy
    auto copy = [&]() {
        if (pre.left > 0) {
            const uint32_t dst = dst0 + put * G::kStage;
            const int rows = min(KT, pre.n - pre_u * KT);
            bool ok[TL];
            int64_t k_at[TL], v_at[TL];  // bytes from the plane's start
#pragma unroll
            for (int i = 0; i < TL; ++i) {
                ok[i] = pre_page[i] >= 0 && pre_page[i] < c.num_pages;
                if (!ok[i]) {            // nothing of this page is read
                    set_status(a.status, AWQ_ERR_BAD_INDEX);
                    pre_page[i] = 0;
                }
                k_at[i] = (pre_page[i] * c.k.page_stride + pre_place[i] * c.k.token_stride) * G::kElem + k_head;
                v_at[i] = k_at[i];
                if (!a.same_strides)
                    v_at[i] = (pre_page[i] * c.v.page_stride + pre_place[i] * c.v.token_stride) * G::kElem + v_head;
            }
            if (paged16) {
                const int64_t k_step = kRowsPer * c.k.token_stride * G::kElem, v_step = kRowsPer * c.v.token_stride * G::kElem;
#pragma unroll
                for (int sub = 0; sub < SUB; ++sub) {
                    const int good = __shfl_sync(~0u, static_cast<int>(ok[0]), sub);
                    const int64_t k0 = __shfl_sync(~0u, k_at[0], sub), v0 = a.same_strides ? k0 : __shfl_sync(~0u, v_at[0], sub);
                    const char *kp = k_data + k0 + sub_row * c.k.token_stride * G::kElem + ch * 16;
                    const char *vp = v_data + v0 + sub_row * c.v.token_stride * G::kElem + ch * 16;
                    const int have = good ? rows - 16 * sub - sub_row : 0;       // rows from this lane's first on
                    if (in_row) {
#pragma unroll
                        for (int i = 0; i < 16 / kRowsPer; ++i) {
                            const int r = 16 * sub + i * kRowsPer;               // + sub_row, which is below kRowsPer
                            const uint32_t at = (dst + r * G::kRow) ^ ((G::kRow >= 128 ? r & 7 : (r >> 1) & 3) << 4);
                            const uint32_t size = i * kRowsPer < have ? 16 : 0;
                            cp_async_16_zfill(at, kp, size, policy);
                            cp_async_16_zfill(at + G::kPlane, vp, size, policy);
                            kp += k_step;
                            vp += v_step;
                        }
                    }
                }
            } else {
#pragma unroll 4
                for (int i = 0; i < KT / kRowsPer; ++i) {
                    const int r = i * kRowsPer;
                    const int row = r + sub_row;
                    int64_t k0 = k_at[0], v0 = v_at[0];
                    int good = ok[0];
                    if (TL > 1 && r >= 32) {
                        k0 = k_at[TL - 1];
                        v0 = v_at[TL - 1];
                        good = ok[TL - 1];
                    }
                    k0 = __shfl_sync(~0u, k0, row % 32);
                    v0 = __shfl_sync(~0u, v0, row % 32);
                    good = __shfl_sync(~0u, good, row % 32);
                    const uint32_t at = (dst + r * G::kRow) ^ ((G::kRow >= 128 ? r & 7 : (r >> 1) & 3) << 4);
                    const uint32_t size = good && row < rows ? 16 : 0;
                    if (in_row) {
                        cp_async_16_zfill(at, k_data + k0 + ch * 16, size, policy);
                        cp_async_16_zfill(at + G::kPlane, v_data + v0 + ch * 16, size, policy);
                    }
                }
            }
            ++pre_u;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        put = put + 1 == G::kStages ? 0 : put + 1;
        find();
    };
    k_head = (a.row_tiles == 1 ? pre.s : pre.s / a.row_tiles) * c.k.head_stride * G::kElem;
    v_head = (a.row_tiles == 1 ? pre.s : pre.s / a.row_tiles) * c.v.head_stride * G::kElem;
    find();
#pragma unroll 1
    for (int i = 0; i < G::kStages - 1; ++i) copy();

    // element of the head that row `hi` (0: g, 1: g + 8) of output tile i is
    auto column = [&](int i, int hi) { return FP8 ? 16 * i + 2 * g + hi : 16 * i + g + 8 * hi; };

    // ldmatrix rows of this lane: 16 tokens x 2 chunks, tokens first for K and
    // for e4m3 V, chunks first for 16-bit V
    const uint32_t k_lane = ring_addr + G::at((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
    const uint32_t v_lane = ring_addr + G::kPlane + (FP8 ? G::at((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4)
                                                         : G::at((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1));
    int get = 0;                         // ring slot of the next unit
    int unit0 = begin + warp * per_warp;  // flat number of the segment's first unit of the warp
    while (seg.left > 0) {
        const int end = seg.end();
        const int kv_head = a.row_tiles == 1 ? seg.s : seg.s / a.row_tiles, tile = seg.s - kv_head * a.row_tiles;
        const int rows_here = min(kAttnRows, a.group - tile * kAttnRows);
        const int head0 = kv_head * a.group + tile * kAttnRows;

        // ---- Q fragments: head 8 nt + g; the heads of this lane's columns are 8 nt + 2 t4 + j
        uint32_t qf[NT][KS][2];
        float fac[NT][2];                // score to base-2 logarithm
        const uint32_t sign = a.scale < 0.f ? 0x80008000u : 0u;
        if (!kEarlyQ) load_q();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // 16 bytes a lane through shared memory: a fragment's own words would
            // be 4-byte loads from eight rows at a time
            __syncwarp();
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                const int at = 32 * i + lane;
                *reinterpret_cast<uint4 *>(q_space + at / (DP / 8) * G::kQPitch + 16 * (at % (DP / 8))) = q_raw[nt][i];
            }
            __syncwarp();
            if constexpr (FP8) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(q_space + g * G::kQPitch + ks * 32 + 8 * t4);
                    qf[nt][ks][0] = v.x ^ sign;
                    qf[nt][ks][1] = v.y ^ sign;
                }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ks += 2) {
                    uint32_t v[4];
                    ldmatrix_x4(v, smem_u32(q_space) + (lane & 7) * G::kQPitch + ks * 32 + (lane >> 3) * 16);
                    qf[nt][ks][0] = v[0] ^ sign;
                    qf[nt][ks][1] = v[1] ^ sign;
                    qf[nt][ks + 1][0] = v[2] ^ sign;
                    qf[nt][ks + 1][1] = v[3] ^ sign;
                }
            }
            float f = fabsf(a.scale) * c.k.scale * kLog2e;
            if constexpr (FP8 && !std::is_same<T, __half>::value) {
                float top = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 x = unpack2<T>(qf[nt][ks][i]);
                        top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
                    }
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                // 2^-e and 2^e of the head's largest element, e kept where both are normal
                const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 2), 252);
                const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                f *= __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 x = unpack2<T>(qf[nt][ks][i]);
                        qf[nt][ks][i] = pack2<C>(x.x * down, x.y * down);
                    }
            }
            f = fminf(fmaxf(f, kMinFactor), FLT_MAX);      // (finite: a score of 0 stays 0)
            fac[nt][0] = __shfl_sync(~0u, f, 8 * t4);
            fac[nt][1] = __shfl_sync(~0u, f, 8 * t4 + 4);
        }

        float o[KS][NT][4];
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.f;
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
        }

        for (int u = seg.u; u < end; ++u) {
            asm volatile("cp.async.wait_group %0;" ::"n"(G::kStages - 2) : "memory");
            __syncwarp();
            const uint32_t kst = k_lane + get * G::kStage, vst = v_lane + get * G::kStage;
            get = get + 1 == G::kStages ? 0 : get + 1;

            // ---- S' = K Q'
            float s[SUB][NT][4];
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub) {
                float x[2][NT][4] = {};          // two chains of products
#pragma unroll
                for (int ks = 0; ks < KS; ks += FP8 ? 2 : 1) {
                    if (ks * 16 < D) {
                        uint32_t k4[4];
                        ldmatrix_x4(k4, (kst + 16 * sub * G::kRow) ^ ((FP8 ? ks : 2 * ks) << 4));
                        if constexpr (FP8) {
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                uint32_t a0, a1, a2, a3;
                                e4m3x4_to_f16x4(k4[2 * j], a0, a2);
                                e4m3x4_to_f16x4(k4[2 * j + 1], a1, a3);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816<C>(x[j][nt], a0, a1, a2, a3, qf[nt][ks + j][0], qf[nt][ks + j][1]);
                            }
                        } else {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<C>(x[ks & 1][nt], k4[0], k4[1], k4[2], k4[3], qf[nt][ks][0], qf[nt][ks][1]);
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[sub][nt][j] = x[0][nt][j] + x[1][nt][j];
            }

            // ---- softmax over the unit
            const int left = seg.n - u * KT;
            if (left < KT) {
#pragma unroll
                for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (16 * sub + g + 8 * (j >> 1) >= left) s[sub][nt][j] = -INFINITY;
            }
            float top[NT][2];
            bool grew = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    top[nt][j] = -INFINITY;
#pragma unroll
                    for (int sub = 0; sub < SUB; ++sub)
                        top[nt][j] = fmaxf(top[nt][j], fmaxf(s[sub][nt][j], s[sub][nt][2 + j]));
                    top[nt][j] *= fac[nt][j];
                    grew |= top[nt][j] - (kLazy + kRaise) > m[nt][j];
                }
            if (__any_sync(~0u, grew)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float mn = fmaxf(m[nt][j], col_max(top[nt][j]) - kRaise);
                        const float corr = m[nt][j] == mn ? 1.f : fast_exp2(m[nt][j] - mn);
                        m[nt][j] = mn;
                        l[nt][j] *= corr;
#pragma unroll
                        for (int i = 0; i < KS; ++i) {
                            o[i][nt][j] *= corr;
                            o[i][nt][2 + j] *= corr;
                        }
                    }
            }
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub) {
                uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float base = m[nt][j & 1] == -INFINITY ? 0.f : m[nt][j & 1];
                        p[j] = fast_exp2(fmaf(s[sub][nt][j], fac[nt][j & 1], -base));
                        l[nt][j & 1] += p[j];
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        split2<C>(p[2 * h], p[2 * h + 1], ph[nt][h], pl[nt][h]);
                        ph[nt][h] = movmatrix_trans(ph[nt][h]);
                        pl[nt][h] = movmatrix_trans(pl[nt][h]);
                    }
                }
                // ---- O' += V' P'
                if constexpr (FP8) {
#pragma unroll
                    for (int i = 0; i < KS; i += 2) {
                        if (i * 16 < D) {
                            uint32_t v4[4];
                            ldmatrix_x4_trans(v4, (vst + 16 * sub * G::kRow) ^ (i << 4));
#pragma unroll
                            for (int j = 0; j < 2; ++j) {        // 16 elements: the even ones are rows 0-7, the odd ones 8-15
                                uint32_t a0, a1, a2, a3;
                                e4m3x4_to_f16x4(__byte_perm(v4[2 * j], 0, 0x3120), a0, a1);
                                e4m3x4_to_f16x4(__byte_perm(v4[2 * j + 1], 0, 0x3120), a2, a3);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    mma16816<C>(o[i + j][nt], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
                                    mma16816<C>(o[i + j][nt], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                                }
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        if (i * 16 < D) {
                            uint32_t v4[4];
                            ldmatrix_x4_trans(v4, (vst + 16 * sub * G::kRow) ^ (i << 5));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816<C>(o[i][nt], v4[0], v4[1], v4[2], v4[3], ph[nt][0], ph[nt][1]);
                                mma16816<C>(o[i][nt], v4[0], v4[1], v4[2], v4[3], pl[nt][0], pl[nt][1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();                               // every lane has read the slot that is filled next
            copy();
        }

#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) l[nt][j] = col_sum(l[nt][j]);
        const bool starts = seg.u == 0, ends = end == seg.units();
        if (starts && ends) {
            // ---- the warp has the whole segment: the output
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = 8 * nt + 2 * t4 + j;
                    if (r >= rows_here) continue;
                    const float inv = l[nt][j] > 0.f ? c.v.scale / l[nt][j] : l[nt][j];   // l is 0 (no weight) or NaN otherwise
                    T *out = static_cast<T *>(a.out.data) + seg.b * a.out.token_stride + (head0 + r) * a.out.head_stride;
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        if constexpr (FP8) {
                            if (column(i, 0) < D)
                                *reinterpret_cast<uint32_t *>(out + column(i, 0)) = pack2<T>(o[i][nt][j] * inv, o[i][nt][2 + j] * inv);
                        } else {
                            if (column(i, 0) < D) out[column(i, 0)] = from_f32<T>(o[i][nt][j] * inv);
                            if (column(i, 1) < D) out[column(i, 1)] = from_f32<T>(o[i][nt][2 + j] * inv);
                        }
                    }
                    if (a.lse && g == 0)
                        a.lse[static_cast<int64_t>(seg.b) * a.q_heads + head0 + r] = (m[nt][j] + __log2f(l[nt][j])) * kLn2;
                }
        } else {
            // ---- a part: the warp's first segment in the workspace, its last
            // one over the ring, whose units have all been used
            const bool last = seg.left == end - seg.u;
            float *buf = block_parts + warp * kPiece;
            if (last) {
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                buf = reinterpret_cast<float *>(ring);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float *row = buf + (8 * nt + 2 * t4 + j) * G::kPitch;
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        row[column(i, 0)] = o[i][nt][j];
                        row[column(i, 1)] = o[i][nt][2 + j];
                    }
                    if (g == 0) *reinterpret_cast<float2 *>(row + DP) = make_float2(m[nt][j], l[nt][j]);
                }
            if (lane == 0) s_meta[2 * warp + last] = PartMeta{unit0 - seg.u, seg.b, seg.s};
        }
        unit0 += end - seg.u;
        seg.next_segment(view);
        if (kEarlyQ && seg.left > 0) load_q();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    if (G::kPartsFit && s_meta[2 * warp].seg_begin >= 0) {
        // back from the workspace, beside the last part, while other warps still work
        const float *src = block_parts + warp * kPiece;
        float *dst = reinterpret_cast<float *>(ring) + 8 * NT * G::kPitch;
#pragma unroll 4
        for (int i = 4 * lane; i < 8 * NT * G::kPitch; i += 128)
            *reinterpret_cast<float4 *>(dst + i) = __ldcg(reinterpret_cast<const float4 *>(src + i));
    }
    __syncthreads();

    // ---- the warps' parts, in order; those of one segment are neighbours: a
    // group. Lane e of every warp looks at part e; the group's first lane, its
    // head, knows the rest of it.
    const PartMeta mt = s_meta[lane < 2 * kWarps ? lane : 0];
    const uint32_t valid = __ballot_sync(~0u, lane < 2 * kWarps && mt.seg_begin >= 0);
    const uint32_t below = valid & ((1u << lane) - 1);
    const int before_it = __shfl_sync(~0u, mt.seg_begin, below ? 31 - __clz(below) : lane);
    const bool head = ((valid >> lane) & 1) && (!below || before_it != mt.seg_begin);
    const uint32_t heads = __ballot_sync(~0u, head);
    int first = 0, last = 0;             // blocks of the head's segment
    bool cut = false;                    // it does not lie inside this block
    int head0 = 0, rows = 0;
    if (head) {
        const int kv_head = a.row_tiles == 1 ? mt.s : mt.s / a.row_tiles, tile = mt.s - kv_head * a.row_tiles;
        rows = min(kAttnRows, a.group - tile * kAttnRows);
        head0 = kv_head * a.group + tile * kAttnRows;
        first = mt.seg_begin / per;
        last = (mt.seg_begin + (view.len(mt.b) + KT - 1) / KT - 1) / per;
        cut = first != last;
    }
    const uint32_t cuts = __ballot_sync(~0u, cut);
    auto piece_of = [&](int seg_begin, int block) {              // slot 0: the segment that holds the block's first unit
        return a.parts + (2 * block + (seg_begin <= static_cast<int64_t>(block) * per ? 0 : 1)) * static_cast<int64_t>(kPiece);
    };

    // Pass 0 turns a group's parts into an output or the block's piece of a cut
    // segment, pass 1 the pieces of the cut segments that this block is the last
    // to leave into outputs. One loop for both: its instructions are fetched
    // once, and their first fetch is most of the time of a pass.
    uint32_t todo = heads;
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        int turn = 0;                    // the warp whose turn it is: the rows go round the warps, group after group
#pragma unroll 1
        for (; todo; todo &= todo - 1) {
            const int hl = __ffs(todo) - 1;
            const uint32_t after = heads & ~((2u << hl) - 1);
            const uint32_t mask = valid & ~((1u << hl) - 1) & (after ? (after & (0u - after)) - 1 : ~0u);
            const int seg_begin = __shfl_sync(~0u, mt.seg_begin, hl), b = __shfl_sync(~0u, mt.b, hl);
            const int h0 = __shfl_sync(~0u, head0, hl), nrows = __shfl_sync(~0u, rows, hl);
            const int from = __shfl_sync(~0u, first, hl), to = __shfl_sync(~0u, last, hl);
            const int n = pass ? to - from + 1 : 32 - __clz(mask) - hl;
#pragma unroll 1
            for (int r = turn <= warp ? warp - turn : warp - turn + kWarps; r < nrows; r += kWarps) {
                constexpr int kCols = (DP + 127) / 128;      // turns of 4 columns per lane
                float mx = -INFINITY, sum = 0.f;
                float4 v[kCols];
#pragma unroll
                for (int c4 = 0; c4 < kCols; ++c4) v[c4] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                for (int e0 = 0; e0 < n; e0 += G::kJoinRows) {
                    const int cnt = min(G::kJoinRows, n - e0), e = e0 + lane;
                    const float *row = reinterpret_cast<const float *>(ring) + lane * G::kPitch;
                    bool ok = lane < cnt;
                    if (pass) {
                        // the pieces' rows into the warp's ring, all in flight together
                        __syncwarp();
                        uint32_t dst = ring_addr + 16 * lane;
                        const float *next = a.parts + 2 * (from + e0) * static_cast<int64_t>(kPiece) + r * G::kPitch + 4 * lane;
                        const float *src = e0 ? next : piece_of(seg_begin, from) + r * G::kPitch + 4 * lane;
#pragma unroll 2
                        for (int k = 0; k < cnt; ++k, dst += 4 * G::kPitch, src = next) {
                            next += 2 * kPiece;      // every later block has its piece in slot 0
#pragma unroll
                            for (int c4 = 0; c4 < DP + 4; c4 += 128)
                                if (4 * lane + c4 < DP + 4)
                                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 4 * c4), "l"(src + c4)
                                                 : "memory");
                        }
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        __syncwarp();
                    } else {
                        // a warp's last part is in its ring, its first one beside it or in the workspace
                        ok = ok && ((mask >> (hl + e)) & 1);
                        const int w = (hl + e) >> 1;
                        row = reinterpret_cast<const float *>(smem + w * G::kStages * G::kStage);
                        if (!((hl + e) & 1)) row = G::kPartsFit ? row + 8 * NT * G::kPitch : block_parts + w * kPiece;
                        row += r * G::kPitch;
                    }
                    // a lane per row for the maximum, the weights and the sum, then one per 4 columns
                    const float2 ml = ok ? *reinterpret_cast<const float2 *>(row + DP) : make_float2(-INFINITY, 0.f);
                    const float top = fmaxf(mx, warp_max(ml.x)), base = top == -INFINITY ? 0.f : top;
                    const float weight = fast_exp2(ml.x - base), old = fast_exp2(mx - base);
                    mx = top;
                    sum = sum * old + warp_sum(weight * ml.y);
#pragma unroll
                    for (int c4 = 0; c4 < kCols; ++c4) v[c4] = make_float4(v[c4].x * old, v[c4].y * old, v[c4].z * old, v[c4].w * old);
                    // four rows at a time
                    const uint64_t row_addr = G::kPartsFit ? smem_u32(row) : reinterpret_cast<uint64_t>(row);
                    uint32_t rest = __ballot_sync(~0u, ok);
#pragma unroll 1
                    while (rest) {
                        float4 x[4][kCols];
                        float f[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const bool some = rest != 0;
                            const int from_lane = some ? __ffs(rest) - 1 : 0;
                            rest &= rest - 1;
                            f[k] = __shfl_sync(~0u, weight, from_lane);
                            // 32 bits of a shared address where no row is in the workspace
                            const uint64_t src =
                                (G::kPartsFit ? __shfl_sync(~0u, static_cast<uint32_t>(row_addr), from_lane)
                                              : __shfl_sync(~0u, row_addr, from_lane)) +
                                16 * lane;
#pragma unroll
                            for (int c4 = 0; c4 < kCols; ++c4) {
                                x[k][c4] = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (some && 4 * lane + 128 * c4 < DP)
                                    x[k][c4] = G::kPartsFit ? lds_f4(static_cast<uint32_t>(src) + 512 * c4)
                                                            : *reinterpret_cast<const float4 *>(src + 512 * c4);
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int c4 = 0; c4 < kCols; ++c4) {
                                v[c4].x += f[k] * x[k][c4].x;
                                v[c4].y += f[k] * x[k][c4].y;
                                v[c4].z += f[k] * x[k][c4].z;
                                v[c4].w += f[k] * x[k][c4].w;
                            }
                    }
                }
                if (pass || !((cuts >> hl) & 1)) {
                    const float inv = sum > 0.f ? c.v.scale / sum : sum;     // the sum is 0 (no weight) or NaN otherwise
                    T *const out = static_cast<T *>(a.out.data) + b * a.out.token_stride + (h0 + r) * a.out.head_stride;
#pragma unroll
                    for (int c4 = 0; c4 < kCols; ++c4)
                        if (const int d = 4 * lane + 128 * c4; d < D)
                            *reinterpret_cast<uint2 *>(out + d) =
                                make_uint2(pack2<T>(v[c4].x * inv, v[c4].y * inv), pack2<T>(v[c4].z * inv, v[c4].w * inv));
                    if (a.lse && lane == 0) a.lse[static_cast<int64_t>(b) * a.q_heads + h0 + r] = (mx + __log2f(sum)) * kLn2;
                } else {
                    float *const piece = piece_of(seg_begin, blockIdx.x) + r * G::kPitch;
#pragma unroll
                    for (int c4 = 0; c4 < kCols; ++c4)
                        if (const int d = 4 * lane + 128 * c4; d < D) *reinterpret_cast<float4 *>(piece + d) = v[c4];
                    if (lane == 0) *reinterpret_cast<float2 *>(piece + DP) = make_float2(mx, sum);
                }
            }
            turn = (turn + nrows) % kWarps;
        }
        if (pass || !cuts) break;
        __syncthreads();
        if (warp == 0) {
            bool joins = false;
            if (cut) {
                // orders the block's pieces (through the barrier) before the
                // count, and the others' before what follows it
                joins = atom_add_acq_rel(a.counters + first, 1) == last - first;
                if (joins) a.counters[first] = 0;
            }
            const uint32_t which = __ballot_sync(~0u, joins);
            if (lane == 0) s_joins = which;
        }
        __syncthreads();
        todo = s_joins;
    }
}

template <typename T, bool FP8, int DP, int NT>
awq_status launch_attn_g(const AttnArgs &a, int sms, cudaStream_t st)
{
    using G = Geo<FP8, DP, NT>;
    const awq_status r = set_smem(attn_kernel<T, FP8, DP, NT>, G::kSmem);
    if (r) return r;
    return launch(attn_kernel<T, FP8, DP, NT>, dim3(std::min(sms, kAttnMaxCtas)), dim3(G::kThreads), G::kSmem,
                  1, st, a);
}

template <typename T, bool FP8, int DP>
awq_status launch_attn_dp(const AttnArgs &a, int sms, cudaStream_t st)
{
    return a.group <= 8 ? launch_attn_g<T, FP8, DP, 1>(a, sms, st) : launch_attn_g<T, FP8, DP, 2>(a, sms, st);
}

template <typename T, bool FP8>
awq_status launch_attn_t(const AttnArgs &a, int sms, cudaStream_t st)
{
    switch (attn_padded_dim(a.cache.head_dim)) {
    case 64: return launch_attn_dp<T, FP8, 64>(a, sms, st);
    case 128: return launch_attn_dp<T, FP8, 128>(a, sms, st);
    default: return launch_attn_dp<T, FP8, 256>(a, sms, st);
    }
}

}  // namespace

awq_status launch_attention(const AttnArgs &a, int dtype, int sms, cudaStream_t st)
{
    const bool fp8 = a.cache.dtype == AWQ_DTYPE_E4M3;
    if (dtype == AWQ_DTYPE_F16) return fp8 ? launch_attn_t<__half, true>(a, sms, st) : launch_attn_t<__half, false>(a, sms, st);
    return fp8 ? launch_attn_t<__nv_bfloat16, true>(a, sms, st) : launch_attn_t<__nv_bfloat16, false>(a, sms, st);
}

}  // namespace awq
