// awq_paged_attention: one new token per sequence over the paged cache.
//
// Work is counted in units of 16 cached tokens of one (sequence, KV head, tile
// of query heads), a segment, numbered segment by segment; block c of G takes
// units [c * per, (c + 1) * per), whatever segments they belong to, so every
// block reads the same number of cache bytes however ragged the batch is. A
// segment that lies inside one block is finished there; one that is cut leaves
// a piece (running maximum, sum, unnormalised output, all fp32) per block in
// the workspace, and the block that finishes last joins the pieces in block
// order, so the result does not depend on which one that is.
//
// Within a block each warp works alone: units go to the warps round-robin,
// each warp copies its unit's 16 K and 16 V rows (cp.async, 16 bytes a lane,
// STAGES units deep, running on into the next segment) and keeps its own
// maximum, sum and output; the warps' results are merged per segment.
//
// Per unit and warp, with up to 16 query heads as the rows of the tensor-core
// tile (mma.m16n8k16, fp32 accumulators):
//   S[16 x 16]  = Q K^T, K rows read with ldmatrix as the B operand
//   m' = max(m, rowmax S), P = exp2(S - m'), l = l * 2^(m - m') + sum P
//   O[16 x D]   = O * 2^(m - m') + P V, V rows read with ldmatrix.trans
// S is scaled to base-2 logarithms in fp32. P enters the tensor core as two
// 16-bit terms, P = hi + lo, so its rounding does not reach the output: with
// at most 8 query heads the lo terms are rows 8-15 of the same tile (free),
// else they are a second product.
//
// e4m3 planes are expanded to fp16 in registers (exact): a 4-byte lane of an
// ldmatrix row holds 4 neighbouring elements of the head, so Q's elements are
// dealt to the fragments in the same order (the dot product does not care),
// and V's columns come out in an order that the output's store undoes. bf16 Q
// becomes fp16 with its row's power of two taken out (exact to 2^-24 of the
// row's largest element).
//
// Bound: 4 * group operations per cached element of 1 or 2 bytes, so the
// bytes decide; mma.sync at 16 rows has a few times the rate that they need.
#include <algorithm>
#include <type_traits>

#include "awq_decoder_kernels.cuh"
#include "awq_launch.cuh"

namespace awq {

namespace {

constexpr int kUnit = 16;              // cached tokens of a unit
constexpr int kWarps = 4;
constexpr int kAttnThreads = kWarps * 32;
constexpr int kLens = 128;             // sequence lengths kept in shared memory
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
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

// Two e4m3 codes as an fp16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
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

__device__ __forceinline__ float quad_max(float v)
{
    v = fmaxf(v, __shfl_xor_sync(~0u, v, 1));
    return fmaxf(v, __shfl_xor_sync(~0u, v, 2));
}
__device__ __forceinline__ float quad_sum(float v)
{
    v += __shfl_xor_sync(~0u, v, 1);
    return v + __shfl_xor_sync(~0u, v, 2);
}

struct BatchView {
    const int32_t *seq_lens;
    const int32_t *s_len;     // lengths of sequences b0 .. b0 + kLens - 1
    int b0, batch, max_len;
    int per_seq;              // segments of a sequence: KV heads x head tiles

    __device__ __forceinline__ int len(int b) const
    {
        const int i = b - b0;
        const int n = i < kLens ? s_len[i] : seq_lens[b];
        return n < 0 ? 0 : n > max_len ? max_len : n;
    }
};

// A position in the flat order of units: segment (b, s) of n tokens, unit u.
struct Cursor {
    int b, s, n, u;
    int64_t left;             // units from u to the end of the block's range

    __device__ __forceinline__ int units() const { return (n + kUnit - 1) / kUnit; }
    // the segment's units that belong to the block: [u, end())
    __device__ __forceinline__ int end() const
    {
        const int e = units();
        return left < e - u ? u + static_cast<int>(left) : e;
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

template <bool FP8, int DP, bool GS8>
struct Geo {
    static constexpr int kElem = FP8 ? 1 : 2;
    static constexpr int kRow = DP * kElem;             // bytes of a token's row in shared memory
    static constexpr int kChunks = kRow / 16;
    static constexpr int kPlane = kUnit * kRow;
    static constexpr int kStage = 2 * kPlane;           // K rows, then V rows
    static constexpr int kRows = GS8 ? 8 : 16;          // query heads of a tile
    static constexpr int kBlocks = kStage >= 16384 ? 1 : 2;      // resident per multiprocessor
    static constexpr int kMergeRow = DP + 2;            // output, maximum, sum
    static constexpr int kMerge = 2 * kRows * kMergeRow * 4;
    // as many units in flight as a block's share of shared memory holds
    static constexpr int kShare = (kBlocks == 1 ? 227 : 112) * 1024 + (kBlocks == 1 ? 0 : 640);
    static constexpr int kFit = (kShare - kMerge) / (kWarps * kStage);
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kSmem = kWarps * kStages * kStage + kMerge;
    static_assert(kStages >= 2, "a unit in flight beside the one in use");

    // 16-byte chunk c of row r, placed so that 8 rows of one chunk fall into
    // different banks
    static __device__ __forceinline__ uint32_t at(int r, int c)
    {
        const int sw = kRow >= 128 ? (r & 7) : ((r >> 1) & 3);
        return static_cast<uint32_t>(r * kRow + ((c ^ sw) << 4));
    }
};

template <typename T, bool FP8, int DP, bool GS8>
__global__ void __launch_bounds__(kAttnThreads, Geo<FP8, DP, GS8>::kBlocks) attn_kernel(const AttnArgs a)
{
    using G = Geo<FP8, DP, GS8>;
    using C = typename std::conditional<FP8, __half, T>::type;   // the tensor core's type
    constexpr int KS = DP / 16;                                   // 16-element steps of a head
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int32_t s_len[kLens];
    __shared__ int64_t s_scan[kWarps + 1];
    __shared__ int64_t s_first[2];                                // first sequence of the block, units before it
    __shared__ int32_t s_ticket;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    const awq_kv_cache &c = a.cache;
    const int D = c.head_dim;
    float *const merge = reinterpret_cast<float *>(smem + kWarps * G::kStages * G::kStage);
    uint8_t *const ring = smem + warp * G::kStages * G::kStage;
    const uint32_t ring_addr = smem_u32(ring);

    // chunks past the head's end are never copied: they stay zero
    for (int i = lane; i < G::kStages * G::kStage / 16; i += 32)
        reinterpret_cast<uint4 *>(ring)[i] = make_uint4(0, 0, 0, 0);

    BatchView view;
    view.seq_lens = a.seq_lens;
    view.s_len = s_len;
    view.batch = a.batch;
    {
        const int64_t most = static_cast<int64_t>(a.max_pages) * c.page_size;
        view.max_len = most > 0x7fffffe0 ? 0x7fffffe0 : static_cast<int>(most);
    }
    view.per_seq = c.num_heads * a.row_tiles;

    grid_dependency_wait();
    grid_launch_dependents();

    // ---- total units, and the block's range
    const int per_thread = (a.batch + kAttnThreads - 1) / kAttnThreads;
    const int b_lo = tid * per_thread, b_hi = min(a.batch, b_lo + per_thread);
    int64_t mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        int n = a.seq_lens[b];
        if (n < 0 || n > view.max_len) {
            if (blockIdx.x == 0) set_status(a.status, AWQ_ERR_BAD_INDEX);
            n = n < 0 ? 0 : view.max_len;
        }
        mine += (n + kUnit - 1) / kUnit;
        // a sequence without tokens: zeros, spread over the blocks
        if (n == 0 && b % gridDim.x == blockIdx.x) {
            for (int h = 0; h < a.q_heads; ++h) {
                T *o = static_cast<T *>(a.out.data) + b * a.out.token_stride + h * a.out.head_stride;
                for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4 *>(o + d) = make_uint4(0, 0, 0, 0);
                if (a.lse) a.lse[static_cast<int64_t>(b) * a.q_heads + h] = -INFINITY;
            }
        }
    }
    mine *= view.per_seq;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int64_t total = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    // at least a unit per warp, and whole rounds of the warps
    int64_t per = (total + gridDim.x - 1) / gridDim.x;
    per = (per + kWarps - 1) / kWarps * kWarps;
    const int64_t begin = blockIdx.x * per;
    if (begin >= total) return;
    if (begin >= before && begin < before + mine) {
        int b = b_lo;
        int64_t at = before;
        while (true) {
            int n = a.seq_lens[b];
            n = n < 0 ? 0 : n > view.max_len ? view.max_len : n;
            const int64_t u = static_cast<int64_t>((n + kUnit - 1) / kUnit) * view.per_seq;
            if (begin < at + u) break;
            at += u;
            ++b;
        }
        s_first[0] = b;
        s_first[1] = at;
    }
    __syncthreads();
    view.b0 = static_cast<int>(s_first[0]);
    for (int i = tid; i < kLens; i += kAttnThreads) s_len[i] = view.b0 + i < a.batch ? a.seq_lens[view.b0 + i] : 0;
    __syncthreads();

    Cursor seg;                          // the segment being computed
    seg.b = view.b0;
    seg.n = view.len(seg.b);
    {
        const int64_t local = begin - s_first[1];
        seg.s = static_cast<int>(local / seg.units());
        seg.u = static_cast<int>(local - static_cast<int64_t>(seg.s) * seg.units());
        seg.left = min(per, total - begin);
    }

    // ---- the copies run ahead of the computation
    Cursor pre = seg;                    // u: the segment's first unit of the block
    int pre_u = pre.u + warp;            // the warp's next unit to copy
    int pre_end = pre.end();
    int32_t pre_page = 0;                // page of this lane's token of that unit
    const bool lane_v = lane >= 16;
    const int lane_tok = lane & 15;
    const awq_kv_plane &plane = lane_v ? c.v : c.k;

    auto find = [&]() {                  // skip segments without units for this warp
        while (pre.left > 0 && pre_u >= pre_end) {
            pre.next_segment(view);
            pre_u = pre.u + warp;
            pre_end = pre.left > 0 ? pre.end() : 0;
        }
        if (pre.left > 0) {
            const int tok = min(pre_u * kUnit + lane_tok, pre.n - 1);
            pre_page = __ldg(a.page_table + pre.b * a.table_stride + tok / c.page_size);
        }
    };
    int put = 0;                         // ring slot of the next copy
    auto copy = [&]() {
        if (pre.left > 0) {
            const int tok = pre_u * kUnit + lane_tok;
            const bool in_seq = tok < pre.n;
            const bool ok = pre_page >= 0 && pre_page < c.num_pages;
            if (in_seq && !ok) set_status(a.status, AWQ_ERR_BAD_INDEX);
            const int place = tok % c.page_size;
            const int head = pre.s / a.row_tiles;
            const char *src = static_cast<const char *>(plane.data);
            if (in_seq && ok)
                src += (pre_page * plane.page_stride + place * plane.token_stride + head * plane.head_stride) * G::kElem;
            const uint32_t bytes = in_seq && ok ? 16u : 0u;
            const uint32_t dst = ring_addr + put * G::kStage;
            const uint64_t packed = reinterpret_cast<uint64_t>(src);
#pragma unroll
            for (int i = 0; i < 2 * kUnit * G::kChunks / 32; ++i) {
                const int idx = i * 32 + lane;
                const int row = idx / G::kChunks, ch = idx % G::kChunks;   // rows 16-31: V
                const uint64_t base = __shfl_sync(~0u, packed, row);
                const uint32_t size = __shfl_sync(~0u, bytes, row);
                if (ch * 16 < D * G::kElem)
                    cp_async_16_zfill(dst + (row >= kUnit ? G::kPlane : 0) + G::at(row & 15, ch),
                                      reinterpret_cast<const char *>(base) + (size ? ch * 16 : 0), size);
            }
            pre_u += kWarps;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        put = put + 1 == G::kStages ? 0 : put + 1;
        find();
    };
    find();
#pragma unroll
    for (int i = 0; i < G::kStages - 1; ++i) copy();

    int get = 0;                         // ring slot of the next unit
    int64_t unit0 = begin;               // flat number of the segment's first unit of the block
    while (seg.left > 0) {
        const int end = seg.end();
        const int kv_head = seg.s / a.row_tiles, tile = seg.s % a.row_tiles;
        const int rows_here = min(kAttnRows, a.group - tile * kAttnRows);
        const int head0 = kv_head * a.group + tile * kAttnRows;
        const int rg[2] = {g, g + 8};

        // ---- Q fragments: rows g and g + 8
        uint32_t qf[KS][4];
        float fac[2];                    // score to base-2 logarithm
        const T *qb = static_cast<const T *>(a.q.data) + seg.b * a.q.token_stride;
#pragma unroll
        for (int r = 0; r < (GS8 ? 1 : 2); ++r) {
            const bool ok = rg[r] < rows_here;
            const T *q = qb + (head0 + (ok ? rg[r] : 0)) * a.q.head_stride;
            uint32_t raw[KS][2];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int d0 = ks * 16 + (FP8 ? 4 * t4 : 2 * t4), d1 = ks * 16 + (FP8 ? 4 * t4 + 2 : 2 * t4 + 8);
                raw[ks][0] = ok && d0 < D ? *reinterpret_cast<const uint32_t *>(q + d0) : 0u;
                raw[ks][1] = ok && d1 < D ? *reinterpret_cast<const uint32_t *>(q + d1) : 0u;
            }
            fac[r] = a.scale * c.k.scale * kLog2e;
            if constexpr (FP8 && !std::is_same<T, __half>::value) {
                float top = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 x = unpack2<T>(raw[ks][i]);
                        top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
                    }
                top = quad_max(top);
                // 2^-e and 2^e of the row's largest element, e kept where both are normal
                const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 2), 252);
                const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                fac[r] *= __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 x = unpack2<T>(raw[ks][i]);
                        raw[ks][i] = pack2<C>(x.x * down, x.y * down);
                    }
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                qf[ks][r] = raw[ks][0];
                qf[ks][2 + r] = raw[ks][1];
            }
        }
        if constexpr (GS8) {
            fac[1] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) qf[ks][1] = qf[ks][3] = 0u;
        }

        float o[DP / 8][4];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (int u = seg.u + warp; u < end; u += kWarps) {
            asm volatile("cp.async.wait_group %0;" ::"n"(G::kStages - 2) : "memory");
            __syncwarp();
            const uint32_t kst = ring_addr + get * G::kStage, vst = kst + G::kPlane;
            get = get + 1 == G::kStages ? 0 : get + 1;

            // ---- S = Q K^T
            float s[2][4] = {};
            if constexpr (FP8) {
#pragma unroll
                for (int ks = 0; ks < KS; ks += 2) {
                    uint32_t k4[4];
                    if (ks * 16 < D) {
                        ldmatrix_x4(k4, kst + G::at((lane & 7) + ((lane >> 3) & 1) * 8, ks + (lane >> 4)));
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int n = 0; n < 2; ++n)
                                mma16816<C>(s[n], qf[ks + j][0], qf[ks + j][1], qf[ks + j][2], qf[ks + j][3],
                                            e4m3x2_to_f16x2(k4[2 * j + n]), e4m3x2_to_f16x2(k4[2 * j + n] >> 16));
                    }
                }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t k4[4];
                    if (ks * 16 < D) {
                        ldmatrix_x4(k4, kst + G::at((lane & 7) + (lane >> 4) * 8, 2 * ks + ((lane >> 3) & 1)));
                        mma16816<C>(s[0], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], k4[0], k4[1]);
                        mma16816<C>(s[1], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], k4[2], k4[3]);
                    }
                }
            }

            // ---- softmax over the unit
            const int left = seg.n - u * kUnit;          // tokens of the unit that exist, if below 16
            constexpr int R = GS8 ? 1 : 2;
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float &x = s[n][2 * r + j];
                        x *= fac[r];
                        if (8 * n + 2 * t4 + j >= left) x = -INFINITY;
                        top[r] = fmaxf(top[r], x);
                    }
                top[r] = quad_max(top[r]);
            }
            bool grew = false;
#pragma unroll
            for (int r = 0; r < R; ++r) grew |= top[r] > m[r];
            if (__any_sync(~0u, grew)) {
                float corr[2] = {1.f, 1.f};
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float mn = fmaxf(m[r], top[r]);
                    corr[r] = m[r] == mn ? 1.f : fast_exp2(m[r] - mn);
                    m[r] = mn;
                    l[r] *= corr[r];
                }
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) {
                    o[i][0] *= corr[0];
                    o[i][1] *= corr[0];
                    o[i][2] *= GS8 ? corr[0] : corr[1];
                    o[i][3] *= GS8 ? corr[0] : corr[1];
                }
            }
            uint32_t p[4], pl[4];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float base = m[r] == -INFINITY ? 0.f : m[r];
                float e[4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        e[2 * n + j] = fast_exp2(s[n][2 * r + j] - base);
                        l[r] += e[2 * n + j];
                    }
                split2<C>(e[0], e[1], p[r], pl[r]);
                split2<C>(e[2], e[3], p[2 + r], pl[2 + r]);
            }
            if constexpr (GS8) {                        // rows 8-15: the lo terms
                p[1] = pl[0];
                p[3] = pl[2];
            }

            // ---- O += P V
#pragma unroll
            for (int ks = 0; ks < (FP8 ? KS / 2 : KS); ++ks) {
                uint32_t v4[4];
                if (ks * (FP8 ? 32 : 16) < D) {
                    ldmatrix_x4_trans(v4, vst + G::at((lane & 7) + ((lane >> 3) & 1) * 8, 2 * ks + (lane >> 4)));
                    if constexpr (FP8) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {   // 16 columns: the even ones, the odd ones
                            const uint32_t x = __byte_perm(v4[2 * j], 0, 0x3120), y = __byte_perm(v4[2 * j + 1], 0, 0x3120);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t b0 = e4m3x2_to_f16x2(h ? x >> 16 : x), b1 = e4m3x2_to_f16x2(h ? y >> 16 : y);
                                float (&acc)[4] = o[4 * ks + 2 * j + h];
                                mma16816<C>(acc, p[0], p[1], p[2], p[3], b0, b1);
                                if constexpr (!GS8) mma16816<C>(acc, pl[0], pl[1], pl[2], pl[3], b0, b1);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            mma16816<C>(o[2 * ks + j], p[0], p[1], p[2], p[3], v4[2 * j], v4[2 * j + 1]);
                            if constexpr (!GS8) mma16816<C>(o[2 * ks + j], pl[0], pl[1], pl[2], pl[3], v4[2 * j], v4[2 * j + 1]);
                        }
                    }
                }
            }
            __syncwarp();                               // every lane has read the slot that is filled next
            copy();
        }

        // ---- the warps' results become one (in warp 0)
        constexpr int R = GS8 ? 1 : 2;
        if constexpr (GS8) {
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) {
                o[i][0] += o[i][2];
                o[i][1] += o[i][3];
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = quad_sum(l[r]);
#pragma unroll
        for (int step = kWarps / 2; step > 0; step >>= 1) {
            __syncthreads();
            if (warp >= step && warp < 2 * step) {
                float *buf = merge + (warp - step) * G::kRows * G::kMergeRow;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float *row = buf + rg[r] * G::kMergeRow;
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i)
                        *reinterpret_cast<float2 *>(row + 8 * i + 2 * t4) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
                    if (t4 == 0) {
                        row[DP] = m[r];
                        row[DP + 1] = l[r];
                    }
                }
            }
            __syncthreads();
            if (warp < step) {
                const float *buf = merge + warp * G::kRows * G::kMergeRow;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float *row = buf + rg[r] * G::kMergeRow;
                    const float m2 = row[DP], mn = fmaxf(m[r], m2);
                    const float w1 = m[r] == -INFINITY ? 0.f : fast_exp2(m[r] - mn);
                    const float w2 = m2 == -INFINITY ? 0.f : fast_exp2(m2 - mn);
                    m[r] = mn;
                    l[r] = l[r] * w1 + row[DP + 1] * w2;
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i) {
                        const float2 x = *reinterpret_cast<const float2 *>(row + 8 * i + 2 * t4);
                        o[i][2 * r] = o[i][2 * r] * w1 + x.x * w2;
                        o[i][2 * r + 1] = o[i][2 * r + 1] * w1 + x.y * w2;
                    }
                }
            }
        }

        // ---- whole segment: the output; else a piece
        // element of the head that o[i][2r + j] is
        auto column = [&](int i, int j) {
            return FP8 ? (i >> 1) * 16 + 4 * t4 + 2 * j + (i & 1) : 8 * i + 2 * t4 + j;
        };
        const bool whole = seg.u == 0 && end == seg.units();
        if (whole) {
            if (warp == 0) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (rg[r] >= rows_here) continue;
                    const int h = head0 + rg[r];
                    const float inv = l[r] > 0.f ? c.v.scale / l[r] : l[r];       // l is 0 (no output) or NaN otherwise
                    T *out = static_cast<T *>(a.out.data) + seg.b * a.out.token_stride + h * a.out.head_stride;
                    if constexpr (FP8) {
#pragma unroll
                        for (int i = 0; i < DP / 8; i += 2) {
                            const int d = column(i, 0);                            // four neighbours: d .. d + 3
                            if (d < D)
                                *reinterpret_cast<uint2 *>(out + d) =
                                    make_uint2(pack2<T>(o[i][2 * r] * inv, o[i + 1][2 * r] * inv),
                                               pack2<T>(o[i][2 * r + 1] * inv, o[i + 1][2 * r + 1] * inv));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < DP / 8; ++i) {
                            const int d = column(i, 0);
                            if (d < D)
                                *reinterpret_cast<uint32_t *>(out + d) = pack2<T>(o[i][2 * r] * inv, o[i][2 * r + 1] * inv);
                        }
                    }
                    if (a.lse && t4 == 0)
                        a.lse[static_cast<int64_t>(seg.b) * a.q_heads + h] = (m[r] + log2f(l[r])) * kLn2;
                }
            }
        } else {
            // blocks of the segment, and this one's piece (a block's first
            // segment has its slot 0, a later one slot 1)
            const int64_t seg_begin = unit0 - seg.u, seg_end = seg_begin + seg.units();
            const int first = static_cast<int>(seg_begin / per), last = static_cast<int>((seg_end - 1) / per);
            constexpr int kPiece = kAttnRows * G::kMergeRow;
            float *piece = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + (unit0 == begin ? 0 : 1)) * kPiece;
            if (warp == 0) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (rg[r] >= rows_here) continue;
                    float *row = piece + rg[r] * G::kMergeRow;
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) row[column(i, j)] = o[i][2 * r + j];
                    if (t4 == 0) {
                        row[DP] = m[r];
                        row[DP + 1] = l[r];
                    }
                }
                __threadfence();
                __syncwarp();
                if (lane == 0) s_ticket = atomicAdd(a.counters + first, 1);
            }
            __syncthreads();
            if (s_ticket == last - first) {
                __threadfence();
                if (tid == 0) a.counters[first] = 0;
                const float *first_piece =
                    a.parts + (2 * static_cast<int64_t>(first) + (seg_begin == first * per ? 0 : 1)) * kPiece;
                const int cols = D / 2;
                for (int i = tid; i < rows_here * cols; i += kAttnThreads) {
                    const int r = i / cols, d = 2 * (i - r * cols);
                    const int64_t at = static_cast<int64_t>(r) * G::kMergeRow;
                    float mx = __ldcg(first_piece + at + DP);
                    for (int p = first + 1; p <= last; ++p)
                        mx = fmaxf(mx, __ldcg(a.parts + 2 * static_cast<int64_t>(p) * kPiece + at + DP));
                    const float base = mx == -INFINITY ? 0.f : mx;
                    float sum = 0.f, x = 0.f, y = 0.f;
                    for (int p = first; p <= last; ++p) {
                        const float *src = (p == first ? first_piece : a.parts + 2 * static_cast<int64_t>(p) * kPiece) + at;
                        const float w = fast_exp2(__ldcg(src + DP) - base);
                        const float2 v = __ldcg(reinterpret_cast<const float2 *>(src + d));
                        sum += w * __ldcg(src + DP + 1);
                        x += w * v.x;
                        y += w * v.y;
                    }
                    const float inv = sum > 0.f ? c.v.scale / sum : sum;
                    const int h = head0 + r;
                    *reinterpret_cast<uint32_t *>(static_cast<T *>(a.out.data) + seg.b * a.out.token_stride +
                                                  h * a.out.head_stride + d) = pack2<T>(x * inv, y * inv);
                    if (a.lse && d == 0) a.lse[static_cast<int64_t>(seg.b) * a.q_heads + h] = (mx + log2f(sum)) * kLn2;
                }
            }
        }
        unit0 += end - seg.u;
        seg.next_segment(view);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, bool FP8, int DP, bool GS8>
awq_status launch_attn_g(const AttnArgs &a, int sms, cudaStream_t st)
{
    using G = Geo<FP8, DP, GS8>;
    const awq_status r = set_smem(attn_kernel<T, FP8, DP, GS8>, G::kSmem);
    if (r) return r;
    return launch(attn_kernel<T, FP8, DP, GS8>, dim3(std::min(sms * G::kBlocks, kAttnMaxCtas)), dim3(kAttnThreads), G::kSmem,
                  1, st, a);
}

template <typename T, bool FP8, int DP>
awq_status launch_attn_dp(const AttnArgs &a, int sms, cudaStream_t st)
{
    return a.group <= 8 ? launch_attn_g<T, FP8, DP, true>(a, sms, st) : launch_attn_g<T, FP8, DP, false>(a, sms, st);
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
