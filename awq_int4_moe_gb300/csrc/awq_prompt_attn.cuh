// awq_prompt_attention and awq_chunk_attention: causal attention of n new
// tokens per sequence, over K and V packed like q or in the paged cache, on the
// 5th-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// Rows. The G query heads of a KV head see the same keys, so a sequence's rows
// are its (token, head of the group) pairs, token by token: row r is token r / G,
// head r % G, and sees the keys before limit(r) = L - n + r / G + 1. A unit is
// 256 consecutive rows of one sequence and KV head (128 where a head is larger
// than 128): no row of a tile is padding but at a sequence's end, a key is
// copied once for all heads that read it, and the diagonal cuts few tiles.
//
// One pass over the keys, 128 at a time (base-2 logarithms, all fp32):
//   S = Q K'                                    tensor core, into tensor memory
//   m' = max(m, S f), P = exp2(S f - m'), l = l 2^(m - m') + sum P      registers
//   O = O 2^(m - m') + P V                      tensor core, P from tensor memory
// m is raised only where a score passes it by more than 2^8, so that O is scaled
// (a round trip through registers) for the first tiles of a row and then hardly
// ever; P stays below 2^8 times the maximum's own weight.
//
// Steps. Two score tiles are in flight, one per softmax warpgroup ("slot"): while
// one is turned into weights, the tensor core works for the other.
//   wide (more than 128 rows): slot w has rows 128 w .. of every key tile;
//   narrow (up to 128 rows, few new tokens over a long context): both have the
//     same rows and every other key tile; their outputs are joined in tensor
//     memory at the end;
//   heads larger than 128: one warpgroup, its score tile double-buffered.
// Tensor memory: S (and P over it, 16 bits) 2 x 128 columns, O 2 x 128 or 256.
//
// Warps: 0-7 softmax and output, a thread per row (nothing crosses lanes in a
// step); 8 and 9 issue the MMAs of a slot each; the rest load (and make V finite where
// rows are masked). Units are found one
// ahead of their use, by warp 9, or over e4m3 by warp 11. All meet at mbarriers, every
// wait is bounded (2^18 tries within a block, a time for other blocks). Registers go
// where the scores are (208 or 200 a thread there): with 227 KB
// of shared memory in use what spills comes back from L2.
//
// Copies are TMA boxes into 128-byte swizzled stages of 128 keys x 128 columns: of K
// and V as many keys as the largest power of two up to 128 that divides the page (any page
// size and stride will do), of Q whole tokens, for which a unit has a whole number
// of them. Where Q cannot come so (more than 256 heads of one, or fewer bits than
// it has) threads copy it. e4m3 tiles come as codes and are expanded to fp16 in
// shared memory by four warps: kind::f8f6f4 would want the weights and q in 8 bits.
//
// Balance. Units are numbered sequence by sequence, head by head, tile by tile;
// their costs (a unit's keys and a fixed part) have a closed form, and every
// block takes an equal share of the sum, whatever units it belongs to. A unit
// that is cut (between pairs of key tiles, not within kPiece of its ends) leaves its parts in the
// workspace; at the end the blocks that share it wait for the last one and each
// join a part of its rows, in block order, so the same inputs give the same bits.
//
// Bound. Wide units over 16-bit keys: per key tile and slot 4 x 2 x 128^3 / 8192
// = 2048 cycles of the tensor core for both slots against some 2750 measured: the
// chain scores, maximum, exponentials (128 a thread, 4 cycles a warp's
// instruction) and product of a slot is not quite hidden by the other's. Then a unit's
// turnaround (its last product, the stores, the next one's Q: 9000 cycles). Narrow
// units: the bytes of K and V (87 % of the copy bandwidth); over e4m3 the warps that copy
// and expand (some 1200 cycles a tile each), beside softmax warps that take rows of
// padding too. Small calls: launch, scan, and some ten dependent steps.
// Device time: one prompt of 8192 tokens, 32 heads over 8 of 128, 410 us (1.34
// PFLOP/s); 1024 tokens over 32768, 391 us; 13 ragged prompts up to 1999, 171 us; 4
// prompts with heads of 256, 143 us; 4 new tokens for each of 32 sequences over an e4m3
// cache, 150 us (3.6 TB/s of it); a prompt of 48, 11 us.
// Tried, and slower: the scores read twice from tensor memory instead of kept in
// registers, the first weights taken against the old maximum before the new one
// is known (414 -> 456 us), one issuing warp for both slots (by a fifth),
// rolled loops over the MMAs, outputs transposed by shuffles before their stores.
#pragma once

#include <cfloat>
#include <climits>
#include <type_traits>

#include "awq_launch.cuh"
#include "awq_prompt_units.cuh"
#include "awq_tc.cuh"

namespace awq {

namespace {

constexpr float kChunkLazy = 8.f;      // a score raises the maximum when it passes it by this (base 2)
// fp16 weights are taken against 2^-7 of the maximum: they stay below 2^15 and
// keep 31 bits below the maximum's own before they vanish.
constexpr float kChunkRaiseF16 = 7.f;
// Least factor that turns a score into a base-2 logarithm: with 0 a masked score of
// -infinity would be NaN. The smallest fp32 makes 2^-21 of the largest score.
constexpr float kChunkMinFactor = 1.40129846e-45f;
constexpr float kChunkLn2 = 0.6931471805599453f;
constexpr int kMmaWarp = 8, kLoaderWarp = 10;
constexpr int kUnits = 3;              // units in shared memory
constexpr int kWaitTries = 1 << 18;    // of 4 to 33 us, as measured: 1 to 9 s

template <int DP, bool FP8>
struct ChunkGeo {
    // e4m3: 10 copies codes, 11 finds the units, 12-15 expand the codes; else 10 and 11 copy
    // 64 columns each, or 10 copies and 11 makes tiles of V finite
    static constexpr bool kGuardWarp = !FP8 && DP == 64;
    static constexpr int kThreads = FP8 ? 512 : 384, kFillWarp = FP8 ? 12 : 10, kFillWarps = FP8 ? 4 : kGuardWarp ? 1 : 2;
    static constexpr int QT = DP <= 128 ? 2 : 1;            // row tiles of a unit
    static constexpr int R = 128 * QT;
    static constexpr int SC = DP < 128 ? DP : 128;          // columns of a stage
    static constexpr int HV = DP / SC;                      // stages of a key tile
    static constexpr int kStage = kChunkKeys * SC * 2;
    static constexpr int kStages = (FP8 ? 96 : 160) * 1024 / kStage;
    // e4m3 stages on their way to fp16, at most
    static constexpr int kRaw = FP8 ? kChunkCodeBytes / (kStage / 2) : 0;
    static constexpr int kQSub = R * 128;                   // 64 columns of Q
    static constexpr int kQ = DP / 64 * kQSub;
    // after Q and the stages: maxima and sums that two slots exchange, rows' powers of two, barriers
    static constexpr int oStages = kQ, oRaw = oStages + kStages * kStage, oMl = oRaw + kRaw * kStage / 2, oExp = oMl + 2 * 128 * 8,
                         oUnits = oExp + 2 * 256, oBars = oUnits + kUnits * 64,
                         kRawBars = FP8 ? kRaw : kGuardWarp ? kStages : 1,
                         kBars = 2 * kStages + 2 + 2 + 2 + 2 + 2 + 5 + 2 * kUnits + 2 * kRawBars,
                         oMisc = oBars + kBars * 8, kSmem = oMisc + 40;
    static constexpr uint32_t kTmemO = 256;                 // first column of O; S at 0 and 128
    static_assert(kSmem <= 227 * 1024, "shared memory of a block");
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ uint64_t pack_f2(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack_f2(uint64_t v, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 32 columns of the warp's 32 lanes; complete after tc_wait_ld32().
__device__ __forceinline__ void tc_ld32_async(uint32_t taddr, float *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
        "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]),
          "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]),
          "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]),
          "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr));
}
// Waits for the loads; the registers pass through so that no use of them is
// moved above the wait.
__device__ __forceinline__ void tc_wait_ld32(float *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]),
                   "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]), "+f"(r[16]),
                   "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]), "+f"(r[24]),
                   "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])
                 :
                 : "memory");
}

// Shared memory matrix descriptor of V as the B operand, MN-major: rows of 64
// columns (128 bytes, 128-byte swizzle), 1024 bytes from 8 keys to the next 8,
// 16 KB from 64 columns to the next 64.
__device__ __forceinline__ uint64_t umma_desc_v(uint32_t addr)
{
    uint64_t d = static_cast<uint64_t>((addr & 0x3FFFF) >> 4);
    d |= static_cast<uint64_t>((kChunkKeys * 128) >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= 1ull << 46;
    d |= 2ull << 61;
    return d;
}
// kind::f16, 128 rows, N columns, fp32 accumulator; bf16 operands; A negated (bit
// 13); B MN-major.
__device__ __forceinline__ uint32_t chunk_idesc(int N, bool bf16, bool negative, bool b_mn)
{
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (negative ? 1u << 13 : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
           (128u >> 4 << 24);
}

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 bytes, or zeros where `bytes` is 0.
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// 4D TMA tile load (coordinates innermost first).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *m, uint64_t *bar, int c0, int c1, int c2, int c3)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void sts_v4(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Four e4m3 codes as two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t four, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}
__device__ __forceinline__ int atomic_add_acq_rel(int32_t *p, int v)
{
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// Whether one of four pairs of 16-bit values is not finite: an exponent of ones
// carries into the sign's place.
template <typename C>
__device__ __forceinline__ uint32_t not_finite4(uint4 v)
{
    constexpr uint32_t M = std::is_same<C, __half>::value ? 0x7C007C00u : 0x7F807F80u;
    constexpr uint32_t one = std::is_same<C, __half>::value ? 0x04000400u : 0x00800080u;
    return (((v.x & M) + one) | ((v.y & M) + one) | ((v.z & M) + one) | ((v.w & M) + one)) & 0x80008000u;
}

// A pair of 16-bit values with those that are not finite made 0.
template <typename C>
__device__ __forceinline__ uint32_t finite_pair(uint32_t v)
{
    constexpr uint32_t M = std::is_same<C, __half>::value ? 0x7C00u : 0x7F80u;
    uint32_t r = v;
    if ((v & M) == M) r &= 0xFFFF0000u;
    if ((v & (M << 16)) == (M << 16)) r &= 0x0000FFFFu;
    return r;
}

__device__ __forceinline__ void st_v8(void *p, const uint32_t *r)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
                 "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void st_v4(void *p, const uint32_t *r)
{
    asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

// Which of the columns c .. c + 31 of V hold a value that is not finite at a key
// that the row sees, among the tiles whose values were made finite on their way
// to the tensor core. Reads them again: nothing of it runs on finite values.
template <typename T, bool FP8>
__device__ __forceinline__ uint32_t not_finite_seen(const ChunkArgs &a, const Unit &u, int limit, int c)
{
    const awq_kv_plane &pl = a.cache.v;
    const int from = max(u.all0 / kChunkKeys, u.k0) * kChunkKeys, to = min(limit, u.k1 * kChunkKeys);
    uint32_t mask = 0;
#pragma unroll 1
    for (int key = from; key < to; ++key) {
        int64_t off;
        if (a.page_table) {
            const int page = key / a.cache.page_size, id = a.page_table[u.b * a.table_stride + page];
            if (id < 0 || id >= a.cache.num_pages) continue;
            off = id * pl.page_stride + (key - page * a.cache.page_size) * pl.token_stride;
        } else {
            off = (static_cast<int64_t>(u.q0) + key) * pl.token_stride;
        }
        off += u.h * pl.head_stride;
#pragma unroll 1
        for (int i = 0; i < 32 && c + i < a.cache.head_dim; ++i) {
            bool bad;
            if constexpr (FP8) {
                bad = (static_cast<const uint8_t *>(pl.data)[off + c + i] & 0x7F) == 0x7F;
            } else {
                const uint32_t v = static_cast<const uint16_t *>(pl.data)[off + c + i];
                constexpr uint32_t M = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
                bad = (v & M) == M;
            }
            mask |= (bad ? 1u : 0u) << i;
        }
    }
    return mask;
}

// The blocks that share a cut unit, for a whole warp: the first one, and where
// `list` is given all of them, with this block's place and their number.
__device__ __forceinline__ int sharing_blocks(const Unit &u, int64_t per, int lane, int16_t *list, int &me, int &count)
{
    const int c0 = first_block(u, per), c1 = last_block(u, per);
    int first = -1;
    count = 0;
    me = 0;
    for (int base = c0; base <= c1; base += 32) {
        const int c = base + lane;
        const bool in = c <= c1 && shares(u, per, c);
        const uint32_t all = __ballot_sync(~0u, in);
        if (all == 0) continue;
        if (first < 0) first = base + __ffs(all) - 1;
        if (!list) break;
        const int place = count + __popc(all & ((1u << lane) - 1));
        if (in) list[place] = static_cast<int16_t>(c);
        if (static_cast<int>(blockIdx.x) >= base && static_cast<int>(blockIdx.x) < base + 32)
            me = count + __popc(all & ((1u << (blockIdx.x - base)) - 1));
        count += __popc(all);
    }
    return first;
}

// ----------------------------------------------------------------- the kernel

template <typename T, bool FP8, int DP>
__global__ void __launch_bounds__(ChunkGeo<DP, FP8>::kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                      const __grid_constant__ CUtensorMap map_q, const __grid_constant__ ChunkArgs a)
{
    using G = ChunkGeo<DP, FP8>;
    using C = typename std::conditional<FP8, __half, T>::type;      // the tensor core's type
    constexpr bool kBf16 = std::is_same<C, __nv_bfloat16>::value;
    constexpr bool kScaledQ = FP8 && !std::is_same<T, C>::value;    // bf16 q as fp16 with a power of two taken out
    constexpr float kRaise = kBf16 ? 0.f : kChunkRaiseF16;
    constexpr int kThreads = G::kThreads, FW = G::kFillWarps;
    constexpr int NST = G::kStages, HV = G::HV, SC = G::SC, QT = G::QT;

    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *const stages = smem + G::oStages;
    float2 *const s_ml = reinterpret_cast<float2 *>(smem + G::oMl);          // [2][128]
    uint8_t *const s_exp = smem + G::oExp;                                   // [2][256]
    uint64_t *const full = reinterpret_cast<uint64_t *>(smem + G::oBars);
    uint64_t *const empty = full + NST;
    uint64_t *const q_full = empty + NST, *const q_empty = q_full + 1;
    uint64_t *const s_full = q_empty + 1;        // [2]
    uint64_t *const p_half = s_full + 2;         // [2]: weights of 64 keys
    uint64_t *const p_full = p_half + 2;         // [2]
    uint64_t *const o_done = p_full + 2;         // [2]
    uint64_t *const drain = o_done + 2;
    uint64_t *const both = drain + 2;                                        // both softmax warpgroups
    uint64_t *const one = drain + 3;                                         // [2]: each by itself
    uint64_t *const u_full = drain + 5, *const u_empty = u_full + kUnits;    // [kUnits]
    uint64_t *const raw_full = u_empty + kUnits, *const raw_empty = raw_full + G::kRawBars;   // codes; tiles to be made finite
    Unit *const s_unit = reinterpret_cast<Unit *>(smem + G::oUnits);
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem + G::oMisc);
    int *const s_first = reinterpret_cast<int *>(smem + G::oMisc + 4);
    int64_t *const s_first_at = reinterpret_cast<int64_t *>(smem + G::oMisc + 8);
    int *const s_bad = reinterpret_cast<int *>(smem + G::oMisc + 16);        // [4]
    uint64_t *const s_start = reinterpret_cast<uint64_t *>(smem + G::oMisc + 32);

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0);
    const int D = a.cache.head_dim;
    if (smem_u32(smem) & 1023) {                 // (the tiles' swizzle needs it)
        if (tid == 0) set_status(a.status, AWQ_ERR_CUDA);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], FP8 ? FW : 2);
            mbar_init(&empty[i], QT);            // the issuers
        }
        mbar_init(q_full, kScaledQ || !a.q_box ? 32 * FW : 1);
        mbar_init(q_empty, QT);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_half[i], 4);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&drain[i], 1);
        mbar_init(both, 8);
        for (int i = 0; i < 2; ++i) mbar_init(&one[i], 4);
        for (int i = 0; i < G::kRawBars; ++i) {
            mbar_init(&raw_full[i], FP8 || G::kGuardWarp ? 1 : 2);
            mbar_init(&raw_empty[i], FW);
        }
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(&u_full[i], 1);
            mbar_init(&u_empty[i], (FP8 ? 5 : 2) + QT + 8);      // copying and filling, issuers, softmax
        }
        for (int i = 0; i < 4; ++i) s_bad[i] = 0;
        fence_barrier_init();
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
    }
    if (warp == kMmaWarp) tc_alloc(tmem_slot, 512);
    grid_dependency_wait();
    grid_launch_dependents();
    if (tid == kThreads - 1) *s_start = global_timer_ns();

    // ---- the sum of all costs, and the first unit of the block's share
    int64_t x0, x1, per_cta;
    {
        int64_t *const scan = reinterpret_cast<int64_t *>(s_ml);             // [16], where no copy goes
        const Span span = sequences_of(a.batch, tid, kThreads);
        int64_t mine = 0;
        for (int b = span.lo; b < span.hi; ++b) {
            const Sequence s = sequence_at(a, b);
            if (s.bad && blockIdx.x == 0) set_status(a.status, AWQ_ERR_BAD_INDEX);
            mine += Costs(s, a, QT == 2).head * a.cache.num_heads;
        }
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) scan[warp] = incl;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        int64_t before = incl - mine, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            const int64_t v = scan[w];
            if (w < warp) before += v;
            total += v;
        }
        per_cta = share_of(total, gridDim.x);
        x0 = min(total, per_cta * blockIdx.x);
        x1 = min(total, x0 + per_cta);
        if (x0 < x1 && x0 >= before && x0 < before + mine) {
            int b = span.lo;
            for (;; ++b) {
                const int64_t c = Costs(sequence_at(a, b), a, QT == 2).head * a.cache.num_heads;
                if (x0 < before + c) break;
                before += c;
            }
            *s_first = b;
            *s_first_at = before;
        }
        __syncthreads();
    }
    const uint32_t tmem = *tmem_slot;
    // Waits give up after kWaitTries suspensions; what a
    // role does after that is harmless and ends soon, as it waits no more. The status
    // is set once, at the end.
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!ok || mbar_try_wait(bar, parity)) return;
        int left = kWaitTries;
#pragma unroll 1
        while (!mbar_try_wait_sleep(bar, parity, 20000))
            if (--left == 0) {
                ok = false;
                break;
            }
    };
    // Both (their answers, of 100 cycles each, come together).
    auto wait_two = [&](uint64_t *bar0, uint32_t parity0, uint64_t *bar1, uint32_t parity1) {
        const bool in0 = mbar_try_wait(bar0, parity0), in1 = mbar_try_wait(bar1, parity1);
        if (!in0) wait(bar0, parity0);
        if (!in1) wait(bar1, parity1);
    };
    // The role's next unit (the ordinal-th, from 1) in shared memory; NULL after the
    // last one. It is given back, by one thread of each warp, with done_with().
    auto next_unit = [&](int ordinal) -> const Unit * {
        const int i = (ordinal - 1) % kUnits;
        wait(&u_full[i], (ordinal - 1) / kUnits & 1);
        ok = __all_sync(~0u, ok);                    // (a warp gives up as one)
        const Unit *const v = s_unit + i;
        return ok && v->b >= 0 ? v : nullptr;
    };
    auto done_with = [&](int ordinal) { mbar_arrive(&u_empty[(ordinal - 1) % kUnits]); };
    if (warp >= kMmaWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FP8 ? 56 : 88));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(FP8 ? 200 : 208));
    // The units, found one after another.
    auto make_unit = [&](UnitWalk<QT == 2> &walk, int made) {
        if (made >= kUnits) wait(&u_empty[made % kUnits], (made / kUnits - 1) & 1);
        Unit v;
        const bool found = walk.next(a, v);
        if (!found) v.b = -1;
        if (lane == 0) {
            s_unit[made % kUnits] = v;
            mbar_arrive(&u_full[made % kUnits]);
        }
        return found;
    };
    auto first_unit = [&]() { return UnitWalk<QT == 2>(a, x0, x1, x0 < x1 ? *s_first : 0, x0 < x1 ? *s_first_at : 0); };

    if (FP8 && warp == kLoaderWarp + 1) {
        UnitWalk<QT == 2> walk = first_unit();
        int made = 0;
#pragma unroll 1
        while (make_unit(walk, made) && ok) ++made;
    } else if (warp >= kLoaderWarp) {
        // ------------------------------------------------------- loader
        const int lw = FW == 1 ? 0 : warp - G::kFillWarp;
        // ---- Q of a unit, 16 bytes a thread: RP rows of CH chunks a warp and turn, so a
        // thread's rows are as far apart as the warps reach and its token and head go on by additions.
        auto load_q = [&](const Unit &u, int ordinal) {
            if (!kScaledQ && a.q_box) {
                // boxes of whole tokens: units begin with one
                if (lw) return;
                if (ordinal > 1) wait(q_empty, (ordinal - 2) & 1);
                const int rows = a.q_box * a.group, boxes = (u.rows + rows - 1) / rows, all = boxes * ((D + 63) / 64);
                if (lane == 0) mbar_arrive_expect_tx(q_full, all * rows * 128);
                __syncwarp();
                for (int i = lane; i < all; i += 32) {
                    const int sub = i / boxes, box = i - sub * boxes;
                    tma_load_3d(smem + sub * G::kQSub + box * rows * 128, &map_q, q_full, sub * 64, u.h * a.group,
                                u.q0 + u.row0 / a.group + box * a.q_box);
                }
                return;
            }
            constexpr int CH = DP / 8, RP = 32 / CH;
            const int ch = lane % CH, first = lw * RP + lane / CH, turn_rows = FW * RP;
            const bool col = ch * 8 < D, pad = ch * 8 < (D + 15) / 16 * 16;
            const uint32_t group = a.group, row = u.row0 + first;
            uint32_t g = row % group;
            const T *src = static_cast<const T *>(a.q.data) + (u.q0 + static_cast<int64_t>(row / group)) * a.q.token_stride +
                           (static_cast<int64_t>(u.h) * group + g) * a.q.head_stride + ch * 8;
            const int64_t next_token = a.q.token_stride - static_cast<int64_t>(group) * a.q.head_stride;
            const int64_t turn = (turn_rows / group) * a.q.token_stride + (turn_rows % group) * a.q.head_stride;
            if (ordinal > 1) wait(q_empty, (ordinal - 2) & 1);
            const int rows = u.rows > 128 ? G::R : 128;                 // (the rows of a tile are all written)
#pragma unroll 4
            for (int r = first; r < rows; r += turn_rows) {
                const bool in = r < u.rows && col;
                const uint32_t dst = smem_u32(smem) + (ch >> 3) * G::kQSub + sw128_offset(r, ch & 7);
                if constexpr (kScaledQ) {
                    // the row's largest magnitude to [2^14, 2^15)
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (in) v = *reinterpret_cast<const uint4 *>(src);
                    float f[8];
                    const uint32_t raw[4] = {v.x, v.y, v.z, v.w};
                    float top = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = unpack2<T>(raw[i]);
                        f[2 * i] = x.x;
                        f[2 * i + 1] = x.y;
                        top = max3(top, fabsf(x.x), fabsf(x.y));
                    }
#pragma unroll
                    for (int m = CH / 2; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, m));
                    const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -112);
                    const float by = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
                    if (pad)
                        sts_v4(dst, make_uint4(pack2<__half>(f[0] * by, f[1] * by), pack2<__half>(f[2] * by, f[3] * by),
                                               pack2<__half>(f[4] * by, f[5] * by), pack2<__half>(f[6] * by, f[7] * by)));
                    if (ch == 0) s_exp[(ordinal & 1) * 256 + r] = static_cast<uint8_t>(e + 112);
                } else {
                    if (pad) cp_async_16_or_zero(dst, in ? src : static_cast<const T *>(a.q.data), in ? 16 : 0);
                }
                src += turn;
                g += turn_rows % group;
                if (g >= group) {
                    g -= group;
                    src += next_token;
                }
            }
            if constexpr (kScaledQ) {
                fence_proxy_async();
                mbar_arrive(q_full);
            } else {
                cp_async_arrive_noinc(q_full);
            }
        };
        // A unit's tiles in the order that they are used up: K 0 .. ahead - 1, then V j, K j
        // + ahead .. (`ahead` is 1 where both slots use a tile, else 2).
        struct Tiles {
            int n, ahead, k, v;                              // tiles; K's and V's so far
            __device__ __forceinline__ Tiles(const Unit &u)
                : n(u.k1 - u.k0), ahead(QT == 2 && u.rows > 128 ? 1 : 2), k(0), v(0) {}
            __device__ __forceinline__ bool more() const { return v < n; }
            __device__ __forceinline__ bool is_v() const { return k - v == ahead || k == n; }
            __device__ __forceinline__ int tile() const { return is_v() ? v : k; }
            __device__ __forceinline__ void next()
            {
                if (is_v()) ++v;
                else ++k;
            }
        };
        // A place in a ring: stage and the parity of its filling.
        struct Ring {
            uint32_t i = 0, phase = 0;
            __device__ __forceinline__ void next(uint32_t n)
            {
                if (++i == n) {
                    i = 0;
                    phase ^= 1;
                }
            }
        };
        // Copies are boxes of a.box keys, as many as lie in one page wherever they begin;
        // nothing of boxes past the unit's keys (their place is -1). Boxes of less than 4
        // keys: lane i has the i-th box of a tile, every 32nd more is found late.
        const int box = a.box, boxes = kChunkKeys / box;
        auto find = [&](const Unit &u, uint32_t key, int &page, int &place) {
            page = 0;
            place = -1;
            if (key >= static_cast<uint32_t>(u.keys)) return;
            if (!a.page_table) {
                place = u.q0 + key;
                return;
            }
            const int at = a.page_shift ? __umulhi(key, a.page_magic) >> (a.page_shift - 1) : key;
            place = key - at * a.cache.page_size;
            page = a.page_table[u.b * a.table_stride + at];
        };
        auto usable = [&](int page, int place) {
            if (place < 0) return false;
            if (static_cast<uint32_t>(page) < static_cast<uint32_t>(a.page_table ? a.cache.num_pages : 1)) return true;
            set_status(a.status, AWQ_ERR_BAD_INDEX);
            return false;
        };
        // One stage (from column d0 on) of the tile at key0, of which the lane has the
        // lane_box-th box, at `page` and `place`, `in` where it is to be copied. Lane 0
        // arrives at `bar` with the bytes.
        auto copy = [&](const Unit &u, bool is_v, int key0, int lane_box, int page, int place, bool in, int d0, uint32_t dst,
                        int row_bytes, uint64_t *bar) {
            const CUtensorMap *const map = is_v ? &map_v : &map_k;
            const int head = a.head_step[is_v] * u.h, step = a.page_step[is_v];
            const int bytes = box * row_bytes, apart = FP8 ? box * code_row_bytes(row_bytes, box) : bytes;
            int count = __popc(__ballot_sync(~0u, in));
            auto expect = [&]() {
                if (lane == 0) mbar_arrive_expect_tx(bar, count * bytes);
                __syncwarp();
                if (in) tma_load_4d(dst + lane_box * apart, map, bar, d0, place, head, step * page);
            };
            if (boxes <= 32) {
                expect();
                return;
            }
            // Pages of a token or two, and odd ones. All of the lane's boxes are asked for at
            // once where registers allow it (4 new tokens of 32 sequences, pages of one token:
            // e4m3 1384 -> 1027 us; 16-bit heads above 64 would lose 3 to 8 % on all pages).
            if constexpr (FP8 || DP == 64) {
                int pg[3], pl[3];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    pg[i] = 0;
                    pl[i] = -1;
                    if (32 * (i + 1) < boxes) find(u, key0 + (lane + 32 * (i + 1)) * box, pg[i], pl[i]);
                }
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    if (!usable(pg[i], pl[i])) pl[i] = -1;
                    count += __popc(__ballot_sync(~0u, pl[i] >= 0));
                }
                expect();
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (pl[i] >= 0) tma_load_4d(dst + (lane + 32 * (i + 1)) * apart, map, bar, d0, pl[i], head, step * pg[i]);
            } else {
#pragma unroll 1
                for (int i = lane + 32; i < boxes; i += 32) {
                    int pg, pl;
                    find(u, key0 + i * box, pg, pl);
                    count += __popc(__ballot_sync(~0u, usable(pg, pl)));
                }
                expect();
#pragma unroll 1
                for (int i = lane + 32; i < boxes; i += 32) {
                    int pg, pl;
                    find(u, key0 + i * box, pg, pl);
                    if (usable(pg, pl)) tma_load_4d(dst + i * apart, map, bar, d0, pl, head, step * pg);
                }
            }
        };
        // a V tile that some row of the unit does not see in full: values that are not
        // finite would reach it as 0 times themselves
        auto guarded = [&](const Unit &u, bool is_v, int key0) { return is_v && key0 + kChunkKeys > u.all0; };

        Ring to;                                             // the next stage to fill
        int ordinal = 0;
        // 64 columns of a V tile in 16 bits, made finite from a key on (a multiple of 4 B);
        // then the stage's arrival. B loads are in flight. The unit is marked for
        // not_finite_seen() only where one lies before the unit's last key: past it are the rest of
        // a page and what another kernel left in the stage, which no row sees.
        auto make_finite = [&](uint32_t tile, int from, int keys, uint64_t *bar) {
            constexpr int B = G::kGuardWarp ? 4 : 8;
#pragma unroll 1
            for (int key = from; key < kChunkKeys; key += 4 * B) {
                const uint32_t at = tile + key * 128 + lane * 16;
                uint4 v[B];
#pragma unroll
                for (int k = 0; k < B; ++k) v[k] = lds_v4(at + k * 512);
                uint32_t bad = 0;
#pragma unroll
                for (int k = 0; k < B; ++k) bad |= not_finite4<C>(v[k]);
                auto seen = [&](int k) { return key + 4 * k + (lane >> 3) < keys; };
                auto put = [&](int k, uint4 x) {
                    sts_v4(at + k * 512, make_uint4(finite_pair<C>(x.x), finite_pair<C>(x.y), finite_pair<C>(x.z), finite_pair<C>(x.w)));
                };
                // (hardly ever run, but its registers and length count: rolled, 4 prompts with heads of
                // 256 take 145 us, not 156; unrolled, 13 ragged prompts with heads of 128 171, not 175)
                if (bad) {
                    if constexpr (DP > 128) {
#pragma unroll 1
                        for (int k = 0; k < B; ++k) {
                            const uint4 x = lds_v4(at + k * 512);
                            if (not_finite4<C>(x) && seen(k)) s_bad[ordinal & 3] = ordinal;
                            put(k, x);
                        }
                    } else {
                        bool mark = false;
#pragma unroll
                        for (int k = 0; k < B; ++k) mark |= not_finite4<C>(v[k]) && seen(k);
                        if (mark) s_bad[ordinal & 3] = ordinal;
#pragma unroll
                        for (int k = 0; k < B; ++k) put(k, v[k]);
                    }
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        if constexpr (FP8) {
            // One warp copies codes, up to kRaw stages ahead; four expand them, a row's 16
            // codes a thread.
            constexpr int CH = SC / 16, RP = 32 / CH;
            const uint32_t raw0 = smem_u32(smem + G::oRaw);
            const uint32_t code_row = code_row_bytes(SC, box), raw_stage = kChunkKeys * code_row;
            const uint32_t raws = SC == 128 || code_row == SC ? G::kRaw : G::kRaw / 2;
            Ring raw;
            if (warp == kLoaderWarp) {
                // A lane has a box of one of the next tiles, and the one as many tiles on: a
                // page's number is asked for well before it is used (asked for one tile
                // ahead, as with 16 bits, it held every tile back: 201 -> 187 us for 4 new
                // tokens of 32 sequences; there, registers are short and it lost 4 %).
                const int per = min(boxes, 32), tiles = 32 / per, lane_box = lane & (per - 1), lane_tile = lane / per;
                struct Places {
                    int page, place, page1, place1;          // of the lane's box, and of its next one
                } of_k, of_v;
                auto look = [&](const Unit &u, int tile, int &page, int &place) {
                    find(u, static_cast<uint32_t>(u.k0 + tile) * kChunkKeys + lane * box, page, place);
                };
                // The page and place of the lane's box if it is one of the tile's, else place
                // -1; on to the next tile.
                auto take = [&](const Unit &u, Places &p, int tile, int &page, int &place) {
                    page = p.page;
                    place = (tile & (tiles - 1)) == lane_tile ? p.place : -1;
                    if (((tile + 1) & (tiles - 1)) == 0) {
                        p.page = p.page1;
                        p.place = p.place1;
                        look(u, tile + 1 + tiles, p.page1, p.place1);
                    }
                };
                uint32_t copied = 0;
                while (const Unit *const next = next_unit(++ordinal)) {
                    const Unit u = *next;               // (in registers: not read again behind every barrier)
                    Tiles t(u);
                    look(u, 0, of_k.page, of_k.place);
                    look(u, tiles, of_k.page1, of_k.place1);
                    of_v = of_k;
#pragma unroll 1
                    while (t.more()) {
                        const bool is_v = t.is_v();
                        const int tile = t.tile(), key0 = (u.k0 + tile) * kChunkKeys;
                        int page, place;
                        if (is_v) take(u, of_v, tile, page, place);
                        else take(u, of_k, tile, page, place);
                        const bool in = usable(page, place);
                        t.next();
#pragma unroll
                        for (int hh = 0; hh < HV; ++hh) {
                            wait(&raw_empty[raw.i], raw.phase ^ 1);
                            copy(u, is_v, key0, lane_box, page, place, in, hh * SC, raw0 + raw.i * raw_stage, SC, &raw_full[raw.i]);
                            raw.next(raws);
                            ++copied;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) done_with(ordinal);
                }
                if (!ok)                                     // as below
                    for (uint32_t i = copied > raws ? copied - raws : 0; i < copied; ++i)
                        mbar_wait_bounded(&raw_full[i % raws], i / raws & 1, a.timeout_ns);
            } else {
                // Lanes of the second 64 columns take the row beside theirs, whose swizzle has
                // the other parity, so that neither load nor store hits a bank twice. RP rows
                // on, the swizzle changes with their number's last bits alone.
                const int ch = lane % CH, row = lw * 32 + (lane / CH ^ ch >> 2);
                const uint32_t at0 = (ch >> 2) * (kChunkKeys * 128) + sw128_offset(row, (ch & 3) * 2);
                const uint32_t at1 = (ch >> 2) * (kChunkKeys * 128) + sw128_offset(row + RP, (ch & 3) * 2);
                while (const Unit *const next = next_unit(++ordinal)) {
                    const Unit u = *next;
                    load_q(u, ordinal);
                    Tiles t(u);
                    // the first tile that is guarded, and the unit's keys in the last one
                    const int guarded_from = u.all0 / kChunkKeys - u.k0, last_keys = u.keys - (u.k1 - 1) * kChunkKeys;
#pragma unroll 1
                    while (t.more()) {
                        const bool guard = t.is_v() && t.v >= guarded_from;
                        t.next();
#pragma unroll 1
                        for (int hh = 0; hh < HV; ++hh) {
                            const uint32_t tile = smem_u32(stages) + to.i * G::kStage;
                            const uint32_t from = raw0 + raw.i * raw_stage + row * code_row + ch * 16, step = RP * code_row;
                            wait_two(&empty[to.i], to.phase ^ 1, &raw_full[raw.i], raw.phase);
                            // (unrolled where rows alternate between two offsets)
                            auto place_of = [&](int i) { return tile + (RP == 4 && i & 1 ? at1 + (i - 1) * (RP * 128) : at0 + i * (RP * 128)); };
                            auto expand = [&](const uint4 &v, uint4 &lo, uint4 &hi) {
                                e4m3x4_f16x4(v.x, lo.x, lo.y);
                                e4m3x4_f16x4(v.y, lo.z, lo.w);
                                e4m3x4_f16x4(v.z, hi.x, hi.y);
                                e4m3x4_f16x4(v.w, hi.z, hi.w);
                            };
                            if (guard) {
#pragma unroll 1
                                for (int i = 0; i < 32 / RP; ++i) {
                                    uint4 lo, hi;
                                    expand(lds_v4(from + i * step), lo, hi);
                                    if (not_finite4<C>(lo) | not_finite4<C>(hi)) {
                                        // (marked as in make_finite(); t.v is V's tile after this one, and the
                                        // row comes from its address: registers are short)
                                        if (t.v < t.n || static_cast<int>((from + i * step - raw0) / code_row % kChunkKeys) < last_keys)
                                            s_bad[ordinal & 3] = ordinal;
                                        lo = make_uint4(finite_pair<C>(lo.x), finite_pair<C>(lo.y), finite_pair<C>(lo.z), finite_pair<C>(lo.w));
                                        hi = make_uint4(finite_pair<C>(hi.x), finite_pair<C>(hi.y), finite_pair<C>(hi.z), finite_pair<C>(hi.w));
                                    }
                                    sts_v4(place_of(i), lo);
                                    sts_v4(place_of(i) ^ 16, hi);
                                }
                            } else {
                                constexpr int B = 4;                 // loads in flight
                                uint4 v[B];
#pragma unroll
                                for (int i = 0; i < B; ++i) v[i] = lds_v4(from + i * step);
#pragma unroll
                                for (int i = 0; i < 32 / RP; ++i) {
                                    uint4 lo, hi;
                                    expand(v[i % B], lo, hi);
                                    if (i + B < 32 / RP) v[i % B] = lds_v4(from + (i + B) * step);
                                    sts_v4(place_of(i), lo);
                                    sts_v4(place_of(i) ^ 16, hi);
                                }
                            }
                            fence_proxy_async();
                            __syncwarp();
                            if (lane == 0) {
                                mbar_arrive(&raw_empty[raw.i]);
                                mbar_arrive(&full[to.i]);
                            }
                            to.next(NST);
                            raw.next(raws);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) done_with(ordinal);
                }
            }
        } else if (!G::kGuardWarp || warp == kLoaderWarp) {
            uint32_t guard_phase = 0, filled = 0;
            int page = 0, place = -1;                        // of the lane's box of the next tile
            while (const Unit *const next = next_unit(++ordinal)) {
                const Unit &u = *next;
                Tiles t(u);
                if (t.more()) find(u, (u.k0 + t.tile()) * kChunkKeys + lane * box, page, place);
                bool has_q = false;
#pragma unroll 1
                while (true) {
                    if (!has_q && (t.k == 1 || !t.more())) {
                        load_q(u, ordinal);                  // behind K's first tile, which has room earlier
                        has_q = true;
                    }
                    if (!t.more()) break;
                    const bool is_v = t.is_v(), in = lane < boxes && usable(page, place);
                    const int key0 = (u.k0 + t.tile()) * kChunkKeys, pg = page, pl = place;
                    const bool guard = guarded(u, is_v, key0);
                    t.next();
                    if (t.more()) find(u, (u.k0 + t.tile()) * kChunkKeys + lane * box, page, place);
#pragma unroll 1
                    for (int hh = 0; hh < HV; ++hh) {
                        // a warp copies 64 columns
                        const int d0 = hh * SC + lw * 64;
                        const bool part = G::kGuardWarp || d0 < D;
                        const uint32_t dst = smem_u32(stages) + to.i * G::kStage + lw * (kChunkKeys * 128);
                        uint64_t *const bar = !guard ? &full[to.i] : G::kGuardWarp ? &raw_full[to.i] : raw_full;
                        wait(&empty[to.i], to.phase ^ 1);
                        if (part) copy(u, is_v, key0, lane, pg, pl, in, d0, dst, 128, bar);
                        else if (lane == 0) mbar_arrive(bar);
                        if (G::kGuardWarp) {
                            if (lane == 0) mbar_arrive(&full[to.i]);     // (the other arrival is the bytes' or the next warp's)
                        } else if (guard) {
                            wait(raw_full, guard_phase);
                            guard_phase ^= 1;
                            make_finite(dst, part ? 0 : kChunkKeys, u.keys - key0, &full[to.i]);
                        }
                        to.next(NST);
                        ++filled;
                    }
                }
                __syncwarp();
                if (lane == 0) done_with(ordinal);
            }
            // after a time-out: the copies in flight end before the block does
            if (!ok)
                for (uint32_t i = filled > NST ? filled - NST : 0; i < filled; ++i)
                    mbar_wait_bounded(&full[i % NST], i / NST & 1, a.timeout_ns);
        } else {
            // Makes the guarded tiles of V finite: done by the warp that copies, each holds
            // the next unit's Q and K back by 4000 cycles (40 short prompts with heads of 64
            // 86 -> 79 us, 64 sequences that decode 157 -> 148). Larger heads keep both
            // warps for the copies (1024 tokens over pages of 32 388 us, with one 404).
            uint32_t base = 0, phases = 0;                   // the unit's first filling; a bit per stage
            while (const Unit *const next = next_unit(++ordinal)) {
                const Unit &u = *next;
                const int n = u.k1 - u.k0, k0 = u.k0, all0 = u.all0, ahead = QT == 2 && u.rows > 128 ? 1 : 2;
#pragma unroll 1
                for (int j = max(0, all0 / kChunkKeys - k0); j < n; ++j) {
                    const uint32_t st = (base + j + min(n, j + ahead)) % NST;
                    wait(&raw_full[st], phases >> st & 1);
                    phases ^= 1u << st;
                    // its keys that some row does not see, from a multiple of 16 on
                    make_finite(smem_u32(stages) + st * G::kStage, max(0, all0 - (k0 + j) * kChunkKeys) & ~15, u.keys - (k0 + j) * kChunkKeys, &full[st]);
                }
                base += 2 * n;
                __syncwarp();
                if (lane == 0) done_with(ordinal);
            }
        }
        // (and the last Q that was asked for: of the unit before the one that did not come)
        if (!ok && warp == G::kFillWarp && ordinal > 1) mbar_wait_bounded(q_full, ordinal & 1, a.timeout_ns);
        cp_async_commit();
        cp_async_wait_group<0>();
    } else if (warp >= kMmaWarp) {
        // ------------------------------------------------------- MMA issuers
        // A warp for each slot: what a warp does between its MMAs (a barrier's answer
        // takes 100 cycles, a commit 50) is hidden behind the other's. All lanes run
        // the code, one elected lane issues, places in the ring advance without
        // divisions. The second one finds the units as well, each while the one
        // before is at work.
        const int me = warp - kMmaWarp;
        // (not with e4m3, where a warp of its own does)
        constexpr bool kFinds = !FP8;
        int made = 0;
        bool all_made = !kFinds || me == 0;
        UnitWalk<QT == 2> walk = all_made ? UnitWalk<QT == 2>(a, 0, 0, 0, 0) : first_unit();
#pragma unroll 1
        while (!all_made && (QT == 1 ? ok : made == 0)) all_made = !make_unit(walk, made++);
        if (me < QT) {
            const int k_steps = (D + 15) / 16;               // of Q K'; times 16: columns of P V
            const uint64_t q_desc = umma_desc_sw128(smem_u32(smem));
            const uint64_t k_desc = umma_desc_sw128(smem_u32(stages)), v_desc = umma_desc_v(smem_u32(stages));
            const uint32_t qk_id = chunk_idesc(kChunkKeys, kBf16, a.negative, false);
            struct Place {
                uint32_t st, phase;
                __device__ __forceinline__ void advance(uint32_t by)
                {
                    st += by;
#pragma unroll 1
                    while (st >= NST) {
                        st -= NST;
                        phase ^= 1;
                    }
                }
            };
            auto commit = [&](uint64_t *bar) {
                if (elect_one()) tc_commit(bar);
            };
            Place kp, vp;                                    // of the next K and V tile
            uint32_t pos = 0;                                // the unit's first stage
            uint32_t p_phase = 0;                            // a bit per slot
            // S[slot] = Q[tile] K' and O[acc] (+)= P[slot] V
            auto qk = [&](int slot, int tile) {
                Place at = kp;
#pragma unroll
                for (int hh = 0; hh < HV; ++hh) {
                    if (HV > 1) wait(&full[at.st], at.phase);
                    const uint64_t da = q_desc + ((tile * (128 * 128) + hh * (SC / 64) * G::kQSub) >> 4);
                    const uint64_t db = k_desc + (at.st * G::kStage >> 4);
                    const int ks = k_steps - hh * (SC / 16);
                    auto step = [&](int k) {
                        const uint32_t in = (k & 3) * 2, sub = k >> 2;       // 16 columns on, 64 columns on
                        tc_mma_f16(tmem + slot * 128, da + in + sub * (G::kQSub >> 4), db + in + sub * (128 * 128 >> 4), qk_id,
                                   k > 0 || hh > 0);
                    };
                    if (elect_one()) {
                        if (ks >= SC / 16) {
#pragma unroll
                            for (int k = 0; k < SC / 16; ++k) step(k);
                        } else {
#pragma unroll 1
                            for (int k = 0; k < ks; ++k) step(k);
                        }
                        if (hh == HV - 1) tc_commit(&s_full[slot]);
                        tc_commit(&empty[at.st]);
                    }
                    at.advance(1);
                }
            };
            auto pv = [&](int slot, int acc, bool more) {
                const uint32_t phase = p_phase >> slot & 1;
                p_phase ^= 1u << slot;
                wait(&p_half[slot], phase);
                tc_fence_after();
                Place at = vp;
#pragma unroll
                for (int hh = 0; hh < HV; ++hh) {
                    if (HV > 1) wait(&full[at.st], at.phase);
                    const int cols = min(SC, k_steps * 16 - hh * SC);
                    const uint64_t db = v_desc + (at.st * G::kStage >> 4);
                    const uint32_t id = chunk_idesc(cols, kBf16, false, true), d = tmem + G::kTmemO + acc * 128 + hh * 128;
                    constexpr int kHalf = kChunkKeys / 32;
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kHalf; ++k)
                            tc_mma_f16_tmem_a(d, tmem + slot * 128 + k * 8, db + k * (2048 >> 4), id, k > 0 || more);
                    }
                    if (hh == 0) {
                        wait(&p_full[slot], phase);
                        tc_fence_after();
                    }
                    if (elect_one()) {
#pragma unroll
                        for (int k = kHalf; k < 2 * kHalf; ++k)
                            tc_mma_f16_tmem_a(d, tmem + slot * 128 + k * 8, db + k * (2048 >> 4), id, 1);
                        tc_commit(&empty[at.st]);
                    }
                    at.advance(1);
                }
            };
            int ordinal = 0;
            while (const Unit *const next = next_unit(ordinal + 1)) {
                const int n = __shfl_sync(~0u, next->k1 - next->k0, 0);
                const int n0 = __shfl_sync(~0u, next->n0, 0);        // (the first slot's rows see fewer keys)
                const bool wide = QT == 2 && __shfl_sync(~0u, next->rows, 0) > 128;
                ++ordinal;
                if (lane == 0) done_with(ordinal);
                const int ahead = wide ? min(1, n) : min(2, n);
                kp.st = pos % NST;                           // the unit's first stage
                kp.phase = pos / NST & 1;
                vp = kp;
                vp.advance(ahead * HV);
                wait(q_full, (ordinal - 1) & 1);
                fence_proxy_async();
                if constexpr (QT == 2) {
                    // Wide: every tile, the first slot up to n0; narrow: every other. A warp
                    // waits for all stages in their order, and gives back at once those that
                    // it has no use for (a stage that it passed over could be two fillings
                    // ahead of the phase that it waits for).
                    const int end = me == 0 ? n0 : n;
                    auto mine = [&](int j) { return wide ? j < end : (j & 1) == me; };
                    const int last = wide ? end - 1 : n - 1 - ((n - 1 - me) & 1);
                    auto give_back = [&](Place at) {
                        if (lane == 0) mbar_arrive(&empty[at.st]);
                    };
                    bool more = false;                       // the accumulator holds something
                    if (last < 0) commit(q_empty);
#pragma unroll 1
                    for (int j = -ahead; j <= n; ++j) {
                        // (the unit after the next would wait for this warp itself)
                        if (kFinds && j == min(0, n) && !all_made && made == ordinal) all_made = !make_unit(walk, made++);
                        if (j == n) break;
                        const bool next = j + ahead < n;
                        if (next && j >= 0) wait_two(&full[kp.st], kp.phase, &full[vp.st], vp.phase);
                        else if (next) wait(&full[kp.st], kp.phase);
                        else wait(&full[vp.st], vp.phase);
                        if (j >= 0) {
                            if (mine(j)) {
                                pv(me, me, more);
                                more = true;
                                if (j == last) commit(&o_done[me]);
                            } else {
                                give_back(vp);
                            }
                            vp.advance(j < n - ahead ? 2 : 1);
                        }
                        if (next) {
                            if (mine(j + ahead)) {
                                qk(me, wide ? me : 0);
                                if (j + ahead == last) commit(q_empty);
                            } else {
                                give_back(kp);
                            }
                            kp.advance(j + 1 < 0 ? 1 : 2);
                        }
                    }
                } else {
                    // S is double-buffered: P V of tile s - 2, then Q K' of tile s
#pragma unroll 1
                    for (int s = 0; s < n + 2; ++s) {
                        if (s >= 2) {
                            pv(s & 1, 0, s > 2);
                            vp.advance(s - 2 < n - ahead ? 2 * HV : HV);
                            commit(&o_done[s & 1]);
                        }
                        if (s < n) {
                            qk(s & 1, 0);
                            kp.advance(s + 1 < ahead ? HV : 2 * HV);
                            if (s + 1 == n) commit(q_empty);
                        }
                    }
                    if (n == 0) commit(q_empty);
                }
                pos += 2 * n * HV;
            }
            // every MMA has completed before the block gives up its tensor memory
            commit(&drain[me]);
            if (!mbar_wait_bounded(&drain[me], 0, a.timeout_ns)) ok = false;
        }
    } else {
        // ------------------------------------------------------- softmax and output
        const int w = warp >> 2, row = (warp & 3) * 32 + lane;               // this thread's row of a tile
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        uint32_t s_phase = 0, o_phase = 0;                                   // a bit per slot: score tiles, products with V
        int last = 0;                                                        // slot of the latest product
        // Units that are cut at their begin and at their end: a lane's word of the
        // first (lanes 0-15) and of the second.
        uint32_t shared_unit = 0, has_shared = 0;
        int ordinal = 0;
        float *const my_parts = a.parts + static_cast<int64_t>(blockIdx.x) * 2 * chunk_piece_floats(DP);
        // Both warpgroups meet.
        uint32_t met = 0;
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(both);
            wait(both, met);
            met ^= 1;
            ok = __all_sync(~0u, ok);
        };
        while (const Unit *const next = next_unit(ordinal + 1)) {
            const Unit &u = *next;
            ++ordinal;
            const int n = u.k1 - u.k0, k0 = u.k0;
            const bool wide = QT == 2 && u.rows > 128;
            const int in_unit = wide ? w * 128 + row : row;                  // this thread's row of the unit
            const int limit = row_limit(u.ctx, u.row0 + min(in_unit, u.rows - 1), a.group);
            // its slot's key tiles: first, step, end
            const int n0 = wide && w == 0 ? u.n0 : n;
            const int j0 = QT == 2 && !wide ? w : 0, step = QT == 2 && !wide ? 2 : 1;
            const bool idle = QT == 1 && w == 1;
            const int all_see = wide && w == 1 ? u.all1 : u.all0;            // keys that every row of the tile sees
            float m = -INFINITY, l = 0.f, factor = 0.f;
            bool first = true;
            for (int j = idle ? n0 : j0; j < n0; j += step) {
                const int slot = QT == 2 ? w : j & 1, acc = QT == 2 ? w : 0;
                wait(&s_full[slot], s_phase >> slot & 1);
                s_phase ^= 1u << slot;
                ok = __all_sync(~0u, ok);
                tc_fence_after();
                const uint32_t s_addr = lanes + slot * 128;
                if (first) {
                    factor = a.factor;
                    if constexpr (kScaledQ) factor *= __uint_as_float(static_cast<uint32_t>(
                        max(1, s_exp[(ordinal & 1) * 256 + (wide ? w * 128 : 0) + row] - 112 - 14 + 127)) << 23);
                    // (finite: a score of 0 stays 0)
                    factor = fminf(fmaxf(factor, kChunkMinFactor), FLT_MAX);
                }
                float s[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32) tc_ld32_async(s_addr + c, s + c);
                const int key0 = (k0 + j) * kChunkKeys;
#pragma unroll
                for (int c = 0; c < 128; c += 32) tc_wait_ld32(s + c);
                if (key0 + kChunkKeys > all_see) {
                    const int seen = limit - key0;
#pragma unroll
                    for (int c = 0; c < 128; c += 32) {
                        // a bit for each key of 32 that the row sees
                        const uint32_t bits = seen >= c + 32 ? ~0u : seen <= c ? 0u : (1u << (seen - c)) - 1;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(bits >> i & 1)) s[c + i] = -INFINITY;
                    }
                }
                float top[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) top[i] = fmaxf(s[i], s[i + 4]);
#pragma unroll
                for (int c = 8; c < 128; c += 8)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top[i] = max3(top[i], s[c + i], s[c + i + 4]);
                const float t = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * factor;
                // (row by row, so that a row's bits do not depend on its neighbours)
                const bool raise = t > m + kChunkLazy || (m == -INFINITY && t > -INFINITY);
                if (__any_sync(~0u, raise)) {
                    const float by = raise ? ex2(m - t) : 1.f;
                    m = raise ? t : m;
                    l *= by;
                    if (!first) {
                        // O so far is behind the product of the step before
                        if (QT == 1) {
                            wait(&o_done[last], (o_phase >> last & 1) ^ 1);
                            ok = __all_sync(~0u, ok);
                            tc_fence_after();
                        }
                        if (ok) {
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t o[16];
                                tc_ld16(lanes + G::kTmemO + acc * 128 + c, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
                                tc_st16(lanes + G::kTmemO + acc * 128 + c, o);
                            }
                        }
                    }
                }
                first = false;
                const float shift = m == -INFINITY ? 0.f : kRaise - m;
                const uint64_t f2 = pack_f2(factor, factor), c2 = pack_f2(shift, shift);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x, y;
                        unpack_f2(fma_f2(pack_f2(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), f2, c2), x, y);
                        x = ex2(x);
                        y = ex2(y);
                        p[i] = pack2<C>(x, y);
                        sum[i & 3] = add_f2(sum[i & 3], pack_f2(x, y));
                    }
                    tc_st16(s_addr + 16 * c, p);
                    if (c & 1) {
                        // the product may begin with the first half
                        tc_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&(c == 1 ? p_half : p_full)[slot]);
                    }
                }
                if (QT == 1) o_phase ^= 1u << slot;
                last = slot;
                float x, y;
                unpack_f2(add_f2(add_f2(sum[0], sum[1]), add_f2(sum[2], sum[3])), x, y);
                l += x + y;
            }
            // ---- the unit's output, or this block's piece of it
            const int acc = QT == 2 ? w : 0;
            const bool valid = in_unit < u.rows, cut = u.cut();
            const int my_row = u.row0 + (valid ? in_unit : u.rows - 1), G_ = a.group;
            if (!first) {
                if (QT == 2) o_phase ^= 1u << last;
                wait(&o_done[last], (o_phase >> last & 1) ^ 1);
                ok = __all_sync(~0u, ok);
            }
            tc_fence_after();
            const bool merge = QT == 2 && !wide, both_store = QT == 1 || merge;
            float w0 = 1.f, w1 = 0.f;                                        // weights of the two accumulators
            if (QT == 1) {
                // the other warpgroup stores half of the columns
                if (w == 0) s_ml[row] = make_float2(m, l);
                tc_fence_before();
                meet();
                tc_fence_after();
                m = s_ml[row].x;
                l = s_ml[row].y;
            }
            if (merge) {
                s_ml[w * 128 + row] = make_float2(m, l);
                tc_fence_before();
                meet();
                tc_fence_after();
                const float2 x = s_ml[row], y = s_ml[128 + row];
                m = fmaxf(x.x, y.x);
                const float ref = m == -INFINITY ? 0.f : m;
                w0 = ex2(x.x - ref);
                w1 = ex2(y.x - ref);
                l = x.y * w0 + y.y * w1;
            }
            if (ok) {
                const bool some = both_store ? n > 0 : !first;                    // an accumulator holds something
                float4 *const piece = reinterpret_cast<float4 *>(my_parts + (u.k0 > 0 ? 0 : 1) * chunk_piece_floats(DP) +
                                                                 (wide ? w : 0) * static_cast<int64_t>(chunk_piece_floats(DP) / QT));
                const float inv = l == 0.f ? 0.f : a.cache.v.scale / l;
                const uint32_t tok = static_cast<uint32_t>(my_row) / static_cast<uint32_t>(G_), g = my_row - tok * G_;
                const int64_t out_row = static_cast<int64_t>(u.q0) + tok, head = static_cast<int64_t>(u.h) * G_ + g;
                T *const out = static_cast<T *>(a.out.data) + out_row * a.out.token_stride + head * a.out.head_stride;
                const bool sectors = __all_sync(~0u, (reinterpret_cast<uintptr_t>(out) & 31) == 0);
                const bool guard = s_bad[ordinal & 3] == ordinal;            // values of V that are not finite were left out
                // one tile of rows: each warpgroup takes half of the columns
                const int c0 = both_store ? w * (DP / 2) : 0, c1 = both_store ? c0 + DP / 2 : DP;
#pragma unroll 1
                for (int c = c0; c < c1; c += 32) {
                    if (c >= D) break;
                    float o[32];
                    if (some) {
                        tc_ld32_async(lanes + G::kTmemO + (both_store ? 0 : acc * 128) + c, o);
                        tc_wait_ld32(o);
                        if (merge && n > 1) {
                            float o1[32];
                            tc_ld32_async(lanes + G::kTmemO + 128 + c, o1);
                            tc_wait_ld32(o1);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = o[i] * w0 + o1[i] * w1;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0.f;
                    }
                    if (guard) {
                        const uint32_t mask = valid ? not_finite_seen<T, FP8>(a, u, limit, c) : 0;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (mask >> i & 1) o[i] = __int_as_float(0x7FC00000);
                        __syncwarp();
                    }
                    if (cut) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            piece[((c + i) >> 2) * 128 + row] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    } else {
                        // 32 bytes of a row a lane: whole sectors, without the rows changing
                        // lanes (a transposition by shuffles took longer than it saved)
                        uint32_t r[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = pack2<T>(o[2 * i] * inv, o[2 * i + 1] * inv);
                        if (valid) {
#pragma unroll
                            for (int i = 0; i < 16; i += 8) {
                                if (c + 2 * i + 16 <= D && sectors) {
                                    st_v8(out + c + 2 * i, r + i);
                                } else {
                                    if (c + 2 * i < D) st_v4(out + c + 2 * i, r + i);
                                    if (c + 2 * i + 8 < D) st_v4(out + c + 2 * i + 8, r + i + 4);
                                }
                            }
                        }
                    }
                }
                if (!both_store || w == 0) {
                    if (cut) {
                        float *const ml = reinterpret_cast<float *>(piece) + 128 * DP;
                        ml[row] = m == -INFINITY ? m : m - kRaise;
                        ml[128 + row] = l;
                    } else if (valid && a.lse) {
                        a.lse[out_row * a.q_heads + head] = l == 0.f ? -INFINITY : (m - kRaise + log2f(l)) * kChunkLn2;
                    }
                }
            }
            if (both_store) {
                tc_fence_before();
                meet();
                tc_fence_after();
            }
            if (cut) {
                const int which = u.k0 > 0 ? 0 : 1;
                if (lane >> 4 == which) shared_unit = reinterpret_cast<const uint32_t *>(&u)[lane & 15];
                has_shared |= 1u << which;
                __threadfence();
                meet();
                if (warp == 0) {
                    int me, count;
                    const int begun = sharing_blocks(u, per_cta, lane, nullptr, me, count);
                    if (lane == 0 && ok) atomic_add_acq_rel(a.counters + 2 * begun, 1);
                }
            }
            __syncwarp();
            if (lane == 0) done_with(ordinal);
        }
        // ---- the cut units: each of the blocks that share one joins a part of it. It is a
        // chain of waits for L2: where the block has two, each warpgroup has one.
        meet();                                                              // (all tiles are read)
        if (has_shared) {
            // Shared memory is free once the last Q has come, too: nothing above waits for
            // that of a unit of which nothing is seen, the issuers do before they drain.
            wait(&drain[0], 0);
            if (QT == 2) wait(&drain[1], 0);
            ok = __all_sync(~0u, ok);
            const bool two = has_shared == 3;
            const int at_once = two ? 128 : 256, me_tid = two ? tid & 127 : tid;
            const int which = two ? w : has_shared >> 1;
            int16_t *const list = reinterpret_cast<int16_t *>(smem + G::oMl + (two ? w * 1024 : 0));   // [kChunkMaxCtas], then place, number, first
            Unit *const kept = reinterpret_cast<Unit *>(smem + G::oMl + (two ? w * 1024 : 0) + 512);
            // Those that join a unit meet; they wait longer than the one that waits for the
            // other blocks, which may be later by some part of what this block took itself.
            auto limit = [&]() { return a.timeout_ns + (global_timer_ns() - *s_start); };
            uint64_t *const joining = two ? &one[w] : both;
            uint32_t joined = two ? 0 : met;
            auto join_sync = [&]() {
                __syncwarp();
                if (lane == 0) mbar_arrive(joining);
                if (ok && !mbar_try_wait(joining, joined) && !mbar_wait_bounded(joining, joined, 2 * limit())) ok = false;
                joined ^= 1;
                ok = __all_sync(~0u, ok);
            };
            if (me_tid < 32) {
                if (lane >> 4 == which) reinterpret_cast<uint32_t *>(kept)[lane & 15] = shared_unit;
                __syncwarp();
                int me, count;
                const int begun = sharing_blocks(*kept, per_cta, lane, list, me, count);
                if (lane == 0) {
                    list[kChunkMaxCtas] = static_cast<int16_t>(me);
                    list[kChunkMaxCtas + 1] = static_cast<int16_t>(count);
                    list[kChunkMaxCtas + 2] = static_cast<int16_t>(begun);
                    bool late = false;                   // (not `ok`: this warp still meets the others)
                    if (ok && ld_acquire_gpu(a.counters + 2 * begun) < count) {
                        const uint64_t t0 = global_timer_ns(), most = limit();
                        while (!late && ld_acquire_gpu(a.counters + 2 * begun) < count) late = global_timer_ns() - t0 > most;
                    }
                    if (late) set_status(a.status, AWQ_ERR_DEVICE_TIMEOUT);
                    if (!ok || late) list[kChunkMaxCtas + 1] = 0;
                }
            }
            join_sync();
            const Unit v = *kept;
            // (after a time-out: no parts, and nothing to do but to meet)
            const int me = list[kChunkMaxCtas], count = ok ? list[kChunkMaxCtas + 1] : 0, begun = list[kChunkMaxCtas + 2];
            const int rows = count ? v.rows : 0, items = rows * (D / 8);
            const int lo = count ? static_cast<int>(static_cast<int64_t>(items) * me / count) : 0;
            const int hi = count ? static_cast<int>(static_cast<int64_t>(items) * (me + 1) / count) : 0;
            auto part = [&](int i, int r) {                                  // of the i-th block: row r's tile
                return a.parts + (static_cast<int64_t>(list[i]) * 2 + (i == 0 ? 1 : 0)) * chunk_piece_floats(DP) +
                       (r >> 7) * static_cast<int64_t>(chunk_piece_floats(DP) / QT);
            };
            // the parts' weights, a row a thread: [part][256], the second unit's from the
            // other end (all parts of both are no more than the blocks and one)
            static_assert((kChunkMaxCtas + 1) * 256 * sizeof(float) <= G::oMl, "weights of the parts");
            float *const weights = reinterpret_cast<float *>(smem + (two && w == 1 ? G::oMl - 1024 : 0));
            const int next_part = two && w == 1 ? -256 : 256;
            for (int r = me_tid; r < rows; r += at_once) {
                float top = -INFINITY, sum = 0.f;
#pragma unroll 4
                for (int i = 0; i < count; ++i) top = fmaxf(top, __ldcg(part(i, r) + 128 * DP + (r & 127)));
                const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll 4
                for (int i = 0; i < count; ++i) {
                    const float *const ml = part(i, r) + 128 * DP + (r & 127);
                    const float w = ex2(__ldcg(ml) - ref);
                    weights[i * next_part + r] = w;
                    sum += __ldcg(ml + 128) * w;
                }
                const float inv = sum == 0.f ? 0.f : a.cache.v.scale / sum;
                for (int i = 0; i < count; ++i) weights[i * next_part + r] *= inv;
                if (me == 0 && a.lse) {
                    const uint32_t at = v.row0 + r, tok = at / static_cast<uint32_t>(a.group), g = at - tok * a.group;
                    a.lse[(static_cast<int64_t>(v.q0) + tok) * a.q_heads + static_cast<int64_t>(v.h) * a.group + g] =
                        sum == 0.f ? -INFINITY : (top + log2f(sum)) * kChunkLn2;
                }
            }
            join_sync();
            constexpr int IT = 4;                                            // items of a thread at a time
#pragma unroll 1
            for (int base = lo + me_tid; base < hi; base += IT * at_once) {
                float f[IT][8];
#pragma unroll
                for (int k = 0; k < IT; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[k][e] = 0.f;
#pragma unroll 1
                for (int i = 0; i < count; ++i) {
                    float4 x[IT], y[IT];
#pragma unroll
                    for (int k = 0; k < IT; ++k) {
                        const int item = min(base + k * at_once, hi - 1), chunk = item / rows, r = item - chunk * rows;
                        const float4 *const p = reinterpret_cast<const float4 *>(part(i, r)) + 2 * chunk * 128 + (r & 127);
                        x[k] = __ldcg(p);
                        y[k] = __ldcg(p + 128);
                    }
#pragma unroll
                    for (int k = 0; k < IT; ++k) {
                        const int item = min(base + k * at_once, hi - 1), r = item % rows;
                        const float by = weights[i * next_part + r];
                        const float z[8] = {x[k].x, x[k].y, x[k].z, x[k].w, y[k].x, y[k].y, y[k].z, y[k].w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[k][e] += z[e] * by;
                    }
                }
#pragma unroll
                for (int k = 0; k < IT; ++k) {
                    const int item = base + k * at_once;
                    if (item >= hi) break;
                    const int chunk = item / rows, r = item - chunk * rows;
                    const uint32_t at = v.row0 + r, tok = at / static_cast<uint32_t>(a.group), g = at - tok * a.group;
                    const int64_t out_row = static_cast<int64_t>(v.q0) + tok, head = static_cast<int64_t>(v.h) * a.group + g;
                    store_elems<T, 8>(static_cast<T *>(a.out.data) + out_row * a.out.token_stride + head * a.out.head_stride + 8 * chunk, f[k]);
                }
            }
            // the last block to leave makes the counters ready for the next call
            join_sync();
            if (me_tid == 0 && count && atomic_add_acq_rel(a.counters + 2 * begun + 1, 1) == count - 1) {
                a.counters[2 * begun] = 0;
                a.counters[2 * begun + 1] = 0;
            }
        }
    }
    if (!ok) set_status(a.status, AWQ_ERR_DEVICE_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tc_dealloc(tmem, 512);
}

// A plane as [page][head][token of a page][element], boxes of `box` tokens.
template <bool FP8, int DP>
bool plane_map(CUtensorMap *m, const ChunkArgs &a, const awq_kv_plane &p)
{
    const cuuint64_t elem = FP8 ? 1 : 2;
    const bool paged = a.page_table;
    // (a stride that is not used or 0 makes its dimension one)
    const auto dim = [](int64_t n, int64_t stride) { return static_cast<cuuint64_t>(stride ? n : 1); };
    const auto bytes = [&](int64_t stride) { return static_cast<cuuint64_t>(stride ? stride * elem : 16); };
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.cache.head_dim), dim(paged ? a.cache.page_size : a.tokens, p.token_stride),
                                dim(a.cache.num_heads, p.head_stride), dim(paged ? a.cache.num_pages : 1, p.page_stride)};
    const cuuint64_t strides[3] = {bytes(p.token_stride), bytes(p.head_stride), bytes(p.page_stride)};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(FP8 ? ChunkGeo<DP, FP8>::SC : 64), static_cast<cuuint32_t>(a.box), 1, 1};
    return encode_tensor_map(m, FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, p.data, dims, strides, box,
                             FP8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

template <typename T, bool FP8, int DP>
awq_status launch_chunk_d(const ChunkArgs &a, int sms, cudaStream_t st)
{
    CUtensorMap map_k, map_v, map_q{};
    if (!plane_map<FP8, DP>(&map_k, a, a.cache.k) || !plane_map<FP8, DP>(&map_v, a, a.cache.v)) return AWQ_ERR_CUDA;
    if (a.q_box && !(FP8 && !std::is_same<T, __half>::value)) {
        const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.cache.head_dim), static_cast<cuuint64_t>(a.q_heads), static_cast<cuuint64_t>(a.tokens)};
        const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.q_heads > 1 ? a.q.head_stride * 2 : 16),
                                       static_cast<cuuint64_t>(a.tokens > 1 ? a.q.token_stride * 2 : 16)};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.group), static_cast<cuuint32_t>(a.q_box)};
        if (!encode_tensor_map(&map_q, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, a.q.data, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
            return AWQ_ERR_CUDA;
    }
    const awq_status r = set_smem(chunk_attn_kernel<T, FP8, DP>, ChunkGeo<DP, FP8>::kSmem);
    if (r) return r;
    const int grid = sms < kChunkMaxCtas ? sms : kChunkMaxCtas;
    return launch_ex(chunk_attn_kernel<T, FP8, DP>, dim3(grid), dim3(ChunkGeo<DP, FP8>::kThreads), ChunkGeo<DP, FP8>::kSmem, 1, true, st, map_k, map_v, map_q, a);
}

template <typename T, bool FP8>
awq_status launch_chunk(const ChunkArgs &a, int sms, cudaStream_t st)
{
    const int dp = attn_padded_dim(a.cache.head_dim);
    return dp == 64    ? launch_chunk_d<T, FP8, 64>(a, sms, st)
           : dp == 128 ? launch_chunk_d<T, FP8, 128>(a, sms, st)
                       : launch_chunk_d<T, FP8, 256>(a, sms, st);
}

}  // namespace

}  // namespace awq
