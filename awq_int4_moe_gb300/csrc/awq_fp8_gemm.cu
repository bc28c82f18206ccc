// awq_fp8_gemm: out = sum over 128-blocks j of K of
//   a_scales[m][j] b_scales[n / 128][j] (a[m][j-block] . b[n][j-block]),
// e4m3 operands on the 5th-generation tensor cores (tcgen05 kind::f8f6f4).
//
// The tensor core multiplies one K block of 128 at a time (four K = 32
// instructions) into one of several fp32 accumulators in tensor memory; the
// epilogue warps read it back, multiply by the block's scale and add it to
// fp32 registers while the next ones are filled, so a block's scale is applied
// exactly once and the sums stay in fp32.
//
// One operand's 128 rows are the UMMA M side, TN rows of the other its N side:
//   few tokens (SWAP): weights on the M side, so that a tile of 16 tokens wastes
//     no tensor-core rows on padding and the weights, which are the bytes, stream
//     in full 128-row boxes; a lane of tensor memory is an output column, a
//     column a token, whose scale is read from shared memory;
//   many tokens: tokens on the M side, 128 or 256 weight rows on the N side; a
//     lane is a token, and each epilogue warp's 64 columns share one weight
//     scale, so the factor is one register.
// Where the tiles do not fill the card, a cluster of CS blocks shares a tile: each
// takes a part of K, the partial sums meet in distributed shared memory and are
// added in block order.
//
// Warps: the epilogue ones first (a warp reads the tensor-memory lanes 32 (w
// mod 4) ..), then the producer (TMA boxes of 128 bytes of K, 128-byte swizzle),
// then the MMA issuer; they meet at mbarriers, every wait is bounded.
//
// Bound: few tokens by the weights' bytes (1 x 16384 x 16384: 43.3 us, 6.2
// TB/s), or by start and cluster sum where those are few (1 x 3584 x 2560: 4.4
// us); many tokens by the accumulators' hand-over (8192 x 5120 x 8192: 326 us,
// 2,110 TFLOP/s; the same products without it 216 us, 3,180 TFLOP/s).
#include <algorithm>
#include <atomic>

#include "awq_decoder_kernels.cuh"
#include "awq_launch.cuh"
#include "awq_tc.cuh"

namespace awq {

namespace {

constexpr int kTM = 128;                    // rows of the UMMA M side
constexpr int kKB = 128;                    // bytes of a K block
constexpr int kRasterRows = 16;             // token tiles that a band of the tile order spans

template <int TN, bool SWAP>
struct GemmGeo {
    static constexpr int kDepth = TN == 256 ? 2 : 4;             // accumulators in tensor memory
    static constexpr int kCols = TN < 64 ? TN : 64;              // columns of an epilogue warp
    static constexpr int kEpiWarps = 4 * (TN / kCols);
    static constexpr int kThreads = (kEpiWarps + 2) * 32;
    static constexpr int kA = kTM * kKB, kB = TN * kKB, kStage = kA + kB;
    // two blocks per multiprocessor where the tile is small
    static constexpr int kBlocks = TN <= 64 ? 2 : 1;
    static constexpr int kStages = (kBlocks == 2 ? 104 : 192) * 1024 / kStage;
    static constexpr int kTmemCols = kDepth * TN < 32 ? 32 : kDepth * TN;
    static constexpr int kFactors = SWAP ? kEpiWarps * 2 * TN * 4 : 0;
    static constexpr int kOut = SWAP ? 0 : kEpiWarps * 2048;     // 32 rows of 32 columns per epilogue warp
    static constexpr int kBars = 2 * kStages + 2 * kDepth + 1;
    static constexpr int kSmem = 1024 + kStages * kStage + kFactors + kOut + kBars * 8 + 16;
    // partial sums of a cluster's blocks, over the operand stages
    static constexpr int kPartRow = SWAP ? kTM : TN + 4;
    static_assert((SWAP ? TN : kTM) * kPartRow * 4 <= kStages * kStage || TN == 256, "partial sums fit");
};

__device__ __forceinline__ void tc_mma_f8(uint32_t tmem, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 columns of the warp's 32 lanes; complete after tc_wait_ld().
__device__ __forceinline__ void tc_ld16_async(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// Waits for the loads; the registers pass through so that no use of them is
// moved above the wait.
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// Pairs of fp32 values in one 64-bit register: acc += (a, b) * f.
__device__ __forceinline__ uint64_t pair(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ void fma2(uint64_t &acc, uint32_t a, uint32_t b, uint64_t f)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(a), "r"(b));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(d), "l"(f));
}

// Tile `t` of token tiles x weight tiles, in bands of kRasterRows token tiles
// (weight tile by weight tile within a band), so that the blocks at work share
// operands in L2.
__device__ __forceinline__ int2 tile_at(int t, int m_tiles, int n_tiles)
{
    const int band = t / (kRasterRows * n_tiles);
    const int rows = min(kRasterRows, m_tiles - band * kRasterRows);
    const int in = t - band * kRasterRows * n_tiles;
    return make_int2(band * kRasterRows + in % rows, in / rows);
}

template <typename T, int TN, bool SWAP>
__global__ void __launch_bounds__(GemmGeo<TN, SWAP>::kThreads, GemmGeo<TN, SWAP>::kBlocks)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_m, const __grid_constant__ CUtensorMap map_n, const GemmArgs p,
                int cluster)
{
    using G = GemmGeo<TN, SWAP>;
    constexpr int EW = G::kEpiWarps, NC = G::kCols;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    float *factors = reinterpret_cast<float *>(smem + G::kStages * G::kStage);
    uint8_t *const out_space = smem + G::kStages * G::kStage + G::kFactors;
    uint64_t *full = reinterpret_cast<uint64_t *>(out_space + G::kOut);
    uint64_t *empty = full + G::kStages;
    uint64_t *acc_full = empty + G::kStages;          // [depth]
    uint64_t *acc_empty = acc_full + G::kDepth;       // [depth]
    uint64_t *drain = acc_empty + G::kDepth;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < G::kDepth; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], EW);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
        prefetch_tmap(&map_m);
        prefetch_tmap(&map_n);
    }
    if (warp == 0) tc_alloc(tmem_slot, G::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();
    grid_launch_dependents();

    // rows of the M side and of the N side, and the tiles of both
    const int rows_m = SWAP ? p.N : p.M, rows_n = SWAP ? p.M : p.N;
    const int tiles_m = (rows_m + kTM - 1) / kTM, tiles_n = (rows_n + TN - 1) / TN;
    const int tiles = tiles_m * tiles_n;
    const int KB = (p.K + kKB - 1) / kKB;
    const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int kb0 = static_cast<int>(static_cast<int64_t>(KB) * rank / cluster);
    const int kb1 = static_cast<int>(static_cast<int64_t>(KB) * (rank + 1) / cluster);
    const int tile0 = blockIdx.x / cluster, tile_step = gridDim.x / cluster;    // one tile each where cluster > 1

    if (warp == EW) {
        // ---------------- producer ----------------
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int t = tile0; ok && t < tiles; t += tile_step) {
                const int2 tl = tile_at(t, tiles_m, tiles_n);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % G::kStages;
                    if (it >= G::kStages && !mbar_wait_bounded(&empty[s], ((it / G::kStages) + 1) & 1, p.timeout_ns)) {
                        set_status(p.status, AWQ_ERR_DEVICE_TIMEOUT);
                        ok = false;
                        break;
                    }
                    uint8_t *dst = smem + s * G::kStage;
                    mbar_arrive_expect_tx(&full[s], G::kStage);
                    tma_load_2d(dst, &map_m, &full[s], kb * kKB, tl.x * kTM);
                    tma_load_2d(dst + G::kA, &map_n, &full[s], kb * kKB, tl.y * TN);
                }
            }
            // after a time-out: the copies in flight end before the block does
            if (!ok)
                for (int i = std::max(0, it - G::kStages); i < it; ++i)
                    mbar_wait_bounded(&full[i % G::kStages], (i / G::kStages) & 1, p.timeout_ns);
        }
    } else if (warp == EW + 1) {
        // ---------------- MMA issuer ----------------
        if (lane == 0) {
            constexpr uint32_t idesc = umma_idesc_f16(kTM, TN);      // e4m3 x e4m3 -> fp32 has the same fields
            int it = 0;
            bool ok = true;
            for (int t = tile0; ok && t < tiles; t += tile_step) {
                for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                    const int s = it % G::kStages, buf = it % G::kDepth;
                    if (!mbar_wait_bounded(&full[s], (it / G::kStages) & 1, p.timeout_ns)) ok = false;
                    const uint32_t at = smem_u32(smem + s * G::kStage);
                    const uint64_t da = umma_desc_sw128(at);
                    if (ok && it >= G::kDepth &&
                        !mbar_wait_bounded(&acc_empty[buf], ((it / G::kDepth) + 1) & 1, p.timeout_ns))
                        ok = false;
                    if (ok) {
                        tc_fence_after();
                        const uint64_t db = umma_desc_sw128(at + G::kA);
#pragma unroll
                        for (int k = 0; k < 4; ++k) tc_mma_f8(tmem + buf * TN, da + 2 * k, db + 2 * k, idesc, k > 0);
                        tc_commit(&empty[s]);
                        tc_commit(&acc_full[buf]);
                    }
                }
            }
            if (!ok) set_status(p.status, AWQ_ERR_DEVICE_TIMEOUT);
            if (!ok) {
                tc_commit(drain);
                mbar_wait_bounded(drain, 0, p.timeout_ns);
            }
        }
    } else {
        // ---------------- epilogue ----------------
        const int quarter = warp & 3, col0 = (warp >> 2) * NC;       // tensor-memory lanes, first column
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + col0;
        const int l = quarter * 32 + lane;                           // this thread's row of the M side
        float *fac = factors + warp * 2 * TN;
        // 0, which the compiler does not see: barrier addresses that it knows
        // to be uniform go through the uniform registers, whose latency is on
        // the path of every K block (M 8192, N 5120, K 8192: 344 us against 326)
        const int none = col0 / TN;
        int it = 0;
        bool ok = true;
        for (int t = tile0; ok && t < tiles; t += tile_step) {
            const int2 tl = tile_at(t, tiles_m, tiles_n);
            const int m0 = tl.x * kTM, n0 = tl.y * TN;
            uint64_t acc[NC / 2];                                    // pairs of columns
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) acc[i] = 0;
            // the scales of the next K block
            const float *wb = p.b_scales + static_cast<int64_t>((SWAP ? m0 : min(n0 + col0, p.N - 1)) / AWQ_FP8_BLOCK) * KB;
            constexpr int F = SWAP ? (TN + 31) / 32 : 1;
            float next[F];
            auto fetch = [&](int kb) {
                const float w = wb[kb];
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    const int tok = SWAP ? n0 + lane + 32 * i : m0 + l;
                    next[i] = tok < p.M && (TN >= 32 || !SWAP || lane < TN)
                                  ? p.a_scales[static_cast<int64_t>(tok) * KB + kb] * w
                                  : 0.f;
                }
            };
            fetch(kb0);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int buf = it % G::kDepth, bar = buf + none;
                const uint64_t mine = pair(next[0], next[0]);
                float *const fb = fac + (it & 1) * TN;
                if constexpr (SWAP) {
#pragma unroll
                    for (int i = 0; i < F; ++i)
                        if (TN >= 32 || lane < TN) fb[lane + 32 * i] = next[i];
                    __syncwarp();
                }
                if (kb + 1 < kb1) fetch(kb + 1);
                if (!mbar_wait_bounded(&acc_full[bar], (it / G::kDepth) & 1, p.timeout_ns)) {
                    if (lane == 0) set_status(p.status, AWQ_ERR_DEVICE_TIMEOUT);
                    ok = false;
                }
                if (!__all_sync(~0u, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t d[2][16];
                tc_ld16_async(taddr + buf * TN, d[0]);
#pragma unroll
                for (int c = 0; c < NC / 16; ++c) {
                    tc_wait_ld(d[c & 1]);
                    if (c + 1 < NC / 16) tc_ld16_async(taddr + buf * TN + (c + 1) * 16, d[(c + 1) & 1]);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        uint64_t f0 = mine, f1 = mine;
                        if constexpr (SWAP) {
                            const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(fb + c * 16 + i);
                            f0 = f.x;
                            f1 = f.y;
                        }
                        fma2(acc[c * 8 + i / 2], d[c & 1][i], d[c & 1][i + 1], f0);
                        fma2(acc[c * 8 + i / 2 + 1], d[c & 1][i + 2], d[c & 1][i + 3], f1);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[bar]);
            }
            if (!ok) break;
            T *out = static_cast<T *>(p.out);
            if (cluster > 1) {
                // this block's part of the sum, over the operand stages: every
                // copy into them has been consumed
                float *part = reinterpret_cast<float *>(smem);
#pragma unroll
                for (int i = 0; i < NC; i += 4) {
                    const float2 x = unpair(acc[i / 2]), y = unpair(acc[i / 2 + 1]);
                    if constexpr (SWAP) {
                        part[(col0 + i) * G::kPartRow + l] = x.x;
                        part[(col0 + i + 1) * G::kPartRow + l] = x.y;
                        part[(col0 + i + 2) * G::kPartRow + l] = y.x;
                        part[(col0 + i + 3) * G::kPartRow + l] = y.y;
                    } else {
                        *reinterpret_cast<float4 *>(part + l * G::kPartRow + col0 + i) = make_float4(x.x, x.y, y.x, y.y);
                    }
                }
            } else if constexpr (SWAP) {
                const int n = m0 + l;
                if (n < p.N)
#pragma unroll
                    for (int i = 0; i < NC; i += 2) {
                        const float2 x = unpair(acc[i / 2]);
                        const int tok = n0 + col0 + i;
                        if (tok < p.M) out[static_cast<int64_t>(tok) * p.ldo + n] = from_f32<T>(x.x);
                        if (tok + 1 < p.M) out[static_cast<int64_t>(tok + 1) * p.ldo + n] = from_f32<T>(x.y);
                    }
            } else {
                // through shared memory, 32 columns at a time, so that
                // neighbouring lanes store neighbouring columns
                uint8_t *const space = out_space + warp * 2048;
                const int m = m0 + quarter * 32, n = n0 + col0;
                const bool wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0 && p.ldo % 8 == 0;
#pragma unroll
                for (int c = 0; c < NC / 32; ++c) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 x = unpair(acc[c * 16 + j * 4 + i]);
                            w[i] = pack2<T>(x.x, x.y);
                        }
                        *reinterpret_cast<uint4 *>(space + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = 8 * j + (lane >> 2), q = lane & 3, col = n + 32 * c + 8 * q;
                        const uint4 v = *reinterpret_cast<const uint4 *>(space + r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
                        if (m + r >= p.M || col >= p.N) continue;
                        T *dst = out + static_cast<int64_t>(m + r) * p.ldo + col;
                        if (wide && col + 8 <= p.N) {
                            *reinterpret_cast<uint4 *>(dst) = v;
                        } else {
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (col + i < p.N)
                                    reinterpret_cast<uint16_t *>(dst)[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
                        }
                    }
                    __syncwarp();
                }
            }
        }
    }

    if (cluster > 1) {
        __syncwarp();
        cluster_sync();
        // block `rank` adds its share of the tile from every block, in order
        const int2 tl = tile_at(tile0, tiles_m, tiles_n);
        const int m0 = tl.x * kTM, n0 = tl.y * TN;
        const float *part = reinterpret_cast<const float *>(smem);
        T *out = static_cast<T *>(p.out);
        // SWAP: rows of the partial sums are tokens; else M-side rows, also tokens
        constexpr int kRows = SWAP ? TN : kTM, kRow4 = (SWAP ? kTM : TN) / 4;
        const int tok0 = SWAP ? n0 : m0, col_base = SWAP ? m0 : n0;
        const int rows = min(kRows, p.M - tok0), r0 = rows * rank / cluster, r1 = rows * (rank + 1) / cluster;
        for (int i = tid; i < (r1 - r0) * kRow4; i += G::kThreads) {
            const int r = r0 + i / kRow4, c = i % kRow4 * 4, n = col_base + c;
            if (n >= p.N) continue;      // nothing is read that no store needs: see the barrier below
            // all blocks' values on their way together, then added in block order
            float4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < cluster) v[k] = ld_shared_cluster_f4(map_shared_rank(part + r * G::kPartRow + c, k));
            float4 sum = v[0];
#pragma unroll
            for (int k = 1; k < 8; ++k)
                if (k < cluster) {
                    sum.x += v[k].x;
                    sum.y += v[k].y;
                    sum.z += v[k].z;
                    sum.w += v[k].w;
                }
            T *dst = out + static_cast<int64_t>(tok0 + r) * p.ldo + n;
            if (n + 4 <= p.N && (reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
                *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(sum.x, sum.y), pack2<T>(sum.z, sum.w));
            } else {
                const float f[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < p.N) dst[j] = from_f32<T>(f[j]);
            }
        }
        // no block leaves while its sums are read; all that this warp reads has
        // arrived (the stores above took it), and it has written nothing that
        // the others wait for
        __syncwarp();
        cluster_arrive_relaxed();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tc_dealloc(tmem, G::kTmemCols);
    if (cluster > 1) {
        __syncwarp();
        cluster_wait();
    }
}

bool make_map(CUtensorMap *m, const uint8_t *base, int64_t ld, int rows, int K, int box_rows)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t str[1] = {static_cast<cuuint64_t>(ld)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kKB), static_cast<cuuint32_t>(box_rows)};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// Clusters of `size` blocks that the device holds at once, one block on a
// multiprocessor (looked up once per device and size: a property of the device
// and the kernel).
template <typename T, int TN, bool SWAP>
int resident_clusters(int size)
{
    using G = GemmGeo<TN, SWAP>;
    static std::atomic<int> known[64][9] = {};       // count + 1
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
    if (dev < 64)
        if (const int n = known[dev][size].load(std::memory_order_relaxed)) return n - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(G::kThreads);
    cfg.dynamicSmemBytes = G::kSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fp8_gemm_kernel<T, TN, SWAP>, &cfg) != cudaSuccess) return 0;
    if (dev < 64) known[dev][size].store(n + 1, std::memory_order_relaxed);
    return n;
}

template <typename T, int TN, bool SWAP>
awq_status launch_gemm_tile(const GemmArgs &g, const uint8_t *a, int64_t lda, const uint8_t *b, int64_t ldb, int sms,
                            cudaStream_t st)
{
    using G = GemmGeo<TN, SWAP>;
    CUtensorMap mm, mn;
    if (!make_map(&mm, SWAP ? b : a, SWAP ? ldb : lda, SWAP ? g.N : g.M, g.K, kTM) ||
        !make_map(&mn, SWAP ? a : b, SWAP ? lda : ldb, SWAP ? g.M : g.N, g.K, TN))
        return AWQ_ERR_CUDA;
    const int64_t tiles = static_cast<int64_t>(((SWAP ? g.N : g.M) + kTM - 1) / kTM) * (((SWAP ? g.M : g.N) + TN - 1) / TN);
    if (tiles > 0x3fffffff) return AWQ_ERR_UNSUPPORTED_SHAPE;
    const int KB = (g.K + kKB - 1) / kKB;
    const awq_status r = set_smem(fp8_gemm_kernel<T, TN, SWAP>, G::kSmem);
    if (r) return r;
    // Blocks per tile: as many, up to 8, as still run all at once with one block
    // per multiprocessor (one token, N = 3584, K = 2560, 28 tiles: 9.1 us with 1,
    // 4.4 with 5, 5.2 with 8), or with kBlocks of them where that gives fewer
    // than 4 (64 tokens, N = K = 5120, 40 tiles: 10.2 us with 3, 9.3 with 6; 7 do
    // not all fit: 15.7).
    int cluster = 1;
    if (TN < 256) {
        auto most = [&](int blocks) {
            int n = std::min(KB, 8);
            while (n > 1 && tiles > blocks * resident_clusters<T, TN, SWAP>(n)) --n;
            return n;
        };
        cluster = most(1);
        if (cluster < 4 && G::kBlocks > 1) cluster = most(G::kBlocks);
    }
    const int grid = cluster > 1 ? static_cast<int>(tiles) * cluster
                                 : static_cast<int>(std::min<int64_t>(tiles, sms * G::kBlocks));
    return launch(fp8_gemm_kernel<T, TN, SWAP>, dim3(grid), dim3(G::kThreads), G::kSmem, cluster, st, mm, mn, g, cluster);
}

template <typename T>
awq_status launch_gemm_t(const GemmArgs &g, const uint8_t *a, int64_t lda, const uint8_t *b, int64_t ldb, int sms,
                         cudaStream_t st)
{
    if (g.M <= 16) return launch_gemm_tile<T, 16, true>(g, a, lda, b, ldb, sms, st);
    if (g.M <= 32) return launch_gemm_tile<T, 32, true>(g, a, lda, b, ldb, sms, st);
    if (g.M <= 64) return launch_gemm_tile<T, 64, true>(g, a, lda, b, ldb, sms, st);
    // Tiles of 128 x 256 take 3 / 2 of the time of tiles of 128 x 128 (the
    // accumulators' hand-over costs as much as half of the products), so they
    // win where they save a third of the rounds: M 512, N = K = 5120: 26 us
    // against 35; M 1024, N 5120, K 2560: 30 against 28; M 4096: 65 against 78.
    const int64_t mt = (g.M + 127) / 128, nt = (g.N + 127) / 128, nt2 = (g.N + 255) / 256;
    if (3 * ((mt * nt2 + sms - 1) / sms) < 2 * ((mt * nt + sms - 1) / sms))
        return launch_gemm_tile<T, 256, false>(g, a, lda, b, ldb, sms, st);
    return launch_gemm_tile<T, 128, false>(g, a, lda, b, ldb, sms, st);
}

}  // namespace

awq_status launch_fp8_gemm(const GemmArgs &g, const uint8_t *a, int64_t lda, const uint8_t *b, int64_t ldb, int dtype,
                           int sms, cudaStream_t st)
{
    return dtype == AWQ_DTYPE_F16 ? launch_gemm_t<__half>(g, a, lda, b, ldb, sms, st)
                                  : launch_gemm_t<__nv_bfloat16>(g, a, lda, b, ldb, sms, st);
}

}  // namespace awq
