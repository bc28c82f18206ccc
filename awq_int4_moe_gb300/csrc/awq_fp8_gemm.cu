// awq_fp8_gemm: out = sum over 128-blocks j of K of
//   a_scales[m][j] b_scales[n / 128][j] (a[m][j-block] . b[n][j-block]),
// e4m3 operands on the 5th-generation tensor cores (tcgen05 kind::f8f6f4).
//
// The tensor core multiplies one K block of 128 at a time (four K = 32
// instructions) into one of two fp32 accumulators in tensor memory; the
// epilogue warps read it back, multiply by the block's scale and add it to
// fp32 registers while the other accumulator is filled, so a block's scale is
// applied exactly once and the sums stay in fp32.
//
// One operand's 128 rows are the UMMA M side, TN rows of the other its N side:
//   few tokens (SWAP): weights on the M side, so that a tile of 16 tokens wastes
//     no tensor-core rows on padding and the weights, which are the bytes, stream
//     in full 128-row boxes; a lane of tensor memory is an output column, a
//     column a token, whose scale is read from shared memory;
//   many tokens: tokens on the M side, 128 or 256 weight rows on the N side; a
//     lane is a token, and each epilogue warp's 128 columns share one weight
//     scale, so the factor is one register.
// Where the tiles do not fill the card, a cluster of CS blocks shares a tile: each
// takes a part of K, the partial sums meet in distributed shared memory and are
// added in block order.
//
// Warps: the epilogue ones first (a warp reads the tensor-memory lanes 32 (w
// mod 4) ..), then the producer (TMA boxes of 128 bytes of K, 128-byte swizzle),
// then the MMA issuer; they meet at mbarriers, every wait is bounded.
#include <algorithm>

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
    static constexpr int kCols = TN < 64 ? TN : 64;              // accumulator columns of an epilogue warp
    static constexpr int kEpiWarps = 4 * (TN / kCols);
    static constexpr int kThreads = (kEpiWarps + 2) * 32;
    static constexpr int kA = kTM * kKB, kB = TN * kKB, kStage = kA + kB;
    // two blocks per multiprocessor where the tile is small
    static constexpr int kBlocks = TN <= 64 ? 2 : 1;
    static constexpr int kStages = (kBlocks == 2 ? 104 : 200) * 1024 / kStage;
    static constexpr int kTmemCols = 2 * TN < 32 ? 32 : 2 * TN;
    static constexpr int kFactors = SWAP ? kEpiWarps * 2 * TN * 4 : 0;
    static constexpr int kBars = 2 * kStages + 5;
    static constexpr int kSmem = 1024 + kStages * kStage + kFactors + kBars * 8 + 16;
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

// (x, y) += (a, b) * (s, t)
__device__ __forceinline__ void fma2(float &x, float &y, uint32_t a, uint32_t b, float s, float t)
{
    uint64_t acc, d, f;
    asm("mov.b64 %0, {%1, %2};" : "=l"(acc) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(a), "r"(b));
    asm("mov.b64 %0, {%1, %2};" : "=l"(f) : "f"(s), "f"(t));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(d), "l"(f));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(acc));
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
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + G::kStages * G::kStage + G::kFactors);
    uint64_t *empty = full + G::kStages;
    uint64_t *acc_full = empty + G::kStages;          // [2]
    uint64_t *acc_empty = acc_full + 2;               // [2]
    uint64_t *drain = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
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
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % G::kStages, buf = it & 1;
                    if ((it >= 2 && !mbar_wait_bounded(&acc_empty[buf], ((it >> 1) + 1) & 1, p.timeout_ns)) ||
                        !mbar_wait_bounded(&full[s], (it / G::kStages) & 1, p.timeout_ns)) {
                        set_status(p.status, AWQ_ERR_DEVICE_TIMEOUT);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = smem_u32(smem + s * G::kStage);
                    const uint64_t da = umma_desc_sw128(at), db = umma_desc_sw128(at + G::kA);
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc_mma_f8(tmem + buf * TN, da + 2 * k, db + 2 * k, idesc, k > 0);
                    tc_commit(&empty[s]);
                    tc_commit(&acc_full[buf]);
                }
            }
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
        int it = 0;
        bool ok = true;
        for (int t = tile0; ok && t < tiles; t += tile_step) {
            const int2 tl = tile_at(t, tiles_m, tiles_n);
            const int m0 = tl.x * kTM, n0 = tl.y * TN;
            float acc[NC];
#pragma unroll
            for (int i = 0; i < NC; ++i) acc[i] = 0.f;
            // the scales of the next K block
            const float *wb = p.b_scales + static_cast<int64_t>((SWAP ? m0 : min(n0 + col0, p.N - 1)) / AWQ_FP8_BLOCK) * KB;
            constexpr int F = SWAP ? (TN + 31) / 32 : 1;
            float next[F];
            auto fetch = [&](int kb) {
                const float w = __ldg(wb + kb);
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    const int tok = SWAP ? n0 + lane + 32 * i : m0 + l;
                    next[i] = tok < p.M && (TN >= 32 || !SWAP || lane < TN)
                                  ? __ldg(p.a_scales + static_cast<int64_t>(tok) * KB + kb) * w
                                  : 0.f;
                }
            };
            fetch(kb0);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int buf = it & 1;
                const float mine = next[0];
                if constexpr (SWAP) {
#pragma unroll
                    for (int i = 0; i < F; ++i)
                        if (TN >= 32 || lane < TN) fac[buf * TN + lane + 32 * i] = next[i];
                    __syncwarp();
                }
                if (kb + 1 < kb1) fetch(kb + 1);
                if (!mbar_wait_bounded(&acc_full[buf], (it >> 1) & 1, p.timeout_ns)) {
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
                        float4 f = make_float4(mine, mine, mine, mine);
                        if constexpr (SWAP) f = *reinterpret_cast<const float4 *>(fac + buf * TN + c * 16 + i);
                        fma2(acc[c * 16 + i], acc[c * 16 + i + 1], d[c & 1][i], d[c & 1][i + 1], f.x, f.y);
                        fma2(acc[c * 16 + i + 2], acc[c * 16 + i + 3], d[c & 1][i + 2], d[c & 1][i + 3], f.z, f.w);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[buf]);
            }
            if (!ok) break;
            T *out = static_cast<T *>(p.out);
            if (cluster > 1) {
                // this block's part of the sum, over the operand stages: every
                // copy into them has been consumed
                float *part = reinterpret_cast<float *>(smem);
                if constexpr (SWAP) {
#pragma unroll
                    for (int i = 0; i < NC; ++i) part[i * G::kPartRow + l] = acc[i];
                } else {
#pragma unroll
                    for (int i = 0; i < NC; i += 4)
                        *reinterpret_cast<float4 *>(part + l * G::kPartRow + col0 + i) =
                            make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
                }
            } else if constexpr (SWAP) {
                const int n = m0 + l;
                if (n < p.N)
#pragma unroll
                    for (int i = 0; i < NC; ++i)
                        if (n0 + i < p.M) out[static_cast<int64_t>(n0 + i) * p.ldo + n] = from_f32<T>(acc[i]);
            } else {
                const int m = m0 + l, n = n0 + col0;
                if (m < p.M && n < p.N) {
                    T *row = out + static_cast<int64_t>(m) * p.ldo + n;
                    if (n + NC <= p.N && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {
#pragma unroll
                        for (int i = 0; i < NC; i += 8)
                            *reinterpret_cast<uint4 *>(row + i) =
                                make_uint4(pack2<T>(acc[i], acc[i + 1]), pack2<T>(acc[i + 2], acc[i + 3]),
                                           pack2<T>(acc[i + 4], acc[i + 5]), pack2<T>(acc[i + 6], acc[i + 7]));
                    } else {
#pragma unroll
                        for (int i = 0; i < NC; ++i)
                            if (n + i < p.N) row[i] = from_f32<T>(acc[i]);
                    }
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
        const int r0 = kRows * rank / cluster, r1 = min(kRows * (rank + 1) / cluster, p.M - tok0);
        for (int i = tid; i < (r1 - r0) * kRow4; i += G::kThreads) {
            const int r = r0 + i / kRow4, c = i % kRow4 * 4;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < cluster; ++k) {
                const float4 v = ld_shared_cluster_f4(map_shared_rank(part + r * G::kPartRow + c, k));
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
            }
            const int n = col_base + c;
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
        cluster_sync();                  // no block leaves while its sums are read
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tc_dealloc(tmem, G::kTmemCols);
}

bool make_map(CUtensorMap *m, const uint8_t *base, int64_t ld, int rows, int K, int box_rows)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t str[1] = {static_cast<cuuint64_t>(ld)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kKB), static_cast<cuuint32_t>(box_rows)};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
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
    // blocks per tile: as many as keep the grid within the blocks that fit
    int cluster = 1;
    if (TN < 256)
        cluster = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({8, KB, sms * G::kBlocks / tiles})));
    const int grid = cluster > 1 ? static_cast<int>(tiles) * cluster
                                 : static_cast<int>(std::min<int64_t>(tiles, sms * G::kBlocks));
    const awq_status r = set_smem(fp8_gemm_kernel<T, TN, SWAP>, G::kSmem);
    if (r) return r;
    return launch(fp8_gemm_kernel<T, TN, SWAP>, dim3(grid), dim3(G::kThreads), G::kSmem, cluster, st, mm, mn, g, cluster);
}

template <typename T>
awq_status launch_gemm_t(const GemmArgs &g, const uint8_t *a, int64_t lda, const uint8_t *b, int64_t ldb, int sms,
                         cudaStream_t st)
{
    if (g.M <= 16) return launch_gemm_tile<T, 16, true>(g, a, lda, b, ldb, sms, st);
    if (g.M <= 32) return launch_gemm_tile<T, 32, true>(g, a, lda, b, ldb, sms, st);
    if (g.M <= 64) return launch_gemm_tile<T, 64, true>(g, a, lda, b, ldb, sms, st);
    const int64_t wide = static_cast<int64_t>((g.M + 127) / 128) * ((g.N + 255) / 256);
    if (wide >= sms) return launch_gemm_tile<T, 256, false>(g, a, lda, b, ldb, sms, st);
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
