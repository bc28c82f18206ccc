// Kernel-side declarations of the decoder-layer operators (awq_decoder.h):
// argument blocks, launchers and the conversions they share.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/awq_decoder.h"
#include "awq_ptx.cuh"

namespace awq {

// x / y for 0 <= x, 0 < y, short where both fit 32 bits (nearly always; a
// 64-bit division is a long way through code that runs once).
__device__ __forceinline__ int64_t div_up_to_64(int64_t x, int64_t y)
{
    if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return x / y;
}

// ------------------------------------------------------------ conversions

// fp32 as one 16-bit activation (round to nearest even).
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __half from_f32<__half>(float v)
{
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}

// Two fp32 values as a 16-bit pair, `lo` in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A 16-bit pair as two fp32 values.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

// Two fp32 values as an e4m3 pair, `lo` in the low byte (nearest even,
// saturating at +-448; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d)
{
    return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}

// N (1, 4 or 8) consecutive 16-bit elements, 4 and 8 in one aligned access: as
// loaded, and as fp32.
template <int N>
struct RawElems {
    static_assert(N == 1 || N == 4 || N == 8, "1, 4 or 8 elements");
    uint32_t w[N == 1 ? 1 : N / 2];
};

template <int N, typename T>
__device__ __forceinline__ RawElems<N> load_raw(const T *p)
{
    RawElems<N> r;
    if constexpr (N == 8) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        r.w[0] = v.x;
        r.w[1] = v.y;
        r.w[2] = v.z;
        r.w[3] = v.w;
    } else if constexpr (N == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = v.x;
        r.w[1] = v.y;
    } else {
        r.w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
    return r;
}

template <typename T, int N>
__device__ __forceinline__ void unpack_raw(const RawElems<N> &r, float (&f)[N])
{
    if constexpr (N == 1) {
        f[0] = unpack2<T>(r.w[0]).x;
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 x = unpack2<T>(r.w[i]);
            f[2 * i] = x.x;
            f[2 * i + 1] = x.y;
        }
    }
}

template <typename T, int N>
__device__ __forceinline__ void load_elems(const T *p, float (&f)[N])
{
    unpack_raw<T>(load_raw<N>(p), f);
}

template <typename T, int N>
__device__ __forceinline__ void store_elems(T *p, const float (&f)[N])
{
    if constexpr (N == 8) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                                                   pack2<T>(f[6], f[7]));
    } else if constexpr (N == 4) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
    } else {
        static_assert(N == 1, "1, 4 or 8 elements");
        *p = from_f32<T>(f[0]);
    }
}

template <int N>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&f)[N])
{
    if constexpr (N == 8) {
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
    } else if constexpr (N == 4) {
        *reinterpret_cast<uint32_t *>(p) = pack_e4m3x4(f[0], f[1], f[2], f[3]);
    } else {
        static_assert(N == 1, "1, 4 or 8 elements");
        *p = static_cast<uint8_t>(pack_e4m3x2(f[0], 0.f));
    }
}

// A group's scale and the factor its values are multiplied by.
__device__ __forceinline__ float2 group_scale(float amax)
{
    const float a = fmaxf(amax, AWQ_FP8_MIN_AMAX);
    return make_float2(a / 448.f, 448.f / a);
}

// ---------------------------------------------------------- argument blocks

struct NormArgs {
    const void *x, *residual, *weight;
    void *residual_out, *out;
    uint8_t *out_q;
    float *out_scales;
    int64_t ldx, ldr, ldro, ldo, ldq;
    float eps;
    int32_t rows, hidden;
};

struct QuantArgs {
    const void *x;
    uint8_t *q;
    float *scales;
    int64_t ldx, ldq;
    int32_t rows, cols;
};

struct RopeArgs {
    awq_heads q, q_out, k, v;
    const int32_t *positions;
    const float *cos_sin;
    const int64_t *slots;
    awq_kv_cache cache;
    int32_t *status;
    int32_t max_positions, rotary_dim, interleaved, tokens, q_heads;
};

struct AttnArgs {
    awq_heads q, out;
    awq_kv_cache cache;
    const int32_t *page_table;
    const int32_t *seq_lens;
    float *lse;
    int32_t *counters;     // [kAttnMaxCtas], zero between calls
    float *parts;          // split pieces, see awq_attn.cu
    int32_t *status;
    int64_t table_stride;
    int32_t max_pages, batch, q_heads, group, row_tiles;
    uint32_t page_magic;   // token / page_size = umulhi(token, magic) >> (shift - 1); shift 0: page size 1
    int32_t page_shift;
    int32_t same_strides;  // K and V have the same strides
    float scale;
};

struct GemmArgs {
    const float *a_scales, *b_scales;
    void *out;
    int64_t ldo;
    int32_t *status;
    int32_t M, N, K;
    uint64_t timeout_ns;
};

// ---------------------------------------------------------------- launchers

// Vectors of 16 bytes where `wide`, else any size and alignment.
awq_status launch_norm(const NormArgs &a, int dtype, bool wide, int sms, cudaStream_t st);
awq_status launch_quantize(const QuantArgs &a, int dtype, bool wide, int sms, cudaStream_t st);
// vec: elements per access (8, 4 or 1).
awq_status launch_rope(const RopeArgs &a, int dtype, int vec, int sms, cudaStream_t st);

// The attention's grid never exceeds this many blocks of this many warps (its
// workspace holds a counter and two pieces per block and a part per warp).
constexpr int kAttnMaxCtas = 160;
constexpr int kAttnMaxWarps = 12;
constexpr int kAttnRows = 16;          // query heads of one tile
constexpr size_t kAttnCounterBytes = (kAttnMaxCtas * sizeof(int32_t) + 255) / 256 * 256;
// Padded head size of the kernel that takes `dim`.
constexpr int attn_padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
// Floats of a row of a part or piece: output, maximum, sum; 16-byte rows, and
// heads two apart fall eight banks apart.
constexpr int attn_part_pitch(int padded_dim) { return padded_dim + 4; }
constexpr size_t attn_workspace_bytes(int dim)
{
    return kAttnCounterBytes +
           static_cast<size_t>(kAttnMaxCtas) * (2 + kAttnMaxWarps) * kAttnRows * attn_part_pitch(attn_padded_dim(dim)) *
               sizeof(float);
}
awq_status launch_attention(const AttnArgs &a, int dtype, int sms, cudaStream_t st);

awq_status launch_fp8_gemm(const GemmArgs &g, const uint8_t *a, int64_t lda, const uint8_t *b, int64_t ldb, int dtype,
                           int sms, cudaStream_t st);

// awq_moe_api.cu
int current_sm_count();
bool encode_tensor_map(CUtensorMap *m, CUtensorMapDataType dt, int rank, const void *base, const cuuint64_t *dims,
                       const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swz,
                       CUtensorMapL2promotion l2);

}  // namespace awq
