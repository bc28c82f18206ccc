// awq_rope_append: rotation of q and k by position and the append of k and v
// to the paged cache, in one pass over them.
//
// One block per token (and slice of its heads, for few tokens): a thread
// keeps the cos and sin of its pairs in registers and walks over the heads.
// Per head an item is VEC pairs: two accesses of VEC elements half a rotation
// apart, or one access of VEC elements (VEC / 2 pairs) where pairs are
// interleaved; what is not rotated is copied in accesses of VEC elements. A
// handful of operations per element: bound by the bytes for many tokens, by
// the launch for few.
#include "awq_decoder_kernels.cuh"
#include "awq_launch.cuh"

namespace awq {

namespace {

constexpr int kRopeThreads = 256;

// A cache element's address and the stores in its type.
template <typename T, bool FP8, int N>
__device__ __forceinline__ void store_cache(void *base, int64_t at, const float (&f)[N], float inv)
{
    if constexpr (FP8) {
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = f[i] * inv;
        store_e4m3<N>(static_cast<uint8_t *>(base) + at, v);
    } else {
        store_elems<T, N>(static_cast<T *>(base) + at, f);
    }
}

// N table values, aligned to N floats where N > 1.
template <int N>
__device__ __forceinline__ void load_table(const float *p, float (&f)[N])
{
    if constexpr (N == 8 || N == 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + i);
            f[i] = v.x;
            f[i + 1] = v.y;
            f[i + 2] = v.z;
            f[i + 3] = v.w;
        }
    } else if constexpr (N == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        f[0] = v.x;
        f[1] = v.y;
    } else {
        f[0] = *p;
    }
}

// blockDim.x: items of a head that run side by side; blockDim.y: heads.
template <typename T, bool FP8, int VEC, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = blockIdx.x;
    const awq_kv_cache &c = a.cache;
    const int64_t slot = a.slots[t];
    const int pos = a.positions[t];
    if (pos < 0 || pos >= a.max_positions || slot >= static_cast<int64_t>(c.num_pages) * c.page_size) {
        if (blockIdx.y == 0 && threadIdx.x == 0 && threadIdx.y == 0) set_status(a.status, AWQ_ERR_BAD_INDEX);
        return;
    }
    const bool keep = slot >= 0;
    const int64_t page = keep ? slot / c.page_size : 0, place = keep ? slot - page * c.page_size : 0;
    const int64_t k_at = page * c.k.page_stride + place * c.k.token_stride;
    const int64_t v_at = page * c.v.page_stride + place * c.v.token_stride;
    const float k_inv = 1.f / c.k.scale, v_inv = 1.f / c.v.scale;
    const T *q = static_cast<const T *>(a.q.data) + t * a.q.token_stride;
    T *qo = static_cast<T *>(a.q_out.data) + t * a.q_out.token_stride;
    const T *k = static_cast<const T *>(a.k.data) + t * a.k.token_stride;
    const T *v = static_cast<const T *>(a.v.data) + t * a.v.token_stride;
    const float *row = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim;
    const int half = a.rotary_dim / 2;
    const int head0 = blockIdx.y * blockDim.y + threadIdx.y, head_step = gridDim.y * blockDim.y;
    // heads: q's, then k's
    const int heads = a.q_heads + (keep ? c.num_heads : 0);

    constexpr int P = INTER ? (VEC == 1 ? 1 : VEC / 2) : VEC;      // pairs of an item
    for (int i = threadIdx.x * P; i < half; i += blockDim.x * P) {
        float cs[P], sn[P];
        load_table<P>(row + i, cs);
        load_table<P>(row + half + i, sn);
        for (int h = head0; h < heads; h += head_step) {
            const bool is_q = h < a.q_heads;
            const T *src = is_q ? q + h * a.q.head_stride : k + (h - a.q_heads) * a.k.head_stride;
            if constexpr (INTER && VEC > 1) {
                float x[VEC], y[VEC];
                load_elems<T, VEC>(src + 2 * i, x);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    y[2 * j] = x[2 * j] * cs[j] - x[2 * j + 1] * sn[j];
                    y[2 * j + 1] = x[2 * j + 1] * cs[j] + x[2 * j] * sn[j];
                }
                if (is_q)
                    store_elems<T, VEC>(qo + h * a.q_out.head_stride + 2 * i, y);
                else
                    store_cache<T, FP8, VEC>(c.k.data, k_at + (h - a.q_heads) * c.k.head_stride + 2 * i, y, k_inv);
            } else {
                const int lo = INTER ? 2 * i : i, hi = INTER ? 2 * i + 1 : i + half;
                float x[P], y[P], u[P], w[P];
                load_elems<T, P>(src + lo, x);
                load_elems<T, P>(src + hi, y);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    u[j] = x[j] * cs[j] - y[j] * sn[j];
                    w[j] = y[j] * cs[j] + x[j] * sn[j];
                }
                if (is_q) {
                    store_elems<T, P>(qo + h * a.q_out.head_stride + lo, u);
                    store_elems<T, P>(qo + h * a.q_out.head_stride + hi, w);
                } else {
                    const int64_t at = k_at + (h - a.q_heads) * c.k.head_stride;
                    store_cache<T, FP8, P>(c.k.data, at + lo, u, k_inv);
                    store_cache<T, FP8, P>(c.k.data, at + hi, w, k_inv);
                }
            }
        }
    }
    // the part of q and k past the rotation
    for (int d = a.rotary_dim + threadIdx.x * VEC; d < c.head_dim; d += blockDim.x * VEC) {
        for (int h = head0; h < heads; h += head_step) {
            const bool is_q = h < a.q_heads;
            float x[VEC];
            load_elems<T, VEC>((is_q ? q + h * a.q.head_stride : k + (h - a.q_heads) * a.k.head_stride) + d, x);
            if (is_q)
                store_elems<T, VEC>(qo + h * a.q_out.head_stride + d, x);
            else
                store_cache<T, FP8, VEC>(c.k.data, k_at + (h - a.q_heads) * c.k.head_stride + d, x, k_inv);
        }
    }
    if (!keep) return;
    for (int h = head0; h < c.num_heads; h += head_step)
        for (int d = threadIdx.x * VEC; d < c.head_dim; d += blockDim.x * VEC) {
            float x[VEC];
            load_elems<T, VEC>(v + h * a.v.head_stride + d, x);
            store_cache<T, FP8, VEC>(c.v.data, v_at + h * c.v.head_stride + d, x, v_inv);
        }
}

template <typename T, bool FP8, int VEC>
awq_status launch_rope_v(const RopeArgs &a, cudaStream_t st)
{
    // side by side: the items of a head's rotation (of its copy, without one)
    const int pairs = a.interleaved && VEC > 1 ? VEC / 2 : VEC;
    int bx = a.rotary_dim ? (a.rotary_dim / 2 + pairs - 1) / pairs : (a.cache.head_dim + VEC - 1) / VEC;
    bx = bx < 1 ? 1 : bx > kRopeThreads ? kRopeThreads : bx;
    const int heads = a.q_heads + a.cache.num_heads;
    int by = kRopeThreads / bx;
    if (by > heads) by = heads;
    return a.interleaved
               ? launch(rope_kernel<T, FP8, VEC, true>, dim3(a.tokens), dim3(bx, by), 0, 1, st, a)
               : launch(rope_kernel<T, FP8, VEC, false>, dim3(a.tokens), dim3(bx, by), 0, 1, st, a);
}

template <typename T, bool FP8>
awq_status launch_rope_t(const RopeArgs &a, int vec, cudaStream_t st)
{
    return vec == 8   ? launch_rope_v<T, FP8, 8>(a, st)
           : vec == 4 ? launch_rope_v<T, FP8, 4>(a, st)
                      : launch_rope_v<T, FP8, 1>(a, st);
}

}  // namespace

awq_status launch_rope(const RopeArgs &a, int dtype, int vec, cudaStream_t st)
{
    const bool fp8 = a.cache.dtype == AWQ_DTYPE_E4M3;
    if (dtype == AWQ_DTYPE_F16) return fp8 ? launch_rope_t<__half, true>(a, vec, st) : launch_rope_t<__half, false>(a, vec, st);
    return fp8 ? launch_rope_t<__nv_bfloat16, true>(a, vec, st) : launch_rope_t<__nv_bfloat16, false>(a, vec, st);
}

}  // namespace awq
