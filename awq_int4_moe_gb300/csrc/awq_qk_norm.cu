// awq_qk_norm_rope_append: RMS norm of each head of q and k, rotation by
// position and the append of k and v to the paged cache, in one pass.
//
// One block per token, its rows q's heads, k's and v's (a v row is copied).
//
// Heads of up to 256 elements in whole, aligned chunks of 8 (head_rows_kernel): a
// chunk a lane, the row's sum of squares by shuffles over its 8 to 32 lanes. With
//   out[j] = (x[j] by) (w[j] cos) + (x'[j] by) (w'[j] sin),  by = 1 / rms,
// x' the other element of the pair (from the lane half a rotation away, or the
// neighbour in the chunk), the token's products of weights, cosines and signed
// sines are formed once and a row costs four products and a sum per element.
// From 3 tokens per multiprocessor on a token is one warp's, which forms those
// products once for all its rows and has two rows on their way; below that a token's q, k
// and v are blocks of their own, of as many threads as they have chunks. 32 + 2 x 8 heads
// of 128, a warp against blocks: 64 tokens 7.2 / 3.0 us, 300 7.4 / 5.8, 600 7.5 / 9.0,
// 1200 8.4 / 16, 8191 40 / 109.
//
// Any other shape (head_norm_kernel): a row is dealt in items to 1 to 32
// neighbouring lanes: an item is VEC pairs half a rotation apart (two accesses
// of VEC elements), VEC / 2 interleaved pairs or VEC elements past the rotation (one
// access). A row of more than 32 items is read twice, its second time from L1.
//
// Bound by the bytes for many tokens (a prompt of 8191: 189 MB, 68 % of the copy
// bandwidth; what is missing is the latency of a warp's first rows and loads on their way: a
// multiprocessor holds 32 of its blocks of one warp), by the launch and dependent loads for few.
#include <algorithm>
#include <type_traits>

#include "awq_launch.cuh"
#include "awq_prompt_kernels.cuh"
#include "awq_rope.cuh"

namespace awq {

namespace {

template <typename T, bool FP8, int VEC, bool INTER, int THREADS>
__global__ void __launch_bounds__(THREADS, 768 / THREADS) head_norm_kernel(const HeadNormArgs n, int lanes_log2)
{
    using Row = Pairs<T, VEC, INTER>;
    constexpr int P = Row::P, kAhead = 2;
    const RopeArgs &a = n.rope;
    const awq_kv_cache &c = a.cache;
    const int t = blockIdx.x;
    const int half = a.rotary_dim / 2, rot_items = half / P, items = rot_items + (c.head_dim - a.rotary_dim) / VEC;
    const int k_row = a.q_heads, v_row = k_row + c.num_heads, all_rows = v_row + c.num_heads;
    const int lanes = 1 << lanes_log2, it0 = threadIdx.x & (lanes - 1), r0 = threadIdx.x >> lanes_log2;
    const int step = blockDim.x >> lanes_log2;
    const float per_dim = 1.f / c.head_dim;

    // item `it` of a row at src: the elements of a rotation, or VEC past it
    auto load = [&](Row &x, const T *src, int it) {
        if (it < rot_items) x.load(src, it * P, half);
        else *reinterpret_cast<RawElems<VEC> *>(&x.a) = load_raw<VEC>(src + a.rotary_dim + (it - rot_items) * VEC);
    };
    // an item as fp32, e[0 .. VEC) and, for pairs of two accesses, f
    auto unpack = [&](const Row &x, float (&e)[VEC], float (&f)[VEC], bool rot) {
        unpack_raw<T>(*reinterpret_cast<const RawElems<VEC> *>(&x.a), e);
        if constexpr (!Row::kOne) {
            if (rot) unpack_raw<T>(x.b, f);
        }
    };

    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t slot = a.slots[t];
    const int pos = a.positions[t];
    auto source = [&](int r) {
        const awq_heads &h = r < k_row ? a.q : r < v_row ? a.k : a.v;
        return static_cast<const T *>(h.data) + t * h.token_stride +
               static_cast<int64_t>(r - (r < k_row ? 0 : r < v_row ? k_row : v_row)) * h.head_stride;
    };
    Row ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (it0 < items && r0 + i * step < all_rows) load(ahead[i], source(r0 + i * step), it0);
    Row wq, wk;                                          // the item's weights
    if (it0 < items) {
        load(wq, static_cast<const T *>(n.q_weight), it0);
        load(wk, static_cast<const T *>(n.k_weight), it0);
    }
    if (pos < 0 || pos >= a.max_positions || slot >= static_cast<int64_t>(c.num_pages) * c.page_size) {
        if (threadIdx.x == 0) set_status(a.status, AWQ_ERR_BAD_INDEX);
        return;
    }
    const int64_t page = slot < 0 ? 0 : div_up_to_64(slot, c.page_size), place = slot < 0 ? 0 : slot - page * c.page_size;
    const float *const table = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim;
    const int rows = slot < 0 ? k_row : all_rows;        // an unused token: q's alone
    float cs0[P], sn0[P];
    if (it0 < rot_items) {
        load_table<P>(table + it0 * P, cs0);
        load_table<P>(table + half + it0 * P, sn0);
    }

    // the item of row r, scaled by `by` and its weight (q and k), turned, stored
    auto finish = [&](const Row &x, const Row &w, int it, int r, float by, const float (&cs)[P], const float (&sn)[P]) {
        const bool rot = it < rot_items, norm = r < v_row;
        float e[VEC], f[VEC];
        unpack(x, e, f, rot);
        if (norm) {
            float we[VEC], wf[VEC];
            unpack(w, we, wf, rot);
#pragma unroll
            for (int i = 0; i < VEC; ++i) e[i] = e[i] * by * we[i];
            if constexpr (!Row::kOne) {
                if (rot) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) f[i] = f[i] * by * wf[i];
                }
            }
            if (rot) {
                if constexpr (Row::kOne) {
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const float u = e[2 * j] * cs[j] - e[2 * j + 1] * sn[j];
                        e[2 * j + 1] = e[2 * j + 1] * cs[j] + e[2 * j] * sn[j];
                        e[2 * j] = u;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const float u = e[j] * cs[j] - f[j] * sn[j];
                        f[j] = f[j] * cs[j] + e[j] * sn[j];
                        e[j] = u;
                    }
                }
            }
        }
        auto put = [&](int d, const float (&y)[VEC]) {
            if (r < k_row) {
                store_elems<T>(static_cast<T *>(a.q_out.data) + t * a.q_out.token_stride + r * a.q_out.head_stride + d, y);
            } else {
                const awq_kv_plane &p = r < v_row ? c.k : c.v;
                store_cache<T, FP8>(p.data, page * p.page_stride + place * p.token_stride +
                                                (r - (r < v_row ? k_row : v_row)) * p.head_stride + d, y, 1.f / p.scale);
            }
        };
        if (!rot) {
            put(a.rotary_dim + (it - rot_items) * VEC, e);
        } else if constexpr (Row::kOne) {
            put(2 * it * P, e);
        } else {
            put(INTER ? 2 * it : it * P, e);
            put(INTER ? 2 * it + 1 : it * P + half, f);
        }
    };
    auto squares = [&](const Row &x, int it) {
        const bool rot = it < rot_items;
        float e[VEC], f[VEC], s = 0.f;
        unpack(x, e, f, rot);
#pragma unroll
        for (int i = 0; i < VEC; ++i) s = fmaf(e[i], e[i], s);
        if constexpr (!Row::kOne) {
            if (rot) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) s = fmaf(f[i], f[i], s);
            }
        }
        return s;
    };

    const int turns = (rows + step - 1) / step;          // (the same for a warp's lanes, which shuffle)
    for (int turn = 0; turn < turns; turn += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = r0 + (turn + i) * step;
            const bool in = r < rows;
            float sum = 0.f;
            if (in && it0 < items) {
                sum = squares(ahead[i], it0);
                for (int it = it0 + lanes; it < items; it += lanes) {
                    Row x;
                    load(x, source(r), it);
                    sum += squares(x, it);
                }
            }
            for (int m = lanes / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(~0u, sum, m);
            if (!in || it0 >= items) continue;
            const float by = rsqrtf(sum * per_dim + n.eps);
            finish(ahead[i], r < k_row ? wq : wk, it0, r, by, cs0, sn0);
            for (int it = it0 + lanes; it < items; it += lanes) {
                Row x, w;
                load(x, source(r), it);
                if (r < v_row) load(w, static_cast<const T *>(r < k_row ? n.q_weight : n.k_weight), it);
                float cs[P], sn[P];
                if (it < rot_items) {
                    load_table<P>(table + it * P, cs);
                    load_table<P>(table + half + it * P, sn);
                }
                finish(x, w, it, r, by, cs, sn);
            }
        }
        // the rows after the next
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = r0 + (turn + kAhead + i) * step;
            if (it0 < items && r < rows) load(ahead[i], source(r), it0);
        }
    }
}

__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t pair_f2(float2 v)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ float2 parts_f2(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

// What a row becomes: q's and k's are normed and turned, k's and v's go to the cache.
enum class Part { Q, K, V };

template <typename T, bool FP8, bool INTER, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) head_rows_kernel(const HeadNormArgs n, int lanes_log2)
{
    constexpr int kAhead = THREADS == 32 ? 2 : 1;        // rows on their way
    // few tokens: a block for each part of one
    const bool split = gridDim.y > 1;
    const int first = blockIdx.y;
    const RopeArgs &a = n.rope;
    const awq_kv_cache &c = a.cache;
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    const int lanes = 1 << lanes_log2, it = threadIdx.x & (lanes - 1), r0 = threadIdx.x >> lanes_log2;
    const int step = blockDim.x >> lanes_log2;
    const bool on = it * 8 < c.head_dim, rot = it * 8 < a.rotary_dim;
    const int half = a.rotary_dim / 2, half_items = half / 8;
    const float per_dim = 1.f / c.head_dim;

    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t slot = a.slots[t];
    const int pos = a.positions[t];
    auto row_of = [&](const awq_heads &h, int r) {
        return static_cast<T *>(h.data) + t * h.token_stride + r * h.head_stride + it * 8;
    };
    auto load = [&](const T *p, bool in) { return in ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0); };
    uint4 x[kAhead];                                     // the next rows, the first ones before all else
    const awq_heads &begin = first == 0 ? a.q : first == 1 ? a.k : a.v;
    const int begin_count = first == 0 ? a.q_heads : c.num_heads;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = load(row_of(begin, r0 + i * step), on && r0 + i * step < begin_count);
    // the lane that has the other elements of the pairs
    const int other = INTER || !rot ? it : it < half_items ? it + half_items : it - half_items;
    const int from = (lane & ~(lanes - 1)) | other;
    if (pos < 0 || pos >= a.max_positions || slot >= static_cast<int64_t>(c.num_pages) * c.page_size) {
        if (threadIdx.x == 0) set_status(a.status, AWQ_ERR_BAD_INDEX);
        return;
    }
    // cosines, and sines with the sign that they have in this element's sum
    float cs[8], sn[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        cs[j] = 1.f;
        sn[j] = 0.f;
    }
    if (rot) {
        const float *const table = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim;
        if constexpr (INTER) {
            float u[4], w[4];
            load_table<4>(table + it * 4, u);
            load_table<4>(table + half + it * 4, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                cs[j] = u[j / 2];
                sn[j] = j & 1 ? w[j / 2] : -w[j / 2];
            }
        } else {
            const int at = (it < half_items ? it : it - half_items) * 8;
            load_table<8>(table + at, cs);
            load_table<8>(table + half + at, sn);
            if (it < half_items) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sn[j] = -sn[j];
            }
        }
    }

    // The rows of one part: `count` of them from `src` on, to `dst`; the next part's
    // first rows are loaded before it ends.
    auto rows_of = [&](auto part, const awq_heads &src, int count, const void *weight, void *dst, int64_t dst_stride, float inv,
                       const awq_heads *then, int then_count) {
        constexpr Part P = decltype(part)::value;
        uint64_t wc[4], ws[4];                           // weights times cosines and sines, in pairs
        if constexpr (P != Part::V) {
            const uint4 own = load(static_cast<const T *>(weight) + it * 8, on), its = load(static_cast<const T *>(weight) + other * 8, on);
            const uint32_t o[4] = {own.x, own.y, own.z, own.w}, p[4] = {its.x, its.y, its.z, its.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 w = unpack2<T>(o[j]);
                float2 v = unpack2<T>(p[j]);
                if constexpr (INTER) v = make_float2(v.y, v.x);
                wc[j] = pair_f2(make_float2(w.x * cs[2 * j] * inv, w.y * cs[2 * j + 1] * inv));
                ws[j] = pair_f2(make_float2(v.x * sn[2 * j] * inv, v.y * sn[2 * j + 1] * inv));
            }
        }
        const T *in = row_of(src, r0);
        char *out = static_cast<char *>(dst);
        constexpr int kElem = P != Part::Q && FP8 ? 1 : 2;
        out += (r0 * dst_stride + it * 8) * kElem;
        const int64_t in_step = step * src.head_stride, out_step = step * dst_stride * kElem;
        const int turns = (count + step - 1) / step;     // (the same for a warp's lanes, which shuffle)
#pragma unroll 1
        for (int turn = 0; turn < turns; turn += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i, in += in_step, out += out_step) {
                const int r = r0 + (turn + i) * step;
                const uint32_t raw[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                if (on && r + kAhead * step < count) x[i] = *reinterpret_cast<const uint4 *>(in + kAhead * in_step);
                else if (then && turn + kAhead >= turns) x[i] = load(row_of(*then, r0 + i * step), on && r0 + i * step < then_count);
                uint64_t e[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) e[j] = pair_f2(unpack2<T>(raw[j]));
                float y[8];
                if constexpr (P == Part::V) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 p = parts_f2(e[j]);
                        y[2 * j] = FP8 ? p.x * inv : p.x;
                        y[2 * j + 1] = FP8 ? p.y * inv : p.y;
                    }
                } else {
                    uint64_t ss = mul_f2(e[0], e[0]);
#pragma unroll
                    for (int j = 1; j < 4; ++j) ss = fma_f2(e[j], e[j], ss);
                    const float2 s2 = parts_f2(ss);
                    float sum = s2.x + s2.y;
                    for (int m = lanes / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(~0u, sum, m);
                    const float by = rsqrtf(sum * per_dim + n.eps);
                    const uint64_t by2 = pair_f2(make_float2(by, by));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint64_t o;                      // the pairs' other elements
                        if constexpr (INTER) {
                            const float2 v = parts_f2(e[j]);
                            o = pair_f2(make_float2(v.y, v.x));
                        } else {
                            o = pair_f2(unpack2<T>(__shfl_sync(~0u, raw[j], from)));
                        }
                        // (scaled first: a product of large values would pass fp32's range)
                        uint64_t v = mul_f2(mul_f2(e[j], by2), wc[j]);
                        if (rot) v = fma_f2(mul_f2(o, by2), ws[j], v);
                        const float2 p = parts_f2(v);
                        y[2 * j] = p.x;
                        y[2 * j + 1] = p.y;
                    }
                }
                if (on && r < count) {
                    if constexpr (kElem == 1) store_e4m3<8>(reinterpret_cast<uint8_t *>(out), y);
                    else store_elems<T>(reinterpret_cast<T *>(out), y);
                }
            }
        }
    };
    using std::integral_constant;
    const bool append = slot >= 0;                       // an unused token: q's alone
    if (first == 0)
        rows_of(integral_constant<Part, Part::Q>(), a.q, a.q_heads, n.q_weight, static_cast<T *>(a.q_out.data) + t * a.q_out.token_stride,
                a.q_out.head_stride, 1.f, append && !split ? &a.k : nullptr, c.num_heads);
    if (!append || (split && first == 0)) return;
    const int64_t page = div_up_to_64(slot, c.page_size), place = slot - page * c.page_size;
    auto plane = [&](const awq_kv_plane &p) {
        return static_cast<char *>(p.data) + (page * p.page_stride + place * p.token_stride) * (FP8 ? 1 : 2);
    };
    if (first <= 1)
        rows_of(integral_constant<Part, Part::K>(), a.k, c.num_heads, n.k_weight, plane(c.k), c.k.head_stride, FP8 ? 1.f / c.k.scale : 1.f,
            split ? nullptr : &a.v, c.num_heads);
    if (split && first == 1) return;
    rows_of(integral_constant<Part, Part::V>(), a.v, c.num_heads, nullptr, plane(c.v), c.v.head_stride, FP8 ? 1.f / c.v.scale : 1.f,
            nullptr, 0);
}

template <typename T, bool FP8, bool INTER, int THREADS>
awq_status launch_head_rows_i(const HeadNormArgs &n, cudaStream_t st)
{
    int log2 = 0;
    while (8 << log2 < n.rope.cache.head_dim) ++log2;
    // q's rows spread evenly over as few turns as the block's threads allow, in whole warps
    const int64_t rows = std::max(n.rope.q_heads, n.rope.cache.num_heads);
    const int most = THREADS >> log2;
    const int64_t turns = (rows + most - 1) / most;
    const int threads = static_cast<int>((rows + turns - 1) / turns) << log2;
    return launch(head_rows_kernel<T, FP8, INTER, THREADS>, dim3(n.rope.tokens, THREADS == 32 ? 1 : 3), dim3((threads + 31) / 32 * 32), 0, 1, st, n, log2);
}

template <typename T, bool FP8>
awq_status launch_head_rows(const HeadNormArgs &n, int sms, cudaStream_t st)
{
    const bool inter = n.rope.interleaved;
    if (n.rope.tokens >= 3 * sms)
        return inter ? launch_head_rows_i<T, FP8, true, 32>(n, st) : launch_head_rows_i<T, FP8, false, 32>(n, st);
    return inter ? launch_head_rows_i<T, FP8, true, 256>(n, st) : launch_head_rows_i<T, FP8, false, 256>(n, st);
}

template <typename T, bool FP8, int VEC, bool INTER, int THREADS>
awq_status launch_head_norm_i(const HeadNormArgs &n, cudaStream_t st)
{
    constexpr int P = Pairs<T, VEC, INTER>::P;
    const RopeArgs &a = n.rope;
    const int items = a.rotary_dim / 2 / P + (a.cache.head_dim - a.rotary_dim) / VEC;
    int log2 = 0;
    while (log2 < 5 && 1 << log2 < items) ++log2;
    // the rows spread evenly over as few turns as the block's threads allow, in whole warps
    const int64_t rows = static_cast<int64_t>(a.q_heads) + 2 * a.cache.num_heads;
    const int most = THREADS >> log2;
    const int64_t turns = (rows + most - 1) / most;
    const int threads = static_cast<int>((rows + turns - 1) / turns) << log2;
    return launch(head_norm_kernel<T, FP8, VEC, INTER, THREADS>, dim3(a.tokens), dim3((threads + 31) / 32 * 32), 0, 1, st, n, log2);
}

template <typename T, bool FP8, int VEC>
awq_status launch_head_norm_n(const HeadNormArgs &n, int sms, cudaStream_t st)
{
    const bool inter = n.rope.interleaved;
    if (n.rope.tokens >= 8 * sms)
        return inter ? launch_head_norm_i<T, FP8, VEC, true, 64>(n, st) : launch_head_norm_i<T, FP8, VEC, false, 64>(n, st);
    return inter ? launch_head_norm_i<T, FP8, VEC, true, 256>(n, st) : launch_head_norm_i<T, FP8, VEC, false, 256>(n, st);
}

template <typename T, bool FP8>
awq_status launch_head_norm_t(const HeadNormArgs &n, int vec, int sms, cudaStream_t st)
{
    if (vec == 8 && n.rope.cache.head_dim <= 256) return launch_head_rows<T, FP8>(n, sms, st);
    return vec >= 4 ? launch_head_norm_n<T, FP8, 4>(n, sms, st) : launch_head_norm_n<T, FP8, 1>(n, sms, st);
}

}  // namespace

awq_status launch_head_norm(const HeadNormArgs &n, int dtype, int vec, int sms, cudaStream_t st)
{
    const bool fp8 = n.rope.cache.dtype == AWQ_DTYPE_E4M3;
    if (dtype == AWQ_DTYPE_F16) return fp8 ? launch_head_norm_t<__half, true>(n, vec, sms, st) : launch_head_norm_t<__half, false>(n, vec, sms, st);
    return fp8 ? launch_head_norm_t<__nv_bfloat16, true>(n, vec, sms, st) : launch_head_norm_t<__nv_bfloat16, false>(n, vec, sms, st);
}

}  // namespace awq
