// awq_qk_norm_rope_append: RMS norm of each head of q and k, rotation by
// position and the append of k and v to the paged cache, in one pass.
//
// One block per token, its rows q's heads, k's and v's (a v row is copied). A
// row is dealt in items to 1 to 32 neighbouring lanes: an item is VEC pairs half
// a rotation apart (two accesses of VEC elements), VEC / 2 interleaved pairs or
// VEC elements past the rotation (one access), so that a lane keeps its item in
// registers from the sum of squares, which the row's lanes add by shuffles, to
// the store. Only a row of more than 32 items is read twice, its second time
// from L1. Bound by the bytes for many tokens, by the launch and dependent loads
// for few.
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
    return vec == 8   ? launch_head_norm_n<T, FP8, 8>(n, sms, st)
           : vec == 4 ? launch_head_norm_n<T, FP8, 4>(n, sms, st)
                      : launch_head_norm_n<T, FP8, 1>(n, sms, st);
}

}  // namespace

awq_status launch_head_norm(const HeadNormArgs &n, int dtype, int vec, int sms, cudaStream_t st)
{
    const bool fp8 = n.rope.cache.dtype == AWQ_DTYPE_E4M3;
    if (dtype == AWQ_DTYPE_F16) return fp8 ? launch_head_norm_t<__half, true>(n, vec, sms, st) : launch_head_norm_t<__half, false>(n, vec, sms, st);
    return fp8 ? launch_head_norm_t<__nv_bfloat16, true>(n, vec, sms, st) : launch_head_norm_t<__nv_bfloat16, false>(n, vec, sms, st);
}

}  // namespace awq
