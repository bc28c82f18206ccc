// awq_rope_append: rotation of q and k by position and the append of k and v
// to the paged cache, in one pass over them.
//
// One block per token: its rows are q's heads, k's and v's (a v row is a row
// that is not turned), a thread takes the same VEC pairs of up to two or so of
// them. Per row an item is VEC pairs: two accesses of VEC elements half a
// rotation apart, or one access of VEC elements (VEC / 2 pairs) where pairs are
// interleaved; what is not rotated is copied in accesses of VEC elements. A
// handful of operations per element: bound by the bytes for many tokens, by
// the launch and three dependent loads for few.
#include "awq_decoder_kernels.cuh"
#include "awq_launch.cuh"

namespace awq {

namespace {


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

// One head's pairs: loaded, then turned and stored.
template <typename T, int VEC, bool INTER>
struct Pairs {
    static constexpr int P = INTER ? (VEC == 1 ? 1 : VEC / 2) : VEC;      // pairs of an item
    static constexpr bool kOne = INTER && VEC > 1;                        // both halves in one access
    RawElems<kOne ? VEC : P> a;
    RawElems<kOne ? 1 : P> b;

    __device__ __forceinline__ void load(const T *src, int i, int half)
    {
        if constexpr (kOne) {
            a = load_raw<VEC>(src + 2 * i);
        } else {
            a = load_raw<P>(src + (INTER ? 2 * i : i));
            b = load_raw<P>(src + (INTER ? 2 * i + 1 : i + half));
        }
    }

    // store(element, values) puts neighbouring elements
    template <typename Store>
    __device__ __forceinline__ void turn(bool rotate, const float (&cs)[P], const float (&sn)[P], int i, int half, Store store) const
    {
        float x[P], y[P];
        if constexpr (kOne) {
            float t[VEC];
            unpack_raw<T>(a, t);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                x[j] = t[2 * j];
                y[j] = t[2 * j + 1];
            }
        } else {
            unpack_raw<T>(a, x);
            unpack_raw<T>(b, y);
        }
        if (rotate) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float u = x[j] * cs[j] - y[j] * sn[j];
                y[j] = y[j] * cs[j] + x[j] * sn[j];
                x[j] = u;
            }
        }
        if constexpr (kOne) {
            float t[VEC];
#pragma unroll
            for (int j = 0; j < P; ++j) {
                t[2 * j] = x[j];
                t[2 * j + 1] = y[j];
            }
            store(2 * i, t);
        } else {
            store(INTER ? 2 * i : i, x);
            store(INTER ? 2 * i + 1 : i + half, y);
        }
    }
};

// blockDim.x: items of a row that run side by side; blockDim.y: rows. The
// elements do not depend on the position: a thread's first kAhead rows are on
// their way while the position, the slot and then the row of the table are.
// THREADS: at most this many a block (1,024 a multiprocessor).
template <typename T, bool FP8, int VEC, bool INTER, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) rope_kernel(const RopeArgs a)
{
    using Row = Pairs<T, VEC, INTER>;
    constexpr int P = Row::P, kAhead = 2;
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = blockIdx.x;
    const awq_kv_cache &c = a.cache;
    const int64_t slot = a.slots[t];
    const int pos = a.positions[t];
    const int half = a.rotary_dim / 2;
    const int k_row = a.q_heads, v_row = k_row + c.num_heads, all_rows = v_row + c.num_heads;
    auto source = [&](int r) {
        const awq_heads &h = r < k_row ? a.q : r < v_row ? a.k : a.v;
        return static_cast<const T *>(h.data) + t * h.token_stride + (r - (r < k_row ? 0 : r < v_row ? k_row : v_row)) * h.head_stride;
    };
    const int i0 = threadIdx.x * P, r0 = threadIdx.y, step = blockDim.y;
    Row ahead[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n)
        if (i0 < half && r0 + n * step < all_rows) ahead[n].load(source(r0 + n * step), i0, half);
    const int d0 = a.rotary_dim + threadIdx.x * VEC;     // the part past the rotation
    RawElems<VEC> rest[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n)
        if (d0 < c.head_dim && r0 + n * step < all_rows) rest[n] = load_raw<VEC>(source(r0 + n * step) + d0);

    if (pos < 0 || pos >= a.max_positions || slot >= static_cast<int64_t>(c.num_pages) * c.page_size) {
        if (threadIdx.x == 0 && threadIdx.y == 0) set_status(a.status, AWQ_ERR_BAD_INDEX);
        return;
    }
    const int64_t page = slot < 0 ? 0 : div_up_to_64(slot, c.page_size), place = slot < 0 ? 0 : slot - page * c.page_size;
    const float *table = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim;
    const int rows = slot < 0 ? k_row : all_rows;        // an unused token: q's alone

    // VEC neighbouring elements of row r from element d on
    auto put = [&](int r, int d, auto &f) {
        if (r < k_row) {
            store_elems<T>(static_cast<T *>(a.q_out.data) + t * a.q_out.token_stride + r * a.q_out.head_stride + d, f);
        } else {
            const awq_kv_plane &p = r < v_row ? c.k : c.v;
            store_cache<T, FP8>(p.data, page * p.page_stride + place * p.token_stride +
                                            (r - (r < v_row ? k_row : v_row)) * p.head_stride + d, f, 1.f / p.scale);
        }
    };
    for (int i = i0; i < half; i += blockDim.x * P) {
        float cs[P], sn[P];
        load_table<P>(table + i, cs);
        load_table<P>(table + half + i, sn);
        int r = r0;
        if (i == i0) {
#pragma unroll
            for (int n = 0; n < kAhead; ++n, r += step)
                if (r < rows) ahead[n].turn(r < v_row, cs, sn, i, half, [&](int d, auto &f) { put(r, d, f); });
        }
        for (; r < rows; r += step) {
            Row x;
            x.load(source(r), i, half);
            x.turn(r < v_row, cs, sn, i, half, [&](int d, auto &f) { put(r, d, f); });
        }
    }
    for (int d = d0; d < c.head_dim; d += blockDim.x * VEC) {
        float x[VEC];
        int r = r0;
        if (d == d0) {
#pragma unroll
            for (int n = 0; n < kAhead; ++n, r += step)
                if (r < rows) {
                    unpack_raw<T>(rest[n], x);
                    put(r, d, x);
                }
        }
        for (; r < rows; r += step) {
            load_elems<T, VEC>(source(r) + d, x);
            put(r, d, x);
        }
    }
}

template <typename T, bool FP8, int VEC, int THREADS>
awq_status launch_rope_v(const RopeArgs &a, cudaStream_t st)
{
    // side by side: the items of a row's rotation (of its copy, without one);
    // the rows spread evenly over as few turns as the block's threads allow
    const int pairs = a.interleaved && VEC > 1 ? VEC / 2 : VEC;
    int bx = a.rotary_dim ? (a.rotary_dim / 2 + pairs - 1) / pairs : (a.cache.head_dim + VEC - 1) / VEC;
    bx = bx > THREADS ? THREADS : bx;
    const int64_t rows = static_cast<int64_t>(a.q_heads) + 2 * a.cache.num_heads;
    const int64_t turns = (rows + THREADS / bx - 1) / (THREADS / bx);
    const int by = static_cast<int>((rows + turns - 1) / turns);
    return a.interleaved
               ? launch(rope_kernel<T, FP8, VEC, true, THREADS>, dim3(a.tokens), dim3(bx, by), 0, 1, st, a)
               : launch(rope_kernel<T, FP8, VEC, false, THREADS>, dim3(a.tokens), dim3(bx, by), 0, 1, st, a);
}

template <typename T, bool FP8, int VEC>
awq_status launch_rope_n(const RopeArgs &a, int sms, cudaStream_t st)
{
    // Many tokens: two warps each, whose work per token (its slot, page and
    // addresses) is then spread over more rows (8191 tokens of 48 rows of 128:
    // 36 us, 43 with eight warps); few: more threads a token (16 tokens: 1.7 us,
    // 2.8 with two warps).
    return a.tokens >= 8 * sms ? launch_rope_v<T, FP8, VEC, 64>(a, st) : launch_rope_v<T, FP8, VEC, 256>(a, st);
}

template <typename T, bool FP8>
awq_status launch_rope_t(const RopeArgs &a, int vec, int sms, cudaStream_t st)
{
    return vec == 8   ? launch_rope_n<T, FP8, 8>(a, sms, st)
           : vec == 4 ? launch_rope_n<T, FP8, 4>(a, sms, st)
                      : launch_rope_n<T, FP8, 1>(a, sms, st);
}

}  // namespace

awq_status launch_rope(const RopeArgs &a, int dtype, int vec, int sms, cudaStream_t st)
{
    const bool fp8 = a.cache.dtype == AWQ_DTYPE_E4M3;
    if (dtype == AWQ_DTYPE_F16) return fp8 ? launch_rope_t<__half, true>(a, vec, sms, st) : launch_rope_t<__half, false>(a, vec, sms, st);
    return fp8 ? launch_rope_t<__nv_bfloat16, true>(a, vec, sms, st) : launch_rope_t<__nv_bfloat16, false>(a, vec, sms, st);
}

}  // namespace awq
