// awq_add_rmsnorm and awq_quantize_fp8.
//
//   r = x + residual, y = r / sqrt(mean(r^2) + eps) * w, and y in e4m3 with
//   a scale of amax / 448 per group of 128 columns.
//
// Each element is read once and written once per output: a row lives in the
// registers of one block (or one warp) between its sum of squares and its
// outputs. About six operations per element: bound by the bytes for many
// rows (8192 x 5120 with residual, 52.8 us, 6.4 TB/s), by the launch and one
// block's dependent steps for few (1.7 us).
//
// Columns are dealt so that a quantisation group never leaves a warp: with
// 16-byte accesses (wide) 16 neighbouring lanes hold a group, 8 columns each;
// otherwise a warp holds it, lane l the columns l, l + 32, l + 64, l + 96 (one
// element per access, neighbouring lanes side by side). Its amax is a few
// shuffles.
#include <algorithm>

#include "awq_decoder_kernels.cuh"
#include "awq_launch.cuh"

namespace awq {

namespace {

// The columns of chunk j that thread `tid` of the R threads of a row holds.
template <bool WIDE>
struct Columns;
template <>
struct Columns<true> {
    static constexpr int kElems = 8;
    static __device__ __forceinline__ int first(int j, int R, int tid) { return (j * R + tid) * 8; }
    static constexpr int kGroupLanes = 16;
};
template <>
struct Columns<false> {
    static constexpr int kElems = 4;
    static __device__ __forceinline__ int first(int j, int R, int tid) { return (j * R + (tid & ~31)) * 4 + (tid & 31); }
    static constexpr int kGroupLanes = 32;
};

// A chunk's columns as loaded (0 past the row's end), and as fp32.
struct RawCols {
    uint32_t w[4];                       // wide: 8 packed elements; else one in each
};

template <typename T, bool WIDE>
__device__ __forceinline__ RawCols load_raw_cols(const T *row, int c, int n)
{
    RawCols r = {{0, 0, 0, 0}};
    if constexpr (WIDE) {
        if (c < n) {
            const RawElems<8> v = load_raw<8>(row + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) r.w[i] = v.w[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + 32 * i < n) r.w[i] = load_raw<1>(row + c + 32 * i).w[0];
    }
    return r;
}

template <typename T, bool WIDE>
__device__ __forceinline__ void unpack_cols(const RawCols &r, float (&f)[Columns<WIDE>::kElems])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = unpack2<T>(r.w[i]);
        if constexpr (WIDE) {
            f[2 * i] = x.x;
            f[2 * i + 1] = x.y;
        } else {
            f[i] = x.x;
        }
    }
}

template <typename T, bool WIDE>
__device__ __forceinline__ void load_cols(const T *row, int c, int n, float (&f)[Columns<WIDE>::kElems])
{
    unpack_cols<T, WIDE>(load_raw_cols<T, WIDE>(row, c, n), f);
}

template <typename T, bool WIDE>
__device__ __forceinline__ void store_cols(T *row, int c, int n, const float (&f)[Columns<WIDE>::kElems])
{
    if constexpr (WIDE) {
        if (c < n) store_elems<T, 8>(row + c, f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + 32 * i < n) row[c + 32 * i] = from_f32<T>(f[i]);
    }
}

// The group's values (0 past the row's end) as e4m3 and its scale. Every
// lane of the warp calls this.
template <bool WIDE>
__device__ __forceinline__ void quantize_cols(const float (&y)[Columns<WIDE>::kElems], int c, int n, uint8_t *q,
                                              float *scales, int lane)
{
    constexpr int E = Columns<WIDE>::kElems;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) amax = fmaxf(amax, fabsf(y[i]));
#pragma unroll
    for (int o = Columns<WIDE>::kGroupLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
    const float2 s = group_scale(amax);
    float v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = y[i] * s.y;
    if constexpr (WIDE) {
        if (c < n) store_e4m3<8>(q + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + 32 * i < n) store_e4m3<1>(q + c + 32 * i, {v[i]});
    }
    if ((lane & (Columns<WIDE>::kGroupLanes - 1)) == 0 && c < n) scales[c / AWQ_FP8_BLOCK] = s.x;
}

// NV chunks of a row per thread. THREADS 128: a row per warp, blockDim.x / 32
// rows side by side; else a row per block. A block goes on to the row that is
// gridDim.x (x 4) further, whose loads are on their way while the present
// row is summed and written.
template <typename T, bool WIDE, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormArgs a)
{
    constexpr int E = Columns<WIDE>::kElems;
    constexpr bool ROW_WARP = THREADS == 128;
    __shared__ float s_sum[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = ROW_WARP ? 32 : blockDim.x;
    const int tid = ROW_WARP ? lane : threadIdx.x;
    const int64_t step = ROW_WARP ? static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5) : gridDim.x;
    int64_t row = ROW_WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
    const int n = a.hidden;
    grid_dependency_wait();
    grid_launch_dependents();
    if (row >= a.rows) return;              // whole warps (ROW_WARP) or never
    RawCols x[NV], res[NV];
    auto fetch = [&](int64_t at) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            x[j] = load_raw_cols<T, WIDE>(static_cast<const T *>(a.x) + at * a.ldx, Columns<WIDE>::first(j, R, tid), n);
        if (a.residual) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                res[j] = load_raw_cols<T, WIDE>(static_cast<const T *>(a.residual) + at * a.ldr, Columns<WIDE>::first(j, R, tid), n);
        }
    };
    fetch(row);
    RawCols weight[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) weight[j] = load_raw_cols<T, WIDE>(static_cast<const T *>(a.weight), Columns<WIDE>::first(j, R, tid), n);
    for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
        float r[NV][E];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            unpack_cols<T, WIDE>(x[j], r[j]);
            if (a.residual) {
                float t[E];
                unpack_cols<T, WIDE>(res[j], t);
#pragma unroll
                for (int i = 0; i < E; ++i) r[j][i] += t[i];
            }
#pragma unroll
            for (int i = 0; i < E; ++i) sum += r[j][i] * r[j][i];
        }
        if (row + step < a.rows) fetch(row + step);
        if (a.residual_out) {
            T *ro = static_cast<T *>(a.residual_out) + row * a.ldro;
#pragma unroll
            for (int j = 0; j < NV; ++j) store_cols<T, WIDE>(ro, Columns<WIDE>::first(j, R, tid), n, r[j]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if constexpr (!ROW_WARP) {
            // written again two rows on, with the next row's barrier between
            if (lane == 0) s_sum[turn][warp] = sum;
            __syncthreads();
            sum = lane < static_cast<int>(blockDim.x >> 5) ? s_sum[turn][lane] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        }
        const float inv = 1.f / sqrtf(sum / static_cast<float>(n) + a.eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = Columns<WIDE>::first(j, R, tid);
            float w[E];
            unpack_cols<T, WIDE>(weight[j], w);
#pragma unroll
            for (int i = 0; i < E; ++i) r[j][i] = r[j][i] * inv * w[i];
            if (a.out) store_cols<T, WIDE>(static_cast<T *>(a.out) + row * a.ldo, c, n, r[j]);
            if (a.out_q)
                quantize_cols<WIDE>(r[j], c, n, a.out_q + row * a.ldq,
                                    a.out_scales + row * ((n + AWQ_FP8_BLOCK - 1) / AWQ_FP8_BLOCK), lane);
        }
    }
}

// A warp takes U neighbouring steps of 256 (wide) or 128 columns of a row, all
// their loads in flight together.
template <typename T, bool WIDE, int U>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantArgs a, int steps_per_row)
{
    constexpr int kCols = 32 * Columns<WIDE>::kElems;
    const int lane = threadIdx.x & 31;
    const int64_t s = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t row = s / steps_per_row;
    if (row >= a.rows) return;                          // whole warps
    const int c0 = static_cast<int>(s - row * steps_per_row) * kCols * U + Columns<WIDE>::first(0, 32, lane);
    grid_dependency_wait();
    grid_launch_dependents();
    float v[U][Columns<WIDE>::kElems];
#pragma unroll
    for (int u = 0; u < U; ++u) load_cols<T, WIDE>(static_cast<const T *>(a.x) + row * a.ldx, c0 + u * kCols, a.cols, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
        quantize_cols<WIDE>(v[u], c0 + u * kCols, a.cols, a.q + row * a.ldq,
                            a.scales + row * ((a.cols + AWQ_FP8_BLOCK - 1) / AWQ_FP8_BLOCK), lane);
}

// Steps of a warp and blocks of a multiprocessor where there are many steps
// (6000 x 8192, row stride 8448: 24.3 us; 4 steps with 5 blocks 28.6, with 3
// blocks 26.7; 8 steps with 2 blocks 25.3).
constexpr int kManySteps = 4, kManyBlocks = 4;

// The same for many steps, with a grid that stays: a warp goes on to the steps
// that are all the grid's warps further (row_step rows and col_step times U
// steps), whose loads are on their way while the present ones are written.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256, kManyBlocks) quantize_many_kernel(const QuantArgs a, int steps_per_row, int row_step, int col_step)
{
    constexpr int U = kManySteps, kCols = 32 * Columns<WIDE>::kElems;
    const int lane = threadIdx.x & 31;
    const int first = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    int64_t row = first / steps_per_row;
    int step = first - static_cast<int>(row) * steps_per_row;
    grid_dependency_wait();
    grid_launch_dependents();
    RawCols x[U];
    auto fetch = [&]() {
#pragma unroll
        for (int u = 0; u < U; ++u)
            x[u] = load_raw_cols<T, WIDE>(static_cast<const T *>(a.x) + row * a.ldx,
                                          (step * U + u) * kCols + Columns<WIDE>::first(0, 32, lane), a.cols);
    };
    if (row < a.rows) fetch();
    while (row < a.rows) {                              // whole warps
        float v[U][Columns<WIDE>::kElems];
#pragma unroll
        for (int u = 0; u < U; ++u) unpack_cols<T, WIDE>(x[u], v[u]);
        const int64_t at = row;
        const int c0 = step * U * kCols + Columns<WIDE>::first(0, 32, lane);
        row += row_step;
        step += col_step;
        if (step >= steps_per_row) {
            step -= steps_per_row;
            ++row;
        }
        if (row < a.rows) fetch();
#pragma unroll
        for (int u = 0; u < U; ++u)
            quantize_cols<WIDE>(v[u], c0 + u * kCols, a.cols, a.q + at * a.ldq,
                                a.scales + at * ((a.cols + AWQ_FP8_BLOCK - 1) / AWQ_FP8_BLOCK), lane);
    }
}

template <typename T, bool WIDE, int NV, int THREADS>
awq_status launch_norm_nv(const NormArgs &a, int threads, int sms, cudaStream_t st)
{
    const int64_t rows = THREADS == 128 ? 4 : 1;         // rows of a block (64 bits: the sum may pass 2^31)
    const int64_t grid = std::min<int64_t>((a.rows + rows - 1) / rows, sms * std::max(1, 2048 / threads));
    return launch(norm_kernel<T, WIDE, NV, THREADS>, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, 1, st, a);
}

template <typename T, bool WIDE>
awq_status launch_norm_w(const NormArgs &a, int sms, cudaStream_t st)
{
    constexpr int kChunk = 32 * Columns<WIDE>::kElems;   // columns of a warp's chunk
    const int chunks = (a.hidden + kChunk - 1) / kChunk;
    // A row per warp up to 4 chunks (16384 x 1024: 24.5 us; a row per block 26),
    // else a row per block: a chunk per warp for few rows (fewer steps in a
    // row's time), two where the rows are many and the row has more than 12
    // chunks (8192 x 5120: 52.9 us, 62 with one; 4096 x 8192: 23.6, 28.5 with
    // one, 26 with four). Narrow accesses take one up to 32 chunks, then four in
    // blocks of up to 512 threads, whose registers let two blocks share a
    // multiprocessor (8192 x 5120, stride 5125: 94.3 us, 143 with two chunks;
    // 4000 x 6001: 51.9, 81.2; as e4m3 too, 4000 x 4501: 61.9, 57.3).
    // Rows that need 1,024 threads with four chunks or more have 64 registers a
    // thread for them, and the compiler spills: wide from 16385 columns on 200 to
    // 310 bytes (2000 x 32768 with residual: 127 us bf16, 113 fp16, floor 77),
    // narrow from 8193 about 100 (2000 x 16383: 135 us, floor 39) and from 16385
    // 860 (2000 x 32767: 459 us, floor 77).
    if (chunks == 1) return launch_norm_nv<T, WIDE, 1, 128>(a, 128, sms, st);
    if (chunks == 2) return launch_norm_nv<T, WIDE, 2, 128>(a, 128, sms, st);
    if (chunks <= 4) return launch_norm_nv<T, WIDE, 4, 128>(a, 128, sms, st);
    const int most = WIDE && a.rows >= 4 * sms ? 12 : 32;
    if (chunks <= most) return launch_norm_nv<T, WIDE, 1, 1024>(a, 32 * chunks, sms, st);
    if constexpr (WIDE) {
        if (chunks <= 64) return launch_norm_nv<T, WIDE, 2, 1024>(a, 32 * ((chunks + 1) / 2), sms, st);
        return launch_norm_nv<T, WIDE, 4, 1024>(a, 32 * ((chunks + 3) / 4), sms, st);
    } else {
        if (chunks <= 64) return launch_norm_nv<T, WIDE, 4, 512>(a, 32 * ((chunks + 3) / 4), sms, st);
        if (chunks <= 128) return launch_norm_nv<T, WIDE, 4, 1024>(a, 32 * ((chunks + 3) / 4), sms, st);
        return launch_norm_nv<T, WIDE, 8, 1024>(a, 32 * ((chunks + 7) / 8), sms, st);
    }
}

template <typename T>
awq_status launch_norm_t(const NormArgs &a, bool wide, int sms, cudaStream_t st)
{
    return wide ? launch_norm_w<T, true>(a, sms, st) : launch_norm_w<T, false>(a, sms, st);
}

template <typename T, bool WIDE, int U>
awq_status launch_quantize_u(const QuantArgs &a, cudaStream_t st)
{
    const int per = 32 * Columns<WIDE>::kElems * U;
    const int steps_per_row = (a.cols + per - 1) / per;
    const int64_t blocks = (static_cast<int64_t>(a.rows) * steps_per_row + 7) / 8;
    if (blocks > 0x7fffffff) return AWQ_ERR_UNSUPPORTED_SHAPE;
    return launch(quantize_kernel<T, WIDE, U>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, 1, st, a, steps_per_row);
}

template <typename T, bool WIDE>
awq_status launch_quantize_w(const QuantArgs &a, int sms, cudaStream_t st)
{
    // One step a warp where the warps should spread (48 x 4096: 1.2 us, 1.5 with
    // two), two where there are several rounds of them (2000 x 2560: 3.1 us;
    // 16384 x 2560: 27.6 us with one, 23.0 with two), and a grid that stays where
    // there are many rounds and few of its steps lie past a row's end (16384 x
    // 2560: 22.0 us; 6000 x 8192, stride 8448: 24.3, 26.6 with two steps a warp;
    // 8000 x 2560: 12.0, 12.3; but 4000 x 2560: 7.3, 6.1, and 16384 x 400: 6.6, 4.5).
    const int per = 32 * Columns<WIDE>::kElems, row_steps = (a.cols + per - 1) / per;
    const int many_steps = (row_steps + kManySteps - 1) / kManySteps;
    const int64_t steps = static_cast<int64_t>(a.rows) * row_steps;
    if (steps >= 400ll * sms && 4ll * kManySteps * many_steps <= 5ll * row_steps) {
        const int warps = 8 * kManyBlocks * sms;
        return launch(quantize_many_kernel<T, WIDE>, dim3(kManyBlocks * sms), dim3(256), 0, 1, st, a, many_steps,
                      warps / many_steps, warps % many_steps);
    }
    return steps >= 64ll * sms ? launch_quantize_u<T, WIDE, 2>(a, st) : launch_quantize_u<T, WIDE, 1>(a, st);
}

template <typename T>
awq_status launch_quantize_t(const QuantArgs &a, bool wide, int sms, cudaStream_t st)
{
    return wide ? launch_quantize_w<T, true>(a, sms, st) : launch_quantize_w<T, false>(a, sms, st);
}

}  // namespace

awq_status launch_norm(const NormArgs &a, int dtype, bool wide, int sms, cudaStream_t st)
{
    return dtype == AWQ_DTYPE_F16 ? launch_norm_t<__half>(a, wide, sms, st) : launch_norm_t<__nv_bfloat16>(a, wide, sms, st);
}

awq_status launch_quantize(const QuantArgs &a, int dtype, bool wide, int sms, cudaStream_t st)
{
    return dtype == AWQ_DTYPE_F16 ? launch_quantize_t<__half>(a, wide, sms, st)
                                  : launch_quantize_t<__nv_bfloat16>(a, wide, sms, st);
}

}  // namespace awq
