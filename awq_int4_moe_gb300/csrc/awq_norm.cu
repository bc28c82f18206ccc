// awq_add_rmsnorm and awq_quantize_fp8.
//
//   r = x + residual, y = r / sqrt(mean(r^2) + eps) * w, and y in e4m3 with
//   a scale of amax / 448 per group of 128 columns.
//
// Each element is read once and written once per output: a row lives in the
// registers of one block (or one warp) between its sum of squares and its
// outputs. About six operations per element: bound by the bytes for many
// rows, by the launch and one block's dependent steps for few.
//
// Columns are dealt so that a quantisation group never leaves a warp: with
// 16-byte accesses (wide) 16 neighbouring lanes hold a group, 8 columns each;
// otherwise a warp holds it, lane l the columns l, l + 32, l + 64, l + 96 (one
// element per access, neighbouring lanes side by side). Its amax is a few
// shuffles.
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

template <typename T, bool WIDE>
__device__ __forceinline__ void load_cols(const T *row, int c, int n, float (&f)[Columns<WIDE>::kElems])
{
    if constexpr (WIDE) {
        if (c < n)
            load_elems<T, 8>(row + c, f);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = c + 32 * i < n ? to_f32(row[c + 32 * i]) : 0.f;
    }
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

// NV chunks of a row per thread. ROW_WARP: a row per warp, blockDim.x / 32
// rows per block; else a row per block.
template <typename T, bool WIDE, int NV, bool ROW_WARP>
__global__ void __launch_bounds__(ROW_WARP ? 128 : 1024) norm_kernel(const NormArgs a)
{
    constexpr int E = Columns<WIDE>::kElems;
    __shared__ float s_sum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = ROW_WARP ? 32 : blockDim.x;
    const int tid = ROW_WARP ? lane : threadIdx.x;
    const int64_t row = ROW_WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
    const int n = a.hidden;
    grid_dependency_wait();
    grid_launch_dependents();
    if (row >= a.rows) return;              // whole warps (ROW_WARP) or never
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    float r[NV][E];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_cols<T, WIDE>(x, Columns<WIDE>::first(j, R, tid), n, r[j]);
    if (a.residual) {
        const T *res = static_cast<const T *>(a.residual) + row * a.ldr;
        float t[NV][E];
#pragma unroll
        for (int j = 0; j < NV; ++j) load_cols<T, WIDE>(res, Columns<WIDE>::first(j, R, tid), n, t[j]);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < E; ++i) r[j][i] += t[j][i];
    }
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) sum += r[j][i] * r[j][i];
    if (a.residual_out) {
        T *ro = static_cast<T *>(a.residual_out) + row * a.ldro;
#pragma unroll
        for (int j = 0; j < NV; ++j) store_cols<T, WIDE>(ro, Columns<WIDE>::first(j, R, tid), n, r[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if constexpr (!ROW_WARP) {
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        sum = lane < static_cast<int>(blockDim.x >> 5) ? s_sum[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    }
    const float inv = 1.f / sqrtf(sum / static_cast<float>(n) + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = Columns<WIDE>::first(j, R, tid);
        float w[E];
        load_cols<T, WIDE>(static_cast<const T *>(a.weight), c, n, w);
#pragma unroll
        for (int i = 0; i < E; ++i) r[j][i] = r[j][i] * inv * w[i];
        if (a.out) store_cols<T, WIDE>(static_cast<T *>(a.out) + row * a.ldo, c, n, r[j]);
        if (a.out_q)
            quantize_cols<WIDE>(r[j], c, n, a.out_q + row * a.ldq,
                                a.out_scales + row * ((n + AWQ_FP8_BLOCK - 1) / AWQ_FP8_BLOCK), lane);
    }
}

// One warp per step of 256 (wide) or 128 columns of a row.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantArgs a, int64_t steps, int steps_per_row)
{
    constexpr int kCols = 32 * Columns<WIDE>::kElems;
    const int lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); s < steps; s += stride) {
        const int64_t row = s / steps_per_row;
        const int c = static_cast<int>(s - row * steps_per_row) * kCols + Columns<WIDE>::first(0, 32, lane);
        float v[Columns<WIDE>::kElems];
        load_cols<T, WIDE>(static_cast<const T *>(a.x) + row * a.ldx, c, a.cols, v);
        quantize_cols<WIDE>(v, c, a.cols, a.q + row * a.ldq,
                            a.scales + row * ((a.cols + AWQ_FP8_BLOCK - 1) / AWQ_FP8_BLOCK), lane);
    }
}

template <typename T, bool WIDE, int NV>
awq_status launch_norm_nv(const NormArgs &a, int row_threads, cudaStream_t st)
{
    if (row_threads == 32)
        return launch(norm_kernel<T, WIDE, NV, true>, dim3((a.rows + 3) / 4), dim3(128), 0, 1, st, a);
    return launch(norm_kernel<T, WIDE, NV, false>, dim3(a.rows), dim3(row_threads), 0, 1, st, a);
}

template <typename T>
awq_status launch_norm_t(const NormArgs &a, bool wide, cudaStream_t st)
{
    // chunks of the row a warp holds: 256 columns wide, 128 otherwise
    const int chunks = (a.hidden + (wide ? 255 : 127)) / (wide ? 256 : 128);
    // a row per warp up to 4 chunks, else a row per block of up to 32 warps
    const int nv = chunks <= 4 ? chunks : (chunks + 31) / 32;
    const int threads = chunks <= 4 ? 32 : (chunks + nv - 1) / nv * 32;
    if (wide)
        return nv == 1   ? launch_norm_nv<T, true, 1>(a, threads, st)
               : nv == 2 ? launch_norm_nv<T, true, 2>(a, threads, st)
                         : launch_norm_nv<T, true, 4>(a, threads, st);
    return nv == 1   ? launch_norm_nv<T, false, 1>(a, threads, st)
           : nv == 2 ? launch_norm_nv<T, false, 2>(a, threads, st)
           : nv <= 4 ? launch_norm_nv<T, false, 4>(a, threads, st)
                     : launch_norm_nv<T, false, 8>(a, threads, st);
}

template <typename T>
awq_status launch_quantize_t(const QuantArgs &a, bool wide, int sms, cudaStream_t st)
{
    const int per = wide ? 256 : 128;
    const int steps_per_row = (a.cols + per - 1) / per;
    const int64_t steps = static_cast<int64_t>(a.rows) * steps_per_row;
    const int grid = static_cast<int>(min(steps / 8 + (steps % 8 != 0), static_cast<int64_t>(sms) * 64));
    return wide ? launch(quantize_kernel<T, true>, dim3(grid), dim3(256), 0, 1, st, a, steps, steps_per_row)
                : launch(quantize_kernel<T, false>, dim3(grid), dim3(256), 0, 1, st, a, steps, steps_per_row);
}

}  // namespace

awq_status launch_norm(const NormArgs &a, int dtype, bool wide, int, cudaStream_t st)
{
    return dtype == AWQ_DTYPE_F16 ? launch_norm_t<__half>(a, wide, st) : launch_norm_t<__nv_bfloat16>(a, wide, st);
}

awq_status launch_quantize(const QuantArgs &a, int dtype, bool wide, int sms, cudaStream_t st)
{
    return dtype == AWQ_DTYPE_F16 ? launch_quantize_t<__half>(a, wide, sms, st)
                                  : launch_quantize_t<__nv_bfloat16>(a, wide, sms, st);
}

}  // namespace awq
