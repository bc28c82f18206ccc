// Pairs of a head's elements, their rotation and the stores to a paged cache:
// what the append with and without the norm of each head share.
#pragma once

#include "awq_decoder_kernels.cuh"

namespace awq {

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

}  // namespace awq
