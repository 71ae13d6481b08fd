// Rows of float32, bfloat16 or binary16 values: 16-byte pieces read and
// written at any alignment of the element type, and the bounds that let a
// division by a run-time constant be two multiplications.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ivfpq {

// Workgroups of one launch (a multiple of 8): a launch takes fewer than 2^32 threads.
constexpr int64_t most_blocks(int threads) { return (0xFFFFFFFFll / threads) & ~7ll; }

// Element types of the row operators (ivfpq_type of the header).
enum RowType { kF32 = 0, kBF16 = 1, kF16 = 2 };

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A 16-byte piece of a row (4 float32 or 8 sixteen-bit values).  The target
// reads global memory at any element alignment, so one wide load serves rows
// of odd length and views alike.
template <typename T>
struct Piece {
    static constexpr int N = 16 / (int)sizeof(T);
    typedef T V __attribute__((ext_vector_type(N), aligned(sizeof(T))));
    float v[N];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = 0.f;
    }
    // valid: elements inside the row; the others read as zero
    __device__ __forceinline__ void load(const T *p, int valid)
    {
        if (valid >= N) {
            const V w = *reinterpret_cast<const V *>(p);
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = (float)w[i];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = i < valid ? (float)p[i] : 0.f;
        }
    }
    // NT: past the caches, for rows that nothing reads soon
    template <bool NT = false>
    __device__ __forceinline__ void store(T *p, int valid) const
    {
        if (valid >= N) {
            V w;
#pragma unroll
            for (int i = 0; i < N; ++i)
                w[i] = (T)v[i];
            if constexpr (NT)
                __builtin_nontemporal_store(w, reinterpret_cast<V *>(p));
            else
                *reinterpret_cast<V *>(p) = w;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < valid)
                    p[i] = (T)v[i];
        }
    }
};

// n / c for 32-bit n and a divisor known on the host: the high word of
// n * (floor(2^64 / c) + 1), exact for every n < 2^32 (c >= 2).
struct FastDiv {
    uint32_t c = 1;
    uint64_t m = 0;
    FastDiv() = default;
    explicit FastDiv(uint32_t divisor) : c(divisor), m(divisor > 1 ? ~0ull / divisor + 1 : 0) {}
    __device__ __forceinline__ uint32_t div(uint32_t n) const
    {
        return c == 1 ? n : (uint32_t)__umul64hi((uint64_t)n, m);
    }
};

} // namespace ivfpq
