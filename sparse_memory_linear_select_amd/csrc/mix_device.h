// Device helpers shared by the sequence mixers: element conversion and vector
// loads and stores of float32 and bfloat16 rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdm {
namespace {

using bf16 = __bf16;

// V consecutive elements, moved by one access of sizeof(T) * V bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> vload(const T *p)
{
    return *reinterpret_cast<const Vec<T, V> *>(p);
}

template <typename T, int V>
__device__ __forceinline__ void vstore(T *p, const Vec<T, V> &v)
{
    *reinterpret_cast<Vec<T, V> *>(p) = v;
}

// Tokens of sequence b: lengths[b] clamped to [0, T], or T.
__device__ __forceinline__ int64_t seq_len(const int32_t *lengths, int64_t b, int64_t T)
{
    if (!lengths) return T;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n > T ? T : n;
}

}  // namespace
}  // namespace sdm
