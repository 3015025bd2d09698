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

// ------------------------------------------------------------------------
// 16x16 matrix products of a wave.  A fragment holds, for lane l, row (or
// column) l % 16 of the operand and the 8 k indices (l / 16) * 8 .. + 7 of a
// block of 32; the result holds column l % 16 and rows (l / 16) * 4 .. + 3.
// Bfloat16 takes one v_mfma_f32_16x16x32_bf16; float32 takes eight
// v_mfma_f32_16x16x4_f32, the i-th with element i of every lane (a sum over k
// does not care which k indices share an instruction).

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct Mat;

template <>
struct Mat<bf16> {
    using Frag = bf16x8;
    using Half = bf16x4;
    // A float32 weight is carried to about 24 bits by three bfloat16 terms.
    static constexpr int kTerms = 3;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

template <>
struct Mat<float> {
    using Frag = f32x8;
    using Half = f32x4;
    static constexpr int kTerms = 1;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c)
    {
#pragma unroll
        for (int i = 0; i < 8; i++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
};

// Rounds 8 float32 values to a fragment.
template <typename T>
__device__ __forceinline__ typename Mat<T>::Frag round_frag(f32x8 v)
{
    typename Mat<T>::Frag f;
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = (T)v[i];
    return f;
}

// 8 float32 values as kTerms fragments that add up to them (bfloat16: the
// rounded value, the rounded rest, and the rest of that; float32: the values).
template <typename T>
__device__ __forceinline__ void split_frag(f32x8 v, typename Mat<T>::Frag (&f)[Mat<T>::kTerms])
{
#pragma unroll
    for (int n = 0; n < Mat<T>::kTerms; n++) {
        f[n] = round_frag<T>(v);
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] -= (float)f[n][i];
    }
}

// Row fragment of a row-major LDS tile: rows row0 + l % 16, k from k0.
template <typename T>
__device__ __forceinline__ typename Mat<T>::Frag frag_row(const T *tile, int ld, int row0, int k0)
{
    const int l = threadIdx.x & 63;
    return *reinterpret_cast<const typename Mat<T>::Frag *>(tile + (row0 + (l & 15)) * ld + k0 +
                                                            (l >> 4) * 8);
}

// Column fragment: columns col0 + l % 16, k (the tile's rows) from k0.
template <typename T>
__device__ __forceinline__ typename Mat<T>::Frag frag_col(const T *tile, int ld, int k0, int col0)
{
    const int l = threadIdx.x & 63;
    const T *p = tile + (k0 + (l >> 4) * 8) * ld + col0 + (l & 15);
    typename Mat<T>::Frag f;
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = p[i * ld];
    return f;
}

// Fills a ROWS x COLS tile in LDS (row stride LD) from rows of a strided
// tensor; rows from `rows` and columns from `cols` on become zero and are not
// read.  vec: every row starts on 16 bytes and cols is a multiple of 16 bytes.
template <typename T, int ROWS, int COLS, int LD, int THREADS>
__device__ __forceinline__ void load_tile(T *tile, const T *src, int64_t stride, int rows, int cols,
                                          bool vec)
{
    constexpr int V = 16 / sizeof(T);
    constexpr int PER = COLS / V;
    const int tid = threadIdx.x;
    for (int e = tid; e < ROWS * PER; e += THREADS) {
        const int r = e / PER, c = (e % PER) * V;
        Vec<T, V> v;
        if (vec && r < rows && c < cols) {
            v = vload<T, V>(src + r * stride + c);
        } else {
#pragma unroll
            for (int i = 0; i < V; i++)
                v.e[i] = r < rows && c + i < cols ? src[r * stride + c + i] : (T)0.f;
        }
        vstore<T, V>(tile + r * LD + c, v);
    }
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ bool rows_aligned(const void *p, int64_t s0, int64_t s1, int cols, int esize)
{
    return (((uintptr_t)p | (uintptr_t)(s0 * esize) | (uintptr_t)(s1 * esize) |
             (uintptr_t)(cols * esize)) & 15u) == 0;
}

}  // namespace
}  // namespace sdm
