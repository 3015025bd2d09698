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
    return __builtin_convertvector(v, typename Mat<T>::Frag);
}

// 8 float32 values as kTerms fragments that add up to them (bfloat16: the
// rounded value, the rounded rest, and the rest of that; float32: the values).
template <typename T>
__device__ __forceinline__ void split_frag(f32x8 v, typename Mat<T>::Frag (&f)[Mat<T>::kTerms])
{
#pragma unroll
    for (int n = 0; n < Mat<T>::kTerms; n++) {
        f[n] = round_frag<T>(v);
        v -= __builtin_convertvector(f[n], f32x8);
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

// Four rows of column l % 16 of a 16-column block of an LDS tile, rows from
// row0 (the same for the 16 lanes that share l / 16).  Bfloat16: the gfx950
// transposing read, in which lane l of the 16 fetches 8 bytes of row l / 4 and
// receives column l of the 4 x 16 block.
__device__ __forceinline__ bf16x4 col4(const bf16 *tile, int ld, int row0, int col0)
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    const int li = threadIdx.x & 15;
    const bf16 *p = tile + (row0 + (li >> 2)) * ld + col0 + (li & 3) * 4;
    return __builtin_bit_cast(
        bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p));
}

__device__ __forceinline__ f32x4 col4(const float *tile, int ld, int row0, int col0)
{
    const float *p = tile + row0 * ld + col0 + (threadIdx.x & 15);
    return f32x4{p[0], p[ld], p[2 * ld], p[3 * ld]};
}

// Column fragment: columns col0 + l % 16, k (the tile's rows) from k0.
template <typename T>
__device__ __forceinline__ typename Mat<T>::Frag frag_col(const T *tile, int ld, int k0, int col0)
{
    const int r = k0 + ((threadIdx.x & 63) >> 4) * 8;
    return __builtin_shufflevector(col4(tile, ld, r, col0), col4(tile, ld, r + 4, col0), 0, 1, 2, 3, 4,
                                   5, 6, 7);
}

// Fragments whose k order is that of two accumulator tiles, 16 apart: k0 + 4 g
// .. + 3 and k0 + 16 + 4 g .. + 3 with g = l / 16.  A column fragment, a row
// fragment, and the accumulator tiles themselves, rounded.
template <typename T>
__device__ __forceinline__ typename Mat<T>::Frag frag_col_pair(const T *tile, int ld, int k0, int col0)
{
    const int r = k0 + ((threadIdx.x & 63) >> 4) * 4;
    return __builtin_shufflevector(col4(tile, ld, r, col0), col4(tile, ld, r + 16, col0), 0, 1, 2, 3, 4,
                                   5, 6, 7);
}

template <typename T>
__device__ __forceinline__ typename Mat<T>::Frag frag_row_pair(const T *tile, int ld, int row0, int k0)
{
    const int l = threadIdx.x & 63;
    const T *q = tile + (row0 + (l & 15)) * ld + k0 + (l >> 4) * 4;
    return __builtin_shufflevector(*reinterpret_cast<const typename Mat<T>::Half *>(q),
                                   *reinterpret_cast<const typename Mat<T>::Half *>(q + 16), 0, 1, 2, 3,
                                   4, 5, 6, 7);
}

template <typename T>
__device__ __forceinline__ typename Mat<T>::Frag frag_acc(f32x4 a, f32x4 b)
{
    return round_frag<T>(__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Reads of a strided tensor through a buffer descriptor: an element offset that
// is masked out (kOut) is not read and gives zero, with no branch around the
// load.  VEC: 16-byte accesses (rows on 16 bytes, columns a multiple of them);
// else element by element.  Offsets from the descriptor's base stay below
// 2^31 bytes: the base is the tile's first row, and row strides are limited.
constexpr uint32_t kOut = 0x80000000u;

template <typename T>
struct Source {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ explicit Source(const T *p)
        : r(__builtin_amdgcn_make_buffer_rsrc((void *)p, 0, (int)kOut, 0x27000))
    {
    }
    // V elements from element offset `off`, `n` of them (vectors: all or none)
    template <int V, bool VEC>
    __device__ __forceinline__ Vec<T, V> read(uint32_t off, int n) const
    {
        static_assert(V * sizeof(T) == 16, "16-byte vectors");
        if constexpr (VEC) {
            using Out = Vec<T, V>;
            return __builtin_bit_cast(
                Out,
                __builtin_amdgcn_raw_buffer_load_b128(r, n > 0 ? off * (uint32_t)sizeof(T) : kOut, 0, 0));
        } else {
            Vec<T, V> v;
#pragma unroll
            for (int i = 0; i < V; i++) {
                const uint32_t at = i < n ? (off + i) * (uint32_t)sizeof(T) : kOut;
                if constexpr (sizeof(T) == 2)
                    v.e[i] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0));
                else
                    v.e[i] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
            }
            return v;
        }
    }
};

// Writes through a buffer descriptor: four elements from element offset `off`,
// of which `n` are stored (vectors: all or none), with no branch.
template <typename T>
struct Sink {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ explicit Sink(T *p)
        : r(__builtin_amdgcn_make_buffer_rsrc((void *)p, 0, (int)kOut, 0x27000))
    {
    }
    template <bool VEC>
    __device__ __forceinline__ void write4(uint32_t off, int n, f32x4 v) const
    {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        const auto out = __builtin_convertvector(v, typename Mat<T>::Half);
        if constexpr (VEC) {
            const uint32_t at = n > 0 ? off * (uint32_t)sizeof(T) : kOut;
            if constexpr (sizeof(T) == 2)
                __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, out), r, at, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, out), r, at, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t at = i < n ? (off + i) * (uint32_t)sizeof(T) : kOut;
                if constexpr (sizeof(T) == 2)
                    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, (T)out[i]), r, at, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, (T)out[i]), r, at, 0, 0);
            }
        }
    }
};

// A ROWS x COLS tile (LDS row stride LD) in two steps, so that a load can be in
// flight while the previous tile is worked on: rows of a strided tensor to
// registers, registers to LDS.  Rows from `rows` and columns from `cols` on
// become zero and are not read.
template <typename T, int ROWS, int COLS, int LD, int THREADS, bool VEC>
struct TileRegs {
    static constexpr int V = 16 / sizeof(T);
    static constexpr int PER = COLS / V;
    static constexpr int N = (ROWS * PER + THREADS - 1) / THREADS;
    static constexpr bool kWhole = ROWS * PER % THREADS == 0;
    Vec<T, V> v[N];

    __device__ __forceinline__ void load(const T *src, int64_t stride, int rows, int cols)
    {
        const Source<T> s(src);
#pragma unroll
        for (int u = 0; u < N; u++) {
            const int e = threadIdx.x + u * THREADS;
            const int r = e / PER, c = (e % PER) * V;
            v[u] = s.template read<V, VEC>((uint32_t)r * (uint32_t)stride + c, r < rows && r < ROWS ? cols - c : 0);
        }
    }
    __device__ __forceinline__ void store(T *tile) const
    {
#pragma unroll
        for (int u = 0; u < N; u++) {
            const int e = threadIdx.x + u * THREADS;
            if (kWhole || e < ROWS * PER) vstore<T, V>(tile + (e / PER) * LD + (e % PER) * V, v[u]);
        }
    }
};

template <typename T, int ROWS, int COLS, int LD, int THREADS, bool VEC>
__device__ __forceinline__ void load_tile(T *tile, const T *src, int64_t stride, int rows, int cols)
{
    TileRegs<T, ROWS, COLS, LD, THREADS, VEC> t;
    t.load(src, stride, rows, cols);
    t.store(tile);
}

// Columns c .. c + 3 of a row of D, rounded; those from D on are not stored.
template <typename T, bool VEC>
__device__ __forceinline__ void store4(T *row, int c, int D, f32x4 v)
{
    const auto out = __builtin_convertvector(v, typename Mat<T>::Half);
    if constexpr (VEC) {
        if (c < D) *reinterpret_cast<typename Mat<T>::Half *>(row + c) = out;
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (c + i < D) row[c + i] = out[i];
    }
}

// A whole row of D: v[j] holds columns 16 j + 4 g .. + 3.  bfloat16 lanes g and
// g ^ 1 first trade halves of two neighbouring blocks, so that a lane stores 16
// bytes and a row gets 64 in one piece.
template <typename T, int DT, bool VEC>
__device__ __forceinline__ void store_row(T *row, int D, const f32x4 *v)
{
    const int g = (threadIdx.x & 63) >> 4;
    if constexpr (VEC && sizeof(T) == 2) {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        const int c0 = 16 * (g & 1) + 4 * (g & 2);
#pragma unroll
        for (int j = 0; j < DT; j += 2) {
            const u32x2 a = __builtin_bit_cast(u32x2, __builtin_convertvector(v[j], typename Mat<T>::Half));
            const u32x2 b = __builtin_bit_cast(u32x2, __builtin_convertvector(v[j + 1], typename Mat<T>::Half));
            const auto x = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
            const auto y = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
            if (16 * j + c0 < D) *reinterpret_cast<u32x4 *>(row + 16 * j + c0) = u32x4{x[0], y[0], x[1], y[1]};
        }
    } else {
#pragma unroll
        for (int j = 0; j < DT; j++) store4<T, VEC>(row, 16 * j + 4 * g, D, v[j]);
    }
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

}  // namespace
}  // namespace sdm
