// Causal attention with a sliding window and sinks: query i sees key j where
// j <= i and (i - j < window or j < sinks).  Hq / Hk query heads share a key
// head.
//
// Scores are computed transposed, S^T = K Q^T, so that a lane holds one query
// (column) and four neighbouring keys: the softmax of a query is a reduction
// over registers and two lane exchanges, and P^T is already the right operand
// of O^T += V^T P^T.  One pass over the keys with the running maximum m and
// sum l of 2^{s - m}, s in units of log2.
#include "mix_internal.h"

#include "lane_ops.h"
#include "mix_device.h"

namespace sdm {
namespace {

constexpr int kRows = 64;     // queries of a workgroup: 16 a wave
constexpr int kKeys = 64;     // keys of a tile
constexpr int kThreads = 256;
constexpr int kSinkRows = 512;  // queries whose sink gradients one workgroup sums

struct WinDims {
    int B, Hq, Hk, D;
    int64_t T, W;
    int S;
    float c2;                   // scale * log2 e
    float scale;
    int64_t qb, qt, qh, kb, kt, kh, vb, vt, vh;
    int64_t cap;                // rows of the cache: S + W
    int nq;                     // query tiles
};

// Tokens of sequence b before the call.
__device__ __forceinline__ int64_t seq_pos(const int64_t *pos, int64_t b)
{
    return pos && pos[b] > 0 ? pos[b] : 0;
}

__device__ __forceinline__ int64_t cache_slot(int64_t p, int64_t S, int64_t W)
{
    return p < S ? p : S + (p - S) % W;
}

// Fills a 64-row tile: row r from row_of(r) (null: zeros).  D columns, padded
// with zeros to COLS.
template <typename T, int COLS, int LD, typename F>
__device__ __forceinline__ void load_rows(T *tile, F row_of, int D, bool vec)
{
    constexpr int V = 16 / sizeof(T);
    constexpr int PER = COLS / V;
    for (int e = threadIdx.x; e < 64 * PER; e += kThreads) {
        const int r = e / PER, c = (e % PER) * V;
        const T *src = row_of(r);
        Vec<T, V> v;
        if (vec && src && c < D) {
            v = vload<T, V>(src + c);
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) v.e[i] = src && c + i < D ? src[c + i] : (T)0.f;
        }
        vstore<T, V>(tile + r * LD + c, v);
    }
}

// Fragment of a row in global memory: 8 elements from k, zeros from D on.
template <typename T>
__device__ __forceinline__ typename Mat<T>::Frag frag_global(const T *src, int k, int D, bool vec)
{
    typename Mat<T>::Frag f;
    if (src && vec && k < D) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int u = 0; u < 8 / V; u++) {
            const Vec<T, V> v = vload<T, V>(src + k + u * V);
#pragma unroll
            for (int i = 0; i < V; i++) f[u * V + i] = v.e[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = src && k + i < D ? src[k + i] : (T)0.f;
    }
    return f;
}

// The keys that the queries i0 .. i1 (positions) can see, as one list: the
// sinks in front of every window, then the keys from lo on.  Entry v is a sink
// that is always seen where v < S; jr(v) = its position - i0 (for entries in
// front of lo some number below that of lo: they precede every query).
struct KeyList {
    int64_t lo;     // first key of the window part
    int ns, total;  // sinks in front of it; entries
    int shift;      // jr(v) = v + shift
    __device__ KeyList(int64_t i0, int64_t i1, int64_t W, int S)
    {
        lo = i0 - W + 1 > 0 ? i0 - W + 1 : 0;
        ns = S < lo ? S : (int)lo;
        total = ns + (int)(i1 - lo + 1);
        shift = (int)(lo - i0) - ns;
    }
    __device__ int64_t key(int v) const { return v < ns ? v : lo + (v - ns); }
};

// What 16 neighbouring entries from v0 are to 16 neighbouring queries from ir0
// (relative to i0): 0 none is seen, 1 some are, 2 all are.
__device__ __forceinline__ int block_sight(int v0, int shift, int ir0, int W, int S)
{
    const int j0 = v0 + shift, j1 = j0 + 15, ir1 = ir0 + 15;
    if (j0 > ir1 || (v0 >= S && j1 <= ir0 - W)) return 0;
    return j1 <= ir0 && (j0 > ir1 - W || v0 + 15 < S) ? 2 : 1;
}

// A 64-row tile in two steps, as TileRegs, from rows given by pointers.  Every
// access is to a row that exists: columns from D on hold the row's first ones
// (finite numbers that meet zeros in the other operand, or columns nobody
// stores).
template <typename T, int COLS, int LD, bool VEC>
struct RowRegs {
    static constexpr int V = 16 / sizeof(T);
    static constexpr int PER = COLS / V;
    static constexpr int N = 64 * PER / kThreads;
    Vec<T, V> v[N];

    template <typename F>
    __device__ __forceinline__ void load(F row_of, int D)
    {
#pragma unroll
        for (int u = 0; u < N; u++) {
            const int e = threadIdx.x + u * kThreads;
            const int c = (e % PER) * V;
            const T *src = row_of(e / PER);
            if constexpr (VEC) {
                v[u] = vload<T, V>(src + (c < D ? c : 0));
            } else {
#pragma unroll
                for (int i = 0; i < V; i++) v[u].e[i] = src[c + i < D ? c + i : 0];
            }
        }
    }
    __device__ __forceinline__ void store(T *tile) const
    {
#pragma unroll
        for (int u = 0; u < N; u++) {
            const int e = threadIdx.x + u * kThreads;
            vstore<T, V>(tile + (e / PER) * LD + (e % PER) * V, v[u]);
        }
    }
};

// Workgroups are dealt to the 8 XCDs in turn; a run of neighbouring indexes on
// one XCD shares its L2.
__device__ __forceinline__ int64_t xcd_index(int64_t id, int64_t n)
{
    const int64_t per = n / 8, cut = per * 8;
    return id < cut ? (id % 8) * per + id / 8 : id;
}

__device__ __forceinline__ float pair_max(float x, int m)
{
    uint32_t lo, hi;
    pair_vals(__float_as_uint(x), m, lo, hi);
    return fmaxf(__uint_as_float(lo), __uint_as_float(hi));
}

// A wave holds QN blocks of 16 queries, over which it uses each fragment of K
// and V twice: the same queries of two heads that share a key head (HP = 2),
// or 32 neighbouring queries.  A workgroup is four waves: 64 queries of two
// heads, or 64 QN queries of one.
template <typename T, int DT, int QN, int HP, bool VEC, bool CACHE>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 && DT <= 8 ? 2 : 1) void window_fwd_kernel(
    WinDims d, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
    const T *__restrict__ ck, const T *__restrict__ cv, const int64_t *__restrict__ pos,
    const int32_t *__restrict__ lengths, T *__restrict__ o, float *__restrict__ lse)
{
    using M = Mat<T>;
    using Half = typename M::Half;
    constexpr int LD = DT * 16 + 8;
    constexpr int QR = HP == 2 ? 16 : 16 * QN;   // queries of a wave
    constexpr int kBufs = 4 * 64 * LD * (int)sizeof(T) <= 160 * 1024 ? 2 : 1;
    __shared__ __align__(32) T Ks[kBufs][kKeys * LD];
    __shared__ __align__(32) T Vs[kBufs][kKeys * LD];

    const int64_t blk = xcd_index(blockIdx.x, gridDim.x);
    const int qt = (int)(blk % d.nq);
    const int64_t bh = blk / d.nq;
    const int h0 = (int)(bh % (d.Hq / HP)) * HP;
    const int64_t b = bh / (d.Hq / HP);
    const int hk = h0 / (d.Hq / d.Hk);
    const int64_t len = seq_len(lengths, b, d.T);
    const int64_t p0 = CACHE ? seq_pos(pos, b) : 0;
    const int64_t t0 = (int64_t)qt * 4 * QR;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l = threadIdx.x & 63, g = l >> 4;
    const int W = (int)d.W, S = d.S;
    int ir[QN];                  // the lane's queries, relative to t0
    int64_t at[QN];              // their rows of o and lse
#pragma unroll
    for (int u = 0; u < QN; u++) {
        ir[u] = QR * w + (HP == 2 ? 0 : 16 * u) + (l & 15);
        at[u] = (b * d.T + t0 + ir[u]) * d.Hq + h0 + (HP == 2 ? u : 0);
    }
    f32x4 O[QN][DT];
    float m[QN], sum[QN];
#pragma unroll
    for (int u = 0; u < QN; u++) {
        m[u] = -INFINITY;
        sum[u] = 0.f;
#pragma unroll
        for (int j = 0; j < DT; j++) O[u][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (t0 < len) {
        typename M::Frag qf[QN][DT / 2];
#pragma unroll
        for (int u = 0; u < QN; u++) {
            const T *row = t0 + ir[u] < len ? q + b * d.qb + (t0 + ir[u]) * d.qt +
                                                  (h0 + (HP == 2 ? u : 0)) * d.qh
                                            : nullptr;
#pragma unroll
            for (int ks = 0; ks < DT / 2; ks++) qf[u][ks] = frag_global<T>(row, 32 * ks + 8 * g, d.D, VEC);
        }
        const int64_t last = (t0 + 4 * QR < len ? t0 + 4 * QR : len) - 1;
        const KeyList kl(p0 + t0, p0 + last, d.W, S);
        const int nt = (kl.total + kKeys - 1) / kKeys;
        const T *kn = k + b * d.kb + hk * d.kh, *vn = v + b * d.vb + hk * d.vh;
        RowRegs<T, DT * 16, LD, VEC> rk, rv;
        const auto fetch = [&](int n) {
            const auto key = [&](int r) {
                const int e = n * kKeys + r;
                return kl.key(e < kl.total ? e : kl.total - 1);
            };
            rk.load([&](int r) {
                const int64_t j = key(r);
                if (CACHE && j < p0) return ck + ((b * d.cap + cache_slot(j, S, W)) * d.Hk + hk) * d.D;
                return kn + (j - p0) * d.kt;
            }, d.D);
            rv.load([&](int r) {
                const int64_t j = key(r);
                if (CACHE && j < p0) return cv + ((b * d.cap + cache_slot(j, S, W)) * d.Hk + hk) * d.D;
                return vn + (j - p0) * d.vt;
            }, d.D);
        };
        fetch(0);
        rk.store(Ks[0]);
        rv.store(Vs[0]);
        __syncthreads();
        for (int n = 0; n < nt; n++) {
            const int buf = kBufs == 2 ? n & 1 : 0;
            if (n + 1 < nt) fetch(n + 1);
            const int v0 = n * kKeys;
            int sight[QN][4];
            bool any = false;
#pragma unroll
            for (int u = 0; u < QN; u++)
#pragma unroll
                for (int kt = 0; kt < 4; kt++) {
                    sight[u][kt] = HP == 2 && u ? sight[0][kt]
                                                : block_sight(v0 + 16 * kt, kl.shift,
                                                              QR * w + (HP == 2 ? 0 : 16 * u), W, S);
                    any = any || sight[u][kt];
                }
            if (any) {
                f32x4 s[QN][4];
#pragma unroll
                for (int kt = 0; kt < 4; kt++) {
                    bool need = false;
#pragma unroll
                    for (int u = 0; u < QN; u++) {
                        s[u][kt] = f32x4{0.f, 0.f, 0.f, 0.f};
                        need = need || sight[u][kt];
                    }
                    if (need)
#pragma unroll
                        for (int ks = 0; ks < DT / 2; ks++) {
                            const auto a = frag_row<T>(Ks[buf], LD, 16 * kt, 32 * ks);
#pragma unroll
                            for (int u = 0; u < QN; u++) s[u][kt] = M::mma(a, qf[u][ks], s[u][kt]);
                        }
                }
                typename M::Frag pf[QN][2];
#pragma unroll
                for (int u = 0; u < QN; u++) {
                    float top = -INFINITY;
#pragma unroll
                    for (int kt = 0; kt < 4; kt++) {
                        if (sight[u][kt] == 2) {
                            s[u][kt] *= d.c2;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const int ve = v0 + 16 * kt + 4 * g + e, jr = ve + kl.shift;
                                const bool see = jr <= ir[u] && (ve < S || jr > ir[u] - W);
                                s[u][kt][e] = see ? s[u][kt][e] * d.c2 : -INFINITY;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 4; e++) top = fmaxf(top, s[u][kt][e]);
                    }
                    top = pair_max(pair_max(top, 16), 32);
                    // The sums are held relative to m, which follows the maximum only where
                    // it has grown by more than 2^8: weights up to 2^8 lose nothing.
                    if (__any(top > m[u] + 8.f)) {
                        const float mn = fmaxf(m[u], top);
                        const float keep = mn == -INFINITY ? 0.f : exp2_fast(m[u] - mn);
                        m[u] = mn;
                        sum[u] *= keep;
#pragma unroll
                        for (int j = 0; j < DT; j++) O[u][j] *= keep;
                    }
                    const float base = m[u] == -INFINITY ? 0.f : m[u];
#pragma unroll
                    for (int kt = 0; kt < 4; kt++)
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            s[u][kt][e] = exp2_fast(s[u][kt][e] - base);
                            sum[u] += s[u][kt][e];
                        }
                    // the weights are rounded to the inputs' type for the product with V
                    pf[u][0] = frag_acc<T>(s[u][0], s[u][1]);
                    pf[u][1] = frag_acc<T>(s[u][2], s[u][3]);
                }
#pragma unroll
                for (int kp = 0; kp < 2; kp++) {
                    bool need = false;
#pragma unroll
                    for (int u = 0; u < QN; u++) need = need || sight[u][2 * kp] || sight[u][2 * kp + 1];
                    if (!need) continue;
#pragma unroll
                    for (int j = 0; j < DT; j++) {
                        const auto a = frag_col_pair<T>(Vs[buf], LD, 32 * kp, 16 * j);
#pragma unroll
                        for (int u = 0; u < QN; u++) O[u][j] = M::mma(a, pf[u][kp], O[u][j]);
                    }
                }
            }
            if (kBufs == 1) __syncthreads();
            if (n + 1 < nt) {
                rk.store(Ks[kBufs == 2 ? buf ^ 1 : 0]);
                rv.store(Vs[kBufs == 2 ? buf ^ 1 : 0]);
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int u = 0; u < QN; u++) {
        const int64_t t = t0 + ir[u];
        float all = xor_add(xor_add(sum[u], 16), 32);
        if (t >= d.T) continue;
        const bool live = t < len;
        const float inv = live ? 1.f / all : 0.f;
        T *op = o + at[u] * d.D;
#pragma unroll
        for (int j = 0; j < DT; j++) {
            const int c = 16 * j + 4 * g;
            const f32x4 r = live ? O[u][j] * inv : f32x4{0.f, 0.f, 0.f, 0.f};
            store4<T, VEC>(op, c, d.D, r);
        }
        if (g == 0) lse[at[u]] = live ? (m[u] + log2f(all)) * 0.6931471805599453f : 0.f;
    }
}

// ------------------------------------------------------------ single tokens
// One token of every sequence against its rolling cache, whose rows are read
// as they lie (a softmax does not ask for an order).  LK = D / 8 lanes share a
// row, 8 columns each; a wave takes 64 / LK rows at a time, for the R query
// heads of the workgroup, and keeps the running softmax of its rows.  Bound by
// the cache's bytes, or for short windows by latency: all loads of a step are
// issued before any is used, and there is one launch (with `splits`, which
// share the rows of a long cache among workgroups, and a joining one).
constexpr int kStepWaves = 8;

template <typename T, int LK, int R, bool VEC>
__global__ __launch_bounds__(64 * kStepWaves) void window_step_kernel(
    WinDims d, int groups, int splits, const T *__restrict__ q, const T *__restrict__ k,
    const T *__restrict__ v, T *ck, T *cv, const int64_t *__restrict__ pos,
    const int32_t *__restrict__ lengths, T *__restrict__ o, float *__restrict__ lse,
    float *__restrict__ part)
{
    constexpr int KW = 64 / LK;
    constexpr int V = 16 / sizeof(T);
    constexpr int kStepRows = R >= 4 ? 4 : 8;   // row loads of a lane in flight, for K and for V
    __shared__ __align__(32) float Os[kStepWaves][R][LK * 8];
    __shared__ float Ms[kStepWaves][R], Zs[kStepWaves][R];
    const int split = blockIdx.x % splits;
    const int64_t r0 = blockIdx.x / splits;
    const int grp = (int)(r0 % groups);
    const int64_t r1 = r0 / groups;
    const int hk = (int)(r1 % d.Hk);
    const int64_t b = r1 / d.Hk;
    const int per = d.Hq / d.Hk, h0 = hk * per + grp * R, hn = per - grp * R < R ? per - grp * R : R;
    const int tid = threadIdx.x, l = tid & 63, w = tid >> 6, kg = l / LK, c0 = (l % LK) * 8;
    if (seq_len(lengths, b, 1) == 0) {
        if (split == 0)
            for (int e = tid; e < hn * d.D; e += 64 * kStepWaves) {
                o[(b * d.Hq + h0 + e / d.D) * d.D + e % d.D] = (T)0.f;
                if (e % d.D == 0) lse[b * d.Hq + h0 + e / d.D] = 0.f;
            }
        return;
    }
    const int64_t p = seq_pos(pos, b), slot = cache_slot(p, d.S, d.W);
    const int64_t rows = p + 1 < d.cap ? p + 1 : d.cap;
    const T *kn = k + b * d.kb + hk * d.kh, *vn = v + b * d.vb + hk * d.vh;
    const int64_t step = (int64_t)d.Hk * d.D;
    T *kc = ck + (b * d.cap * d.Hk + hk) * d.D, *vc = cv + (b * d.cap * d.Hk + hk) * d.D;
    if (split == 0 && grp == 0 && tid < d.D) {   // nobody reads this row of the cache
        kc[slot * step + tid] = kn[tid];
        vc[slot * step + tid] = vn[tid];
    }
    const int64_t share = (rows + splits - 1) / splits;
    const int64_t first = split * share, end = first + share < rows ? first + share : rows;

    const auto read8 = [&](const T *row, bool in) {
        typename Mat<T>::Frag f;
        if constexpr (VEC) {
            const T *src = row + (c0 < d.D ? c0 : 0);   // a column that exists: meets zeros of q
#pragma unroll
            for (int u = 0; u < 8 / V; u++) {
                const Vec<T, V> x = vload<T, V>(src + u * V);
#pragma unroll
                for (int i = 0; i < V; i++) f[u * V + i] = x.e[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) f[i] = in && c0 + i < d.D ? row[c0 + i] : (T)0.f;
        }
        return f;
    };
    f32x8 qf[R], O[R];
    float m[R], z[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const bool in = r < hn && c0 < d.D;
        qf[r] = __builtin_convertvector(read8(q + b * d.qb + (h0 + (r < hn ? r : 0)) * d.qh, in), f32x8) *
                (in ? d.c2 : 0.f);
        O[r] = f32x8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        m[r] = -INFINITY;
        z[r] = 0.f;
    }
    for (int64_t j0 = first; j0 < end; j0 += kStepWaves * kStepRows * KW) {
        typename Mat<T>::Frag kf[kStepRows], vf[kStepRows];
#pragma unroll
        for (int u = 0; u < kStepRows; u++) {
            int64_t j = j0 + (u * kStepWaves + w) * KW + kg;
            if (j >= end) j = end - 1;                       // a row that exists, masked below
            const bool cur = j == slot;
            kf[u] = read8(cur ? kn : kc + j * step, true);
            vf[u] = read8(cur ? vn : vc + j * step, true);
        }
#pragma unroll
        for (int r = 0; r < R; r++) {
            float s[kStepRows], top = m[r];
#pragma unroll
            for (int u = 0; u < kStepRows; u++) {
                float a = 0.f;
#pragma unroll
                for (int i = 0; i < 8; i++) a = fmaf(qf[r][i], (float)kf[u][i], a);
#pragma unroll
                for (int x = 1; x < LK; x <<= 1) a = xor_add(a, x);
                s[u] = j0 + (u * kStepWaves + w) * KW + kg < end ? a : -INFINITY;
                top = fmaxf(top, s[u]);
            }
            const float base = top == -INFINITY ? 0.f : top;
            const float keep = exp2_fast(m[r] - base);
            m[r] = top;
            z[r] *= keep;
            O[r] *= keep;
#pragma unroll
            for (int u = 0; u < kStepRows; u++) {
                const float e = exp2_fast(s[u] - base);
                z[r] += e;
                O[r] += __builtin_convertvector(vf[u], f32x8) * e;
            }
        }
    }
    // join the row groups of the wave, then the waves
#pragma unroll
    for (int r = 0; r < R; r++) {
        float top = m[r];
#pragma unroll
        for (int x = LK; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
        const float f = top == -INFINITY ? 0.f : exp2_fast(m[r] - top);
        float zz = z[r] * f;
        O[r] *= f;
#pragma unroll
        for (int x = LK; x < 64; x <<= 1) {
            zz = xor_add(zz, x);
#pragma unroll
            for (int i = 0; i < 8; i++) O[r][i] = xor_add(O[r][i], x);
        }
        if (kg == 0) *reinterpret_cast<f32x8 *>(&Os[w][r][c0]) = O[r];
        if (l == 0) {
            Ms[w][r] = top;
            Zs[w][r] = zz;
        }
    }
    __syncthreads();
    for (int e = tid; e < hn * d.D; e += 64 * kStepWaves) {
        const int r = e / d.D, c = e % d.D;
        float top = -INFINITY, zz = 0.f, acc = 0.f;
#pragma unroll
        for (int x = 0; x < kStepWaves; x++) top = fmaxf(top, Ms[x][r]);
        if (top > -INFINITY)
#pragma unroll
            for (int x = 0; x < kStepWaves; x++) {
                const float f = exp2_fast(Ms[x][r] - top);
                zz = fmaf(Zs[x][r], f, zz);
                acc = fmaf(Os[x][r][c], f, acc);
            }
        const int64_t row = b * d.Hq + h0 + r;
        if (splits == 1) {
            o[row * d.D + c] = (T)(acc / zz);
            if (c == 0) lse[row] = (top + log2f(zz)) * 0.6931471805599453f;
        } else {
            float *pp = part + (row * splits + split) * (d.D + 2);
            pp[c] = acc;
            if (c == 0) {
                pp[d.D] = top;
                pp[d.D + 1] = zz;
            }
        }
    }
}

// o and lse of a query head from its splits.
template <typename T>
__global__ __launch_bounds__(kThreads) void window_join_kernel(WinDims d, int splits,
                                                               const int32_t *__restrict__ lengths,
                                                               const float *__restrict__ part,
                                                               T *__restrict__ o, float *__restrict__ lse)
{
    const int64_t row = blockIdx.x;
    if (seq_len(lengths, row / d.Hq, 1) == 0) return;   // written as zeros already
    const float *pp = part + row * splits * (d.D + 2);
    float top = -INFINITY, z = 0.f, acc = 0.f;
    for (int x = 0; x < splits; x++) top = fmaxf(top, pp[x * (d.D + 2) + d.D]);
    const int c = threadIdx.x;
    for (int x = 0; x < splits; x++) {
        const float *q = pp + x * (d.D + 2);
        const float f = exp2_fast(q[d.D] - top);
        z = fmaf(q[d.D + 1], f, z);
        if (c < d.D) acc = fmaf(q[c], f, acc);
    }
    if (c < d.D) o[row * d.D + c] = (T)(acc / z);
    if (c == 0) lse[row] = (top + log2f(z)) * 0.6931471805599453f;
}

// The call's last tokens into the rolling cache: the sinks, and the newest
// `window` tokens behind them.
template <typename T>
__global__ __launch_bounds__(kThreads) void window_cache_kernel(
    WinDims d, int64_t span, const T *__restrict__ k, const T *__restrict__ v, T *__restrict__ ck,
    T *__restrict__ cv, const int64_t *__restrict__ pos, const int32_t *__restrict__ lengths)
{
    // rows 0 .. S - 1 of `span` are the call's first S tokens, the others its last W
    const int64_t r = blockIdx.x % span, b = blockIdx.x / span;
    const int64_t len = seq_len(lengths, b, d.T);
    const int64_t p0 = seq_pos(pos, b);
    const int64_t nf = d.S < d.T ? d.S : d.T;
    const int64_t t = r < nf ? r : len - 1 - (r - nf);
    if (t < 0 || t >= len) return;
    const int64_t p = p0 + t;
    if (r < nf ? p >= d.S : p < d.S) return;
    const int64_t at = (b * d.cap + cache_slot(p, d.S, d.W)) * d.Hk * d.D;
    for (int e = threadIdx.x; e < d.Hk * d.D; e += kThreads) {
        const int h = e / d.D, c = e % d.D;
        ck[at + e] = k[b * d.kb + t * d.kt + h * d.kh + c];
        cv[at + e] = v[b * d.vb + t * d.vt + h * d.vh + c];
    }
}

// dQ^T += K^T dS^T over the keys, with P^T recomputed from lse and
// dS = P (dP - delta) scale, dP^T = V dO^T, delta = sum_c dO o (also left in
// the workspace for the other kernel).  Blocks and tiles as in the forward.
template <typename T, int DT, int QN, int HP, bool VEC>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 && DT <= 8 ? 2 : 1) void window_dq_kernel(
    WinDims d, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
    const T *__restrict__ o, const T *__restrict__ dout, const float *__restrict__ lse,
    const int32_t *__restrict__ lengths, float *__restrict__ delta, T *__restrict__ dq)
{
    using M = Mat<T>;
    constexpr int LD = DT * 16 + 8;
    constexpr int QR = HP == 2 ? 16 : 16 * QN;
    constexpr int kBufs = 4 * 64 * LD * (int)sizeof(T) <= 160 * 1024 ? 2 : 1;
    __shared__ __align__(32) T Ks[kBufs][kKeys * LD];
    __shared__ __align__(32) T Vs[kBufs][kKeys * LD];

    const int64_t blk = xcd_index(blockIdx.x, gridDim.x);
    const int qt = (int)(blk % d.nq);
    const int64_t bh = blk / d.nq;
    const int h0 = (int)(bh % (d.Hq / HP)) * HP;
    const int64_t b = bh / (d.Hq / HP);
    const int hk = h0 / (d.Hq / d.Hk);
    const int64_t len = seq_len(lengths, b, d.T);
    const int64_t t0 = (int64_t)qt * 4 * QR;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l = threadIdx.x & 63, g = l >> 4;
    const int W = (int)d.W, S = d.S;
    int ir[QN];
    int64_t at[QN];
    f32x4 O[QN][DT];
#pragma unroll
    for (int u = 0; u < QN; u++) {
        ir[u] = QR * w + (HP == 2 ? 0 : 16 * u) + (l & 15);
        at[u] = (b * d.T + t0 + ir[u]) * d.Hq + h0 + (HP == 2 ? u : 0);
#pragma unroll
        for (int j = 0; j < DT; j++) O[u][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (t0 < len) {
        typename M::Frag qf[QN][DT / 2], gf[QN][DT / 2];
        float L[QN], dl[QN];
#pragma unroll
        for (int u = 0; u < QN; u++) {
            const bool live = t0 + ir[u] < len;
            const T *row = live ? q + b * d.qb + (t0 + ir[u]) * d.qt + (h0 + (HP == 2 ? u : 0)) * d.qh
                                : nullptr;
            const T *grow = live ? dout + at[u] * d.D : nullptr;
            const T *orow = live ? o + at[u] * d.D : nullptr;
            float s = 0.f;
#pragma unroll
            for (int ks = 0; ks < DT / 2; ks++) {
                qf[u][ks] = frag_global<T>(row, 32 * ks + 8 * g, d.D, VEC);
                gf[u][ks] = frag_global<T>(grow, 32 * ks + 8 * g, d.D, VEC);
                const auto of = frag_global<T>(orow, 32 * ks + 8 * g, d.D, VEC);
#pragma unroll
                for (int i = 0; i < 8; i++) s = fmaf((float)gf[u][ks][i], (float)of[i], s);
            }
            dl[u] = xor_add(xor_add(s, 16), 32);
            if (live && g == 0) delta[at[u]] = dl[u];
            L[u] = live ? lse[at[u]] * 1.4426950408889634f : 0.f;
        }
        const int64_t last = (t0 + 4 * QR < len ? t0 + 4 * QR : len) - 1;
        const KeyList kl(t0, last, d.W, S);
        const int nt = (kl.total + kKeys - 1) / kKeys;
        const T *kn = k + b * d.kb + hk * d.kh, *vn = v + b * d.vb + hk * d.vh;
        RowRegs<T, DT * 16, LD, VEC> rk, rv;
        const auto fetch = [&](int n) {
            const auto key = [&](int r) {
                const int e = n * kKeys + r;
                return kl.key(e < kl.total ? e : kl.total - 1);
            };
            rk.load([&](int r) { return kn + key(r) * d.kt; }, d.D);
            rv.load([&](int r) { return vn + key(r) * d.vt; }, d.D);
        };
        fetch(0);
        rk.store(Ks[0]);
        rv.store(Vs[0]);
        __syncthreads();
        for (int n = 0; n < nt; n++) {
            const int buf = kBufs == 2 ? n & 1 : 0;
            if (n + 1 < nt) fetch(n + 1);
            const int v0 = n * kKeys;
#pragma unroll
            for (int kp = 0; kp < 2; kp++) {
                int sight[QN][2];
                bool any = false;
#pragma unroll
                for (int u = 0; u < QN; u++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        sight[u][e] = HP == 2 && u ? sight[0][e]
                                                   : block_sight(v0 + 32 * kp + 16 * e, kl.shift,
                                                                 QR * w + (HP == 2 ? 0 : 16 * u), W, S);
                        any = any || sight[u][e];
                    }
                if (!any) continue;
                f32x4 s[QN][2], dp[QN][2];
#pragma unroll
                for (int kt = 0; kt < 2; kt++) {
#pragma unroll
                    for (int u = 0; u < QN; u++) s[u][kt] = dp[u][kt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ks = 0; ks < DT / 2; ks++) {
                        const auto ka = frag_row<T>(Ks[buf], LD, 32 * kp + 16 * kt, 32 * ks);
                        const auto va = frag_row<T>(Vs[buf], LD, 32 * kp + 16 * kt, 32 * ks);
#pragma unroll
                        for (int u = 0; u < QN; u++) {
                            s[u][kt] = M::mma(ka, qf[u][ks], s[u][kt]);
                            dp[u][kt] = M::mma(va, gf[u][ks], dp[u][kt]);
                        }
                    }
                }
                typename M::Frag sf[QN];
#pragma unroll
                for (int u = 0; u < QN; u++) {
#pragma unroll
                    for (int kt = 0; kt < 2; kt++)
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const float p = exp2_fast(fmaf(s[u][kt][e], d.c2, -L[u]));
                            float ds = p * (dp[u][kt][e] - dl[u]) * d.scale;
                            if (sight[u][kt] != 2) {
                                const int ve = v0 + 32 * kp + 16 * kt + 4 * g + e, jr = ve + kl.shift;
                                ds = jr <= ir[u] && (ve < S || jr > ir[u] - W) ? ds : 0.f;
                            }
                            s[u][kt][e] = ds;
                        }
                    // dS is rounded to the inputs' type for the product with K
                    sf[u] = frag_acc<T>(s[u][0], s[u][1]);
                }
#pragma unroll
                for (int j = 0; j < DT; j++) {
                    const auto a = frag_col_pair<T>(Ks[buf], LD, 32 * kp, 16 * j);
#pragma unroll
                    for (int u = 0; u < QN; u++) O[u][j] = M::mma(a, sf[u], O[u][j]);
                }
            }
            if (kBufs == 1) __syncthreads();
            if (n + 1 < nt) {
                rk.store(Ks[kBufs == 2 ? buf ^ 1 : 0]);
                rv.store(Vs[kBufs == 2 ? buf ^ 1 : 0]);
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int u = 0; u < QN; u++) {
        const int64_t t = t0 + ir[u];
        if (t >= d.T) continue;
#pragma unroll
        for (int j = 0; j < DT; j++)
            store4<T, VEC>(dq + at[u] * d.D, 16 * j + 4 * g, d.D,
                           t < len ? O[u][j] : f32x4{0.f, 0.f, 0.f, 0.f});
    }
}

// dK and dV: a lane holds one key of KN blocks of 16 (columns) and four
// neighbouring queries (rows), a workgroup 64 KN keys, over the query heads of
// their key head.  SINKS = false: the queries that some window over the keys
// reaches; the sums of sinks go to part 0 of `parts`.  SINKS = true: the sinks
// for the queries behind those, 512 a workgroup, into parts 1 ..
template <typename T, int DT, int KN, bool VEC, bool SINKS>
__global__ __launch_bounds__(kThreads) void window_dkv_kernel(
    WinDims d, int ntiles, int nparts, const T *__restrict__ q, const T *__restrict__ k,
    const T *__restrict__ v, const T *__restrict__ dout, const float *__restrict__ lse,
    const float *__restrict__ delta, const int32_t *__restrict__ lengths, T *__restrict__ dk,
    T *__restrict__ dv, float *__restrict__ parts)
{
    using M = Mat<T>;
    constexpr int LD = DT * 16 + 8;
    constexpr int KR = 64 * KN;                   // keys of a workgroup
    constexpr int kBufs = 4 * 64 * LD * (int)sizeof(T) <= 156 * 1024 ? 2 : 1;
    __shared__ __align__(32) T Qs[kBufs][kRows * LD];
    __shared__ __align__(32) T Gs[kBufs][kRows * LD];
    __shared__ __align__(16) float Ls[kBufs][kRows], Dl[kBufs][kRows];

    int64_t rest = xcd_index(blockIdx.x, gridDim.x);
    int part = 0;
    if (SINKS) {
        part = 1 + (int)(rest % (nparts - 1));
        rest /= nparts - 1;
    }
    const int kt = (int)(rest % ntiles);
    rest /= ntiles;
    const int hk = (int)(rest % d.Hk);
    const int64_t b = rest / d.Hk;
    const int64_t len = seq_len(lengths, b, d.T);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l = threadIdx.x & 63, g = l >> 4;
    const int W = (int)d.W, S = d.S;
    const int64_t j0 = (int64_t)kt * KR;
    const int k0 = 16 * KN * w;                   // the wave's keys, relative to j0
    const int sinks = (int)(S > j0 ? S - j0 : 0);   // keys below this one are sinks
    const int per = d.Hq / d.Hk;
    f32x4 dK[KN][DT], dV[KN][DT];
#pragma unroll
    for (int u = 0; u < KN; u++)
#pragma unroll
        for (int n = 0; n < DT; n++) dK[u][n] = dV[u][n] = f32x4{0.f, 0.f, 0.f, 0.f};

    // the queries: [first, end)
    const int64_t reach = j0 + KR - 1 + d.W;
    int64_t first = j0, end = reach < len ? reach : len;
    if (SINKS) {
        first = (int64_t)(part - 1) * kSinkRows;
        end = first + kSinkRows < len ? first + kSinkRows : len;
        if (first < reach) first = reach;   // nearer queries are in part 0
    }
    if (j0 < len && first < end) {
        typename M::Frag kf[KN][DT / 2], vf[KN][DT / 2];
#pragma unroll
        for (int u = 0; u < KN; u++) {
            const int64_t j = j0 + k0 + 16 * u + (l & 15);
            const T *krow = j < len ? k + b * d.kb + j * d.kt + hk * d.kh : nullptr;
            const T *vrow = j < len ? v + b * d.vb + j * d.vt + hk * d.vh : nullptr;
#pragma unroll
            for (int ks = 0; ks < DT / 2; ks++) {
                kf[u][ks] = frag_global<T>(krow, 32 * ks + 8 * g, d.D, VEC);
                vf[u][ks] = frag_global<T>(vrow, 32 * ks + 8 * g, d.D, VEC);
            }
        }
        const int nq = (int)((end - first + kRows - 1) / kRows);
        RowRegs<T, DT * 16, LD, VEC> rq, rg;
        float rl, rd;
        const auto fetch = [&](int n) {
            const int h = hk * per + n / nq;
            const int64_t t0 = first + (int64_t)(n % nq) * kRows;
            const auto row = [&](int r) { return t0 + r < end ? t0 + r : end - 1; };
            rq.load([&](int r) { return q + b * d.qb + row(r) * d.qt + h * d.qh; }, d.D);
            rg.load([&](int r) { return dout + ((b * d.T + row(r)) * d.Hq + h) * d.D; }, d.D);
            if (threadIdx.x < kRows) {
                const int64_t at = (b * d.T + row(threadIdx.x)) * d.Hq + h;
                rl = lse[at] * 1.4426950408889634f;
                rd = delta[at];
            }
        };
        const auto put = [&](int buf) {
            rq.store(Qs[buf]);
            rg.store(Gs[buf]);
            if (threadIdx.x < kRows) {
                Ls[buf][threadIdx.x] = rl;
                Dl[buf][threadIdx.x] = rd;
            }
        };
        fetch(0);
        put(0);
        __syncthreads();
        for (int n = 0; n < per * nq; n++) {
            const int buf = kBufs == 2 ? n & 1 : 0;
            if (n + 1 < per * nq) fetch(n + 1);
            // first query of the tile relative to j0 (sinks: any number behind all keys will do)
            const int64_t t0 = first + (int64_t)(n % nq) * kRows;
            const int q0 = SINKS ? KR : (int)(t0 - j0);
            const int qend = q0 + (int)(end - t0);
#pragma unroll
            for (int half = 0; half < 2; half++) {
                const int r0 = 32 * half;
                int sight[KN];
                bool any = false;
#pragma unroll
                for (int u = 0; u < KN; u++) {  // as block_sight, for 16 keys and 32 queries
                    const int c0 = k0 + 16 * u, c1 = c0 + 15, s0 = q0 + r0, s1 = s0 + 31;
                    const bool none = c0 > s1 || s0 >= qend ||
                                      (SINKS ? c0 >= sinks : c0 >= sinks && s0 - c1 >= W);
                    const bool all = c1 <= s0 && s1 < qend && (c1 < sinks || (!SINKS && s1 - c0 < W));
                    sight[u] = none ? 0 : all ? 2 : 1;
                    any = any || sight[u];
                }
                if (!any) continue;
                f32x4 p[KN][2], ds[KN][2];
#pragma unroll
                for (int e2 = 0; e2 < 2; e2++) {
                    f32x4 s[KN], dp[KN];
#pragma unroll
                    for (int u = 0; u < KN; u++) s[u] = dp[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ks = 0; ks < DT / 2; ks++) {
                        const auto qa = frag_row<T>(Qs[buf], LD, r0 + 16 * e2, 32 * ks);
                        const auto ga = frag_row<T>(Gs[buf], LD, r0 + 16 * e2, 32 * ks);
#pragma unroll
                        for (int u = 0; u < KN; u++) {
                            s[u] = M::mma(qa, kf[u][ks], s[u]);
                            dp[u] = M::mma(ga, vf[u][ks], dp[u]);
                        }
                    }
                    const f32x4 L = *reinterpret_cast<const f32x4 *>(Ls[buf] + r0 + 16 * e2 + 4 * g);
                    const f32x4 D = *reinterpret_cast<const f32x4 *>(Dl[buf] + r0 + 16 * e2 + 4 * g);
#pragma unroll
                    for (int u = 0; u < KN; u++)
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            float pe = exp2_fast(fmaf(s[u][e], d.c2, -L[e]));
                            float de = pe * (dp[u][e] - D[e]) * d.scale;
                            if (sight[u] != 2) {
                                const int kr = k0 + 16 * u + (l & 15), qr = q0 + r0 + 16 * e2 + 4 * g + e;
                                const bool see = kr <= qr && qr < qend &&
                                                 (kr < sinks || (!SINKS && qr - kr < W));
                                pe = see ? pe : 0.f;
                                de = see ? de : 0.f;
                            }
                            p[u][e2][e] = pe;
                            ds[u][e2][e] = de;
                        }
                }
                // P and dS are rounded to the inputs' type for the products with dO and Q
                typename M::Frag pf[KN], sf[KN];
#pragma unroll
                for (int u = 0; u < KN; u++) {
                    pf[u] = frag_acc<T>(p[u][0], p[u][1]);
                    sf[u] = frag_acc<T>(ds[u][0], ds[u][1]);
                }
#pragma unroll
                for (int c = 0; c < DT; c++) {
                    const auto ga = frag_col_pair<T>(Gs[buf], LD, r0, 16 * c);
                    const auto qa = frag_col_pair<T>(Qs[buf], LD, r0, 16 * c);
#pragma unroll
                    for (int u = 0; u < KN; u++) {
                        dV[u][c] = M::mma(ga, pf[u], dV[u][c]);
                        dK[u][c] = M::mma(qa, sf[u], dK[u][c]);
                    }
                }
            }
            if (kBufs == 1) __syncthreads();
            if (n + 1 < per * nq) put(kBufs == 2 ? buf ^ 1 : 0);
            __syncthreads();
        }
    }
#pragma unroll
    for (int u = 0; u < KN; u++) {
        const int kr = k0 + 16 * u + (l & 15);
        const int64_t j = j0 + kr;
        const bool sink = parts && kr < sinks;
        if (j >= d.T || (SINKS && !sink)) continue;
        const int64_t at = ((b * d.T + j) * d.Hk + hk) * d.D;
        float *pp = sink ? parts + ((((int64_t)part * d.B + b) * d.Hk + hk) * d.S + j) * 2 * d.D : nullptr;
#pragma unroll
        for (int c = 0; c < DT; c++) {
            if (sink) {
                store4<float, false>(pp, 16 * c + 4 * g, d.D, dK[u][c]);
                store4<float, false>(pp + d.D, 16 * c + 4 * g, d.D, dV[u][c]);
            } else {
                store4<T, VEC>(dk + at, 16 * c + 4 * g, d.D, dK[u][c]);
                store4<T, VEC>(dv + at, 16 * c + 4 * g, d.D, dV[u][c]);
            }
        }
    }
}

// dK and dV of the sinks: the sum of their parts, in order.
template <typename T>
__global__ __launch_bounds__(kThreads) void window_sinks_kernel(WinDims d, int nparts,
                                                                const float *__restrict__ parts,
                                                                T *__restrict__ dk, T *__restrict__ dv)
{
    const int64_t r = blockIdx.x;   // (b, hk, j)
    const int64_t j = r % d.S, bh = r / d.S, hk = bh % d.Hk, b = bh / d.Hk;
    if (j >= d.T) return;
    const int64_t step = (int64_t)d.B * d.Hk * d.S * 2 * d.D;
    for (int c = threadIdx.x; c < 2 * d.D; c += kThreads) {
        float s = 0.f;
        for (int n = 0; n < nparts; n++) s += parts[n * step + r * 2 * d.D + c];
        T *out = c < d.D ? dk : dv;
        out[((b * d.T + j) * d.Hk + hk) * d.D + (c < d.D ? c : c - d.D)] = (T)s;
    }
}

// -------------------------------------------------------------------- host

WinDims dims_of(const sdm_window_desc &s)
{
    WinDims d = {};
    d.B = s.B;
    d.Hq = s.Hq;
    d.Hk = s.Hk;
    d.D = s.D;
    d.T = s.T;
    d.W = s.window;
    d.S = s.sinks;
    d.scale = s.scale;
    d.c2 = (float)((double)s.scale * 1.4426950408889634);
    d.qb = s.q_batch;
    d.qt = s.q_token;
    d.qh = s.q_head;
    d.kb = s.k_batch;
    d.kt = s.k_token;
    d.kh = s.k_head;
    d.vb = s.v_batch;
    d.vt = s.v_token;
    d.vh = s.v_head;
    d.cap = s.sinks + s.window;
    d.nq = (int)((s.T + kRows - 1) / kRows);
    return d;
}

// Keys of a wave of the dK, dV kernel in blocks of 16: two, so that each
// fragment of Q and dO serves 32 keys, unless D = 256 fills the registers.
constexpr int key_blocks(int D) { return D <= 128 ? 2 : 1; }

struct BackPlan {
    size_t delta, parts, total;
    int nparts, ktiles;
};

BackPlan back_plan(const sdm_window_desc &s)
{
    BackPlan p = {};
    size_t at = ((size_t)s.B * s.T * s.Hq * 4 + 255) & ~(size_t)255;
    // sinks that queries see from behind their window
    if (s.sinks > 0 && s.T > s.window) {
        const int64_t keys = 64 * key_blocks(s.D), rows = s.sinks < s.T ? s.sinks : s.T;
        p.nparts = 1 + (int)((s.T + kSinkRows - 1) / kSinkRows);
        p.ktiles = (int)((rows + keys - 1) / keys);
        p.parts = at;
        at += (size_t)p.nparts * s.B * s.Hk * s.sinks * 2 * s.D * 4;
    }
    p.total = at;
    return p;
}

template <typename T, int DT, bool VEC>
hipError_t forward(const WindowArgs &a, hipStream_t stream)
{
    WinDims d = dims_of(a.d);
    constexpr int QN = DT == 16 ? 1 : 2;  // D = 256 fills the registers with one
    const auto run = [&](auto kernel, int hp, int queries) {
        d.nq = (int)((d.T + queries - 1) / queries);
        kernel<<<(unsigned)((int64_t)d.B * (d.Hq / hp) * d.nq), kThreads, 0, stream>>>(
            d, (const T *)a.q, (const T *)a.k, (const T *)a.v, (const T *)a.cache_k,
            (const T *)a.cache_v, a.pos, a.lengths, (T *)a.o, a.lse);
    };
    // heads in pairs where an even number of them shares a key head
    const bool pairs = QN == 2 && (d.Hq / d.Hk) % 2 == 0;
    if (a.pos)
        pairs ? run(window_fwd_kernel<T, DT, QN, QN, VEC, true>, 2, 64)
              : run(window_fwd_kernel<T, DT, QN, 1, VEC, true>, 1, 64 * QN);
    else
        pairs ? run(window_fwd_kernel<T, DT, QN, QN, VEC, false>, 2, 64)
              : run(window_fwd_kernel<T, DT, QN, 1, VEC, false>, 1, 64 * QN);
    if (a.cache_k) {
        const int64_t span = (d.S < d.T ? d.S : d.T) + (d.W < d.T ? d.W : d.T);
        window_cache_kernel<T><<<(unsigned)(span * d.B), kThreads, 0, stream>>>(
            d, span, (const T *)a.k, (const T *)a.v, (T *)a.cache_k, (T *)a.cache_v, a.pos, a.lengths);
    }
    return hipGetLastError();
}

template <typename T, int DT, bool VEC>
hipError_t backward(const WindowArgs &a, hipStream_t stream)
{
    WinDims d = dims_of(a.d);
    const BackPlan p = back_plan(a.d);
    constexpr int QN = DT == 16 ? 1 : 2, KN = key_blocks(DT * 16);
    const T *q = (const T *)a.q, *k = (const T *)a.k, *v = (const T *)a.v, *dout = (const T *)a.dout;
    float *delta = (float *)a.ws, *parts = p.nparts ? (float *)(a.ws + p.parts) : nullptr;
    const auto run = [&](auto kernel, int hp, int queries) {
        d.nq = (int)((d.T + queries - 1) / queries);
        kernel<<<(unsigned)((int64_t)d.B * (d.Hq / hp) * d.nq), kThreads, 0, stream>>>(
            d, q, k, v, (const T *)a.oin, dout, a.lse_in, a.lengths, delta, (T *)a.dq);
    };
    if (QN == 2 && (d.Hq / d.Hk) % 2 == 0)
        run(window_dq_kernel<T, DT, QN, QN, VEC>, 2, 64);
    else
        run(window_dq_kernel<T, DT, QN, 1, VEC>, 1, 64 * QN);
    const int ntiles = (int)((d.T + 64 * KN - 1) / (64 * KN));
    window_dkv_kernel<T, DT, KN, VEC, false><<<(unsigned)((int64_t)d.B * d.Hk * ntiles), kThreads, 0, stream>>>(
        d, ntiles, p.nparts, q, k, v, dout, a.lse_in, delta, a.lengths, (T *)a.dk, (T *)a.dv, parts);
    if (p.nparts) {
        window_dkv_kernel<T, DT, KN, VEC, true>
            <<<(unsigned)((int64_t)d.B * d.Hk * p.ktiles * (p.nparts - 1)), kThreads, 0, stream>>>(
                d, p.ktiles, p.nparts, q, k, v, dout, a.lse_in, delta, a.lengths, (T *)a.dk, (T *)a.dv,
                parts);
        window_sinks_kernel<T><<<(unsigned)((int64_t)d.B * d.Hk * d.S), kThreads, 0, stream>>>(
            d, p.nparts, parts, (T *)a.dk, (T *)a.dv);
    }
    return hipGetLastError();
}

// Query heads of a workgroup of the single-token kernel, and the workgroups
// that share a cache: enough for every compute unit where there are few
// streams, each with at least 256 rows.
struct StepPlan {
    int R, groups, splits;
};

StepPlan step_plan(const sdm_window_desc &s)
{
    StepPlan p;
    const int per = s.Hq / s.Hk;
    p.R = per == 1 ? 1 : per == 2 ? 2 : per <= 4 ? 4 : 8;
    p.groups = (per + p.R - 1) / p.R;
    const int64_t units = (int64_t)s.B * s.Hk * p.groups, rows = s.sinks + s.window;
    int64_t n = (256 + units - 1) / units;
    if (n > rows / 256) n = rows / 256;
    p.splits = n < 1 ? 1 : n > 64 ? 64 : (int)n;
    return p;
}

bool is_step(const sdm_window_desc &d, bool cont) { return cont && d.T == 1; }

template <typename T, int LK, bool VEC>
hipError_t step(const WindowArgs &a, hipStream_t stream)
{
    const WinDims d = dims_of(a.d);
    const StepPlan p = step_plan(a.d);
    const auto run = [&](auto kernel) {
        kernel<<<(unsigned)((int64_t)d.B * d.Hk * p.groups * p.splits), 64 * kStepWaves, 0, stream>>>(
            d, p.groups, p.splits, (const T *)a.q, (const T *)a.k, (const T *)a.v, (T *)a.cache_k,
            (T *)a.cache_v, a.pos, a.lengths, (T *)a.o, a.lse, (float *)a.ws);
    };
    switch (p.R) {
    case 1: run(window_step_kernel<T, LK, 1, VEC>); break;
    case 2: run(window_step_kernel<T, LK, 2, VEC>); break;
    case 4: run(window_step_kernel<T, LK, 4, VEC>); break;
    default: run(window_step_kernel<T, LK, 8, VEC>); break;
    }
    if (p.splits > 1)
        window_join_kernel<T><<<(unsigned)((int64_t)d.B * d.Hq), kThreads, 0, stream>>>(
            d, p.splits, a.lengths, (const float *)a.ws, (T *)a.o, a.lse);
    return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t dispatch_d(const WindowArgs &a, bool back, hipStream_t stream)
{
    if (!back && is_step(a.d, a.pos)) {  // lanes of a row
        if (a.d.D <= 32) return step<T, 4, VEC>(a, stream);
        if (a.d.D <= 64) return step<T, 8, VEC>(a, stream);
        if (a.d.D <= 128) return step<T, 16, VEC>(a, stream);
        return step<T, 32, VEC>(a, stream);
    }
    // head columns padded to 32, 64, 128 or 256
    if (a.d.D <= 32) return back ? backward<T, 2, VEC>(a, stream) : forward<T, 2, VEC>(a, stream);
    if (a.d.D <= 64) return back ? backward<T, 4, VEC>(a, stream) : forward<T, 4, VEC>(a, stream);
    if (a.d.D <= 128) return back ? backward<T, 8, VEC>(a, stream) : forward<T, 8, VEC>(a, stream);
    return back ? backward<T, 16, VEC>(a, stream) : forward<T, 16, VEC>(a, stream);
}

template <typename T>
hipError_t dispatch(const WindowArgs &a, bool back, hipStream_t stream)
{
    const sdm_window_desc &d = a.d;
    const bool vec = d.D % 8 == 0 &&
                     rows_on_16(a.q, d.q_batch, d.q_token, d.q_head, d.D, sizeof(T)) &&
                     rows_on_16(a.k, d.k_batch, d.k_token, d.k_head, d.D, sizeof(T)) &&
                     rows_on_16(a.v, d.v_batch, d.v_token, d.v_head, d.D, sizeof(T));
    return vec ? dispatch_d<T, true>(a, back, stream) : dispatch_d<T, false>(a, back, stream);
}

}  // namespace

size_t window_forward_ws(const sdm_window_desc &d, bool cont)
{
    if (!is_step(d, cont)) return 0;
    const StepPlan p = step_plan(d);
    return p.splits == 1 ? 0 : (size_t)d.B * d.Hq * p.splits * (d.D + 2) * 4;
}
size_t window_backward_ws(const sdm_window_desc &d) { return back_plan(d).total; }

hipError_t launch_window_forward(const WindowArgs &a, hipStream_t stream)
{
    return a.d.dtype == SDM_F32 ? dispatch<float>(a, false, stream) : dispatch<bf16>(a, false, stream);
}

hipError_t launch_window_backward(const WindowArgs &a, hipStream_t stream)
{
    return a.d.dtype == SDM_F32 ? dispatch<float>(a, true, stream) : dispatch<bf16>(a, true, stream);
}

}  // namespace sdm
