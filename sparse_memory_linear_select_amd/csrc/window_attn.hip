// Causal attention with a sliding window and sinks: query i sees key j where
// j <= i and (i - j < window or j < sinks).  Hq / Hk query heads share a key
// head.
//
// Scores are computed transposed, S^T = K Q^T, so that a lane holds one query
// (column) and four neighbouring keys: the softmax of a query is a reduction
// over registers and two lane exchanges, and P^T is already the right operand
// of O^T += V^T P^T.  One pass over the keys with the running maximum m and
// sum l of 2^{s - m}, s in units of log2.
#include <type_traits>

#include "mix_internal.h"

#include "lane_ops.h"
#include "mix_device.h"

namespace sdm {
namespace {

constexpr int kTile = 64;     // keys (or queries) of a tile in LDS
constexpr int kThreads = 256; // of the kernels whose waves hold queries
constexpr int kFewKeys = 64;  // fewer visible keys: delta from the keys
constexpr int kKeys = 64;     // keys of a workgroup of the dK, dV kernel: 16 for each of four waves
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

// 8 elements from k of a row, zeros from D on (VEC: all or none).
template <typename T, bool VEC>
__device__ __forceinline__ typename Mat<T>::Frag frag_global(const T *row, int k, int D)
{
    typename Mat<T>::Frag f;
    if constexpr (VEC) {
        constexpr int V = 16 / sizeof(T);
        const T *src = row + (k < D ? k : 0);
#pragma unroll
        for (int u = 0; u < 8 / V; u++) {
            const Vec<T, V> v = vload<T, V>(src + u * V);
#pragma unroll
            for (int i = 0; i < V; i++) f[u * V + i] = k < D ? v.e[i] : (T)0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const T v = row[k + i < D ? k + i : 0];
            f[i] = k + i < D ? v : (T)0.f;
        }
    }
    return f;
}

// The keys that the queries i0 .. i1 (positions) can see, as one list: the
// sinks in front of every window (unless they are taken apart), then the keys
// from lo on.  Entries v < always are sinks that every later query sees; jr(v)
// = the position of entry v - i0 (for entries in front of lo some number below
// that of lo: they precede every query).
struct KeyList {
    int64_t lo;        // first key of the window part
    int front;         // sinks in front of it
    int ns, total;     // sinks in the list; entries
    int always;
    int shift;         // jr(v) = v + shift
    __device__ KeyList(int64_t i0, int64_t i1, int64_t W, int S, bool apart)
    {
        lo = i0 - W + 1 > 0 ? i0 - W + 1 : 0;
        front = S < lo ? S : (int)lo;
        ns = apart ? 0 : front;
        total = ns + (int)(i1 - lo + 1);
        always = S - (front - ns);
        shift = (int)(lo - i0) - ns;
    }
    __device__ int64_t key(int v) const { return v < ns ? v : lo + (v - ns); }
};

// (Masks of single numbers below are written with & and |: && and || become
// branches, and a wave that branches waits for every read in turn.)
// What 16 neighbouring entries from v0 are to 16 neighbouring queries from ir0
// (relative to i0): 0 none is seen, 1 some are, 2 all are.
__device__ __forceinline__ int block_sight(int v0, int shift, int ir0, int W, int always)
{
    const int j0 = v0 + shift, j1 = j0 + 15, ir1 = ir0 + 15;
    if (j0 > ir1 || (v0 >= always && j1 <= ir0 - W)) return 0;
    return j1 <= ir0 && (j0 > ir1 - W || v0 + 15 < always) ? 2 : 1;
}

// A 64-row tile in two steps, as TileRegs, from rows given by pointers.  Every
// access is to a row that exists: columns from D on hold the row's first ones
// (finite numbers that meet zeros in the other operand, or columns nobody
// stores).
template <typename T, int COLS, int LD, bool VEC, int THREADS>
struct RowRegs {
    static constexpr int V = 16 / sizeof(T);
    static constexpr int PER = COLS / V;
    static constexpr int N = (kTile * PER + THREADS - 1) / THREADS;
    static constexpr bool kWhole = kTile * PER % THREADS == 0;
    Vec<T, V> v[N];

    template <typename F>
    __device__ __forceinline__ void load(F row_of, int D)
    {
#pragma unroll
        for (int u = 0; u < N; u++) {
            const int e = threadIdx.x + u * THREADS;
            const int c = (e % PER) * V, r = e / PER;
            const T *src = row_of(kWhole || r < kTile ? r : kTile - 1);
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
            const int e = threadIdx.x + u * THREADS;
            if (kWhole || e < kTile * PER) vstore<T, V>(tile + (e / PER) * LD + (e % PER) * V, v[u]);
        }
    }
};

// Few sinks in front of the windows are taken apart from the list, as a block of
// 16 keys of their own: at the head of the list they would cost a whole tile
// (with 64 queries and a window of 128, 195 entries are four tiles and 191 three).
constexpr int kFewSinks = 16;

// Fills a 16-row tile from rows given by pointers (which exist).
template <typename T, int COLS, int LD, bool VEC, int THREADS, typename F>
__device__ __forceinline__ void load_few(T *tile, F row_of, int D)
{
    constexpr int V = 16 / sizeof(T);
    constexpr int PER = COLS / V;
    for (int e = threadIdx.x; e < kFewSinks * PER; e += THREADS) {
        const int c = (e % PER) * V, r = e / PER;
        const T *src = row_of(r);
        Vec<T, V> v;
        if constexpr (VEC) {
            v = vload<T, V>(src + (c < D ? c : 0));
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) v.e[i] = src[c + i < D ? c + i : 0];
        }
        vstore<T, V>(tile + r * LD + c, v);
    }
}

// Column fragment of a 16-row tile for weights frag_acc(tile, zeros).
template <typename T>
__device__ __forceinline__ typename Mat<T>::Frag frag_col_few(const T *tile, int ld, int col0)
{
    const auto zero = __builtin_convertvector(f32x4{0.f, 0.f, 0.f, 0.f}, typename Mat<T>::Half);
    return __builtin_shufflevector(col4(tile, ld, ((threadIdx.x & 63) >> 4) * 4, col0), zero, 0, 1, 2, 3, 4,
                                   5, 6, 7);
}

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
// heads, or 64 QN queries of one, and two workgroups share a compute unit.  (One
// block a wave, eight waves a workgroup, reads LDS twice as often and runs no
// more waves: 200 us instead of 165 for 8 x 4096 tokens, 16 and 8 heads of 128,
// window 128.)  The next tile of keys is loaded while one is worked on; bfloat16
// tiles go to a second buffer, float32 ones (35 KB) leave the LDS to a second
// workgroup instead (3 x 1333 tokens, 6 and 2 heads of 72, window 301: 66 us
// instead of 83).  Bound by the latency between HBM and the tiles: 133 us for the
// bfloat16 shape above, 3.0 TB/s (window 1: 98); long windows by the matrix
// products (window 1000: 397 us).
template <typename T, int DT, int QN, int HP, bool VEC, bool CACHE>
__global__ __launch_bounds__(kThreads, DT <= 8 ? 2 : 1) void window_fwd_kernel(
    WinDims d, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
    const T *__restrict__ ck, const T *__restrict__ cv, const int64_t *__restrict__ pos,
    const int32_t *__restrict__ lengths, T *__restrict__ o, float *__restrict__ lse)
{
    using M = Mat<T>;
    using Half = typename M::Half;
    constexpr int LD = DT * 16 + 8;
    constexpr int QR = HP == 2 ? 16 : 16 * QN;   // queries of a wave
    constexpr int kBufs = sizeof(T) == 2 ? 2 : 1;
    __shared__ __align__(32) T Ks[kBufs][kTile * LD];
    __shared__ __align__(32) T Vs[kBufs][kTile * LD];
    // float32 tiles leave no room for the sinks' beside a second workgroup
    constexpr bool kApart = sizeof(T) == 2;
    __shared__ __align__(32) T Few[2][kApart ? kFewSinks * LD : 1];

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
        const int64_t last = (t0 + 4 * QR < len ? t0 + 4 * QR : len) - 1;
        const KeyList kl(p0 + t0, p0 + last, d.W, S, kApart && S <= kFewSinks);
        const int few = kl.front - kl.ns;
        const int nt = (kl.total + kTile - 1) / kTile;
        const T *kn = k + b * d.kb + hk * d.kh, *vn = v + b * d.vb + hk * d.vh;
        const auto krow = [&](int64_t j) {
            if (CACHE && j < p0) return ck + ((b * d.cap + cache_slot(j, S, W)) * d.Hk + hk) * d.D;
            return kn + (j - p0) * d.kt;
        };
        const auto vrow = [&](int64_t j) {
            if (CACHE && j < p0) return cv + ((b * d.cap + cache_slot(j, S, W)) * d.Hk + hk) * d.D;
            return vn + (j - p0) * d.vt;
        };
        RowRegs<T, DT * 16, LD, VEC, kThreads> rk, rv;
        const auto fetch = [&](int n) {
            const auto key = [&](int r) {
                const int e = n * kTile + r;
                return kl.key(e < kl.total ? e : kl.total - 1);
            };
            rk.load([&](int r) { return krow(key(r)); }, d.D);
            rv.load([&](int r) { return vrow(key(r)); }, d.D);
        };
        fetch(0);
        typename M::Frag qf[QN][DT / 2];
#pragma unroll
        for (int u = 0; u < QN; u++) {
            const int64_t tr = t0 + ir[u] <= last ? t0 + ir[u] : last;   // a row that exists
            const T *row = q + b * d.qb + tr * d.qt + (h0 + (HP == 2 ? u : 0)) * d.qh;
#pragma unroll
            for (int ks = 0; ks < DT / 2; ks++) qf[u][ks] = frag_global<T, VEC>(row, 32 * ks + 8 * g, d.D);
        }
        if (kApart && few > 0) {
            load_few<T, DT * 16, LD, VEC, kThreads>(Few[0], [&](int r) { return krow(r < few ? r : few - 1); }, d.D);
            load_few<T, DT * 16, LD, VEC, kThreads>(Few[1], [&](int r) { return vrow(r < few ? r : few - 1); }, d.D);
        }
        rk.store(Ks[0]);
        rv.store(Vs[0]);
        __syncthreads();
        if (kApart && few > 0) {
            const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
            typename M::Frag pf[QN];
#pragma unroll
            for (int u = 0; u < QN; u++) {
                f32x4 s = zero;
#pragma unroll
                for (int ks = 0; ks < DT / 2; ks++)
                    s = M::mma(frag_row<T>(Few[0], LD, 0, 32 * ks), qf[u][ks], s);
                float top = -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    s[e] = 4 * g + e < few ? s[e] * d.c2 : -INFINITY;
                    top = fmaxf(top, s[e]);
                }
                m[u] = pair_max(pair_max(top, 16), 32);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    s[e] = exp2_fast(s[e] - m[u]);
                    sum[u] += s[e];
                }
                pf[u] = frag_acc<T>(s, zero);
            }
#pragma unroll
            for (int j = 0; j < DT; j++) {
                const auto a = frag_col_few<T>(Few[1], LD, 16 * j);
#pragma unroll
                for (int u = 0; u < QN; u++) O[u][j] = M::mma(a, pf[u], O[u][j]);
            }
        }
        for (int n = 0; n < nt; n++) {
            const int buf = kBufs == 2 ? n & 1 : 0;
            fetch(n + 1 < nt ? n + 1 : n);
            const int v0 = n * kTile;
            int sight[QN][4];
            bool any = false;
#pragma unroll
            for (int u = 0; u < QN; u++)
#pragma unroll
                for (int kt = 0; kt < 4; kt++) {
                    sight[u][kt] = HP == 2 && u ? sight[0][kt]
                                                : block_sight(v0 + 16 * kt, kl.shift,
                                                              QR * w + (HP == 2 ? 0 : 16 * u), W, kl.always);
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
                                const bool see = (jr <= ir[u]) & ((ve < kl.always) | (jr > ir[u] - W));
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
            rk.store(Ks[kBufs == 2 ? buf ^ 1 : 0]);
            rv.store(Vs[kBufs == 2 ? buf ^ 1 : 0]);
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
        for (int j = 0; j < DT; j++) O[u][j] = live ? O[u][j] * inv : f32x4{0.f, 0.f, 0.f, 0.f};
        store_row<T, DT, VEC>(op, d.D, O[u]);
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
// share the rows of a long cache among workgroups, and a joining one).  32
// streams, 16 and 8 heads of 128, window 128, bfloat16: 8 us.
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

// Gradients of the sinks.  Few queries see a key, but all later ones a sink, so
// their sums are split: part 0 holds the queries that the dK, dV kernel visits
// for the keys' windows, the others each a part of the queries behind.  With at
// most 16 sinks (and 128 columns) the dQ kernel, which has their weights at hand, sums the parts
// (one a workgroup; `near` = its queries): those of the sinks that stand in
// front of all its windows.  With more, the dK, dV kernel runs once more, for
// the sinks alone.
struct SinkParts {
    float *sums;     // [part][B][Hk][S][2 D]: dK, dV; null: no query sees a sink from behind its window
    int near;        // queries of a dQ workgroup that sums its part, or 0
    int nparts;
};

__device__ __forceinline__ float *sink_part(const SinkParts &p, const WinDims &d, int64_t part, int64_t b,
                                            int hk)
{
    return p.sums + ((part * d.B + b) * d.Hk + hk) * d.S * 2 * d.D;
}

// dQ^T += K^T dS^T over the keys, with P^T recomputed from lse and
// dS = P (dP - delta) scale, dP^T = V dO^T, delta = sum_c dO o = sum_j P_j dP_j
// (also left in the workspace for the other kernel).  Rows and tiles as in the
// forward.  A bfloat16 o was rounded, which delta feels where few keys share a
// row's weight: with n equal weights dS is off by 1 / sqrt(n - 1) of a rounding.
// Queries that may see fewer than kFewKeys keys get delta from a walk of its own
// over their keys, at most three tiles: delta + sum_j P_j (dP_j - delta)
// (backward of 8 x 4096 tokens, 16 and 8 heads of 128, window 32, 4 sinks: 438 us
// instead of 414).  Bound, like the forward, by the latency between HBM and the
// tiles: 269 us with window 128, 670 MB.
template <typename T, int DT, int QN, int HP, bool VEC, bool FEW>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 && DT <= 8 ? 2 : 1) void window_dq_kernel(
    WinDims d, SinkParts sp, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
    const T *__restrict__ o, const T *__restrict__ dout, const float *__restrict__ lse,
    const int32_t *__restrict__ lengths, float *__restrict__ delta, T *__restrict__ dq)
{
    using M = Mat<T>;
    using Frag = typename M::Frag;
    constexpr int LD = DT * 16 + 8;
    constexpr int QR = HP == 2 ? 16 : 16 * QN;    // queries of a wave
    constexpr int kRows = 64 * QN;                // rows of the workgroup
    constexpr int LS = kRows + 8;
    constexpr int kBufs = sizeof(T) == 2 ? 2 : 1;
    __shared__ __align__(32) T Ks[kBufs * kTile * LD];  // at the end (FEW) the rows of Q and dO
    __shared__ __align__(32) T Vs[kBufs * kTile * LD];
    // the sinks' K and V, then their P and dS: [key][row]
    __shared__ __align__(32) T Few[2][FEW ? kFewSinks * (LS > LD ? LS : LD) : 1];
    static_assert(!FEW || kBufs * kTile >= kRows, "room for the rows");

    const int64_t blk = xcd_index(blockIdx.x, gridDim.x);
    const int qt = (int)(blk % d.nq);
    const int64_t bh = blk / d.nq;
    const int h0 = (int)(bh % (d.Hq / HP)) * HP;
    const int64_t b = bh / (d.Hq / HP);
    const int hk = h0 / (d.Hq / d.Hk);
    const int64_t len = seq_len(lengths, b, d.T);
    const int64_t t0 = (int64_t)qt * 4 * QR;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l = threadIdx.x & 63, g = l >> 4, li = l & 15;
    const int W = (int)d.W, S = d.S;
    int ir[QN];
    bool alone[QN];   // a query that sees one key: its weight is 1, whatever the score
    f32x4 O[QN][DT];
#pragma unroll
    for (int u = 0; u < QN; u++) {
        ir[u] = QR * w + (HP == 2 ? 0 : 16 * u) + li;
        alone[u] = t0 + ir[u] == 0;
#pragma unroll
        for (int j = 0; j < DT; j++) O[u][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (t0 < len) {
        const int64_t last = (t0 + 4 * QR < len ? t0 + 4 * QR : len) - 1;
        const KeyList kl(t0, last, d.W, S, FEW);
        const int nt = (kl.total + kTile - 1) / kTile;
        const T *kn = k + b * d.kb + hk * d.kh, *vn = v + b * d.vb + hk * d.vh;
        RowRegs<T, DT * 16, LD, VEC, kThreads> rk, rv;
        const auto fetch = [&](int n) {
            const auto key = [&](int r) {
                const int e = n * kTile + r;
                return kl.key(e < kl.total ? e : kl.total - 1);
            };
            rk.load([&](int r) { return kn + key(r) * d.kt; }, d.D);
            rv.load([&](int r) { return vn + key(r) * d.vt; }, d.D);
        };
        fetch(0);
        Frag qf[QN][DT / 2], gf[QN][DT / 2];
        float L[QN], dl[QN];
#pragma unroll
        for (int u = 0; u < QN; u++) {
            const bool live = t0 + ir[u] <= last;
            const int64_t tr = live ? t0 + ir[u] : last;   // a row that exists
            const int h = h0 + (HP == 2 ? u : 0);
            const int64_t ar = (b * d.T + tr) * d.Hq + h;
            float s = 0.f;
#pragma unroll
            for (int ks = 0; ks < DT / 2; ks++) {
                qf[u][ks] = frag_global<T, VEC>(q + b * d.qb + tr * d.qt + h * d.qh, 32 * ks + 8 * g, d.D);
                gf[u][ks] = frag_global<T, VEC>(dout + ar * d.D, 32 * ks + 8 * g, d.D);
                const Frag of = frag_global<T, VEC>(o + ar * d.D, 32 * ks + 8 * g, d.D);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    gf[u][ks][i] = live ? gf[u][ks][i] : (T)0.f;
                    s = fmaf((float)gf[u][ks][i], (float)of[i], s);
                }
            }
            dl[u] = xor_add(xor_add(s, 16), 32);
            L[u] = lse[ar] * 1.4426950408889634f;
        }
        const bool few = FEW && kl.front > 0;
        if (few) {
            const auto row = [&](int r) { return r < kl.front ? r : kl.front - 1; };
            load_few<T, DT * 16, LD, VEC, kThreads>(Few[0], [&](int r) { return kn + row(r) * d.kt; }, d.D);
            load_few<T, DT * 16, LD, VEC, kThreads>(Few[1], [&](int r) { return vn + row(r) * d.vt; }, d.D);
        }
        rk.store(Ks);
        rv.store(Vs);
        __syncthreads();
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        // P and dS (without the scale) of the sinks in front
        const auto front = [&](f32x4 *s, f32x4 *dp) {
#pragma unroll
            for (int u = 0; u < QN; u++) {
                s[u] = dp[u] = zero;
#pragma unroll
                for (int ks = 0; ks < DT / 2; ks++) {
                    s[u] = M::mma(frag_row<T>(Few[0], LD, 0, 32 * ks), qf[u][ks], s[u]);
                    dp[u] = M::mma(frag_row<T>(Few[1], LD, 0, 32 * ks), gf[u][ks], dp[u]);
                }
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float p = exp2_fast(fmaf(s[u][e], d.c2, -L[u]));
                    const float ds = p * (dp[u][e] - dl[u]);
                    s[u][e] = 4 * g + e < kl.front ? p : 0.f;
                    dp[u][e] = 4 * g + e < kl.front ? ds : 0.f;
                }
            }
        };
        // One walk over the tiles, from the one in buffer `at` on: of dQ, or of eps, the
        // rows' sums of P (dP - delta), which leaves the first tile in the next buffer.
        f32x4 eps[QN];
        int at = 0;
        const auto walk = [&](auto sum) {
            constexpr bool kSum = decltype(sum)::value;
            for (int n = 0; n < nt; n++) {
                const int buf = kBufs == 2 ? at : 0;
                const T *Kt = Ks + buf * kTile * LD, *Vt = Vs + buf * kTile * LD;
                fetch(n + 1 < nt ? n + 1 : kSum ? 0 : n);
                const int v0 = n * kTile;
#pragma unroll
                for (int kp = 0; kp < 2; kp++) {
                    int sight[QN][2];
                    int any = 0;
#pragma unroll
                    for (int u = 0; u < QN; u++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            sight[u][e] = HP == 2 && u ? sight[0][e]
                                                       : block_sight(v0 + 32 * kp + 16 * e, kl.shift,
                                                                     QR * w + (HP == 2 ? 0 : 16 * u), W, kl.always);
                            any |= sight[u][e];
                        }
                    if (!any) continue;
                    f32x4 s[QN][2], dp[QN][2];
#pragma unroll
                    for (int kt = 0; kt < 2; kt++) {
#pragma unroll
                        for (int u = 0; u < QN; u++) s[u][kt] = dp[u][kt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int ks = 0; ks < DT / 2; ks++) {
                            const auto ka = frag_row<T>(Kt, LD, 32 * kp + 16 * kt, 32 * ks);
                            const auto va = frag_row<T>(Vt, LD, 32 * kp + 16 * kt, 32 * ks);
#pragma unroll
                            for (int u = 0; u < QN; u++) {
                                s[u][kt] = M::mma(ka, qf[u][ks], s[u][kt]);
                                dp[u][kt] = M::mma(va, gf[u][ks], dp[u][kt]);
                            }
                        }
                    }
                    Frag sf[QN];
#pragma unroll
                    for (int u = 0; u < QN; u++) {
#pragma unroll
                        for (int kt = 0; kt < 2; kt++) {
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const float p = exp2_fast(fmaf(s[u][kt][e], d.c2, -L[u]));
                                dp[u][kt][e] = p * (dp[u][kt][e] - dl[u]);
                                if (!kSum) dp[u][kt][e] *= d.scale;
                            }
                            if (sight[u][kt] != 2)
#pragma unroll
                                for (int e = 0; e < 4; e++) {
                                    const int ve = v0 + 32 * kp + 16 * kt + 4 * g + e, jr = ve + kl.shift;
                                    const bool see = (jr <= ir[u]) & ((ve < kl.always) | (jr > ir[u] - W));
                                    dp[u][kt][e] = see & !alone[u] ? dp[u][kt][e] : 0.f;
                                }
                        }
                        // dS is rounded to the inputs' type for the product with K
                        if constexpr (kSum)
                            eps[u] += dp[u][0] + dp[u][1];
                        else
                            sf[u] = frag_acc<T>(dp[u][0], dp[u][1]);
                    }
                    if constexpr (!kSum)
#pragma unroll
                        for (int j = 0; j < DT; j++) {
                            const auto a = frag_col_pair<T>(Kt, LD, 32 * kp, 16 * j);
#pragma unroll
                            for (int u = 0; u < QN; u++) O[u][j] = M::mma(a, sf[u], O[u][j]);
                        }
                }
                if (kBufs == 1) __syncthreads();
                rk.store(Ks + (kBufs == 2 ? (buf ^ 1) * kTile * LD : 0));
                rv.store(Vs + (kBufs == 2 ? (buf ^ 1) * kTile * LD : 0));
                __syncthreads();
                at ^= 1;
            }
        };
        // (float32: o is as good as the sum)
        const bool exact = sizeof(T) == 2 && (d.W + S < kFewKeys || t0 < kFewKeys);
        if (exact) {
            f32x4 s[QN], dp[QN];
            if (few) front(s, dp);
#pragma unroll
            for (int u = 0; u < QN; u++) eps[u] = few ? dp[u] : zero;
            walk(std::true_type{});
#pragma unroll
            for (int u = 0; u < QN; u++)
                dl[u] += xor_add(xor_add((eps[u][0] + eps[u][1]) + (eps[u][2] + eps[u][3]), 16), 32);
        }
#pragma unroll
        for (int u = 0; u < QN; u++)
            if (t0 + ir[u] <= last && g == 0) delta[(b * d.T + t0 + ir[u]) * d.Hq + h0 + (HP == 2 ? u : 0)] = dl[u];
        if (few) {
            f32x4 s[QN], dp[QN];
            front(s, dp);
            Frag sf[QN];
#pragma unroll
            for (int u = 0; u < QN; u++) {
                dp[u] *= d.scale;
                sf[u] = frag_acc<T>(dp[u], zero);
            }
#pragma unroll
            for (int j = 0; j < DT; j++) {
                const auto a = frag_col_few<T>(Few[0], LD, 16 * j);
#pragma unroll
                for (int u = 0; u < QN; u++) O[u][j] = M::mma(a, sf[u], O[u][j]);
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < QN; u++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int at = (4 * g + e) * LS + 16 * (w * QN + u) + li;
                    Few[0][at] = (T)s[u][e];
                    Few[1][at] = (T)dp[u][e];
                }
        }
        walk(std::false_type{});
        if constexpr (FEW) {
            if (few) {   // dK, dV of the sinks in front over the workgroup's rows
#pragma unroll
                for (int u = 0; u < QN; u++)
#pragma unroll
                    for (int ks = 0; ks < DT / 2; ks++) {
                        const int at = (16 * (w * QN + u) + li) * LD + 32 * ks + 8 * g;
                        *reinterpret_cast<Frag *>(Ks + at) = qf[u][ks];
                        *reinterpret_cast<Frag *>(Vs + at) = gf[u][ks];
                    }
                __syncthreads();
                const int per = d.Hq / d.Hk / HP;
                float *pp = sink_part(sp, d, 1 + (int64_t)qt * per + (h0 / HP) % per, b, hk);
                for (int c = w; c < 2 * DT; c += 4) {
                    const bool isV = c >= DT;
                    const int c0 = 16 * (isV ? c - DT : c);
                    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ks = 0; ks < kRows / 32; ks++)
                        acc = M::mma(frag_row<T>(Few[isV ? 0 : 1], LS, 0, 32 * ks),
                                     frag_col<T>(isV ? Vs : Ks, LD, 32 * ks, c0), acc);
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (4 * g + e < kl.front && c0 + li < d.D)
                            pp[(4 * g + e) * 2 * d.D + (isV ? d.D : 0) + c0 + li] = acc[e];
                }
            }
        }
    }
#pragma unroll
    for (int u = 0; u < QN; u++) {
        const int64_t t = t0 + ir[u];
        if (t >= d.T) continue;
        T *row = dq + ((b * d.T + t) * d.Hq + h0 + (HP == 2 ? u : 0)) * d.D;
#pragma unroll
        for (int j = 0; j < DT; j++) O[u][j] = t < len ? O[u][j] : f32x4{0.f, 0.f, 0.f, 0.f};
        store_row<T, DT, VEC>(row, d.D, O[u]);
    }
}

// dK and dV of 64 keys, 16 a wave, over the query heads of their key head: a
// lane holds one key (column) and four neighbouring queries (rows).  Two
// workgroups share a compute unit; 128 keys and eight waves in one load fewer
// tiles but start and end together (backward of 8 x 4096 tokens, 16 and 8 heads
// of 128, window 128: 540 us instead of 507; this kernel 237 us, 540 MB).  SINKS:
// the sinks alone, for the queries behind part 0, 512 a workgroup, into parts 1 ..
template <typename T, int DT, bool VEC, bool SINKS>
__global__ __launch_bounds__(kThreads, sizeof(T) * DT <= 16 ? 2 : 1) void window_dkv_kernel(
    WinDims d, SinkParts sp, int ntiles, const T *__restrict__ q, const T *__restrict__ k,
    const T *__restrict__ v, const T *__restrict__ dout, const float *__restrict__ lse,
    const float *__restrict__ delta, const int32_t *__restrict__ lengths, T *__restrict__ dk,
    T *__restrict__ dv)
{
    using M = Mat<T>;
    constexpr int LD = DT * 16 + 8;
    constexpr int kBufs = sizeof(T) == 2 || DT <= 8 ? 2 : 1;
    __shared__ __align__(32) T Qs[kBufs][kTile * LD];
    __shared__ __align__(32) T Gs[kBufs][kTile * LD];
    __shared__ __align__(16) float Ls[kBufs][kTile], Dl[kBufs][kTile];

    int64_t rest = xcd_index(blockIdx.x, gridDim.x);
    int part = 0;
    if (SINKS) {
        part = 1 + (int)(rest % (sp.nparts - 1));
        rest /= sp.nparts - 1;
    }
    const int kt = (int)(rest % ntiles);
    rest /= ntiles;
    const int hk = (int)(rest % d.Hk);
    const int64_t b = rest / d.Hk;
    const int64_t len = seq_len(lengths, b, d.T);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l = threadIdx.x & 63, g = l >> 4;
    const int W = (int)d.W;
    const int64_t j0 = (int64_t)kt * kKeys;
    const int k0 = 16 * w, kr = k0 + (l & 15);    // the wave's first key and the lane's, relative to j0
    const int64_t j = j0 + kr;
    const int sinks = (int)(d.S > j0 ? d.S - j0 : 0);   // keys below this one are sinks
    const int per = d.Hq / d.Hk;
    f32x4 dK[DT], dV[DT];
#pragma unroll
    for (int n = 0; n < DT; n++) dK[n] = dV[n] = f32x4{0.f, 0.f, 0.f, 0.f};

    // The queries [first, end).  Where the dQ kernel sums the sinks in front of a
    // workgroup's windows, the queries of the last workgroup that has one inside
    // are visited here.
    const int64_t reach = j0 + kKeys - 1 + d.W + (sinks ? sp.near : 0);
    int64_t first = j0, end = reach < len ? reach : len;
    if (SINKS) {
        first = (int64_t)(part - 1) * kSinkRows;
        end = first + kSinkRows < len ? first + kSinkRows : len;
        if (first < reach) first = reach;   // nearer queries are in part 0
    }
    if (j0 < len && first < end) {
        typename M::Frag kf[DT / 2], vf[DT / 2];
        const int64_t jr = j < len ? j : len - 1;  // a row that exists; no query sees its copy
        const int nq = (int)((end - first + kTile - 1) / kTile);
        RowRegs<T, DT * 16, LD, VEC, kThreads> rq, rg;
        float rl, rd;
        const auto fetch = [&](int n) {
            const int h = hk * per + n / nq;
            const int64_t t0 = first + (int64_t)(n % nq) * kTile;
            const auto row = [&](int r) { return t0 + r < end ? t0 + r : end - 1; };
            rq.load([&](int r) { return q + b * d.qb + row(r) * d.qt + h * d.qh; }, d.D);
            rg.load([&](int r) { return dout + ((b * d.T + row(r)) * d.Hq + h) * d.D; }, d.D);
            const int64_t at = (b * d.T + row(l)) * d.Hq + h;
            rl = lse[at] * 1.4426950408889634f;
            rd = delta[at];
        };
        const auto put = [&](int buf) {
            rq.store(Qs[buf]);
            rg.store(Gs[buf]);
            if (threadIdx.x < kTile) {
                Ls[buf][l] = rl;
                Dl[buf][l] = rd;
            }
        };
        fetch(0);
#pragma unroll
        for (int ks = 0; ks < DT / 2; ks++) {
            kf[ks] = frag_global<T, VEC>(k + b * d.kb + jr * d.kt + hk * d.kh, 32 * ks + 8 * g, d.D);
            vf[ks] = frag_global<T, VEC>(v + b * d.vb + jr * d.vt + hk * d.vh, 32 * ks + 8 * g, d.D);
        }
        put(0);
        __syncthreads();
        for (int n = 0; n < per * nq; n++) {
            const int buf = kBufs == 2 ? n & 1 : 0;
            fetch(n + 1 < per * nq ? n + 1 : n);
            // first query of the tile relative to j0 (sinks: any number behind all keys will do)
            const int64_t t0 = first + (int64_t)(n % nq) * kTile;
            const int q0 = SINKS ? kKeys : (int)(t0 - j0);
            const int qend = q0 + (int)(end - t0);
#pragma unroll
            for (int half = 0; half < 2; half++) {
                const int r0 = 32 * half, k1 = k0 + 15, s0 = q0 + r0, s1 = s0 + 31;
                // as block_sight, for 16 keys and 32 queries
                const bool none = k0 > s1 || s0 >= qend ||
                                  (k0 >= sinks && (SINKS || s0 - k1 >= W));
                const bool all = k1 <= s0 && s1 < qend &&
                                 (SINKS ? k1 < sinks : s1 - k0 < W || (k1 < sinks && !sp.near));
                if (none) continue;
                f32x4 p[2], ds[2];
#pragma unroll
                for (int e2 = 0; e2 < 2; e2++) {
                    f32x4 s = {0.f, 0.f, 0.f, 0.f}, dp = s;
#pragma unroll
                    for (int ks = 0; ks < DT / 2; ks++) {
                        s = M::mma(frag_row<T>(Qs[buf], LD, r0 + 16 * e2, 32 * ks), kf[ks], s);
                        dp = M::mma(frag_row<T>(Gs[buf], LD, r0 + 16 * e2, 32 * ks), vf[ks], dp);
                    }
                    const f32x4 L = *reinterpret_cast<const f32x4 *>(Ls[buf] + r0 + 16 * e2 + 4 * g);
                    const f32x4 D = *reinterpret_cast<const f32x4 *>(Dl[buf] + r0 + 16 * e2 + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        p[e2][e] = exp2_fast(fmaf(s[e], d.c2, -L[e]));
                        ds[e2][e] = p[e2][e] * (dp[e] - D[e]) * d.scale;
                    }
                    if (!all)
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const int qr = q0 + r0 + 16 * e2 + 4 * g + e;
                            // a sink: all, or (near) where it stands in the query's workgroup's list
                            // behind its first window key
                            const int from = sp.near ? qr & ~(sp.near - 1) : kr;
                            const bool see = (kr <= qr) & (qr < qend) &
                                             (SINKS ? kr < sinks
                                                    : (qr - kr < W) | ((kr < sinks) & (from - kr < W)));
                            p[e2][e] = see ? p[e2][e] : 0.f;
                            // the first query sees one key, whose weight is 1 whatever the score
                            ds[e2][e] = see & (SINKS | (j0 + qr != 0)) ? ds[e2][e] : 0.f;
                        }
                }
                // P and dS are rounded to the inputs' type for the products with dO and Q
                const auto pf = frag_acc<T>(p[0], p[1]), sf = frag_acc<T>(ds[0], ds[1]);
#pragma unroll
                for (int c = 0; c < DT; c++) {
                    dV[c] = M::mma(frag_col_pair<T>(Gs[buf], LD, r0, 16 * c), pf, dV[c]);
                    dK[c] = M::mma(frag_col_pair<T>(Qs[buf], LD, r0, 16 * c), sf, dK[c]);
                }
            }
            if (kBufs == 1) __syncthreads();
            put(kBufs == 2 ? buf ^ 1 : 0);
            __syncthreads();
        }
    }
    const bool sink = sp.sums && kr < sinks;
    if (j >= d.T || (SINKS && !sink)) return;
    const int64_t at = ((b * d.T + j) * d.Hk + hk) * d.D;
    float *pp = sink ? sink_part(sp, d, part, b, hk) + j * 2 * d.D : nullptr;
    if (sink) {
        store_row<float, DT, false>(pp, d.D, dK);
        store_row<float, DT, false>(pp + d.D, d.D, dV);
    } else {
        store_row<T, DT, VEC>(dk + at, d.D, dK);
        store_row<T, DT, VEC>(dv + at, d.D, dV);
    }
}

// dK and dV of the sinks: the sum of their parts, in order: 8 strided sums of a
// column, joined pairwise.  Parts of workgroups without the sink in front of
// their windows were not written (near).
template <typename T>
__global__ __launch_bounds__(1024) void window_sinks_kernel(WinDims d, SinkParts sp, int per,
                                                            const int32_t *__restrict__ lengths,
                                                            T *__restrict__ dk, T *__restrict__ dv)
{
    __shared__ float sums[8][128];
    const int64_t r = blockIdx.x;   // (b, hk, j)
    const int64_t j = r % d.S, bh = r / d.S, hk = bh % d.Hk, b = bh / d.Hk;
    if (j >= d.T) return;
    const int64_t len = seq_len(lengths, b, d.T);
    const int64_t step = (int64_t)d.B * d.Hk * d.S * 2 * d.D;
    const int x = threadIdx.x, y = threadIdx.y;
    for (int c0 = 0; c0 < 2 * d.D; c0 += 128) {
        const int c = c0 + x;
        float s = 0.f;
        if (c < 2 * d.D) {
            const float *src = sp.sums + r * 2 * d.D + c;
            if (y == 0) s = src[0];
            for (int n = 1 + y; n < sp.nparts; n += 8) {
                if (sp.near) {
                    const int64_t t0 = (int64_t)((n - 1) / per) * sp.near;
                    if (t0 >= len || t0 - d.W + 1 <= j) continue;
                }
                s += src[n * step];
            }
        }
        __syncthreads();
        sums[y][x] = s;
        for (int n = 4; n > 0; n >>= 1) {
            __syncthreads();
            if (y < n) sums[y][x] += sums[y + n][x];
        }
        if (y == 0 && c < 2 * d.D) {
            T *out = c < d.D ? dk : dv;
            out[((b * d.T + j) * d.Hk + hk) * d.D + (c < d.D ? c : c - d.D)] = (T)sums[0][x];
        }
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
    return d;
}

// Blocks of 16 queries of a wave (D = 256 fills the registers with one, float32
// LDS with the tiles), and the heads of a workgroup: two where an even number
// of them shares a key head.
constexpr int query_blocks(int D, int esize) { return D <= 128 && esize == 2 ? 2 : 1; }
int blocks_of(const sdm_window_desc &s) { return query_blocks(s.D, s.dtype == SDM_F32 ? 4 : 2); }
int head_pair(const sdm_window_desc &s)
{
    return blocks_of(s) == 2 && (s.Hq / s.Hk) % 2 == 0 ? 2 : 1;
}
int queries_of(const sdm_window_desc &s) { return 64 * blocks_of(s) / head_pair(s); }

struct BackPlan {
    size_t parts, total;
    int near, nparts, ktiles;
};

BackPlan back_plan(const sdm_window_desc &s)
{
    BackPlan p = {};
    size_t at = ((size_t)s.B * s.T * s.Hq * 4 + 255) & ~(size_t)255;   // delta
    // sinks that queries see from behind their window
    if (s.sinks > 0 && s.T > s.window) {
        const int hp = head_pair(s);
        // the dQ kernel sums few sinks itself, where LDS holds its rows
        if (s.sinks <= kFewSinks && s.D <= 128) {
            p.near = queries_of(s);
            p.nparts = 1 + (int)((s.T + p.near - 1) / p.near) * (s.Hq / s.Hk / hp);
        } else {
            const int64_t rows = s.sinks < s.T ? s.sinks : s.T;
            p.nparts = 1 + (int)((s.T + kSinkRows - 1) / kSinkRows);
            p.ktiles = (int)((rows + kKeys - 1) / kKeys);
        }
        p.parts = at;
        at += (size_t)p.nparts * s.B * s.Hk * s.sinks * 2 * s.D * 4;
    }
    p.total = at;
    return p;
}

template <typename T, int DT, bool VEC>
hipError_t forward(const WindowArgs &a, hipStream_t stream)
{
    constexpr int QN = query_blocks(DT * 16, sizeof(T));
    WinDims d = dims_of(a.d);
    const int hp = head_pair(a.d), queries = queries_of(a.d);
    d.nq = (int)((d.T + queries - 1) / queries);
    const auto run = [&](auto kernel) {
        kernel<<<(unsigned)((int64_t)d.B * (d.Hq / hp) * d.nq), kThreads, 0, stream>>>(
            d, (const T *)a.q, (const T *)a.k, (const T *)a.v, (const T *)a.cache_k,
            (const T *)a.cache_v, a.pos, a.lengths, (T *)a.o, a.lse);
    };
    if (a.pos)
        hp == 2 ? run(window_fwd_kernel<T, DT, QN, QN, VEC, true>)
                : run(window_fwd_kernel<T, DT, QN, 1, VEC, true>);
    else
        hp == 2 ? run(window_fwd_kernel<T, DT, QN, QN, VEC, false>)
                : run(window_fwd_kernel<T, DT, QN, 1, VEC, false>);
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
    if (d.W == 1 && d.S == 0) d.scale = 0.f;   // every query sees one key: scores have no gradient
    const BackPlan p = back_plan(a.d);
    constexpr int QN = query_blocks(DT * 16, sizeof(T));
    const int hp = head_pair(a.d), queries = queries_of(a.d);
    const T *q = (const T *)a.q, *k = (const T *)a.k, *v = (const T *)a.v, *dout = (const T *)a.dout;
    float *delta = (float *)a.ws;
    const SinkParts sp = {p.nparts ? (float *)(a.ws + p.parts) : nullptr, p.near, p.nparts};
    d.nq = (int)((d.T + queries - 1) / queries);
    const auto run = [&](auto kernel) {
        kernel<<<(unsigned)((int64_t)d.B * (d.Hq / hp) * d.nq), kThreads, 0, stream>>>(
            d, sp, q, k, v, (const T *)a.oin, dout, a.lse_in, a.lengths, delta, (T *)a.dq);
    };
    constexpr bool kCan = DT <= 8;   // few sinks: up to 128 columns
    if (p.near)
        hp == 2 ? run(window_dq_kernel<T, DT, QN, QN, VEC, kCan>)
                : run(window_dq_kernel<T, DT, QN, 1, VEC, kCan>);
    else
        hp == 2 ? run(window_dq_kernel<T, DT, QN, QN, VEC, false>)
                : run(window_dq_kernel<T, DT, QN, 1, VEC, false>);
    const int ntiles = (int)((d.T + kKeys - 1) / kKeys);
    window_dkv_kernel<T, DT, VEC, false><<<(unsigned)((int64_t)d.B * d.Hk * ntiles), kThreads, 0, stream>>>(
        d, sp, ntiles, q, k, v, dout, a.lse_in, delta, a.lengths, (T *)a.dk, (T *)a.dv);
    if (p.ktiles)
        window_dkv_kernel<T, DT, VEC, true>
            <<<(unsigned)((int64_t)d.B * d.Hk * p.ktiles * (p.nparts - 1)), kThreads, 0, stream>>>(
                d, sp, p.ktiles, q, k, v, dout, a.lse_in, delta, a.lengths, (T *)a.dk, (T *)a.dv);
    if (p.nparts)
        window_sinks_kernel<T><<<(unsigned)((int64_t)d.B * d.Hk * d.S), dim3(128, 8), 0, stream>>>(
            d, sp, d.Hq / d.Hk / hp, a.lengths, (T *)a.dk, (T *)a.dv);
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
