// Selective state space scan: one decay per head and token, B and C shared by
// the heads of a group.  Per head, with D_t = softplus(dt_t + bias):
//   S_t = a_t S_{t-1} + D_t x_t B_t^T,  a_t = e^{D_t A},   y_t = S_t C_t + D x_t
//
// In chunks of 64 tokens, with c_t the running sum of log2 a in the chunk
// (kept as two float32 that hold it to 48 bits, so that differences of large
// sums stay exact) and S the state before the chunk:
//   y_t = 2^{c_t} S C_t + sum_{s <= t} M_ts x_s,   M_ts = (C_t.B_s) 2^{c_t - c_s} D_s
//   S  <- 2^{c_63} S + sum_s x_s (w_s B_s)^T,      w_s = 2^{c_63 - c_s} D_s
// which are 16x16 matrix products.  Every exponent is a sum of logs of decays
// (<= 0 for A <= 0), so nothing is divided by a decay.
#include "mix_internal.h"

#include "lane_ops.h"
#include "mix_device.h"

namespace sdm {
namespace {

constexpr int Q = 64;         // tokens of a chunk
constexpr int kSlice = 64;    // columns of x that a workgroup holds: 16 a wave
constexpr int kThreads = 256;
constexpr int kMaxSegs = 256;   // segments of the time axis
constexpr int LX = kSlice + 8;  // LDS row stride of 64-wide tiles

// LDS leaves these kernels two waves a SIMD, so the compiler may use half of the
// registers for each and need not hold loads back to save some.
#define TWO_WAVES __attribute__((amdgpu_waves_per_eu(2, 2)))

struct ScanDims {
    int B, H, P, N, G;
    int64_t T;
    int nc;                    // chunks
    int nps;                   // slices of x's columns
    int nseg, cps;             // segments of the time axis, chunks of each
    int64_t xb, xt, bb, bt, cb, ct;
};

// ------------------------------------------------------------------ decays
// delta[bh][t] = D_t and cs[bh][t] = c_t (high and low part) for whole chunks;
// tokens behind a sequence's length have D = 0 (the state passes unchanged).
// A wave per (sequence, chunk, head); lane = token.
template <typename T>
__global__ __launch_bounds__(kThreads) void scan_prep_kernel(
    ScanDims d, const T *__restrict__ dt, const float *__restrict__ A,
    const float *__restrict__ bias, const int32_t *__restrict__ lengths, int softplus,
    float *__restrict__ delta, float2 *__restrict__ cs)
{
    const int64_t u = (int64_t)blockIdx.x * 4 + threadIdx.y;
    if (u >= (int64_t)d.B * d.nc * d.H) return;
    const int h = (int)(u % d.H);
    const int64_t bc = u / d.H;
    const int c = (int)(bc % d.nc);
    const int64_t b = bc / d.nc;
    const int64_t t = (int64_t)c * Q + threadIdx.x;
    float v = 0.f;
    if (t < seq_len(lengths, b, d.T)) {
        v = (float)dt[(b * d.T + t) * d.H + h] + (bias ? bias[h] : 0.f);
        if (softplus) v = v > 20.f ? v : log1pf(expf(v));
    }
    double l = (double)v * (double)A[h] * 1.4426950408889634;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(l, m);
        if ((int)threadIdx.x >= m) l += o;
    }
    const int64_t at = ((b * d.H + h) * d.nc + c) * Q + threadIdx.x;
    delta[at] = v;
    const float hi = (float)l;
    cs[at] = make_float2(hi, (float)(l - (double)hi));
}

// 2^{c_t - c_s}
__device__ __forceinline__ float decay(float2 t, float2 s)
{
    return exp2_fast((t.x - s.x) + (t.y - s.y));
}

// x of the lane n to the left in the 16-lane row, 0 for the row's first n lanes.
template <int n>
__device__ __forceinline__ float row_shr(float x)
{
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x110 | n, 0xF, 0xF, true));
}

// x of the lane n to the right, 0 for the row's last n lanes.
template <int n>
__device__ __forceinline__ float row_shl(float x)
{
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x100 | n, 0xF, 0xF, true));
}

// The tiles on and under the diagonal of a 4 x 4 grid: 0 (0,0), 1 (1,0), 2 (1,1) ..
__device__ __forceinline__ int tile_row(int id) { return id < 1 ? 0 : id < 3 ? 1 : id < 6 ? 2 : 3; }
__device__ __forceinline__ int tile_id(int row, int col) { return row * (row + 1) / 2 + col; }

// One wave's part of a state: S^T, tiles j0 .. j0 + NJ - 1 of 16 rows n, rows
// (l / 16) * 4 + i of each, column p of the lane.  In the caller's [P][N]
// layout or the workspace's [N][P].
template <int NJ>
__device__ __forceinline__ void state_load(f32x4 (&S)[NJ], const float *src, bool api, int j0, int p, int P,
                                           int N)
{
    const int n0 = 16 * j0 + 4 * ((threadIdx.x & 63) >> 4);
    const int64_t sp = api ? N : 1, sn = api ? 1 : P;
    const float *q = src ? src + p * sp + n0 * sn : nullptr;
#pragma unroll
    for (int j = 0; j < NJ; j++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            S[j][i] = src && p < P && n0 + 16 * j + i < N ? q[(16 * j + i) * sn] : 0.f;
}

template <int NJ>
__device__ __forceinline__ void state_store(const f32x4 (&S)[NJ], float *dst, bool api, int j0, int p, int P,
                                            int N)
{
    const int n0 = 16 * j0 + 4 * ((threadIdx.x & 63) >> 4);
    if (p >= P) return;
    const int64_t sp = api ? N : 1, sn = api ? 1 : P;
    float *q = dst + p * sp + n0 * sn;
#pragma unroll
    for (int j = 0; j < NJ; j++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (n0 + 16 * j + i < N) q[(16 * j + i) * sn] = S[j][i];
}

// The weighted columns w_s U[s], columns col0 .. + 15 of U, for state_add.
// They are carried to 24 bits (three bfloat16 terms), so the float32 state
// keeps its precision whatever the inputs' type.
template <typename T>
struct Weighted {
    typename Mat<T>::Frag f[2][Mat<T>::kTerms];
    __device__ __forceinline__ Weighted(const T *U, const float *wt, int col0)
    {
        const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int ks = 0; ks < 2; ks++) {
            const auto u = frag_col_pair<T>(U, LX, 32 * ks, col0);
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(wt + 32 * ks + g * 4);
            const f32x4 hi = *reinterpret_cast<const f32x4 *>(wt + 32 * ks + 16 + g * 4);
            split_frag<T>(__builtin_convertvector(u, f32x8) *
                              __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7),
                          f[ks]);
        }
    }
};

// S <- scale S + sum_s V[s]^T (w_s U[s]) for one chunk, tiles j0 .. of the rows n.
template <typename T, int NJ, int LN>
__device__ __forceinline__ void state_add(f32x4 *S, const T *V, const Weighted<T> &u, float scale, int j0)
{
    using M = Mat<T>;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
        S[j] *= scale;
#pragma unroll
        for (int ks = 0; ks < 2; ks++) {
            const auto a = frag_col_pair<T>(V, LN, 32 * ks, 16 * (j0 + j));
#pragma unroll
            for (int n = 0; n < M::kTerms; n++) S[j] = M::mma(a, u.f[ks][n], S[j]);
        }
    }
}

// ----------------------------------------------------------------- forward
// A workgroup walks the chunks of one (sequence, head, slice of 64 columns,
// segment) in order.  Its eight waves work in two roles, so that every SIMD
// has two waves whose waits fall at different times: waves 0 .. 3 hold the
// state in registers, 16 columns each, update it and hand it to the others
// through LDS, rounded (read before a step's barrier, replaced behind it); waves
// 4 .. 7 compute M (shared through LDS) and y, 16 columns each.  Products are taken transposed (M^T, y^T, S^T): a lane then
// holds one token and four neighbouring columns, so that a token's decay is
// one number a lane, stores take four columns, and the state's accumulators
// are the next product's operand as they stand.  The next two chunks' tiles
// are on their way from HBM while a chunk is worked on; with kBufs = 2 they go
// to a second set of tiles (as long as two sets fit into 160 KB of LDS).  Bound by
// the time of a step's dependent reads, products and barriers, 2.0 us at N = 64
// and 3.1 at N = 128: 8 x 4096 tokens, 16 heads of 128 x 64, bfloat16: 133 us for
// the call, 2.1 TB/s; four waves a SIMD spill (273 us).
template <typename T, int NT, bool VEC>
__global__ __launch_bounds__(2 * kThreads) TWO_WAVES void scan_walk_kernel(
    ScanDims d, const T *__restrict__ x, const T *__restrict__ Bm, const T *__restrict__ Cm,
    const float *__restrict__ D, const float *__restrict__ delta, const float2 *__restrict__ cs,
    const int32_t *__restrict__ lengths, const float *init, int init_api, float *state,
    T *__restrict__ y)
{
    using M = Mat<T>;
    using Frag = typename M::Frag;
    using Half = typename M::Half;
    constexpr int LN = NT * 16 + 8;
    constexpr int kBufs = sizeof(T) == 2 || NT == 2 ? 2 : 1;
    constexpr int NF = NT / 2;
    __shared__ __align__(32) T Xs[kBufs][Q * LX];
    __shared__ __align__(32) T Bs[kBufs][Q * LN];
    __shared__ __align__(32) T Cs[kBufs][Q * LN];
    __shared__ __align__(32) T Ms[Q * LX];
    __shared__ __align__(32) Frag Sf[4][NF][64];
    __shared__ __align__(16) float dl[kBufs][Q], wt[kBufs][Q];
    __shared__ __align__(16) float2 cc[kBufs][Q];

    const int seg = blockIdx.x % d.nseg;
    const int64_t r0 = blockIdx.x / d.nseg;
    const int ps = (int)(r0 % d.nps);
    const int64_t bh = r0 / d.nps;
    const int h = (int)(bh % d.H);
    const int64_t b = bh / d.H;
    const int grp = h / (d.H / d.G);
    const int64_t len = seq_len(lengths, b, d.T);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave & 3;
    const bool keeper = wave < 4;
    const int l = threadIdx.x & 63, g = l >> 4, li = l & 15;
    const int pcols = d.P - ps * kSlice < kSlice ? d.P - ps * kSlice : kSlice;
    const T *xp = x + b * d.xb + (int64_t)h * d.P + ps * kSlice;
    const T *bp = Bm + b * d.bb + (int64_t)grp * d.N;
    const T *cp = Cm + b * d.cb + (int64_t)grp * d.N;
    const float Dh = D ? D[h] : 0.f;

    // a chunk's tiles in registers
    struct Ahead {
        TileRegs<T, Q, kSlice, LX, 2 * kThreads, VEC> x;
        TileRegs<T, Q, NT * 16, LN, 2 * kThreads, VEC> b, c;
        float d;
        float2 me, tot;
    };
    const auto rows_of = [&](int c) {
        const int64_t n = len - (int64_t)c * Q;
        return n < 0 ? 0 : n < Q ? (int)n : Q;
    };
    const auto fetch = [&](Ahead &r, int c) {
        const int64_t t0 = (int64_t)c * Q;
        const int rows = rows_of(c);
        r.x.load(xp + t0 * d.xt, d.xt, rows, pcols);
        r.b.load(bp + t0 * d.bt, d.bt, rows, d.N);
        r.c.load(cp + t0 * d.ct, d.ct, rows, d.N);
        const int64_t at = (bh * d.nc + c) * Q;
        r.me = cs[at + l];
        r.tot = cs[at + Q - 1];
        r.d = delta[at + l];
    };
    const auto put = [&](const Ahead &r, int n) {
        r.x.store(Xs[n]);
        r.b.store(Bs[n]);
        r.c.store(Cs[n]);
        if (threadIdx.x < Q) {
            dl[n][threadIdx.x] = r.d;
            cc[n][threadIdx.x] = r.me;
            wt[n][threadIdx.x] = decay(r.tot, r.me) * r.d;
        }
    };

    const int c0 = seg * d.cps, c1 = c0 + d.cps < d.nc ? c0 + d.cps : d.nc;
    Ahead r0a, r1a;
    fetch(r0a, c0);
    f32x4 S[NT];
    const int pl = ps * kSlice + 16 * w + li;
    const auto hand_over = [&]() {
#pragma unroll
        for (int j = 0; j < NF; j++) Sf[w][j][l] = frag_acc<T>(S[2 * j], S[2 * j + 1]);
    };
    if (keeper) {
        const float *src = init;
        if (src) src += (init_api ? bh : bh * d.nseg + seg) * (int64_t)d.P * d.N;
        state_load<NT>(S, src, init_api, 0, pl, d.P, d.N);
        hand_over();
    } else if (w < 2) {
        // the two tiles right of the diagonal that products read: sources behind the tokens
        const int t = 32 * w + li;
        const Half zero = __builtin_convertvector(f32x4{0.f, 0.f, 0.f, 0.f}, Half);
        *reinterpret_cast<Half *>(Ms + t * LX + 32 * w + 16 + 4 * g) = zero;
    }
    put(r0a, 0);
    fetch(r1a, c0 + 1 < c1 ? c0 + 1 : c0);
    __syncthreads();
    // Chunk c, with chunk c + 1 in `next`, and chunk c + 2 to be asked for (at the
    // end the last one once more).  No load or store stands behind a branch, so a
    // wait for one chunk's loads leaves the next one's in flight.
    const auto chunk = [&](int c, int n, Ahead &next, Ahead &far) {
        const int64_t t0 = (int64_t)c * Q;
        const int rows = rows_of(c);
        fetch(far, c + 2 < c1 ? c + 2 : c1 - 1);
        if (keeper) {
            const float2 tot = cc[n][Q - 1];
            const float scale = exp2_fast(tot.x + tot.y);
            const Weighted<T> u(Xs[n], wt[n], 16 * w);
            state_add<T, NF, LN>(S, Bs[n], u, scale, 0);
            __syncthreads();
            state_add<T, NF, LN>(S + NF, Bs[n], u, scale, NF);
            hand_over();
        } else {
            // M^T: the ten 16 x 16 tiles on and under the diagonal, tokens in columns.
            // Three a wave, with no branch between them (the last tile three times over):
            // what a step costs is the time of its dependent reads and products.
            f32x4 acc[3];
#pragma unroll
            for (int k = 0; k < 3; k++) {
                const int id = w + 4 * k < 9 ? w + 4 * k : 9;  // (0,0) (1,0) (1,1) (2,0) ..
                const int tt = tile_row(id), st = id - tile_id(tt, 0);
                acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < NF; ks++)
                    acc[k] = M::mma(frag_row<T>(Bs[n], LN, 16 * st, 32 * ks),
                                    frag_row<T>(Cs[n], LN, 16 * tt, 32 * ks), acc[k]);
            }
#pragma unroll
            for (int k = 0; k < 3; k++) {
                const int id = w + 4 * k < 9 ? w + 4 * k : 9;
                const int tt = tile_row(id), st = id - tile_id(tt, 0);
                const int t = 16 * tt + li, s0 = 16 * st + 4 * g;
                const float2 ct = cc[n][t];
                const f32x4 ds = *reinterpret_cast<const f32x4 *>(dl[n] + s0);
                const f32x4 c0 = *reinterpret_cast<const f32x4 *>(cc[n] + s0);
                const f32x4 c1 = *reinterpret_cast<const f32x4 *>(cc[n] + s0 + 2);
                const f32x4 f = {decay(ct, make_float2(c0[0], c0[1])), decay(ct, make_float2(c0[2], c0[3])),
                                 decay(ct, make_float2(c1[0], c1[1])), decay(ct, make_float2(c1[2], c1[3]))};
                const f32x4 v = acc[k] * f * ds;
#pragma unroll
                for (int i = 0; i < 4; i++) acc[k][i] = s0 + i <= t ? v[i] : 0.f;
                // the decayed scores are rounded to the inputs' type for the product with x
                *reinterpret_cast<Half *>(Ms + t * LX + s0) = __builtin_convertvector(acc[k], Half);
            }
            // y^T for the wave's columns.  What comes from the state needs no M, so it is
            // taken before the barrier; the state came rounded to the inputs' type.
            Frag sf[NF], xf[2];
#pragma unroll
            for (int j = 0; j < NF; j++) sf[j] = Sf[w][j][l];
#pragma unroll
            for (int ks = 0; ks < 2; ks++) xf[ks] = frag_col<T>(Xs[n], LX, 32 * ks, 16 * w);
            f32x4 yr[4];
#pragma unroll
            for (int r = 0; r < 4; r++) {
                yr[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < NF; j++)
                    yr[r] = M::mma(sf[j], frag_row_pair<T>(Cs[n], LN, 16 * r, 32 * j), yr[r]);
                const float2 ct = cc[n][16 * r + li];
                yr[r] *= exp2_fast(ct.x + ct.y);
            }
            __syncthreads();
            const int p = ps * kSlice + 16 * w + 4 * g;
            const Sink<T> out(y + ((b * d.T + t0) * d.H + h) * d.P);
            const uint32_t hp = (uint32_t)d.H * d.P;
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int t = 16 * r + li;
                f32x4 acc = yr[r];
#pragma unroll
                for (int ks = 0; ks <= r / 2; ks++)
                    acc = M::mma(xf[ks], frag_row<T>(Ms, LX, 16 * r, 32 * ks), acc);
                const auto xv = *reinterpret_cast<const Half *>(Xs[n] + t * LX + 16 * w + 4 * g);
                acc += __builtin_convertvector(xv, f32x4) * Dh;
                if (t >= rows) acc = f32x4{0.f, 0.f, 0.f, 0.f};
                out.template write4<VEC>((uint32_t)t * hp + p, t0 + t < d.T ? d.P - p : 0, acc);
            }
        }
        if (kBufs == 1) __syncthreads();
        put(next, kBufs == 2 ? n ^ 1 : 0);
        __syncthreads();
    };
    for (int c = c0;;) {
        chunk(c, 0, r1a, r0a);
        if (++c == c1) break;
        chunk(c, kBufs - 1, r0a, r1a);
        if (++c == c1) break;
    }
    if (keeper && seg == d.nseg - 1)
        state_store<NT>(S, state + bh * (int64_t)d.P * d.N, true, 0, pl, d.P, d.N);
}

// A tile of `each` lies as the lanes hold it: element (n, p) = (16 j + 4 g + i,
// 16 w + li) at each_at(j, w, i) + 16 g + li, so that a store covers 256 bytes in
// one piece, and so do the gradient kernel's reads (whole backward of 8 x 4096
// tokens, 16 heads of 128 x 64: 506 us; with rows of p 523).
__device__ __forceinline__ constexpr int each_at(int j, int w, int i) { return (j * 4 + w) * 256 + 64 * i; }

// States alone.  Forward: U = x, V = B, weights 2^{c_63 - c_s} D_s; `each` gets
// the state before every chunk.  Reverse: U = dy, V = C, weights 2^{c_t},
// chunks from last to first: the gradient G of the state,
//   G <- 2^{c_63} G + sum_t 2^{c_t} C_t dy_t^T,
// and `each` gets G behind every chunk; a tile per slice, whose rows and columns
// beyond N and P are zero.  `end` gets the last one: per segment in the
// workspace's layout, or (end_api) the caller's gradient.  Waves w and w + 4 hold
// the same 16 columns, each one half of the rows n.  The backward runs both
// directions in one launch: a walk is bound by the time of its steps, and two
// walks share a compute unit (both directions of 8 x 4096 tokens, 16 heads of
// 128 x 64: 178 us, 4.5 TB/s, most of it the states written).
template <typename T>
struct StateJob {
    const T *U, *V;
    int64_t ub, ut, vb, vt;
    const float *init;
    float *each, *end;
    int rev, init_api, end_api;
};

template <typename T, int NT, bool VEC, bool EACH>
__global__ __launch_bounds__(2 * kThreads) void scan_state_kernel(
    ScanDims d, const float *__restrict__ delta, const float2 *__restrict__ cs,
    const int32_t *__restrict__ lengths, StateJob<T> job0, StateJob<T> job1)
{
    constexpr int LN = NT * 16 + 8;
    constexpr int NJ = NT / 2;
    __shared__ __align__(32) T Us[2][Q * LX];
    __shared__ __align__(32) T Vs[2][Q * LN];
    __shared__ __align__(16) float wt[2][Q];
    __shared__ float scale[2];

    const StateJob<T> job = blockIdx.y ? job1 : job0;
    const int seg = blockIdx.x % d.nseg;
    const int64_t r0 = blockIdx.x / d.nseg;
    const int ps = (int)(r0 % d.nps);
    const int64_t bh = r0 / d.nps;
    const int h = (int)(bh % d.H);
    const int64_t b = bh / d.H;
    const int grp = h / (d.H / d.G);
    const int64_t len = seq_len(lengths, b, d.T);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave & 3, j0 = (wave >> 2) * NJ;
    const int pcols = d.P - ps * kSlice < kSlice ? d.P - ps * kSlice : kSlice;
    const int p = ps * kSlice + 16 * w + (threadIdx.x & 15);
    const int64_t PN = (int64_t)d.P * d.N;
    const T *up = job.U + b * job.ub + (int64_t)h * d.P + ps * kSlice;
    const T *vp = job.V + b * job.vb + (int64_t)grp * d.N;

    const int c0 = seg * d.cps, c1 = c0 + d.cps < d.nc ? c0 + d.cps : d.nc;
    struct Ahead {
        TileRegs<T, Q, kSlice, LX, 2 * kThreads, VEC> u;
        TileRegs<T, Q, NT * 16, LN, 2 * kThreads, VEC> v;
        float d;
        float2 me, tot;
    };
    const auto chunk_of = [&](int k) { return job.rev ? c0 + c1 - 1 - k : k; };
    const auto fetch = [&](Ahead &r, int k) {
        const int c = chunk_of(k);
        const int64_t t0 = (int64_t)c * Q;
        const int rows = len - t0 < 0 ? 0 : len - t0 < Q ? (int)(len - t0) : Q;
        r.u.load(up + t0 * job.ut, job.ut, rows, pcols);
        r.v.load(vp + t0 * job.vt, job.vt, rows, d.N);
        const int64_t at = (bh * d.nc + c) * Q;
        r.me = cs[at + (threadIdx.x & 63)];
        r.tot = cs[at + Q - 1];
        r.d = delta[at + (threadIdx.x & 63)];
    };
    const auto put = [&](const Ahead &r, int n) {
        r.u.store(Us[n]);
        r.v.store(Vs[n]);
        if (threadIdx.x < Q)
            wt[n][threadIdx.x] = job.rev ? exp2_fast(r.me.x + r.me.y) : decay(r.tot, r.me) * r.d;
        if (threadIdx.x == 0) scale[n] = exp2_fast(r.tot.x + r.tot.y);
    };
    Ahead r0a, r1a;
    fetch(r0a, c0);
    f32x4 S[NJ];
    {
        const float *src = job.init;
        if (src) src += (job.init_api ? bh : bh * d.nseg + seg) * PN;
        state_load<NJ>(S, src, job.init_api, j0, p, d.P, d.N);
    }
    put(r0a, 0);
    fetch(r1a, c0 + 1 < c1 ? c0 + 1 : c0);
    __syncthreads();
    const auto step = [&](int k, int n, Ahead &next, Ahead &far) {
        fetch(far, k + 2 < c1 ? k + 2 : c1 - 1);
        if constexpr (EACH) {
            float *q = job.each + ((bh * d.nc + chunk_of(k)) * d.nps + ps) * (NT * 16 * kSlice) +
                       each_at(j0, w, 0) + (threadIdx.x & 63);
#pragma unroll
            for (int j = 0; j < NJ; j++)
#pragma unroll
                for (int i = 0; i < 4; i++) q[each_at(j, 0, i)] = S[j][i];
        }
        const Weighted<T> u(Us[n], wt[n], 16 * w);
        state_add<T, NJ, LN>(S, Vs[n], u, scale[n], j0);
        put(next, n ^ 1);
        __syncthreads();
    };
    for (int k = c0;;) {
        step(k, 0, r1a, r0a);
        if (++k == c1) break;
        step(k, 1, r0a, r1a);
        if (++k == c1) break;
    }
    if (!job.end) return;
    if (!job.end_api)
        state_store<NJ>(S, job.end + (bh * d.nseg + seg) * PN, false, j0, p, d.P, d.N);
    else if (seg == (job.rev ? 0 : d.nseg - 1))
        state_store<NJ>(S, job.end + bh * PN, true, j0, p, d.P, d.N);
}

// Joins the segments: from each segment's own contribution (`own`, computed
// from zero) and the state before the first one, the state before every
// segment, in the order of the walk.
__global__ __launch_bounds__(kThreads) void scan_join_kernel(ScanDims d, const float2 *__restrict__ cs,
                                                             int rev, const float *first,
                                                             const float *__restrict__ own,
                                                             float *__restrict__ start)
{
    __shared__ float keep[kMaxSegs];
    const int64_t PN = (int64_t)d.P * d.N;
    const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t bh = blockIdx.y;
    for (int seg = threadIdx.x; seg < d.nseg; seg += kThreads) {
        const int c0 = seg * d.cps, c1 = c0 + d.cps < d.nc ? c0 + d.cps : d.nc;
        double sum = 0.0;
        for (int c = c0; c < c1; c++) {
            const float2 t = cs[(bh * d.nc + c) * Q + Q - 1];
            sum += (double)t.x + (double)t.y;
        }
        keep[seg] = exp2_fast((float)sum);
    }
    __syncthreads();
    if (e >= PN) return;
    const int n = (int)(e / d.P), p = (int)(e % d.P);
    float S = first ? first[bh * PN + (int64_t)p * d.N + n] : 0.f;
#pragma unroll 8
    for (int k = 0; k < d.nseg; k++) {
        const int seg = rev ? d.nseg - 1 - k : k;
        start[(bh * d.nseg + seg) * PN + e] = S;
        S = fmaf(keep[seg], S, own[(bh * d.nseg + seg) * PN + e]);
    }
}

// ---------------------------------------------------------------- backward
// Gradients of one chunk from the state S before it, the gradient G of the
// state behind it and the inputs.  With E_ts = 2^{c_t - c_s}, for s <= t:
//   dx_s = sum_t M_ts dy_t + w_s G B_s + D dy_s
//   dC_t = sum_h sum_s W_ts B_s + 2^{c_t} S^T dy_t,     W_ts = (dy_t.x_s) E_ts D_s
//   dB_s = sum_h sum_t W_ts C_t + w_s G^T x_s
//   dD_s = sum_t e_ts + 2^{c_63 - c_s} B_s.(G^T x_s) + A dl_s,  e_ts = (C_t.B_s)(dy_t.x_s) E_ts
// and the gradient of a token's log decay collects what flows across it: pairs
// of a source before it (in the chunk, or S) and a target from it on (in the
// chunk, or G),
//   dl_r = sum_{s < r <= t} e_ts D_s + sum_{t >= r} 2^{c_t} dy_t.S C_t
//        + sum_{s < r} w_s x_s.G B_s + 2^{c_63} <G, S>,
// which is made of such sums alone, never of the difference of two long ones.
// The pairs in the chunk are summed as prefixes over s of every row t, then
// over t: a small flow across a boundary keeps its own precision beside large
// pairs on one side of it.  S and G enter the products for dC, dB and dD to 24
// bits.
//
// A workgroup of eight waves owns a chunk and a block of the heads of a group,
// whose sums for dB and dC stay in registers: waves 0 .. 3 hold those for dC,
// a quarter of the columns n each, waves 4 .. 7 those for dB.  The ten 16 x 16
// tiles on and under the diagonal of the 64 x 64 products are dealt to the
// waves; dx is split into 16 columns and half of the tokens a wave.  The next
// slice of x, dy, S and G is loaded while one is worked on.  What a head's
// dD and dl need is left in LDS, and summed up for four heads at a time, by a
// wave each.  8 x 4096 tokens, 16 heads of 128 x 64, bfloat16: about 300 us of
// the backward's 476, 3.1 TB/s of x, dy, dx and both states; no registers are left
// for loads further ahead.
constexpr int kBatch = 4;

// What the waves leave for a head's token gradients.
struct HeadSums {
    float2 cc[Q];
    float dl[Q], wt[Q], et[Q];   // D_t, w_t, 2^{c_63 - c_t}
    float colE[10][16];          // per tile: sum_t e_ts
    float cross[10][16];         //   pairs with both ends in the tile that cross column r
    float rows[Q][4];            //   sum_s e_ts D_s of row t
    float all[10];               //   the tile's sum
    float dotC[4][Q], dotB[4][Q];  // per quarter of n: C_t.(S^T dy_t), B_s.(G^T x_s)
    float gs[4], dd[8];          // <G, S> and sum dy x, in parts
};

template <typename T, int NT, bool VEC>
__global__ __launch_bounds__(2 * kThreads) TWO_WAVES void scan_grad_kernel(
    ScanDims d, int hblocks, const T *__restrict__ x, const T *__restrict__ dy,
    const T *__restrict__ Bm, const T *__restrict__ Cm, const float *__restrict__ A,
    const float *__restrict__ D, const float *__restrict__ delta, const float2 *__restrict__ cs,
    const int32_t *__restrict__ lengths, int softplus, const float *__restrict__ Sws,
    const float *__restrict__ Gws, T *__restrict__ dx, T *__restrict__ ddt, T *__restrict__ dB,
    T *__restrict__ dC, float *__restrict__ parts, float *__restrict__ hsum)
{
    using M = Mat<T>;
    using Frag = typename M::Frag;
    using Half = typename M::Half;
    constexpr int LN = NT * 16 + 8;
    constexpr int NW = NT >= 4 ? NT / 4 : 1;      // 16-column tiles of n per wave
    constexpr int NF = NT / 2;
    constexpr int kBufs = sizeof(T) == 2 ? 2 : 1;
    constexpr bool kGs = sizeof(T) == 2;          // G, rounded, through LDS
    constexpr int kTile = NT * 16 * kSlice;       // floats of a state tile
    constexpr bool kEarly = NT < 8;
    __shared__ __align__(32) T Xs[kBufs][Q * LX];
    __shared__ __align__(32) T Ys[kBufs][Q * LX];
    __shared__ __align__(32) T Bs[Q * LN];
    __shared__ __align__(32) T Cs[Q * LN];
    __shared__ __align__(32) T Ms[Q * LX];        // M, then W
    __shared__ __align__(32) T Gs[kGs ? kBufs : 1][kGs ? NT * 16 * LX : 1];
    __shared__ __align__(16) HeadSums hs[kBatch];

    const int hb = blockIdx.x % hblocks;
    const int64_t r0 = blockIdx.x / hblocks;
    const int grp = (int)(r0 % d.G);
    const int64_t r1 = r0 / d.G;
    const int c = (int)(r1 % d.nc);
    const int64_t b = r1 / d.nc;
    const int per = d.H / d.G;
    const int h0 = grp * per + (int)((int64_t)per * hb / hblocks);
    const int h1 = grp * per + (int)((int64_t)per * (hb + 1) / hblocks);
    const int64_t t0 = (int64_t)c * Q;
    const int64_t len = seq_len(lengths, b, d.T);
    const int rows = len - t0 < 0 ? 0 : len - t0 < Q ? (int)(len - t0) : Q;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave & 3;
    const bool sideB = wave >= 4;
    const int l = threadIdx.x & 63, g = l >> 4, li = l & 15;
    const int nt0 = w * NW;                       // the wave's column tiles of n
    const bool ncols = nt0 < NT;

    // one slice of x, dy, S and G in flight
    TileRegs<T, Q, kSlice, LX, 2 * kThreads, VEC> rx, ry;
    f32x4 rS[2][NW][2], rG[2][NW][2];             // rows n = 16 j + li, columns 32 ks + 8 g ..
    const int64_t yt = (int64_t)d.H * d.P;
    const auto fetch = [&](int step) {
        const int h = h0 + step / d.nps, ps = step % d.nps;
        const int pcols = d.P - ps * kSlice < kSlice ? d.P - ps * kSlice : kSlice;
        rx.load(x + b * d.xb + t0 * d.xt + (int64_t)h * d.P + ps * kSlice, d.xt, rows, pcols);
        ry.load(dy + (b * d.T + t0) * yt + (int64_t)h * d.P + ps * kSlice, yt, rows, pcols);
    };
    const auto fetch_states = [&](int step) {
        if (!ncols) return;
        const int h = h0 + step / d.nps, ps = step % d.nps;
        const int64_t at = (((b * d.H + h) * d.nc + c) * d.nps + ps) * kTile + each_at(nt0, g >> 1, li & 3) +
                           16 * (li >> 2) + 8 * (g & 1);
#pragma unroll
        for (int ks = 0; ks < 2; ks++)
#pragma unroll
            for (int j = 0; j < NW; j++)
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    const int64_t e = at + each_at(j, 2 * ks, 0) + 4 * u;
                    rS[ks][j][u] = *reinterpret_cast<const f32x4 *>(Sws + e);
                    if (sideB) rG[ks][j][u] = *reinterpret_cast<const f32x4 *>(Gws + e);
                }
    };
    fetch(0);
    fetch_states(0);
    load_tile<T, Q, NT * 16, LN, 2 * kThreads, VEC>(
        Bs, Bm + b * d.bb + t0 * d.bt + (int64_t)grp * d.N, d.bt, rows, d.N);
    load_tile<T, Q, NT * 16, LN, 2 * kThreads, VEC>(
        Cs, Cm + b * d.cb + t0 * d.ct + (int64_t)grp * d.N, d.ct, rows, d.N);
    __syncthreads();

    // the wave's tiles: `wave`, and for waves 0 and 1 also 8 and 9
    const int ntile = wave < 2 ? 2 : 1;
    f32x4 CB[2], E[2], DX[2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
        CB[k] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (k >= ntile) continue;
        const int id = wave + 8 * k, tr = tile_row(id), tc = id - tile_id(tr, 0);
#pragma unroll
        for (int ks = 0; ks < NF; ks++)
            CB[k] = M::mma(frag_row<T>(Cs, LN, 16 * tr, 32 * ks), frag_row<T>(Bs, LN, 16 * tc, 32 * ks),
                           CB[k]);
    }
    f32x4 sum[4][NW];                             // dC^T or dB^T: rows n, column = token
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
        for (int j = 0; j < NW; j++) sum[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // tiles right of the diagonal that products read stay zero
    if (wave < 2) {
        const int t = 32 * wave + 4 * g, s = 32 * wave + 16 + li;
#pragma unroll
        for (int i = 0; i < 4; i++) Ms[(t + i) * LX + s] = (T)0.f;
    }

    const int steps = (h1 - h0) * d.nps;
    f32x4 acc[4][NW];
    float gdot = 0.f, ddot = 0.f;
    for (int step = 0; step < steps; step++) {
        const int hn = step / d.nps, h = h0 + hn, ps = step % d.nps, slot = hn % kBatch;
        const int buf = kBufs == 2 ? step & 1 : 0;
        HeadSums &H = hs[slot];
        if (ps == 0) {
            __syncthreads();  // the head before is done with W, and at slot 0 its batch with hs
            if (slot == 0) {
                const int hh = h + (int)(threadIdx.x >> 6), s = threadIdx.x >> 6;
                if (s < kBatch && hh < h1) {
                    const int64_t at = ((b * d.H + hh) * d.nc + c) * Q;
                    const float2 me = cs[at + l];
                    const float dv = delta[at + l], e = decay(cs[at + Q - 1], me);
                    hs[s].cc[l] = me;
                    hs[s].dl[l] = dv;
                    hs[s].et[l] = e;
                    hs[s].wt[l] = e * dv;
                }
                __syncthreads();
            }
#pragma unroll
            for (int k = 0; k < 2; k++) {
                DX[k] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (k >= ntile) continue;
                const int id = wave + 8 * k, tr = tile_row(id), tc = id - tile_id(tr, 0);
                const int s = 16 * tc + li;
                const float2 ccs = H.cc[s];
                const float ds = H.dl[s];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int t = 16 * tr + 4 * g + i;
                    const float e = decay(H.cc[t], ccs);
                    E[k][i] = s <= t ? e : 0.f;
                    Ms[t * LX + s] = (T)(CB[k][i] * E[k][i] * ds);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; r++)
#pragma unroll
                for (int j = 0; j < NW; j++) acc[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            gdot = ddot = 0.f;
        }
        if (kBufs == 1 && step) __syncthreads();
        rx.store(Xs[buf]);
        ry.store(Ys[buf]);
        // the state of the wave's side in three terms, of one half of the columns at a time
        // where N = 128 leaves no registers for both
        Frag sf[kEarly ? 2 : 1][NW][M::kTerms];
        const auto split = [&](int ks, int at) {
#pragma unroll
            for (int j = 0; j < NW; j++) {
                f32x8 v;
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] = sideB ? rG[ks][j][i / 4][i % 4] : rS[ks][j][i / 4][i % 4];
                split_frag<T>(v, sf[at][j]);
            }
        };
        if constexpr (kEarly)
            if (ncols) {
                split(0, 0);
                split(1, 1);
            }
        if (ncols && sideB)
#pragma unroll
            for (int ks = 0; ks < 2; ks++)
#pragma unroll
                for (int j = 0; j < NW; j++) {
#pragma unroll
                    for (int u = 0; u < 2; u++)
#pragma unroll
                        for (int i = 0; i < 4; i++) gdot = fmaf(rS[ks][j][u][i], rG[ks][j][u][i], gdot);
                    if constexpr (kGs)
                        *reinterpret_cast<Frag *>(Gs[buf] + (16 * (nt0 + j) + li) * LX + 32 * ks + 8 * g) =
                            frag_acc<T>(rG[ks][j][0], rG[ks][j][1]);
                }
        __syncthreads();
        if (step + 1 < steps) {
            fetch(step + 1);
            if (kEarly) fetch_states(step + 1);
        }
        // dy.x for the wave's tiles
#pragma unroll
        for (int k = 0; k < 2; k++) {
            if (k >= ntile) continue;
            const int id = wave + 8 * k, tr = tile_row(id), tc = id - tile_id(tr, 0);
#pragma unroll
            for (int ks = 0; ks < 2; ks++)
                DX[k] = M::mma(frag_row<T>(Ys[buf], LX, 16 * tr, 32 * ks),
                               frag_row<T>(Xs[buf], LX, 16 * tc, 32 * ks), DX[k]);
        }
        // S^T dy or G^T x, transposed: rows n, column = token
        if (ncols) {
            const T *src = sideB ? Xs[buf] : Ys[buf];
#pragma unroll
            for (int ks = 0; ks < 2; ks++) {
                if constexpr (!kEarly) split(ks, 0);
                Frag a[4];
#pragma unroll
                for (int r = 0; r < 4; r++) a[r] = frag_row<T>(src, LX, 16 * r, 32 * ks);
#pragma unroll
                for (int m = 0; m < M::kTerms; m++)
#pragma unroll
                    for (int j = 0; j < NW; j++)
#pragma unroll
                        for (int r = 0; r < 4; r++)
                            acc[r][j] = M::mma(sf[kEarly ? ks : 0][j][m], a[r], acc[r][j]);
            }
        }
        if (!kEarly && step + 1 < steps) fetch_states(step + 1);
        // dx^T: 16 columns (rows here) and half of the tokens
        {
            Frag gn[NF], yc[2];
            const float *Gh = Gws + (((b * d.H + h) * d.nc + c) * d.nps + ps) * kTile +
                              each_at(g >> 1, w, 0) + 32 * (g & 1) + li;
#pragma unroll
            for (int kk = 0; kk < NF; kk++) {
                if constexpr (kGs) {
                    gn[kk] = frag_col<T>(Gs[buf], LX, 32 * kk, 16 * w);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++) gn[kk][i] = Gh[each_at(2 * kk, 0, i & 3) + 16 * (i >> 2)];
                }
            }
#pragma unroll
            for (int ks = 0; ks < 2; ks++) yc[ks] = frag_col<T>(Ys[buf], LX, 32 * ks, 16 * w);
            const int p = ps * kSlice + 16 * w + 4 * g;
#pragma unroll
            for (int q = 0; q < 2; q++) {
                const int r = sideB ? 2 + q : q, s = 16 * r + li;
                f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk < NF; kk++)
                    o = M::mma(gn[kk], frag_row<T>(Bs, LN, 16 * r, 32 * kk), o);
                o *= H.wt[s];
#pragma unroll
                for (int ks = 0; ks < 2; ks++)
                    if (ks || !sideB) o = M::mma(yc[ks], frag_col<T>(Ms, LX, 32 * ks, 16 * r), o);
                const f32x4 gy = __builtin_convertvector(
                    *reinterpret_cast<const Half *>(Ys[buf] + s * LX + 16 * w + 4 * g), f32x4);
                const f32x4 xv = __builtin_convertvector(
                    *reinterpret_cast<const Half *>(Xs[buf] + s * LX + 16 * w + 4 * g), f32x4);
#pragma unroll
                for (int i = 0; i < 4; i++) ddot = fmaf(gy[i], xv[i], ddot);
                o += gy * (D ? D[h] : 0.f);
                if (s >= rows) o = f32x4{0.f, 0.f, 0.f, 0.f};
                if (t0 + s < d.T)
                    store4<T, VEC>(dx + ((b * d.T + t0 + s) * d.H + h) * d.P, p, d.P, o);
            }
        }
        if (ps + 1 < d.nps) continue;

        // the head's last slice: W, and the sums that its token gradients are made of
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; k++) {
            if (k >= ntile) continue;
            const int id = wave + 8 * k, tr = tile_row(id), tc = id - tile_id(tr, 0);
            const int s = 16 * tc + li;
            const float ds = H.dl[s];
            float cE = 0.f, cS = 0.f, whole = 0.f;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int t = 16 * tr + 4 * g + i;
                const float wv = DX[k][i] * E[k][i];
                const float e = wv * CB[k][i];
                Ms[t * LX + s] = (T)(wv * ds);    // rounded for the products with B and C
                cE += e;
                float q = e * ds;                 // prefix over the tile's 16 columns
                q += row_shr<1>(q);
                q += row_shr<2>(q);
                q += row_shr<4>(q);
                q += row_shr<8>(q);
                cS += s <= t ? row_shr<1>(q) : 0.f;
                if (li == 15) H.rows[t][tc] = q;
                whole += q;
            }
            cE = xor_add(xor_add(cE, 16), 32);
            cS = xor_add(xor_add(cS, 16), 32);
            whole = xor_add(xor_add(whole, 16), 32);
            if (g == 0) {
                H.colE[id][li] = cE;
                H.cross[id][li] = cS;
                if (li == 15) H.all[id] = whole;
            }
        }
        if (ncols) {
            const T *own = sideB ? Bs : Cs;
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int t = 16 * r + li;
                const float2 ct = H.cc[t];
                const float f = sideB ? H.wt[t] : exp2_fast(ct.x + ct.y);
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < NW; j++) {
                    const f32x4 v = __builtin_convertvector(
                        *reinterpret_cast<const Half *>(own + t * LN + 16 * (nt0 + j) + 4 * g), f32x4);
#pragma unroll
                    for (int i = 0; i < 4; i++) dot = fmaf(acc[r][j][i], v[i], dot);
                    sum[r][j] += acc[r][j] * f;
                }
                dot = xor_add(xor_add(dot, 16), 32);
                if (g == 0) (sideB ? H.dotB : H.dotC)[w][t] = dot;
            }
        } else if (g == 0) {
#pragma unroll
            for (int r = 0; r < 4; r++) (sideB ? H.dotB : H.dotC)[w][16 * r + li] = 0.f;
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            gdot = xor_add(gdot, m);
            ddot = xor_add(ddot, m);
        }
        if (l == 0) {
            if (sideB) H.gs[w] = gdot;
            H.dd[wave] = ddot;
        }
        __syncthreads();
        if (ncols) {
            const T *other = sideB ? Cs : Bs;
#pragma unroll
            for (int j = 0; j < NW; j++)
#pragma unroll
                for (int ks = 0; ks < 2; ks++) {
                    const Frag f = frag_col<T>(other, LN, 32 * ks, 16 * (nt0 + j));
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        if (!sideB && ks <= r / 2)
                            sum[r][j] = M::mma(f, frag_row<T>(Ms, LX, 16 * r, 32 * ks), sum[r][j]);
                        if (sideB && ks >= r / 2)
                            sum[r][j] = M::mma(f, frag_col<T>(Ms, LX, 32 * ks, 16 * r), sum[r][j]);
                    }
                }
        }
        if (slot + 1 < kBatch && h + 1 < h1) continue;

        // token gradients of the batch: a wave per head, lane = token
        if (wave <= slot) {
            const HeadSums &K = hs[wave];
            const int hh = h - slot + wave, k = l >> 4;
            const float2 tot = K.cc[Q - 1], me = K.cc[l];
            const float dC_ = (K.dotC[0][l] + K.dotC[1][l]) + (K.dotC[2][l] + K.dotC[3][l]);
            const float dB_ = (K.dotB[0][l] + K.dotB[1][l]) + (K.dotB[2][l] + K.dotB[3][l]);
            float ce = 0.f, cross = 0.f, left = 0.f;
#pragma unroll
            for (int r = 0; r < 4; r++)
                if (r >= k) {
                    ce += K.colE[tile_id(r, k)][li];
                    cross += K.cross[tile_id(r, k)][li];
                }
            // sources in tiles left of the token's: rows from it on in its own row of tiles ...
#pragma unroll
            for (int q = 0; q < 3; q++)
                if (q < k) left += K.rows[l][q];
            left += row_shl<1>(left);
            left += row_shl<2>(left);
            left += row_shl<4>(left);
            left += row_shl<8>(left);
            cross += left;
            // ... and whole tiles under that
#pragma unroll
            for (int r = 0; r < 4; r++)
#pragma unroll
                for (int q = 0; q < 3; q++)
                    if (r > k && q < k) cross += K.all[tile_id(r, q)];
            float suf = exp2_fast(me.x + me.y) * dC_;
            float pre = K.wt[l] * dB_;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const float a = __shfl_down(suf, m), q = __shfl_up(pre, m);
                if (l + m < 64) suf += a;
                if (l >= m) pre += q;
            }
            const float up = __shfl_up(pre, 1), before = l ? up : 0.f;
            const float pass = exp2_fast(tot.x + tot.y) * ((K.gs[0] + K.gs[1]) + (K.gs[2] + K.gs[3]));
            const float dv = K.dl[l];
            const float dlr = l < rows ? (cross + suf) + (before + pass) : 0.f;
            float dz = l < rows ? fmaf(A[hh], dlr, fmaf(K.et[l], dB_, ce)) : 0.f;
            if (softplus) dz *= -expm1f(-dv);
            if (t0 + l < d.T) ddt[(b * d.T + t0 + l) * d.H + hh] = (T)dz;
            float pa = dv * dlr, pb = dz;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                pa = xor_add(pa, m);
                pb = xor_add(pb, m);
            }
            if (l == 0) {
                float *q = parts + ((b * d.nc + c) * d.H + hh) * 3;
                q[0] = pa;
                q[1] = ((K.dd[0] + K.dd[1]) + (K.dd[2] + K.dd[3])) + ((K.dd[4] + K.dd[5]) + (K.dd[6] + K.dd[7]));
                q[2] = pb;
            }
        }
    }
    if (!ncols) return;
#pragma unroll
    for (int r = 0; r < 4; r++) {
        const int t = 16 * r + li;
        if (t0 + t >= d.T) continue;
        const int64_t at = ((b * d.T + t0 + t) * d.G + grp) * d.N;
#pragma unroll
        for (int j = 0; j < NW; j++) {
            const f32x4 v = t < rows ? sum[r][j] : f32x4{0.f, 0.f, 0.f, 0.f};
            const int n = 16 * (nt0 + j) + 4 * g;
            if (hblocks == 1)
                store4<T, VEC>((sideB ? dB : dC) + at, n, d.N, v);
            else
                store4<float, VEC>(hsum + (2 * hb + sideB) * ((int64_t)d.B * d.T * d.G * d.N) + at, n, d.N, v);
        }
    }
}

// dC and dB from the sums of the blocks of heads.
template <typename T>
__global__ __launch_bounds__(kThreads) void scan_heads_kernel(int64_t all, int hblocks,
                                                              const float *__restrict__ hsum,
                                                              T *__restrict__ dB, T *__restrict__ dC)
{
    const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (e >= all) return;
    float c = 0.f, b = 0.f;
    for (int k = 0; k < hblocks; k++) {
        c += hsum[(2 * k) * all + e];
        b += hsum[(2 * k + 1) * all + e];
    }
    dC[e] = (T)c;
    dB[e] = (T)b;
}

// dA, dD and ddt_bias of a head: the sum over sequences and chunks.
__global__ __launch_bounds__(kThreads) void scan_params_kernel(int64_t rows, int H,
                                                               const float *__restrict__ parts,
                                                               float *dA, float *dD, float *dbias)
{
    __shared__ double sums[kThreads];
    const int h = blockIdx.x, which = blockIdx.y;
    float *out = which == 0 ? dA : which == 1 ? dD : dbias;
    if (!out) return;
    double s = 0.0;
    for (int64_t r = threadIdx.x; r < rows; r += kThreads) s += (double)parts[(r * H + h) * 3 + which];
    sums[threadIdx.x] = s;
    for (int n = kThreads / 2; n > 0; n >>= 1) {
        __syncthreads();
        if ((int)threadIdx.x < n) sums[threadIdx.x] += sums[threadIdx.x + n];
    }
    if (threadIdx.x == 0) out[h] = (float)sums[0];
}

// ------------------------------------------------------------ single tokens
// One token: the state is read, updated and written once, which is all that
// counts (P N floats each way a head).  LN lanes share a row of the state, four
// columns each; a workgroup takes 32 rows.  32 streams, 16 heads of 128 x 64:
// 10 us, 3.4 TB/s.
constexpr int kStepRows = 32;

template <typename T, int LN, bool VEC>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(
    ScanDims d, const T *__restrict__ x, const T *__restrict__ dt, const T *__restrict__ Bm,
    const T *__restrict__ Cm, const float *__restrict__ A, const float *__restrict__ D,
    const float *__restrict__ bias, const int32_t *__restrict__ lengths, int softplus, int cont,
    float *__restrict__ state, T *__restrict__ y)
{
    constexpr int PASS = kThreads / LN;   // rows at a time
    constexpr int NP = kStepRows > PASS ? kStepRows / PASS : 1;
    const int nrb = (d.P + kStepRows - 1) / kStepRows;
    const int rb = blockIdx.x % nrb;
    const int64_t bh = blockIdx.x / nrb;
    const int h = (int)(bh % d.H), grp = h / (d.H / d.G);
    const int64_t b = bh / d.H;
    const bool on = seq_len(lengths, b, 1) > 0;
    const int n = (threadIdx.x % LN) * 4, r = threadIdx.x / LN;
    float *sp = state + bh * (int64_t)d.P * d.N + n;
    f32x4 S[NP];
    float xv[NP];
    T xr[NP];
    // all loads first
#pragma unroll
    for (int u = 0; u < NP; u++) {
        const int p = rb * kStepRows + u * PASS + r;
        S[u] = f32x4{0.f, 0.f, 0.f, 0.f};
        xr[u] = (T)0.f;
        if (p >= d.P || (NP == 1 && r >= kStepRows)) continue;
        if (cont) {
            if constexpr (VEC) {
                if (n < d.N) S[u] = *reinterpret_cast<const f32x4 *>(sp + (int64_t)p * d.N);
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (n + i < d.N) S[u][i] = sp[(int64_t)p * d.N + i];
            }
        }
        if (on) xr[u] = x[b * d.xb + (int64_t)h * d.P + p];
    }
    f32x4 Bv = {0.f, 0.f, 0.f, 0.f}, Cv = Bv;
    float delta = 0.f;
    if (on) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (n + i < d.N) {
                Bv[i] = (float)Bm[b * d.bb + (int64_t)grp * d.N + n + i];
                Cv[i] = (float)Cm[b * d.cb + (int64_t)grp * d.N + n + i];
            }
        delta = (float)dt[b * d.H + h] + (bias ? bias[h] : 0.f);
        if (softplus) delta = delta > 20.f ? delta : log1pf(expf(delta));
    }
    const float a = expf(delta * A[h]), Dh = D ? D[h] : 0.f;
#pragma unroll
    for (int u = 0; u < NP; u++) {
        const int p = rb * kStepRows + u * PASS + r;
        if (p >= d.P || (NP == 1 && r >= kStepRows)) continue;
        xv[u] = (float)xr[u];
        if (on) S[u] = S[u] * a + Bv * (delta * xv[u]);
        float s = fmaf(S[u][0], Cv[0], S[u][1] * Cv[1]) + fmaf(S[u][2], Cv[2], S[u][3] * Cv[3]);
#pragma unroll
        for (int m = 1; m < LN; m <<= 1) s = xor_add(s, m);
        if constexpr (VEC) {
            if (n < d.N) *reinterpret_cast<f32x4 *>(sp + (int64_t)p * d.N) = S[u];
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (n + i < d.N) sp[(int64_t)p * d.N + i] = S[u][i];
        }
        if (n == 0) y[bh * d.P + p] = (T)(on ? fmaf(Dh, xv[u], s) : 0.f);
    }
}

// -------------------------------------------------------------------- host

struct Plan {
    ScanDims d;
    int hblocks;
    size_t delta, cs, own[2], start[2], S, G, parts, hsum, total;
};

constexpr int64_t kFill = 256;   // compute units

Plan plan_of(const sdm_scan_desc &s, bool backward)
{
    Plan p = {};
    ScanDims &d = p.d;
    d.B = s.B;
    d.H = s.H;
    d.P = s.P;
    d.N = s.N;
    d.G = s.G;
    d.T = s.T;
    d.nc = (int)((s.T + Q - 1) / Q);
    d.nps = (s.P + kSlice - 1) / kSlice;
    // Few chains: the time axis is split into segments, enough for a workgroup on
    // every compute unit, which first run for their states alone.  A segment is at
    // least two chunks, or eight in the backward, whose two walks share a launch
    // and take no longer steps (5 x 777 tokens, 6 heads, float32: forward 67 us in
    // one segment and 38 in six; backward 71 and 85).
    const int64_t units = (int64_t)s.B * s.H * d.nps, least = backward ? 8 : 2;
    int64_t seg = (kFill + units - 1) / units;
    if (seg > d.nc / least) seg = d.nc / least;
    if (seg < 1) seg = 1;
    d.cps = (int)((d.nc + seg - 1) / seg);
    d.nseg = (d.nc + d.cps - 1) / d.cps;
    d.xb = s.x_batch;
    d.xt = s.x_token;
    d.bb = s.B_batch;
    d.bt = s.B_token;
    d.cb = s.C_batch;
    d.ct = s.C_token;
    // Blocks of a group's heads: the number with the fewest rounds of workgroups
    // (one a compute unit) times heads of a workgroup, counting its tiles of B and
    // C and its last stores as one head more; the fewest blocks of those.
    const int64_t grads = (int64_t)s.B * d.nc * s.G, per = s.H / s.G;
    int64_t best = 0;
    for (int64_t hb = 1; hb <= per && hb <= kFill; hb++) {
        const int64_t cost = (grads * hb + kFill - 1) / kFill * ((per + hb - 1) / hb + 1);
        if (hb == 1 || cost < best) {
            best = cost;
            p.hblocks = (int)hb;
        }
    }

    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) & ~(size_t)255;
        return here;
    };
    const size_t bh = (size_t)s.B * s.H, PN = (size_t)s.P * s.N;
    p.delta = take(bh * d.nc * Q * 4);
    p.cs = take(bh * d.nc * Q * 8);
    if (d.nseg > 1) {
        for (int k = 0; k < (backward ? 2 : 1); k++) {
            p.own[k] = take(bh * d.nseg * PN * 4);
            p.start[k] = take(bh * d.nseg * PN * 4);
        }
    }
    if (backward) {
        const size_t tile = (size_t)(s.N <= 32 ? 32 : s.N <= 64 ? 64 : 128) * kSlice * 4;
        p.S = take(bh * d.nc * d.nps * tile);
        p.G = take(bh * d.nc * d.nps * tile);
        p.parts = take((size_t)s.B * d.nc * s.H * 3 * 4);
        if (p.hblocks > 1) p.hsum = take((size_t)p.hblocks * 2 * s.B * s.T * s.G * s.N * 4);
    }
    p.total = at;
    return p;
}

template <typename T>
void run_prep(const ScanArgs &a, const Plan &p, float *delta, float2 *cs, hipStream_t stream)
{
    const int64_t waves = (int64_t)p.d.B * p.d.nc * p.d.H;
    scan_prep_kernel<T><<<(unsigned)((waves + 3) / 4), dim3(64, 4), 0, stream>>>(
        p.d, (const T *)a.dt, a.A, a.dt_bias, a.lengths, a.d.softplus, delta, cs);
}

// The walks of `jobs` over whole sequences.  With more than one segment each
// segment first runs from zero, for the state before every one (in `start`).
template <typename T, int NT, bool VEC>
void run_segments(const ScanArgs &a, const Plan &p, StateJob<T> *jobs, int njobs, const float *delta,
                  const float2 *cs, hipStream_t stream)
{
    const ScanDims &d = p.d;
    if (d.nseg == 1) return;
    const dim3 grid((unsigned)((int64_t)d.B * d.H * d.nps * d.nseg), njobs);
    StateJob<T> own[2];
    for (int k = 0; k < njobs; k++) {
        own[k] = jobs[k];
        own[k].init = nullptr;
        own[k].each = nullptr;
        own[k].end = (float *)(a.ws + p.own[k]);
        own[k].end_api = 0;
    }
    scan_state_kernel<T, NT, VEC, false><<<grid, 2 * kThreads, 0, stream>>>(d, delta, cs, a.lengths, own[0],
                                                                    own[njobs - 1]);
    for (int k = 0; k < njobs; k++) {
        float *start = (float *)(a.ws + p.start[k]);
        scan_join_kernel<<<dim3((d.P * d.N + kThreads - 1) / kThreads, d.B * d.H), kThreads, 0, stream>>>(
            d, cs, jobs[k].rev, jobs[k].init, own[k].end, start);
        jobs[k].init = start;
        jobs[k].init_api = 0;
    }
}

template <typename T, int NT, bool VEC>
hipError_t forward(const ScanArgs &a, hipStream_t stream)
{
    const Plan p = plan_of(a.d, false);
    const ScanDims &d = p.d;
    float *delta = (float *)(a.ws + p.delta);
    float2 *cs = (float2 *)(a.ws + p.cs);
    run_prep<T>(a, p, delta, cs, stream);
    const T *x = (const T *)a.x, *Bm = (const T *)a.Bm, *Cm = (const T *)a.Cm;
    StateJob<T> job = {x, Bm, d.xb, d.xt, d.bb, d.bt, a.cont ? a.state : nullptr, nullptr, nullptr, 0, 1, 0};
    run_segments<T, NT, VEC>(a, p, &job, 1, delta, cs, stream);
    scan_walk_kernel<T, NT, VEC>
        <<<(unsigned)((int64_t)d.B * d.H * d.nps * d.nseg), 2 * kThreads, 0, stream>>>(
            d, x, Bm, Cm, a.D, delta, cs, a.lengths, job.init, job.init_api, a.state, (T *)a.y);
    return hipGetLastError();
}

template <typename T, int NT, bool VEC>
hipError_t backward(const ScanArgs &a, hipStream_t stream)
{
    const Plan p = plan_of(a.d, true);
    const ScanDims &d = p.d;
    float *delta = (float *)(a.ws + p.delta);
    float2 *cs = (float2 *)(a.ws + p.cs);
    float *S = (float *)(a.ws + p.S), *G = (float *)(a.ws + p.G);
    float *parts = (float *)(a.ws + p.parts), *hsum = (float *)(a.ws + p.hsum);
    const T *x = (const T *)a.x, *Bm = (const T *)a.Bm, *Cm = (const T *)a.Cm, *dy = (const T *)a.dy;
    const int64_t yt = (int64_t)d.H * d.P, yb = d.T * yt;
    run_prep<T>(a, p, delta, cs, stream);
    StateJob<T> jobs[2] = {{x, Bm, d.xb, d.xt, d.bb, d.bt, a.state0, S, nullptr, 0, 1, 0},
                           {dy, Cm, yb, yt, d.cb, d.ct, a.dstateT, G, a.dstate0, 1, 1, 1}};
    run_segments<T, NT, VEC>(a, p, jobs, 2, delta, cs, stream);
    scan_state_kernel<T, NT, VEC, true>
        <<<dim3((unsigned)((int64_t)d.B * d.H * d.nps * d.nseg), 2), 2 * kThreads, 0, stream>>>(
            d, delta, cs, a.lengths, jobs[0], jobs[1]);
    scan_grad_kernel<T, NT, VEC>
        <<<(unsigned)((int64_t)d.B * d.nc * d.G * p.hblocks), 2 * kThreads, 0, stream>>>(
            d, p.hblocks, x, dy, Bm, Cm, a.A, a.D, delta, cs, a.lengths, a.d.softplus, S, G, (T *)a.dx,
            (T *)a.ddt, (T *)a.dB, (T *)a.dC, parts, hsum);
    if (p.hblocks > 1) {
        const int64_t all = (int64_t)d.B * d.T * d.G * d.N;
        scan_heads_kernel<T><<<(unsigned)((all + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
            all, p.hblocks, hsum, (T *)a.dB, (T *)a.dC);
    }
    scan_params_kernel<<<dim3(d.H, 3), kThreads, 0, stream>>>((int64_t)d.B * d.nc, d.H, parts, a.dA,
                                                            a.dD, a.ddt_bias);
    return hipGetLastError();
}

template <typename T>
hipError_t step(const ScanArgs &a, hipStream_t stream)
{
    const Plan p = plan_of(a.d, false);
    const ScanDims &d = p.d;
    const unsigned grid = (unsigned)((int64_t)d.B * d.H * ((d.P + kStepRows - 1) / kStepRows));
    const auto run = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, stream>>>(
            d, (const T *)a.x, (const T *)a.dt, (const T *)a.Bm, (const T *)a.Cm, a.A, a.D, a.dt_bias,
            a.lengths, a.d.softplus, a.cont, a.state, (T *)a.y);
    };
    const bool vec = d.N % 4 == 0;  // rows of the state on 16 bytes
    if (d.N <= 32)
        vec ? run(scan_step_kernel<T, 8, true>) : run(scan_step_kernel<T, 8, false>);
    else if (d.N <= 64)
        vec ? run(scan_step_kernel<T, 16, true>) : run(scan_step_kernel<T, 16, false>);
    else
        vec ? run(scan_step_kernel<T, 32, true>) : run(scan_step_kernel<T, 32, false>);
    return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t dispatch_n(const ScanArgs &a, bool back, hipStream_t stream)
{
    // the state's columns, padded to 32, 64 or 128
    if (a.d.N <= 32) return back ? backward<T, 2, VEC>(a, stream) : forward<T, 2, VEC>(a, stream);
    if (a.d.N <= 64) return back ? backward<T, 4, VEC>(a, stream) : forward<T, 4, VEC>(a, stream);
    return back ? backward<T, 8, VEC>(a, stream) : forward<T, 8, VEC>(a, stream);
}

template <typename T>
hipError_t dispatch(const ScanArgs &a, bool back, hipStream_t stream)
{
    const sdm_scan_desc &d = a.d;
    if (!back && d.T == 1) return step<T>(a, stream);
    const bool vec = rows_on_16(a.x, d.x_batch, d.x_token, 0, d.P, sizeof(T)) &&
                     rows_on_16(a.Bm, d.B_batch, d.B_token, 0, d.N, sizeof(T)) &&
                     rows_on_16(a.Cm, d.C_batch, d.C_token, 0, d.N, sizeof(T));
    return vec ? dispatch_n<T, true>(a, back, stream) : dispatch_n<T, false>(a, back, stream);
}

}  // namespace

size_t scan_forward_ws(const sdm_scan_desc &d) { return d.T == 1 ? 0 : plan_of(d, false).total; }
size_t scan_backward_ws(const sdm_scan_desc &d) { return plan_of(d, true).total; }

hipError_t launch_scan_forward(const ScanArgs &a, hipStream_t stream)
{
    return a.d.dtype == SDM_F32 ? dispatch<float>(a, false, stream) : dispatch<bf16>(a, false, stream);
}

hipError_t launch_scan_backward(const ScanArgs &a, hipStream_t stream)
{
    return a.d.dtype == SDM_F32 ? dispatch<float>(a, true, stream) : dispatch<bf16>(a, true, stream);
}

}  // namespace sdm
