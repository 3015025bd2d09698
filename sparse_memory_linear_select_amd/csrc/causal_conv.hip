// Short causal depthwise convolution over the token axis, with an optional
// SiLU, its continuation from the last K - 1 rows, and its backward.
//
// With xe = [K - 1 rows before the sequence, x], per channel:
//   z_t = bias + sum_k w_k xe[t + k],   y_t = z_t  or  z_t / (1 + e^-z_t)
//   dz_t = dy_t  or  dy_t s (1 + z_t (1 - s)),  s = 1 / (1 + e^-z_t)
//   dxe[j] = sum_k w_k dz[j - k],   dw_k = sum_t dz_t xe[t + k],   dbias = sum_t dz_t
//
// Bound by HBM: x is read and y written once (2 K flops an element).  A thread
// owns V neighbouring channels (16 bytes where the layout allows) and a run of
// tokens, and keeps the K-row window in registers, so every row is loaded once
// plus K - 1 rows of overlap per run.  Sums stay in float32; each output is
// rounded once.
#include "mix_internal.h"

#include "mix_device.h"

namespace sdm {
namespace {

constexpr int kLanes = 64;      // channel vectors of a backward workgroup
constexpr int kRuns = 4;        // token runs of a backward workgroup
constexpr int kThreads = 256;
constexpr int kFwdRun = 24;     // tokens of a forward run
constexpr int kAhead = 4;       // rows of a forward run loaded before they are used

struct ConvDims {
    int64_t T;
    int C, silu;
    int64_t xb, xt;             // strides of x, in elements
    int nvec;                   // channel vectors
    int runs;                   // forward: token runs of a sequence
    int cblocks, tblocks, run;  // backward: workgroups along channels and tokens, tokens of a run
};

// 1 / (1 + e^-z) by the hardware's exponential and reciprocal, one unit in the
// last place each (z log2 e is off by |z| 2^-24, where the result is e^z or 1).
__device__ __forceinline__ float sigmoid(float z)
{
    return __builtin_amdgcn_rcpf(1.f + exp2_fast(-1.44269504f * z));
}

// The K taps of V channels, and their bias.
template <int V, int K>
__device__ __forceinline__ void load_taps(const float *__restrict__ weight, const float *__restrict__ bias,
                                          int c, float (&w)[K][V], float (&bs)[V])
{
    const float *p = weight + (int64_t)c * K;
    float flat[V * K];
    if constexpr (V * K % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V * K; i += 4) {
            const Vec<float, 4> q = vload<float, 4>(p + i);
#pragma unroll
            for (int e = 0; e < 4; e++) flat[i + e] = q.e[e];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * K; i++) flat[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < V; i++) {
        bs[i] = bias ? bias[c + i] : 0.f;
#pragma unroll
        for (int k = 0; k < K; k++) w[k][i] = flat[i * K + k];
    }
}

// A thread: V channels and a run of 24 tokens.  Rows are loaded four at a
// time and without a branch (rows behind the sequence stand for its last one),
// so that they are in flight together.  8 x 4096 tokens of 2176 bfloat16
// channels: 67 us, 4.2 TB/s (eight rows at a time 83 us, sixteen 108; runs of 16
// tokens 72, of 64 97).
template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(
    ConvDims d, int64_t total, const T *__restrict__ x, const float *__restrict__ weight,
    const float *__restrict__ bias, const int32_t *__restrict__ lengths, int cont, T *state,
    T *__restrict__ y)
{
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (id >= total) return;
    const int c = (int)(id % d.nvec) * V;
    const int64_t rest = id / d.nvec;
    const int64_t b = rest / d.runs, t0 = (rest % d.runs) * kFwdRun;
    const int64_t len = seq_len(lengths, b, d.T);
    const int64_t t1 = t0 + kFwdRun < d.T ? t0 + kFwdRun : d.T;
    const T *xp = x + b * d.xb + c;
    T *yp = y + (b * d.T) * d.C + c;
    const int64_t last = len > 0 ? len - 1 : 0;

    float w[K][V], bs[V];
    load_taps<V, K>(weight, bias, c, w, bs);
    // win: the K - 1 rows before the run
    Vec<T, V> win[K - 1];
#pragma unroll
    for (int k = 0; k < K - 1; k++) {
        const int64_t r = t0 - (K - 1) + k;
        if (r >= 0 && r < len) {
            win[k] = vload<T, V>(xp + r * d.xt);
        } else if (t0 == 0 && cont) {
            win[k] = vload<T, V>(state + (b * (K - 1) + k) * d.C + c);
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) win[k].e[i] = (T)0.f;
        }
    }
    // The run at token 0 is the only reader of the old state, so it also
    // writes the new one: row r is xe[len + r], an old row where len is short.
    if (t0 == 0) {
        for (int r = 0; r < K - 1; r++) {
            const int64_t e = len + r;
            Vec<T, V> row;
            if (e >= K - 1) {
                row = vload<T, V>(xp + (e - (K - 1)) * d.xt);
            } else {
                row = win[0];
#pragma unroll
                for (int k = 1; k < K - 1; k++)
                    if (e == k) row = win[k];
            }
            vstore<T, V>(state + (b * (K - 1) + r) * d.C + c, row);
        }
    }

    for (int64_t t = t0; t < t1; t += kAhead) {
        Vec<T, V> nx[kAhead];
        if (len > 0) {
#pragma unroll
            for (int u = 0; u < kAhead; u++)
                nx[u] = vload<T, V>(xp + (t + u < last ? t + u : last) * d.xt);
        }
#pragma unroll
        for (int u = 0; u < kAhead; u++) {
            if (t + u >= t1) break;
            Vec<T, V> out;
#pragma unroll
            for (int i = 0; i < V; i++) {
                float z = bs[i];
#pragma unroll
                for (int k = 0; k < K - 1; k++) z = fmaf(w[k][i], (float)win[k].e[i], z);
                z = fmaf(w[K - 1][i], (float)nx[u].e[i], z);
                out.e[i] = (T)(t + u < len ? d.silu ? z * sigmoid(z) : z : 0.f);
            }
#pragma unroll
            for (int k = 0; k + 1 < K - 1; k++) win[k] = win[k + 1];
            win[K - 2] = nx[u];
            vstore<T, V>(yp + (t + u) * d.C, out);
        }
    }
}

// One workgroup: 64 channel vectors x 4 runs of tokens.  A run at token t0
// computes dz for its tokens and the K - 1 after them, and writes dx of its
// own tokens; the sums for dweight and dbias are joined over the four runs in
// LDS and written as one row of `partial` per workgroup, which
// conv_reduce_kernel adds in a fixed order.  Four tokens are loaded at a time:
// 8 x 4096 x 2176 bfloat16 take 181 us, 2.4 TB/s, bound by the window, gradients
// and sums that each channel keeps in registers (two at a time 194 us, eight
// 243; 5 x 1021 x 1090 float32 19.4 us, 3.4 TB/s).
template <typename T, int V, int K>
__global__ __launch_bounds__(kLanes *kRuns) void conv_bwd_kernel(
    ConvDims d, const T *__restrict__ x, const T *__restrict__ dy,
    const float *__restrict__ weight, const float *__restrict__ bias,
    const int32_t *__restrict__ lengths, const T *__restrict__ state0,
    const T *__restrict__ dstateT, T *__restrict__ dx, T *__restrict__ dstate0,
    float *__restrict__ partial)
{
    constexpr int kGroup = 4;   // tokens loaded before they are used
    __shared__ float sums[kRuns - 1][kLanes * V];
    const int cb = blockIdx.x % d.cblocks;
    const int64_t rest = blockIdx.x / d.cblocks;
    const int tb = (int)(rest % d.tblocks);
    const int64_t b = rest / d.tblocks;
    const int c = (cb * kLanes + (int)threadIdx.x) * V;
    const int64_t t0 = ((int64_t)tb * kRuns + threadIdx.y) * d.run;
    const bool live = c < d.C && t0 < d.T;

    float acc[K + 1][V];  // dw_0 .. dw_{K-1}, dbias
#pragma unroll
    for (int k = 0; k <= K; k++)
#pragma unroll
        for (int i = 0; i < V; i++) acc[k][i] = 0.f;

    if (live) {
        const int64_t len = seq_len(lengths, b, d.T);
        const int64_t t1 = t0 + d.run < d.T ? t0 + d.run : d.T;
        const int64_t last = len > 0 ? len - 1 : 0;
        const T *xp = x + b * d.xb + c;
        const T *gp = dy + (b * d.T) * d.C + c;
        T *op = dx + (b * d.T) * d.C + c;
        float w[K][V], bs[V];
        load_taps<V, K>(weight, bias, c, w, bs);
        float win[K][V];  // xe[t .. t + K - 1]
        float dz[K][V];   // dz[t - K + 1 .. t]
#pragma unroll
        for (int k = 0; k < K; k++)
#pragma unroll
            for (int i = 0; i < V; i++) win[k][i] = dz[k][i] = 0.f;
#pragma unroll
        for (int k = 0; k < K - 1; k++) {
            const int64_t r = t0 - (K - 1) + k;
            Vec<T, V> v;
            if (r >= 0 && r < len)
                v = vload<T, V>(xp + r * d.xt);
            else if (t0 == 0 && state0)
                v = vload<T, V>(state0 + (b * (K - 1) + k) * d.C + c);
            else
                continue;
#pragma unroll
            for (int i = 0; i < V; i++) win[k + 1][i] = (float)v.e[i];
        }
        for (int64_t tg = t0; tg < t1 + K - 1; tg += kGroup) {
            Vec<T, V> xv[kGroup], gv[kGroup];
            if (len > 0) {
#pragma unroll
                for (int u = 0; u < kGroup; u++) {
                    const int64_t r = tg + u < last ? tg + u : last;
                    xv[u] = vload<T, V>(xp + r * d.xt);
                    gv[u] = vload<T, V>(gp + r * d.C);
                }
            }
#pragma unroll
            for (int u = 0; u < kGroup; u++) {
                const int64_t t = tg + u;
                if (t >= t1 + K - 1) break;
                const bool in = t < len, mine = t < t1;
#pragma unroll
                for (int i = 0; i < V; i++) {
#pragma unroll
                    for (int k = 0; k + 1 < K; k++) {
                        dz[k][i] = dz[k + 1][i];
                        win[k][i] = win[k + 1][i];
                    }
                    win[K - 1][i] = (float)xv[u].e[i];
                    float g = (float)gv[u].e[i];
                    if (d.silu) {
                        float z = bs[i];
#pragma unroll
                        for (int k = 0; k < K; k++) z = fmaf(w[k][i], win[k][i], z);
                        const float s = sigmoid(z);
                        g *= s * fmaf(z, 1.f - s, 1.f);
                    }
                    g = in ? g : 0.f;
                    dz[K - 1][i] = g;
                    const float own = mine ? g : 0.f;
#pragma unroll
                    for (int k = 0; k < K; k++) acc[k][i] = fmaf(own, in ? win[k][i] : 0.f, acc[k][i]);
                    acc[K][i] += own;
                }
                // dxe[t] is complete: row t - (K - 1) of x, or row t of the old state
                const int64_t r = t - (K - 1);
                if (r < t0 && !(t0 == 0 && r < 0 && dstate0)) continue;
                Vec<T, V> out;
#pragma unroll
                for (int i = 0; i < V; i++) {
                    float s = 0.f;
                    // dz[K - 1 - k] is dz_{t - k}
#pragma unroll
                    for (int k = 0; k < K; k++) s = fmaf(w[k][i], dz[K - 1 - k][i], s);
                    if (dstateT && t >= len && t - len < K - 1)
                        s += (float)dstateT[(b * (K - 1) + (t - len)) * d.C + c + i];
                    out.e[i] = (T)s;
                }
                if (r >= 0)
                    vstore<T, V>(op + r * d.C, out);
                else
                    vstore<T, V>(dstate0 + (b * (K - 1) + t) * d.C + c, out);
            }
        }
    }
    float *row = partial + (rest * (K + 1)) * d.C;
#pragma unroll
    for (int k = 0; k <= K; k++) {
        __syncthreads();
        if (threadIdx.y > 0)
#pragma unroll
            for (int i = 0; i < V; i++) sums[threadIdx.y - 1][threadIdx.x * V + i] = acc[k][i];
        __syncthreads();
        if (threadIdx.y == 0 && c < d.C)
#pragma unroll
            for (int i = 0; i < V; i++) {
                float s = acc[k][i];
#pragma unroll
                for (int r = 0; r < kRuns - 1; r++) s += sums[r][threadIdx.x * V + i];
                row[(int64_t)k * d.C + c + i] = s;
            }
    }
}

// dweight[c][k] and dbias[c]: the sum of `rows` partial rows, in a fixed
// order: 16 strided sums of a column, joined pairwise.
__global__ __launch_bounds__(1024) void conv_reduce_kernel(const float *__restrict__ partial,
                                                           int64_t rows, int K, int C,
                                                           float *__restrict__ dweight,
                                                           float *__restrict__ dbias)
{
    __shared__ float sums[16][64];
    const int c = blockIdx.x * 64 + threadIdx.x;
    const int k = blockIdx.y;
    float s = 0.f;
    if (c < C)
        for (int64_t r = threadIdx.y; r < rows; r += 16)
            s += partial[(r * (K + 1) + k) * C + c];
    sums[threadIdx.y][threadIdx.x] = s;
    for (int n = 8; n > 0; n >>= 1) {
        __syncthreads();
        if ((int)threadIdx.y < n) sums[threadIdx.y][threadIdx.x] += sums[threadIdx.y + n][threadIdx.x];
    }
    if (threadIdx.y == 0 && c < C) {
        if (k < K)
            dweight[(int64_t)c * K + k] = sums[0][threadIdx.x];
        else if (dbias)
            dbias[c] = sums[0][threadIdx.x];
    }
}

ConvDims dims_of(const sdm_conv_desc &d, int V)
{
    ConvDims m;
    m.T = d.T;
    m.C = d.C;
    m.silu = d.silu;
    m.xb = d.x_batch;
    m.xt = d.x_token;
    m.nvec = (d.C + V - 1) / V;
    m.runs = (int)((d.T + kFwdRun - 1) / kFwdRun);
    m.cblocks = (m.nvec + kLanes - 1) / kLanes;
    // Backward runs of 32 tokens; of 16 where the workgroups would not fill the
    // 256 compute units four times (shorter runs overlap more and leave more sums).
    m.run = (int64_t)d.B * m.cblocks * ((d.T + 127) / 128) >= 1024 ? 32 : 16;
    m.tblocks = (int)((d.T + kRuns * m.run - 1) / (kRuns * m.run));
    return m;
}

bool aligned_to(const void *p, size_t n) { return ((uintptr_t)p % n) == 0; }

// Channels per thread: as many as one 16-byte access holds where every row of
// every tensor starts on such a boundary, half or a quarter of that for rows
// that start on 8 or 4 bytes, else one.
int vector_width(const ConvArgs &a, int esize)
{
    for (int v = 16 / esize; v > 1; v >>= 1) {
        const size_t bytes = (size_t)v * esize;
        if (a.d.C % v == 0 && a.d.x_batch % v == 0 && a.d.x_token % v == 0 &&
            aligned_to(a.x, bytes))
            return v;
    }
    return 1;
}

template <typename T, int V, int K>
hipError_t run_conv(const ConvArgs &a, bool backward, hipStream_t stream)
{
    const ConvDims m = dims_of(a.d, V);
    if (!backward) {
        const int64_t total = (int64_t)m.nvec * m.runs * a.d.B;
        conv_fwd_kernel<T, V, K><<<(unsigned)((total + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
            m, total, (const T *)a.x, a.weight, a.bias, a.lengths, a.cont, (T *)a.state, (T *)a.y);
    } else {
        const dim3 grid((unsigned)((int64_t)m.cblocks * m.tblocks * a.d.B)), block(kLanes, kRuns);
        conv_bwd_kernel<T, V, K><<<grid, block, 0, stream>>>(
            m, (const T *)a.x, (const T *)a.dy, a.weight, a.bias, a.lengths, (const T *)a.state0,
            (const T *)a.dstateT, (T *)a.dx, (T *)a.dstate0, a.partial);
        conv_reduce_kernel<<<dim3((a.d.C + 63) / 64, K + 1), dim3(64, 16), 0, stream>>>(
            a.partial, (int64_t)m.tblocks * a.d.B, K, a.d.C, a.dweight, a.dbias);
    }
    return hipGetLastError();
}

template <typename T, int V>
hipError_t run_conv_k(const ConvArgs &a, bool backward, hipStream_t stream)
{
    switch (a.d.K) {
    case 2: return run_conv<T, V, 2>(a, backward, stream);
    case 3: return run_conv<T, V, 3>(a, backward, stream);
    case 4: return run_conv<T, V, 4>(a, backward, stream);
    case 5: return run_conv<T, V, 5>(a, backward, stream);
    case 6: return run_conv<T, V, 6>(a, backward, stream);
    case 7: return run_conv<T, V, 7>(a, backward, stream);
    default: return run_conv<T, V, 8>(a, backward, stream);
    }
}

hipError_t dispatch_conv(const ConvArgs &a, bool backward, hipStream_t stream)
{
    if (a.d.dtype == SDM_F32) {
        switch (vector_width(a, 4)) {
        case 4: return run_conv_k<float, 4>(a, backward, stream);
        case 2: return run_conv_k<float, 2>(a, backward, stream);
        default: return run_conv_k<float, 1>(a, backward, stream);
        }
    }
    switch (vector_width(a, 2)) {
    case 8: return run_conv_k<bf16, 8>(a, backward, stream);
    case 4: return run_conv_k<bf16, 4>(a, backward, stream);
    case 2: return run_conv_k<bf16, 2>(a, backward, stream);
    default: return run_conv_k<bf16, 1>(a, backward, stream);
    }
}

}  // namespace

size_t conv_backward_ws(const sdm_conv_desc &d)
{
    // the most rows of sums that any vector width leaves: runs of 16 tokens
    return (size_t)((d.T + 16 * kRuns - 1) / (16 * kRuns)) * d.B * (d.K + 1) * d.C * sizeof(float);
}

hipError_t launch_conv_forward(const ConvArgs &a, hipStream_t stream)
{
    return dispatch_conv(a, false, stream);
}

hipError_t launch_conv_backward(const ConvArgs &a, hipStream_t stream)
{
    return dispatch_conv(a, true, stream);
}

}  // namespace sdm
