// C ABI of the sequence mixers: argument validation and launches.  Every
// check happens before the first HIP call; see include/sdm.h for the contract.
#include "mix_internal.h"

#include <math.h>

namespace {

using sdm::set_error;

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned_el(const void *p, sdm_dtype t) { return ((uintptr_t)p & (t == SDM_F32 ? 3u : 1u)) == 0; }

sdm_status hip_fail(hipError_t e, const char *what)
{
    return set_error(SDM_ERR_HIP, "%s: %s (%s)", what, hipGetErrorName(e), hipGetErrorString(e));
}

// A dense tensor: required (null refused) or optional, 16-byte aligned.
sdm_status check_dense(const void *p, const char *name, bool required = true)
{
    if (!p) return required ? set_error(SDM_ERR_ARG, "null %s", name) : SDM_OK;
    if (!aligned16(p)) return set_error(SDM_ERR_ARG, "%s must be 16-byte aligned", name);
    return SDM_OK;
}

// A strided input: element-aligned.
sdm_status check_strided(const void *p, const char *name, sdm_dtype t)
{
    if (!p) return set_error(SDM_ERR_ARG, "null %s", name);
    if (!aligned_el(p, t)) return set_error(SDM_ERR_ARG, "%s must be aligned to its elements", name);
    return SDM_OK;
}

sdm_status check_lengths(const int32_t *p)
{
    if (p && ((uintptr_t)p & 3u)) return set_error(SDM_ERR_ARG, "lengths must be 4-byte aligned");
    return SDM_OK;
}

sdm_status check_batch(int B, int64_t T, sdm_dtype dtype)
{
    if (B < 1) return set_error(SDM_ERR_ARG, "B must be >= 1 (got %d)", B);
    if (T < 1) return set_error(SDM_ERR_ARG, "T must be >= 1 (got %lld)", (long long)T);
    if (T >= (int64_t)1 << 31)
        return set_error(SDM_ERR_UNSUPPORTED, "T must be < 2^31 (got %lld)", (long long)T);
    if (dtype != SDM_F32 && dtype != SDM_BF16)
        return set_error(SDM_ERR_ARG, "dtype must be SDM_F32 or SDM_BF16 (got %d)", (int)dtype);
    return SDM_OK;
}

// The kernels address the rows of a tile with 31-bit offsets.
sdm_status check_stride(int64_t token)
{
    if (token >= (int64_t)1 << 22)
        return set_error(SDM_ERR_UNSUPPORTED, "token strides must be < 2^22 elements (got %lld)",
                         (long long)token);
    return SDM_OK;
}

sdm_status check_workspace(const void *ws, size_t have, size_t need)
{
    if (need && !ws) return set_error(SDM_ERR_ARG, "null workspace");
    if (!aligned16(ws)) return set_error(SDM_ERR_ARG, "workspace must be 16-byte aligned");
    if (have < need)
        return set_error(SDM_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
    return SDM_OK;
}

#define CHECK(expr)                          \
    do {                                     \
        const sdm_status st_ = (expr);       \
        if (st_ != SDM_OK) return st_;       \
    } while (0)

// ------------------------------------------------------------- convolution

sdm_status check_conv(const sdm_conv_desc *d)
{
    if (!d) return set_error(SDM_ERR_ARG, "null descriptor");
    CHECK(check_batch(d->B, d->T, d->dtype));
    if (d->C < 1 || d->K < 1)
        return set_error(SDM_ERR_ARG, "C and K must be >= 1 (got %d %d)", d->C, d->K);
    if (d->silu != 0 && d->silu != 1)
        return set_error(SDM_ERR_ARG, "silu must be 0 or 1 (got %d)", d->silu);
    if (d->x_batch < 0 || d->x_token < 0)
        return set_error(SDM_ERR_ARG, "strides must be >= 0");
    if (d->K < 2 || d->K > 8)
        return set_error(SDM_ERR_UNSUPPORTED, "2 <= K <= 8 is supported (got %d)", d->K);
    if ((double)d->B * (double)d->T * d->C >= 1099511627776.0)
        return set_error(SDM_ERR_UNSUPPORTED, "B*T*C must be < 2^40");
    // workgroups of the scalar form: one launch holds fewer than 2^31
    if ((double)d->B * (double)((d->T + 63) / 64) * (double)((d->C + 63) / 64) >= 2147483648.0)
        return set_error(SDM_ERR_UNSUPPORTED, "B * ceil(T/64) * ceil(C/64) must be < 2^31");
    return SDM_OK;
}

// -------------------------------------------------------------------- scan

sdm_status check_scan(const sdm_scan_desc *d)
{
    if (!d) return set_error(SDM_ERR_ARG, "null descriptor");
    CHECK(check_batch(d->B, d->T, d->dtype));
    if (d->H < 1 || d->P < 1 || d->N < 1 || d->G < 1)
        return set_error(SDM_ERR_ARG, "H, P, N, G must be >= 1 (got %d %d %d %d)", d->H, d->P, d->N,
                         d->G);
    if (d->H % d->G)
        return set_error(SDM_ERR_ARG, "G = %d must divide H = %d", d->G, d->H);
    if (d->softplus != 0 && d->softplus != 1)
        return set_error(SDM_ERR_ARG, "softplus must be 0 or 1 (got %d)", d->softplus);
    if (d->x_batch < 0 || d->x_token < 0 || d->B_batch < 0 || d->B_token < 0 || d->C_batch < 0 ||
        d->C_token < 0)
        return set_error(SDM_ERR_ARG, "strides must be >= 0");
    if (d->N > 128) return set_error(SDM_ERR_UNSUPPORTED, "N <= 128 is supported (got %d)", d->N);
    CHECK(check_stride(d->x_token));
    CHECK(check_stride(d->B_token));
    CHECK(check_stride(d->C_token));
    if (d->P > 65536) return set_error(SDM_ERR_UNSUPPORTED, "P <= 65536 is supported (got %d)", d->P);
    if ((double)d->B * (double)d->T * d->H >= 2147483648.0)
        return set_error(SDM_ERR_UNSUPPORTED, "B*T*H must be < 2^31");
    if ((double)d->B * d->H * ((d->P + 31) / 32) >= 2147483648.0)
        return set_error(SDM_ERR_UNSUPPORTED, "B*H*ceil(P/32) must be < 2^31");
    if ((double)d->B * d->H >= 65536.0)
        return set_error(SDM_ERR_UNSUPPORTED, "B*H must be < 65536");
    if ((int64_t)d->H * d->P >= (int64_t)1 << 22)
        return set_error(SDM_ERR_UNSUPPORTED, "H*P must be < 2^22");
    return SDM_OK;
}

sdm_status check_scan_inputs(const sdm_scan_desc *d, const void *x, const void *dt, const void *Bm,
                             const void *Cm, const float *A, const float *D, const float *dt_bias,
                             const int32_t *lengths)
{
    CHECK(check_strided(x, "x", d->dtype));
    CHECK(check_dense(dt, "dt"));
    CHECK(check_strided(Bm, "Bm", d->dtype));
    CHECK(check_strided(Cm, "Cm", d->dtype));
    CHECK(check_dense(A, "A"));
    CHECK(check_dense(D, "D", false));
    CHECK(check_dense(dt_bias, "dt_bias", false));
    return check_lengths(lengths);
}

// --------------------------------------------------------------- attention

sdm_status check_window(const sdm_window_desc *d)
{
    if (!d) return set_error(SDM_ERR_ARG, "null descriptor");
    CHECK(check_batch(d->B, d->T, d->dtype));
    if (d->Hq < 1 || d->Hk < 1 || d->D < 1)
        return set_error(SDM_ERR_ARG, "Hq, Hk, D must be >= 1 (got %d %d %d)", d->Hq, d->Hk, d->D);
    if (d->Hq % d->Hk)
        return set_error(SDM_ERR_ARG, "Hk = %d must divide Hq = %d", d->Hk, d->Hq);
    if (d->window < 1) return set_error(SDM_ERR_ARG, "window must be >= 1 (got %lld)", (long long)d->window);
    if (d->sinks < 0) return set_error(SDM_ERR_ARG, "sinks must be >= 0 (got %d)", d->sinks);
    if (!isfinite(d->scale)) return set_error(SDM_ERR_ARG, "scale must be finite");
    if (d->q_batch < 0 || d->q_token < 0 || d->q_head < 0 || d->k_batch < 0 || d->k_token < 0 ||
        d->k_head < 0 || d->v_batch < 0 || d->v_token < 0 || d->v_head < 0)
        return set_error(SDM_ERR_ARG, "strides must be >= 0");
    if (d->D > 256) return set_error(SDM_ERR_UNSUPPORTED, "D <= 256 is supported (got %d)", d->D);
    if (d->sinks > 1024)
        return set_error(SDM_ERR_UNSUPPORTED, "sinks <= 1024 is supported (got %d)", d->sinks);
    if (d->window >= (int64_t)1 << 30)
        return set_error(SDM_ERR_UNSUPPORTED, "window must be < 2^30");
    const double rows = (double)(d->sinks < d->T ? d->sinks : d->T) +
                        (double)(d->window < d->T ? d->window : d->T);
    if ((double)d->B * d->Hq * (double)((d->T + 63) / 64) >= 2147483648.0 ||
        (double)d->B * rows >= 2147483648.0)
        return set_error(SDM_ERR_UNSUPPORTED,
                         "B*Hq*ceil(T/64) and B*(min(sinks, T) + min(window, T)) must be < 2^31");
    return SDM_OK;
}

}  // namespace

extern "C" {

sdm_status sdm_conv_forward(const sdm_conv_desc *d, const void *x, const float *weight,
                            const float *bias, const int32_t *lengths, unsigned flags, void *y,
                            void *state, void *stream)
{
    CHECK(check_conv(d));
    if (flags & ~SDM_FLAG_CONTINUE) return set_error(SDM_ERR_ARG, "unknown flags 0x%x", flags);
    CHECK(check_strided(x, "x", d->dtype));
    CHECK(check_dense(weight, "weight"));
    CHECK(check_dense(bias, "bias", false));
    CHECK(check_lengths(lengths));
    CHECK(check_dense(y, "y"));
    CHECK(check_dense(state, "state"));
    sdm::ConvArgs a = {};
    a.d = *d;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.lengths = lengths;
    a.cont = flags & SDM_FLAG_CONTINUE;
    a.y = y;
    a.state = state;
    const hipError_t e = sdm::launch_conv_forward(a, (hipStream_t)stream);
    return e == hipSuccess ? SDM_OK : hip_fail(e, "convolution launch");
}

sdm_status sdm_conv_backward_workspace_size(const sdm_conv_desc *d, size_t *bytes)
{
    if (!bytes) return set_error(SDM_ERR_ARG, "null bytes pointer");
    *bytes = 0;
    CHECK(check_conv(d));
    *bytes = sdm::conv_backward_ws(*d);
    return SDM_OK;
}

sdm_status sdm_conv_backward(const sdm_conv_desc *d, const void *x, const float *weight,
                             const float *bias, const int32_t *lengths, const void *dy,
                             const void *state, const void *dstateT, void *workspace,
                             size_t ws_bytes, void *dx, float *dweight, float *dbias,
                             void *dstate, void *stream)
{
    CHECK(check_conv(d));
    CHECK(check_strided(x, "x", d->dtype));
    CHECK(check_dense(weight, "weight"));
    CHECK(check_dense(bias, "bias", false));
    CHECK(check_lengths(lengths));
    CHECK(check_dense(dy, "dy"));
    CHECK(check_dense(state, "state", false));
    CHECK(check_dense(dstateT, "dstateT", false));
    CHECK(check_dense(dx, "dx"));
    CHECK(check_dense(dweight, "dweight"));
    CHECK(check_dense(dbias, "dbias", false));
    CHECK(check_dense(dstate, "dstate", false));
    CHECK(check_workspace(workspace, ws_bytes, sdm::conv_backward_ws(*d)));
    sdm::ConvArgs a = {};
    a.d = *d;
    a.x = x;
    a.dy = dy;
    a.weight = weight;
    a.bias = bias;
    a.lengths = lengths;
    a.state0 = state;
    a.dstateT = dstateT;
    a.dx = dx;
    a.dstate0 = dstate;
    a.dweight = dweight;
    a.dbias = dbias;
    a.partial = (float *)workspace;
    const hipError_t e = sdm::launch_conv_backward(a, (hipStream_t)stream);
    return e == hipSuccess ? SDM_OK : hip_fail(e, "convolution backward launch");
}

sdm_status sdm_scan_workspace_size(const sdm_scan_desc *d, size_t *bytes)
{
    if (!bytes) return set_error(SDM_ERR_ARG, "null bytes pointer");
    *bytes = 0;
    CHECK(check_scan(d));
    *bytes = sdm::scan_forward_ws(*d);
    return SDM_OK;
}

sdm_status sdm_scan_forward(const sdm_scan_desc *d, const void *x, const void *dt, const void *Bm,
                            const void *Cm, const float *A, const float *D, const float *dt_bias,
                            const int32_t *lengths, unsigned flags, void *workspace,
                            size_t ws_bytes, void *y, float *state, void *stream)
{
    CHECK(check_scan(d));
    if (flags & ~SDM_FLAG_CONTINUE) return set_error(SDM_ERR_ARG, "unknown flags 0x%x", flags);
    CHECK(check_scan_inputs(d, x, dt, Bm, Cm, A, D, dt_bias, lengths));
    CHECK(check_dense(y, "y"));
    CHECK(check_dense(state, "state"));
    CHECK(check_workspace(workspace, ws_bytes, sdm::scan_forward_ws(*d)));
    sdm::ScanArgs a = {};
    a.d = *d;
    a.x = x;
    a.dt = dt;
    a.Bm = Bm;
    a.Cm = Cm;
    a.A = A;
    a.D = D;
    a.dt_bias = dt_bias;
    a.lengths = lengths;
    a.cont = flags & SDM_FLAG_CONTINUE;
    a.y = y;
    a.state = state;
    a.ws = (unsigned char *)workspace;
    const hipError_t e = sdm::launch_scan_forward(a, (hipStream_t)stream);
    return e == hipSuccess ? SDM_OK : hip_fail(e, "scan launch");
}

sdm_status sdm_scan_backward_workspace_size(const sdm_scan_desc *d, size_t *bytes)
{
    if (!bytes) return set_error(SDM_ERR_ARG, "null bytes pointer");
    *bytes = 0;
    CHECK(check_scan(d));
    *bytes = sdm::scan_backward_ws(*d);
    return SDM_OK;
}

sdm_status sdm_scan_backward(const sdm_scan_desc *d, const void *x, const void *dt,
                             const void *Bm, const void *Cm, const float *A, const float *D,
                             const float *dt_bias, const int32_t *lengths, const void *dy,
                             const float *state, const float *dstateT, void *workspace,
                             size_t ws_bytes, void *dx, void *ddt, void *dB, void *dC, float *dA,
                             float *dD, float *ddt_bias, float *dstate, void *stream)
{
    CHECK(check_scan(d));
    CHECK(check_scan_inputs(d, x, dt, Bm, Cm, A, D, dt_bias, lengths));
    CHECK(check_dense(dy, "dy"));
    CHECK(check_dense(state, "state", false));
    CHECK(check_dense(dstateT, "dstateT", false));
    CHECK(check_dense(dx, "dx"));
    CHECK(check_dense(ddt, "ddt"));
    CHECK(check_dense(dB, "dB"));
    CHECK(check_dense(dC, "dC"));
    CHECK(check_dense(dA, "dA"));
    CHECK(check_dense(dD, "dD", false));
    CHECK(check_dense(ddt_bias, "ddt_bias", false));
    CHECK(check_dense(dstate, "dstate", false));
    CHECK(check_workspace(workspace, ws_bytes, sdm::scan_backward_ws(*d)));
    sdm::ScanArgs a = {};
    a.d = *d;
    a.x = x;
    a.dt = dt;
    a.Bm = Bm;
    a.Cm = Cm;
    a.A = A;
    a.D = D;
    a.dt_bias = dt_bias;
    a.lengths = lengths;
    a.dy = dy;
    a.state0 = state;
    a.dstateT = dstateT;
    a.dx = dx;
    a.ddt = ddt;
    a.dB = dB;
    a.dC = dC;
    a.dA = dA;
    a.dD = dD;
    a.ddt_bias = ddt_bias;
    a.dstate0 = dstate;
    a.ws = (unsigned char *)workspace;
    const hipError_t e = sdm::launch_scan_backward(a, (hipStream_t)stream);
    return e == hipSuccess ? SDM_OK : hip_fail(e, "scan backward launch");
}

sdm_status sdm_window_workspace_size(const sdm_window_desc *d, unsigned flags, size_t *bytes)
{
    if (!bytes) return set_error(SDM_ERR_ARG, "null bytes pointer");
    *bytes = 0;
    CHECK(check_window(d));
    if (flags & ~SDM_FLAG_CONTINUE) return set_error(SDM_ERR_ARG, "unknown flags 0x%x", flags);
    *bytes = sdm::window_forward_ws(*d, flags & SDM_FLAG_CONTINUE);
    return SDM_OK;
}

sdm_status sdm_window_forward(const sdm_window_desc *d, const void *q, const void *k,
                              const void *v, const int32_t *lengths, unsigned flags,
                              void *cache_k, void *cache_v, const int64_t *pos, void *workspace,
                              size_t ws_bytes, void *o, float *lse, void *stream)
{
    CHECK(check_window(d));
    if (flags & ~SDM_FLAG_CONTINUE) return set_error(SDM_ERR_ARG, "unknown flags 0x%x", flags);
    const bool cont = flags & SDM_FLAG_CONTINUE;
    CHECK(check_strided(q, "q", d->dtype));
    CHECK(check_strided(k, "k", d->dtype));
    CHECK(check_strided(v, "v", d->dtype));
    CHECK(check_lengths(lengths));
    CHECK(check_dense(cache_k, "cache_k", cont));
    CHECK(check_dense(cache_v, "cache_v", cont));
    if (!cache_k != !cache_v) return set_error(SDM_ERR_ARG, "cache_k and cache_v come together");
    if (cont && !pos) return set_error(SDM_ERR_ARG, "SDM_FLAG_CONTINUE needs pos");
    if (!cont && pos) return set_error(SDM_ERR_ARG, "pos needs SDM_FLAG_CONTINUE");
    if ((uintptr_t)pos & 7u) return set_error(SDM_ERR_ARG, "pos must be 8-byte aligned");
    CHECK(check_dense(o, "o"));
    CHECK(check_dense(lse, "lse"));
    CHECK(check_workspace(workspace, ws_bytes, sdm::window_forward_ws(*d, cont)));
    sdm::WindowArgs a = {};
    a.d = *d;
    a.q = q;
    a.k = k;
    a.v = v;
    a.lengths = lengths;
    a.pos = pos;
    a.cache_k = cache_k;
    a.cache_v = cache_v;
    a.o = o;
    a.lse = lse;
    a.ws = (unsigned char *)workspace;
    const hipError_t e = sdm::launch_window_forward(a, (hipStream_t)stream);
    return e == hipSuccess ? SDM_OK : hip_fail(e, "attention launch");
}

sdm_status sdm_window_backward_workspace_size(const sdm_window_desc *d, size_t *bytes)
{
    if (!bytes) return set_error(SDM_ERR_ARG, "null bytes pointer");
    *bytes = 0;
    CHECK(check_window(d));
    *bytes = sdm::window_backward_ws(*d);
    return SDM_OK;
}

sdm_status sdm_window_backward(const sdm_window_desc *d, const void *q, const void *k,
                               const void *v, const void *o, const float *lse, const void *dout,
                               const int32_t *lengths, void *workspace, size_t ws_bytes, void *dq,
                               void *dk, void *dv, void *stream)
{
    CHECK(check_window(d));
    CHECK(check_strided(q, "q", d->dtype));
    CHECK(check_strided(k, "k", d->dtype));
    CHECK(check_strided(v, "v", d->dtype));
    CHECK(check_dense(o, "o"));
    CHECK(check_dense(lse, "lse"));
    CHECK(check_dense(dout, "dout"));
    CHECK(check_lengths(lengths));
    CHECK(check_dense(dq, "dq"));
    CHECK(check_dense(dk, "dk"));
    CHECK(check_dense(dv, "dv"));
    CHECK(check_workspace(workspace, ws_bytes, sdm::window_backward_ws(*d)));
    sdm::WindowArgs a = {};
    a.d = *d;
    a.q = q;
    a.k = k;
    a.v = v;
    a.oin = o;
    a.lse_in = lse;
    a.dout = dout;
    a.lengths = lengths;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.ws = (unsigned char *)workspace;
    const hipError_t e = sdm::launch_window_backward(a, (hipStream_t)stream);
    return e == hipSuccess ? SDM_OK : hip_fail(e, "attention backward launch");
}

}  // extern "C"
