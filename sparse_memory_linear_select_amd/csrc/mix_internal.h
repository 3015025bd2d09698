// Internal declarations of the sequence mixers beside the SDM core: the short
// causal convolution, the selective state space scan and sliding-window
// attention (not installed).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sdm.h"

namespace sdm {

// Thread-local error text of the C entry points (sdm_api.cpp).
sdm_status set_error(sdm_status s, const char *fmt, ...);

// Whether rows of a strided tensor start on 16 bytes and hold whole 16-byte
// vectors of `cols` elements.
inline bool rows_on_16(const void *p, int64_t s0, int64_t s1, int64_t s2, int64_t cols, int esize)
{
    return (((uintptr_t)p | (uintptr_t)(s0 * esize) | (uintptr_t)(s1 * esize) |
             (uintptr_t)(s2 * esize) | (uintptr_t)(cols * esize)) & 15u) == 0;
}

struct ConvArgs {
    sdm_conv_desc d;
    const void *x, *dy;
    const float *weight, *bias;
    const int32_t *lengths;
    bool cont;              // forward: `state` holds the rows before x
    const void *state0;     // backward: rows before x, or null
    const void *dstateT;    // backward: gradient of the final state, or null
    void *y, *state;        // forward outputs
    void *dx, *dstate0;     // backward outputs
    float *dweight, *dbias;
    float *partial;         // backward: [blocks][K + 1][C] sums
};
size_t conv_backward_ws(const sdm_conv_desc &d);
hipError_t launch_conv_forward(const ConvArgs &a, hipStream_t stream);
hipError_t launch_conv_backward(const ConvArgs &a, hipStream_t stream);

struct ScanArgs {
    sdm_scan_desc d;
    const void *x, *dt, *Bm, *Cm;
    const float *A, *D, *dt_bias;
    const int32_t *lengths;
    bool cont;                      // forward: `state` holds the state before x
    void *y;
    float *state;
    const void *dy;                 // backward
    const float *state0, *dstateT;
    void *dx, *ddt, *dB, *dC;
    float *dA, *dD, *ddt_bias, *dstate0;
    unsigned char *ws;
};
size_t scan_forward_ws(const sdm_scan_desc &d);
size_t scan_backward_ws(const sdm_scan_desc &d);
hipError_t launch_scan_forward(const ScanArgs &a, hipStream_t stream);
hipError_t launch_scan_backward(const ScanArgs &a, hipStream_t stream);

struct WindowArgs {
    sdm_window_desc d;
    const void *q, *k, *v;
    const int32_t *lengths;
    const int64_t *pos;             // tokens before this call, or null for none
    void *cache_k, *cache_v;        // or null
    void *o;
    float *lse;
    const void *oin, *dout;         // backward
    const float *lse_in;
    void *dq, *dk, *dv;
    unsigned char *ws;
};
size_t window_forward_ws(const sdm_window_desc &d, bool cont);
size_t window_backward_ws(const sdm_window_desc &d);
hipError_t launch_window_forward(const WindowArgs &a, hipStream_t stream);
hipError_t launch_window_backward(const WindowArgs &a, hipStream_t stream);

}  // namespace sdm
