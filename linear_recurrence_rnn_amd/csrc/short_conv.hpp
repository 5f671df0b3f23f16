// short_conv.hpp -- host-visible interface of the short causal convolution (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace linrec {

constexpr int kConvMaxK = 8;  // taps: a lane keeps its filters and inputs in registers

struct ConvShape {
    int64_t B, T, C;
    int K, act, dtype;
    const int* lengths;  // (B) device, or null
};

struct ConvArgs {
    const void* x;       // (B,T,C)
    const float* weight; // (C,K)
    const float* bias;   // (C), or null
    const void* s_in;    // (B,K-1,C), or null (zero)
    void* y;             // (B,T,C)
    void* s_out;         // (B,K-1,C), or null; may be s_in
};

struct ConvBwdArgs {
    const void* gy;      // (B,T,C)
    const void* gs_out;  // (B,K-1,C), or null
    void* gx;            // (B,T,C)
    float *gweight, *gbias;  // (C,K), (C) (null without bias)
    void* gs_in;         // (B,K-1,C), or null; not gs_out, which other runs read
    float* part;         // workspace: (walkers,K+1,C) partial sums
};

hipError_t run_short_conv(const ConvShape& s, const ConvArgs& A, hipStream_t st);
hipError_t run_short_conv_backward(const ConvShape& s, const ConvArgs& A, const ConvBwdArgs& g, hipStream_t st);
// Bytes of ConvBwdArgs::part: a pure function of the sizes (and not of pointers' alignment).
size_t short_conv_backward_ws_bytes(const ConvShape& s);

}  // namespace linrec
