// rms_norm.hpp -- host-visible interface of the root-mean-square norm behind a residual's addition
// (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace linrec {

constexpr int kRmsMaxC = 8192;  // channels: a workgroup holds a row in registers

struct RmsArgs {
    int64_t N, C;
    int dtype, rtype;     // of x, y and gx; of the residual, the sum and the sum's gradients
    float eps;
    const void* x;        // (N,C)
    const void* res;      // (N,C), or null
    const float* weight;  // (C)
    void* y;              // (N,C)
    void* sum;            // (N,C); null without res
    // backward: the sum (x itself where there was no residual), the upstream gradients
    const void* s;        // (N,C) of rtype
    const void *gy, *gsum;  // (N,C) of dtype; of rtype, or null
    void *gx, *gs;        // (N,C) of dtype, or null where gs says the same; of rtype
    float* gweight;       // (C)
    float* part;          // workspace: (walkers,C) partial sums
};

hipError_t run_rms_norm(const RmsArgs& A, hipStream_t st);
hipError_t run_rms_norm_backward(const RmsArgs& A, hipStream_t st);
// Bytes of RmsArgs::part: a pure function of the sizes (and not of pointers' alignment).
size_t rms_norm_backward_ws_bytes(int64_t N, int64_t C);

}  // namespace linrec
