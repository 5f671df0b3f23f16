// group_norm.hpp -- host-visible interface of the per-token group norm (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace linrec {

constexpr int kNormMaxGroup = 8192;  // channels of a group: 32 a lane, 256 lanes
constexpr int kActNone = 0, kActSilu = 1;

struct NormArgs {
    const void *x, *gate;        // (N,C); gate may be null
    const float *weight, *bias;  // (C)
    void* y;                     // (N,C), forward
    const void* gy;              // (N,C), backward from here on
    void *gx, *ggate;            // (N,C)
    float *gweight, *gbias;      // (C)
    float* part;                 // workspace: (workers, 2, C) partial sums
    int64_t N, C;
    int G, D;                    // groups, channels of one
    float eps;
    int act, dtype;
};

hipError_t run_group_norm(const NormArgs& A, hipStream_t st);
hipError_t run_group_norm_backward(const NormArgs& A, hipStream_t st);
// Bytes of NormArgs::part: a pure function of the sizes (and not of pointers' alignment).
size_t group_norm_backward_ws_bytes(int64_t N, int64_t C, int G);

}  // namespace linrec
