// row_ops.hpp -- what the kernels of the selective scan, the short convolution and the root-mean-square norm share:
// the logistic function, the tokens of a row that are there, sums over lanes and over rows of partial sums.
#pragma once

#include "elem_types.hpp"

namespace linrec {

__device__ __forceinline__ float logistic(float t) {
    // e^{-t} may be infinite: the reciprocal is then 0.
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-t * kLog2e));
}

// Tokens of row b that are there.
__device__ __forceinline__ int64_t tokens_of(const int* lengths, int64_t T, int64_t b) {
    if (!lengths) return T;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : (n < T ? n : T);
}

// v summed over this lane and the one that the DPP permutation CTRL exchanges it with.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// The sum of column j of (rows, cols) partial sums, in the lanes of strip 0 (the first 16 of a workgroup of 256, a
// column each): 16 strips of rows at once, then the strips in order.
__device__ __forceinline__ float fold_column(const float* __restrict__ part, int64_t rows, int64_t cols, int64_t j,
                                             float (&lds)[16][17]) {
    const int cx = threadIdx.x & 15, strip = threadIdx.x >> 4;
    float v = 0.f;
    if (j < cols)
#pragma unroll 4
        for (int64_t r = strip; r < rows; r += 16) v += part[r * cols + j];
    lds[strip][cx] = v;
    __syncthreads();
    if (strip == 0) {
#pragma unroll
        for (int i = 1; i < 16; ++i) v += lds[i][cx];
    }
    return v;
}

}  // namespace linrec
