// short_conv.hip -- the short causal convolution of each channel, forward and backward.
//
//   pre_t = bias + sum_k w[k] x_{t-K+1+k},   y_t = act(pre_t)
// where x before the first token is the carried state (K-1 inputs) or zero.  In the order of one
// line of inputs, state first: line index i = t + K - 1, and the state behind the last token is
// the line's elements len .. len + K - 2.
//
// Backward, with q_t = gy_t act'(pre_t):
//   gw[k] = sum q_t x_{t-K+1+k},  gbias = sum q_t,
//   gline[i] = sum_k w[k] q_{i-k}  (+ gs_out[i - len] for len <= i < len + K - 1)
// of which the first K-1 elements are the carried state's gradient and the others x's.
//
// A lane takes VEC neighbouring channels (16 bytes) and walks down a run of tokens with the last K-1
// inputs, and backwards also the last K-1 of q, in registers, so a token is read once but for the K-1
// before (and, backwards, behind) a run.  Both directions are bound by memory.  The sums over tokens
// are kept in registers over a walker's runs, go to the workspace and are added in walker order.
#include "short_conv.hpp"
#include "group_norm.hpp"  // the activations' codes
#include "elem_types.hpp"

namespace linrec {

namespace {

constexpr int kRun = 16;  // tokens of a run

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

__device__ __forceinline__ float logistic(float t) {
    // e^{-t} may be infinite: the reciprocal is then 0.
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-t * kLog2e));
}

__device__ __forceinline__ int64_t row_length(const ConvShape& s, int64_t b) {
    if (!s.lengths) return s.T;
    const int64_t n = s.lengths[b];
    return n < 0 ? 0 : (n < s.T ? n : s.T);
}

template <class E, int VEC>
__device__ __forceinline__ void load_vec(const E* __restrict__ p, float* __restrict__ out) {
    if constexpr (VEC == 1) out[0] = (float)*p;
    else load16<E>(p, out);
}
template <class E, int VEC, bool NT>
__device__ __forceinline__ void store_vec(E* __restrict__ p, const float* __restrict__ in) {
    if constexpr (VEC == 1) *p = (E)in[0];
    else store16<E, NT>(p, in);
}

// Input at token t (which may lie in the state, t < 0) of row b, channels c..; zero where there is none.
template <class E, int VEC>
__device__ __forceinline__ void load_input(const ConvShape& s, const ConvArgs& A, int64_t b, int64_t t, int64_t len,
                                           int64_t c, float* __restrict__ out) {
    if (t >= 0 && t < len) {
        load_vec<E, VEC>(reinterpret_cast<const E*>(A.x) + (b * s.T + t) * s.C + c, out);
    } else if (t < 0 && A.s_in) {
        load_vec<E, VEC>(reinterpret_cast<const E*>(A.s_in) + (b * (s.K - 1) + t + s.K - 1) * s.C + c, out);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) out[j] = 0.f;
    }
}

template <int K, int VEC>
__device__ __forceinline__ void load_filters(const ConvArgs& A, int64_t c, float (&w)[K][VEC], float (&bias)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][j] = A.weight[(c + j) * K + k];
        bias[j] = A.bias ? A.bias[c + j] : 0.f;
    }
}

// Four runs a workgroup, 64 lanes of VEC channels each.
template <class E, int K, int VEC>
__global__ __launch_bounds__(256) void short_conv_kernel(ConvShape s, ConvArgs A, int64_t runs, int64_t cols) {
    const int64_t col = blockIdx.x % cols, run = blockIdx.x / cols * 4 + (threadIdx.x >> 6);
    const int64_t c = (col * 64 + (threadIdx.x & 63)) * VEC;
    if (c >= s.C || run >= s.B * runs) return;
    const int64_t b = run / runs, t0 = run % runs * kRun, len = row_length(s, b);
    float w[K][VEC], bias[VEC];
    load_filters<K, VEC>(A, c, w, bias);
    float x[K][VEC];  // x[k] = x_{t-K+1+k}
#pragma unroll
    for (int k = 0; k < K - 1; ++k) load_input<E, VEC>(s, A, b, t0 - (K - 1) + k, len, c, x[k + 1]);
    // The first run of a row also writes the state, which may be the one that was read: all that
    // is needed of that is in registers before.
    float keep[K > 1 ? K - 1 : 1][VEC];
    const bool states = A.s_out && t0 == 0;
    if (states) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) load_input<E, VEC>(s, A, b, len - (K - 1) + k, len, c, keep[k]);
    }
#pragma unroll 4
    for (int i = 0; i < kRun; ++i) {
        const int64_t t = t0 + i;
        if (t >= s.T) break;
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
#pragma unroll
            for (int j = 0; j < VEC; ++j) x[k][j] = x[k + 1][j];
        load_input<E, VEC>(s, A, b, t, len, c, x[K - 1]);
        float y[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            float v = bias[j];
#pragma unroll
            for (int k = 0; k < K; ++k) v = fmaf(w[k][j], x[k][j], v);
            if (s.act == kActSilu) v *= logistic(v);
            y[j] = t < len ? v : 0.f;
        }
        store_vec<E, VEC, true>(reinterpret_cast<E*>(A.y) + (b * s.T + t) * s.C + c, y);
    }
    if (states) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
            store_vec<E, VEC, false>(reinterpret_cast<E*>(A.s_out) + (b * (K - 1) + k) * s.C + c, keep[k]);
    }
}

// Walkers of 64 lanes, four a workgroup; a walker takes every (4 * walkers)-th run.
template <class E, int K, int VEC>
__global__ __launch_bounds__(256) void short_conv_bwd_kernel(ConvShape s, ConvArgs A, ConvBwdArgs g, int64_t runs,
                                                             int64_t cols, int64_t walkers) {
    __shared__ float acc[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t col = blockIdx.x % cols, walker = blockIdx.x / cols;
    const int64_t c = (col * 64 + lane) * VEC;
    const bool live = c < s.C;
    float gw[K][VEC], gb[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        gb[j] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) gw[k][j] = 0.f;
    }
    if (live) {
        float w[K][VEC], bias[VEC];
        load_filters<K, VEC>(A, c, w, bias);
        for (int64_t run = walker * 4 + wave; run < s.B * runs; run += walkers * 4) {
            const int64_t b = run / runs, t0 = run % runs * kRun, len = row_length(s, b);
            float x[K][VEC], q[K][VEC];  // q[k] = q_{t-k}
#pragma unroll
            for (int k = 0; k < K - 1; ++k) {
                load_input<E, VEC>(s, A, b, t0 - (K - 1) + k, len, c, x[k + 1]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) q[k][j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) q[K - 1][j] = 0.f;
            float gs[K > 1 ? K - 1 : 1][VEC];  // gs_out: it may be overwritten
            if (g.gs_out) {
#pragma unroll
                for (int k = 0; k < K - 1; ++k)
                    load_vec<E, VEC>(reinterpret_cast<const E*>(g.gs_out) + (b * (K - 1) + k) * s.C + c, gs[k]);
            }
            // Tokens up to K-1 beyond the run: x's gradient at a token needs the q behind it.
#pragma unroll 1
            for (int i = 0; i < kRun + K - 1; ++i) {
                const int64_t t = t0 + i, out = t - (K - 1);
                const bool mine = i < kRun;
                if (out >= s.T) break;
#pragma unroll
                for (int k = 0; k < K - 1; ++k)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) x[k][j] = x[k + 1][j];
#pragma unroll
                for (int k = K - 1; k > 0; --k)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) q[k][j] = q[k - 1][j];
                load_input<E, VEC>(s, A, b, t, len, c, x[K - 1]);
                if (t < len) {
                    load_vec<E, VEC>(reinterpret_cast<const E*>(g.gy) + (b * s.T + t) * s.C + c, q[0]);
                    if (s.act == kActSilu) {
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            float v = bias[j];
#pragma unroll
                            for (int k = 0; k < K; ++k) v = fmaf(w[k][j], x[k][j], v);
                            const float sg = logistic(v);
                            q[0][j] *= sg * fmaf(v, 1.f - sg, 1.f);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) q[0][j] = 0.f;
                }
                if (mine) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        gb[j] += q[0][j];
#pragma unroll
                        for (int k = 0; k < K; ++k) gw[k][j] = fmaf(q[0][j], x[k][j], gw[k][j]);
                    }
                }
                // The line's element t, token `out`: a run's own tokens, and the state's before the first.
                if (out < t0 && t0 > 0) continue;
                if (out < 0 && !g.gs_in) continue;
                float v[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    v[j] = 0.f;
#pragma unroll
                    for (int k = 0; k < K; ++k) v[j] = fmaf(w[k][j], q[k][j], v[j]);
                }
                if (g.gs_out && t >= len && t < len + K - 1) {
#pragma unroll
                    for (int k = 0; k < K - 1; ++k)
                        if (t - len == k)
#pragma unroll
                            for (int j = 0; j < VEC; ++j) v[j] += gs[k][j];
                }
                E* p = out >= 0 ? reinterpret_cast<E*>(g.gx) + (b * s.T + out) * s.C + c
                                : reinterpret_cast<E*>(g.gs_in) + (b * (K - 1) + t) * s.C + c;
                store_vec<E, VEC, false>(p, v);
            }
        }
    }
    // This workgroup's sums: the four waves in order.
    float* const part = g.part + walker * (K + 1) * s.C + c;
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            __syncthreads();
            acc[wave][lane] = k < K ? gw[k < K ? k : 0][j] : gb[j];
            __syncthreads();
            if (wave == 0 && live) part[k * s.C + j] = acc[0][lane] + acc[1][lane] + acc[2][lane] + acc[3][lane];
        }
}

// Sum of the walkers' partial sums, 16 strips of walkers at once, then the strips in order.
__global__ __launch_bounds__(256) void short_conv_fold_kernel(const float* __restrict__ part, int64_t rows, int64_t C,
                                                              int K, float* __restrict__ gw, float* __restrict__ gb) {
    __shared__ float lds[16][17];
    const int cx = threadIdx.x & 15, strip = threadIdx.x >> 4;
    const int64_t cols = (K + 1) * C, j = (int64_t)blockIdx.x * 16 + cx;
    float v = 0.f;
    if (j < cols)
#pragma unroll 4
        for (int64_t r = strip; r < rows; r += 16) v += part[r * cols + j];
    lds[strip][cx] = v;
    __syncthreads();
    if (strip != 0 || j >= cols) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) v += lds[i][cx];
    const int64_t k = j / C, c = j % C;
    if (k < K) gw[c * K + k] = v;
    else if (gb) gb[c] = v;
}

// Runs of a row: one at least, for the state of a row without tokens.
int64_t runs_of(const ConvShape& s) { return s.T ? ceil_div(s.T, kRun) : 1; }

// Walkers: four workgroups a CU over all channels, but no more than there are runs.
int64_t walkers_of(const ConvShape& s) {
    const int64_t cols = ceil_div(s.C, 64 * (s.dtype == kBf16 ? 8 : 4));
    int64_t n = ceil_div(1024, cols);
    const int64_t most = ceil_div(s.B * runs_of(s), 4);
    return n < most ? n : most;
}

template <class E, int K, int VEC>
hipError_t launch(const ConvShape& s, const ConvArgs& A, const ConvBwdArgs* g, hipStream_t st) {
    const int64_t cols = ceil_div(s.C, 64 * VEC), runs = runs_of(s);
    if (!g) {
        hipLaunchKernelGGL((short_conv_kernel<E, K, VEC>), dim3((unsigned)(cols * ceil_div(s.B * runs, 4))), dim3(256), 0,
                           st, s, A, runs, cols);
        return hipGetLastError();
    }
    const int64_t walkers = walkers_of(s);
    hipLaunchKernelGGL((short_conv_bwd_kernel<E, K, VEC>), dim3((unsigned)(cols * walkers)), dim3(256), 0, st, s, A, *g,
                       runs, cols, walkers);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(short_conv_fold_kernel, dim3((unsigned)ceil_div((K + 1) * s.C, 16)), dim3(256), 0, st, g->part,
                       walkers, s.C, K, g->gweight, g->gbias);
    return hipGetLastError();
}

template <class E, int VEC>
hipError_t by_taps(const ConvShape& s, const ConvArgs& A, const ConvBwdArgs* g, hipStream_t st) {
    switch (s.K) {
        case 1: return launch<E, 1, VEC>(s, A, g, st);
        case 2: return launch<E, 2, VEC>(s, A, g, st);
        case 3: return launch<E, 3, VEC>(s, A, g, st);
        case 4: return launch<E, 4, VEC>(s, A, g, st);
        case 5: return launch<E, 5, VEC>(s, A, g, st);
        case 6: return launch<E, 6, VEC>(s, A, g, st);
        case 7: return launch<E, 7, VEC>(s, A, g, st);
        default: return launch<E, 8, VEC>(s, A, g, st);
    }
}

template <class E>
hipError_t by_alignment(const ConvShape& s, const ConvArgs& A, const ConvBwdArgs* g, hipStream_t st) {
    // 16-byte accesses where every row of every tensor starts on 16 bytes.
    uintptr_t all = (uintptr_t)A.x | (uintptr_t)A.s_in | (uintptr_t)A.y | (uintptr_t)A.s_out;
    if (g) all |= (uintptr_t)g->gy | (uintptr_t)g->gs_out | (uintptr_t)g->gx | (uintptr_t)g->gs_in;
    const bool wide = s.C % ElemVec<E>::n == 0 && all % 16 == 0;
    return wide ? by_taps<E, ElemVec<E>::n>(s, A, g, st) : by_taps<E, 1>(s, A, g, st);
}

}  // namespace

hipError_t run_short_conv(const ConvShape& s, const ConvArgs& A, hipStream_t st) {
    return s.dtype == kBf16 ? by_alignment<bf16_t>(s, A, nullptr, st) : by_alignment<float>(s, A, nullptr, st);
}

size_t short_conv_backward_ws_bytes(const ConvShape& s) {
    return (size_t)walkers_of(s) * (size_t)(s.K + 1) * (size_t)s.C * sizeof(float);
}

hipError_t run_short_conv_backward(const ConvShape& s, const ConvArgs& A, const ConvBwdArgs& g, hipStream_t st) {
    return s.dtype == kBf16 ? by_alignment<bf16_t>(s, A, &g, st) : by_alignment<float>(s, A, &g, st);
}

}  // namespace linrec
