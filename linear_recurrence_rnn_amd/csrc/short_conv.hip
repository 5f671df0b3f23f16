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
// A lane takes VEC neighbouring channels and walks down a run of tokens with the last K-1
// inputs, and backwards also the last K-1 of q, in registers, so a token is read once but for the K-1
// before (and, backwards, behind) a run; the next tokens are on their way meanwhile.  Both
// directions are bound by memory.  The sums over tokens are kept in registers over a wave's runs, go to the
// workspace and are added in the order of the waves.
#include <algorithm>

#include "short_conv.hpp"
#include "group_norm.hpp"  // the activations' codes
#include "row_ops.hpp"

namespace linrec {

namespace {

// Tokens asked for at once.  Forward, 8 x 4096 tokens of 2560 bfloat16 channels take 65 us with four (5.2
// TB/s), 67 with eight and 72 with two; backward 121 with two (4.2 TB/s), 135 with four.
constexpr int kForwardAhead = 4, kBackwardAhead = 2;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

__device__ __forceinline__ int64_t row_length(const ConvShape& s, int64_t b) { return tokens_of(s.lengths, s.T, b); }

// VEC elements as they come from memory, and their values.
template <class E, int VEC> struct Raw { typedef E type __attribute__((ext_vector_type(VEC))); };
template <class E> struct Raw<E, 1> { typedef E type; };

// Row `row` (the same for the wave) of p, a lane's channels from byte `off`: the form that takes two
// scalar registers and one vector register for the address.
template <class E, int VEC>
__device__ __forceinline__ typename Raw<E, VEC>::type load_raw(const void* p, int64_t row, int64_t C, unsigned off) {
    const char* const base = reinterpret_cast<const char*>(reinterpret_cast<const E*>(p) + row * C);
    return *reinterpret_cast<const typename Raw<E, VEC>::type*>(base + off);
}
template <class E, int VEC>
__device__ __forceinline__ void values(const typename Raw<E, VEC>::type& v, bool there, float (&out)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        if constexpr (VEC == 1) out[j] = there ? (float)v : 0.f;
        else out[j] = there ? (float)v[j] : 0.f;
    }
}
template <class E, int VEC>
__device__ __forceinline__ void store_vec(void* p, int64_t row, int64_t C, unsigned off, const float (&in)[VEC]) {
    typename Raw<E, VEC>::type v;
    if constexpr (VEC == 1) v = (E)in[0];
    else
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = (E)in[j];
    char* const base = reinterpret_cast<char*>(reinterpret_cast<E*>(p) + row * C);
    *reinterpret_cast<typename Raw<E, VEC>::type*>(base + off) = v;
}

// Input at token t (which may lie in the state, t < 0) of row b, channels c..; zero where there is none.
template <class E, int VEC>
__device__ __forceinline__ void load_input(const ConvShape& s, const ConvArgs& A, int64_t b, int64_t t, int64_t len,
                                           unsigned off, float (&out)[VEC]) {
    if (t >= 0 && t < len) {
        values<E, VEC>(load_raw<E, VEC>(A.x, b * s.T + t, s.C, off), true, out);
    } else if (t < 0 && A.s_in) {
        values<E, VEC>(load_raw<E, VEC>(A.s_in, b * (s.K - 1) + t + s.K - 1, s.C, off), true, out);
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

// One run a wave, four a workgroup, 64 lanes of VEC channels each.
template <class E, int K, int VEC>
__global__ __launch_bounds__(256) void short_conv_kernel(ConvShape s, ConvArgs A, int64_t runs, int64_t run_tokens,
                                                         int64_t cols) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t col = blockIdx.x % cols, run = blockIdx.x / cols * 4 + wave;
    const int64_t c = (col * 64 + (threadIdx.x & 63)) * VEC;
    const unsigned off = (unsigned)c * (unsigned)sizeof(E);
    if (c >= s.C || run >= s.B * runs) return;
    const int64_t b = run / runs, t0 = run % runs * run_tokens, len = row_length(s, b);
    const int64_t t_end = t0 + run_tokens < s.T ? t0 + run_tokens : s.T;
    // Tokens that are absent or behind the run are read as the last one that is neither, and not used.
    const int64_t t_live = t_end < len ? t_end : len;
    typename Raw<E, VEC>::type next[kForwardAhead];
    const auto fetch = [&](int64_t t) {
#pragma unroll
        for (int u = 0; u < kForwardAhead; ++u)
            next[u] = load_raw<E, VEC>(A.x, b * s.T + (t + u < t_live ? t + u : t_live - 1), s.C, off);
    };
    if (t0 < t_live) fetch(t0);
    float w[K][VEC], bias[VEC];
    load_filters<K, VEC>(A, c, w, bias);
    float x[K][VEC];  // x[k] = x_{t-K+1+k}
#pragma unroll
    for (int k = 0; k < K - 1; ++k) load_input<E, VEC>(s, A, b, t0 - (K - 1) + k, len, off, x[k + 1]);
    // The first run of a row also writes the state, which may be the one that was read: all that
    // is needed of that is in registers before.
    float keep[K > 1 ? K - 1 : 1][VEC];
    const bool states = A.s_out && t0 == 0;
    if (states) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) load_input<E, VEC>(s, A, b, len - (K - 1) + k, len, off, keep[k]);
    }
    int64_t t1 = t0;
    for (; t1 < t_live; t1 += kForwardAhead) {
        typename Raw<E, VEC>::type now[kForwardAhead];
#pragma unroll
        for (int u = 0; u < kForwardAhead; ++u) now[u] = next[u];
        if (t1 + kForwardAhead < t_live) fetch(t1 + kForwardAhead);
#pragma unroll
        for (int u = 0; u < kForwardAhead; ++u) {
            const int64_t t = t1 + u;
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int j = 0; j < VEC; ++j) x[k][j] = x[k + 1][j];
            values<E, VEC>(now[u], t < len, x[K - 1]);
            float y[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float v = bias[j];
#pragma unroll
                for (int k = 0; k < K; ++k) v = fmaf(w[k][j], x[k][j], v);
                if (s.act == kActSilu) v *= logistic(v);
                y[j] = t < len ? v : 0.f;
            }
            if (t < t_end) store_vec<E, VEC>(A.y, b * s.T + t, s.C, off, y);
        }
    }
    float none[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) none[j] = 0.f;
    for (; t1 < t_end; ++t1) store_vec<E, VEC>(A.y, b * s.T + t1, s.C, off, none);
    if (states) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) store_vec<E, VEC>(A.s_out, b * (K - 1) + k, s.C, off, keep[k]);
    }
}

template <class E, int K, int VEC>
__global__ __launch_bounds__(256) void short_conv_bwd_kernel(ConvShape s, ConvArgs A, ConvBwdArgs g, int64_t runs,
                                                             int64_t run_tokens, int64_t cols) {
    __shared__ float acc[4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t col = blockIdx.x % cols, walker = blockIdx.x / cols, walkers = gridDim.x / cols;
    const int64_t c = (col * 64 + lane) * VEC;
    const unsigned off = (unsigned)c * (unsigned)sizeof(E);
    const bool live = c < s.C;
    float gw[K][VEC], gb[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        gb[j] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) gw[k][j] = 0.f;
    }
    float w[K][VEC], bias[VEC];
    if (live) load_filters<K, VEC>(A, c, w, bias);
    for (int64_t run = walker * 4 + wave; live && run < s.B * runs; run += walkers * 4) {
        const int64_t b = run / runs, t0 = run % runs * run_tokens, len = row_length(s, b);
        const int64_t t_end = t0 + run_tokens < s.T ? t0 + run_tokens : s.T;
        // The line's elements up to K-1 tokens beyond the run: x's gradient at a token needs the q behind it.
        // Absent tokens are read as the last one that is there and not used.
        typename Raw<E, VEC>::type nx[kBackwardAhead], ny[kBackwardAhead];
        const auto fetch = [&](int64_t t) {
#pragma unroll
            for (int u = 0; u < kBackwardAhead; ++u) {
                const int64_t row = b * s.T + (t + u < len ? t + u : len - 1);
                nx[u] = load_raw<E, VEC>(A.x, row, s.C, off);
                ny[u] = load_raw<E, VEC>(g.gy, row, s.C, off);
            }
        };
        if (t0 < len) fetch(t0);
        float x[K][VEC], q[K][VEC];  // x[k] = x_{t-K+1+k}, q[k] = q_{t-k}
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (k < K - 1) load_input<E, VEC>(s, A, b, t0 - (K - 1) + k, len, off, x[k + 1 < K ? k + 1 : 0]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) q[k][j] = 0.f;
        }
        for (int64_t t1 = t0; t1 < t_end + K - 1; t1 += kBackwardAhead) {
            typename Raw<E, VEC>::type vx[kBackwardAhead], vy[kBackwardAhead];
#pragma unroll
            for (int u = 0; u < kBackwardAhead; ++u) vx[u] = nx[u], vy[u] = ny[u];
            if (t1 + kBackwardAhead < len && t1 + kBackwardAhead < t_end + K - 1) fetch(t1 + kBackwardAhead);
#pragma unroll
            for (int u = 0; u < kBackwardAhead; ++u) {
                const int64_t t = t1 + u, out = t - (K - 1);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
#pragma unroll
                    for (int k = 0; k < K - 1; ++k) x[k][j] = x[k + 1][j];
#pragma unroll
                    for (int k = K - 1; k > 0; --k) q[k][j] = q[k - 1][j];
                }
                values<E, VEC>(vx[u], t < len, x[K - 1]);
                values<E, VEC>(vy[u], t < len, q[0]);
                if (s.act == kActSilu) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        float v = bias[j];
#pragma unroll
                        for (int k = 0; k < K; ++k) v = fmaf(w[k][j], x[k][j], v);
                        const float sg = logistic(v);
                        q[0][j] = t < len ? q[0][j] * (sg * fmaf(v, 1.f - sg, 1.f)) : 0.f;
                    }
                }
                if (t < t_end) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        gb[j] += q[0][j];
#pragma unroll
                        for (int k = 0; k < K; ++k) gw[k][j] = fmaf(q[0][j], x[k][j], gw[k][j]);
                    }
                }
                // The line's element t, token `out`: the run's own tokens, and the state's before the first.
                if (out >= t_end || (out < t0 && t0 > 0) || (out < 0 && !g.gs_in)) continue;
                float v[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    v[j] = 0.f;
#pragma unroll
                    for (int k = 0; k < K; ++k) v[j] = fmaf(w[k][j], q[k][j], v[j]);
                }
                if (g.gs_out && t >= len && t < len + K - 1) {
                    float gs[VEC];
                    values<E, VEC>(load_raw<E, VEC>(g.gs_out, b * (K - 1) + t - len, s.C, off), true, gs);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) v[j] += gs[j];
                }
                if (out >= 0) store_vec<E, VEC>(g.gx, b * s.T + out, s.C, off, v);
                else store_vec<E, VEC>(g.gs_in, b * (K - 1) + t, s.C, off, v);
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

// Sum of the workgroups' partial sums, 16 strips of them at once, then the strips in order.
__global__ __launch_bounds__(256) void short_conv_fold_kernel(const float* __restrict__ part, int64_t rows, int64_t C,
                                                              int K, float* __restrict__ gw, float* __restrict__ gb) {
    __shared__ float lds[16][17];
    const int64_t cols = (K + 1) * C, j = (int64_t)blockIdx.x * 16 + (threadIdx.x & 15);
    const float v = fold_column(part, rows, cols, j, lds);
    if (threadIdx.x >= 16 || j >= cols) return;
    const int64_t k = j / C, c = j % C;
    if (k < K) gw[c * K + k] = v;
    else if (gb) gb[c] = v;
}

constexpr int kVec = 4;  // channels of a lane

// Tokens of a run: as many as leave `waves` waves of 64 lanes with `vec` channels each to the chip, 16 at least; a row has
// one run at least, for its state if it has no tokens.  A wave takes one run or, `bounded`, as many as leave no more
// than that many waves.
struct ConvPlan {
    int64_t run_tokens, runs, groups;  // runs of a row; workgroups a column of channels
};
ConvPlan plan(const ConvShape& s, int64_t waves, int vec, bool bounded) {
    ConvPlan p{};
    const int64_t cols = ceil_div(s.C, 64 * vec);
    int64_t runs = waves / cols / s.B;  // of a row, so that all of them fit
    if (runs < 1) runs = 1;
    int64_t n = ceil_div(s.T, runs);
    n = ceil_div(n < 16 ? 16 : n, 4) * 4;
    p.run_tokens = n;
    p.runs = s.T ? ceil_div(s.T, n) : 1;
    p.groups = ceil_div(s.B * p.runs, 4);
    if (bounded) p.groups = std::min(p.groups, std::max<int64_t>(waves / cols / 4, 1));
    return p;
}
// Forward four times what the chip holds at once, so that ragged rows even out: a batch of 16 ragged
// rows of up to 2000 tokens takes 43 us, 47 with half as many waves; full rows care little.  With one channel a lane runs
// as long as with four, and so four times the waves: 8 x 4096 tokens of 2562 channels take 151 us, 164 with as many.
// Backward what it holds, and no more: 16 workgroups more than that cost a second round (174 us for 135), and
// each leaves K + 1 rows of partial sums.  Many short rows are taken by the same waves: a training step of 65536 rows of 4
// tokens, 256 channels, takes 211 us, 359 with a wave a row (and 84 MB of partial sums for 5).  One channel a lane: 8 x 4096
// tokens of 250 channels 40.4 us, 44.4 with four times the waves, of 2562 in float32 481 and 489.
constexpr int64_t kForwardWaves = 16384, kBackwardWaves = 4096;

template <class E, int K, int VEC>
hipError_t launch(const ConvShape& s, const ConvArgs& A, const ConvBwdArgs* g, hipStream_t st) {
    const int64_t cols = ceil_div(s.C, 64 * VEC);
    if (!g) {
        const ConvPlan p = plan(s, kForwardWaves, kVec, false);
        hipLaunchKernelGGL((short_conv_kernel<E, K, VEC>), dim3((unsigned)(cols * p.groups)), dim3(256), 0, st, s, A,
                           p.runs, p.run_tokens, cols);
        return hipGetLastError();
    }
    const ConvPlan p = plan(s, kBackwardWaves, VEC, true);
    hipLaunchKernelGGL((short_conv_bwd_kernel<E, K, VEC>), dim3((unsigned)(cols * p.groups)), dim3(256), 0, st, s, A, *g,
                       p.runs, p.run_tokens, cols);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(short_conv_fold_kernel, dim3((unsigned)ceil_div((K + 1) * s.C, 16)), dim3(256), 0, st, g->part,
                       p.groups, s.C, K, g->gweight, g->gbias);
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
    // Accesses of four elements where every row of every tensor starts on that.
    uintptr_t all = (uintptr_t)A.x | (uintptr_t)A.s_in | (uintptr_t)A.y | (uintptr_t)A.s_out;
    if (g) all |= (uintptr_t)g->gy | (uintptr_t)g->gs_out | (uintptr_t)g->gx | (uintptr_t)g->gs_in;
    const bool wide = s.C % kVec == 0 && all % (kVec * sizeof(E)) == 0;
    return wide ? by_taps<E, kVec>(s, A, g, st) : by_taps<E, 1>(s, A, g, st);
}

}  // namespace

hipError_t run_short_conv(const ConvShape& s, const ConvArgs& A, hipStream_t st) {
    return s.dtype == kBf16 ? by_alignment<bf16_t>(s, A, nullptr, st) : by_alignment<float>(s, A, nullptr, st);
}

size_t short_conv_backward_ws_bytes(const ConvShape& s) {
    const int64_t groups = std::max(plan(s, kBackwardWaves, kVec, true).groups, plan(s, kBackwardWaves, 1, true).groups);
    return (size_t)groups * (size_t)(s.K + 1) * (size_t)s.C * sizeof(float);
}

hipError_t run_short_conv_backward(const ConvShape& s, const ConvArgs& A, const ConvBwdArgs& g, hipStream_t st) {
    return s.dtype == kBf16 ? by_alignment<bf16_t>(s, A, &g, st) : by_alignment<float>(s, A, &g, st);
}

}  // namespace linrec
