// group_norm.hip -- group norm of each token's channels with an activation or a gate, and its
// gradients; x (N,C) with the channels last, G groups of D = C/G.
//
//   n = (x - mean) / sqrt(var + eps),  y = n w + b,  out = act(y)  or  y act(gate)
//
// mean and var are over the D channels of one token's group (biased variance), taken in passes over
// registers: the mean, then the mean of what it leaves (the float32 mean's own rounding, which would
// be a common offset of every n: 1e-4 of it at a mean of 1000 times the spread), then the squares.
// A mean that is large beside the spread so costs no digits that the inputs have.
//
// Backward, with dy = go act'(y) (no gate) or go act(gate):
//   dw = sum_tokens dy n,  db = sum_tokens dy,  dgate = go y act'(gate)
//   dx = rstd (dn - mean(dn) - n mean(dn n)),  dn = dy w
// The statistics are formed again from x, which has to be read anyway: nothing is kept by
// the forward.
//
// LPR lanes hold one token's group, EPL channels each; a wave holds 64/LPR neighbouring
// groups of one token (a workgroup of 256 lanes one group when LPR = 256) and walks down the
// tokens with its weights and its dw, db sums in registers.  The walkers' sums go to the
// workspace and are added in walker order by a second kernel, so results do not depend on
// timing.  Both directions are bound by memory: 32768 tokens of 2560 bfloat16 channels in 20 gated
// groups take 96 us forward (5.2 TB/s, what a copy of 1 GiB reaches) and 170 us backward (4.9).
#include "group_norm.hpp"
#include "elem_types.hpp"

namespace linrec {

namespace {

__device__ __forceinline__ float sigmoidf(float t) {
    // e^{-t} may be infinite: the reciprocal is then 0.
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-t * kLog2e));
}

// Sum over the LPR lanes of a group, the same bits in every lane.
template <int LPR>
__device__ __forceinline__ float group_sum(float v, float* lds) {
#pragma unroll
    for (int o = 1; o < (LPR < 64 ? LPR : 64); o <<= 1) v += __shfl_xor(v, o);
    if constexpr (LPR > 64) {
        __syncthreads();  // the previous sum has been read
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = lds[0];
#pragma unroll
        for (int w = 1; w < LPR / 64; ++w) v += lds[w];
    }
    return v;
}

// EPL channels of one lane: VEC consecutive ones from each of EPL/VEC stretches of LPR*VEC.
template <int LPR, int VEC>
__device__ __forceinline__ int chan(int i, int gl) { return (i / VEC) * (LPR * VEC) + gl * VEC + i % VEC; }

template <class E, int LPR, int EPL, bool WIDE, bool NT>
__device__ __forceinline__ void load_row(const E* __restrict__ p, int gl, int D, bool live, float* __restrict__ out) {
    constexpr int VEC = WIDE ? ElemVec<E>::n : 1;
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < EPL; i += VEC) {
            const int c = chan<LPR, VEC>(i, gl);
            if (live && c < D) load16<E, NT>(p + c, out + i);
            else
#pragma unroll
                for (int j = 0; j < VEC; ++j) out[i + j] = 0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int c = chan<LPR, VEC>(i, gl);
            out[i] = (live && c < D) ? (float)p[c] : 0.f;
        }
    }
}

template <class E, int LPR, int EPL, bool WIDE>
__device__ __forceinline__ void store_row(E* __restrict__ p, int gl, int D, bool live, const float* __restrict__ in) {
    constexpr int VEC = WIDE ? ElemVec<E>::n : 1;
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < EPL; i += VEC) {
            const int c = chan<LPR, VEC>(i, gl);
            if (live && c < D) store16<E, true>(p + c, in + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int c = chan<LPR, VEC>(i, gl);
            if (live && c < D) p[c] = (E)in[i];
        }
    }
}

// Per-channel parameters of a lane (float32).
template <int LPR, int EPL, int VEC>
__device__ __forceinline__ void load_chan(const float* __restrict__ p, int gl, int D, bool live, float* __restrict__ out) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int c = chan<LPR, VEC>(i, gl);
        out[i] = (live && c < D) ? p[c] : 0.f;
    }
}

// x -> n in place (0 in the lanes past the group); returns rstd.
template <int LPR, int EPL, int VEC>
__device__ __forceinline__ float normalise(float* __restrict__ x, int gl, int D, float eps, float* lds) {
    const float inv = 1.f / (float)D;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) s += x[i];
    const float mean = group_sum<LPR>(s, lds) * inv;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        x[i] = chan<LPR, VEC>(i, gl) < D ? x[i] - mean : 0.f;
        s += x[i];
    }
    const float rest = group_sum<LPR>(s, lds) * inv;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        x[i] = chan<LPR, VEC>(i, gl) < D ? x[i] - rest : 0.f;
        q = fmaf(x[i], x[i], q);
    }
    const float rstd = rsqrtf(fmaf(group_sum<LPR>(q, lds), inv, eps));
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] *= rstd;
    return rstd;
}

// Where a lane works: its group, its place in it, and its walker among the tokens.
template <int LPR>
struct Place {
    int gl, group;
    bool live;
    int64_t n0, step;
    __device__ Place(const NormArgs& A) {
        constexpr int RPW = LPR < 64 ? 64 / LPR : 1;  // groups of a wave
        const int lane = threadIdx.x & 63;
        gl = (int)threadIdx.x % LPR;
        if constexpr (LPR <= 64) {
            group = (int)blockIdx.x * RPW + lane / LPR;
            n0 = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6);
            step = (int64_t)gridDim.y * 4;
        } else {
            group = (int)blockIdx.x;
            n0 = blockIdx.y;
            step = gridDim.y;
        }
        live = group < A.G;
    }
};

template <class E, int LPR, int EPL, bool WIDE, bool GATE>
__global__ __launch_bounds__(256) void group_norm_kernel(NormArgs A) {
    constexpr int VEC = WIDE ? ElemVec<E>::n : 1;
    __shared__ float lds[4];
    const Place<LPR> P(A);
    const int64_t col = (int64_t)P.group * A.D;
    float w[EPL], b[EPL];
    load_chan<LPR, EPL, VEC>(A.weight + col, P.gl, A.D, P.live, w);
    load_chan<LPR, EPL, VEC>(A.bias + col, P.gl, A.D, P.live, b);
    for (int64_t n = P.n0; n < A.N; n += P.step) {
        const int64_t at = n * A.C + col;
        float x[EPL], z[GATE ? EPL : 1];
        load_row<E, LPR, EPL, WIDE, true>(reinterpret_cast<const E*>(A.x) + at, P.gl, A.D, P.live, x);
        if constexpr (GATE)
            load_row<E, LPR, EPL, WIDE, true>(reinterpret_cast<const E*>(A.gate) + at, P.gl, A.D, P.live, z);
        normalise<LPR, EPL, VEC>(x, P.gl, A.D, A.eps, lds);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float y = fmaf(x[i], w[i], b[i]);
            const float t = GATE ? z[i] : y;
            const float a = A.act == kActSilu ? t * sigmoidf(t) : t;
            x[i] = GATE ? y * a : a;
        }
        store_row<E, LPR, EPL, WIDE>(reinterpret_cast<E*>(A.y) + at, P.gl, A.D, P.live, x);
    }
}

template <class E, int LPR, int EPL, bool WIDE, bool GATE>
__global__ __launch_bounds__(256) void group_norm_bwd_kernel(NormArgs A) {
    constexpr int VEC = WIDE ? ElemVec<E>::n : 1;
    __shared__ float lds[4];
    __shared__ float acc[LPR <= 64 ? 4 : 1][LPR <= 64 ? 64 : 1];
    const Place<LPR> P(A);
    const int64_t col = (int64_t)P.group * A.D;
    float w[EPL], b[EPL], sw[EPL], sb[EPL];
    load_chan<LPR, EPL, VEC>(A.weight + col, P.gl, A.D, P.live, w);
    load_chan<LPR, EPL, VEC>(A.bias + col, P.gl, A.D, P.live, b);
#pragma unroll
    for (int i = 0; i < EPL; ++i) sw[i] = sb[i] = 0.f;
    const float inv = 1.f / (float)A.D;
    for (int64_t n = P.n0; n < A.N; n += P.step) {
        const int64_t at = n * A.C + col;
        float x[EPL], g[EPL], z[GATE ? EPL : 1];
        load_row<E, LPR, EPL, WIDE, true>(reinterpret_cast<const E*>(A.x) + at, P.gl, A.D, P.live, x);
        load_row<E, LPR, EPL, WIDE, true>(reinterpret_cast<const E*>(A.gy) + at, P.gl, A.D, P.live, g);
        if constexpr (GATE)
            load_row<E, LPR, EPL, WIDE, true>(reinterpret_cast<const E*>(A.gate) + at, P.gl, A.D, P.live, z);
        const float rstd = normalise<LPR, EPL, VEC>(x, P.gl, A.D, A.eps, lds);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float y = fmaf(x[i], w[i], b[i]);
            const float t = GATE ? z[i] : y;
            float a = t, da = 1.f;
            if (A.act == kActSilu) {
                const float sg = sigmoidf(t);
                a = t * sg;
                da = sg * fmaf(t, 1.f - sg, 1.f);
            }
            if constexpr (GATE) z[i] = g[i] * y * da;
            const float dy = g[i] * (GATE ? a : da);
            sw[i] = fmaf(dy, x[i], sw[i]);
            sb[i] += dy;
            g[i] = dy * w[i];
            s1 += g[i];
            s2 = fmaf(g[i], x[i], s2);
        }
        s1 = group_sum<LPR>(s1, lds) * inv;
        s2 = group_sum<LPR>(s2, lds) * inv;
#pragma unroll
        for (int i = 0; i < EPL; ++i) g[i] = rstd * (g[i] - s1 - x[i] * s2);
        store_row<E, LPR, EPL, WIDE>(reinterpret_cast<E*>(A.gx) + at, P.gl, A.D, P.live, g);
        if constexpr (GATE)
            store_row<E, LPR, EPL, WIDE>(reinterpret_cast<E*>(A.ggate) + at, P.gl, A.D, P.live, z);
    }
    // This workgroup's sums: the four walkers in wave order, one channel of a lane at a time.
    float* pw = A.part + (int64_t)blockIdx.y * 2 * A.C + col;
    float* pb = pw + A.C;
#pragma unroll
    for (int i = 0; i < 2 * EPL; ++i) {
        float v = i < EPL ? sw[i % EPL] : sb[i % EPL];
        if constexpr (LPR <= 64) {
            const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
            __syncthreads();
            acc[wave][lane] = v;
            __syncthreads();
            v = acc[0][lane] + acc[1][lane] + acc[2][lane] + acc[3][lane];
            if (wave) continue;
        }
        const int c = chan<LPR, VEC>(i % EPL, P.gl);
        if (P.live && c < A.D) (i < EPL ? pw : pb)[c] = v;
    }
}

// Sum of the walkers' partial sums: column j of (rows, cols) added over the rows, 16 strips of
// rows in parallel, then the strips in order.
__global__ __launch_bounds__(256) void group_norm_fold_kernel(const float* __restrict__ part, int64_t rows, int64_t C,
                                                              float* __restrict__ gw, float* __restrict__ gb) {
    __shared__ float lds[16][17];
    const int cx = threadIdx.x & 15, strip = threadIdx.x >> 4;
    const int64_t j = (int64_t)blockIdx.x * 16 + cx;
    float s = 0.f;
    if (j < 2 * C)
#pragma unroll 4
        for (int64_t r = strip; r < rows; r += 16) s += part[r * 2 * C + j];
    lds[strip][cx] = s;
    __syncthreads();
    if (strip == 0 && j < 2 * C) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += lds[i][cx];
        if (j < C) gw[j] = s;
        else gb[j - C] = s;
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Lanes and channels per lane of a group of D channels.
struct NormPlan {
    int lpr, epl;
    int64_t gx, gy;  // grid: groups of a wave, walkers
};

NormPlan plan(int64_t N, int64_t C, int G, bool backward) {
    const int D = (int)(C / G);
    NormPlan p{};
    if (D > 2048) {
        p.lpr = 256, p.epl = 32;
    } else if (D > 512) {
        p.lpr = 64, p.epl = D > 1024 ? 32 : 16;
    } else {
        p.epl = 8, p.lpr = 4;
        while (p.lpr * 8 < D) p.lpr <<= 1;
    }
    p.gx = p.lpr <= 64 ? ceil_div(G, 64 / p.lpr) : G;
    const int64_t tokens = p.lpr <= 64 ? 4 : 1;
    // Workgroups to fill the chip, each walking as many tokens as that leaves, so that the weights are
    // loaded once for several.  Forward, five a CU: 32768 tokens of 2560 gated bfloat16 channels take
    // 96 us, 103 at 1024 and at 4096 workgroups; 8192 of 768 take 17, 17 and 32.  Backward, four a CU,
    // as its partial sums grow with them: 165 us, 260 at 512 and 177 at 2048; 8192 of 768 30, 33 and 39.
    const int64_t want = backward ? 1024 : 1280;
    p.gy = ceil_div(N, tokens);
    const int64_t cap = ceil_div(want, p.gx);
    if (p.gy > cap) p.gy = cap;
    if (p.gy > 65535) p.gy = 65535;
    return p;
}

template <class E, int LPR, int EPL, bool WIDE>
hipError_t launch(const NormArgs& A, const NormPlan& p, bool backward, hipStream_t st) {
    const dim3 grid((unsigned)p.gx, (unsigned)p.gy);
    if (backward) {
        if (A.gate) hipLaunchKernelGGL((group_norm_bwd_kernel<E, LPR, EPL, WIDE, true>), grid, dim3(256), 0, st, A);
        else hipLaunchKernelGGL((group_norm_bwd_kernel<E, LPR, EPL, WIDE, false>), grid, dim3(256), 0, st, A);
    } else {
        if (A.gate) hipLaunchKernelGGL((group_norm_kernel<E, LPR, EPL, WIDE, true>), grid, dim3(256), 0, st, A);
        else hipLaunchKernelGGL((group_norm_kernel<E, LPR, EPL, WIDE, false>), grid, dim3(256), 0, st, A);
    }
    return hipGetLastError();
}

template <class E, bool WIDE>
hipError_t by_size(const NormArgs& A, const NormPlan& p, bool backward, hipStream_t st) {
    if (p.lpr == 256) return launch<E, 256, 32, WIDE>(A, p, backward, st);
    if (p.epl == 32) return launch<E, 64, 32, WIDE>(A, p, backward, st);
    if (p.epl == 16) return launch<E, 64, 16, WIDE>(A, p, backward, st);
    switch (p.lpr) {
        case 4: return launch<E, 4, 8, WIDE>(A, p, backward, st);
        case 8: return launch<E, 8, 8, WIDE>(A, p, backward, st);
        case 16: return launch<E, 16, 8, WIDE>(A, p, backward, st);
        case 32: return launch<E, 32, 8, WIDE>(A, p, backward, st);
        default: return launch<E, 64, 8, WIDE>(A, p, backward, st);
    }
}

template <class E>
hipError_t by_alignment(const NormArgs& A, const NormPlan& p, bool backward, hipStream_t st) {
    // 16-byte accesses where every row of every tensor starts on 16 bytes.
    uintptr_t all = (uintptr_t)A.x | (uintptr_t)A.gate;
    all |= backward ? ((uintptr_t)A.gy | (uintptr_t)A.gx | (uintptr_t)A.ggate) : (uintptr_t)A.y;
    const bool wide = A.D % ElemVec<E>::n == 0 && all % 16 == 0;
    return wide ? by_size<E, true>(A, p, backward, st) : by_size<E, false>(A, p, backward, st);
}

}  // namespace

hipError_t run_group_norm(const NormArgs& A, hipStream_t st) {
    const NormPlan p = plan(A.N, A.C, A.G, false);
    return A.dtype == kBf16 ? by_alignment<bf16_t>(A, p, false, st) : by_alignment<float>(A, p, false, st);
}

size_t group_norm_backward_ws_bytes(int64_t N, int64_t C, int G) {
    return (size_t)plan(N, C, G, true).gy * 2 * (size_t)C * sizeof(float);
}

hipError_t run_group_norm_backward(const NormArgs& A, hipStream_t st) {
    const NormPlan p = plan(A.N, A.C, A.G, true);
    const hipError_t e = A.dtype == kBf16 ? by_alignment<bf16_t>(A, p, true, st) : by_alignment<float>(A, p, true, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(group_norm_fold_kernel, dim3((unsigned)ceil_div(2 * A.C, 16)), dim3(256), 0, st, A.part, p.gy,
                       A.C, A.gweight, A.gbias);
    return hipGetLastError();
}

}  // namespace linrec
