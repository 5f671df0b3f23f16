// rms_norm.hip -- the root-mean-square norm of each token's channels behind the addition of the
// residual, and its gradients; x (N,C), the channels last.
//
//   s = x + r (stored in r's type),  n = s / sqrt(mean(s^2) + eps),  y = n w
//
// The norm is that of s as stored, so that the backward, which starts from the stored s, is
// its gradient.  With rstd = 1/sqrt(mean(s^2) + eps) and v = gy w:
//   gs = gsum + rstd (v - n mean(v n)),  gw = sum_tokens gy n
// gs is the gradient of x and of r alike.
//
// LPR lanes hold a token's row, 8 NV channels each in registers: one pass over memory.  A wave
// (LPR 64) or a workgroup (LPR 256) walks down the tokens with its weights, and backwards its sums
// of gw, in registers; the walkers' sums go to the workspace and are added in walker order.  Bound by
// memory: the next row is on its way while one is worked on, without which the backward took 277 us
// for 113 (32768 tokens of 2560 bfloat16 channels), four barriers a row between its loads.
#include "rms_norm.hpp"
#include "row_ops.hpp"

namespace linrec {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Sum over the LPR lanes of a row, the same bits in every lane.  In a workgroup of several waves two
// sums in a row use `lds` of their own, so that one barrier each is enough.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* lds) {
    v = add_dpp<0xb1>(v);   // quad_perm [1,0,3,2]
    v = add_dpp<0x4e>(v);   // quad_perm [2,3,0,1]
    v = add_dpp<0x141>(v);  // row_half_mirror
    v = add_dpp<0x140>(v);  // row_mirror
    if constexpr (LPR > 16) {
        const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
        const u32x2 p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if constexpr (LPR > 64) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = lds[0];
#pragma unroll
        for (int w = 1; w < LPR / 64; ++w) v += lds[w];
    }
    return v;
}

// Channels of a lane: 8 neighbouring ones from each of NV stretches of LPR * 8.
template <int LPR>
__device__ __forceinline__ int chan(int i, int rl) { return (i / 8) * (LPR * 8) + rl * 8 + i % 8; }

// A lane's 8 NV elements of a row, as they come from memory: asked for a row ahead.
template <int TYPE, int LPR, int NV, bool WIDE>
struct RawRow {
    static constexpr int kWords = TYPE == kBf16 ? 1 : 2;  // 16-byte words of 8 elements
    u32x4 v[WIDE ? NV * kWords : 1];
    float f[WIDE ? 1 : 8 * NV];
    __device__ __forceinline__ void load(const void* p, int64_t at, int rl, int C) {
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = chan<LPR>(8 * i, rl);
#pragma unroll
                for (int k = 0; k < kWords; ++k) {
                    const u32x4* const q = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(p) + (at + c) * (2 * kWords)) + k;
                    if (c < C) v[i * kWords + k] = __builtin_nontemporal_load(q);
                    else v[i * kWords + k] = u32x4{0u, 0u, 0u, 0u};
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8 * NV; ++i) {
                const int c = chan<LPR>(i, rl);
                f[i] = c >= C ? 0.f
                       : TYPE == kBf16 ? (float)reinterpret_cast<const bf16_t*>(p)[at + c]
                                       : reinterpret_cast<const float*>(p)[at + c];
            }
        }
    }
    __device__ __forceinline__ void get(float (&out)[8 * NV]) const {
#pragma unroll
        for (int i = 0; i < 8 * NV; ++i) {
            if constexpr (!WIDE) out[i] = f[i];
            else if constexpr (TYPE == kBf16) out[i] = __uint_as_float(i & 1 ? v[i / 8][i % 8 / 2] & 0xffff0000u : v[i / 8][i % 8 / 2] << 16);
            else out[i] = __uint_as_float(v[i / 4][i % 4]);
        }
    }
};

template <int LPR, int NV, bool WIDE>
__device__ __forceinline__ void store_row(void* p, int type, int64_t at, int rl, int C, const float (&in)[8 * NV]) {
#pragma unroll
    for (int i = 0; i < 8 * NV; i += 8) {
        const int c = chan<LPR>(i, rl);
        if constexpr (WIDE) {
            if (c >= C) continue;
            if (type == kBf16) {
                store16<bf16_t, true>(reinterpret_cast<bf16_t*>(p) + at + c, in + i);
            } else {
                store16<float, true>(reinterpret_cast<float*>(p) + at + c, in + i);
                store16<float, true>(reinterpret_cast<float*>(p) + at + c + 4, in + i + 4);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (c + j >= C) continue;
                if (type == kBf16) reinterpret_cast<bf16_t*>(p)[at + c + j] = (bf16_t)in[i + j];
                else reinterpret_cast<float*>(p)[at + c + j] = in[i + j];
            }
        }
    }
}

template <int LPR, int NV>
__device__ __forceinline__ void load_weight(const float* __restrict__ p, int rl, int C, float (&out)[8 * NV]) {
#pragma unroll
    for (int i = 0; i < 8 * NV; ++i) {
        const int c = chan<LPR>(i, rl);
        out[i] = c < C ? p[c] : 0.f;
    }
}

// Where a lane works: its place in the row, and its walker among the tokens.
template <int LPR>
struct Walk {
    int rl;
    int64_t first, step;
    __device__ Walk() {
        constexpr int R = 256 / LPR;  // rows of a workgroup
        rl = (int)threadIdx.x % LPR;
        first = (int64_t)blockIdx.x * R + threadIdx.x / LPR;
        step = (int64_t)gridDim.x * R;
    }
};

template <int DT, int RT, int LPR, int NV, bool WIDE, bool RES>
__global__ __launch_bounds__(256) void rms_norm_kernel(RmsArgs A) {
    __shared__ float lds[2][4];
    const Walk<LPR> P;
    const int C = (int)A.C;
    const float inv = 1.f / (float)C;
    RawRow<DT, LPR, NV, WIDE> nx;
    RawRow<RT, LPR, NV, WIDE> nr;
    const auto fetch = [&](int64_t n) {
        nx.load(A.x, n * A.C, P.rl, C);
        if constexpr (RES) nr.load(A.res, n * A.C, P.rl, C);
    };
    if (P.first < A.N) fetch(P.first);
    float w[8 * NV];
    load_weight<LPR, NV>(A.weight, P.rl, C, w);
    int turn = 0;
    for (int64_t n = P.first; n < A.N; n += P.step, turn ^= 1) {
        float x[8 * NV], r[8 * NV];
        nx.get(x);
        if constexpr (RES) nr.get(r);
        if (n + P.step < A.N) fetch(n + P.step);
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < 8 * NV; ++i) {
                x[i] += r[i];
                if constexpr (RT == kBf16) x[i] = (float)(bf16_t)x[i];
            }
            store_row<LPR, NV, WIDE>(A.sum, RT, n * A.C, P.rl, C, x);
        }
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < 8 * NV; ++i) q = fmaf(x[i], x[i], q);
        const float rstd = rsqrtf(fmaf(row_sum<LPR>(q, lds[turn]), inv, A.eps));
#pragma unroll
        for (int i = 0; i < 8 * NV; ++i) x[i] = x[i] * rstd * w[i];
        store_row<LPR, NV, WIDE>(A.y, DT, n * A.C, P.rl, C, x);
    }
}

template <int DT, int RT, int LPR, int NV, bool WIDE, bool GSUM>
__global__ __launch_bounds__(256) void rms_norm_bwd_kernel(RmsArgs A) {
    constexpr int R = 256 / LPR;
    __shared__ float lds[2][4];
    __shared__ float acc[R > 1 ? 256 : 1];
    const Walk<LPR> P;
    const int C = (int)A.C;
    const float inv = 1.f / (float)C;
    RawRow<RT, LPR, NV, WIDE> ns, ng;
    RawRow<DT, LPR, NV, WIDE> ny;
    const auto fetch = [&](int64_t n) {
        ns.load(A.s, n * A.C, P.rl, C);
        ny.load(A.gy, n * A.C, P.rl, C);
        if constexpr (GSUM) ng.load(A.gsum, n * A.C, P.rl, C);
    };
    if (P.first < A.N) fetch(P.first);
    float w[8 * NV], gw[8 * NV];
    load_weight<LPR, NV>(A.weight, P.rl, C, w);
#pragma unroll
    for (int i = 0; i < 8 * NV; ++i) gw[i] = 0.f;
    for (int64_t n = P.first; n < A.N; n += P.step) {
        float x[8 * NV], v[8 * NV], r[8 * NV];
        ns.get(x);
        ny.get(v);
        if constexpr (GSUM) ng.get(r);
        if (n + P.step < A.N) fetch(n + P.step);
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < 8 * NV; ++i) q = fmaf(x[i], x[i], q);
        const float rstd = rsqrtf(fmaf(row_sum<LPR>(q, lds[0]), inv, A.eps));
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8 * NV; ++i) {
            x[i] *= rstd;
            gw[i] = fmaf(v[i], x[i], gw[i]);
            v[i] *= w[i];
            m = fmaf(v[i], x[i], m);
        }
        m = row_sum<LPR>(m, lds[1]) * inv;
#pragma unroll
        for (int i = 0; i < 8 * NV; ++i) {
            v[i] = rstd * fmaf(-x[i], m, v[i]);
            if constexpr (GSUM) v[i] += r[i];
        }
        store_row<LPR, NV, WIDE>(A.gs, RT, n * A.C, P.rl, C, v);
        if (DT != RT && A.gx) store_row<LPR, NV, WIDE>(A.gx, DT, n * A.C, P.rl, C, v);
    }
    // This workgroup's sums, the rows' walkers in order.
    float* const part = A.part + (int64_t)blockIdx.x * A.C;
#pragma unroll
    for (int i = 0; i < 8 * NV; ++i) {
        float v = gw[i];
        const int c = chan<LPR>(i, P.rl);
        if constexpr (R > 1) {
            __syncthreads();
            acc[threadIdx.x] = v;
            __syncthreads();
            if ((int)threadIdx.x >= LPR) continue;
#pragma unroll
            for (int k = 1; k < R; ++k) v += acc[k * LPR + threadIdx.x];
        }
        if (c < C) part[c] = v;
    }
}

// Sum of the walkers' partial sums, 16 strips of walkers at once, then the strips in order.
__global__ __launch_bounds__(256) void rms_norm_fold_kernel(const float* __restrict__ part, int64_t rows, int64_t C,
                                                            float* __restrict__ gw) {
    __shared__ float lds[16][17];
    const int64_t j = (int64_t)blockIdx.x * 16 + (threadIdx.x & 15);
    const float v = fold_column(part, rows, C, j, lds);
    if (threadIdx.x < 16 && j < C) gw[j] = v;
}

struct RmsPlan {
    int lpr, nv;
    int64_t wg;
};

RmsPlan plan(int64_t N, int64_t C, bool backward) {
    RmsPlan p{};
    p.lpr = C <= 128 ? 16 : C <= 1024 ? 64 : 256;
    p.nv = C <= 512 ? 1 : C <= 1024 ? 2 : C <= 2048 ? 1 : C <= 4096 ? 2 : 4;
    p.wg = ceil_div(N, 256 / p.lpr);
    // Two workgroups a CU, backward three, each with its next row on its way while it works on one: 32768
    // tokens of 2560 bfloat16 channels take 111 us forward (6.0 TB/s; 124 and 128 with four and eight) and 113
    // backward (5.9; 122 and 140 with two and four).
    const int64_t most = backward ? 768 : 512;
    if (p.wg > most) p.wg = most;
    return p;
}

template <int DT, int RT, int LPR, int NV, bool WIDE>
hipError_t launch(const RmsArgs& A, const RmsPlan& p, bool backward, hipStream_t st) {
    const dim3 grid((unsigned)p.wg);
    if (!backward) {
        if (A.res) hipLaunchKernelGGL((rms_norm_kernel<DT, RT, LPR, NV, WIDE, true>), grid, dim3(256), 0, st, A);
        else hipLaunchKernelGGL((rms_norm_kernel<DT, RT, LPR, NV, WIDE, false>), grid, dim3(256), 0, st, A);
    } else {
        if (A.gsum) hipLaunchKernelGGL((rms_norm_bwd_kernel<DT, RT, LPR, NV, WIDE, true>), grid, dim3(256), 0, st, A);
        else hipLaunchKernelGGL((rms_norm_bwd_kernel<DT, RT, LPR, NV, WIDE, false>), grid, dim3(256), 0, st, A);
    }
    return hipGetLastError();
}

template <int DT, int RT, bool WIDE>
hipError_t by_size(const RmsArgs& A, const RmsPlan& p, bool backward, hipStream_t st) {
    if (p.lpr == 16) return launch<DT, RT, 16, 1, WIDE>(A, p, backward, st);
    if (p.lpr == 64 && p.nv == 1) return launch<DT, RT, 64, 1, WIDE>(A, p, backward, st);
    if (p.lpr == 64) return launch<DT, RT, 64, 2, WIDE>(A, p, backward, st);
    if (p.nv == 1) return launch<DT, RT, 256, 1, WIDE>(A, p, backward, st);
    if (p.nv == 2) return launch<DT, RT, 256, 2, WIDE>(A, p, backward, st);
    return launch<DT, RT, 256, 4, WIDE>(A, p, backward, st);
}

template <int DT, int RT>
hipError_t by_alignment(const RmsArgs& A, bool backward, hipStream_t st) {
    // 16-byte accesses where every lane's 8 channels of every tensor start on 16 bytes.
    const RmsPlan p = plan(A.N, A.C, backward);
    uintptr_t all = backward ? ((uintptr_t)A.s | (uintptr_t)A.gy | (uintptr_t)A.gsum | (uintptr_t)A.gx | (uintptr_t)A.gs)
                             : ((uintptr_t)A.x | (uintptr_t)A.res | (uintptr_t)A.y | (uintptr_t)A.sum);
    const bool wide = A.C % 8 == 0 && all % 16 == 0;
    return wide ? by_size<DT, RT, true>(A, p, backward, st) : by_size<DT, RT, false>(A, p, backward, st);
}

hipError_t by_type(const RmsArgs& A, bool backward, hipStream_t st) {
    if (A.dtype == kF32) return by_alignment<kF32, kF32>(A, backward, st);
    if (A.rtype == kF32) return by_alignment<kBf16, kF32>(A, backward, st);
    return by_alignment<kBf16, kBf16>(A, backward, st);
}

}  // namespace

hipError_t run_rms_norm(const RmsArgs& A, hipStream_t st) { return by_type(A, false, st); }

size_t rms_norm_backward_ws_bytes(int64_t N, int64_t C) {
    return (size_t)plan(N, C, true).wg * (size_t)C * sizeof(float);
}

hipError_t run_rms_norm_backward(const RmsArgs& A, hipStream_t st) {
    const hipError_t e = by_type(A, true, st);
    if (e != hipSuccess) return e;
    const RmsPlan p = plan(A.N, A.C, true);
    hipLaunchKernelGGL(rms_norm_fold_kernel, dim3((unsigned)ceil_div(A.C, 16)), dim3(256), 0, st, A.part, p.wg, A.C,
                       A.gweight);
    return hipGetLastError();
}

}  // namespace linrec
