// gated_delta_step.hip -- the gated delta rule token by token, the state in registers: one
// token for decoding, a few for the shortest sequences.
//
// With m = S^T k and p = S^T q over the state before the token, and w = beta (v - a m):
//   o = scale (a p + (q.k) w),   S' = a S + k w^T
// so one reduction over the rows of S serves both products, and S is read and written once.
//
// A workgroup of 256 threads owns TV = 4*LC columns of one head's state: LC lanes across the
// columns (four each, one 16-byte load per row) and 256/LC row lanes, each holding every
// (256/LC)-th row.  LC = 8 (128-byte pieces of rows, four workgroups a head at 128 channels)
// measured no slower than 16 or 32 anywhere: 37.6, 38.1 and 39.2 us a call from Python at 64 users x
// 20 heads of 128x128 (the kernel alone 30: 5.6 TB/s), 8.9 us at one user, half of it the call.
// Sums over rows: shuffles within the wave, then the four waves' partial sums through LDS in wave
// order.  One token moves 8 Dk Dv bytes a head for 9 Dk Dv
// operations, so it is bound by memory where there are many heads and by the latency of one
// dependent load, two barriers and the launch where there are few.
#include "gated_delta.hpp"
#include "elem_types.hpp"

namespace linrec {

namespace {

// LC: lanes across columns; VEC: Dv % 4 == 0 and 16-byte aligned states.
template <class E, int LC, bool VEC>
__global__ __launch_bounds__(256) void delta_recurrent_kernel(DeltaShape s, DeltaFwdArgs A, int ntile) {
    constexpr int RG = 256 / LC;             // row lanes
    constexpr int R = kDeltaMaxDk / RG;      // rows per thread
    constexpr int TV = 4 * LC;
    __shared__ float kq[2][2][kDeltaMaxDk];  // [buffer][k, q][row]
    __shared__ float part[2][4][9][LC];      // [buffer][wave][m0..3, p0..3, qk][column lane]
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int cl = tid % LC, rl = tid / LC;
    int64_t blk = blockIdx.x;
    const int tile = (int)(blk % ntile);
    blk /= ntile;
    const int h = (int)(blk % s.Hv);
    const int64_t b = blk / s.Hv;
    const int hk = h / (s.Hv / s.Hk);
    const int Dk = s.Dk, Dv = s.Dv, c0 = tile * TV + 4 * cl;
    int64_t T = s.T;
    if (s.lengths) {
        const int64_t len = s.lengths[b];
        T = len < 0 ? 0 : (len < T ? len : T);
    }
    const int64_t sb = (b * s.Hv + h) * (int64_t)Dk * Dv;
    // This thread's 4 columns of its rows rl, rl + RG, ...
    float S[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = rl + r * RG;
#pragma unroll
        for (int j = 0; j < 4; ++j) S[r][j] = 0.f;
        if (A.s_in && row < Dk) {
            const float* p = A.s_in + sb + (int64_t)row * Dv + c0;
            if constexpr (VEC) {
                if (c0 < Dv) load16<float>(p, S[r]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c0 + j < Dv) S[r][j] = p[j];
            }
        }
    }
    for (int64_t t = 0; t < T; ++t) {
        const int buf = (int)(t & 1);
        const int64_t tk = ((b * s.T + t) * s.Hk + hk) * Dk, tv = (b * s.T + t) * s.Hv + h;
        {
            const int which = tid >> 7, row = tid & 127;
            const E* src = reinterpret_cast<const E*>(which ? A.q : A.k) + tk;
            kq[buf][which][row] = row < Dk ? (float)src[row] : 0.f;
        }
        const float a = __expf((float)reinterpret_cast<const E*>(A.g)[tv]);
        const float beta = (float)reinterpret_cast<const E*>(A.beta)[tv];
        const E* vp = reinterpret_cast<const E*>(A.v) + tv * Dv + c0;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = c0 + j < Dv ? (float)vp[j] : 0.f;
        __syncthreads();
        float sum[9] = {};
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float kk = kq[buf][0][rl + r * RG], qq = kq[buf][1][rl + r * RG];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum[j] = fmaf(S[r][j], kk, sum[j]);
                sum[4 + j] = fmaf(S[r][j], qq, sum[4 + j]);
            }
            sum[8] = fmaf(kk, qq, sum[8]);
        }
        // The wave's row lanes of one column lane sit LC lanes apart.
#pragma unroll
        for (int o = LC; o < 64; o <<= 1)
#pragma unroll
            for (int i = 0; i < 9; ++i) sum[i] += __shfl_xor(sum[i], o);
        if (lane < LC)
#pragma unroll
            for (int i = 0; i < 9; ++i) part[buf][wave][i][lane] = sum[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 9; ++i) {
            sum[i] = part[buf][0][i][cl];
#pragma unroll
            for (int w = 1; w < 4; ++w) sum[i] += part[buf][w][i][cl];
        }
        float w[4], o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = beta * fmaf(-a, sum[j], v[j]);
            o[j] = s.scale * fmaf(a, sum[4 + j], sum[8] * w[j]);
        }
        if (rl == 0) {
            E* op = reinterpret_cast<E*>(A.o) + tv * Dv + c0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c0 + j < Dv) op[j] = (E)o[j];
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float kk = kq[buf][0][rl + r * RG];
#pragma unroll
            for (int j = 0; j < 4; ++j) S[r][j] = fmaf(kk, w[j], a * S[r][j]);
        }
        // The other buffer pair is written next; this one two tokens on, past two barriers.
    }
    // Absent tokens: zero outputs.
    if (rl == 0)
        for (int64_t t = T; t < s.T; ++t) {
            E* op = reinterpret_cast<E*>(A.o) + ((b * s.T + t) * s.Hv + h) * Dv + c0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c0 + j < Dv) op[j] = (E)0.f;
        }
    if (A.s_out) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = rl + r * RG;
            if (row >= Dk) continue;
            float* p = A.s_out + sb + (int64_t)row * Dv + c0;
            if constexpr (VEC) {
                if (c0 < Dv) store16<float>(p, S[r]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c0 + j < Dv) p[j] = S[r][j];
            }
        }
    }
}

template <class E>
hipError_t launch(const DeltaShape& s, const DeltaFwdArgs& A, hipStream_t st) {
    constexpr int LC = 8;
    const int ntile = (s.Dv + 4 * LC - 1) / (4 * LC);
    const int64_t nb = s.B * s.Hv * ntile;
    const bool vec = s.Dv % 4 == 0 && ((uintptr_t)A.s_in % 16) == 0 && ((uintptr_t)A.s_out % 16) == 0;
    if (vec)
        hipLaunchKernelGGL((delta_recurrent_kernel<E, LC, true>), dim3((unsigned)nb), dim3(256), 0, st, s, A, ntile);
    else
        hipLaunchKernelGGL((delta_recurrent_kernel<E, LC, false>), dim3((unsigned)nb), dim3(256), 0, st, s, A, ntile);
    return hipGetLastError();
}

}  // namespace

hipError_t run_delta_recurrent(const DeltaShape& s, const DeltaFwdArgs& A, hipStream_t st) {
    return s.dtype == kBf16 ? launch<bf16_t>(s, A, st) : launch<float>(s, A, st);
}

}  // namespace linrec
