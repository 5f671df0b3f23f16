// selective_scan.hip -- the selective state space scan, forward and for one token.
//
//   d_t = softplus(dt_t + bias),  h_t[n] = e^{d_t A[n]} h_{t-1}[n] + d_t u_t B_t[n],
//   y_t = (sum_n C_t[n] h_t[n] + D u_t) silu(z_t)
//
// Nothing is shared between channels but B_t and C_t, so there is no matrix product in it: each
// state takes an exponential (a quarter of the rate) and four multiply-adds, and with 16 states a
// channel that, and not the few bytes of u, dt, z and y, is what bounds it.
//
// A workgroup owns 64 channels of one group and one segment of the tokens.  Lane = channel; wave w
// holds the states w*NPT .. w*NPT+NPT-1 of every channel in registers and walks down the tokens.  B_t
// and C_t are the same for all lanes: they come by scalar loads, in float32 (a small kernel before this
// one lays them out), and cost no vector instruction.  What depends on the channel alone (the
// softplus, d u, the gate) is formed once per token, 16 tokens at a time and 16/W by each wave,
// and goes to the waves through LDS; the waves' shares of y come back the same way and are added in
// wave order.
//
// Where the rows and channels are too few to fill the chip, the rows are cut into segments: each
// segment's state from a zero state, and the sum of its steps (the decay over a segment is e^{A sum}),
// then the states that enter the segments one after the other, then the segments again from those.
#include "selective_math.hpp"

namespace linrec {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// B and C as float32, (B,T,G,W,2,NPT), zero beyond N and for absent tokens.
template <class E>
__global__ __launch_bounds__(256) void sel_prepare_kernel(SelShape s, const E* __restrict__ Bm,
                                                          const E* __restrict__ Cm, float* __restrict__ bc, int npt,
                                                          int np, int64_t total) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int j = (int)(i % (2 * np));
        const int64_t tok = i / (2 * np) / s.G;  // b * T + t
        const int w = j / (2 * npt), r = j % (2 * npt);
        const int n = w * npt + r % npt;
        const int64_t b = tok / s.T;
        float v = 0.f;
        if (n < s.N && tok - b * s.T < row_length(s, b)) v = (float)(r < npt ? Bm : Cm)[i / (2 * np) * s.N + n];
        bc[i] = v;
    }
}

// AGG: the segment's state from zero, and the sum of its steps, instead of outputs.
template <class E, int W, int NPT, bool AGG>
__global__ __launch_bounds__(64 * W) void sel_forward_kernel(SelShape s, SelArgs A, const float* __restrict__ bc,
                                                             float* __restrict__ agg, float* __restrict__ sum,
                                                             float* __restrict__ keep, int64_t segs,
                                                             int64_t seg_tiles, int group_tiles) {
    constexpr int TW = kSelTile / W;  // tokens a wave stages
    __shared__ f32x2 din[kSelTile][64];                       // d, d u
    __shared__ float part[AGG ? 1 : W][AGG ? 1 : kSelTile][64];  // the waves' shares of y
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t blk = blockIdx.x;
    const int tile = (int)(blk % (s.G * group_tiles));
    blk /= s.G * group_tiles;
    const int64_t seg = blk % segs, b = blk / segs;
    const int grp = tile / group_tiles, Cg = (int)(s.C / s.G);
    const int in_group = (tile % group_tiles) * 64 + lane;
    const bool live = in_group < Cg;
    const int64_t c = (int64_t)grp * Cg + (live ? in_group : Cg - 1);
    const int64_t t_begin = seg * seg_tiles * kSelTile;
    const int64_t t_end = seg == segs - 1 ? s.T : t_begin + seg_tiles * kSelTile;
    const int64_t len = row_length(s, b);
    const bool last = seg == segs - 1;
    const int n0 = w * NPT, Np = (s.N + 3) / 4 * 4;

    float h[NPT], a2[NPT];
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        const int n = n0 + i;
        a2[i] = n < s.N ? A.A[c * s.N + n] * kLog2e : 0.f;
        h[i] = 0.f;
        if (!AGG && n < s.N) {
            if (segs > 1) h[i] = agg[state_at(s, b * segs + seg, n, c)];
            else if (A.s_in) h[i] = A.s_in[(b * s.C + c) * s.N + n];
        }
    }
    const float bias = A.bias ? A.bias[c] : 0.f;
    const float Dc = A.D ? A.D[c] : 0.f;
    float total = 0.f;

    for (int64_t t0 = t_begin; t0 < t_end; t0 += kSelTile) {
        if constexpr (!AGG) {
            if (keep && live) {
#pragma unroll
                for (int i = 0; i < NPT; ++i)
                    if (n0 + i < Np)
                        keep[state_at(s, b * ((s.T + kSelTile - 1) / kSelTile) + t0 / kSelTile, n0 + i, c)] = h[i];
            }
        }
        // This wave's tokens of the tile.
        float u[TW], z[TW];
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const int64_t t = t0 + w * TW + i;
            const bool there = live && t < len && t < t_end;
            const int64_t at = (b * s.T + t) * s.C + c;
            u[i] = z[i] = 0.f;
            float d = 0.f;
            if (there) {
                u[i] = (float)reinterpret_cast<const E*>(A.u)[at];
                d = (float)reinterpret_cast<const E*>(A.dt)[at] + bias;
                if (!AGG && A.z) z[i] = (float)reinterpret_cast<const E*>(A.z)[at];
                float sig;
                if (s.softplus) d = softplus(d, sig);
            }
            const f32x2 v = {d, d * u[i]};
            din[w * TW + i][lane] = v;
        }
        __syncthreads();
        const float* row = bc + (((b * s.T + t0) * s.G + grp) * W + w) * (2 * NPT);
        const int64_t row_step = (int64_t)s.G * W * (2 * NPT);
        const int m = t_end - t0 < kSelTile ? (int)(t_end - t0) : kSelTile;
        float subtotal = 0.f;
        for (int t = 0; t < m; ++t) {
            float v[2 * NPT];
            load_uniform<2 * NPT>(row + t * row_step, v);
            const f32x2 x = din[t][lane];
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < NPT; ++i) {
                h[i] = fmaf(fast_exp2(x[0] * a2[i]), h[i], x[1] * v[i]);
                y = fmaf(v[NPT + i], h[i], y);
            }
            if constexpr (AGG) subtotal += x[0];
            else part[w][t][lane] = y;
        }
        total += subtotal;
        __syncthreads();
        if constexpr (!AGG) {
            if (A.y && live) {
#pragma unroll
                for (int i = 0; i < TW; ++i) {
                    const int64_t t = t0 + w * TW + i;
                    if (t >= t_end) break;
                    float y = Dc * u[i];
#pragma unroll
                    for (int k = 0; k < W; ++k) y += part[k][w * TW + i][lane];
                    if (A.z) y *= z[i] * logistic(z[i]);
                    reinterpret_cast<E*>(A.y)[(b * s.T + t) * s.C + c] = (E)(t < len ? y : 0.f);
                }
            }
        }
    }
    if (!live) return;
    if constexpr (AGG) {
#pragma unroll
        for (int i = 0; i < NPT; ++i)
            if (n0 + i < Np) agg[state_at(s, b * segs + seg, n0 + i, c)] = h[i];
        if (w == 0) sum[(b * segs + seg) * s.C + c] = total;
    } else if (last && A.s_out) {
#pragma unroll
        for (int i = 0; i < NPT; ++i)
            if (n0 + i < s.N) A.s_out[(b * s.C + c) * s.N + n0 + i] = h[i];
    }
}

// One element of every state and row: the blocks' shares become the states that enter them.
template <bool REV>
__global__ __launch_bounds__(256) void sel_join_kernel(SelShape s, const float* __restrict__ A, float* __restrict__ v,
                                                       const float* __restrict__ sum, int64_t blocks,
                                                       const float* in, float* out) {
    const int64_t per = (int64_t)((s.N + 3) / 4) * 4 * s.C;
    const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (j >= s.B * per) return;
    const int64_t b = j / per, e = j % per;
    const int64_t c = e / 4 % s.C;
    const int n = (int)(e / (4 * s.C)) * 4 + (int)(e & 3);
    const int64_t at = (b * s.C + c) * s.N + n;
    const float a2 = n < s.N ? A[c * s.N + n] * kLog2e : 0.f;
    float x = in && n < s.N ? in[at] : 0.f;
    for (int64_t i = 0; i < blocks; ++i) {
        const int64_t k = b * blocks + (REV ? blocks - 1 - i : i);
        const float own = v[k * per + e];
        v[k * per + e] = x;
        x = fmaf(fast_exp2(a2 * sum[k * s.C + c]), x, own);
    }
    if (out && n < s.N) out[at] = x;
}

// One token: LN lanes a channel, four states each.
template <class E, bool VEC>
__global__ __launch_bounds__(256) void sel_step_kernel(SelShape s, SelArgs A, int ln) {
    const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = j / ln;  // b * C + c
    const int n0 = (int)(j % ln) * 4;
    const bool live = row < s.B * s.C;
    const int64_t b = live ? row / s.C : 0, c = live ? row % s.C : 0;
    float y = 0.f, u = 0.f;
    if (live) {
        u = (float)reinterpret_cast<const E*>(A.u)[row];
        float d = (float)reinterpret_cast<const E*>(A.dt)[row] + (A.bias ? A.bias[c] : 0.f), sig;
        if (s.softplus) d = softplus(d, sig);
        const int64_t bg = (b * s.G + c / (s.C / s.G)) * s.N;
        const E* Bm = reinterpret_cast<const E*>(A.Bm) + bg;
        const E* Cm = reinterpret_cast<const E*>(A.Cm) + bg;
        float h[4], a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = a[i] = 0.f;
        if constexpr (VEC) {
            if (n0 < s.N) {
                load16<float>(A.A + c * s.N + n0, a);
                if (A.s_in) load16<float>(A.s_in + row * s.N + n0, h);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n0 + i < s.N) {
                    a[i] = A.A[c * s.N + n0 + i];
                    if (A.s_in) h[i] = A.s_in[row * s.N + n0 + i];
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (n0 + i >= s.N) continue;
            h[i] = fmaf(fast_exp2(d * (a[i] * kLog2e)), h[i], d * u * (float)Bm[n0 + i]);
            y = fmaf((float)Cm[n0 + i], h[i], y);
        }
        if constexpr (VEC) {
            if (n0 < s.N) store16<float>(A.s_out + row * s.N + n0, h);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n0 + i < s.N) A.s_out[row * s.N + n0 + i] = h[i];
        }
    }
    for (int o = 1; o < ln; o <<= 1) y += __shfl_xor(y, o);
    if (live && n0 == 0) {
        if (A.D) y = fmaf(A.D[c], u, y);
        if (A.z) {
            const float z = (float)reinterpret_cast<const E*>(A.z)[row];
            y *= z * logistic(z);
        }
        reinterpret_cast<E*>(A.y)[row] = (E)y;
    }
}

template <class E, int W, int NPT>
hipError_t forward(const SelShape& s, const SelArgs& A, const SelPlan& p, const SelScratch& S, float* keep,
                   hipStream_t st) {
    const int group_tiles = (int)ceil_div(s.C / s.G, 64);
    const dim3 grid((unsigned)(s.B * p.segs * s.G * group_tiles));
    if (p.segs > 1) {
        hipLaunchKernelGGL((sel_forward_kernel<E, W, NPT, true>), grid, dim3(64 * W), 0, st, s, A, S.bc, S.agg, S.sum,
                           (float*)nullptr, p.segs, p.seg_tiles, group_tiles);
        hipError_t e = hipGetLastError();
        if (e == hipSuccess) e = run_sel_join(s, A.A, S.agg, S.sum, p.segs, A.s_in, nullptr, false, st);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((sel_forward_kernel<E, W, NPT, false>), grid, dim3(64 * W), 0, st, s, A, S.bc, S.agg, S.sum,
                       keep, p.segs, p.seg_tiles, group_tiles);
    return hipGetLastError();
}

template <class E>
hipError_t forward_by_states(const SelShape& s, const SelArgs& A, const SelPlan& p, const SelScratch& S, float* keep,
                             hipStream_t st) {
    if (p.npt == 1) return forward<E, 1, 1>(s, A, p, S, keep, st);
    if (p.npt == 2) return forward<E, 1, 2>(s, A, p, S, keep, st);
    if (p.npt == 4) {
        if (p.waves == 1) return forward<E, 1, 4>(s, A, p, S, keep, st);
        if (p.waves == 2) return forward<E, 2, 4>(s, A, p, S, keep, st);
        return forward<E, 4, 4>(s, A, p, S, keep, st);
    }
    if (p.npt == 8) return p.waves == 4 ? forward<E, 4, 8>(s, A, p, S, keep, st) : forward<E, 8, 8>(s, A, p, S, keep, st);
    return forward<E, 8, 16>(s, A, p, S, keep, st);
}

}  // namespace

SelPlan sel_plan(const SelShape& s) {
    SelPlan p{};
    p.npt = s.N <= 1 ? 1 : s.N <= 2 ? 2 : s.N <= 16 ? 4 : s.N <= 64 ? 8 : 16;
    p.waves = s.N <= 4 ? 1 : s.N <= 8 ? 2 : s.N <= 32 ? 4 : 8;
    // Segments until the chip has four waves a SIMD, of four tiles at least.
    const int64_t wg = s.B * s.G * ceil_div(s.C / s.G, 64), tiles = sel_tiles(s);
    int64_t segs = 4096 / (wg * p.waves);
    if (segs > tiles / 4) segs = tiles / 4;
    if (segs < 2) segs = 1;
    p.seg_tiles = ceil_div(tiles, segs);
    p.segs = ceil_div(tiles, p.seg_tiles);
    return p;
}

size_t sel_bc_floats(const SelShape& s, const SelPlan& p) {
    return (size_t)(s.B * s.T * s.G) * 2 * (size_t)(p.npt * p.waves);
}

hipError_t run_sel_prepare(const SelShape& s, const SelArgs& A, const SelPlan& p, const SelScratch& W, hipStream_t st) {
    const int64_t total = (int64_t)sel_bc_floats(s, p);
    int64_t blocks = ceil_div(total, 256);
    if (blocks > 4096) blocks = 4096;
    const int np = p.npt * p.waves;
    if (s.dtype == kBf16)
        hipLaunchKernelGGL((sel_prepare_kernel<bf16_t>), dim3((unsigned)blocks), dim3(256), 0, st, s,
                           (const bf16_t*)A.Bm, (const bf16_t*)A.Cm, W.bc, p.npt, np, total);
    else
        hipLaunchKernelGGL((sel_prepare_kernel<float>), dim3((unsigned)blocks), dim3(256), 0, st, s,
                           (const float*)A.Bm, (const float*)A.Cm, W.bc, p.npt, np, total);
    return hipGetLastError();
}

hipError_t run_sel_forward(const SelShape& s, const SelArgs& A, const SelPlan& p, const SelScratch& W, float* keep,
                           hipStream_t st) {
    return s.dtype == kBf16 ? forward_by_states<bf16_t>(s, A, p, W, keep, st)
                            : forward_by_states<float>(s, A, p, W, keep, st);
}

hipError_t run_sel_join(const SelShape& s, const float* A, float* v, const float* sum, int64_t blocks, const float* in,
                        float* out, bool reverse, hipStream_t st) {
    const dim3 grid((unsigned)ceil_div(s.B * sel_n4(s) * 4 * s.C, 256));
    if (reverse) hipLaunchKernelGGL((sel_join_kernel<true>), grid, dim3(256), 0, st, s, A, v, sum, blocks, in, out);
    else hipLaunchKernelGGL((sel_join_kernel<false>), grid, dim3(256), 0, st, s, A, v, sum, blocks, in, out);
    return hipGetLastError();
}

hipError_t run_sel_step(const SelShape& s, const SelArgs& A, hipStream_t st) {
    int ln = 1;
    while (4 * ln < s.N) ln *= 2;
    const dim3 grid((unsigned)ceil_div(s.B * s.C * ln, 256));
    const bool vec = s.N % 4 == 0 && ((uintptr_t)A.A | (uintptr_t)A.s_in | (uintptr_t)A.s_out) % 16 == 0;
    if (s.dtype == kBf16) {
        if (vec) hipLaunchKernelGGL((sel_step_kernel<bf16_t, true>), grid, dim3(256), 0, st, s, A, ln);
        else hipLaunchKernelGGL((sel_step_kernel<bf16_t, false>), grid, dim3(256), 0, st, s, A, ln);
    } else {
        if (vec) hipLaunchKernelGGL((sel_step_kernel<float, true>), grid, dim3(256), 0, st, s, A, ln);
        else hipLaunchKernelGGL((sel_step_kernel<float, false>), grid, dim3(256), 0, st, s, A, ln);
    }
    return hipGetLastError();
}

}  // namespace linrec
