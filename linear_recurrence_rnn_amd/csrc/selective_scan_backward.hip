// selective_scan_backward.hip -- gradients of the selective state space scan.
//
// With p_t = gy_t silu(z_t) the gradient of the ungated output and G_t the gradient that enters token
// t from its right (G_{T-1} = gs_out):
//   g_t[n] = C_t[n] p_t + G_t[n],   G_{t-1}[n] = a_t[n] g_t[n],   a_t[n] = e^{d_t A[n]}
//   m_t[n] = G_{t-1}[n] h_{t-1}[n]
//   gC_t[n] = sum_c p_t h_t[n],     gB_t[n] = sum_c g_t[n] d_t u_t       (over a group's channels)
//   gd_t = sum_n A[n] m_t[n] + u_t sum_n g_t[n] B_t[n],   gA[n] = sum_t d_t m_t[n]
//   gu_t = D p_t + d_t sum_n g_t[n] B_t[n],   gD = sum_t p_t u_t
//   gdt_t = gd_t softplus'(dt_t + bias),  gbias = sum_t gdt_t,  gz_t = gy_t core_t silu'(z_t)
//
// The rows are cut into blocks of 64 tokens.  First each block's share of the G that leaves it on
// the left, from zero on its right (all blocks at once, as the forward's segments); then the G that
// enters each block, one block after the other (the decay over a block is e^{A sum d}); then all gradients,
// all blocks at once, the states formed again from those the forward kept every 16 tokens.
//
// The last kernel sums over states (for each token and channel) and over channels (for each token
// and state).  A wave holds 8 channels x 8 NT states, lane = 8 (state) + channel: sums over states go
// across lane bits 3 to 5, 16 tokens at once, each step halving the tokens a lane holds, so that
// they end at the lane that has the token's own inputs.  Sums over channels are kept per lane for the
// 16 tokens and over all channel sets the wave walks through, and cross its 8 channel lanes once.
// Sums over blocks, batch rows and channel ranges are partial sums in the workspace, added in
// order by small kernels at the end: nothing depends on timing.
#include "selective_math.hpp"

namespace linrec {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The G that leaves each block on its left, from zero, and the sum of its steps.
template <class E, int W, int NPT>
__global__ __launch_bounds__(64 * W) void sel_reverse_kernel(SelShape s, SelArgs A, const E* __restrict__ gy,
                                                             const float* __restrict__ bc, float* __restrict__ out,
                                                             float* __restrict__ sum, int blocks, int group_tiles) {
    constexpr int TW = kSelTile / W;
    __shared__ f32x2 din[kSelTile][64];  // d, p
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    unsigned blk = blockIdx.x;
    const int tile = (int)(blk % (unsigned)(s.G * group_tiles));
    blk /= (unsigned)(s.G * group_tiles);
    const int k = (int)(blk % (unsigned)blocks);
    const int64_t b = blk / (unsigned)blocks;
    const int grp = tile / group_tiles, Cg = (int)(s.C / s.G);
    const int in_group = (tile % group_tiles) * 64 + lane;
    const bool live = in_group < Cg;
    const unsigned c = (unsigned)(grp * Cg + (live ? in_group : Cg - 1));
    const int T = (int)s.T, tiles = (T + kSelTile - 1) / kSelTile;
    const int t_begin = k * kSelBlock, len = (int)row_length(s, b);
    const int n0 = w * NPT, Np = (s.N + 3) / 4 * 4;
    float g[NPT], a2[NPT];
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        g[i] = 0.f;
        a2[i] = n0 + i < s.N ? A.A[(int64_t)c * s.N + n0 + i] * kLog2e : 0.f;
    }
    const float bias = A.bias ? A.bias[c] : 0.f;
    float total = 0.f;
    // This wave's tokens of a tile, read while the tile behind it is worked on.  Tokens behind the
    // row's end are read as the last one and not used.
    E dr[TW], zr[TW], gr[TW];
    const auto fetch = [&](int t0) {
        const int64_t base = (b * T + t0) * s.C;
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const int last = T - 1 - t0, j = w * TW + i < last ? w * TW + i : last;
            const unsigned off = (unsigned)j * (unsigned)s.C + c;
            dr[i] = (reinterpret_cast<const E*>(A.dt) + base)[off];
            gr[i] = (gy + base)[off];
            if (A.z) zr[i] = (reinterpret_cast<const E*>(A.z) + base)[off];
        }
    };
    // Tiles of absent tokens alone change nothing.
    const int end = t_begin + kSelBlock < len ? t_begin + kSelBlock : len;
    int t0 = end > t_begin ? (end - 1) / kSelTile * kSelTile : -1;
    if (t0 >= 0) fetch(t0);
    for (; t0 >= t_begin; t0 -= kSelTile) {
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const bool there = live && t0 + w * TW + i < len;
            float d = (float)dr[i] + bias, sig, p = there ? (float)gr[i] : 0.f;
            if (s.softplus) d = softplus(d, sig);
            if (A.z) {
                const float z = there ? (float)zr[i] : 0.f;
                p *= z * logistic(z);
            }
            const f32x2 v = {there ? d : 0.f, p};
            din[w * TW + i][lane] = v;
        }
        if (t0 > t_begin) fetch(t0 - kSelTile);
        __syncthreads();
        const float* row = bc + (((b * tiles + t0 / kSelTile) * s.G + grp) * W + w) * (kSelTile * 2 * NPT);
        constexpr int kGroups = SelGroup<NPT>::kGroups, kTok = SelGroup<NPT>::kTok;
        float subtotal = 0.f;
        SelGroup<NPT> grp_of[2];
        grp_of[0].fetch(row, din, lane, kGroups - 1);
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
            const SelGroup<NPT>& v = grp_of[q & 1];
            if (q + 1 < kGroups) grp_of[(q + 1) & 1].fetch(row, din, lane, kGroups - 2 - q);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = kTok - 1; k >= 0; --k) {
                const f32x2 x = v.x[k];
#pragma unroll
                for (int i = 0; i < NPT; ++i) g[i] = fast_exp2(x[0] * a2[i]) * fmaf(v.C(k, i), x[1], g[i]);
                subtotal += x[0];
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        total += subtotal;
        __syncthreads();
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NPT; ++i)
        if (n0 + i < Np) out[state_at(s, b * blocks + k, n0 + i, c)] = g[i];
    if (w == 0) sum[(b * blocks + k) * s.C + c] = total;
}

// ---- sums across the lanes of a wave ---------------------------------------------------

// Lanes below 32: a summed over lanes l and l+32; the others: b.  (xor 16: by rows of 16.)
__device__ __forceinline__ float fold32(float a, float b) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float fold16(float a, float b) {
    const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// The same with the DPP permutation CTRL, an involution: lanes with `up` false get a's sum.
template <int CTRL>
__device__ __forceinline__ float fold_dpp(float a, float b, bool up) {
    const float own = up ? b : a, other = up ? a : b;
    return own + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(other), CTRL, 0xf, 0xf, true));
}
constexpr int kXor8 = 0x128, kXor7 = 0x141, kXor3 = 0x1b, kXor1 = 0xb1;  // row_ror:8, row_half_mirror, quad_perm

__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

constexpr int kGradWaves = 4, kGradChan = 8;                   // waves, channels of a wave at once
constexpr int kGradStep = kGradWaves * kGradChan;              // channels of a workgroup at once

// LDS of the gradient kernel: the fixed part, and per set of channels of a wave.
template <int NT>
struct GradLds {
    static constexpr int kStates = 8 * NT;
    float bc[2][kSelTile][kStates];
    union {
        f32x4 rec[kGradWaves][kSelTile][kGradChan];  // d, d u, p
        float red[kGradWaves][4 * NT][64];
    };
};

template <class E, int NT>
__global__ __launch_bounds__(64 * kGradWaves) void sel_gradient_kernel(SelShape s, SelArgs A, SelBwdArgs g,
                                                                       const float* __restrict__ keep,
                                                                       SelBwdScratch W, int64_t blocks, int ntiles) {
    constexpr int kStates = 8 * NT;
    extern __shared__ __align__(16) char lds[];
    GradLds<NT>& L = *reinterpret_cast<GradLds<NT>*>(lds);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int d = lane & 7, nl = lane >> 3;
    const int Cg = (int)(s.C / s.G), cut = (int)W.cut, cuts = (int)W.cuts, sets = cut / kGradStep;
    // Per set of channels: G, gA, and the lane's own sums of gD and gbias.
    float* const own = reinterpret_cast<float*>(lds + sizeof(GradLds<NT>)) + (int64_t)w * sets * 64 * (2 * NT + 2) + lane;
    int64_t blk = blockIdx.x;
    const int nt = (int)(blk % ntiles);
    blk /= ntiles;
    const int cu = (int)(blk % cuts);
    blk /= cuts;
    const int grp = (int)(blk % s.G);
    blk /= s.G;
    const int64_t k = blk % blocks, b = blk / blocks;
    const int64_t len = row_length(s, b), tiles = (s.T + kSelTile - 1) / kSelTile;
    const int n0 = nt * kStates + nl * NT, Np = (s.N + 3) / 4 * 4;
    const bool whole = ntiles == 1;  // sums over the states are complete

    for (int i = 0; i < sets * (2 * NT + 2); ++i) own[i * 64] = 0.f;

    for (int q = kSelBlock / kSelTile - 1; q >= 0; --q) {
        const int64_t t0 = k * kSelBlock + q * kSelTile;
        if (t0 >= s.T) continue;
        __syncthreads();  // the previous tile's bc and red have been read
        for (int j = threadIdx.x; j < 2 * kSelTile * kStates; j += 64 * kGradWaves) {
            const int n = nt * kStates + j % kStates, t = j / kStates % kSelTile, o = j / (kStates * kSelTile);
            float v = 0.f;
            if (n < s.N && t0 + t < len)
                v = (float)reinterpret_cast<const E*>(o ? A.Cm : A.Bm)[((b * s.T + t0 + t) * s.G + grp) * s.N + n];
            L.bc[o][t][n - nt * kStates] = v;
        }
        __syncthreads();
        float accB[kSelTile][NT], accC[kSelTile][NT];
#pragma unroll
        for (int t = 0; t < kSelTile; ++t)
#pragma unroll
            for (int i = 0; i < NT; ++i) accB[t][i] = accC[t][i] = 0.f;

        for (int set = 0; set < sets; ++set) {
            const int in_group = cu * cut + set * kGradStep + w * kGradChan + d;
            if (cu * cut + set * kGradStep + w * kGradChan >= Cg) break;
            const bool live = in_group < Cg;
            const int64_t c = (int64_t)grp * Cg + (live ? in_group : Cg - 1);
            float* const mine = own + set * 64 * (2 * NT + 2);
            // This lane's two tokens.
            const float bias = A.bias ? A.bias[c] : 0.f, Dc = A.D ? A.D[c] : 0.f;
            float u[2], dd[2], p[2], sig[2], gzf[2];
            bool there[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t t = t0 + 2 * nl + e;
                there[e] = live && t < len;
                u[e] = dd[e] = p[e] = gzf[e] = 0.f;
                sig[e] = 1.f;
                if (there[e]) {
                    const int64_t at = (b * s.T + t) * s.C + c;
                    u[e] = (float)reinterpret_cast<const E*>(A.u)[at];
                    dd[e] = (float)reinterpret_cast<const E*>(A.dt)[at] + bias;
                    p[e] = (float)reinterpret_cast<const E*>(g.gy)[at];
                    if (A.z) {
                        const float z = (float)reinterpret_cast<const E*>(A.z)[at];
                        const float sg = logistic(z);
                        gzf[e] = p[e] * sg * fmaf(z, 1.f - sg, 1.f);
                        p[e] *= z * sg;
                    }
                    if (s.softplus) dd[e] = softplus(dd[e], sig[e]);
                }
                const f32x4 v = {dd[e], dd[e] * u[e], p[e], 0.f};
                L.rec[w][2 * nl + e][d] = v;
            }
            float a2[NT], G[NT], gA[NT], h0[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int n = n0 + i;
                a2[i] = n < s.N ? A.A[c * s.N + n] * kLog2e : 0.f;
                h0[i] = G[i] = 0.f;
                if (n < s.N) {
                    h0[i] = keep[state_at(s, b * tiles + t0 / kSelTile, n, c)];
                    if (t0 + kSelTile >= s.T || q == kSelBlock / kSelTile - 1)
                        G[i] = W.carry[state_at(s, b * blocks + k, n, c)];
                    else
                        G[i] = mine[i * 64];
                }
                gA[i] = mine[(NT + i) * 64];
            }
            wave_lds_fence();
            // The states of the tile again.
            float h[kSelTile][NT], a[kSelTile][NT];
#pragma unroll
            for (int t = 0; t < kSelTile; ++t) {
                const f32x2 x = *reinterpret_cast<const f32x2*>(&L.rec[w][t][d]);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    a[t][i] = fast_exp2(x[0] * a2[i]);
                    h[t][i] = fmaf(a[t][i], t ? h[t ? t - 1 : 0][i] : h0[i], x[1] * L.bc[0][t][nl * NT + i]);
                }
            }
            // Backwards: q1 = sum A m, q2 = sum g B, q3 = sum C h (over this lane's states).
            float q1[kSelTile], q2[kSelTile], q3[kSelTile];
#pragma unroll
            for (int t = kSelTile - 1; t >= 0; --t) {
                const f32x4 x = L.rec[w][t][d];
                q1[t] = q2[t] = q3[t] = 0.f;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const float Bt = L.bc[0][t][nl * NT + i], Ct = L.bc[1][t][nl * NT + i];
                    const float gt = fmaf(Ct, x[2], G[i]);
                    G[i] = gt * a[t][i];
                    const float m = G[i] * (t ? h[t ? t - 1 : 0][i] : h0[i]);
                    gA[i] = fmaf(x[0], m, gA[i]);
                    q1[t] = fmaf(a2[i], m, q1[t]);
                    q2[t] = fmaf(gt, Bt, q2[t]);
                    q3[t] = fmaf(Ct, h[t][i], q3[t]);
                    accB[t][i] = fmaf(gt, x[1], accB[t][i]);
                    accC[t][i] = fmaf(x[2], h[t][i], accC[t][i]);
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) mine[i * 64] = G[i], mine[(NT + i) * 64] = gA[i];
            // Over the state lanes; lane nl ends with tokens 2 nl and 2 nl + 1.
            const bool up = lane & 8;
            float s1[2], s2[2], s3[2];
            const auto over_states = [&](const float* v, float* out) {
                float r[8], r2[4];
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = fold32(v[j], v[j + 8]);
#pragma unroll
                for (int j = 0; j < 4; ++j) r2[j] = fold16(r[j], r[j + 4]);
#pragma unroll
                for (int j = 0; j < 2; ++j) out[j] = fold_dpp<kXor8>(r2[j], r2[j + 2], up);
            };
            over_states(q1, s1);
            over_states(q2, s2);
            over_states(q3, s3);
            wave_lds_fence();  // rec has been read
            float sD = 0.f, sb = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t t = t0 + 2 * nl + e;
                const int64_t at = (b * s.T + t) * s.C + c;
                if (!live || t >= s.T) continue;
                if (whole) {
                    const float gd = there[e] ? fmaf(u[e], s2[e], s1[e] * kLn2) * sig[e] : 0.f;
                    const float gu = there[e] ? fmaf(Dc, p[e], dd[e] * s2[e]) : 0.f;
                    const float gz = there[e] ? gzf[e] * fmaf(Dc, u[e], s3[e]) : 0.f;
                    reinterpret_cast<E*>(g.gu)[at] = (E)gu;
                    reinterpret_cast<E*>(g.gdt)[at] = (E)gd;
                    if (A.z) reinterpret_cast<E*>(g.gz)[at] = (E)gz;
                    sD = fmaf(p[e], u[e], sD);
                    sb += gd;
                } else {
                    float* o = W.q + ((int64_t)nt * s.B * s.T * s.C + at) * 3;
                    o[0] = s1[e] * kLn2, o[1] = s2[e], o[2] = s3[e];
                }
            }
            mine[(2 * NT) * 64] += sD;
            mine[(2 * NT + 1) * 64] += sb;
        }
        // Over the channel lanes: bit 2 of the lane picks B or C, bits 1 and 0 the token's bits 3, 2.
        float r[4 * NT];
        {
            float x[kSelTile * NT], y[8 * NT];
            const bool up2 = lane & 4, up1 = lane & 2, up0 = lane & 1;
#pragma unroll
            for (int j = 0; j < kSelTile * NT; ++j)
                x[j] = fold_dpp<kXor7>(accB[j / NT][j % NT], accC[j / NT][j % NT], up2);
#pragma unroll
            for (int j = 0; j < 8 * NT; ++j) y[j] = fold_dpp<kXor3>(x[j], x[j + 8 * NT], up1);
#pragma unroll
            for (int j = 0; j < 4 * NT; ++j) r[j] = fold_dpp<kXor1>(y[j], y[j + 4 * NT], up0);
        }
        __syncthreads();  // the last set's rec has been read
#pragma unroll
        for (int j = 0; j < 4 * NT; ++j) L.red[w][j][lane] = r[j];
        __syncthreads();
        for (int j = threadIdx.x; j < 4 * NT * 64; j += 64 * kGradWaves) {
            const int l = j & 63, v = j >> 6;
            float x = L.red[0][v][l];
#pragma unroll
            for (int i = 1; i < kGradWaves; ++i) x += L.red[i][v][l];
            const int o = l >> 2 & 1, t = (l >> 1 & 1) * 8 + (l & 1) * 4 + v / NT;
            const int n = nt * kStates + (l >> 3) * NT + v % NT;
            if (t0 + t < s.T && n < Np)
                W.gBC[((((int64_t)cu * s.B + b) * s.T + t0 + t) * s.G + grp) * 2 * Np + o * Np + n] = t0 + t < len ? x : 0.f;
        }
    }
    // What each set of channels kept.
    for (int set = 0; set < sets; ++set) {
        const int in_group = cu * cut + set * kGradStep + w * kGradChan + d;
        const bool live = in_group < Cg;
        const int64_t c = (int64_t)grp * Cg + in_group;
        const float* const mine = own + set * 64 * (2 * NT + 2);
        if (live) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (n0 + i < Np) W.gA[state_at(s, b * blocks + k, n0 + i, c)] = mine[(NT + i) * 64];
        }
        if (whole) {
            float sD = mine[(2 * NT) * 64], sb = mine[(2 * NT + 1) * 64];
#pragma unroll
            for (int o = 8; o < 64; o <<= 1) sD += __shfl_xor(sD, o), sb += __shfl_xor(sb, o);
            if (live && nl == 0) {
                W.gDb[((b * blocks + k) * 2) * s.C + c] = sD;
                W.gDb[((b * blocks + k) * 2 + 1) * s.C + c] = sb;
            }
        }
    }
}

// More than 16 states: the tiles' sums over states added, and the gradients of each token and
// channel.  A lane walks down one block's tokens of one channel.
template <class E>
__global__ __launch_bounds__(64) void sel_finish_kernel(SelShape s, SelArgs A, SelBwdArgs g, SelBwdScratch W,
                                                        int64_t blocks, int ntiles) {
    const int64_t cols = (s.C + 63) / 64;
    const int64_t c = (int64_t)(blockIdx.x % cols) * 64 + threadIdx.x;
    const int64_t row = blockIdx.x / cols, k = row % blocks, b = row / blocks;
    if (c >= s.C) return;
    const int64_t len = row_length(s, b);
    const float bias = A.bias ? A.bias[c] : 0.f, Dc = A.D ? A.D[c] : 0.f;
    float sD = 0.f, sb = 0.f;
    for (int64_t t = k * kSelBlock; t < (k + 1) * kSelBlock && t < s.T; ++t) {
        const int64_t at = (b * s.T + t) * s.C + c;
        float gu = 0.f, gd = 0.f, gz = 0.f;
        if (t < len) {
            float s1 = 0.f, s2 = 0.f, s3 = 0.f;
            for (int i = 0; i < ntiles; ++i) {
                const float* o = W.q + ((int64_t)i * s.B * s.T * s.C + at) * 3;
                s1 += o[0], s2 += o[1], s3 += o[2];
            }
            const float u = (float)reinterpret_cast<const E*>(A.u)[at];
            float d = (float)reinterpret_cast<const E*>(A.dt)[at] + bias, sig = 1.f;
            float p = (float)reinterpret_cast<const E*>(g.gy)[at];
            if (s.softplus) d = softplus(d, sig);
            if (A.z) {
                const float z = (float)reinterpret_cast<const E*>(A.z)[at];
                const float sg = logistic(z);
                gz = p * sg * fmaf(z, 1.f - sg, 1.f) * fmaf(Dc, u, s3);
                p *= z * sg;
            }
            gd = fmaf(u, s2, s1) * sig;
            gu = fmaf(Dc, p, d * s2);
            sD = fmaf(p, u, sD);
            sb += gd;
        }
        reinterpret_cast<E*>(g.gu)[at] = (E)gu;
        reinterpret_cast<E*>(g.gdt)[at] = (E)gd;
        if (A.z) reinterpret_cast<E*>(g.gz)[at] = (E)gz;
    }
    W.gDb[(row * 2) * s.C + c] = sD;
    W.gDb[(row * 2 + 1) * s.C + c] = sb;
}

// Column sums of (rows, cols), rows added by 16 strips at once, then the strips in order.  The
// column's place in the results: a state's (STATES), or D's and the bias's.
template <bool STATES>
__global__ __launch_bounds__(256) void sel_fold_kernel(SelShape s, const float* __restrict__ part, int64_t rows,
                                                       int64_t cols, float* __restrict__ x, float* __restrict__ y) {
    __shared__ float lds[16][17];
    const int cx = threadIdx.x & 15, strip = threadIdx.x >> 4;
    const int64_t j = (int64_t)blockIdx.x * 16 + cx;
    float v = 0.f;
    if (j < cols)
#pragma unroll 4
        for (int64_t r = strip; r < rows; r += 16) v += part[r * cols + j];
    lds[strip][cx] = v;
    __syncthreads();
    if (strip != 0 || j >= cols) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) v += lds[i][cx];
    if constexpr (STATES) {
        const int n = (int)(j / (4 * s.C)) * 4 + (int)(j & 3);
        if (n < s.N) x[j / 4 % s.C * s.N + n] = v;
    } else if (j < s.C) {
        if (x) x[j] = v;
    } else if (y) {
        y[j - s.C] = v;
    }
}

// B's and C's gradients: the channel ranges' shares added.
template <class E>
__global__ __launch_bounds__(256) void sel_fold_bc_kernel(SelShape s, const float* __restrict__ part, int64_t cuts,
                                                          E* __restrict__ gB, E* __restrict__ gC, int64_t total) {
    const int Np = (s.N + 3) / 4 * 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        float v = 0.f;
        for (int64_t k = 0; k < cuts; ++k) v += part[k * total + i];
        const int j = (int)(i % (2 * Np)), n = j % Np;
        if (n < s.N) (j < Np ? gB : gC)[i / (2 * Np) * s.N + n] = (E)v;
    }
}

template <class E, int W, int NPT>
hipError_t reverse(const SelShape& s, const SelArgs& A, const void* gy, const float* bc, float* out, float* sum,
                   hipStream_t st) {
    const int group_tiles = (int)ceil_div(s.C / s.G, 64);
    const int64_t blocks = sel_blocks(s);
    hipLaunchKernelGGL((sel_reverse_kernel<E, W, NPT>), dim3((unsigned)(s.B * blocks * s.G * group_tiles)),
                       dim3(64 * W), 0, st, s, A, (const E*)gy, bc, out, sum, (int)blocks, group_tiles);
    return hipGetLastError();
}

template <class E>
hipError_t reverse_by_states(const SelShape& s, const SelArgs& A, const SelPlan& p, const void* gy, const float* bc,
                             float* out, float* sum, hipStream_t st) {
    if (p.npt == 1) return reverse<E, 1, 1>(s, A, gy, bc, out, sum, st);
    if (p.npt == 2) return reverse<E, 1, 2>(s, A, gy, bc, out, sum, st);
    if (p.npt == 4) {
        if (p.waves == 1) return reverse<E, 1, 4>(s, A, gy, bc, out, sum, st);
        if (p.waves == 2) return reverse<E, 2, 4>(s, A, gy, bc, out, sum, st);
        return reverse<E, 4, 4>(s, A, gy, bc, out, sum, st);
    }
    if (p.npt == 8)
        return p.waves == 4 ? reverse<E, 4, 8>(s, A, gy, bc, out, sum, st) : reverse<E, 8, 8>(s, A, gy, bc, out, sum, st);
    return reverse<E, 8, 16>(s, A, gy, bc, out, sum, st);
}

template <class E, int NT>
hipError_t gradients(const SelShape& s, const SelArgs& A, const SelBwdArgs& g, const float* keep,
                     const SelBwdScratch& W, hipStream_t st) {
    const int64_t blocks = sel_blocks(s);
    const int ntiles = (int)ceil_div(s.N, 8 * NT);
    const size_t lds = sizeof(GradLds<NT>) + (size_t)(W.cut / kGradChan) * 64 * (2 * NT + 2) * sizeof(float);
    hipLaunchKernelGGL((sel_gradient_kernel<E, NT>), dim3((unsigned)(s.B * blocks * s.G * W.cuts * ntiles)),
                       dim3(64 * kGradWaves), lds, st, s, A, g, keep, W, blocks, ntiles);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || ntiles == 1) return e;
    hipLaunchKernelGGL((sel_finish_kernel<E>), dim3((unsigned)(s.B * blocks * ceil_div(s.C, 64))), dim3(64), 0, st, s,
                       A, g, W, blocks, ntiles);
    return hipGetLastError();
}

template <class E>
hipError_t backward(const SelShape& s, const SelArgs& A, const SelBwdArgs& g, const SelPlan& p, const float* bc,
                    const float* keep, const SelBwdScratch& W, hipStream_t st) {
    const int64_t blocks = sel_blocks(s), rows = s.B * blocks;
    hipError_t e = reverse_by_states<E>(s, A, p, g.gy, bc, W.carry, W.sum, st);
    if (e == hipSuccess) e = run_sel_join(s, A.A, W.carry, W.sum, blocks, g.gs_out, g.gs_in, true, st);
    if (e == hipSuccess) e = s.N <= 8 ? gradients<E, 1>(s, A, g, keep, W, st) : gradients<E, 2>(s, A, g, keep, W, st);
    if (e != hipSuccess) return e;
    const int64_t cols = (int64_t)sel_n4(s) * 4 * s.C;
    hipLaunchKernelGGL((sel_fold_kernel<true>), dim3((unsigned)ceil_div(cols, 16)), dim3(256), 0, st, s, W.gA, rows,
                       cols, g.gA, (float*)nullptr);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (g.gD || g.gbias) {
        hipLaunchKernelGGL((sel_fold_kernel<false>), dim3((unsigned)ceil_div(2 * s.C, 16)), dim3(256), 0, st, s, W.gDb,
                           rows, 2 * s.C, g.gD, g.gbias);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int64_t total = s.B * s.T * s.G * 2 * sel_n4(s) * 4;
    int64_t wg = ceil_div(total, 256);
    if (wg > 8192) wg = 8192;
    hipLaunchKernelGGL((sel_fold_bc_kernel<E>), dim3((unsigned)wg), dim3(256), 0, st, s, W.gBC, W.cuts, (E*)g.gB,
                       (E*)g.gC, total);
    return hipGetLastError();
}

}  // namespace

int64_t sel_cut(const SelShape& s) {
    // Channels of a workgroup of the gradients: up to 128, fewer where that leaves the chip empty.
    const int64_t Cg = s.C / s.G, rows = s.B * sel_blocks(s) * s.G;
    int64_t cut = 128;
    while (cut > kGradStep && rows * ceil_div(Cg, cut) < 1024) cut /= 2;
    return cut;
}

hipError_t run_sel_backward(const SelShape& s, const SelArgs& A, const SelBwdArgs& g, const SelPlan& p, const float* bc,
                            const float* keep, const SelBwdScratch& W, hipStream_t st) {
    return s.dtype == kBf16 ? backward<bf16_t>(s, A, g, p, bc, keep, W, st)
                            : backward<float>(s, A, g, p, bc, keep, W, st);
}

}  // namespace linrec
