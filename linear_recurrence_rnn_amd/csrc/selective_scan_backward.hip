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
// The rows are cut into blocks of 16 to 256 tokens.  First each block's share of the G that leaves it on
// the left, from zero on its right (all blocks at once, as the forward's segments); then the G that
// enters each block, one block after the other (the decay over a block is e^{A sum d}); then all gradients,
// all blocks at once, the states formed again from those the forward kept every 16 tokens.
//
// The last kernel sums over states (for each token and channel) and over channels (for each token
// and state).  Like the forward, a wave holds 64 channels, a lane each, and 4 states of them, with B and C by
// scalar loads; sums over the states are added in the lane and over the waves through LDS.  Sums over the
// lanes are transposed there: 8 values (2 tokens, 4 states) are written as rows of 64 and read back as
// eighths of rows, 8 floats a lane, that the lane adds; what the eight lanes of a row have left is folded for
// 64 values at once.  10 cycles of the vector unit a state for both sums, where folds across the
// lanes alone would take 24.  (float32 products of the matrix unit with columns of ones were slower: on this
// chip they keep the vector unit from its own work, 34 cycles and 35 of it taking 74.)
// Sums over blocks, batch rows and channel ranges are partial sums in the workspace, added in
// order by small kernels at the end: nothing depends on timing.
//
// 8 x 4096 tokens of 2560 channels, 16 states, bfloat16, by trace: reverse 275-295 us, gradients 921-994 (the lower ones
// before the clock falls), partial sums 56.  The vector unit is busy 98% and 96% of the first two.
#include "selective_math.hpp"

namespace linrec {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kBwdNpt = 4;  // states of a lane in the kernels below; a workgroup of W waves has 4 W

// The G that leaves each block on its left, from zero, and the sum of its steps.
template <class E, int W>
__global__ __launch_bounds__(64 * W) void sel_reverse_kernel(SelShape s, SelArgs A, const E* __restrict__ gy,
                                                             const float* __restrict__ bc, float* __restrict__ out,
                                                             float* __restrict__ sum, int blocks, int block, int group_tiles,
                                                             int ntiles) {
    constexpr int TW = kSelTile / W, NPT = kBwdNpt;
    __shared__ f32x2 din[kSelTile][64];  // d, p
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    unsigned blk = place_of(blockIdx.x, gridDim.x, (unsigned)(s.G * group_tiles * ntiles));
    const int tile = (int)(blk % (unsigned)(s.G * group_tiles));
    blk /= (unsigned)(s.G * group_tiles);
    const int nt = (int)(blk % (unsigned)ntiles);
    blk /= (unsigned)ntiles;
    const int k = (int)(blk % (unsigned)blocks);
    const int64_t b = blk / (unsigned)blocks;
    const int grp = tile / group_tiles, Cg = (int)(s.C / s.G);
    const int in_group = (tile % group_tiles) * 64 + lane;
    const bool live = in_group < Cg;
    const unsigned C = (unsigned)s.C, c = (unsigned)(grp * Cg + (live ? in_group : Cg - 1));
    const int T = (int)s.T, tiles = (T + kSelTile - 1) / kSelTile;
    const int t_begin = k * block, len = (int)row_length(s, b);
    const int n0 = (nt * W + w) * NPT;
    float g[NPT], a2[NPT];
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        g[i] = 0.f;
        a2[i] = n0 + i < s.N ? A.A[(int64_t)c * s.N + n0 + i] * kLog2e : 0.f;
    }
    const float bias = A.bias ? A.bias[c] : 0.f;
    const bool gated = A.z != nullptr, soft = s.softplus != 0;
    const void* const zp = gated ? A.z : A.dt;
    float total = 0.f;
    // This wave's tokens of a tile, read while the tile behind it is worked on.  Absent ones are read as
    // the last that is there and not used.
    E dr[TW], zr[TW], gr[TW];
    const auto fetch = [&](int t0, int64_t base) {  // base: the tile's first element
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const int j = t0 + w * TW + i < len ? w * TW + i : len - 1 - t0;
            const unsigned at = ((unsigned)j * C + c) * (unsigned)sizeof(E);
            dr[i] = load_elem<E>(elems<E>(A.dt, base), at);
            gr[i] = load_elem<E>(elems<E>(gy, base), at);
            zr[i] = load_elem<E>(elems<E>(zp, base), at);
        }
    };
    // Tiles of absent tokens alone change nothing.
    const int end = t_begin + block < len ? t_begin + block : len;
    int t0 = end > t_begin ? (end - 1) / kSelTile * kSelTile : t_begin - kSelTile;
    int64_t base = (b * T + t0) * s.C;
    const int step = s.G * ntiles * W * (kSelTile * 2 * NPT);  // of B and C, from tile to tile
    const float* row =
        bc + ((((b * tiles + t_begin / kSelTile) * s.G + grp) * ntiles + nt) * W + w) * (kSelTile * 2 * NPT) +
        (int64_t)((t0 - t_begin) / kSelTile) * step;
    if (t0 >= t_begin) fetch(t0, base);
    for (; t0 >= t_begin; t0 -= kSelTile) {
        float d[TW], p[TW];
#pragma unroll
        for (int i = 0; i < TW; ++i) d[i] = (float)dr[i] + bias, p[i] = (float)gr[i];
        if (soft) {
            float sig;
#pragma unroll
            for (int i = 0; i < TW; ++i) d[i] = softplus(d[i], sig);
        }
        if (gated) {
#pragma unroll
            for (int i = 0; i < TW; ++i) p[i] *= (float)zr[i] * logistic((float)zr[i]);
        }
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const bool there = live && t0 + w * TW + i < len;
            const f32x2 v = {there ? d[i] : 0.f, there ? p[i] : 0.f};
            din[w * TW + i][lane] = v;
        }
        if (t0 > t_begin) base -= kSelTile * s.C;
        fetch(t0 > t_begin ? t0 - kSelTile : t0, base);
        __syncthreads();
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
            for (int r = kTok - 1; r >= 0; --r) {
                const f32x2 x = v.x[r];
#pragma unroll
                for (int i = 0; i < NPT; ++i) g[i] = fast_exp2(x[0] * a2[i]) * fmaf(v.C(r, i), x[1], g[i]);
                subtotal += x[0];
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        total += subtotal;
        row -= step;
        __syncthreads();
    }
    if (!live) return;
    if (n0 < s.N) store16<float>(out + state_at(s, b * blocks + k, n0, c), g);
    if (nt == 0 && w == 0) sum[(b * blocks + k) * s.C + c] = total;
}

// ---- the gradients --------------------------------------------------------------------

// The lanes with `up` false: a summed over the two lanes that the DPP permutation CTRL, an
// involution, exchanges; the others: b.
template <int CTRL>
__device__ __forceinline__ float fold_dpp(float a, float b, bool up) {
    const float own = up ? b : a, other = up ? a : b;
    return own + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(other), CTRL, 0xf, 0xf, true));
}
constexpr int kMirror8 = 0x141, kXor1 = 0xb1, kXor2 = 0x4e;  // quad_perm [1,0,3,2] and [2,3,0,1]

// Tokens of a tile whose decays are kept from the pass over the states to the one back over their gradients.
// The others are formed again, 12 cycles of the vector unit each, so that the registers are enough for three waves
// a SIMD with four waves a workgroup (all kept: two waves, 1245 us for 1045 at the time) and for two with one wave or two.
// Whole training steps of 8 x 4096 tokens of 2560 channels, bfloat16 / float32: 16 states 1770 / 1872 us with six, 1789 / 1894
// with four; 4 states, one wave a workgroup, 1286 / 1592 with six, which leave it one wave a SIMD, 1017 / 1330
// with four; 8 states, two waves, 1325 / 1567 with either.
template <int W>
constexpr int kKeptBy = W == 1 ? 4 : 6;

constexpr int kRowPad = 68;  // floats of a row of 64: an eighth starts on 16 bytes, two rows on other banks

template <int W>
struct GradLds {
    f32x2 du[kSelTile][64];          // d, d u
    float p[kSelTile][64];
    float part[2][W][kSelTile][64];  // the waves' shares of sums over the states
    float rows[W][8][kRowPad];       // 8 values of a wave on their way to being summed over its lanes
};

// WHOLE: one workgroup has all states of its channels, so that its sums over them are complete.
template <class E, int W, bool WHOLE>
__global__ __launch_bounds__(64 * W, W == 4 ? 3 : 2) void sel_gradient_kernel(SelShape s, SelArgs A, SelBwdArgs g,
                                                                              const float* __restrict__ bc,
                                                                              const float* __restrict__ keep,
                                                                              SelBwdScratch S, int blocks, int block, int ntiles) {
    constexpr int NPT = kBwdNpt, TW = kSelTile / W, kPairs = kSelTile / 2, kKept = kKeptBy<W>;
    __shared__ GradLds<W> L;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int Cg = (int)(s.C / s.G), cuts = (int)S.cuts;
    unsigned blk = place_of(blockIdx.x, gridDim.x, (unsigned)(cuts * s.G * ntiles));
    const int cu = (int)(blk % (unsigned)cuts);
    blk /= (unsigned)cuts;
    const int grp = (int)(blk % (unsigned)s.G);
    blk /= (unsigned)s.G;
    const int nt = (int)(blk % (unsigned)ntiles);
    blk /= (unsigned)ntiles;
    const int k = (int)(blk % (unsigned)blocks);
    const int64_t b = blk / (unsigned)blocks;
    const int T = (int)s.T, tiles = (T + kSelTile - 1) / kSelTile, len = (int)row_length(s, b);
    const int t_begin = k * block, t_end = t_begin + block < T ? t_begin + block : T;
    const int n0 = (nt * W + w) * NPT, Np = (s.N + 3) / 4 * 4;
    const unsigned C = (unsigned)s.C;
    const bool gated = A.z != nullptr, soft = s.softplus != 0, states = n0 < s.N;
    const bool live = cu * 64 + lane < Cg;
    const unsigned c = (unsigned)(grp * Cg + (live ? cu * 64 + lane : Cg - 1));

    // Tiles of absent tokens alone: no gradients.
    const int live_end = len < t_end ? (len > t_begin ? (len + kSelTile - 1) / kSelTile * kSelTile : t_begin) : t_end;
    for (int t = live_end + w; t < t_end; t += W) {
        if (WHOLE && live) {
            const int64_t at = (b * T + t) * s.C + c;
            reinterpret_cast<E*>(g.gu)[at] = reinterpret_cast<E*>(g.gdt)[at] = (E)0.f;
            if (gated) reinterpret_cast<E*>(g.gz)[at] = (E)0.f;
        }
        for (int j = lane; j < 2 * W * NPT; j += 64) {
            const int n = nt * W * NPT + j % (W * NPT);
            if (n < Np) S.gBC[((((int64_t)cu * s.B + b) * T + t) * s.G + grp) * 2 * Np + j / (W * NPT) * Np + n] = 0.f;
        }
    }

    // What a lane reads of a tile: its wave's tokens' inputs and its states before the tile, asked for a
    // tile ahead.  Absent tokens are read as the last one that is there, lanes behind the last channel
    // as that, inputs that were not given as others: none of that is used.  Bases of the block, and a
    // lane's byte offsets in it (below 2^32: 64 tokens of at most 2^22 channels, more of fewer).
    const int64_t base = (b * T + t_begin) * s.C;
    const void *const pu = elems<E>(A.u, base), *const pdt = elems<E>(A.dt, base), *const pgy = elems<E>(g.gy, base);
    const void* const pz = elems<E>(gated ? A.z : A.u, base);
    const void* const ph = elems<float>(keep, (b * tiles + t_begin / kSelTile) * Np * s.C + (int64_t)(states ? n0 : 0) * s.C);
    struct Raw {
        E u[TW], dt[TW], z[TW], gy[TW];  // as they come: a conversion would wait for the load
        f32x4 h0;
    } next;
    const auto fetch = [&](int q) {
#pragma unroll
        for (int e = 0; e < TW; ++e) {
            const int t = q * kSelTile + w * TW + e;
            const unsigned at = ((unsigned)(t_begin + t < len ? t : len - 1 - t_begin) * C + c) * (unsigned)sizeof(E);
            next.u[e] = load_elem<E>(pu, at);
            next.dt[e] = load_elem<E>(pdt, at);
            next.gy[e] = load_elem<E>(pgy, at);
            next.z[e] = load_elem<E>(pz, at);
        }
        next.h0 = load_elem<f32x4>(ph, ((unsigned)(q * Np) * C + c * 4) * 4);
    };
    const int q_first = (live_end - t_begin + kSelTile - 1) / kSelTile - 1;
    if (q_first >= 0) fetch(q_first);

    const float bias = A.bias ? A.bias[c] : 0.f, Dc = A.D ? A.D[c] : 0.f;
    float a2[NPT], G[NPT], gA[NPT], sD = 0.f, sb = 0.f;
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        a2[i] = n0 + i < s.N ? A.A[(int64_t)c * s.N + n0 + i] * kLog2e : 0.f;
        G[i] = n0 + i < s.N ? S.carry[state_at(s, b * blocks + k, n0 + i, c)] : 0.f;
        gA[i] = 0.f;
    }
    // A lane's eighth of a row.
    float* const rows = &L.rows[w][0][0];
    const float* const eighth = rows + (lane >> 3) * kRowPad + (lane & 7) * 8;

    // The block's first tile of B and C and of their gradients, and steps from one tile to the next.
    const float* const bc0 =
        bc + ((((b * tiles + t_begin / kSelTile) * s.G + grp) * ntiles + nt) * W + w) * (kSelTile * 2 * NPT);
    float* const gbc0 = S.gBC + ((((int64_t)cu * s.B + b) * T + t_begin) * s.G + grp) * 2 * Np;
    const int bc_step = s.G * ntiles * W * (kSelTile * 2 * NPT), gbc_step = kSelTile * s.G * 2 * Np;
    for (int q = q_first; q >= 0; --q) {
        const int t0 = t_begin + q * kSelTile;
        const float* row = bc0 + (int64_t)q * bc_step;
        // (Whether a token is there is the same for the whole wave.  Of an absent one, or a lane without a
        // channel, d, u and p are zero, which leaves the states and the sums over channels alone.)
        float sig[TW], gzf[TW], us[TW], h0[NPT];
        int own = s.N - n0;
        asm volatile("" : "+s"(own));  // four masks of the wave would be kept

#pragma unroll
        for (int e = 0; e < TW; ++e) {
            const bool there = live && t0 + w * TW + e < len;
            const float raw = (float)next.dt[e] + bias, z = (float)next.z[e], gy = (float)next.gy[e], sg = logistic(z);
            const float d = softplus(raw, sig[e]);
            if (!soft) sig[e] = 1.f;
            gzf[e] = gy * sg * fmaf(z, 1.f - sg, 1.f);
            us[e] = there ? (float)next.u[e] : 0.f;
            const float dd = there ? (soft ? d : raw) : 0.f;
            const f32x2 du = {dd, dd * us[e]};
            L.du[w * TW + e][lane] = du;
            L.p[w * TW + e][lane] = there ? gy * (gated ? z * sg : 1.f) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NPT; ++i) h0[i] = i < own ? next.h0[i] : 0.f;
        __syncthreads();
        // The states of the tile again, their sums q3 = sum C h, and the sums over channels of p h.
        float h[kSelTile][NPT], a[kKept][NPT], shares[kPairs];
        f32x4 eight[2];
        const auto ask_sums = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i) eight[i] = *reinterpret_cast<const f32x4*>(eighth + 4 * i);
        };
        const auto take_sums = [&]() {
            const f32x4 v = eight[0] + eight[1];
            return (v[0] + v[1]) + (v[2] + v[3]);
        };
        // A share of a pair of tokens joins the others: the pair's bits 0, 1 and 2 are the lane's bits 2, 1 and 0.
        float xs[2], ys[2];
        const auto join = [&](int j, bool up) {  // up: the pairs come in order, otherwise from the last
            if (j % 2 != (up ? 1 : 0)) return;
            xs[j / 2 % 2] = fold_dpp<kMirror8>(shares[j & ~1], shares[j | 1], lane & 4);
            if (j / 2 % 2 == (up ? 1 : 0)) ys[j / 4] = fold_dpp<kXor2>(xs[0], xs[1], lane & 2);
        };
        const auto fold = [&]() { return fold_dpp<kXor1>(ys[0], ys[1], lane & 1); };
        {
            typedef SelGroup<NPT, 16> Group;  // pairs of tokens
            constexpr int kGroups = Group::kGroups, kTok = Group::kTok;
            Group of[2];
            float pt[2][2];
            const auto ahead = [&](int j) {
                of[j & 1].fetch(row, L.du, lane, j);
#pragma unroll
                for (int r = 0; r < kTok; ++r) pt[j & 1][r] = L.p[j * kTok + r][lane];
            };
            ahead(0);
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                const Group& v = of[j & 1];
                if (j + 1 < kGroups) ahead(j + 1);
                if (j > 0) {
                    wave_lds_fence();  // the pair before has been written, and is read before the next is
                    ask_sums();
                    wave_lds_fence();
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = 0; r < kTok; ++r) {
                    const int t = j * kTok + r;
                    float q3 = 0.f;
#pragma unroll
                    for (int i = 0; i < NPT; ++i) {
                        const float f = fast_exp2(v.x[r][0] * a2[i]);
                        if (t >= kSelTile - kKept) a[t - (kSelTile - kKept)][i] = f;
                        h[t][i] = fmaf(f, t ? h[t ? t - 1 : 0][i] : h0[i], v.x[r][1] * v.B(r, i));
                        q3 = fmaf(v.C(r, i), h[t][i], q3);
                        rows[(r * NPT + i) * kRowPad + lane] = pt[j & 1][r] * h[t][i];
                    }
                    L.part[0][w][t][lane] = q3;
                }
                __builtin_amdgcn_sched_barrier(0);
                if (j > 0) shares[j - 1] = take_sums(), join(j - 1, true);
            }
            wave_lds_fence();
            ask_sums();
            wave_lds_fence();
            shares[kPairs - 1] = take_sums(), join(kPairs - 1, true);
        }
        const float totC = fold();
        __syncthreads();
        if (gated || !WHOLE) {
            float core[TW];
#pragma unroll
            for (int e = 0; e < TW; ++e) {
                core[e] = L.part[0][0][w * TW + e][lane];
#pragma unroll
                for (int j = 1; j < W; ++j) core[e] += L.part[0][j][w * TW + e][lane];
                if (WHOLE) core[e] = where(t0 + w * TW + e < len, gzf[e] * fmaf(Dc, us[e], core[e]));
            }
            if (live) {
#pragma unroll
                for (int e = 0; e < TW; ++e) {
                    const unsigned at = (unsigned)(q * kSelTile + w * TW + e) * C + c;
                    if (t0 + w * TW + e >= T) break;
                    if constexpr (!WHOLE)
                        store_elem<float>(S.q + ((int64_t)nt * 3 + 2) * s.B * T * s.C + base, at * 4, core[e]);
                    else
                        store_elem<E>((E*)g.gz + base, at * (unsigned)sizeof(E), core[e]);
                }
            }
        }
        __syncthreads();
        // Backwards: q1 = sum A m, q2 = sum g B, and the sums over channels of g d u.
        asm volatile("" : "+s"(row));  // as if it were another one: B and C of a whole tile would be kept in 128 scalar registers
        {
            f32x2 x[2][2];
            float y[2][2];
            f32x16 v[2];
            const auto ahead = [&](int j) {  // the pair of tokens 2 j, 2 j + 1
                typedef const __attribute__((address_space(4))) f32x16_at16* P;
                v[j & 1] = *reinterpret_cast<P>(reinterpret_cast<uintptr_t>(row + j * 16));
#pragma unroll
                for (int r = 0; r < 2; ++r) x[j & 1][r] = L.du[2 * j + r][lane], y[j & 1][r] = L.p[2 * j + r][lane];
            };
            ahead(kPairs - 1);
#pragma unroll
            for (int j = kPairs - 1; j >= 0; --j) {
                if (j > 0) ahead(j - 1);
                if (j == kPairs / 2) fetch(q > 0 ? q - 1 : 0);  // the last time for nothing
                if (j + 1 < kPairs) {
                    wave_lds_fence();
                    ask_sums();
                    wave_lds_fence();
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = 1; r >= 0; --r) {
                    const int t = 2 * j + r;
                    const float d = x[j & 1][r][0], du = x[j & 1][r][1], p = y[j & 1][r];
                    float q1 = 0.f, q2 = 0.f;
#pragma unroll
                    for (int i = 0; i < NPT; ++i) {
                        const float gt = fmaf(v[j & 1][r * 2 * NPT + NPT + i], p, G[i]);
                        G[i] = gt * (t >= kSelTile - kKept ? a[t - (kSelTile - kKept)][i] : fast_exp2(d * a2[i]));
                        const float m = G[i] * (t ? h[t ? t - 1 : 0][i] : h0[i]);
                        gA[i] = fmaf(d, m, gA[i]);
                        q1 = fmaf(a2[i], m, q1);
                        q2 = fmaf(gt, v[j & 1][r * 2 * NPT + i], q2);
                        rows[(r * NPT + i) * kRowPad + lane] = gt * du;
                    }
                    L.part[0][w][t][lane] = q1;
                    L.part[1][w][t][lane] = q2;
                }
#pragma unroll
                for (int i = 0; i < NPT; ++i) asm volatile("" : "+v"(gA[i]));  // now: behind the loop it would keep all m
                __builtin_amdgcn_sched_barrier(0);
                if (j + 1 < kPairs) shares[j + 1] = take_sums(), join(j + 1, false);
            }
            wave_lds_fence();
            ask_sums();
            wave_lds_fence();
            shares[0] = take_sums(), join(0, false);
        }
        const float totB = fold();
        __syncthreads();
        {
            float q1[TW], q2[TW];
#pragma unroll
            for (int e = 0; e < TW; ++e) {
                const int t = w * TW + e;
                q1[e] = L.part[0][0][t][lane], q2[e] = L.part[1][0][t][lane];
#pragma unroll
                for (int j = 1; j < W; ++j) q1[e] += L.part[0][j][t][lane], q2[e] += L.part[1][j][t][lane];
                if constexpr (WHOLE) {
                    const float d = L.du[t][lane][0], p = L.p[t][lane];
                    const bool there = t0 + t < len;
                    q1[e] = where(there, fmaf(us[e], q2[e], q1[e] * kLn2) * sig[e]);
                    q2[e] = where(there, fmaf(Dc, p, d * q2[e]));
                    sD = fmaf(p, us[e], sD);
                    sb += q1[e];
                }
            }
            if (live) {
#pragma unroll
                for (int e = 0; e < TW; ++e) {
                    const unsigned at = (unsigned)(q * kSelTile + w * TW + e) * C + c;
                    if (t0 + w * TW + e >= T) break;
                    if constexpr (WHOLE) {
                        store_elem<E>((E*)g.gu + base, at * (unsigned)sizeof(E), q2[e]);
                        store_elem<E>((E*)g.gdt + base, at * (unsigned)sizeof(E), q1[e]);
                    } else {
                        float* const o = S.q + (int64_t)nt * 3 * s.B * T * s.C + base;
                        store_elem<float>(o, at * 4, q1[e] * kLn2);
                        store_elem<float>(o + s.B * T * s.C, at * 4, q2[e]);
                    }
                }
            }
        }
        // A lane's sums over channels: of a pair of tokens by bits 0 to 2, the token by bit 5 and the state
        // by bits 4 and 3.
        const int t = 8 * (lane & 1) + 2 * (lane & 2) + (lane >> 1 & 2) + (lane >> 5), n = n0 + (lane >> 3 & 3);
        if (t0 + t < T && n < Np) {
            float* const o = gbc0 + (int64_t)q * gbc_step;
            const unsigned at = (unsigned)(t * s.G * 2 * Np + n) * 4;
            store_elem<float>(o, at, t0 + t < len ? totB : 0.f);
            store_elem<float>(o + Np, at, t0 + t < len ? totC : 0.f);
        }
    }
    if (live && states) store16<float>(S.gA + state_at(s, b * blocks + k, n0, c), gA);
    if (!WHOLE) return;
    __syncthreads();  // the last tile's part has been read
    L.part[0][w][0][lane] = sD, L.part[1][w][0][lane] = sb;
    __syncthreads();
    for (int o = w; o < 2; o += W) {
        float v = L.part[o][0][0][lane];
#pragma unroll
        for (int i = 1; i < W; ++i) v += L.part[o][i][0][lane];
        if (live) S.gDb[((b * blocks + k) * 2 + o) * s.C + c] = v;
    }
}

// More than 16 states: the tiles' sums over states added, and the gradients of each token and
// channel.  A workgroup takes 64 tokens of 64 channels at a time, 4 tokens a wave; 32 of those a CU keep the chip
// busy, and 2^22 would be more threads than one launch may have.
constexpr int kFinishGroups = 8192;

template <class E>
__global__ __launch_bounds__(1024) void sel_finish_kernel(SelShape s, SelArgs A, SelBwdArgs g, SelBwdScratch S,
                                                          int64_t blocks, int ntiles) {
    constexpr int kWaves = 16, kTok = kSelBlock / kWaves;
    __shared__ float acc[2][kWaves][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t cols = (s.C + 63) / 64;
    for (int64_t blk = blockIdx.x; blk < s.B * blocks * cols; blk += gridDim.x) {
        const int64_t c = blk % cols * 64 + lane, row = blk / cols, k = row % blocks, b = row / blocks;
        const bool live = c < s.C;
        const int64_t len = row_length(s, b), plane = s.B * s.T * s.C, t0 = k * kSelBlock + w * kTok;
        float sD = 0.f, sb = 0.f;
        if (live) {
            const float bias = A.bias ? A.bias[c] : 0.f, Dc = A.D ? A.D[c] : 0.f;
            // Everything of the four tokens is asked for before any is used; absent ones are read as the row's last one
            // that is there, and nothing where all four are.
            float q[kTok][3];
            E ur[kTok], dr[kTok], pr[kTok], zr[kTok];
            if (t0 < len) {
#pragma unroll
                for (int e = 0; e < kTok; ++e) {
                    q[e][0] = q[e][1] = q[e][2] = 0.f;
                    const int64_t t = t0 + e < len ? t0 + e : len - 1, at = (b * s.T + t) * s.C + c;
                    ur[e] = reinterpret_cast<const E*>(A.u)[at];
                    dr[e] = reinterpret_cast<const E*>(A.dt)[at];
                    pr[e] = reinterpret_cast<const E*>(g.gy)[at];
                    zr[e] = reinterpret_cast<const E*>(A.z ? A.z : A.u)[at];
                    for (int i = 0; i < ntiles; ++i) {
                        const float* o = S.q + (int64_t)i * 3 * plane + at;
#pragma unroll
                        for (int j = 0; j < 3; ++j) q[e][j] += o[j * plane];
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < kTok; ++e) {
                const int64_t t = t0 + e, at = (b * s.T + t) * s.C + c;
                if (t >= s.T) continue;
                float gu = 0.f, gd = 0.f, gz = 0.f;
                if (t < len) {
                    const float u = (float)ur[e];
                    float d = (float)dr[e] + bias, p = (float)pr[e], sig = 1.f;
                    if (s.softplus) d = softplus(d, sig);
                    if (A.z) {
                        const float z = (float)zr[e], sg = logistic(z);
                        gz = p * sg * fmaf(z, 1.f - sg, 1.f) * fmaf(Dc, u, q[e][2]);
                        p *= z * sg;
                    }
                    gd = fmaf(u, q[e][1], q[e][0]) * sig;
                    gu = fmaf(Dc, p, d * q[e][1]);
                    sD = fmaf(p, u, sD);
                    sb += gd;
                }
                reinterpret_cast<E*>(g.gu)[at] = (E)gu;
                reinterpret_cast<E*>(g.gdt)[at] = (E)gd;
                if (A.z) reinterpret_cast<E*>(g.gz)[at] = (E)gz;
            }
        }
        acc[0][w][lane] = sD, acc[1][w][lane] = sb;
        __syncthreads();
        if (w < 2 && live) {
            float v = acc[w][0][lane];
#pragma unroll
            for (int i = 1; i < kWaves; ++i) v += acc[w][i][lane];
            S.gDb[(row * 2 + w) * s.C + c] = v;
        }
        __syncthreads();  // acc has been read
    }
}

// The partial sums: A's gradients over the rows of blocks, those of D and the bias, B's and C's over
// the channel ranges.  Columns of (rows, cols) are added by 16 strips of rows at once, then the
// strips in order; one launch does all three, in as many workgroups each as `wg` says.
struct SelFold {
    unsigned wg[3];
    int64_t rows, share_rows;
};

template <class E>
__global__ __launch_bounds__(256) void sel_fold_kernel(SelShape s, SelBwdArgs g, SelBwdScratch S, SelFold f) {
    __shared__ float lds[16][17];
    const int Np = (s.N + 3) / 4 * 4;
    unsigned blk = blockIdx.x;
    if (blk < f.wg[0]) {
        const int64_t cols = (int64_t)Np * s.C, j = (int64_t)blk * 16 + (threadIdx.x & 15);
        const float v = fold_column(S.gA, f.rows, cols, j, lds);
        const int n = (int)(j / (4 * s.C)) * 4 + (int)(j & 3);
        if (threadIdx.x < 16 && j < cols && n < s.N) g.gA[j / 4 % s.C * s.N + n] = v;
        return;
    }
    blk -= f.wg[0];
    if (blk < f.wg[1]) {
        const int64_t cols = 2 * s.C, j = (int64_t)blk * 16 + (threadIdx.x & 15);
        const float v = fold_column(S.gDb, f.share_rows, cols, j, lds);
        float* const out = j < s.C ? g.gD : g.gbias;
        if (threadIdx.x < 16 && j < cols && out) out[j < s.C ? j : j - s.C] = v;
        return;
    }
    blk -= f.wg[1];
    const int64_t total = s.B * s.T * s.G * 2 * Np;
    for (int64_t i = (int64_t)blk * 256 + threadIdx.x; i < total; i += (int64_t)f.wg[2] * 256) {
        float v = 0.f;
        for (int64_t k = 0; k < S.cuts; ++k) v += S.gBC[k * total + i];
        const int j = (int)(i % (2 * Np)), n = j % Np;
        if (n < s.N) reinterpret_cast<E*>(j < Np ? g.gB : g.gC)[i / (2 * Np) * s.N + n] = (E)v;
    }
}

template <class E, int W>
hipError_t by_waves(const SelShape& s, const SelArgs& A, const SelBwdArgs& g, const float* bc, const float* keep,
                    const SelBwdScratch& S, hipStream_t st) {
    const int64_t blocks = sel_blocks(s);
    const int block = sel_block(s);
    const int ntiles = (int)ceil_div(s.N, kBwdNpt * W), group_tiles = (int)ceil_div(s.C / s.G, 64);
    hipLaunchKernelGGL((sel_reverse_kernel<E, W>), dim3((unsigned)(s.B * blocks * ntiles * s.G * group_tiles)),
                       dim3(64 * W), 0, st, s, A, (const E*)g.gy, bc, S.carry, S.sum, (int)blocks, block, group_tiles, ntiles);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) e = run_sel_join(s, A.A, S.carry, S.sum, blocks, g.gs_out, g.gs_in, true, st);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(s.B * blocks * ntiles * s.G * S.cuts));
    if (W < 4 || ntiles == 1) {
        hipLaunchKernelGGL((sel_gradient_kernel<E, W, true>), grid, dim3(64 * W), 0, st, s, A, g, bc, keep, S, (int)blocks,
                           block, ntiles);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((sel_gradient_kernel<E, 4, false>), grid, dim3(256), 0, st, s, A, g, bc, keep, S, (int)blocks, block,
                       ntiles);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t shares = sel_share_rows(s) / s.B, all = s.B * shares * ceil_div(s.C, 64);
    hipLaunchKernelGGL((sel_finish_kernel<E>), dim3((unsigned)(all < kFinishGroups ? all : kFinishGroups)), dim3(1024), 0,
                       st, s, A, g, S, shares, ntiles);
    return hipGetLastError();
}

template <class E>
hipError_t backward(const SelShape& s, const SelArgs& A, const SelBwdArgs& g, const float* bc, const float* keep,
                    const SelBwdScratch& W, hipStream_t st) {
    const int waves = sel_backward_plan(s).waves;
    hipError_t e = waves == 1   ? by_waves<E, 1>(s, A, g, bc, keep, W, st)
                   : waves == 2 ? by_waves<E, 2>(s, A, g, bc, keep, W, st)
                                : by_waves<E, 4>(s, A, g, bc, keep, W, st);
    if (e != hipSuccess) return e;
    SelFold f{};
    f.rows = s.B * sel_blocks(s);
    f.share_rows = sel_share_rows(s);
    f.wg[0] = (unsigned)ceil_div((int64_t)sel_n4(s) * 4 * s.C, 16);
    f.wg[1] = g.gD || g.gbias ? (unsigned)ceil_div(2 * s.C, 16) : 0;
    const int64_t wg = ceil_div(s.B * s.T * s.G * 2 * sel_n4(s) * 4, 256);
    f.wg[2] = (unsigned)(wg < 8192 ? wg : 8192);
    hipLaunchKernelGGL((sel_fold_kernel<E>), dim3(f.wg[0] + f.wg[1] + f.wg[2]), dim3(256), 0, st, s, g, W, f);
    return hipGetLastError();
}

}  // namespace

SelPlan sel_backward_plan(const SelShape& s) {
    SelPlan p{};
    p.npt = kBwdNpt;
    p.waves = s.N <= 4 ? 1 : s.N <= 8 ? 2 : 4;  // of a workgroup
    p.tiles_n = (int)ceil_div(s.N, kBwdNpt * p.waves);
    return p;
}

hipError_t run_sel_backward(const SelShape& s, const SelArgs& A, const SelBwdArgs& g, const float* bc, const float* keep,
                            const SelBwdScratch& W, hipStream_t st) {
    return s.dtype == kBf16 ? backward<bf16_t>(s, A, g, bc, keep, W, st) : backward<float>(s, A, g, bc, keep, W, st);
}

}  // namespace linrec
