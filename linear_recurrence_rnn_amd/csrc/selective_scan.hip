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
//
// 8 x 1024 tokens of 1536 channels, 16 states, bfloat16: 105 us, of which the segments' states take 38% and
// the outputs 51%; the vector unit is busy 87% and 94% of those.  A state and token costs it 24 cycles for 64
// of them; what a token and channel costs, once per pass, is a quarter to a third of all instructions.
// Channels of one group alone share B and C: groups that are not of whole 64s leave lanes idle.
#include <type_traits>

#include "selective_math.hpp"

namespace linrec {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// B and C as float32, (B,tiles,G,waves,16 tokens,2,npt), zero beyond N, for absent tokens and behind T.
// A workgroup takes 1024 floats of one tile.
template <class E>
__global__ __launch_bounds__(256) void sel_prepare_kernel(SelShape s, const E* __restrict__ Bm,
                                                          const E* __restrict__ Cm, float* __restrict__ bc, int npt,
                                                          int waves, int64_t tiles, int64_t parts) {
    const unsigned per = kSelTile * 2 * npt, all = per * waves * s.G;
    for (int64_t k = blockIdx.x; k < s.B * tiles * parts; k += gridDim.x) {
        const int64_t row = k / parts, b = row / tiles;  // row: b * tiles + tile
        const unsigned first = (unsigned)(k % parts) * 1024, t0 = (unsigned)(row % tiles) * kSelTile;
        const int64_t len = row_length(s, b);
        for (unsigned i = first + threadIdx.x; i < all && i < first + 1024; i += 256) {
            const unsigned j = i % per, w = i / per % waves, g = i / per / waves, r = j % (2 * npt);
            const unsigned t = t0 + j / (2 * npt);
            const int n = (int)(w * npt + r % npt);
            float v = 0.f;
            if (n < s.N && t < len) v = (float)((int)r < npt ? Bm : Cm)[((b * s.T + t) * s.G + g) * s.N + n];
            bc[row * all + i] = v;
        }
    }
}

// AGG: the segment's state from zero, and the sum of its steps, instead of outputs.
template <class E, int W, int NPT, bool AGG>
__global__ __launch_bounds__(64 * W) void sel_forward_kernel(SelShape s, SelArgs A, const float* __restrict__ bc,
                                                             float* __restrict__ agg, float* __restrict__ sum,
                                                             float* __restrict__ keep, int segs, int seg_tiles,
                                                             int group_tiles) {
    constexpr int TW = kSelTile / W;  // tokens a wave stages
    __shared__ f32x2 din[kSelTile][64];                          // d, d u
    __shared__ float part[AGG ? 1 : W][AGG ? 1 : kSelTile][64];  // the waves' shares of y
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int runs = AGG ? segs - 1 : segs;  // nothing needs the last segment's share
    unsigned blk = place_of(blockIdx.x, gridDim.x, (unsigned)(s.G * group_tiles));
    const int tile = (int)(blk % (unsigned)(s.G * group_tiles));
    blk /= (unsigned)(s.G * group_tiles);
    const int seg = (int)(blk % (unsigned)runs);
    const int64_t b = blk / (unsigned)runs;
    const int grp = tile / group_tiles, Cg = (int)(s.C / s.G);
    const int in_group = (tile % group_tiles) * 64 + lane;
    const bool live = in_group < Cg;
    const unsigned c = (unsigned)(grp * Cg + (live ? in_group : Cg - 1));
    const int T = (int)s.T, tiles = (T + kSelTile - 1) / kSelTile;
    const int t_begin = seg * seg_tiles * kSelTile;
    const int t_end = seg == segs - 1 ? T : t_begin + seg_tiles * kSelTile;
    const int len = (int)row_length(s, b);
    const int n0 = w * NPT, Np = (s.N + 3) / 4 * 4;

    float h[NPT], a2[NPT];
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        const int n = n0 + i;
        a2[i] = n < s.N ? A.A[(int64_t)c * s.N + n] * kLog2e : 0.f;
        h[i] = 0.f;
        if (!AGG && n < s.N) {
            if (segs > 1) h[i] = agg[state_at(s, b * segs + seg, n, c)];
            else if (A.s_in) h[i] = A.s_in[(b * s.C + c) * s.N + n];
        }
    }
    const float bias = A.bias ? A.bias[c] : 0.f;
    const float Dc = A.D ? A.D[c] : 0.f;
    float total = 0.f;

    // This wave's tokens of a tile, read while the tile before is worked on.  Absent tokens are read as the last
    // that is there (or the segment's first), a gate that was not given as u: neither is used.
    const bool gated = A.z != nullptr, soft = s.softplus != 0;
    const void* const zp = gated ? A.z : A.u;
    E ur[TW], dr[TW], zr[TW];
    const unsigned C = (unsigned)s.C;
    const int t_stop = len < t_end ? (len > t_begin ? len : t_begin + 1) : t_end;
    const auto fetch = [&](int t0, int64_t at0) {  // at0: the tile's first element
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const int k = t0 + w * TW + i < t_stop ? w * TW + i : t_stop - 1 - t0;
            const unsigned at = ((unsigned)k * C + c) * (unsigned)sizeof(E);
            ur[i] = load_elem<E>(elems<E>(A.u, at0), at);
            dr[i] = load_elem<E>(elems<E>(A.dt, at0), at);
            if (!AGG) zr[i] = load_elem<E>(elems<E>(zp, at0), at);
        }
    };
    // Where this tile's elements, B and C, and kept states are.
    int64_t base = (b * T + t_begin) * s.C;
    const int64_t first = b * tiles + t_begin / kSelTile;
    const float* row = bc + ((first * s.G + grp) * W + w) * (kSelTile * 2 * NPT);
    float* kept = keep + (first * Np + n0 / 4 * 4) * s.C + (n0 & 3);
    int next = t_begin;  // the tile on its way
    int64_t next_base = base;
    fetch(next, next_base);
    for (int t0 = t_begin; t0 < t_end; t0 += kSelTile) {
        if constexpr (!AGG) {
            if (keep && live) {
                if constexpr (NPT % 4 == 0) {
#pragma unroll
                    for (int i = 0; i < NPT; i += 4) {
                        const f32x4 v = {h[i], h[i + 1], h[i + 2], h[i + 3]};
                        if (n0 + i < Np) store_as<f32x4>(kept + i * s.C, c * 16, v);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < NPT; ++i)
                        if (n0 + i < Np) store_as<float>(kept + i, c * 16, h[i]);
                }
            }
            kept += Np * s.C;
        }
        // Whether a token is there is the same for the whole wave; d and d u of an absent one, or of a
        // lane without a channel, are zero, which leaves the states alone.
        float u[TW], z[TW];
        if (t0 < len) {
            float d[TW];
#pragma unroll
            for (int i = 0; i < TW; ++i) d[i] = (float)dr[i] + bias;
            if (soft) {  // outside of the loop: the tokens' chains of instructions then run side by side
                float sig;
#pragma unroll
                for (int i = 0; i < TW; ++i) d[i] = softplus(d[i], sig);
            }
#pragma unroll
            for (int i = 0; i < TW; ++i) {
                const bool there = live && t0 + w * TW + i < len;
                u[i] = (float)ur[i];
                if (!AGG) z[i] = (float)zr[i];
                const f32x2 v = {there ? d[i] : 0.f, there ? d[i] * u[i] : 0.f};
                din[w * TW + i][lane] = v;
            }
        }
        if (next + kSelTile < t_stop) next += kSelTile, next_base += kSelTile * s.C;
        fetch(next, next_base);
        __syncthreads();
        if (t0 < len) {
            float subtotal = 0.f;
            SelGroup<NPT> grp_of[2];
            grp_of[0].fetch(row, din, lane, 0);
#pragma unroll
            for (int q = 0; q < SelGroup<NPT>::kGroups; ++q) {
                const SelGroup<NPT>& v = grp_of[q & 1];
                if (q + 1 < SelGroup<NPT>::kGroups) grp_of[(q + 1) & 1].fetch(row, din, lane, q + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int k = 0; k < SelGroup<NPT>::kTok; ++k) {
                    const f32x2 x = v.x[k];
                    float y = 0.f;
#pragma unroll
                    for (int i = 0; i < NPT; ++i) {
                        h[i] = fmaf(fast_exp2(x[0] * a2[i]), h[i], x[1] * v.B(k, i));
                        y = fmaf(v.C(k, i), h[i], y);
                    }
                    if constexpr (AGG) subtotal += x[0];
                    else part[w][q * SelGroup<NPT>::kTok + k][lane] = y;
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            total += subtotal;
        }
        __syncthreads();
        if constexpr (!AGG) {
            if (A.y) {
                float y[TW];
#pragma unroll
                for (int i = 0; i < TW; ++i) {
                    y[i] = Dc * u[i];
#pragma unroll
                    for (int k = 0; k < W; ++k) y[i] += part[k][w * TW + i][lane];
                    const float gate = z[i] * logistic(z[i]);
                    y[i] = where(t0 + w * TW + i < len, y[i] * (gated ? gate : 1.f));
                }
                if (live) {
                    void* const out = (void*)elems<E>(A.y, base);
#pragma unroll
                    for (int i = 0; i < TW; ++i) {
                        if (t0 + w * TW + i >= t_end) break;
                        store_elem<E>(out, ((unsigned)(w * TW + i) * C + c) * (unsigned)sizeof(E), y[i]);
                    }
                }
            }
        }
        base += kSelTile * s.C;
        row += s.G * W * (kSelTile * 2 * NPT);
    }
    if (!live) return;
    if constexpr (AGG) {
#pragma unroll
        for (int i = 0; i < NPT; ++i)
            if (n0 + i < Np) agg[state_at(s, b * segs + seg, n0 + i, c)] = h[i];
        if (w == 0) sum[(b * segs + seg) * s.C + c] = total;
    } else if (seg == segs - 1 && A.s_out) {
#pragma unroll
        for (int i = 0; i < NPT; ++i)
            if (n0 + i < s.N) A.s_out[(b * s.C + c) * s.N + n0 + i] = h[i];
    }
}

// One element of every state and row: the blocks' shares become the states that enter them.  Bound by the loads'
// latency, one block after the other, hence eight at once: 16384 tokens of 256 channels 128 -> 72 us.
constexpr int kAhead = 8;

// x 2^p.  States that grow (A above zero, or steps below) may grow over a block by more than a float32 holds and be none
// the less one, or zero: the whole part of p goes to the exponent.  A p beyond 1000 either way leaves nothing or infinity.
__device__ __forceinline__ float grown(float x, float p) {
    p = fminf(fmaxf(p, -1000.f), 1000.f);
    const float whole = floorf(p);
    return __builtin_amdgcn_ldexpf(x * fast_exp2(p - whole), (int)whole);
}

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
    // What leaves the last block forwards is not asked for, and its share was not formed.
    const int64_t known = REV ? blocks : blocks - 1;
    const auto place = [&](int64_t i) { return b * blocks + (REV ? blocks - 1 - i : i); };
    // Loads of kAhead blocks at once, and ahead of the stores of those before: not one by one, where they are used.
    float own[2][kAhead], d[2][kAhead];
    const auto load = [&](int64_t i, float (&o)[kAhead], float (&f)[kAhead]) {
#pragma unroll
        for (int r = 0; r < kAhead; ++r) {
            const int64_t k = place(i + r < known ? i + r : known - 1);
            o[r] = v[k * per + e], f[r] = sum[k * s.C + c];
        }
    };
    if (known > 0) load(0, own[0], d[0]);
    const auto group = [&](int64_t i, float (&o)[kAhead], float (&f)[kAhead], float (&o1)[kAhead], float (&f1)[kAhead]) {
        load(i + kAhead, o1, f1);
#pragma unroll
        for (int r = 0; r < kAhead; ++r) asm volatile("" : "+v"(o[r]), "+v"(f[r]));
#pragma unroll
        for (int r = 0; r < kAhead; ++r) {
            if (i + r >= known) break;
            v[place(i + r) * per + e] = x;
            x = grown(x, a2 * f[r]) + o[r];
        }
    };
    for (int64_t i = 0; i < known; i += 2 * kAhead) {
        group(i, own[0], d[0], own[1], d[1]);
        if (i + kAhead < known) group(i + kAhead, own[1], d[1], own[0], d[0]);
    }
    if (!REV) v[place(blocks - 1) * per + e] = x;
    if (out && n < s.N) out[at] = x;
}

// v of lane `I` of each LN lanes (of each four, where they are more).
template <int LN, int I>
__device__ __forceinline__ float of_lane(float v) {
    if constexpr (LN == 1) return v;
    constexpr int ctrl = LN == 2 ? (I | I << 2 | (2 + I) << 4 | (2 + I) << 6) : I * 0x55;  // quad_perm
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, true));
}

// v summed over LN lanes, in every one of them.
template <int LN>
__device__ __forceinline__ float over_lanes(float v) {
    if constexpr (LN > 1) v = add_dpp<0xb1>(v);   // quad_perm [1,0,3,2]
    if constexpr (LN > 2) v = add_dpp<0x4e>(v);   // quad_perm [2,3,0,1]
    if constexpr (LN > 4) v = add_dpp<0x141>(v);  // row_half_mirror
    if constexpr (LN > 8) v = add_dpp<0x140>(v);  // row_mirror
    if constexpr (LN > 16) {
        const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}

// One token.  LN lanes hold a channel's states, four each, and M neighbouring channels of them; what
// depends on the channel alone is formed once, channel i's by lane i.  Bound by memory, the state read and
// written (64 users, 5120 channels of 16 states: 10.2 us, 4.4 TB/s); VEC: 16 bytes of it at once.
template <class E, int LN, bool VEC>
__global__ __launch_bounds__(256) void sel_step_kernel(SelShape s, SelArgs A, unsigned col_blocks) {
    constexpr int M = LN < 4 ? LN : 4, kChan = 256 / LN * M;  // channels of a workgroup
    const unsigned b = blockIdx.x / col_blocks, col = blockIdx.x % col_blocks;
    const unsigned l = threadIdx.x % LN, c0 = col * kChan + threadIdx.x / LN * M;
    const int n0 = (int)l * 4;
    const unsigned C = (unsigned)s.C, Cg = C / (unsigned)s.G;
    const int64_t rows = (int64_t)b * s.C;  // b * C: of the state's rows, and of u
    float h[M][4], a[M][4], Bv[M][4], Cv[M][4];
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const bool live = c0 + i < C;
        const int64_t at = (live ? c0 + i : 0u) * (int64_t)s.N + n0;
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i][j] = a[i][j] = 0.f;
        if constexpr (VEC) {
            if (live && n0 < s.N) {
                load16<float>(A.A + at, a[i]);
                if (A.s_in) load16<float>(A.s_in + rows * s.N + at, h[i]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (live && n0 + j < s.N) {
                    a[i][j] = A.A[at + j];
                    if (A.s_in) h[i][j] = A.s_in[rows * s.N + at + j];
                }
        }
    }
    // B and C: the same for all channels of one group.
#pragma unroll
    for (int i = 0; i < M; ++i) {
        if (i > 0 && s.G == 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) Bv[i][j] = Bv[0][j], Cv[i][j] = Cv[0][j];
            continue;
        }
        const unsigned c = c0 + i < C ? c0 + i : C - 1, g = s.G == 1 ? 0u : c / Cg;
        const int64_t at = ((int64_t)b * s.G + g) * s.N;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + j < s.N ? n0 + j : 0;
            Bv[i][j] = n0 + j < s.N ? (float)reinterpret_cast<const E*>(A.Bm)[at + n] : 0.f;
            Cv[i][j] = n0 + j < s.N ? (float)reinterpret_cast<const E*>(A.Cm)[at + n] : 0.f;
        }
    }
    // This lane's own channel, the same for every fourth lane.
    const unsigned own = l % M;
    const bool mine = l < (unsigned)M && c0 + own < C;
    const unsigned c = c0 + own < C ? c0 + own : C - 1;
    const float u = (float)reinterpret_cast<const E*>(A.u)[rows + c];
    float d = (float)reinterpret_cast<const E*>(A.dt)[rows + c] + (A.bias ? A.bias[c] : 0.f), sig, gate = 1.f;
    const float Dc = A.D ? A.D[c] : 0.f;
    if (A.z) {
        const float z = (float)reinterpret_cast<const E*>(A.z)[rows + c];
        gate = z * logistic(z);
    }
    if (s.softplus) d = softplus(d, sig);
    const float du = d * u;
    float out = 0.f;
    const auto channel = [&](auto index) {
        constexpr int i = decltype(index)::value;
        if constexpr (i < M) {
            const float di = of_lane<LN, i>(d), xi = of_lane<LN, i>(du);
            float y = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[i][j] = fmaf(fast_exp2(di * (a[i][j] * kLog2e)), h[i][j], xi * Bv[i][j]);
                y = fmaf(Cv[i][j], h[i][j], y);
            }
            y = over_lanes<LN>(y);
            out = own == (unsigned)i ? y : out;
            if (c0 + i < C && n0 < s.N) {
                float* const o = A.s_out + (rows + c0 + i) * s.N + n0;
                if constexpr (VEC) {
                    store16<float>(o, h[i]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n0 + j < s.N) o[j] = h[i][j];
                }
            }
        }
    };
    channel(std::integral_constant<int, 0>());
    channel(std::integral_constant<int, 1>());
    channel(std::integral_constant<int, 2>());
    channel(std::integral_constant<int, 3>());
    if (mine) reinterpret_cast<E*>(A.y)[rows + c] = (E)(fmaf(Dc, u, out) * gate);
}

template <class E, int LN>
hipError_t step(const SelShape& s, const SelArgs& A, hipStream_t st) {
    const int64_t col_blocks = ceil_div(s.C, 256 / LN * (LN < 4 ? LN : 4));
    const dim3 grid((unsigned)(s.B * col_blocks));
    const bool vec = s.N % 4 == 0 && ((uintptr_t)A.A | (uintptr_t)A.s_in | (uintptr_t)A.s_out) % 16 == 0;
    if (vec) hipLaunchKernelGGL((sel_step_kernel<E, LN, true>), grid, dim3(256), 0, st, s, A, (unsigned)col_blocks);
    else hipLaunchKernelGGL((sel_step_kernel<E, LN, false>), grid, dim3(256), 0, st, s, A, (unsigned)col_blocks);
    return hipGetLastError();
}

template <class E>
hipError_t step_by_states(const SelShape& s, const SelArgs& A, hipStream_t st) {
    if (s.N <= 4) return step<E, 1>(s, A, st);
    if (s.N <= 8) return step<E, 2>(s, A, st);
    if (s.N <= 16) return step<E, 4>(s, A, st);
    if (s.N <= 32) return step<E, 8>(s, A, st);
    if (s.N <= 64) return step<E, 16>(s, A, st);
    return step<E, 32>(s, A, st);
}

template <class E, int W, int NPT>
hipError_t forward(const SelShape& s, const SelArgs& A, const SelPlan& p, const SelScratch& S, float* keep,
                   hipStream_t st) {
    const int group_tiles = (int)ceil_div(s.C / s.G, 64);
    const int64_t wg = s.B * s.G * group_tiles;
    const int segs = (int)p.segs, seg_tiles = (int)p.seg_tiles;
    if constexpr (!(W == 8 && NPT == 2)) {  // whole rows alone are split like that
        if (segs > 1) {
            hipLaunchKernelGGL((sel_forward_kernel<E, W, NPT, true>), dim3((unsigned)(wg * (segs - 1))), dim3(64 * W), 0, st,
                               s, A, S.bc, S.agg, S.sum, (float*)nullptr, segs, seg_tiles, group_tiles);
            hipError_t e = hipGetLastError();
            if (e == hipSuccess) e = run_sel_join(s, A.A, S.agg, S.sum, p.segs, A.s_in, nullptr, false, st);
            if (e != hipSuccess) return e;
        }
    }
    hipLaunchKernelGGL((sel_forward_kernel<E, W, NPT, false>), dim3((unsigned)(wg * segs)), dim3(64 * W), 0, st, s, A,
                       S.bc, S.agg, S.sum, keep, segs, seg_tiles, group_tiles);
    return hipGetLastError();
}

template <class E>
hipError_t forward_by_states(const SelShape& s, const SelArgs& A, const SelPlan& p, const SelScratch& S, float* keep,
                             hipStream_t st) {
    if (p.npt == 1) return forward<E, 1, 1>(s, A, p, S, keep, st);
    if (p.npt == 2) return p.waves == 1 ? forward<E, 1, 2>(s, A, p, S, keep, st) : forward<E, 8, 2>(s, A, p, S, keep, st);
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
    p.tiles_n = 1;
    p.npt = s.N <= 1 ? 1 : s.N <= 2 ? 2 : s.N <= 16 ? 4 : s.N <= 64 ? 8 : 16;
    p.waves = s.N <= 4 ? 1 : s.N <= 8 ? 2 : s.N <= 32 ? 4 : 8;
    // Segments until there are ten waves a SIMD, of which it holds three (one wave a workgroup) to eight at once: 8 x 4096
    // tokens of 2560 channels take 537 us, 558 with six waves, 549 with sixteen; with 8 states 390, 427 and 391; 32768 of 2048
    // 471, 493 and 462.
    const int64_t wg = s.B * s.G * ceil_div(s.C / s.G, 64), tiles = sel_tiles(s);
    int64_t segs = 10240 / (wg * p.waves);
    // Of two tiles at least, of four in rows of more than 128 tiles, where the states that enter the segments would cost
    // more: 512 tokens of 1536 channels take 26.0 us with twos, 28.7 with fours, 4096 of 256 36.5 and 32.1.  Of one where
    // that leaves SIMDs with two waves, in up to 64 tiles: 500 tokens of 256 take 18.1 us, 20.1 with twos, but 1024 of
    // 1536, with six waves a SIMD, 36.3 and 30.9.
    const int64_t most = tiles <= 64 && wg * p.waves * tiles <= 2048 ? tiles : tiles <= 128 ? tiles / 2 : tiles / 4;
    if (segs > most) segs = most;
    // Each segment but the last is walked twice, so that cut rows keep the chip busy for a time that grows with the
    // workgroups, where whole ones take what one of them takes, alone on its CU or with others, however few they are.
    // Microseconds a tile of 16 tokens, by the number of states: a whole row's workgroup alone on its CU (of 256), one with
    // others, and a workgroup's part of cut rows' time.
    const bool halved = p.npt == 4 && p.waves == 4;  // whole rows may be, below
    const double us[6][3] = {{3.3, 4.4, 0.0033}, {2.45, 3.8, 0.0046}, {1.7, 2.5, 0.0065},
                             {3.27, 4.4, 0.0116}, {4.25, 6.95, 0.0235}, {7.75, 13.3, 0.046}};
    const double* const tile_us = us[s.N <= 4 ? 0 : s.N <= 8 ? 1 : s.N <= 16 ? 2 : s.N <= 32 ? 3 : s.N <= 64 ? 4 : 5];
    const double saved = (double)tiles * (tile_us[wg > 256] - tile_us[2] * (double)wg);
    // Cutting costs two launches and the segments' states written and read.  That model and the measured times of both
    // sides, 1536 or 2560 channels in bfloat16, whole / cut: of 16 states 8 x 128 tokens 20.6 / 31.5 us, 8 x 256 33.7 /
    // 44.3, 4 x 256 33.5 / 31.9, 8 x 512 60 / 68, 8 x 1024 113 / 105, 9 x 4096 651 / 635 (seven segments), 10 x 4096 654 /
    // 692 (six), 8 x 4096 631 / 532 (eight); of 8 24 x 256 57 / 66, 20 x 4096 1114 / 945, 24 x 4096 1124 / 1128; of 4
    // 12 x 128 33.4 / 29.6, 32 x 128 34.4 / 39.1, 32 x 4096 1226 / 1060, 42 x 512 157 / 210; of 32 4 x 128 35 / 38, 2 x 128
    // 34 / 30, 9 x 4096 1152 / 1100, 10 x 4096 1159 / 1216; of 64 4 x 128 44 / 59, 4 x 512 144 / 117, 8 x 1024 281 / 317.
    if (segs < 4 || saved < 16. + 2.5e-4 * (double)(wg * segs) * s.N) segs = 1;
    p.seg_tiles = ceil_div(tiles, segs);
    p.segs = ceil_div(tiles, p.seg_tiles);
    // Whole rows too few for four waves a SIMD: half the states a wave.  77 tokens of 1536 channels take 12.1 us for
    // 15.2, 12 x 1024 of 2560 173 for 182, but 24 x 1024 302 for 291.
    if (p.segs == 1 && halved && wg * 8 <= 4096) p.npt = 2, p.waves = 8;
    return p;
}

size_t sel_bc_floats(const SelShape& s, const SelPlan& p) {
    return (size_t)(s.B * sel_tiles(s) * kSelTile * s.G) * 2 * (size_t)(p.npt * p.waves * p.tiles_n);
}

hipError_t run_sel_prepare(const SelShape& s, const SelArgs& A, const SelPlan& p, float* bc, hipStream_t st) {
    const int64_t rows = s.B * sel_tiles(s), parts = ceil_div((int64_t)sel_bc_floats(s, p) / rows, 1024);
    const dim3 grid((unsigned)(rows * parts < (1 << 20) ? rows * parts : 1 << 20));
    const int waves = p.tiles_n * p.waves;
    if (s.dtype == kBf16)
        hipLaunchKernelGGL((sel_prepare_kernel<bf16_t>), grid, dim3(256), 0, st, s, (const bf16_t*)A.Bm,
                           (const bf16_t*)A.Cm, bc, p.npt, waves, sel_tiles(s), parts);
    else
        hipLaunchKernelGGL((sel_prepare_kernel<float>), grid, dim3(256), 0, st, s, (const float*)A.Bm,
                           (const float*)A.Cm, bc, p.npt, waves, sel_tiles(s), parts);
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
    return s.dtype == kBf16 ? step_by_states<bf16_t>(s, A, st) : step_by_states<float>(s, A, st);
}

}  // namespace linrec
