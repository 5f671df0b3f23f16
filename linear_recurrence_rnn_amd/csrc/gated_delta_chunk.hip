// gated_delta_chunk.hip -- the gated delta rule in chunks of 64 tokens on the matrix units.
//
// Within a chunk, with gam the decays cumulated from its start and S the state before it:
//   G_ij = e^{gam_i - gam_j} k_i.k_j   (i > j)       Z = V - diag(e^gam) K S
//   X = (I + G diag(beta))^{-1} Z                    (x_t of the recurrence, all 64 at once)
//   O = scale diag(e^gam) Q S + P (beta X),   P_ij = scale e^{gam_i - gam_j} q_i.k_j  (i >= j)
//   S' = e^{gam_63} S + K^T diag(e^{gam_63 - gam}) (beta X)
// Every exponent is <= 0, so nothing overflows.  The inverse depends on K, g and beta alone and
// is formed for all chunks at once by the first kernel; the second walks the chunks of a head
// with the state in registers.
#include "gated_delta.hpp"
#include "delta_tile.hpp"

namespace linrec {

namespace {

// ---- the chunks' inverses -------------------------------------------------------------------
// One wave a chunk.  K's fragments serve as both operands of K K^T (the A and B layouts of a
// matrix and its transpose are one).  Lane c then solves for column c of the inverse:
//   t_i = [i = c] - sum_{j<i} A_ij t_j,   A = G diag(beta)
// with the rows of A read from LDS by all lanes at once.
template <class E, int KT, bool VEC>
__global__ __launch_bounds__(64) void delta_prepare_kernel(DeltaShape s, DeltaFwdArgs A, DeltaChunks W, int nc) {
    constexpr int NI = kTerms<E>;
    constexpr int LD = 68;
    __shared__ float a[kChunk * LD];
    __shared__ double gam[kChunk];
    __shared__ float bet[kChunk];
    const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
    const int64_t blk = blockIdx.x;
    const int n = (int)(blk % nc);
    const int64_t bh = blk / nc;
    const int h = (int)(bh % s.Hv), hk = h / (s.Hv / s.Hk);
    const int64_t b = bh / s.Hv;
    const int len = row_length(s, b), t0 = n * kChunk;
    if (t0 >= len) return;  // nothing of this chunk is used
    {
        const bool live = t0 + lane < len;
        const int64_t at = (b * s.T + t0 + lane) * s.Hv + h;
        const double d = live ? decay_of((float)reinterpret_cast<const E*>(A.g)[at]) : 0.0;
        const double c = wave_cumsum(d);
        gam[lane] = c;
        bet[lane] = live ? (float)reinterpret_cast<const E*>(A.beta)[at] : 0.f;
        W.gam[blk * kChunk + lane] = c;
    }
    Frag<NI> kf[4][KT];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int row = t0 + 16 * t + r;
        const E* p = reinterpret_cast<const E*>(A.k) + ((b * s.T + row) * s.Hk + hk) * (int64_t)s.Dk;
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
            E x[8];
            load8<E, VEC>(p + 32 * kk + 8 * g, 32 * kk + 8 * g, s.Dk, row < len, x);
            kf[t][kk] = to_frag<E>(x);
        }
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int jt = 0; jt <= it; ++jt) {
            f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) mma(c, kf[it][kk], kf[jt][kk]);
            const int j = 16 * jt + r;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * it + 4 * g + e;
                a[i * LD + j] = i > j ? c[e] * decay_exp(gam[i], gam[j]) * bet[j] : 0.f;
            }
        }
    __syncthreads();
    float t[kChunk];
    float* out = W.tinv + blk * (kChunk * kChunk) + lane;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        float x = i == lane ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < i; ++j) x = fmaf(-a[i * LD + j], t[j], x);
        t[i] = x;
        out[i * kChunk] = x;
    }
}

// ---- the chain over a head's chunks -----------------------------------------------------------
// A workgroup of four waves owns 64*CT columns of the value channels of one head, a wave 16*CT
// of them, all rows of the state (32*KT, zero past Dk).  K, Q, the inverse and P lie in LDS as
// bfloat16 terms, shared by the waves; V comes from memory in the A layout and is turned into
// the D layout by a product with the identity, which is exact.
//
// Terms: the state and what flows into it (Z, beta X) are taken as three bfloat16 terms, so
// that S keeps float32 precision over any number of chunks; the outputs of bfloat16 calls take
// two terms of S, P and beta X, so that the rounding of the output itself is all there is.
template <class E, int KT, int CT, bool VEC>
struct FwdLds {
    static constexpr int NI = kTerms<E>, NO = NI == 1 ? 2 : 3;  // terms of inputs, of the outputs' operands
    static constexpr int LK = 32 * KT + 8, LT = kChunk + 8;
    bf16_t k[NI][kChunk][LK], q[NI][kChunk][LK];
    bf16_t t[3][kChunk][LT];
    bf16_t p[NO][kChunk][LT];
    double gam[kChunk];
    float eg[kChunk], ew[kChunk], be[kChunk];
};

// What the chain leaves: o, and what the backward starts from (of type KE).
constexpr int kOut = 1, kKeep = 2;

template <class E, class KE, int KT, int CT, bool VEC, int MODE>
__global__ __launch_bounds__(256) void delta_forward_kernel(DeltaShape s, DeltaFwdArgs A, DeltaChunks W, int nc,
                                                            int ntile) {
    typedef FwdLds<E, KT, CT, VEC> Lds;
    constexpr int NI = kTerms<E>, NO = Lds::NO, NS = 3;
    constexpr bool OUT = MODE & kOut, KEEP = MODE & kKeep;
    extern __shared__ __align__(16) char lds_raw[];
    Lds& L = *reinterpret_cast<Lds*>(lds_raw);
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int tile = (int)(blockIdx.x % ntile);
    const int64_t bh = blockIdx.x / ntile;
    const int h = (int)(bh % s.Hv), hk = h / (s.Hv / s.Hk);
    const int64_t b = bh / s.Hv;
    const int len = row_length(s, b);
    const int c0 = tile * 64 * CT + wave * 16 * CT;  // this wave's first value channel
    const int Dk = s.Dk, Dv = s.Dv;
    const int nblk = ntile * 4 * CT;  // blocks of 16 value channels

    // State: D tiles S[kk][half][ct], rows 32kk + tile_row(m, half), columns c0 + 16ct + r.
    f32x4 S[KT][2][CT];
    const int64_t sb = bh * (int64_t)Dk * Dv;
#pragma unroll
    for (int kk = 0; kk < KT; ++kk)
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = 32 * kk + 8 * g + 4 * half + e, col = c0 + 16 * ct + r;
                    S[kk][half][ct][e] = (A.s_in && row < Dk && col < Dv) ? A.s_in[sb + (int64_t)row * Dv + col] : 0.f;
                }
    const Frag<1> ident[2] = {identity_frag(0), identity_frag(1)};

    const int nlive = (len + kChunk - 1) / kChunk;
    for (int n = 0; n < nlive; ++n) {
        const int t0 = n * kChunk;
        const int64_t cb = bh * nc + n;
        __syncthreads();  // the previous chunk's tiles have been read
        // Stage K, Q (4 lanes a row), the inverse, the decays.
        {
            stage_rows<E, KT, VEC>(A.k, s, b, s.Hk, hk, Dk, t0, len, L.k);
            if constexpr (OUT) stage_rows<E, KT, VEC>(A.q, s, b, s.Hk, hk, Dk, t0, len, L.q);
            stage_inverse(W.tinv + cb * (kChunk * kChunk), L.t);
            if (tid < kChunk) {
                const bool on = t0 + tid < len;
                const double gm = W.gam[cb * kChunk + tid], end = W.gam[cb * kChunk + kChunk - 1];
                L.gam[tid] = gm;
                L.eg[tid] = decay_exp(gm, 0.0);
                L.ew[tid] = decay_exp(end, gm);
                L.be[tid] = on ? (float)reinterpret_cast<const E*>(A.beta)[(b * s.T + t0 + tid) * s.Hv + h] : 0.f;
            }
        }
        __syncthreads();
        // P, rows 16*wave..: tiles of K Q^T (rows j, columns i), stored as P[i][j].
        if constexpr (OUT) {
            const int i = 16 * wave + r;
            const double gi = L.gam[i];
            for (int jt = 0; jt <= (wave | 1); ++jt) {
                f32x4 c = {0.f, 0.f, 0.f, 0.f};
                if (jt <= wave)
#pragma unroll
                    for (int kk = 0; kk < KT; ++kk) {
                        const int col = 32 * kk + 8 * g;
                        mma(c, read_row<NI>(L.k, 16 * jt + r, col), read_row<NI>(L.q, i, col));
                    }
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 16 * jt + 4 * g + e;
                    x[e] = j <= i ? s.scale * decay_exp(gi, L.gam[j]) * c[e] : 0.f;
                    x[4 + e] = 0.f;
                }
                const Frag<NO> f = split<NO>(x);
#pragma unroll
                for (int m = 0; m < NO; ++m)
                    *reinterpret_cast<bf16x4*>(&L.p[m][i][16 * jt + 4 * g]) =
                        __builtin_shufflevector(f.t[m], f.t[m], 0, 1, 2, 3);
            }
        }
        // Z = V - e^gam K S and the state's part of O^T.
        f32x4 Z[2][2][CT], O[4][CT];  // Z: rows 32*k2 + tile_row(m, half); O^T: columns 16*tt + r
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    Z[k2][half][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
                    O[2 * k2 + half][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
            Frag<NS> fs[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) fs[ct] = split_tiles<NS>(S[kk][0][ct], S[kk][1][ct]);
            if constexpr (KEEP)  // S before the chunk, turned so that a lane holds 4 value channels
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int which = 0; which < 2; ++which) {
                        f32x4 x = {0.f, 0.f, 0.f, 0.f};
                        mma<NS, 1, kKeptSum<KE>, 1>(x, fs[ct], ident[which]);
                        store4<KE>(reinterpret_cast<KE*>(W.s0) +
                                      ((cb * nblk + c0 / 16 + ct) * (32 * KT) + 32 * kk + 16 * which + r) * 16 + 4 * g,
                                  x);
                    }
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const Frag<NI> fk = read_row<NI>(L.k, 32 * k2 + tile_row(r, half), 32 * kk + 8 * g);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) mma(Z[k2][half][ct], fk, fs[ct]);
                    if constexpr (OUT) {
                        const Frag<NI> fq = read_row<NI>(L.q, 16 * (2 * k2 + half) + r, 32 * kk + 8 * g);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) mma<NS, NI, NO, NI>(O[2 * k2 + half][ct], fs[ct], fq);
                    }
                }
        }
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = t0 + 32 * k2 + tile_row(r, half);
                f32x4 v[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) v[ct] = f32x4{0.f, 0.f, 0.f, 0.f};
                E x[8];
                const int c = c0 + 8 * g;  // 32 columns of one A operand; 16 of them with CT = 1
                const bool on = row < len && (CT == 2 || g < 2);
                load8<E, VEC>(reinterpret_cast<const E*>(A.v) + ((b * s.T + row) * s.Hv + h) * (int64_t)Dv + c, c, Dv,
                              on, x);
                const Frag<NI> fv = to_frag<E>(x);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) mma<NI, 1>(v[ct], fv, ident[ct]);
                const f32x4 eg = *reinterpret_cast<const f32x4*>(&L.eg[32 * k2 + 8 * g + 4 * half]);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        Z[k2][half][ct][e] = fmaf(-eg[e], Z[k2][half][ct][e], v[ct][e]);
                const float so = s.scale * L.eg[16 * (2 * k2 + half) + r];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) O[2 * k2 + half][ct] *= so;
            }
        // X = inverse Z, then U = beta X.
        f32x4 U[2][2][CT];
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) U[k2][half][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kz = 0; kz < 2; ++kz) {
            Frag<NS> fz[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) fz[ct] = split_tiles<NS>(Z[kz][0][ct], Z[kz][1][ct]);
#pragma unroll
            for (int k2 = kz; k2 < 2; ++k2)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const Frag<3> ft = read_row<3>(L.t, 32 * k2 + tile_row(r, half), 32 * kz + 8 * g);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) mma(U[k2][half][ct], ft, fz[ct]);
                }
        }
        Frag<NO> fu[2][CT];   // beta X for the outputs
        Frag<NS> fw[2][CT];   // e^{gam_63 - gam} beta X for the state
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                f32x4 w[2];
                if constexpr (KEEP) {  // X, likewise
                    const Frag<kKeptSum<KE>> fx = split_tiles<kKeptSum<KE>>(U[k2][0][ct], U[k2][1][ct]);
#pragma unroll
                    for (int which = 0; which < 2; ++which) {
                        f32x4 x = {0.f, 0.f, 0.f, 0.f};
                        mma<kKeptSum<KE>, 1>(x, fx, ident[which]);
                        store4<KE>(reinterpret_cast<KE*>(W.x) +
                                      ((cb * nblk + c0 / 16 + ct) * kChunk + 32 * k2 + 16 * which + r) * 16 + 4 * g,
                                  x);
                    }
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int row = 32 * k2 + 8 * g + 4 * half;
                    U[k2][half][ct] *= *reinterpret_cast<const f32x4*>(&L.be[row]);
                    w[half] = U[k2][half][ct] * *reinterpret_cast<const f32x4*>(&L.ew[row]);
                }
                fu[k2][ct] = split_tiles<NO>(U[k2][0][ct], U[k2][1][ct]);
                fw[k2][ct] = split_tiles<NS>(w[0], w[1]);
            }
        // S' = e^{gam_63} S + K^T w.
        const float end = L.eg[kChunk - 1];
#pragma unroll
        for (int kk = 0; kk < KT; ++kk)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) S[kk][half][ct] *= end;
#pragma unroll
                for (int k2 = 0; k2 < 2; ++k2) {
                    const Frag<NI> ft = read_col<NI, true>(L.k, 32 * k2, 32 * kk, half);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) mma(S[kk][half][ct], ft, fw[k2][ct]);
                }
            }
        if constexpr (OUT) {
        __syncthreads();  // P is there
        // O^T += U^T P^T.
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
            for (int k2 = 0; k2 <= tt / 2; ++k2) {
                const Frag<NO> fp = read_row<NO>(L.p, 16 * tt + r, 32 * k2 + 8 * g);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) mma(O[tt][ct], fu[k2][ct], fp);
            }
            const int t = t0 + 16 * tt + r;
            if (t < s.T) {
                E* op = reinterpret_cast<E*>(A.o) + ((b * s.T + t) * s.Hv + h) * (int64_t)Dv;
                const bool live = t < len;
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const f32x4 x = live ? O[tt][ct] : f32x4{0.f, 0.f, 0.f, 0.f};
                    store_cols<E, VEC>(op, c0 + 16 * ct + 4 * g, Dv, x);
                }
            }
        }
        }
    }
    // Chunks past the row's length: zero outputs.
    if constexpr (OUT)
    for (int64_t t = (int64_t)nlive * kChunk + tid / 64; t < s.T; t += 4) {
        E* op = reinterpret_cast<E*>(A.o) + ((b * s.T + t) * s.Hv + h) * (int64_t)Dv;
        for (int c = tile * 64 * CT + lane; c < (tile + 1) * 64 * CT && c < Dv; c += 64) op[c] = (E)0.f;
    }
    if (A.s_out)
#pragma unroll
        for (int kk = 0; kk < KT; ++kk)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = 32 * kk + 8 * g + 4 * half + e, col = c0 + 16 * ct + r;
                        if (row < Dk && col < Dv) A.s_out[sb + (int64_t)row * Dv + col] = S[kk][half][ct][e];
                    }
}

bool vec_ok(const DeltaShape& s, const DeltaFwdArgs& A) {
    const uintptr_t all = (uintptr_t)A.q | (uintptr_t)A.k | (uintptr_t)A.v | (uintptr_t)A.o;
    return s.Dk % 8 == 0 && s.Dv % 8 == 0 && all % 16 == 0;
}

template <class E, int KT, bool VEC>
hipError_t prepare(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    const int64_t nb = delta_chunks(s);
    hipLaunchKernelGGL((delta_prepare_kernel<E, KT, VEC>), dim3((unsigned)nb), dim3(64), 0, st, s, A, W,
                       (int)((s.T + kChunk - 1) / kChunk));
    return hipGetLastError();
}

template <class E, class KE, int KT, int CT, bool VEC, int MODE>
hipError_t forward_mode(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    auto kernel = delta_forward_kernel<E, KE, KT, CT, VEC, MODE>;
    const int bytes = (int)sizeof(FwdLds<E, KT, CT, VEC>);
    // More dynamic LDS than the default 64 KiB has to be asked for.
    hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    const int ntile = (s.Dv + 64 * CT - 1) / (64 * CT);
    hipLaunchKernelGGL(kernel, dim3((unsigned)(s.B * s.Hv * ntile)), dim3(256), bytes, st, s, A, W,
                       (int)((s.T + kChunk - 1) / kChunk), ntile);
    return hipGetLastError();
}

template <class E, int KT, int CT, bool VEC>
hipError_t forward(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    if (!W.x) return forward_mode<E, E, KT, CT, VEC, kOut>(s, A, W, st);
    if (sizeof(E) == 4 || delta_keeps_f32(s.dtype, A.s_in))
        return A.o ? forward_mode<E, float, KT, CT, VEC, kOut | kKeep>(s, A, W, st)
                   : forward_mode<E, float, KT, CT, VEC, kKeep>(s, A, W, st);
    return A.o ? forward_mode<E, E, KT, CT, VEC, kOut | kKeep>(s, A, W, st)
               : forward_mode<E, E, KT, CT, VEC, kKeep>(s, A, W, st);
}

template <class E, bool VEC>
hipError_t prepare_by(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    if (s.Dk <= 32) return prepare<E, 1, VEC>(s, A, W, st);
    if (s.Dk <= 64) return prepare<E, 2, VEC>(s, A, W, st);
    return prepare<E, 4, VEC>(s, A, W, st);
}

template <class E, bool VEC>
hipError_t forward_by(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    if (s.Dk <= 32) return forward<E, 1, 1, VEC>(s, A, W, st);
    if (s.Dk <= 64) return forward<E, 2, 1, VEC>(s, A, W, st);
    return forward<E, 4, 1, VEC>(s, A, W, st);
}

}  // namespace

hipError_t run_delta_prepare(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    const bool vec = vec_ok(s, A);
    if (s.dtype == kBf16) return vec ? prepare_by<bf16_t, true>(s, A, W, st) : prepare_by<bf16_t, false>(s, A, W, st);
    return vec ? prepare_by<float, true>(s, A, W, st) : prepare_by<float, false>(s, A, W, st);
}

hipError_t run_delta_forward(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    const bool vec = vec_ok(s, A);
    if (s.dtype == kBf16) return vec ? forward_by<bf16_t, true>(s, A, W, st) : forward_by<bf16_t, false>(s, A, W, st);
    return vec ? forward_by<float, true>(s, A, W, st) : forward_by<float, false>(s, A, W, st);
}

}  // namespace linrec
