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

// ---- what depends on a chunk alone -----------------------------------------------------------
// One wave a chunk.  K's fragments serve as both operands of K K^T (the A and B layouts of a
// matrix and its transpose are one).  With A = G diag(beta), the inverse's diagonal 32x32 blocks
// come by substitution, the block below them by two products.  Bound by memory where there are many
// chunks: 10240 of 128 key channels take 140 us for 0.67 GB (4.8 TB/s).  Four waves a chunk, each with
// its own tokens, took 10.1 us instead of 12.4 on one chunk of 12 heads but 204 on the 10240.
template <class E, int KT, bool VEC, int NP>
__global__ __launch_bounds__(64) void delta_prepare_kernel(DeltaShape s, DeltaFwdArgs A, DeltaChunks W, int nc) {
    constexpr int NI = kTerms<E>;
    constexpr int LD = 68;
    __shared__ __align__(16) float a[kChunk * LD];
    __shared__ double gam[kChunk];
    __shared__ float bet[kChunk];
    const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
    const int64_t blk = blockIdx.x;
    const BlockPos at(blockIdx.x, s.Hv, nc);
    const int n = at.rest, h = at.h, hk = uniform(h / (s.Hv / s.Hk));
    const int64_t b = at.b;
    const int len = row_length(s, b), t0 = n * kChunk;
    if (t0 >= len) return;  // nothing of this chunk is used
    const Rows K = rows_of<E>(A.k, s, b, s.Hk, hk, s.Dk, t0, len), Q = rows_of<E>(A.q, s, b, s.Hk, hk, s.Dk, t0, len);
    const bool live = t0 + lane < len;
    float gv = 0.f, bb = 0.f;
    if (live) {
        const int64_t tok = (b * s.T + t0 + lane) * s.Hv + h;
        gv = (float)reinterpret_cast<const E*>(A.g)[tok];
        bb = (float)reinterpret_cast<const E*>(A.beta)[tok];
    }
    // All of K and, at one term a value, of Q is on its way before anything is waited for.
    Frag<NI> kf[4][KT];
    E qx[NI == 1 ? 4 : 1][KT][8];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
            E x[8];
            load8<E, VEC>(K, 16 * t + r, 32 * kk + 8 * g, s.Dk, true, x);
            kf[t][kk] = to_frag<E>(x);
        }
    if constexpr (NI == 1)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) load8<E, VEC>(Q, 16 * t + r, 32 * kk + 8 * g, s.Dk, true, qx[t][kk]);
    {
        const double c = wave_cumsum(decay_of(gv));
        gam[lane] = c;
        bet[lane] = bb;
        W.gam[blk * kChunk + lane] = c;
        float* dec = W.dec + blk * (3 * kChunk) + lane;
        dec[0] = decay_exp(c, 0.0);
        dec[kEw] = decay_exp(__shfl(c, 63), c);
        dec[kBe] = bb;
    }
    __syncthreads();
    // A: tiles of K K^T (rows i, columns j).
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
    // P: tiles of K Q^T (rows j, columns i), stored as P[i][j].
    bf16_t* p = reinterpret_cast<bf16_t*>(W.p) + blk * (NP * kChunk * kChunk);
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        Frag<NI> fq[KT];
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
            if constexpr (NI > 1) load8<E, VEC>(Q, 16 * it + r, 32 * kk + 8 * g, s.Dk, true, qx[0][kk]);
            fq[kk] = to_frag<E>(qx[NI == 1 ? it : 0][kk]);
        }
        const int i = 16 * it + r;
        const double gi = gam[i];
#pragma unroll
        for (int jt = 0; jt <= (it | 1); ++jt) {
            f32x4 c = {0.f, 0.f, 0.f, 0.f};
            if (jt <= it)
#pragma unroll
                for (int kk = 0; kk < KT; ++kk) mma(c, kf[jt][kk], fq[kk]);
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = 16 * jt + 4 * g + e;
                x[e] = j <= i ? s.scale * decay_exp(gi, gam[j]) * c[e] : 0.f;
                x[4 + e] = 0.f;
            }
            const Frag<NP> f = split<NP>(x);
#pragma unroll
            for (int m = 0; m < NP; ++m)
                *reinterpret_cast<bf16x4*>(p + (m * kChunk + i) * kChunk + 16 * jt + 4 * g) =
                    __builtin_shufflevector(f.t[m], f.t[m], 0, 1, 2, 3);
        }
    }
    __syncthreads();
    // The inverses of A's two 32x32 diagonal blocks, over them: lane 32*m + c solves for column c
    // of block m, t_i = [i = c] - sum_{j<i} A_ij t_j, A's rows read from LDS by all its lanes at once.
    {
        float* const blkm = a + (lane >> 5) * (32 * LD + 32);
        const int c = lane & 31;
        float t[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            float x = i == c ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) x = fmaf(-blkm[i * LD + j], t[j], x);
            t[i] = x;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 32; ++i) blkm[i * LD + c] = t[i];
        __syncthreads();
    }
    // The block below them: -N_1 (A_10 N_0), three terms of each factor.
    {
        f32x4 y[2][2];  // A_10 N_0: rows tile_row(m, half), columns 16*ct + r
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = a[(8 * g + i) * LD + 16 * ct + r];
            const Frag<3> f = split<3>(x);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float* p = a + (32 + tile_row(r, half)) * LD + 8 * g;
                load16<float>(p, x);
                load16<float>(p + 4, x + 4);
                y[half][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
                mma(y[half][ct], split<3>(x), f);
            }
        }
        const Frag<3> fy[2] = {split_tiles<3>(y[0][0], y[1][0]), split_tiles<3>(y[0][1], y[1][1])};
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float x[8];
            const float* p = a + (32 + 16 * t + r) * LD + 32 + 8 * g;
            load16<float>(p, x);
            load16<float>(p + 4, x + 4);
            const Frag<3> f = split<3>(x);
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                f32x4 z = {0.f, 0.f, 0.f, 0.f};
                mma(z, f, fy[ct]);
#pragma unroll
                for (int e = 0; e < 4; ++e) a[(32 + 16 * t + 4 * g + e) * LD + 16 * ct + r] = -z[e];
            }
        }
        __syncthreads();
    }
    // Out as three terms, a row's 16-byte pieces by neighbouring lanes.
    bf16_t* out = reinterpret_cast<bf16_t*>(W.inv) + blk * (3 * kChunk * kChunk);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int id = lane + 64 * i, row = id >> 3, c = 8 * (id & 7);
        if (row < 32 && c >= 32) continue;
        float x[8];
        load16<float>(a + row * LD + c, x);
        load16<float>(a + row * LD + c + 4, x + 4);
        const Frag<3> f = split<3>(x);
#pragma unroll
        for (int m = 0; m < 3; ++m) *reinterpret_cast<bf16x8*>(out + m * kChunk * kChunk + 8 * id) = f.t[m];
    }
}

// ---- the chain over a head's chunks -----------------------------------------------------------
// A workgroup of NW waves owns 16*NW value channels of one head, a wave 16 of them, all rows of
// the state (32*KT, zero past Dk).  K, Q, the inverse and P lie in LDS as bfloat16 terms, shared
// by the waves; V comes from memory in the A layout and is turned into the D layout by a product
// with the identity, which is exact.  The next chunk's loads are in flight while one is computed.
//
// A chunk costs a workgroup 4.4 us with one wave a SIMD and 7.3 us with two (128x128, bfloat16), by
// the length of its dependent sequence: 1.3 and 2.5 us of that the matrix units are busy.  Two waves
// a SIMD need every value in 256 registers; a spilled one costs a wait for all loads in flight
// (2950 against 2332 us over a row of 32768 tokens).
//
// Terms: the state and what flows into it (Z, beta X) are taken as three bfloat16 terms, so
// that S keeps float32 precision over any number of chunks; the outputs of bfloat16 calls take
// two terms of S, P and beta X, so that the rounding of the output itself is all there is.
template <class E, int KT>
struct FwdLds {
    static constexpr int NI = kTerms<E>, NO = NI == 1 ? 2 : 3;  // terms of inputs, of the outputs' operands
    Mat<KT> k[NI], q[NI];
    Mat<2> t[3], p[NO];  // the inverse, P
    float dec[3 * kChunk];  // e^gam, e^{gam_63 - gam} (from kEw), beta (from kBe)
};

// What the chain leaves: o, what the backward starts from, or a segment's map:
// tiles of its constant part (the walk from a zero state) and then of its matrix (the walk of
// the identity's columns with no values).
constexpr int kOut = 1, kKeep = 2, kMap = 4;

template <class E, int KT, int NW, bool VEC, int MODE>
__global__ __launch_bounds__(64 * NW, (kWavesPerSimd<E, KT, NW>)) void delta_forward_kernel(DeltaShape s, DeltaFwdArgs A,
                                                                                        DeltaChunks W, int nc,
                                                                                        int ntile, int ntile_v,
                                                                                        int segs, int nblk) {
    typedef FwdLds<E, KT> Lds;
    constexpr int NI = kTerms<E>, NO = Lds::NO, NS = 3;
    constexpr bool OUT = MODE & kOut, KEEP = MODE & kKeep, MAP = MODE & kMap;
    extern __shared__ __align__(16) char lds_raw[];
    Lds& L = *reinterpret_cast<Lds*>(lds_raw);
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const LanePos pos;
    const int r = pos.r, g = pos.g;
    const BlockPos at(blockIdx.x, s.Hv, ntile * segs);
    const int tile = uniform(at.rest % ntile), seg = uniform(at.rest / ntile), h = at.h, hk = uniform(h / (s.Hv / s.Hk));
    const int64_t b = at.b, bh = b * s.Hv + h;
    const int len = row_length(s, b);
    const bool matrix = MAP && tile >= ntile_v;  // a tile of the map's matrix
    const int c0 = ((matrix ? tile - ntile_v : tile) * NW + wave) * 16;  // this wave's first value channel, or column
    const int Dk = s.Dk, Dv = s.Dv;

    // State: D tiles S[2kk + half], rows 32kk + tile_row(m, half), columns c0 + r.
    f32x4 S[2 * KT];
    const int64_t sb = bh * (int64_t)Dk * Dv;
    // (With segments also the first one's: the last may write s_out, which may be s_in.)
    const float* s_in = W.segs == 1 ? A.s_in : W.start + (int64_t)seg * (s.B * s.Hv * (int64_t)Dk * Dv);
#pragma unroll
    for (int d = 0; d < 2 * KT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = 32 * (d >> 1) + 8 * g + 4 * (d & 1) + e, col = c0 + r;
            if constexpr (MAP) S[d][e] = matrix && row == col ? 1.f : 0.f;
            else S[d][e] = (s_in && row < Dk && col < Dv) ? s_in[sb + (int64_t)row * Dv + col] : 0.f;
        }

    const int live = (len + kChunk - 1) / kChunk, first = seg * W.seg_len, past = min(first + W.seg_len, nc);
    const int nlive = min(live, past);  // chunks first..nlive-1 are walked
    RowStage<E, KT, 64 * NW> sk, sq;
    SquareStage<3, 64 * NW> si;
    SquareStage<NO, 64 * NW> sp;
    float sd = 0.f;
    ColumnStage<E> sv;
    const auto fetch = [&](int n) {
        const int t0 = n * kChunk;
        sk.template load<VEC>(rows_of<E>(A.k, s, b, s.Hk, hk, Dk, t0, len), Dk);
        si.load(W.inv, bh * nc + n, 3);
        if (tid < 3 * kChunk) sd = W.dec[(bh * nc + n) * (3 * kChunk) + tid];
        sv.template load<VEC>(rows_of<E>(A.v, s, b, s.Hv, h, Dv, t0, len), c0, matrix ? 0 : Dv);
        if constexpr (OUT) {
            sq.template load<VEC>(rows_of<E>(A.q, s, b, s.Hk, hk, Dk, t0, len), Dk);
            sp.load(W.p, bh * nc + n, W.np);
        }
    };
    if (first < nlive) fetch(first);
    for (int n = first; n < nlive; ++n) {
        const int t0 = n * kChunk;
        const int64_t cb = bh * nc + n;
        __syncthreads();  // the previous chunk's tiles have been read
        sk.store(L.k);
        if constexpr (OUT) sq.store(L.q), sp.store(L.p);
        si.store(L.t);
        if (tid < 3 * kChunk) L.dec[tid] = sd;
        const Frag<NI> fv[2] = {to_frag<E>(sv.x[0]), to_frag<E>(sv.x[1])};
        __syncthreads();
        if (n + 1 < nlive) fetch(n + 1);  // in flight while this chunk is computed
        phase();
        // K S and the state's part of O^T.
        f32x4 Z[4], O[4];  // Z[t]: rows 32*(t/2) + tile_row(m, t%2); O^T[t]: columns 16*t + r
#pragma unroll
        for (int t = 0; t < 4; ++t) Z[t] = O[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
            Frag<NI> fk[4], fq[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                fk[t] = read_tile<NI>(L.k, pos, t >> 1, t & 1, kk);
                if constexpr (OUT) fq[t] = read_rows<NI>(L.q, pos, t, kk);
            }
            const Frag<NS> fs = split_tiles<NS>(S[2 * kk], S[2 * kk + 1]);
            mma_rows<4>(Z, fk, fs);
            if constexpr (OUT) mma_cols<4, NS, NI, NO, NI>(O, fs, fq);
            if constexpr (KEEP)  // S before the chunk, turned so that a lane holds 4 value channels
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    f32x4 x = {0.f, 0.f, 0.f, 0.f};
                    mma(x, fs, identity_frag(which));
                    store4<float>(W.s0 + ((cb * nblk + c0 / 16) * (32 * KT) + 32 * kk + 16 * which + r) * 16 + 4 * g,
                                  x);
                }
        }
        // Z = V - e^gam K S.
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            mma(v, fv[t >> 1], identity_frag(t & 1));
            const f32x4 eg = *reinterpret_cast<const f32x4*>(&L.dec[32 * (t >> 1) + 8 * g + 4 * (t & 1)]);
#pragma unroll
            for (int e = 0; e < 4; ++e) Z[t][e] = fmaf(-eg[e], Z[t][e], v[e]);
            if constexpr (OUT) O[t] *= s.scale * L.dec[16 * t + r];
        }
        phase();
        // X = inverse Z (its upper right block is zero).
        f32x4 U[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) U[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        {
            Frag<3> ft[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) ft[t] = read_tile<3>(L.t, pos, t >> 1, t & 1, 0);
            mma_rows<4>(U, ft, split_tiles<NS>(Z[0], Z[1]));
#pragma unroll
            for (int t = 2; t < 4; ++t) ft[t] = read_tile<3>(L.t, pos, 1, t & 1, 1);
            mma_rows<2>(U + 2, ft + 2, split_tiles<NS>(Z[2], Z[3]));
        }
        phase();
        Frag<NO> fu[2];  // beta X for the outputs
        Frag<NS> fw[2];  // e^{gam_63 - gam} beta X for the state
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
            if constexpr (KEEP) {  // X, likewise
                const Frag<3> fx = split_tiles<3>(U[2 * k2], U[2 * k2 + 1]);
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    f32x4 x = {0.f, 0.f, 0.f, 0.f};
                    mma(x, fx, identity_frag(which));
                    store4<float>(W.x +
                                   ((cb * nblk + c0 / 16) * kChunk + 32 * k2 + 16 * which + r) * 16 + 4 * g,
                               x);
                }
            }
            f32x4 w[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = 32 * k2 + 8 * g + 4 * half;
                U[2 * k2 + half] *= *reinterpret_cast<const f32x4*>(&L.dec[kBe + row]);
                w[half] = U[2 * k2 + half] * *reinterpret_cast<const f32x4*>(&L.dec[kEw + row]);
            }
            if constexpr (OUT) fu[k2] = split_tiles<NO>(U[2 * k2], U[2 * k2 + 1]);
            fw[k2] = split_tiles<NS>(w[0], w[1]);
        }
        phase();
        // S' = e^{gam_63} S + K^T w, four tiles at a time.
        const float end = L.dec[kChunk - 1];
        constexpr int T = KT == 1 ? 2 : 4;
#pragma unroll
        for (int d = 0; d < 2 * KT; d += T) {
#pragma unroll
            for (int t = 0; t < T; ++t) S[d + t] *= end;
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
                Frag<NI> ft[T];
#pragma unroll
                for (int t = 0; t < T; ++t) ft[t] = read_col<NI, true>(L.k, pos, k2, 32 * ((d + t) >> 1), t & 1);
                mma_rows<T>(S + d, ft, fw[k2]);
            }
        }
        if constexpr (OUT) {
            phase();
            const Rows out = rows_of<E>(A.o, s, b, s.Hv, h, Dv, t0, (int)s.T);
            // O^T += U^T P^T (P's upper right block is zero).
            Frag<NO> fp[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) fp[t] = read_rows<NO>(L.p, pos, t, 0);
            mma_cols<4>(O, fu[0], fp);
#pragma unroll
            for (int t = 2; t < 4; ++t) fp[t] = read_rows<NO>(L.p, pos, t, 1);
            mma_cols<2>(O + 2, fu[1], fp + 2);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                store_rows<E, VEC>(out, 16 * t + r, c0 + 4 * g, Dv,
                                   t0 + 16 * t + r < len ? O[t] : f32x4{0.f, 0.f, 0.f, 0.f});
        }
    }
    // Chunks past the row's length: zero outputs.
    if constexpr (OUT)
        for (int64_t t = (int64_t)max(live, first) * kChunk + wave; t < s.T && t < (int64_t)past * kChunk; t += NW) {
            E* op = reinterpret_cast<E*>(A.o) + ((b * s.T + t) * s.Hv + h) * (int64_t)Dv;
            for (int c = tile * NW * 16 + lane; c < (tile + 1) * NW * 16 && c < Dv; c += 64) op[c] = (E)0.f;
        }
    if constexpr (MAP) {
        float* m = W.map + ((bh * (W.segs - 1) + seg) * (32 * KT)) * (int64_t)(16 * nblk + 32 * KT);
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 32 * (d >> 1) + 8 * g + 4 * (d & 1) + e;
                if (!matrix || c0 < 32 * KT)
                    m[row * (16 * nblk + 32 * KT) + (matrix ? 16 * nblk : 0) + c0 + r] = S[d][e];
            }
    }
    if (!MAP && A.s_out && seg == segs - 1)
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 32 * (d >> 1) + 8 * g + 4 * (d & 1) + e, col = c0 + r;
                if (row < Dk && col < Dv) A.s_out[sb + (int64_t)row * Dv + col] = S[d][e];
            }
}

// ---- the states before the segments ---------------------------------------------------------------
// start_{g+1} = matrix_g start_g + constant_g, in order.  A workgroup takes 16 value channels of a
// head, a wave 16 rows of the state: the matrix's rows do not depend on the state, so the next
// segment's are on their way while one is multiplied, and a segment costs little more than the
// two barriers around the exchange of the state through LDS.  Three terms of both.
template <int KT>
__global__ __launch_bounds__(128 * KT) void delta_join_kernel(DeltaShape s, DeltaFwdArgs A, DeltaChunks W, int ntile,
                                                              int nblk) {
    __shared__ float st[32 * KT][17];
    const int d = threadIdx.x >> 6;
    const LanePos pos;
    const int r = pos.r, g = pos.g;
    const BlockPos at(blockIdx.x, s.Hv, ntile);
    const int64_t bh = at.b * s.Hv + at.h;
    const int c0 = at.rest * 16, Dk = s.Dk, Dv = s.Dv, ld = 16 * nblk + 32 * KT;
    const int cell = threadIdx.x & 15;  // this thread's column of the rows threadIdx.x / 16 + 8*KT*i
    for (int row = threadIdx.x >> 4; row < 32 * KT; row += 8 * KT)
        st[row][cell] = (A.s_in && row < Dk && c0 + cell < Dv) ? A.s_in[(bh * Dk + row) * Dv + c0 + cell] : 0.f;
    float x[KT][8], c[4];
    const auto fetch = [&](int seg) {
        const float* m = W.map + ((bh * (W.segs - 1) + seg) * (32 * KT)) * (int64_t)ld;
        const float* p = m + (32 * (d >> 1) + tile_row(r, d & 1)) * ld + 16 * nblk + 8 * g;
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
            load16<float>(p + 32 * kk, x[kk]);
            load16<float>(p + 32 * kk + 4, x[kk] + 4);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = m[(32 * (d >> 1) + 8 * g + 4 * (d & 1) + e) * ld + c0 + r];
    };
    fetch(0);
    for (int seg = 0;; ++seg) {
        __syncthreads();  // the state before this segment is there
        float* out = W.start + ((int64_t)seg * s.B * s.Hv + bh) * Dk * Dv;
        for (int row = threadIdx.x >> 4; row < Dk; row += 8 * KT)
            if (c0 + cell < Dv) out[(int64_t)row * Dv + c0 + cell] = st[row][cell];
        if (seg + 1 == W.segs) return;
        f32x4 S = {c[0], c[1], c[2], c[3]};
        Frag<3> fm[KT];
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) fm[kk] = split<3>(x[kk]);
        if (seg + 2 < W.segs) fetch(seg + 1);
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = st[32 * kk + 8 * g + i][r];
            mma(S, fm[kk], split<3>(y));
        }
        __syncthreads();  // all have read it
#pragma unroll
        for (int e = 0; e < 4; ++e) st[32 * (d >> 1) + 8 * g + 4 * (d & 1) + e][r] = S[e];
    }
}

bool vec_ok(const DeltaShape& s, const DeltaFwdArgs& A) {
    const uintptr_t all = (uintptr_t)A.q | (uintptr_t)A.k | (uintptr_t)A.v | (uintptr_t)A.o;
    return s.Dk % 8 == 0 && s.Dv % 8 == 0 && all % 16 == 0;
}

template <class E, int KT, bool VEC>
hipError_t prepare(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    const dim3 grid((unsigned)delta_chunks(s));
    const int nc = (int)((s.T + kChunk - 1) / kChunk);
    if constexpr (sizeof(E) == 2) {
        if (W.np == 2)
            hipLaunchKernelGGL((delta_prepare_kernel<E, KT, VEC, 2>), grid, dim3(64), 0, st, s, A, W, nc);
        else
            hipLaunchKernelGGL((delta_prepare_kernel<E, KT, VEC, 3>), grid, dim3(64), 0, st, s, A, W, nc);
    } else {
        hipLaunchKernelGGL((delta_prepare_kernel<E, KT, VEC, 3>), grid, dim3(64), 0, st, s, A, W, nc);
    }
    return hipGetLastError();
}

template <class E, int KT, int NW, bool VEC, int MODE>
hipError_t forward_nw(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    auto kernel = delta_forward_kernel<E, KT, NW, VEC, MODE>;
    const int bytes = (int)sizeof(FwdLds<E, KT>);
    // More dynamic LDS than the default 64 KiB has to be asked for.
    hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    const int ntile_v = (s.Dv + 16 * NW - 1) / (16 * NW);
    const int ntile = ntile_v + (MODE & kMap ? (32 * KT + 16 * NW - 1) / (16 * NW) : 0);
    const int segs = MODE & kMap ? W.segs - 1 : W.segs;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(s.B * s.Hv * ntile * segs)), dim3(64 * NW), bytes, st, s, A, W,
                       (int)((s.T + kChunk - 1) / kChunk), ntile, ntile_v, segs, delta_blocks(s));
    return hipGetLastError();
}

template <class E, int KT, bool VEC, int MODE>
hipError_t forward_mode(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    if constexpr (sizeof(E) == 2)
        if (delta_wide(s, W.segs)) return forward_nw<E, KT, 8, VEC, MODE>(s, A, W, st);
    return forward_nw<E, KT, 4, VEC, MODE>(s, A, W, st);
}

template <class E, int KT, bool VEC>
hipError_t forward(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    if (W.segs > 1) {
        hipError_t e = forward_mode<E, KT, VEC, kMap>(s, A, W, st);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((delta_join_kernel<KT>), dim3((unsigned)(s.B * s.Hv * ((s.Dv + 15) / 16))), dim3(128 * KT), 0,
                           st, s, A, W, (s.Dv + 15) / 16, delta_blocks(s));
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!W.x) return forward_mode<E, KT, VEC, kOut>(s, A, W, st);
    return A.o ? forward_mode<E, KT, VEC, kOut | kKeep>(s, A, W, st) : forward_mode<E, KT, VEC, kKeep>(s, A, W, st);
}

template <class E, bool VEC>
hipError_t prepare_by(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    if (s.Dk <= 32) return prepare<E, 1, VEC>(s, A, W, st);
    if (s.Dk <= 64) return prepare<E, 2, VEC>(s, A, W, st);
    return prepare<E, 4, VEC>(s, A, W, st);
}

template <class E, bool VEC>
hipError_t forward_by(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    if (s.Dk <= 32) return forward<E, 1, VEC>(s, A, W, st);
    if (s.Dk <= 64) return forward<E, 2, VEC>(s, A, W, st);
    return forward<E, 4, VEC>(s, A, W, st);
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
