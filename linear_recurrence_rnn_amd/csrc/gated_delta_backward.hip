// gated_delta_backward.hip -- gradients of the gated delta rule, in the forward's chunks.
//
// With dO and dS' (the gradient of the state after the chunk), and the forward's G, P, inverse
// N = (I + G diag(beta))^{-1}, X, and state S before the chunk:
//   dU = P^T dO + diag(e^{gam_63 - gam}) K dS'
//   dZ = N^T (beta dU) = dV
//   dS = e^{gam_63} dS' + scale Q^T diag(e^gam) dO - K^T diag(e^gam) dZ
// is a chain over the chunks in reverse (first kernel; it writes dV, in bfloat16 calls also what its
// rounding left of dZ, and every dS').  The rest is local to a chunk (second kernel), with
// H = dO X^T, E = dZ X^T, L_ij = e^{gam_i - gam_j}, q' = scale q, W = e^{gam_63 - gam_j} dS' x_j,
// M_ij = L_ij (q'_i.k_j H_ij - [i > j] k_i.k_j E_ij):
//   dq_i    = scale (e^{gam_i} S dO_i + sum_{j<=i} L_ij beta_j H_ij k_j)
//   dk_j    = beta_j (W_j + sum_{i>=j} L_ij H_ij q'_i - sum_{i>j} L_ij E_ij k_i)
//             - e^{gam_j} S dZ_j - sum_{i<j} L_ji beta_i E_ji k_i
//   dbeta_j = sum_i M_ij + k_j.W_j
//   dg_t    = sum_{i>=t} (q'_i.e^{gam_i} S dO_i - k_i.e^{gam_i} S dZ_i) + sum_{j<t} beta_j k_j.W_j
//             + e^{gam_63} <S, dS'> + sum_{i>=t>j} beta_j M_ij
// (every pair of a write before t and a read at or after t carries e^{g_t}).
#include "gated_delta.hpp"
#include "delta_tile.hpp"

namespace linrec {

namespace {

// ---- the chain of the state's gradient ----------------------------------------------------------
// The forward chain's layout: 16 value channels a wave, dS in registers.  NS terms for the gradient
// of the state and what flows into it: three where it leaves the call in float32, as the gradient
// of a carried state; two (2^-16) where all results are bfloat16.
template <class E, int KT, int NS>
struct ChainLds {
    static constexpr int NI = kTerms<E>;
    Mat<KT> k[NI], q[NI];
    Mat<2> t[NS], p[NS];  // the inverse, P
    float dec[3 * kChunk];  // e^gam, e^{gam_63 - gam} (from kEw), beta (from kBe)
};

template <class E, int KT, int NW, bool VEC, int NS>
__global__ __launch_bounds__(64 * NW, (kWavesPerSimd<E, KT, NW>)) void delta_chain_kernel(DeltaShape s, DeltaBwdArgs A,
                                                                                      DeltaChunks W, int nc, int ntile,
                                                                                      int nblk) {
    typedef ChainLds<E, KT, NS> Lds;
    constexpr int NI = kTerms<E>, NZ = kKeptTerms<E>;
    extern __shared__ __align__(16) char lds_raw[];
    Lds& L = *reinterpret_cast<Lds*>(lds_raw);
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const LanePos pos;
    const int r = pos.r, g = pos.g;
    const BlockPos at(blockIdx.x, s.Hv, ntile);
    const int tile = at.rest, h = at.h, hk = uniform(h / (s.Hv / s.Hk));
    const int64_t b = at.b, bh = b * s.Hv + h;
    const int len = row_length(s, b);
    const int c0 = (tile * NW + wave) * 16;
    const int Dk = s.Dk, Dv = s.Dv;

    f32x4 S[2 * KT];  // dS, in the forward's layout of S
    const int64_t sb = bh * (int64_t)Dk * Dv;
#pragma unroll
    for (int d = 0; d < 2 * KT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = 32 * (d >> 1) + 8 * g + 4 * (d & 1) + e, col = c0 + r;
            S[d][e] = (A.gs_out && row < Dk && col < Dv) ? A.gs_out[sb + (int64_t)row * Dv + col] : 0.f;
        }

    const int nlive = (len + kChunk - 1) / kChunk;
    RowStage<E, KT, 64 * NW> sk, sq;
    SquareStage<NS, 64 * NW> si, sp;
    float sd = 0.f;
    ColumnStage<E> so;
    const auto fetch = [&](int n) {
        const int t0 = n * kChunk;
        sk.template load<VEC>(rows_of<E>(A.k, s, b, s.Hk, hk, Dk, t0, len), Dk);
        si.load(W.inv, bh * nc + n, 3);
        sp.load(W.p, bh * nc + n, W.np);
        if (tid < 3 * kChunk) sd = W.dec[(bh * nc + n) * (3 * kChunk) + tid];
        so.template load<VEC>(rows_of<E>(A.go, s, b, s.Hv, h, Dv, t0, len), c0, Dv);
        sq.template load<VEC>(rows_of<E>(A.q, s, b, s.Hk, hk, Dk, t0, len), Dk);
    };
    if (nlive > 0) fetch(nlive - 1);
    for (int n = nlive - 1; n >= 0; --n) {
        const int t0 = n * kChunk;
        const int64_t cb = bh * nc + n;
        __syncthreads();  // the previous chunk's tiles have been read
        sk.store(L.k);
        sq.store(L.q);
        si.store(L.t);
        sp.store(L.p);
        if (tid < 3 * kChunk) L.dec[tid] = sd;
        const Frag<NI> fv[2] = {to_frag<E>(so.x[0]), to_frag<E>(so.x[1])};
        __syncthreads();
        if (n > 0) fetch(n - 1);  // in flight while this chunk is computed
        phase();
        // K dS' (dS' is also stored, turned so that a lane holds 4 value channels).
        f32x4 U[4];  // rows 32*(t/2) + tile_row(m, t%2)
#pragma unroll
        for (int t = 0; t < 4; ++t) U[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
            Frag<NI> fk[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) fk[t] = read_tile<NI>(L.k, pos, t >> 1, t & 1, kk);
            const Frag<NS> fs = split_tiles<NS>(S[2 * kk], S[2 * kk + 1]);
            mma_rows<4>(U, fk, fs);
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                f32x4 x = {0.f, 0.f, 0.f, 0.f};
                mma(x, fs, identity_frag(which));
                store4<float>(W.ds + ((cb * nblk + c0 / 16) * (32 * KT) + 32 * kk + 16 * which + r) * 16 + 4 * g, x);
            }
        }
        phase();
        // dO in the D layout: as B operand, and scaled for the state's gradient.
        Frag<NI> fo[2];
        Frag<NS> fd[2];
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
            f32x4 d[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                d[half] = f32x4{0.f, 0.f, 0.f, 0.f};
                mma(d[half], fv[k2], identity_frag(half));
                U[2 * k2 + half] *= *reinterpret_cast<const f32x4*>(&L.dec[kEw + 32 * k2 + 8 * g + 4 * half]);
            }
            fo[k2] = split_tiles<NI>(d[0], d[1]);
#pragma unroll
            for (int half = 0; half < 2; ++half)
                d[half] *= s.scale * *reinterpret_cast<const f32x4*>(&L.dec[32 * k2 + 8 * g + 4 * half]);
            fd[k2] = split_tiles<NS>(d[0], d[1]);
        }
        phase();
        // dU += P^T dO (the lower left block is zero), then beta dU.
        {
            Frag<NS> fp[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) fp[t] = read_col<NS, true>(L.p, pos, 1, 32 * (t >> 1), t & 1);
            mma_rows<4>(U, fp, fo[1]);
#pragma unroll
            for (int t = 0; t < 2; ++t) fp[t] = read_col<NS, true>(L.p, pos, 0, 0, t);
            mma_rows<2>(U, fp, fo[0]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) U[t] *= *reinterpret_cast<const f32x4*>(&L.dec[kBe + 32 * (t >> 1) + 8 * g + 4 * (t & 1)]);
        phase();
        // dZ = N^T (beta dU).
        f32x4 Z[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) Z[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        {
            Frag<NS> ft[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) ft[t] = read_col<NS, true>(L.t, pos, 1, 32 * (t >> 1), t & 1);
            mma_rows<4>(Z, ft, split_tiles<NS>(U[2], U[3]));
#pragma unroll
            for (int t = 0; t < 2; ++t) ft[t] = read_col<NS, true>(L.t, pos, 0, 0, t);
            mma_rows<2>(Z, ft, split_tiles<NS>(U[0], U[1]));
        }
        phase();
        const Rows out = rows_of<E>(A.gv, s, b, s.Hv, h, Dv, t0, (int)s.T);
        // dV, turned; and -e^gam dZ for the state's gradient.
        Frag<NS> fz[2];
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
            const Frag<NZ> fx = split_tiles<NZ>(Z[2 * k2], Z[2 * k2 + 1]);
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                f32x4 x = {0.f, 0.f, 0.f, 0.f};
                mma<NZ, 1, NI, 1>(x, fx, identity_frag(which));
                if (t0 + kChunk > len)  // absent tokens: zero, whatever their chunk holds
                    if (t0 + 32 * k2 + 16 * which + r >= len) x = f32x4{0.f, 0.f, 0.f, 0.f};
                store_rows<E, VEC>(out, 32 * k2 + 16 * which + r, c0 + 4 * g, Dv, x);
                if constexpr (NI < NZ) {  // what the rounding left
                    f32x4 y = {0.f, 0.f, 0.f, 0.f};
                    mma(y, Frag<1>{{fx.t[1]}}, identity_frag(which));
                    store_rows<E, VEC>(rows_of<E>(W.dz, s, b, s.Hv, h, Dv, t0, (int)s.T), 32 * k2 + 16 * which + r,
                                       c0 + 4 * g, Dv, y);
                }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half)
                Z[2 * k2 + half] *= -*reinterpret_cast<const f32x4*>(&L.dec[32 * k2 + 8 * g + 4 * half]);
            fz[k2] = split_tiles<NS>(Z[2 * k2], Z[2 * k2 + 1]);
        }
        phase();
        // dS = e^{gam_63} dS' + scale Q^T e^gam dO - K^T e^gam dZ, four tiles at a time.
        const float end = L.dec[kChunk - 1];
        constexpr int T = KT == 1 ? 2 : 4;
#pragma unroll
        for (int d = 0; d < 2 * KT; d += T) {
#pragma unroll
            for (int t = 0; t < T; ++t) S[d + t] *= end;
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
                Frag<NI> fq[T], fk[T];
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    fq[t] = read_col<NI, true>(L.q, pos, k2, 32 * ((d + t) >> 1), t & 1);
                    fk[t] = read_col<NI, true>(L.k, pos, k2, 32 * ((d + t) >> 1), t & 1);
                }
                mma_rows<T>(S + d, fq, fd[k2]);
                mma_rows<T>(S + d, fk, fz[k2]);
            }
        }
    }
    for (int64_t t = (int64_t)nlive * kChunk + wave; t < s.T; t += NW) {
        E* op = reinterpret_cast<E*>(A.gv) + ((b * s.T + t) * s.Hv + h) * (int64_t)Dv;
        for (int c = tile * NW * 16 + lane; c < (tile + 1) * NW * 16 && c < Dv; c += 64) op[c] = (E)0.f;
    }
    if (A.gs_in)
#pragma unroll
        for (int d = 0; d < 2 * KT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 32 * (d >> 1) + 8 * g + 4 * (d & 1) + e, col = c0 + r;
                if (row < Dk && col < Dv) A.gs_in[sb + (int64_t)row * Dv + col] = S[d][e];
            }
}

// ---- the gradients of a chunk ---------------------------------------------------------------------
// A workgroup of eight waves takes one chunk of one key head and goes through the value heads
// that read it, so dq and dk are summed over them in head order, in registers.  A wave owns 16
// key channels (all 64 tokens at 128 key channels, 32 or 16 of them at fewer): dq^T, dk^T and the
// products with S and dS' have its key channels as rows, so every byte of S and dS' is loaded
// once, straight into operands.  dO, dZ and X, which all waves need, go through LDS, 32*SK value
// channels at a time.  The tiles of H^T and E^T (rows j <= its columns i) are dealt to the waves.
//
// Operands are the tensors' own type (one bfloat16 term, or three); what is kept (x, S, dS'), dZ and
// the weights L beta H and L beta E are two terms in bfloat16 calls.  At 128x128 a bfloat16 chunk reads
// 240 KB (half of it S and dS') and writes 33 KB a head: 794 us for 10240 (2.9 GB by the counters, 3.6
// TB/s), bound by one workgroup's loads, products and five barriers following each other (its LDS
// is over half of a CU's; half of its waves' time is waiting).
template <class E, int KT>
struct GradLds {
    static constexpr int NI = kTerms<E>, NX = kKeptTerms<E>, NH = NX;
    static constexpr int SK = NI == 1 ? 4 : 1;
    static constexpr bool ONE = NI == 3;  // no room for both weights: one after the other
    Mat<KT> k[NI], q[NI];
    union {
        struct {
            Mat<SK> go[NI], gz[NX], x[NX];
        };
        struct {
            Mat<2> h[NH], e[ONE ? 1 : NH];  // scale L beta H, L beta E: rows i, columns j
        };
    };
    double gam[kChunk];
    float be[kChunk];
    float col[4][kChunk];  // sums over each tile's i > j of M_ij; M_jj on its own, so that sums that
                           // ought to cancel in dg hold nothing that does not belong there
    float row[2][kChunk], diag[kChunk];
    float a[2 * KT][kChunk], wr[2 * KT][kChunk];
    float dot[8];
};

// x in LDS as terms from its blocks of 16 value channels, 32*SK channels from block b0 on.
template <int N, int SK>
struct BlockStage {
    static constexpr int P = kChunk * 4 * SK, I = (P + 511) / 512;
    float x[I][8];
    __device__ __forceinline__ void load(const float* m, int b0) {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int id = (int)threadIdx.x + 512 * i;
            if (P % 512 != 0 && id >= P) break;
            const float* p = m + ((int64_t)b0 * kChunk * 16 + 8 * id);
            load16<float>(p, x[i]);
            load16<float>(p + 4, x[i] + 4);
        }
    }
    __device__ __forceinline__ void store(Mat<SK>* dst) const {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int id = (int)threadIdx.x + 512 * i, row = (id >> 1) & 63, c = 16 * (id >> 7) + 8 * (id & 1);
            if (P % 512 != 0 && id >= P) break;
            const Frag<N> f = split<N>(x[i]);
#pragma unroll
            for (int m = 0; m < N; ++m) *dst[m].row8(row, c) = f.t[m];
        }
    }
};

// 8 value channels from 32*kv + 8g of row `row` of a matrix kept in blocks of 16 channels.  Through
// a buffer resource: what depends on the lane is one register for all of them.
__device__ __forceinline__ void load_block(const rsrc_t& m, int rows, int row, int kv, int g, float* x) {
    const unsigned lane = 64u * ((g >> 1) * rows + row) + 32u * (g & 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x4 t = __builtin_bit_cast(
            f32x4, __builtin_amdgcn_raw_buffer_load_b128(m, lane + 16u * i, uniform(128 * kv * rows), 0));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * i + e] = t[e];
    }
}

template <int N>
__device__ __forceinline__ Frag<N> negative(Frag<N> f) {
#pragma unroll
    for (int n = 0; n < N; ++n)
        f.t[n] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, f.t[n]) ^ 0x80008000u);
    return f;
}

template <class E, int KT, bool VEC>
__global__ __launch_bounds__(512, 2) void delta_grad_kernel(DeltaShape s, DeltaBwdArgs A, DeltaChunks W, int nc, int,
                                                            int nblk) {
    typedef GradLds<E, KT> Lds;
    constexpr int NI = Lds::NI, NX = Lds::NX, NH = Lds::NH, SK = Lds::SK;
    constexpr int DT = 2 * KT, TW = DT / 2;  // tiles of key channels; token tiles of a wave
    extern __shared__ __align__(16) char lds_raw[];
    Lds& L = *reinterpret_cast<Lds*>(lds_raw);
    const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63;
    LanePos pos;
    const int d0 = wave % DT, tk0 = (wave / DT) * TW;  // this wave's key channel tile, first token tile
    const int it = wave & 3, j0 = wave >> 2;           // its tiles of H^T: columns it, rows j0, j0 + 2
    const BlockPos at(blockIdx.x, s.Hk, nc);
    const int n = at.rest, hk = at.h, rep = s.Hv / s.Hk;
    const int64_t b = at.b;
    const int len = row_length(s, b), t0 = n * kChunk;
    const int Dk = s.Dk, Dv = s.Dv;
    if (t0 >= len) {  // absent tokens: zero gradients
        for (int i = wave; i < kChunk && t0 + i < s.T; i += 8) {
            const int64_t at = ((b * s.T + t0 + i) * s.Hk + hk) * (int64_t)Dk;
            for (int c = lane; c < Dk; c += 64) {
                reinterpret_cast<E*>(A.gq)[at + c] = (E)0.f;
                reinterpret_cast<E*>(A.gk)[at + c] = (E)0.f;
            }
            for (int c = lane; c < rep; c += 64) {
                const int64_t p = (b * s.T + t0 + i) * s.Hv + hk * rep + c;
                reinterpret_cast<E*>(A.gg)[p] = (E)0.f;
                reinterpret_cast<E*>(A.gbeta)[p] = (E)0.f;
            }
        }
        return;
    }
    RowStage<E, KT, 512> sk, sq;
    sk.template load<VEC>(rows_of<E>(A.k, s, b, s.Hk, hk, Dk, t0, len), Dk);
    sq.template load<VEC>(rows_of<E>(A.q, s, b, s.Hk, hk, Dk, t0, len), Dk);

    f32x4 dq[TW], dk[TW];  // rows 16*d0 + 4g.., columns 16*(tk0 + t) + r
#pragma unroll
    for (int t = 0; t < TW; ++t) dq[t] = dk[t] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int hr = 0; hr < rep; ++hr) {
        const int h = hk * rep + hr;
        pos.renew();
        const int r = pos.r, g = pos.g;
        const int64_t cb = (b * s.Hv + h) * nc + n;
        const float* X = W.x + cb * nblk * (kChunk * 16);
        const int kept = nblk * (32 * KT * 16);  // of a chunk
        const rsrc_t S0 = make_rsrc(W.s0 + cb * kept, 4 * kept), DS = make_rsrc(W.ds + cb * kept, 4 * kept);
        const Rows go = rows_of<E>(A.go, s, b, s.Hv, h, Dv, t0, len), gz = rows_of<E>(A.gv, s, b, s.Hv, h, Dv, t0, len);
        const Rows gl = rows_of<E>(W.dz, s, b, s.Hv, h, Dv, t0, len);  // dZ is gz + gl in bfloat16 calls
        f32x4 H[2], Z[2], rq[TW], rk[TW], wk[TW];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) H[i] = Z[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < TW; ++t) rq[t] = rk[t] = wk[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int kv0 = 0; 32 * kv0 < Dv; kv0 += SK) {
            RowStage<E, SK, 512> so, sz, sl;
            BlockStage<NX, SK> sx;
            so.template load<VEC>(go, Dv, 32 * kv0);
            sz.template load<VEC>(gz, Dv, 32 * kv0);
            if constexpr (NI < NX) sl.template load<VEC>(gl, Dv, 32 * kv0);
            sx.load(X, 2 * kv0);
            // S and dS', two slabs of 32 value channels ahead: the first on its way with what goes through
            // LDS, the second in the registers that that leaves, the others as those before are used
            // (more at once were spilled, which waits for every load in flight).
            float xs[SK][8], xd[SK][8];
            const auto states = [&](int from, int to) {
#pragma unroll
                for (int kv = from; kv < to; ++kv) {
                    load_block(S0, 32 * KT, 16 * d0 + r, kv0 + kv, g, xs[kv]);
                    load_block(DS, 32 * KT, 16 * d0 + r, kv0 + kv, g, xd[kv]);
                }
            };
            states(0, 1);
            __syncthreads();  // what lay here has been read
            if (hr == 0 && kv0 == 0) sk.store(L.k), sq.store(L.q);
            if (kv0 == 0 && tid < kChunk) {
                L.gam[tid] = W.gam[cb * kChunk + tid];
                L.be[tid] = t0 + tid < len
                                ? (float)reinterpret_cast<const E*>(A.beta)[(b * s.T + t0 + tid) * s.Hv + h]
                                : 0.f;
            }
            so.store(L.go);
            sz.store(L.gz);
            if constexpr (NI < NX) sl.store(L.gz + 1);
            sx.store(L.x);
            states(1, SK < 2 ? SK : 2);
            __syncthreads();
            pos.renew();
#pragma unroll
            for (int kv = 0; kv < SK; ++kv) {
                if (32 * (kv0 + kv) >= Dv) break;  // blocks past Dv may not have been written
                phase();
                // H^T, E^T: rows j, columns i.
                const Frag<NI> fo = read_rows<NI>(L.go, pos, it, kv);
                const Frag<NX> fz = read_rows<NX>(L.gz, pos, it, kv);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (j0 + 2 * i <= it) {
                        const Frag<NX> f = read_rows<NX>(L.x, pos, j0 + 2 * i, kv);
                        mma(H[i], f, fo);
                        mma(Z[i], f, fz);
                    }
                // S dO, S dZ, dS' x: rows key channels, columns tokens.
                Frag<NI> to[TW];
                Frag<NX> tz[TW], tx[TW];
#pragma unroll
                for (int t = 0; t < TW; ++t) {
                    to[t] = read_rows<NI>(L.go, pos, tk0 + t, kv);
                    tz[t] = read_rows<NX>(L.gz, pos, tk0 + t, kv);
                    tx[t] = read_rows<NX>(L.x, pos, tk0 + t, kv);
                }
                const Frag<NX> fs = split<NX>(xs[kv]), fd = split<NX>(xd[kv]);
                mma_cols<TW>(rq, fs, to);
                mma_cols<TW>(rk, fs, tz);
                mma_cols<TW>(wk, fd, tx);
                if (tk0 == 0)  // <S, dS'>, each byte of them once
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot = fmaf(xs[kv][i], xd[kv][i], dot);
                if (kv + 2 < SK) states(kv + 2, kv + 3);
            }
        }
        phase();
        __syncthreads();  // the slab has been read: the weights lie over it
        pos.renew();
        const double gend = L.gam[kChunk - 1];
        // M, its sums, and the weights scale L beta H and L beta E.
        bf16x4 we[2][NH];
        {
            const int mine = 16 * it + r;
            const double gi = L.gam[mine];
            float rowsum = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int jt = j0 + 2 * i;
                if (jt > (it | 1)) {
                    if (lane < 16) L.col[it][16 * jt + lane] = 0.f;
                    continue;
                }
                f32x4 qk = {0.f, 0.f, 0.f, 0.f}, kk = {0.f, 0.f, 0.f, 0.f};
                if (jt <= it)
#pragma unroll
                    for (int c = 0; c < KT; ++c) {
                        const Frag<NI> fk = read_rows<NI>(L.k, pos, jt, c);
                        mma(qk, fk, read_rows<NI>(L.q, pos, it, c));
                        mma(kk, fk, read_rows<NI>(L.k, pos, it, c));
                    }
                float hw[8], ez[8];
                f32x4 m4;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 16 * jt + 4 * g + e;
                    const float l = j <= mine ? decay_exp(gi, L.gam[j]) : 0.f, ls = j < mine ? l : 0.f;
                    const float bj = L.be[j];
                    const float hh = s.scale * l * H[i][e], zz = ls * Z[i][e];
                    m4[e] = qk[e] * hh - kk[e] * zz;
                    if (j == mine) {
                        L.diag[mine] = m4[e];
                        m4[e] = 0.f;
                    }
                    rowsum = fmaf(bj, m4[e], rowsum);
                    hw[e] = bj * hh;
                    ez[e] = bj * zz;
                    hw[4 + e] = ez[4 + e] = 0.f;
                }
                const Frag<NH> fh = split<NH>(hw), fe = split<NH>(ez);
#pragma unroll
                for (int m = 0; m < NH; ++m) {
                    *quad(&L.h[m], pos, it, jt) = __builtin_shufflevector(fh.t[m], fh.t[m], 0, 1, 2, 3);
                    we[i][m] = __builtin_shufflevector(fe.t[m], fe.t[m], 0, 1, 2, 3);
                    if constexpr (!Lds::ONE) *quad(&L.e[m], pos, it, jt) = we[i][m];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) m4[e] += __shfl_xor(m4[e], o);
                    if (r == 0) L.col[it][16 * jt + 4 * g + e] = m4[e];
                }
            }
            rowsum += __shfl_xor(rowsum, 16);
            rowsum += __shfl_xor(rowsum, 32);
            if (g == 0) L.row[j0][mine] = rowsum;
        }
        // Sums with q and k over the key channels, and the parts of dq, dk from S and dS'.
#pragma unroll
        for (int t = 0; t < TW; ++t) {
            phase();
            const int tt = tk0 + t, tok = 16 * tt + r;
            const double gi = L.gam[tok];
            const float eg = decay_exp(gi, 0.0), ew = decay_exp(gend, gi), be = L.be[tok];
            f32x4 q4 = {0.f, 0.f, 0.f, 0.f}, k4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = NI - 1; m >= 0; --m) {
                const bf16x4 a = *quad(&L.q[m], pos, tt, d0), c = *quad(&L.k[m], pos, tt, d0);
#pragma unroll
                for (int e = 0; e < 4; ++e) q4[e] += (float)a[e], k4[e] += (float)c[e];
            }
            rq[t] *= s.scale * eg;
            rk[t] *= eg;
            wk[t] *= ew;
            float asum = 0.f, wsum = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                asum = fmaf(q4[e], rq[t][e], asum);
                asum = fmaf(-k4[e], rk[t][e], asum);
                wsum = fmaf(k4[e], wk[t][e], wsum);
            }
            asum += __shfl_xor(asum, 16);
            asum += __shfl_xor(asum, 32);
            wsum += __shfl_xor(wsum, 16);
            wsum += __shfl_xor(wsum, 32);
            if (g == 0) L.a[d0][tok] = asum, L.wr[d0][tok] = wsum;
            dq[t] += rq[t];
            dk[t] += be * wk[t] - rk[t];
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o);
        if (lane == 0) L.dot[wave] = dot;
        __syncthreads();  // the weights and the sums are there
        // dq += L beta H k;  dk += (L beta H)^T q' - (L beta E)^T k - (L beta E) k.
        const auto with_h = [&](int k2, const Frag<NI>& fk) {
            const Frag<NI> fq = read_col<NI, false>(L.q, pos, k2, 16 * d0, 0);
#pragma unroll
            for (int t = 0; t < TW; ++t) {  // rows 32*k2.. reach down, or up, to this tile's tokens
                phase();
                const int tt = tk0 + t;
                if (2 * k2 <= tt) mma(dq[t], fk, read_rows<NH>(L.h, pos, tt, k2));
                if (2 * k2 + 1 >= tt) mma(dk[t], fq, read_col<NH, false>(L.h, pos, k2, 16 * tt, 0));
            }
        };
        const auto with_e = [&](int k2, const Frag<NI>& fk, const Mat<2>* e) {
            const Frag<NI> mk = negative(fk);
#pragma unroll
            for (int t = 0; t < TW; ++t) {
                phase();
                const int tt = tk0 + t;
                if (2 * k2 <= tt) mma(dk[t], mk, read_rows<NH>(e, pos, tt, k2));
                if (2 * k2 + 1 >= tt) mma(dk[t], mk, read_col<NH, false>(e, pos, k2, 16 * tt, 0));
            }
        };
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
            const Frag<NI> fk = read_col<NI, false>(L.k, pos, k2, 16 * d0, 0);
            with_h(k2, fk);
            if constexpr (!Lds::ONE) with_e(k2, fk, L.e);
        }
        if constexpr (Lds::ONE) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int m = 0; m < NH; ++m)
                    if (j0 + 2 * i <= (it | 1)) *quad(&L.h[m], pos, it, j0 + 2 * i) = we[i][m];
            __syncthreads();
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) with_e(k2, read_col<NI, false>(L.k, pos, k2, 16 * d0, 0), L.h);
        }
        if (wave == 0) {
            float cs = 0.f, rs = 0.f, as = 0.f, wr = 0.f, dots = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) cs += L.col[w][lane];
#pragma unroll
            for (int w = 0; w < 8; ++w) dots += L.dot[w];
            rs = L.row[0][lane] + L.row[1][lane];
#pragma unroll
            for (int d = 0; d < DT; ++d) as += L.a[d][lane], wr += L.wr[d][lane];
            const float bt = L.be[lane];
            const double a = as, bw = (double)bt * wr, dcr = (double)bt * cs - (double)rs;
            // Sums over the tokens before this one: not the inclusive sum less this token's part, which
            // is far larger than they are where decays are strong.
            const double sa = wave_cumsum(a), sw = __shfl_up(wave_cumsum(bw + dcr), 1);
            const double dg = (__shfl(sa, 63) - sa + a) + (lane ? sw : 0.0) + (double)decay_exp(gend, 0.0) * (double)dots;
            const int t = t0 + lane;
            if (t < s.T) {
                const int64_t at = (b * s.T + t) * s.Hv + h;
                reinterpret_cast<E*>(A.gg)[at] = (E)(t < len ? (float)dg : 0.f);
                reinterpret_cast<E*>(A.gbeta)[at] = (E)(t < len ? cs + L.diag[lane] + wr : 0.f);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < TW; ++t) {
        const int row = 16 * (tk0 + t) + pos.r, c = 16 * d0 + 4 * pos.g;
        if (t0 + kChunk > len)  // absent tokens, as above
            if (t0 + row >= len) dq[t] = dk[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        store_rows<E, VEC>(rows_of<E>(A.gq, s, b, s.Hk, hk, Dk, t0, (int)s.T), row, c, Dk, dq[t]);
        store_rows<E, VEC>(rows_of<E>(A.gk, s, b, s.Hk, hk, Dk, t0, (int)s.T), row, c, Dk, dk[t]);
    }
}

bool vec_ok(const DeltaShape& s, const DeltaBwdArgs& A) {
    const uintptr_t all = (uintptr_t)A.q | (uintptr_t)A.k | (uintptr_t)A.go | (uintptr_t)A.gq | (uintptr_t)A.gk |
                          (uintptr_t)A.gv;
    return s.Dk % 8 == 0 && s.Dv % 8 == 0 && all % 16 == 0;
}

template <class K>
hipError_t launch(K kernel, int64_t blocks, int bytes, hipStream_t st, const DeltaShape& s, const DeltaBwdArgs& A,
                  const DeltaChunks& W, int threads, int ntile) {
    // More dynamic LDS than the default 64 KiB has to be asked for.
    hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), bytes, st, s, A, W,
                       (int)((s.T + kChunk - 1) / kChunk), ntile, delta_blocks(s));
    return hipGetLastError();
}

template <class E, int KT, int NS, bool VEC>
hipError_t backward(const DeltaShape& s, const DeltaBwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    const int bytes = (int)sizeof(ChainLds<E, KT, NS>), wide = (s.Dv + 127) / 128, narrow = (s.Dv + 63) / 64;
    hipError_t e = hipSuccess;
    bool done = false;
    if constexpr (sizeof(E) == 2)
        if ((done = delta_wide(s)))
            e = launch(delta_chain_kernel<E, KT, 8, VEC, NS>, s.B * s.Hv * wide, bytes, st, s, A, W, 512, wide);
    if (!done)
        e = launch(delta_chain_kernel<E, KT, 4, VEC, NS>, s.B * s.Hv * narrow, bytes, st, s, A, W, 256, narrow);
    if (e != hipSuccess) return e;
    return launch(delta_grad_kernel<E, KT, VEC>, s.B * s.Hk * ((s.T + kChunk - 1) / kChunk),
                  (int)sizeof(GradLds<E, KT>), st, s, A, W, 512, 0);
}

template <class E, int NS, bool VEC>
hipError_t by_width(const DeltaShape& s, const DeltaBwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    if (s.Dk <= 32) return backward<E, 1, NS, VEC>(s, A, W, st);
    if (s.Dk <= 64) return backward<E, 2, NS, VEC>(s, A, W, st);
    return backward<E, 4, NS, VEC>(s, A, W, st);
}

template <bool VEC>
hipError_t by_type(const DeltaShape& s, const DeltaBwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    if (s.dtype != kBf16) return by_width<float, 3, VEC>(s, A, W, st);
    return A.s_in ? by_width<bf16_t, 3, VEC>(s, A, W, st) : by_width<bf16_t, 2, VEC>(s, A, W, st);
}

}  // namespace

hipError_t run_delta_backward(const DeltaShape& s, const DeltaBwdArgs& A, const DeltaChunks& W, hipStream_t st) {
    return vec_ok(s, A) ? by_type<true>(s, A, W, st) : by_type<false>(s, A, W, st);
}

}  // namespace linrec
