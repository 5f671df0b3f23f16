// delta_tile.hpp -- matrix tiles of the chunked gated delta rule on the bf16 MFMA.
//
// Products are 16x16x32 (v_mfma_f32_16x16x32_bf16, float32 accumulation).  With l the lane,
// r = l % 16 and g = l / 16, a lane holds
//   A (16 rows x 32):  row r, columns 8g..8g+7          (8 values)
//   B (32 x 16 cols):  column r, rows 8g..8g+7          (8 values)
//   D (16 x 16):       column r, rows 4g..4g+3          (4 values)
// Where the rows of a 32-row block are dealt to two D tiles so that tile 0 holds rows
// 8g..8g+3 and tile 1 rows 8g+4..8g+7 of each lane (`tile_row`), the two tiles together ARE
// the B operand of the next product, and the A operand of the transposed one: a chain of
// products stays in registers.
//
// float32 precision on the bf16 units: a float32 value is the sum of three bfloat16 values
// (8 significant bits each; `split`), and a product of such sums keeps the terms down to
// 2^-16 of the leading one, so what is dropped is below 2^-23 of it (`mma`).  An operand that
// is bfloat16 to begin with is one term.  Six products at the bf16 rate are 2.7 times the
// rate of the float32 MFMA.
#pragma once

#include "elem_types.hpp"
#include "gated_delta.hpp"

namespace linrec {

constexpr int kChunk = 64;  // tokens of a chunk: four D tiles

template <int N> struct Frag { bf16x8 t[N]; };

// Row of a 32-row block held by row m of D tile `half`.
__device__ __forceinline__ int tile_row(int m, int half) { return 8 * (m >> 2) + 4 * half + (m & 3); }

template <int N>
__device__ __forceinline__ Frag<N> split(const float* x) {
    // In pairs: one conversion gives two terms, a shift and a mask give them back as float32.
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        f32x2 r = {x[i], x[i + 1]};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const bf16x2 h = __builtin_convertvector(r, bf16x2);
            f.t[n][i] = h[0];
            f.t[n][i + 1] = h[1];
            if (n + 1 < N) {
                const unsigned u = __builtin_bit_cast(unsigned, h);
                r[0] -= __builtin_bit_cast(float, u << 16);
                r[1] -= __builtin_bit_cast(float, u & 0xffff0000u);
            }
        }
    }
    return f;
}

// The two D tiles of a 32-row block as an operand.
template <int N>
__device__ __forceinline__ Frag<N> split_tiles(const f32x4& a, const f32x4& b) {
    const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return split<N>(x);
}

__device__ __forceinline__ f32x4 mfma(const bf16x8& a, const bf16x8& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// c += a b, the products of terms i, j with i + j below the larger term count; the first M
// terms of each operand only.
template <int NA, int NB, int MA = NA, int MB = NB>
__device__ __forceinline__ void mma(f32x4& c, const Frag<NA>& a, const Frag<NB>& b) {
    constexpr int lim = MA > MB ? MA : MB;
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j)
            if (i + j < lim) c = mfma(a.t[i], b.t[j], c);
}

// The same over several tiles that share an operand, the terms outermost so that neighbouring
// products are independent: c[t] += a[t] b, and c[t] += a b[t].
template <int T, int NA, int NB, int MA = NA, int MB = NB>
__device__ __forceinline__ void mma_rows(f32x4* c, const Frag<NA>* a, const Frag<NB>& b) {
    constexpr int lim = MA > MB ? MA : MB;
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j)
            if (i + j < lim)
#pragma unroll
                for (int t = 0; t < T; ++t) c[t] = mfma(a[t].t[i], b.t[j], c[t]);
}

template <int T, int NA, int NB, int MA = NA, int MB = NB>
__device__ __forceinline__ void mma_cols(f32x4* c, const Frag<NA>& a, const Frag<NB>* b) {
    constexpr int lim = MA > MB ? MA : MB;
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j)
            if (i + j < lim)
#pragma unroll
                for (int t = 0; t < T; ++t) c[t] = mfma(a.t[i], b[t].t[j], c[t]);
}

// Rows of a (B,T,H,D) tensor's head from token t0 on, through a buffer resource: lanes that
// must not load (absent tokens, columns past D) give an offset past its end and get 0, so a
// load is never behind a branch and many are in flight.  64 rows span less than 2^31 bytes
// (the host checks H*D).
struct Rows {
    rsrc_t rs;
    unsigned stride;  // bytes from token to token
};
constexpr unsigned kNowhere = 0x80000000u;

template <class E>
__device__ __forceinline__ Rows rows_of(const void* base, const DeltaShape& s, int64_t b, int H, int h, int D,
                                        int64_t t0) {
    return {make_rsrc(reinterpret_cast<const E*>(base) + ((b * s.T + t0) * H + h) * (int64_t)D, 0x7fffffff),
            (unsigned)(H * D * (int)sizeof(E))};
}

// 8 elements of row `row` from column c; those at columns >= D, or all if !live, are 0.
// VEC: D % 8 == 0 and rows 16-byte aligned.
template <class E, bool VEC>
__device__ __forceinline__ void load8(const Rows& R, int row, int c, int D, bool live, E* __restrict__ out) {
    const unsigned at = (unsigned)row * R.stride + (unsigned)(c * (int)sizeof(E));
    if constexpr (VEC) {
        constexpr int n = ElemVec<E>::n;
        typedef typename ElemVec<E>::type V;
        const unsigned off = live && c < D ? at : kNowhere;
#pragma unroll
        for (int i = 0; i < 8; i += n) {
            const V t = __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b128(R.rs, off + 4 * i, 0, 0));
#pragma unroll
            for (int j = 0; j < n; ++j) out[i + j] = t[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned off = live && c + i < D ? at + (unsigned)(i * (int)sizeof(E)) : kNowhere;
            if constexpr (sizeof(E) == 2)
                out[i] = __builtin_bit_cast(E, __builtin_amdgcn_raw_buffer_load_b16(R.rs, off, 0, 0));
            else
                out[i] = __builtin_bit_cast(E, __builtin_amdgcn_raw_buffer_load_b32(R.rs, off, 0, 0));
        }
    }
}

template <class E> constexpr int kTerms = sizeof(E) == 2 ? 1 : 3;  // bfloat16 terms of an input

// Terms of what the forward keeps for the backward in type KE: written as this many terms'
// sum, read as this many terms in calls on E (two carry float32 kept for bfloat16 tensors).
template <class KE> constexpr int kKeptSum = sizeof(KE) == 2 ? 1 : 3;
template <class E, class KE> constexpr int kKeptTerms = sizeof(KE) == 2 ? 1 : sizeof(E) == 2 ? 2 : 3;

template <class E>
__device__ __forceinline__ Frag<kTerms<E>> to_frag(const E* x) {
    if constexpr (sizeof(E) == 2) {
        Frag<1> f;
#pragma unroll
        for (int i = 0; i < 8; ++i) f.t[0][i] = x[i];
        return f;
    } else {
        return split<3>(x);
    }
}

// Inclusive sum over the 64 lanes of a wave, in float64.
__device__ __forceinline__ double wave_cumsum(double v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// g as summed: -inf (a cleared state) becomes a finite number whose exponential is 0 even
// after 64 of them cancel in a difference with another clearing.
__device__ __forceinline__ double decay_of(float g) { return g < -1e5f ? -1e5 : (double)g; }  // NaN stays

// e^{a - b} of two cumulated decays; the difference in float64, so that it keeps its digits
// behind a cleared state.
__device__ __forceinline__ float decay_exp(double a, double b) {
    return fast_exp2((float)((a - b) * 1.4426950408889634));
}

// Operand of a transposed matrix that lies row-major in LDS: four rows (8-byte pieces at the
// addresses the lanes give, lane 4i + c of a group of 16 giving row i's columns 4c..4c+3) come
// back as lane j holding column j of the four rows.
__device__ __forceinline__ bf16x4 read_transposed(const bf16_t* p) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef s16x4 __attribute__((address_space(3)))* lds_ptr;
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p));
}

// Tokens of batch row b.
__device__ __forceinline__ int row_length(const DeltaShape& s, int64_t b) {
    int64_t len = s.T;
    if (s.lengths) {
        const int64_t n = s.lengths[b];
        len = n < 0 ? 0 : (n < len ? n : len);
    }
    return (int)len;
}

// A chunk of a head on its way to LDS: loads issued for one chunk while another is computed.
// 256 threads, four lanes a row.
template <class E, int KT>
struct RowStage {
    E x[KT][8];
    template <bool VEC>
    __device__ __forceinline__ void load(const Rows& R, int D, int len) {  // len: tokens from the chunk's first
        const int row = threadIdx.x >> 2, quarter = threadIdx.x & 3;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int c = 8 * (quarter + 4 * i);
            load8<E, VEC>(R, row, c, D, row < len, x[i]);
        }
    }
    // As bfloat16 terms into dst[term][row][.], zero past D (of 32*KT) and past the row's length.
    template <int LD>
    __device__ __forceinline__ void store(bf16_t (*dst)[kChunk][LD]) const {
        const int row = threadIdx.x >> 2, quarter = threadIdx.x & 3;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const Frag<kTerms<E>> f = to_frag<E>(x[i]);
#pragma unroll
            for (int m = 0; m < kTerms<E>; ++m)
                *reinterpret_cast<bf16x8*>(&dst[m][row][8 * (quarter + 4 * i)]) = f.t[m];
        }
    }
};

// A chunk's inverse and decays likewise; the inverse as three bfloat16 terms.
template <class E>
struct InverseStage {
    float x[16];
    double gam, end;
    float be;
    __device__ __forceinline__ void load(const DeltaChunks& W, int64_t cb, const Rows& beta, int len) {
        const int row = threadIdx.x >> 2, quarter = threadIdx.x & 3, t = threadIdx.x & 63;
        const float* p = W.tinv + cb * (kChunk * kChunk) + row * kChunk + 8 * quarter;
#pragma unroll
        for (int i = 0; i < 4; ++i) load16<float>(p + 32 * (i >> 1) + 4 * (i & 1), x + 4 * i);
        gam = W.gam[cb * kChunk + t];
        end = W.gam[cb * kChunk + kChunk - 1];
        const unsigned off = t < len ? (unsigned)t * beta.stride : kNowhere;
        if constexpr (sizeof(E) == 2)
            be = (float)__builtin_bit_cast(E, __builtin_amdgcn_raw_buffer_load_b16(beta.rs, off, 0, 0));
        else
            be = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(beta.rs, off, 0, 0));
    }
    template <class Lds>
    __device__ __forceinline__ void store(Lds& L) const {
        const int row = threadIdx.x >> 2, quarter = threadIdx.x & 3, t = threadIdx.x;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const Frag<3> f = split<3>(x + 8 * i);
#pragma unroll
            for (int m = 0; m < 3; ++m) *reinterpret_cast<bf16x8*>(&L.t[m][row][8 * quarter + 32 * i]) = f.t[m];
        }
        if (t < kChunk) {
            L.gam[t] = gam;
            L.eg[t] = decay_exp(gam, 0.0);
            L.ew[t] = decay_exp(end, gam);
            L.be[t] = be;
        }
    }
};

// A wave's 16 value channels of a chunk, as A operands of the four token tiles (the upper 16 of
// an operand's 32 columns are 0).
template <class E>
struct ColumnStage {
    E x[4][8];
    template <bool VEC>
    __device__ __forceinline__ void load(const Rows& R, int c0, int D, int len) {
        const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int row = 32 * (t >> 1) + tile_row(r, t & 1);
            load8<E, VEC>(R, row, c0 + 8 * g, D, row < len && g < 2, x[t]);
        }
    }
};

// Row operand (A or B): 8 columns from c of row `row`.
template <int N, int LD>
__device__ __forceinline__ Frag<N> read_row(const bf16_t (*m)[kChunk][LD], int row, int c) {
    Frag<N> f;
#pragma unroll
    for (int n = 0; n < N; ++n) f.t[n] = *reinterpret_cast<const bf16x8*>(&m[n][row][c]);
    return f;
}

// Column operand of the transposed matrix: rows row0 + 8g.. (32 of them over the wave), columns
// c0 + c(r); PERM: the columns of D tile `half` of a 32-column block, else 16 in order.
template <int N, bool PERM, int LD>
__device__ __forceinline__ Frag<N> read_col(const bf16_t (*m)[kChunk][LD], int row0, int c0, int half) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int row = row0 + 8 * g + (r >> 2), c = PERM ? c0 + 8 * (r & 3) + 4 * half : c0 + 4 * (r & 3);
    Frag<N> f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const bf16x4 lo = read_transposed(&m[n][row][c]), hi = read_transposed(&m[n][row + 4][c]);
        f.t[n] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return f;
}

// B operands of the product with the identity that turns an A operand's 32 rows k into D's
// columns: columns r = k - 16*which.
__device__ __forceinline__ Frag<1> identity_frag(int which) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    Frag<1> f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.t[0][i] = (bf16_t)((8 * g + i) == 16 * which + r ? 1.f : 0.f);
    return f;
}

// Four consecutive elements.
template <class E>
__device__ __forceinline__ void store4(E* p, const f32x4& x) {
    typedef E E4 __attribute__((ext_vector_type(4)));
    E4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = (E)x[e];
    *reinterpret_cast<E4*>(p) = y;
}

// Columns c..c+3 of a row of D; VEC: D % 4 == 0 and the row 4*sizeof(E)-byte aligned.
template <class E, bool VEC>
__device__ __forceinline__ void store_cols(E* row, int c, int D, const f32x4& x) {
    if constexpr (VEC) {
        if (c < D) store4<E>(row + c, x);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < D) row[c + e] = (E)x[e];
    }
}

}  // namespace linrec
