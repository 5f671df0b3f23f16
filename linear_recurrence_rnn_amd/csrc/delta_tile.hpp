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
    Frag<N> f;
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f.t[n][i] = (bf16_t)r[i];
            if (n + 1 < N) r[i] -= (float)f.t[n][i];
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

// 8 elements p[0..7] of which those at c.. >= D, or all if !live, are 0.  VEC: D % 8 == 0 and
// p 16-byte aligned.
template <class E, bool VEC>
__device__ __forceinline__ void load8(const E* __restrict__ p, int c, int D, bool live, E* __restrict__ out) {
    constexpr int n = ElemVec<E>::n;
    typedef typename ElemVec<E>::type V;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 8; i += n) {
            V t = {};
            if (live && c < D) t = *reinterpret_cast<const V*>(p + i);
#pragma unroll
            for (int j = 0; j < n; ++j) out[i + j] = t[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = (live && c + i < D) ? p[i] : (E)0.f;
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

// Stage rows t0.. of a (B,T,H,D) tensor's head h as bfloat16 terms into dst[term][row][LD]: 256
// threads, four lanes a row, zero past D (of 32*KT) and past the row's length.
template <class E, int KT, bool VEC, int LD>
__device__ __forceinline__ void stage_rows(const void* src, const DeltaShape& s, int64_t b, int H, int h, int D, int t0,
                                           int len, bf16_t (*dst)[kChunk][LD]) {
    const int row = threadIdx.x >> 2, quarter = threadIdx.x & 3;
    const E* p = reinterpret_cast<const E*>(src) + ((b * s.T + t0 + row) * H + h) * (int64_t)D;
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const int c = 8 * (quarter + 4 * i);
        E x[8];
        load8<E, VEC>(p + c, c, D, t0 + row < len, x);
        const Frag<kTerms<E>> f = to_frag<E>(x);
#pragma unroll
        for (int m = 0; m < kTerms<E>; ++m) *reinterpret_cast<bf16x8*>(&dst[m][row][c]) = f.t[m];
    }
}

// A chunk's inverse as three bfloat16 terms.
template <int LD>
__device__ __forceinline__ void stage_inverse(const float* __restrict__ src, bf16_t (*dst)[kChunk][LD]) {
    const int row = threadIdx.x >> 2, quarter = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = 8 * (quarter + 4 * i);
        float x[8];
        load16<float>(src + row * kChunk + c, x);
        load16<float>(src + row * kChunk + c + 4, x + 4);
        const Frag<3> f = split<3>(x);
#pragma unroll
        for (int m = 0; m < 3; ++m) *reinterpret_cast<bf16x8*>(&dst[m][row][c]) = f.t[m];
    }
}

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
