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
constexpr int kEw = kChunk, kBe = 2 * kChunk;  // where these start in a chunk's DeltaChunks::dec

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

// A value known to be the same in all lanes, as a scalar: what a buffer resource is made of has
// to be one, or every load through it becomes a loop over the lanes' resources.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Up to 64 rows of a (B,T,H,D) tensor's head from token t0 on, through a buffer resource that
// ends with the row's last token: loads past it, and at the offset kNowhere, return 0.  No load
// is behind a branch, so many are in flight.  (64 rows span less than 2^31 bytes: the host
// checks H*D.)
struct Rows {
    rsrc_t rs;
    unsigned stride;  // bytes from token to token
};
constexpr unsigned kNowhere = 0x80000000u;

template <class E>
__device__ __forceinline__ Rows rows_of(const void* base, const DeltaShape& s, int64_t b, int H, int h, int D, int t0,
                                        int len) {
    const unsigned stride = (unsigned)(H * D * (int)sizeof(E));
    const int left = len - t0 < kChunk ? len - t0 : kChunk;
    const E* p = reinterpret_cast<const E*>(base) + ((b * s.T + t0) * H + h) * (int64_t)D;
    return {__builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(p), (short)0,
                                              uniform((int)stride * (left > 0 ? left : 0)), 0x00020000),
            stride};
}

// 8 elements of row `row` from column c; those at columns >= D, or all if !on, are 0.
// VEC: D % 8 == 0 and rows 16-byte aligned.
template <class E, bool VEC>
__device__ __forceinline__ void load8(const Rows& R, int row, int c, int D, bool on, E* __restrict__ out) {
    const unsigned at = (unsigned)row * R.stride + (unsigned)(c * (int)sizeof(E));
    if constexpr (VEC) {
        constexpr int n = ElemVec<E>::n;
        typedef typename ElemVec<E>::type V;
        const unsigned off = on && c < D ? at : kNowhere;
#pragma unroll
        for (int i = 0; i < 8; i += n) {
            const V t = __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b128(R.rs, off + 4 * i, 0, 0));
#pragma unroll
            for (int j = 0; j < n; ++j) out[i + j] = t[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned off = on && c + i < D ? at + (unsigned)(i * (int)sizeof(E)) : kNowhere;
            if constexpr (sizeof(E) == 2)
                out[i] = __builtin_bit_cast(E, __builtin_amdgcn_raw_buffer_load_b16(R.rs, off, 0, 0));
            else
                out[i] = __builtin_bit_cast(E, __builtin_amdgcn_raw_buffer_load_b32(R.rs, off, 0, 0));
        }
    }
}

// Registers of the chains: half a SIMD's for a wave, or all where a workgroup of four waves has
// the CU to itself (LDS in float32 calls; few heads, see delta_wide, at 128 key channels).
template <class E, int KT, int NW> constexpr int kWavesPerSimd = NW == 8 || (sizeof(E) == 2 && KT < 4) ? 2 : 1;

template <class E> constexpr int kTerms = sizeof(E) == 2 ? 1 : 3;  // bfloat16 terms of an input

// Terms in which the gradients' products take what is kept in float32 (x, the states and their
// gradients) and dZ: two in calls on bfloat16, 2^-16 before each result's own rounding.
template <class E> constexpr int kKeptTerms = sizeof(E) == 2 ? 2 : 3;

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

// A block index as (row, head, rest): rest the fastest of `inner`, then the head of H.
struct BlockPos {
    int64_t b;
    int h, rest;
    __device__ __forceinline__ BlockPos(unsigned blk, int H, int inner) {
        const unsigned row = blk / (unsigned)inner;
        rest = uniform((int)(blk - row * (unsigned)inner));
        h = uniform((int)(row % (unsigned)H));
        b = uniform((int)(row / (unsigned)H));
    }
};

// Tokens of batch row b.
__device__ __forceinline__ int row_length(const DeltaShape& s, int64_t b) {
    int64_t len = s.T;
    if (s.lengths) {
        const int64_t n = s.lengths[b];
        len = n < 0 ? 0 : (n < len ? n : len);
    }
    return uniform((int)len);
}

// A 64-row matrix in LDS, rows of 32*KT bfloat16 values plus 16 bytes.  Rows lie 16 by 16, row
// 4x + a of 16 at place 4a + x: taken 8 lanes at a time (8 rows, one column) the row reads, and 16 at
// a time (4 neighbouring rows, 4 columns) the transposed reads, then fall into banks of their own, and
// every read of a lane is a constant away from one of three places (LanePos).  Conflicts remain all
// the same: 28% of the LDS cycles in the forward chain, 35% in the reverse chain, 36% in the
// gradients (128x128, bfloat16), whose source is not found.
template <int KT>
struct Mat {
    static constexpr int LD = 32 * KT + 8;
    bf16_t v[kChunk * LD];
    __device__ __forceinline__ static int place(int row) { return (row & ~15) | ((row & 3) << 2) | ((row >> 2) & 3); }
    __device__ __forceinline__ bf16x8* row8(int row, int c) { return reinterpret_cast<bf16x8*>(v + place(row) * LD + c); }
};

struct LanePos {
    int r, g;
    int tile;  // place of row tile_row(r, half) less half
    int nat;   // place of row r
    int col;   // place of row 8g + r/4
    __device__ __forceinline__ LanePos() {
        const int lane = threadIdx.x & 63;
        r = lane & 15;
        g = lane >> 4;
        tile = 16 * (r >> 3) + 4 * (r & 3) + 2 * ((r >> 2) & 1);
        nat = 4 * (r & 3) + (r >> 2);
        col = 16 * (g >> 1) + 4 * (r >> 2) + 2 * (g & 1);
    }
    // The same values, but addresses formed from them are formed again: in a loop they would
    // otherwise be kept from before it, in more registers than there are.
    __device__ __forceinline__ void renew() {
        asm volatile("" : "+v"(r), "+v"(g), "+v"(tile), "+v"(nat), "+v"(col));
    }
};

// A chunk of a head on its way to LDS: loads issued for one chunk while another is computed, NT
// threads, 16-byte pieces (of bfloat16) in order.
template <class E, int KT, int NT>
struct RowStage {
    static constexpr int P = kChunk * 4 * KT, I = (P + NT - 1) / NT;
    E x[I][8];
    template <bool VEC>
    __device__ __forceinline__ void load(const Rows& R, int D, int c0 = 0) {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int id = (int)threadIdx.x + i * NT, row = id / (4 * KT), c = 8 * (id % (4 * KT));
            load8<E, VEC>(R, row, c0 + c, D, P % NT == 0 || id < P, x[i]);
        }
    }
    // As bfloat16 terms, zero past D (of 32*KT) and past the row's length.
    __device__ __forceinline__ void store(Mat<KT>* dst) const {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int id = (int)threadIdx.x + i * NT, row = id / (4 * KT), c = 8 * (id % (4 * KT));
            const Frag<kTerms<E>> f = to_frag<E>(x[i]);
            if (P % NT == 0 || id < P)
#pragma unroll
                for (int m = 0; m < kTerms<E>; ++m) *dst[m].row8(row, c) = f.t[m];
        }
    }
};

// N terms of a 64x64 matrix likewise; its upper right 32x32 block, never written, comes as 0.
template <int N, int NT>
struct SquareStage {
    static constexpr int I = N * kChunk * 8 / NT;
    bf16x8 x[I];
    __device__ __forceinline__ void load(const void* src, int64_t cb, int planes) {
        const char* p = reinterpret_cast<const char*>(src) + cb * planes * (kChunk * kChunk * 2);
        const rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), (short)0, N * kChunk * kChunk * 2, 0x00020000);
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int id = (int)threadIdx.x + NT * i;
            const bool upper = (id & 7) >= 4 && ((id >> 3) & 63) < 32;
            x[i] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rs, upper ? kNowhere : 16u * id, 0, 0));
        }
    }
    __device__ __forceinline__ void store(Mat<2>* dst) const {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int id = (int)threadIdx.x + NT * i;
            *dst[id >> 9].row8((id >> 3) & 63, 8 * (id & 7)) = x[i];
        }
    }
};

// A wave's 16 value channels of a chunk as A operands of 32 columns: operand k2 has token tile
// 2*k2 in its first 16 columns and tile 2*k2 + 1 in the others, so that products with
// identity_frag(half) give the D tiles.
template <class E>
struct ColumnStage {
    E x[2][8];
    template <bool VEC>
    __device__ __forceinline__ void load(const Rows& R, int c0, int D) {
        const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2)
            load8<E, VEC>(R, 32 * k2 + tile_row(r, g >> 1), c0 + 8 * (g & 1), D, true, x[k2]);
    }
};

// Row operands (A or B) of columns 32*kk..: rows 32*k2 + tile_row(m, half), or 16*t + m.
template <int N, int KT>
__device__ __forceinline__ Frag<N> read_tile(const Mat<KT>* m, const LanePos& p, int k2, int half, int kk) {
    Frag<N> f;
#pragma unroll
    for (int n = 0; n < N; ++n)
        f.t[n] = *reinterpret_cast<const bf16x8*>(m[n].v + p.tile * Mat<KT>::LD + 8 * p.g +
                                                  ((32 * k2 + half) * Mat<KT>::LD + 32 * kk));
    return f;
}

template <int N, int KT>
__device__ __forceinline__ Frag<N> read_rows(const Mat<KT>* m, const LanePos& p, int t, int kk) {
    Frag<N> f;
#pragma unroll
    for (int n = 0; n < N; ++n)
        f.t[n] = *reinterpret_cast<const bf16x8*>(m[n].v + p.nat * Mat<KT>::LD + 8 * p.g +
                                                  (16 * t * Mat<KT>::LD + 32 * kk));
    return f;
}

// Operands of the transposed matrix: rows 32*k2.. (the product's inner index); columns 32*kk +
// tile_row(m, half) (PERM) or c0 + m.
template <int N, bool PERM, int KT>
__device__ __forceinline__ Frag<N> read_col(const Mat<KT>* m, const LanePos& p, int k2, int c0, int half) {
    Frag<N> f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const bf16_t* at = m[n].v + p.col * Mat<KT>::LD + (PERM ? 8 : 4) * (p.r & 3) +
                           (32 * k2 * Mat<KT>::LD + c0 + 4 * half);
        const bf16x4 lo = read_transposed(at), hi = read_transposed(at + Mat<KT>::LD);
        f.t[n] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return f;
}

// Columns 16*ct + 4g.. of row 16*t + r.
template <int KT>
__device__ __forceinline__ bf16x4* quad(Mat<KT>* m, const LanePos& p, int t, int ct) {
    return reinterpret_cast<bf16x4*>(m->v + p.nat * Mat<KT>::LD + 4 * p.g + (16 * t * Mat<KT>::LD + 16 * ct));
}

// Nothing is scheduled across: keeps a phase's loads from LDS out of the phase before it, whose
// registers they would need.
__device__ __forceinline__ void phase() { __builtin_amdgcn_sched_barrier(0); }

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

// Columns c..c+3 of row `row`; nothing past D or past the rows of R.  Never behind a branch: the
// wait for loads issued before the store then need not wait for the store.
template <class E, bool VEC>
__device__ __forceinline__ void store_rows(const Rows& R, int row, int c, int D, const f32x4& x) {
    const unsigned at = (unsigned)row * R.stride + (unsigned)(c * (int)sizeof(E));
    if constexpr (VEC) {
        typedef E E4 __attribute__((ext_vector_type(4)));
        E4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = (E)x[e];
        const unsigned off = c < D ? at : kNowhere;
        if constexpr (sizeof(E) == 2)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, y), R.rs, off, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), R.rs, off, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned off = c + e < D ? at + (unsigned)(e * (int)sizeof(E)) : kNowhere;
            const E y = (E)x[e];
            if constexpr (sizeof(E) == 2)
                __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, y), R.rs, off, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, y), R.rs, off, 0, 0);
        }
    }
}

}  // namespace linrec
