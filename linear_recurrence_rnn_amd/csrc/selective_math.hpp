// selective_math.hpp -- what the kernels of the selective scan share: the step's softplus and its
// derivative, the gate, scalar loads and the place of a lane's channel.
#pragma once

#include "selective_scan.hpp"
#include "row_ops.hpp"

namespace linrec {

constexpr float kLn2 = 0.69314718055994531f;

// e^x for x <= 0: 2^p for p = x log2(e) as rounded, and what that rounding left of x, x - p ln 2, to first order.
// kLn2 is 2.7e-9 of ln 2 away from it, which costs x * 2^-28 of the result; without the second term the product's
// rounding would cost x * 2^-24, up to four bits of a step of 1e-7.  With bfloat16 tensors too: where steps are
// small, most of x is the bias, which is float32, and so are the states and sums that a step reaches.
__device__ __forceinline__ float exp_neg(float x) {
    x = __builtin_elementwise_maximum(x, -104.f);  // 0 there; a NaN stays one
    const float p = x * kLog2e;
    const float e = fast_exp2(p);
    return fmaf(e, fmaf(-p, kLn2, x), e);
}

// softplus(x) = max(x, 0) + log(1 + e^{-|x|}).  The logarithm of w = 1 + e as rounded, and what
// that rounding lost, e - (w - 1), which is all there is left of a small e.
// sig: the logistic function of x, softplus's derivative.
__device__ __forceinline__ float softplus(float x, float& sig) {
    const float e = exp_neg(-fabsf(x));
    const float w = 1.f + e;
    const float r = __builtin_amdgcn_rcpf(w);
    sig = x >= 0.f ? r : e * r;
    return fmaxf(x, 0.f) + fmaf(__builtin_amdgcn_logf(w), kLn2, e - (w - 1.f));
}

// One element at a wave-uniform base and a lane's byte offset: the form that takes two scalar registers
// and one vector register for the address.
template <class E>
__device__ __forceinline__ E load_elem(const void* base, unsigned at) {
    return *reinterpret_cast<const E*>(reinterpret_cast<const char*>(base) + at);
}
template <class V>
__device__ __forceinline__ void store_as(void* base, unsigned at, V x) {
    *reinterpret_cast<V*>(reinterpret_cast<char*>(base) + at) = x;
}
template <class E>
__device__ __forceinline__ void store_elem(void* base, unsigned at, float x) {
    store_as<E>(base, at, (E)x);
}
template <class E>
__device__ __forceinline__ const void* elems(const void* p, int64_t first) {
    return reinterpret_cast<const E*>(p) + first;
}

// What the states of one wave need of a few tokens: B and C by scalar loads, NF floats, and the
// channels' own pair of floats from LDS.  Scalar loads come back in any order, so a wait for one is a
// wait for all of them and for LDS: both are asked for together, one group ahead of their use.
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef f32x16 f32x16_at16 __attribute__((aligned(16)));  // at 16 bytes, which is what a workspace is sure to start on
static_assert(alignof(f32x16_at16) == 16 && sizeof(f32x16_at16) == 64);

template <int NPT, int NF = 32>
struct SelGroup {
    static constexpr int kTok = NF / 2 / NPT;         // tokens of a group
    static constexpr int kGroups = kSelTile / kTok;   // groups of a tile
    f32x16 bc[NF / 16];
    f32x2 x[kTok];
    // row: the wave's 2*NPT floats of the tile's first token, those of its other tokens behind them.
    __device__ __forceinline__ void fetch(const float* row, const f32x2 (*din)[64], int lane, int q) {
        fetch(row, q);
#pragma unroll
        for (int k = 0; k < kTok; ++k) x[k] = din[q * kTok + k][lane];
    }
    __device__ __forceinline__ void fetch(const float* row, int q) {
        typedef const __attribute__((address_space(4))) f32x16_at16* P;
        const P p = reinterpret_cast<P>(reinterpret_cast<uintptr_t>(row + q * NF));
#pragma unroll
        for (int k = 0; k < NF / 16; ++k) bc[k] = p[k];
    }
    __device__ __forceinline__ float B(int k, int i) const { return bc[(k * 2 * NPT + i) / 16][(k * 2 * NPT + i) % 16]; }
    __device__ __forceinline__ float C(int k, int i) const { return B(k, NPT + i); }
};

// LDS written by lanes of this wave is read by others of it behind this, and what was read may be written.  The wave's
// LDS accesses are carried out in their order anyway: this keeps the compiler to it, and costs no instruction.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// v, or zero: formed in any case, as a branch around it would part it from its neighbours.
__device__ __forceinline__ float where(bool there, float v) {
    asm volatile("" : "+v"(v));
    return there ? v : 0.f;
}

// The workgroup's place among n, such that `together` neighbours, which read the same tokens' lines, run on one of
// the eight chiplets that workgroups go round, and share its cache.
__device__ __forceinline__ unsigned place_of(unsigned i, unsigned n, unsigned together) {
    if (i >= n / (8 * together) * (8 * together)) return i;
    return (i / 8 / together * 8 + i % 8) * together + i / 8 % together;
}

// Tokens of row b that are there.
__device__ __forceinline__ int64_t row_length(const SelShape& s, int64_t b) { return tokens_of(s.lengths, s.T, b); }

// Element (row, n, c) of an array of states between kernels.
__device__ __forceinline__ int64_t state_at(const SelShape& s, int64_t row, int n, int64_t c) {
    return ((row * ((s.N + 3) / 4) + n / 4) * s.C + c) * 4 + (n & 3);
}

}  // namespace linrec
