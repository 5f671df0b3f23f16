// elem_types.hpp -- element types of the operators that take float32 or bfloat16 tensors:
// conversions and 16-byte loads and stores.  All arithmetic is float32; a value is rounded
// to bfloat16 (nearest, ties to even) only when it is stored.
#pragma once

#include "device_common.hpp"

namespace linrec {

typedef __bf16 bf16_t;
typedef bf16_t bf16x2 __attribute__((ext_vector_type(2)));
typedef bf16_t bf16x4 __attribute__((ext_vector_type(4)));
typedef bf16_t bf16x8 __attribute__((ext_vector_type(8)));

// dtype codes of the C ABI (LINREC_F32, LINREC_BF16).
constexpr int kF32 = 0, kBf16 = 1;

template <class E> struct ElemVec;  // elements in 16 bytes
template <> struct ElemVec<float> { static constexpr int n = 4; typedef f32x4 type; };
template <> struct ElemVec<bf16_t> { static constexpr int n = 8; typedef bf16x8 type; };

// n = 16 / sizeof(E) consecutive elements at p (16-byte aligned) as float32.  NT: streamed once.
template <class E, bool NT = false>
__device__ __forceinline__ void load16(const E* __restrict__ p, float* __restrict__ out) {
    typedef typename ElemVec<E>::type V;
    V t;
    if constexpr (NT) t = __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
    else t = *reinterpret_cast<const V*>(p);
#pragma unroll
    for (int i = 0; i < ElemVec<E>::n; ++i) out[i] = (float)t[i];
}

template <class E, bool NT = false>
__device__ __forceinline__ void store16(E* __restrict__ p, const float* __restrict__ in) {
    typedef typename ElemVec<E>::type V;
    V t;
#pragma unroll
    for (int i = 0; i < ElemVec<E>::n; ++i) t[i] = (E)in[i];
    if constexpr (NT) __builtin_nontemporal_store(t, reinterpret_cast<V*>(p));
    else *reinterpret_cast<V*>(p) = t;
}

}  // namespace linrec
