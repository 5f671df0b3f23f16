// gated_delta.hpp -- host-visible interface of the gated delta rule (internal).
//
// Per batch row b and value head h (reading key head h / (Hv / Hk)), with the state S
// (Dk, Dv) and a_t = e^{g_t}:
//   x_t = v_t - (a_t S_{t-1})^T k_t,   S_t = a_t S_{t-1} + beta_t k_t x_t^T,   o_t = scale S_t^T q_t
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace linrec {

constexpr int kDeltaMaxDk = 128;  // key channels a head may have: a wave keeps them all in registers
constexpr int kDeltaMaxDv = 256;

struct DeltaShape {
    int64_t B, T;
    int Hk, Hv, Dk, Dv;
    int dtype;           // kF32 or kBf16: q, k, v, g, beta, o and their gradients
    const int* lengths;  // (B) device, or null: tokens at or beyond a row's length are absent
    float scale;
};

struct DeltaFwdArgs {
    const void *q, *k;   // (B,T,Hk,Dk)
    const void* v;       // (B,T,Hv,Dv)
    const void *g, *beta;  // (B,T,Hv)
    const float* s_in;   // (B,Hv,Dk,Dv), or null (zero)
    void* o;             // (B,T,Hv,Dv)
    float* s_out;        // (B,Hv,Dk,Dv), or null; may be s_in
};

// What the chunked kernels keep of each chunk of 64 tokens, (B*Hv, chunks, ...):
//   tinv  (64,64) float32   (I + strictly lower e^{gam_i - gam_j} (k_i.k_j) beta_j)^{-1}
//   gam   (64) float64      decays cumulated within the chunk
struct DeltaChunks {
    float* tinv;
    double* gam;
};
inline int64_t delta_chunks(const DeltaShape& s) { return s.B * s.Hv * ((s.T + 63) / 64); }

hipError_t run_delta_prepare(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st);
hipError_t run_delta_forward(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st);

// Token by token, the state in registers: decoding and the shortest sequences.
hipError_t run_delta_recurrent(const DeltaShape& s, const DeltaFwdArgs& A, hipStream_t st);

}  // namespace linrec
