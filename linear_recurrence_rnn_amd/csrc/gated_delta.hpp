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
    void* o;             // (B,T,Hv,Dv); null in a call that only keeps for the backward
    float* s_out;        // (B,Hv,Dk,Dv), or null; may be s_in
};

// What the chunked kernels keep of each chunk of 64 tokens, (B*Hv, chunks, ...):
//   inv   (3,64,64)         N = (I + strictly lower e^{gam_i - gam_j} (k_i.k_j) beta_j)^{-1}, as three
//                           bfloat16 terms
//   p     (np,64,64)        P_ij = scale e^{gam_i - gam_j} q_i.k_j (i >= j, else 0), as np terms
//                           (the upper right 32x32 blocks of both are not written)
//   gam   (64) float64      decays cumulated within the chunk
//   dec   (3,64) float32    e^gam, e^{gam_63 - gam}, beta
// and for the backward, in float32, in blocks of 16 value channels (delta_blocks(s) of them, zero
// past Dv).  They enter every gradient: with the states in bfloat16 and dZ as rounded in dV, the
// errors (2-norm) of bfloat16 gradients were 1.2 to 2.2 times their final rounding's where decays are
// slow or a gradient of the final state comes in; so they are that rounding's, to three digits.  A
// training step of 8 x 4096 tokens and 20 heads of 128x128 takes 2206 us for 1890.
//   x     (blocks, 64, 16)       x_t of the recurrence
//   s0    (blocks, dkp, 16)      the state before the chunk, dkp = Dk rounded up (delta_dkp)
//   ds    (blocks, dkp, 16)      the gradient of the state after the chunk
// and, laid out as v, what the bfloat16 result dV = dZ leaves of dZ (bfloat16 calls only):
//   dz    (B,T,Hv,Dv) bfloat16   dZ - dV
struct DeltaChunks {
    void *inv, *p;
    int np;
    double* gam;
    float* dec;
    float* x;  // null: nothing is kept
    float *s0, *ds;
    void* dz;
    // Long rows of few heads are walked in `segs` segments of `seg_len` chunks (1: in one).  A
    // chunk maps the state to (matrix) state + (matrix), so a segment does: `map` holds, for all
    // but the last, (dkp, 16*blocks + dkp) float32, the map's constant part and its matrix;
    // `start` the state before every segment, (segs, B, Hv, Dk, Dv) float32.
    int segs, seg_len;
    float *map, *start;
};
inline int64_t delta_chunks(const DeltaShape& s) { return s.B * s.Hv * ((s.T + 63) / 64); }
inline int delta_blocks(const DeltaShape& s) { return (s.Dv + 127) / 128 * 8; }
// Eight waves to a workgroup (bfloat16 calls) where a head has the value channels for them and
// workgroups of four would be more than the 256 CUs; four, on twice the CUs, else.  1024 tokens,
// four against eight: 128 heads of 128x128 107 us against 122, 136 heads 182 against 133 (training
// step 467 against 525, 661 against 565); of 128x256 64 heads 97 against 115, 68 heads 165 against
// 117; of 64x128 128 heads 78 against 90, 136 heads 108 against 98.
inline bool delta_wide(const DeltaShape& s, int segs = 1) {
    return s.Dv > 64 && s.B * s.Hv * segs * ((s.Dv + 63) / 64) > 256;
}
inline int delta_dkp(const DeltaShape& s) { return s.Dk <= 32 ? 32 : s.Dk <= 64 ? 64 : 128; }

struct DeltaBwdArgs {
    const void *q, *k, *v, *g, *beta;
    const float* s_in;
    const void* go;       // (B,T,Hv,Dv)
    const float* gs_out;  // (B,Hv,Dk,Dv), or null (zero)
    void *gq, *gk;        // (B,T,Hk,Dk)
    void* gv;             // (B,T,Hv,Dv)
    void *gg, *gbeta;     // (B,T,Hv)
    float* gs_in;         // (B,Hv,Dk,Dv), or null; may be gs_out; only with s_in
};

// Segments: as many as fill the chip with workgroups, of eight chunks at least, where that
// divides the chain by six or more (a segment is walked twice, the first time with Dk columns
// more); else one.  One walk against segments, bfloat16 128x128: one head of 48 chunks in six 207
// against 101 us, 42 heads of 96 in six 497 against 374.  Fewer gain less (64 heads of 96 in four
// 550 against 528, one head of 24 in three 111 against 92) and are not taken.  Each segment takes
// delta_segment_length chunks, the last what is left, and none is empty: the last one's workgroups
// alone write the final state.
inline int delta_segments(const DeltaShape& s) {
    const int64_t nc = (s.T + 63) / 64, cols = s.dtype == 1 ? 128 : 64;
    int64_t n = 256 / (s.B * s.Hv * ((s.Dv + cols - 1) / cols));
    n = n < nc / 8 ? n : nc / 8;
    if (n < 6) return 1;
    const int64_t len = (nc + n - 1) / n;
    return (int)((nc + len - 1) / len);
}
inline int delta_segment_length(const DeltaShape& s, int segs) { return (int)(((s.T + 63) / 64 + segs - 1) / segs); }

hipError_t run_delta_prepare(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st);
hipError_t run_delta_forward(const DeltaShape& s, const DeltaFwdArgs& A, const DeltaChunks& W, hipStream_t st);

// The gradients, from what run_delta_prepare and a keeping run_delta_forward left in W.
hipError_t run_delta_backward(const DeltaShape& s, const DeltaBwdArgs& A, const DeltaChunks& W, hipStream_t st);

// Token by token, the state in registers: decoding and the shortest sequences.
hipError_t run_delta_recurrent(const DeltaShape& s, const DeltaFwdArgs& A, hipStream_t st);

}  // namespace linrec
