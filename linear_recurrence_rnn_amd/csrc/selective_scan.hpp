// selective_scan.hpp -- host-visible interface of the selective state space scan (internal).
//
// Per batch row b, channel c (of C, in G groups of C/G) and state n (of N), with g = c / (C/G):
//   d_t = softplus(dt_t + bias)  (or dt_t + bias)
//   h_t[n] = e^{d_t A[n]} h_{t-1}[n] + d_t u_t B_t[g,n]
//   y_t = (sum_n C_t[g,n] h_t[n] + D u_t) silu(z_t)      (without z: no gate)
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace linrec {

constexpr int kSelMaxN = 128;  // states of a channel: 16 a lane, 8 waves
constexpr int kSelTile = 16;   // tokens between two kept states, and staged at once
constexpr int kSelBlock = 64;  // tokens of a workgroup of the backward, up to 4 times as many or as few

struct SelShape {
    int64_t B, T, C;
    int G, N;
    int dtype;           // kF32 or kBf16: u, dt, z, B, C, y and their gradients
    int softplus;
    const int* lengths;  // (B) device, or null: tokens at or beyond a row's length are absent
};

struct SelArgs {
    const void *u, *dt;        // (B,T,C)
    const float* A;            // (C,N)
    const void *Bm, *Cm;       // (B,T,G,N)
    const float *D, *bias;     // (C), or null
    const void* z;             // (B,T,C), or null
    const float* s_in;         // (B,C,N), or null (zero)
    void* y;                   // (B,T,C); null in a call that only keeps for the backward
    float* s_out;              // (B,C,N), or null; may be s_in
};

struct SelBwdArgs {
    const void* gy;            // (B,T,C)
    const float* gs_out;       // (B,C,N), or null
    void *gu, *gdt, *gB, *gC, *gz;  // as u, dt, Bm, Cm, z (gz null without z)
    float *gA, *gD, *gbias;    // as A, D, bias (null where those are)
    float* gs_in;              // (B,C,N), or null; may be gs_out
};

// States between kernels are laid out (rows, N/4 rounded up, C, 4).
inline int sel_n4(const SelShape& s) { return (s.N + 3) / 4; }
inline int64_t sel_tiles(const SelShape& s) { return (s.T + kSelTile - 1) / kSelTile; }

// Tokens of the backward's workgroups.  Longer ones write fewer partial sums and states: a training step of 8 x 4096
// tokens of 2560 channels takes 1922 us with 64, 1867 with 128 and 1852 with 256.  They are for many of them, six times
// the 768 that the chip holds, so that the last ones, and ragged rows, do not leave it idle; and for offsets of 32 bits.
// Shorter ones where the chip holds them all: 4 ragged rows of up to 500 tokens, 200 channels in two groups and 24 states,
// 256 workgroups of 64 tokens or 512 of 32, take 27 and 17 us for the gradients, 12 and 9 for the reverse walk.
inline int64_t sel_block_groups(const SelShape& s, int64_t tokens) {  // workgroups
    return s.B * ((s.T + tokens - 1) / tokens) * s.G * ((s.C / s.G + 63) / 64) * ((s.N + 15) / 16);
}
inline int sel_block(const SelShape& s) {
    int tokens = kSelBlock;
    while (tokens > kSelTile && sel_block_groups(s, tokens / 2) <= 768) tokens /= 2;
    while (tokens < 4 * kSelBlock && sel_block_groups(s, 2 * tokens) >= 4608 && s.C * sel_n4(s) < (1 << 22)) tokens *= 2;
    return tokens;
}
inline int64_t sel_blocks(const SelShape& s) { return (s.T + sel_block(s) - 1) / sel_block(s); }
// Rows of the shares of D's gradient and the bias's: with more than 16 states another kernel forms them.
inline int64_t sel_share_rows(const SelShape& s) {
    return s.B * (s.N > 16 ? (s.T + kSelBlock - 1) / kSelBlock : sel_blocks(s));
}

// How the forward is split: states of a lane, waves of a workgroup, segments of the rows.
struct SelPlan {
    int npt, waves, tiles_n;  // workgroups share the states: tiles_n of them (forward: 1)
    int64_t segs, seg_tiles;  // segments, and tiles of one
};
SelPlan sel_plan(const SelShape& s);
SelPlan sel_backward_plan(const SelShape& s);  // (no segments: the backward has blocks)

// Scratch of the forward: bc, and where the rows are cut into segments `agg` and `sum`.
struct SelScratch {
    float* bc;    // (B,tiles,G,tiles_n*waves,16,2,npt): B and C in float32, zero for absent tokens and behind T
    float* agg;   // (B,segs) rows of states
    float* sum;   // (B,segs,C) sums of d
};
size_t sel_bc_floats(const SelShape& s, const SelPlan& p);

// Scratch of the backward.
struct SelBwdScratch {
    float* carry;  // (B,blocks) rows of states: the gradient that enters each block from its right
    float* sum;    // (B,blocks,C) sums of d
    float* gA;     // (B*blocks) rows of states
    float* gDb;    // (share rows,2,C): D's gradient, bias's
    float* gBC;    // (cuts,B,T,G,2,4*n4): B's and C's gradients by ranges of 64 channels of a group
    float* q;      // (tiles of 16 states,3,B,T,C) where N > 16: sums over the states of one
    int64_t cuts;
};

// keep: (B,tiles) rows of states, the state before each tile; null: not kept.
hipError_t run_sel_prepare(const SelShape& s, const SelArgs& A, const SelPlan& p, float* bc, hipStream_t st);
hipError_t run_sel_forward(const SelShape& s, const SelArgs& A, const SelPlan& p, const SelScratch& W, float* keep,
                           hipStream_t st);
hipError_t run_sel_step(const SelShape& s, const SelArgs& A, hipStream_t st);
// v (B,blocks) rows of states holding each block's share h_k -> the state entering each, in place,
// by s_{k+1} = e^{A sum_k} s_k + h_k from s_0 = in (zero if null), forwards, or backwards with
// reverse; the last result goes to `out` if given.
hipError_t run_sel_join(const SelShape& s, const float* A, float* v, const float* sum, int64_t blocks, const float* in,
                        float* out, bool reverse, hipStream_t st);
hipError_t run_sel_backward(const SelShape& s, const SelArgs& A, const SelBwdArgs& g, const float* bc, const float* keep,
                            const SelBwdScratch& W, hipStream_t st);

}  // namespace linrec
