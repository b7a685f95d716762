// ops.hpp -- internal types of the operators of include/mlstm_ops.h (linear
// attention with a decay for each head, group norm with an activation).
#pragma once

#include "common.hpp"

namespace mlstm {

struct Strides {
    long long s0, s1, s2;
};

// One linear attention over "local" tokens tau = 0 .. n-1 of every (b, h):
//   o_tau  = in_scale e^{g (tau + 1 - shift)} X0^T q_tau
//            + sum_{sigma <= tau} e^{g (tau - sigma)} p_scale (q_tau . k_sigma) v_sigma,
//   X_n    = e^{g n} X0 + up_scale sum_sigma e^{g (n - 1 + shift - sigma)} k_sigma v_sigma^T
// with X [dk x dv].  The forward is one of these; the backward is three (dq
// runs forward with q = do, k = v, v = k; dv and dk run backwards in time,
// where the carried gradient has already decayed once: shift = 1).
struct LinJob {
    const void *q, *k, *v;      // rows of dk, dk and dv elements, io dtype
    void *o;                    // rows of dv elements
    Strides sq, sk, sv, so;     // over (b, h, t)
    const float *X0;            // initial state of each (b, h), NULL = zero
    float *Xn;                  // final state, NULL = not wanted
    long long rs, cs;           // element strides of a state's rows (dk) and columns (dv)
    int dk, dv;
    float p_scale, in_scale, up_scale;
    int shift, reverse;         // reverse: local token tau is token n - 1 - tau
};

struct LinArgs {
    LinJob job[3];
    int njob;
    const float *g;             // [H]
    const int *lengths;         // [B] or NULL
    int B, H, T;
    float *ws;
};

size_t linattn_workspace_floats(int B, int H, int T, int dk, int dv, int io_bf16, int backward);
hipError_t launch_linattn(const LinArgs &a, int io_bf16, hipStream_t s);

struct LinStepArgs {
    const void *q, *k, *v;
    const float *g, *S_in;
    void *o;
    float *S_out;
    Strides sq, sk, sv, so;     // over (b, h)
    float scale;
    int B, H, dk, dv;
};
hipError_t launch_linattn_step(const LinStepArgs &a, int io_bf16, hipStream_t s);

struct GnArgs {
    const void *x, *dy;         // [N, S, G, D]; dy NULL in the forward
    const float *w, *b;         // [G, D] or NULL
    float *mean, *rstd;         // forward: written or NULL; backward: read
    void *y;                    // y, or dx in the backward
    float *dw, *db;             // [G, D] or NULL
    Strides sx, sdy, sy;
    int N, S, G, D;
    int seq;                    // statistics over all positions
    int act;
    float eps;
    float *ws;
};
size_t groupnorm_workspace_floats(int N, int S, int G, int D, int seq, int io_bf16, int backward);
hipError_t launch_groupnorm(const GnArgs &a, int io_bf16, hipStream_t s);

// Decay of one step in base 2: e^g = 2^(decay_log2(g)).  -inf becomes a large
// finite number, so that 0 steps times it is 0 and 1 step is 2^-huge = 0; NaN stays.
__device__ __forceinline__ float decay_log2(float g) {
    const float x = g * 1.4426950408889634f;
    return x < -1e30f ? -1e30f : x;
}

}  // namespace mlstm
