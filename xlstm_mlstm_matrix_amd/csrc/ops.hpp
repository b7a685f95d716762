// ops.hpp -- internal types of the operators of include/mlstm_ops.h (linear
// attention with a decay for each head, the gated delta rule, group norm with an
// activation, norm and rotation of queries and keys).
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

// The gated delta rule; the members of the second half are the backward's.
struct DeltaArgs {
    const void *q, *k, *v;      // [B, Hk, T, dk] x2, [B, H, T, dv]
    const float *g, *beta;      // [B, H, T]
    const float *S0;
    const int *lengths;
    void *o;
    float *S_T;
    Strides sq, sk, sv, sg, sb, so;
    float scale;
    int B, Hk, H, T, dk, dv;
    float *ws;
    const void *d_o;
    const float *dS_T;
    void *dq, *dkk, *dvv;
    float *dg, *db, *dS0;
    Strides sdo, sdq, sdk, sdv, sdg, sdb;
};
// the caller refuses sizes past its limit
size_t deltarule_workspace_floats(int B, int H, int T, int dk, int dv, int io_bf16, int backward);
hipError_t launch_deltarule_fwd(const DeltaArgs &a, int io_bf16, hipStream_t s);
hipError_t launch_deltarule_bwd(const DeltaArgs &a, int io_bf16, hipStream_t s);

struct DeltaStepArgs {
    const void *q, *k, *v;
    const float *g, *beta, *S_in;
    void *o;
    float *S_out;
    Strides sq, sk, sv, sg, sb, so;  // over (b, h)
    float scale;
    int B, Hk, H, dk, dv;
};
hipError_t launch_deltarule_step(const DeltaStepArgs &a, int io_bf16, hipStream_t s);

// Norm and rotation of queries (tensor 0) and keys (tensor 1; H[1] = 0 without).
struct QkArgs {
    const void *x[2], *dy[2];   // dy: backward
    void *y[2];                 // y, or dx in the backward
    const float *w[2];
    float *dw[2];
    Strides sx[2], sdy[2], sy[2];
    const float *freq;
    const int *pos;
    int B, T, H[2], d, nf;
    int pairs;                  // neighbouring channels make a pair
    int norm;                   // mlstm_qknorm_t
    float amp, eps;
    float *ws;
};
size_t qknorm_workspace_floats(int B, int H, int Hk, int T, int d);
hipError_t launch_qknorm(const QkArgs &a, int io_bf16, hipStream_t s);

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
