// ops_api.cpp -- the C ABI of include/mlstm_ops.h: validation and launches.
//
// As in api.cpp, every check runs on the host before any device work, so an
// invalid call enqueues nothing and touches no device.
#include "mlstm_ops.h"

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "hostcheck.hpp"
#include "ops.hpp"

using namespace mlstm;

namespace {

constexpr int kMaxDk = 256, kMaxDv = 512;
// a chunk's rows are addressed through 32-bit byte offsets from its first one
constexpr long long kMaxRowStride = ((long long)1 << 22) - 1;
constexpr int kMaxT = 1 << 30;  // token indices, one segment past the last included, fit 32 bits

// One strided tensor of a call: rows of `d` elements at (i0, i1, i2).
struct View {
    const void *p;
    Strides st;
    int n0, n1, n2, d;
    bool out;
};

Strides dense(long long n1, long long n2, long long d) { return Strides{n1 * n2 * d, n2 * d, d}; }

// The call's strides for tensor i, with those of dimensions of size 1 set to 0.
Strides pick(const mlstm_strides_t *s, int i, Strides dflt, int n0, int n1, int n2) {
    Strides r = s ? Strides{s[i].s0, s[i].s1, s[i].s2} : dflt;
    if (n0 == 1) r.s0 = 0;
    if (n1 == 1) r.s1 = 0;
    if (n2 == 1) r.s2 = 0;
    return r;
}

// Byte extent of a view; false when its offsets overflow or a stride is negative.
bool extent(const View &v, size_t es, Range *r) {
    const long long st[3] = {v.st.s0, v.st.s1, v.st.s2};
    const int n[3] = {v.n0, v.n1, v.n2};
    size_t last = (size_t)v.d;
    for (int i = 0; i < 3; ++i) {
        size_t x;
        if (st[i] < 0 || !mul_ok((size_t)st[i], (size_t)(n[i] - 1), &x) || x > ((size_t)1 << 60)) return false;
        last += x;
    }
    *r = rng(v.p, last * es);
    return true;
}

// No element of the view is at the address of another: taken by rising stride,
// each dimension steps over everything inside it.
bool disjoint_rows(const View &v) {
    long long st[3] = {v.st.s0, v.st.s1, v.st.s2};
    int n[3] = {v.n0, v.n1, v.n2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) {
                const long long t = st[i];
                st[i] = st[j];
                st[j] = t;
                const int m = n[i];
                n[i] = n[j];
                n[j] = m;
            }
    long long span = v.d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (st[i] < span) return false;
        span += st[i] * (n[i] - 1);
    }
    return true;
}

// Strided and dense arguments of a call, and their overlap rules.
struct Extents {
    Range in[12], out[8];
    int ni = 0, no = 0;
    void input(Range r) { in[ni++] = r; }
    void output(Range r) { out[no++] = r; }
    // every output apart from every other argument; `same_ok`: output so may be input si exactly
    bool ok(int so, int si) const {
        for (int o = 0; o < no; ++o) {
            for (int i = 0; i < ni; ++i)
                if (overlaps(out[o], in[i]) && !(o == so && i == si && same(out[o], in[i]))) return false;
            for (int p = o + 1; p < no; ++p)
                if (overlaps(out[o], out[p])) return false;
        }
        return true;
    }
};

// Shapes of a linear attention call; *cells = B * H.
mlstm_status_t lin_dims(int B, int H, int T, int dk, int dv, mlstm_dtype_t io, size_t *cells) {
    if (B <= 0 || H <= 0 || T <= 0 || T > kMaxT || dk <= 0 || dv <= 0) return MLSTM_ERR_SHAPE;
    if (io != MLSTM_F32 && io != MLSTM_BF16) return MLSTM_ERR_UNSUPPORTED;
    if (dk > kMaxDk || dk % 16 || dv > kMaxDv || dv % 16) return MLSTM_ERR_UNSUPPORTED;
    // workgroups are counted in 32 bits; a cell has at most 4096 of them
    if (!mul_ok((size_t)B, (size_t)H, cells) || *cells > (size_t)INT32_MAX / 4096) return MLSTM_ERR_SHAPE;
    return MLSTM_OK;
}

// The strided tensors of a linear attention call: strides, alignment and extents.
mlstm_status_t lin_views(View *v, int n, mlstm_dtype_t io, bool tokens, Extents *x) {
    const size_t es = io == MLSTM_BF16 ? 2 : 4;
    for (int i = 0; i < n; ++i) {
        Range r;
        if (!extent(v[i], es, &r)) return MLSTM_ERR_SHAPE;
        const Strides &s = v[i].st;
        if ((s.s0 * es) % 16 || (s.s1 * es) % 16 || (s.s2 * es) % 16) return MLSTM_ERR_ALIGN;
        if (tokens) {
            if (v[i].n2 == 1)
                v[i].st.s2 = v[i].d;
            else if (s.s2 < v[i].d || s.s2 > kMaxRowStride)
                return MLSTM_ERR_SHAPE;
        }
        if (v[i].out) {
            if (!disjoint_rows(v[i])) return MLSTM_ERR_ALIAS;
            x->output(r);
        } else {
            x->input(r);
        }
    }
    return MLSTM_OK;
}

}  // namespace

extern "C" {

mlstm_status_t mlstm_linattn_fwd_workspace_size(int B, int H, int T, int d_qk, int d_v,
                                                mlstm_dtype_t io, size_t *bytes) {
    if (!bytes) return MLSTM_ERR_NULL;
    size_t cells;
    const mlstm_status_t st = lin_dims(B, H, T, d_qk, d_v, io, &cells);
    if (st != MLSTM_OK) return st;
    *bytes = 4 * linattn_workspace_floats(B, H, T, d_qk, d_v, io == MLSTM_BF16, 0);
    return MLSTM_OK;
}

mlstm_status_t mlstm_linattn_fwd(const void *q, const void *k, const void *v,
                                 const float *log_decay, const float *S0, const int *lengths,
                                 void *o, float *S_T, const mlstm_strides_t *strides, float scale,
                                 int B, int H, int T, int d_qk, int d_v, mlstm_dtype_t io,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    if (!q || !k || !v || !log_decay || !o) return MLSTM_ERR_NULL;
    size_t cells;
    mlstm_status_t st = lin_dims(B, H, T, d_qk, d_v, io, &cells);
    if (st != MLSTM_OK) return st;
    if (!all_aligned({q, k, v, log_decay, S0, lengths, o, S_T, workspace})) return MLSTM_ERR_ALIGN;
    const Strides nk = dense(H, T, d_qk), nv = dense(H, T, d_v);
    View w[4] = {{q, pick(strides, 0, nk, B, H, T), B, H, T, d_qk, false},
                 {k, pick(strides, 1, nk, B, H, T), B, H, T, d_qk, false},
                 {v, pick(strides, 2, nv, B, H, T), B, H, T, d_v, false},
                 {o, pick(strides, 3, nv, B, H, T), B, H, T, d_v, true}};
    Extents x;
    if ((st = lin_views(w, 4, io, true, &x)) != MLSTM_OK) return st;
    const size_t state = cells * d_qk * d_v * 4;
    x.input(rng(log_decay, (size_t)H * 4));
    x.input(rng(S0, state));
    x.input(rng(lengths, (size_t)B * 4));
    x.output(rng(S_T, state));
    const size_t need = 4 * linattn_workspace_floats(B, H, T, d_qk, d_v, io == MLSTM_BF16, 0);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MLSTM_ERR_WORKSPACE;
    if (need > 0) x.output(rng(workspace, need));
    if (!x.ok(1, 4)) return MLSTM_ERR_ALIAS;

    LinArgs a{};
    a.job[0] = LinJob{q, k, v, o, w[0].st, w[1].st, w[2].st, w[3].st, S0, S_T, d_v, 1, d_qk, d_v,
                      scale, scale, 1.0f, 0, 0};
    a.njob = 1;
    a.g = log_decay; a.lengths = lengths;
    a.B = B; a.H = H; a.T = T;
    a.ws = static_cast<float *>(workspace);
    const hipError_t e = launch_linattn(a, io == MLSTM_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLSTM_OK : MLSTM_ERR_HIP;
}

mlstm_status_t mlstm_linattn_step(const void *q, const void *k, const void *v,
                                  const float *log_decay, const float *S_in, void *o, float *S_out,
                                  const mlstm_strides_t *strides, float scale, int B, int H,
                                  int d_qk, int d_v, mlstm_dtype_t io, void *stream) {
    if (!q || !k || !v || !log_decay || !o || !S_out) return MLSTM_ERR_NULL;
    size_t cells;
    mlstm_status_t st = lin_dims(B, H, 1, d_qk, d_v, io, &cells);
    if (st != MLSTM_OK) return st;
    if (!all_aligned({q, k, v, log_decay, S_in, o, S_out})) return MLSTM_ERR_ALIGN;
    const Strides nk = dense(H, 1, d_qk), nv = dense(H, 1, d_v);
    View w[4] = {{q, pick(strides, 0, nk, B, H, 1), B, H, 1, d_qk, false},
                 {k, pick(strides, 1, nk, B, H, 1), B, H, 1, d_qk, false},
                 {v, pick(strides, 2, nv, B, H, 1), B, H, 1, d_v, false},
                 {o, pick(strides, 3, nv, B, H, 1), B, H, 1, d_v, true}};
    Extents x;
    if ((st = lin_views(w, 4, io, false, &x)) != MLSTM_OK) return st;
    const size_t state = cells * d_qk * d_v * 4;
    x.input(rng(log_decay, (size_t)H * 4));
    x.input(rng(S_in, state));
    x.output(rng(S_out, state));
    if (!x.ok(1, 4)) return MLSTM_ERR_ALIAS;

    LinStepArgs a{q, k, v, log_decay, S_in, o, S_out, w[0].st, w[1].st, w[2].st, w[3].st, scale, B, H, d_qk, d_v};
    const hipError_t e = launch_linattn_step(a, io == MLSTM_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLSTM_OK : MLSTM_ERR_HIP;
}

mlstm_status_t mlstm_linattn_bwd_workspace_size(int B, int H, int T, int d_qk, int d_v,
                                                mlstm_dtype_t io, size_t *bytes) {
    if (!bytes) return MLSTM_ERR_NULL;
    size_t cells;
    const mlstm_status_t st = lin_dims(B, H, T, d_qk, d_v, io, &cells);
    if (st != MLSTM_OK) return st;
    *bytes = 4 * linattn_workspace_floats(B, H, T, d_qk, d_v, io == MLSTM_BF16, 1);
    return MLSTM_OK;
}

mlstm_status_t mlstm_linattn_bwd(const void *q, const void *k, const void *v,
                                 const float *log_decay, const float *S0, const int *lengths,
                                 const void *d_o, const float *dS_T, void *dq, void *dk, void *dv,
                                 float *dS0, const mlstm_strides_t *strides, float scale, int B,
                                 int H, int T, int d_qk, int d_v, mlstm_dtype_t io,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    if (!q || !k || !v || !log_decay || !d_o || !dq || !dk || !dv) return MLSTM_ERR_NULL;
    size_t cells;
    mlstm_status_t st = lin_dims(B, H, T, d_qk, d_v, io, &cells);
    if (st != MLSTM_OK) return st;
    if (!all_aligned({q, k, v, log_decay, S0, lengths, d_o, dS_T, dq, dk, dv, dS0, workspace}))
        return MLSTM_ERR_ALIGN;
    const Strides nk = dense(H, T, d_qk), nv = dense(H, T, d_v);
    View w[7] = {{q, pick(strides, 0, nk, B, H, T), B, H, T, d_qk, false},
                 {k, pick(strides, 1, nk, B, H, T), B, H, T, d_qk, false},
                 {v, pick(strides, 2, nv, B, H, T), B, H, T, d_v, false},
                 {d_o, pick(strides, 3, nv, B, H, T), B, H, T, d_v, false},
                 {dq, pick(strides, 4, nk, B, H, T), B, H, T, d_qk, true},
                 {dk, pick(strides, 5, nk, B, H, T), B, H, T, d_qk, true},
                 {dv, pick(strides, 6, nv, B, H, T), B, H, T, d_v, true}};
    Extents x;
    if ((st = lin_views(w, 7, io, true, &x)) != MLSTM_OK) return st;
    const size_t state = cells * d_qk * d_v * 4;
    x.input(rng(log_decay, (size_t)H * 4));
    x.input(rng(S0, state));
    x.input(rng(dS_T, state));
    x.input(rng(lengths, (size_t)B * 4));
    x.output(rng(dS0, state));
    const size_t need = 4 * linattn_workspace_floats(B, H, T, d_qk, d_v, io == MLSTM_BF16, 1);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MLSTM_ERR_WORKSPACE;
    if (need > 0) x.output(rng(workspace, need));
    if (!x.ok(-1, -1)) return MLSTM_ERR_ALIAS;

    LinArgs a{};
    // dq_t = s S_t do_t: the forward's states, read by their value index
    a.job[0] = LinJob{d_o, v, k, dq, w[3].st, w[2].st, w[1].st, w[4].st, S0, nullptr, 1, d_v, d_v, d_qk,
                      scale, scale, 1.0f, 0, 0};
    // dv_t = D_t^T k_t with D_t = e^g D_{t+1} + s q_t do_t^T, from the last token back
    a.job[1] = LinJob{k, q, d_o, dv, w[1].st, w[0].st, w[3].st, w[6].st, dS_T, dS0, d_v, 1, d_qk, d_v,
                      scale, 1.0f, scale, 1, 1};
    // dk_t = D_t v_t
    a.job[2] = LinJob{v, d_o, q, dk, w[2].st, w[3].st, w[0].st, w[5].st, dS_T, nullptr, 1, d_v, d_v, d_qk,
                      scale, 1.0f, scale, 1, 1};
    a.njob = 3;
    a.g = log_decay; a.lengths = lengths;
    a.B = B; a.H = H; a.T = T;
    a.ws = static_cast<float *>(workspace);
    const hipError_t e = launch_linattn(a, io == MLSTM_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLSTM_OK : MLSTM_ERR_HIP;
}

// ---- gated delta rule

namespace {

// Shapes of a delta rule call; *need = workspace bytes of one over sequences.
mlstm_status_t delta_dims(int B, int Hk, int H, int T, int dk, int dv, mlstm_dtype_t io, int backward,
                          size_t *cells, size_t *need) {
    if (Hk <= 0) return MLSTM_ERR_SHAPE;
    const mlstm_status_t st = lin_dims(B, H, T, dk, dv, io, cells);
    if (st != MLSTM_OK) return st;
    if (H % Hk) return MLSTM_ERR_SHAPE;
    if (need) {
        // 2^40 bytes.  A 32-token chunk of a head has at least one KB and below 2^24 bytes of it, so
        // the sizes of what passes here do not overflow.
        if (*cells * (((size_t)T + 31) / 32) > (size_t)1 << 30) return MLSTM_ERR_SHAPE;
        const size_t f = deltarule_workspace_floats(B, H, T, dk, dv, io == MLSTM_BF16, backward);
        if (f > ((size_t)1 << 38)) return MLSTM_ERR_SHAPE;
        *need = 4 * f;
    }
    return MLSTM_OK;
}

// A gate of one float for each (b, h, t): any strides, 4-byte alignment.
mlstm_status_t gate_view(const View &v, Extents *x) {
    Range r;
    if (!extent(v, 4, &r)) return MLSTM_ERR_SHAPE;
    if ((uintptr_t)v.p & 3) return MLSTM_ERR_ALIGN;
    if (v.out) {
        if (!disjoint_rows(v)) return MLSTM_ERR_ALIAS;
        x->output(r);
    } else {
        x->input(r);
    }
    return MLSTM_OK;
}

}  // namespace

mlstm_status_t mlstm_deltarule_fwd_workspace_size(int B, int Hk, int H, int T, int d_qk, int d_v,
                                                  mlstm_dtype_t io, size_t *bytes) {
    if (!bytes) return MLSTM_ERR_NULL;
    size_t cells;
    return delta_dims(B, Hk, H, T, d_qk, d_v, io, 0, &cells, bytes);
}

mlstm_status_t mlstm_deltarule_fwd(const void *q, const void *k, const void *v,
                                   const float *log_decay, const float *beta, const float *S0,
                                   const int *lengths, void *o, float *S_T,
                                   const mlstm_strides_t *strides, float scale, int B, int Hk, int H,
                                   int T, int d_qk, int d_v, mlstm_dtype_t io, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    if (!q || !k || !v || !log_decay || !beta || !o) return MLSTM_ERR_NULL;
    size_t cells, need;
    mlstm_status_t st = delta_dims(B, Hk, H, T, d_qk, d_v, io, 0, &cells, &need);
    if (st != MLSTM_OK) return st;
    if (!all_aligned({q, k, v, S0, lengths, o, S_T, workspace})) return MLSTM_ERR_ALIGN;
    const Strides nk = dense(Hk, T, d_qk), nv = dense(H, T, d_v), ng = dense(H, T, 1);
    View w[4] = {{q, pick(strides, 0, nk, B, Hk, T), B, Hk, T, d_qk, false},
                 {k, pick(strides, 1, nk, B, Hk, T), B, Hk, T, d_qk, false},
                 {v, pick(strides, 2, nv, B, H, T), B, H, T, d_v, false},
                 {o, pick(strides, 5, nv, B, H, T), B, H, T, d_v, true}};
    const View gates[2] = {{log_decay, pick(strides, 3, ng, B, H, T), B, H, T, 1, false},
                           {beta, pick(strides, 4, ng, B, H, T), B, H, T, 1, false}};
    Extents x;
    x.input(rng(S0, cells * d_qk * d_v * 4));
    if ((st = lin_views(w, 4, io, true, &x)) != MLSTM_OK) return st;
    for (const View &v1 : gates)
        if ((st = gate_view(v1, &x)) != MLSTM_OK) return st;
    x.input(rng(lengths, (size_t)B * 4));
    x.output(rng(S_T, cells * d_qk * d_v * 4));
    if (need > 0 && (!workspace || workspace_bytes < need)) return MLSTM_ERR_WORKSPACE;
    if (need > 0) x.output(rng(workspace, need));
    if (!x.ok(1, 0)) return MLSTM_ERR_ALIAS;

    DeltaArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = log_decay; a.beta = beta; a.S0 = S0; a.lengths = lengths;
    a.o = o; a.S_T = S_T;
    a.sq = w[0].st; a.sk = w[1].st; a.sv = w[2].st; a.so = w[3].st;
    a.sg = gates[0].st; a.sb = gates[1].st;
    a.scale = scale;
    a.B = B; a.Hk = Hk; a.H = H; a.T = T; a.dk = d_qk; a.dv = d_v;
    a.ws = static_cast<float *>(workspace);
    const hipError_t e = launch_deltarule_fwd(a, io == MLSTM_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLSTM_OK : MLSTM_ERR_HIP;
}

mlstm_status_t mlstm_deltarule_step(const void *q, const void *k, const void *v,
                                    const float *log_decay, const float *beta, const float *S_in,
                                    void *o, float *S_out, const mlstm_strides_t *strides,
                                    float scale, int B, int Hk, int H, int d_qk, int d_v,
                                    mlstm_dtype_t io, void *stream) {
    if (!q || !k || !v || !log_decay || !beta || !o || !S_out) return MLSTM_ERR_NULL;
    size_t cells;
    mlstm_status_t st = delta_dims(B, Hk, H, 1, d_qk, d_v, io, 0, &cells, nullptr);
    if (st != MLSTM_OK) return st;
    if (!all_aligned({q, k, v, S_in, o, S_out})) return MLSTM_ERR_ALIGN;
    const Strides nk = dense(Hk, 1, d_qk), nv = dense(H, 1, d_v), ng = dense(H, 1, 1);
    View w[4] = {{q, pick(strides, 0, nk, B, Hk, 1), B, Hk, 1, d_qk, false},
                 {k, pick(strides, 1, nk, B, Hk, 1), B, Hk, 1, d_qk, false},
                 {v, pick(strides, 2, nv, B, H, 1), B, H, 1, d_v, false},
                 {o, pick(strides, 5, nv, B, H, 1), B, H, 1, d_v, true}};
    const View gates[2] = {{log_decay, pick(strides, 3, ng, B, H, 1), B, H, 1, 1, false},
                           {beta, pick(strides, 4, ng, B, H, 1), B, H, 1, 1, false}};
    Extents x;
    x.input(rng(S_in, cells * d_qk * d_v * 4));
    if ((st = lin_views(w, 4, io, false, &x)) != MLSTM_OK) return st;
    for (const View &v1 : gates)
        if ((st = gate_view(v1, &x)) != MLSTM_OK) return st;
    x.output(rng(S_out, cells * d_qk * d_v * 4));
    if (!x.ok(1, 0)) return MLSTM_ERR_ALIAS;

    const DeltaStepArgs a{q, k, v, log_decay, beta, S_in, o, S_out, w[0].st, w[1].st, w[2].st, gates[0].st,
                          gates[1].st, w[3].st, scale, B, Hk, H, d_qk, d_v};
    const hipError_t e = launch_deltarule_step(a, io == MLSTM_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLSTM_OK : MLSTM_ERR_HIP;
}

mlstm_status_t mlstm_deltarule_bwd_workspace_size(int B, int Hk, int H, int T, int d_qk, int d_v,
                                                  mlstm_dtype_t io, size_t *bytes) {
    if (!bytes) return MLSTM_ERR_NULL;
    size_t cells;
    return delta_dims(B, Hk, H, T, d_qk, d_v, io, 1, &cells, bytes);
}

mlstm_status_t mlstm_deltarule_bwd(const void *q, const void *k, const void *v,
                                   const float *log_decay, const float *beta, const float *S0,
                                   const int *lengths, const void *d_o, const float *dS_T, void *dq,
                                   void *dk, void *dv, float *dlog_decay, float *dbeta, float *dS0,
                                   const mlstm_strides_t *strides, float scale, int B, int Hk, int H,
                                   int T, int d_qk, int d_v, mlstm_dtype_t io, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    if (!q || !k || !v || !log_decay || !beta || !d_o || !dq || !dk || !dv || !dlog_decay || !dbeta)
        return MLSTM_ERR_NULL;
    size_t cells, need;
    mlstm_status_t st = delta_dims(B, Hk, H, T, d_qk, d_v, io, 1, &cells, &need);
    if (st != MLSTM_OK) return st;
    if (!all_aligned({q, k, v, S0, lengths, d_o, dS_T, dq, dk, dv, dS0, workspace})) return MLSTM_ERR_ALIGN;
    const Strides nk = dense(Hk, T, d_qk), nv = dense(H, T, d_v), ng = dense(H, T, 1);
    View w[7] = {{q, pick(strides, 0, nk, B, Hk, T), B, Hk, T, d_qk, false},
                 {k, pick(strides, 1, nk, B, Hk, T), B, Hk, T, d_qk, false},
                 {v, pick(strides, 2, nv, B, H, T), B, H, T, d_v, false},
                 {d_o, pick(strides, 5, nv, B, H, T), B, H, T, d_v, false},
                 {dq, pick(strides, 6, nk, B, Hk, T), B, Hk, T, d_qk, true},
                 {dk, pick(strides, 7, nk, B, Hk, T), B, Hk, T, d_qk, true},
                 {dv, pick(strides, 8, nv, B, H, T), B, H, T, d_v, true}};
    const View gates[4] = {{log_decay, pick(strides, 3, ng, B, H, T), B, H, T, 1, false},
                           {beta, pick(strides, 4, ng, B, H, T), B, H, T, 1, false},
                           {dlog_decay, pick(strides, 9, ng, B, H, T), B, H, T, 1, true},
                           {dbeta, pick(strides, 10, ng, B, H, T), B, H, T, 1, true}};
    Extents x;
    if ((st = lin_views(w, 7, io, true, &x)) != MLSTM_OK) return st;
    for (const View &v1 : gates)
        if ((st = gate_view(v1, &x)) != MLSTM_OK) return st;
    const size_t state = cells * d_qk * d_v * 4;
    x.input(rng(S0, state));
    x.input(rng(dS_T, state));
    x.input(rng(lengths, (size_t)B * 4));
    x.output(rng(dS0, state));
    if (need > 0 && (!workspace || workspace_bytes < need)) return MLSTM_ERR_WORKSPACE;
    if (need > 0) x.output(rng(workspace, need));
    if (!x.ok(-1, -1)) return MLSTM_ERR_ALIAS;

    DeltaArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = log_decay; a.beta = beta; a.S0 = S0; a.lengths = lengths;
    a.d_o = d_o; a.dS_T = dS_T; a.dq = dq; a.dkk = dk; a.dvv = dv;
    a.dg = dlog_decay; a.db = dbeta; a.dS0 = dS0;
    a.sq = w[0].st; a.sk = w[1].st; a.sv = w[2].st; a.sdo = w[3].st;
    a.sdq = w[4].st; a.sdk = w[5].st; a.sdv = w[6].st;
    a.sg = gates[0].st; a.sb = gates[1].st; a.sdg = gates[2].st; a.sdb = gates[3].st;
    a.scale = scale;
    a.B = B; a.Hk = Hk; a.H = H; a.T = T; a.dk = d_qk; a.dv = d_v;
    a.ws = static_cast<float *>(workspace);
    const hipError_t e = launch_deltarule_bwd(a, io == MLSTM_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLSTM_OK : MLSTM_ERR_HIP;
}

// ---- norm and rotation of queries and keys

namespace {

mlstm_status_t qk_dims(int B, int H, int Hk, bool keys, int T, int d) {
    if (B <= 0 || H <= 0 || (keys && Hk <= 0) || T <= 0 || d <= 0) return MLSTM_ERR_SHAPE;
    if (d > 512) return MLSTM_ERR_UNSUPPORTED;
    size_t n;
    if (!mul_ok((size_t)B, (size_t)T, &n) || !mul_ok(n, (size_t)H + (keys ? (size_t)Hk : 0), &n) || n > (size_t)INT32_MAX)
        return MLSTM_ERR_SHAPE;
    return MLSTM_OK;
}

// Two tensors that interleave in one buffer without meeting, as the queries and keys
// of a fused projection do: with equal strides, the inner dimensions of one lie
// whole between those of the other.
bool interleaved(const View &x, const View &y, size_t es) {
    const View &a = (uintptr_t)x.p <= (uintptr_t)y.p ? x : y, &b = (uintptr_t)x.p <= (uintptr_t)y.p ? y : x;
    const size_t bytes = (uintptr_t)b.p - (uintptr_t)a.p;
    if (bytes % es || bytes / es > ((size_t)1 << 60)) return false;
    const long long delta = (long long)(bytes / es);
    const long long sa[3] = {a.st.s0, a.st.s1, a.st.s2}, sb[3] = {b.st.s0, b.st.s1, b.st.s2};
    const int na[3] = {a.n0, a.n1, a.n2}, nb[3] = {b.n0, b.n1, b.n2};
    long long st[3];
    int dim[3], n = 0;
    for (int i = 0; i < 3; ++i) {
        if (na[i] > 1 && nb[i] > 1 && sa[i] != sb[i]) return false;
        st[i] = na[i] > 1 ? sa[i] : sb[i];
        if (na[i] > 1 || nb[i] > 1) dim[n++] = i;
    }
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if (st[dim[j]] < st[dim[i]]) {
                const int t = dim[i];
                dim[i] = dim[j];
                dim[j] = t;
            }
    // inner dimensions 0 .. m - 1 of both, side by side within one step of dimension m
    long long span_a = a.d, span_b = b.d;
    for (int m = 0;; ++m) {
        if (delta >= span_a && (m == n || delta + span_b <= st[dim[m]])) {
            // ... and the steps of the outer ones are apart from one another
            long long reach = m == n ? 0 : st[dim[m]];
            for (int j = m; j < n; ++j) {
                if (st[dim[j]] < reach) return false;
                reach += st[dim[j]] * (std::max(na[dim[j]], nb[dim[j]]) - 1);
            }
            return true;
        }
        if (m == n) return false;
        span_a += st[dim[m]] * (na[dim[m]] - 1);
        span_b += st[dim[m]] * (nb[dim[m]] - 1);
    }
}

mlstm_status_t qk_call(QkArgs &a, const mlstm_strides_t *strides, int layout, int norm, mlstm_dtype_t io,
                       void *workspace, size_t workspace_bytes, void *stream) {
    const int B = a.B, T = a.T, d = a.d;
    const bool bwd = a.dy[0] != nullptr, keys = a.x[1] != nullptr;
    if (!keys) a.H[1] = 0;
    const mlstm_status_t st = qk_dims(B, a.H[0], a.H[1], keys, T, d);
    if (st != MLSTM_OK) return st;
    if (io != MLSTM_F32 && io != MLSTM_BF16) return MLSTM_ERR_UNSUPPORTED;
    if (layout != MLSTM_ROTARY_HALF && layout != MLSTM_ROTARY_PAIRS) return MLSTM_ERR_UNSUPPORTED;
    if (norm != MLSTM_QKNORM_NONE && norm != MLSTM_QKNORM_RMS && norm != MLSTM_QKNORM_L2) return MLSTM_ERR_UNSUPPORTED;
    if (!(a.eps >= 0.0f)) return MLSTM_ERR_UNSUPPORTED;
    if (a.nf < 0 || a.nf > d / 2) return MLSTM_ERR_SHAPE;
    if (a.nf > 0 && !a.freq) return MLSTM_ERR_NULL;
    const size_t es = io == MLSTM_BF16 ? 2 : 4;
    // element alignment suffices for rows; the tables are float32 and int32
    for (const void *p : {a.x[0], a.x[1], a.dy[0], a.dy[1], (const void *)a.y[0], (const void *)a.y[1]})
        if ((uintptr_t)p % es) return MLSTM_ERR_ALIGN;
    if (!all_aligned({a.w[0], a.w[1], a.dw[0], a.dw[1], a.freq, a.pos, workspace})) return MLSTM_ERR_ALIGN;
    Range in[2][2] = {}, out[2] = {}, dense_in[4], dense_out[3];
    View views[3][2] = {};
    int at = 0;
    for (int role = 0; role < 3; ++role)  // x, dy, y
        for (int i = 0; i < 2; ++i) {
            if (role == 1 && !bwd) continue;
            const int n = a.H[i];
            Strides &s = role == 0 ? a.sx[i] : role == 1 ? a.sdy[i] : a.sy[i];
            Range &r = role == 2 ? out[i] : in[role][i];
            const void *p = role == 0 ? a.x[i] : role == 1 ? a.dy[i] : a.y[i];
            r = Range{0, 0};
            if (n > 0) {
                s = pick(strides, at, dense(n, T, d), B, n, T);
                const View v{p, s, B, n, T, d, role == 2};
                views[role][i] = v;
                if (!extent(v, es, &r)) return MLSTM_ERR_SHAPE;
                if (role == 2 && !disjoint_rows(v)) return MLSTM_ERR_ALIAS;
            }
            ++at;
        }
    const size_t par = (size_t)d * 4;
    dense_in[0] = rng(a.w[0], par);
    dense_in[1] = rng(a.w[1], par);
    dense_in[2] = rng(a.freq, (size_t)a.nf * 4);
    dense_in[3] = rng(a.nf > 0 ? a.pos : nullptr, (size_t)B * T * 4);
    dense_out[0] = rng(a.dw[0], par);
    dense_out[1] = rng(a.dw[1], par);
    const size_t need = a.dw[0] || a.dw[1] ? 4 * qknorm_workspace_floats(B, a.H[0], a.H[1], T, d) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return MLSTM_ERR_WORKSPACE;
    dense_out[2] = need > 0 ? rng(workspace, need) : Range{0, 0};
    const auto eq = [](const Strides &x, const Strides &y) { return x.s0 == y.s0 && x.s1 == y.s1 && x.s2 == y.s2; };
    for (int i = 0; i < 2; ++i) {
        for (int j = 0; j < 2; ++j) {
            // a row is read whole before it is written: y over its own x (dx over its own dy)
            const bool own_x = i == j && !bwd && a.y[i] == a.x[i] && eq(a.sy[i], a.sx[i]);
            const bool own_dy = i == j && bwd && a.y[i] == a.dy[i] && eq(a.sy[i], a.sdy[i]);
            if (overlaps(out[i], in[0][j]) && !own_x && !interleaved(views[2][i], views[0][j], es)) return MLSTM_ERR_ALIAS;
            if (bwd && overlaps(out[i], in[1][j]) && !own_dy && !interleaved(views[2][i], views[1][j], es))
                return MLSTM_ERR_ALIAS;
        }
        for (const Range &r : dense_in)
            if (overlaps(out[i], r)) return MLSTM_ERR_ALIAS;
        for (const Range &r : dense_out)
            if (overlaps(out[i], r)) return MLSTM_ERR_ALIAS;
    }
    if (overlaps(out[0], out[1]) && !interleaved(views[2][0], views[2][1], es)) return MLSTM_ERR_ALIAS;
    for (int i = 0; i < 3; ++i) {
        for (const Range &r : dense_in)
            if (overlaps(dense_out[i], r)) return MLSTM_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(dense_out[i], dense_out[j])) return MLSTM_ERR_ALIAS;
        for (int j = 0; j < 2; ++j)
            if (overlaps(dense_out[i], in[0][j]) || (bwd && overlaps(dense_out[i], in[1][j]))) return MLSTM_ERR_ALIAS;
    }
    a.pairs = layout == MLSTM_ROTARY_PAIRS;
    a.norm = norm;
    a.ws = static_cast<float *>(workspace);
    const hipError_t e = launch_qknorm(a, io == MLSTM_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MLSTM_OK : MLSTM_ERR_HIP;
}

}  // namespace

mlstm_status_t mlstm_qknorm_fwd(const void *q, const void *k, const float *q_weight,
                                const float *k_weight, const float *inv_freq,
                                const int *positions, void *yq, void *yk,
                                const mlstm_strides_t *strides, int B, int H, int Hk, int T, int d,
                                int n_freq, mlstm_rotary_t layout, float amplitude,
                                mlstm_qknorm_t norm, float eps, mlstm_dtype_t io, void *stream) {
    if (!q || !yq || (k == nullptr) != (yk == nullptr)) return MLSTM_ERR_NULL;
    QkArgs a{};
    a.x[0] = q; a.x[1] = k; a.y[0] = yq; a.y[1] = yk;
    a.w[0] = q_weight; a.w[1] = k ? k_weight : nullptr;
    a.freq = inv_freq; a.pos = positions;
    a.B = B; a.T = T; a.H[0] = H; a.H[1] = Hk; a.d = d; a.nf = n_freq;
    a.amp = amplitude; a.eps = eps;
    return qk_call(a, strides, layout, norm, io, nullptr, 0, stream);
}

mlstm_status_t mlstm_qknorm_bwd_workspace_size(int B, int H, int Hk, int T, int d, size_t *bytes) {
    if (!bytes) return MLSTM_ERR_NULL;
    const mlstm_status_t st = qk_dims(B, H, Hk, Hk != 0, T, d);
    if (st != MLSTM_OK) return st;
    *bytes = 4 * qknorm_workspace_floats(B, H, Hk, T, d);
    return MLSTM_OK;
}

mlstm_status_t mlstm_qknorm_bwd(const void *q, const void *k, const void *dyq, const void *dyk,
                                const float *q_weight, const float *k_weight, const float *inv_freq,
                                const int *positions, void *dq, void *dk, float *dq_weight,
                                float *dk_weight, const mlstm_strides_t *strides, int B, int H,
                                int Hk, int T, int d, int n_freq, mlstm_rotary_t layout,
                                float amplitude, mlstm_qknorm_t norm, float eps, mlstm_dtype_t io,
                                void *workspace, size_t workspace_bytes, void *stream) {
    if (!q || !dyq || !dq || (k == nullptr) != (dyk == nullptr) || (k == nullptr) != (dk == nullptr))
        return MLSTM_ERR_NULL;
    QkArgs a{};
    a.x[0] = q; a.x[1] = k; a.dy[0] = dyq; a.dy[1] = dyk; a.y[0] = dq; a.y[1] = dk;
    a.w[0] = q_weight; a.w[1] = k ? k_weight : nullptr;
    a.dw[0] = dq_weight; a.dw[1] = k ? dk_weight : nullptr;
    a.freq = inv_freq; a.pos = positions;
    a.B = B; a.T = T; a.H[0] = H; a.H[1] = Hk; a.d = d; a.nf = n_freq;
    a.amp = amplitude; a.eps = eps;
    return qk_call(a, strides, layout, norm, io, workspace, workspace_bytes, stream);
}

mlstm_status_t mlstm_rope_frequencies(int n_freq, double base, mlstm_rope_scaling_t scaling,
                                      double factor, int context, double fast, double slow,
                                      float *inv_freq, float *amplitude) {
    if (!inv_freq || !amplitude) return MLSTM_ERR_NULL;
    if (n_freq <= 0 || !(base > 1.0) || !(factor >= 1.0) || isinf(base) || isinf(factor)) return MLSTM_ERR_SHAPE;
    const double turn = 6.283185307179586476925286766559;
    double lo = 0.0, hi = 0.0, amp = 1.0;
    switch (scaling) {
        case MLSTM_ROPE_PLAIN:
        case MLSTM_ROPE_LINEAR:
            break;
        case MLSTM_ROPE_BASE:
            if (n_freq < 2) return MLSTM_ERR_SHAPE;
            // the last exponent is -(n - 1) / n: this divides its frequency by the factor
            base *= pow(factor, (double)n_freq / (n_freq - 1));
            break;
        case MLSTM_ROPE_RAMP: {
            if (context < 1 || !(slow > 0.0) || !(fast > slow) || isinf(fast)) return MLSTM_ERR_SHAPE;
            // pair index at which the context holds so many turns: context f_i / turn = turns
            const auto index = [&](double turns) { return n_freq * log(context / (turn * turns)) / log(base); };
            lo = index(fast);
            hi = index(slow);
            amp = 0.1 * log(factor) + 1.0;
            break;
        }
        default:
            return MLSTM_ERR_UNSUPPORTED;
    }
    for (int i = 0; i < n_freq; ++i) {
        double f = pow(base, -(double)i / n_freq);
        if (scaling == MLSTM_ROPE_LINEAR) f /= factor;
        if (scaling == MLSTM_ROPE_RAMP) {
            const double r = fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0);  // 0: kept, 1: divided
            f = f * (1.0 - r) + f / factor * r;
        }
        inv_freq[i] = (float)f;
    }
    *amplitude = (float)amp;
    return MLSTM_OK;
}

// ---- group norm

static mlstm_status_t gn_dims(int N, int S, int G, int D, mlstm_norm_over_t over, mlstm_dtype_t io) {
    if (N <= 0 || S <= 0 || G <= 0 || D <= 0) return MLSTM_ERR_SHAPE;
    if (io != MLSTM_F32 && io != MLSTM_BF16) return MLSTM_ERR_UNSUPPORTED;
    if (over != MLSTM_NORM_TOKEN && over != MLSTM_NORM_SEQUENCE) return MLSTM_ERR_UNSUPPORTED;
    // positions, channels and samples x groups are counted in 32 bits, and so are
    // workgroups of at least 16 channels of a sample, four for each 64
    size_t n;
    if (!mul_ok((size_t)G, (size_t)D, &n) || n > (size_t)INT32_MAX / 2) return MLSTM_ERR_SHAPE;
    if (!mul_ok((size_t)N, (size_t)S, &n) || n > (size_t)INT32_MAX / 2) return MLSTM_ERR_SHAPE;
    if (!mul_ok((size_t)N, (size_t)G, &n) || n > (size_t)INT32_MAX / 2) return MLSTM_ERR_SHAPE;
    if (!mul_ok((size_t)N, ((size_t)G * D + 63) / 64, &n) || n > (size_t)INT32_MAX / 8) return MLSTM_ERR_SHAPE;
    return MLSTM_OK;
}

static mlstm_status_t gn_call(GnArgs &a, const mlstm_strides_t *strides, mlstm_norm_over_t over, mlstm_act_t act,
                       mlstm_dtype_t io, void *workspace, size_t workspace_bytes, void *stream) {
    const int N = a.N, S = a.S, G = a.G, D = a.D;
    const mlstm_status_t st = gn_dims(N, S, G, D, over, io);
    if (st != MLSTM_OK) return st;
    if (act != MLSTM_ACT_NONE && act != MLSTM_ACT_SILU && act != MLSTM_ACT_GELU) return MLSTM_ERR_UNSUPPORTED;
    if (!a.dy && !(a.eps > 0.0f)) return MLSTM_ERR_UNSUPPORTED;
    if (!all_aligned({a.x, a.dy, a.w, a.b, a.mean, a.rstd, a.y, a.dw, a.db, workspace})) return MLSTM_ERR_ALIGN;
    const bool bwd = a.dy != nullptr;
    const size_t es = io == MLSTM_BF16 ? 2 : 4;
    const Strides nd = dense(S, G, D);
    a.sx = pick(strides, 0, nd, N, S, G);
    if (bwd) a.sdy = pick(strides, 1, nd, N, S, G);
    a.sy = pick(strides, bwd ? 2 : 1, nd, N, S, G);
    Extents e;
    Range r;
    if (!extent(View{a.x, a.sx, N, S, G, D, false}, es, &r)) return MLSTM_ERR_SHAPE;
    e.input(r);
    if (bwd) {
        if (!extent(View{a.dy, a.sdy, N, S, G, D, false}, es, &r)) return MLSTM_ERR_SHAPE;
        e.input(r);
    }
    const View y{a.y, a.sy, N, S, G, D, true};
    if (!extent(y, es, &r)) return MLSTM_ERR_SHAPE;
    if (!disjoint_rows(y)) return MLSTM_ERR_ALIAS;
    e.output(r);
    const size_t par = (size_t)G * D * 4, stat = (size_t)N * G * 4 * (over == MLSTM_NORM_TOKEN ? (size_t)S : 1);
    e.input(rng(a.w, par));
    e.input(rng(a.b, par));
    if (bwd) {
        e.input(rng(a.mean, stat));
        e.input(rng(a.rstd, stat));
        e.output(rng(a.dw, par));
        e.output(rng(a.db, par));
    } else {
        e.output(rng(a.mean, stat));
        e.output(rng(a.rstd, stat));
    }
    a.seq = over == MLSTM_NORM_SEQUENCE;
    a.act = act;
    const size_t need = 4 * groupnorm_workspace_floats(N, S, G, D, a.seq, io == MLSTM_BF16, bwd);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MLSTM_ERR_WORKSPACE;
    if (need > 0) e.output(rng(workspace, need));
    if (!e.ok(-1, -1)) return MLSTM_ERR_ALIAS;
    a.ws = static_cast<float *>(workspace);
    const hipError_t err = launch_groupnorm(a, io == MLSTM_BF16, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? MLSTM_OK : MLSTM_ERR_HIP;
}

mlstm_status_t mlstm_groupnorm_workspace_size(int N, int S, int G, int D, mlstm_norm_over_t over,
                                              mlstm_dtype_t io, int backward, size_t *bytes) {
    if (!bytes) return MLSTM_ERR_NULL;
    const mlstm_status_t st = gn_dims(N, S, G, D, over, io);
    if (st != MLSTM_OK) return st;
    *bytes = 4 * groupnorm_workspace_floats(N, S, G, D, over == MLSTM_NORM_SEQUENCE, io == MLSTM_BF16, backward != 0);
    return MLSTM_OK;
}

mlstm_status_t mlstm_groupnorm_fwd(const void *x, const float *weight, const float *bias, void *y,
                                   float *mean, float *rstd, const mlstm_strides_t *strides, int N,
                                   int S, int G, int D, mlstm_norm_over_t over, mlstm_act_t act,
                                   float eps, mlstm_dtype_t io, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    if (!x || !y || (mean == nullptr) != (rstd == nullptr)) return MLSTM_ERR_NULL;
    GnArgs a{};
    a.x = x; a.w = weight; a.b = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    a.N = N; a.S = S; a.G = G; a.D = D; a.eps = eps;
    return gn_call(a, strides, over, act, io, workspace, workspace_bytes, stream);
}

mlstm_status_t mlstm_groupnorm_bwd(const void *x, const void *dy, const float *mean,
                                   const float *rstd, const float *weight, const float *bias,
                                   void *dx, float *dweight, float *dbias,
                                   const mlstm_strides_t *strides, int N, int S, int G, int D,
                                   mlstm_norm_over_t over, mlstm_act_t act, mlstm_dtype_t io,
                                   void *workspace, size_t workspace_bytes, void *stream) {
    if (!x || !dy || !mean || !rstd || !dx) return MLSTM_ERR_NULL;
    GnArgs a{};
    a.x = x; a.dy = dy; a.w = weight; a.b = bias; a.y = dx;
    a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    a.dw = dweight; a.db = dbias;
    a.N = N; a.S = S; a.G = G; a.D = D;
    return gn_call(a, strides, over, act, io, workspace, workspace_bytes, stream);
}

}  // extern "C"
