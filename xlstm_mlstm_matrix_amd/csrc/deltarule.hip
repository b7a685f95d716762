// deltarule.hip -- the gated delta rule over whole sequences, token by token.
//
//   S <- e^g S;  x = v - S^T k;  u = beta x;  S <- S + k u^T;  o = scale S^T q,
// and backwards with D = dL/dS behind a token:
//   D <- D + scale q do^T;  du = D^T k;  dbeta = du . x;  dv = beta du;
//   dk = D u - (e^g S_before) dv;  dq = scale S do;  D <- e^g (D - k dv^T).
// A decay scales all later outputs and the final state, less what v adds:
//   dg_t = sum_{s >= t} (q.dq + k.dk - 2 beta dbeta)_s + <dS_T, S_T>.
#include "ops.hpp"

namespace mlstm {

namespace {

constexpr int BV = 64;  // value columns of a workgroup

__device__ __forceinline__ int tokens(const DeltaArgs &a, int b) {
    return a.lengths ? max(0, min(a.lengths[b], a.T)) : a.T;
}
__device__ __forceinline__ float decay(const DeltaArgs &a, int b, int h, long long t) {
    return __builtin_amdgcn_exp2f(decay_log2(a.g[b * a.sg.s0 + h * a.sg.s1 + t * a.sg.s2]));
}
__device__ __forceinline__ float strength(const DeltaArgs &a, int b, int h, long long t) {
    return a.beta[b * a.sb.s0 + h * a.sb.s1 + t * a.sb.s2];
}

struct Ws {
    float *x, *du, *gq, *gk, *st, *dG;
};
Ws make_ws(const DeltaArgs &a) {
    const size_t n = (size_t)a.B * a.H * a.T, c = (size_t)a.B * a.H;
    Ws w;
    w.x = a.ws;
    w.du = w.x + n * a.dv;
    w.gq = w.du + n * a.dv;
    w.gk = w.gq + n * a.dk;
    w.st = w.gk + n * a.dk;
    w.dG = w.st + c * a.dk * a.dv;
    return w;
}

// 64 columns of a head: 4 wavefronts hold 64 rows each.
template <typename IO, bool REV>
__global__ __launch_bounds__(256) void column_kernel(DeltaArgs a, Ws w) {
    __shared__ float ks[256], qs[256], red[2][4][BV];
    const int ntile = (a.dv + BV - 1) / BV;
    const int tile = blockIdx.x % ntile, bh = blockIdx.x / ntile, b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const int tid = threadIdx.x, c = tid & 63, rg = tid >> 6, col = tile * BV + c;
    const bool ok = col < a.dv;
    const int n = tokens(a, b);
    float S[64];
    const float *S0 = REV ? a.dS_T : a.S0;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
        const int r = rg * 64 + i;
        S[i] = S0 && ok && r < a.dk ? S0[((size_t)bh * a.dk + r) * a.dv + col] : 0.0f;
    }
    for (int s = 0; s < n; ++s) {
        const long long t = REV ? n - 1 - s : s;
        const IO *q = (const IO *)a.q + b * a.sq.s0 + hk * a.sq.s1 + t * a.sq.s2;
        const IO *k = (const IO *)a.k + b * a.sk.s0 + hk * a.sk.s1 + t * a.sk.s2;
        __syncthreads();
        ks[tid] = tid < a.dk ? to_f(k[tid]) : 0.0f;
        qs[tid] = tid < a.dk ? to_f(q[tid]) : 0.0f;
        const float gam = decay(a, b, h, t), beta = strength(a, b, h, t);
        const size_t row = ((size_t)bh * a.T + t) * a.dv + col;
        __syncthreads();
        float acc = 0.0f;
        if constexpr (REV) {
            const float go = ok ? a.scale * to_f(((const IO *)a.d_o)[b * a.sdo.s0 + h * a.sdo.s1 + t * a.sdo.s2 + col]) : 0.0f;
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                S[i] += qs[rg * 64 + i] * go;
                acc += ks[rg * 64 + i] * S[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                S[i] *= gam;
                acc += ks[rg * 64 + i] * S[i];
            }
        }
        red[0][rg][c] = acc;
        __syncthreads();
        acc = (red[0][0][c] + red[0][1][c]) + (red[0][2][c] + red[0][3][c]);
        if constexpr (REV) {
            const float dv = beta * acc;
            if (ok && rg == 0) {
                w.du[row] = acc;
                ((IO *)a.dvv)[b * a.sdv.s0 + h * a.sdv.s1 + t * a.sdv.s2 + col] = from_f<IO>(dv);
            }
#pragma unroll
            for (int i = 0; i < 64; ++i) S[i] = gam * (S[i] - ks[rg * 64 + i] * dv);
        } else {
            const float v = ok ? to_f(((const IO *)a.v)[b * a.sv.s0 + h * a.sv.s1 + t * a.sv.s2 + col]) : 0.0f;
            const float x = v - acc;
            float y = 0.0f;
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                S[i] += ks[rg * 64 + i] * (beta * x);
                y += qs[rg * 64 + i] * S[i];
            }
            red[1][rg][c] = y;
            if (w.x && ok && rg == 0) w.x[row] = x;
            __syncthreads();
            y = (red[1][0][c] + red[1][1][c]) + (red[1][2][c] + red[1][3][c]);
            if (a.o && ok && rg == 0)
                ((IO *)a.o)[b * a.so.s0 + h * a.so.s1 + t * a.so.s2 + col] = from_f<IO>(a.scale * y);
        }
    }
    IO *out = REV ? (IO *)a.dvv : (IO *)a.o;
    const Strides so = REV ? a.sdv : a.so;
    for (long long t = n + rg; t < a.T; t += 4)
        if (out && ok) out[b * so.s0 + h * so.s1 + t * so.s2 + col] = from_f<IO>(0.0f);
    float *Sn = REV ? a.dS0 : a.S_T;
    if (!Sn) return;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
        const int r = rg * 64 + i;
        if (ok && r < a.dk) Sn[((size_t)bh * a.dk + r) * a.dv + col] = S[i];
    }
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m);
    return x;
}

// One row of the memory a wavefront, given every token's x and du.
template <typename IO, bool REV>
__global__ __launch_bounds__(64) void row_kernel(DeltaArgs a, Ws w) {
    const int r = blockIdx.x % a.dk, bh = blockIdx.x / a.dk, b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const int lane = threadIdx.x, n = tokens(a, b);
    float S[8];
    const float *S0 = REV ? a.dS_T : a.S0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        S[i] = S0 && lane + 64 * i < a.dv ? S0[((size_t)bh * a.dk + r) * a.dv + lane + 64 * i] : 0.0f;
    for (int s = 0; s < n; ++s) {
        const long long t = REV ? n - 1 - s : s;
        const float gam = decay(a, b, h, t), beta = strength(a, b, h, t);
        const float k = to_f(((const IO *)a.k)[b * a.sk.s0 + hk * a.sk.s1 + t * a.sk.s2 + r]);
        const float q = to_f(((const IO *)a.q)[b * a.sq.s0 + hk * a.sq.s1 + t * a.sq.s2 + r]);
        const IO *go = (const IO *)a.d_o + b * a.sdo.s0 + h * a.sdo.s1 + t * a.sdo.s2;
        const size_t row = (size_t)bh * a.T + t;
        float y = 0.0f, z = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = lane + 64 * i;
            const bool ok = c < a.dv;
            const float x = ok ? w.x[row * a.dv + c] : 0.0f, dv = ok ? beta * w.du[row * a.dv + c] : 0.0f;
            const float o = ok ? to_f(go[c]) : 0.0f;
            if constexpr (REV) {
                S[i] += a.scale * q * o;
                y += S[i] * (beta * x);
                S[i] = gam * (S[i] - k * dv);
            } else {
                S[i] *= gam;
                y -= S[i] * dv;
                S[i] += k * (beta * x);
                z += a.scale * S[i] * o;
            }
        }
        y = wave_sum(y);
        if constexpr (!REV) z = wave_sum(z);
        if (lane == 0) {
            if constexpr (REV) {
                w.gk[row * a.dk + r] += y;
            } else {
                w.gk[row * a.dk + r] = y;
                w.gq[row * a.dk + r] = z;
            }
        }
    }
    if constexpr (!REV)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 64 * i < a.dv) w.st[((size_t)bh * a.dk + r) * a.dv + lane + 64 * i] = S[i];
}

// dbeta and the decay's share of each token, one wavefront a token
template <typename IO>
__global__ __launch_bounds__(64) void token_kernel(DeltaArgs a, Ws w) {
    const long long row = blockIdx.x;
    const int bh = (int)(row / a.T), b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const long long t = row % a.T;
    const int lane = threadIdx.x;
    float db = 0.0f, dG = 0.0f;
    if (t < tokens(a, b)) {
        const IO *q = (const IO *)a.q + b * a.sq.s0 + hk * a.sq.s1 + t * a.sq.s2;
        const IO *k = (const IO *)a.k + b * a.sk.s0 + hk * a.sk.s1 + t * a.sk.s2;
        for (int c = lane; c < a.dv; c += 64) db += w.x[row * a.dv + c] * w.du[row * a.dv + c];
        for (int c = lane; c < a.dk; c += 64)
            dG += to_f(q[c]) * w.gq[row * a.dk + c] + to_f(k[c]) * w.gk[row * a.dk + c];
        db = wave_sum(db);
        dG = wave_sum(dG) - 2.0f * strength(a, b, h, t) * db;
    }
    if (lane == 0) {
        a.db[b * a.sdb.s0 + h * a.sdb.s1 + t * a.sdb.s2] = db;
        w.dG[row] = dG;
    }
}

__global__ __launch_bounds__(64) void decay_kernel(DeltaArgs a, Ws w) {
    const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H, n = tokens(a, b);
    const size_t size = (size_t)a.dk * a.dv;
    double sum = 0.0;
    if (a.dS_T)
        for (size_t i = threadIdx.x; i < size; i += 64) sum += (double)a.dS_T[bh * size + i] * w.st[bh * size + i];
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
    if (threadIdx.x != 0) return;
    for (long long t = a.T - 1; t >= 0; --t) {
        if (t < n) sum += w.dG[(size_t)bh * a.T + t];
        a.dg[b * a.sdg.s0 + h * a.sdg.s1 + t * a.sdg.s2] = t < n && decay(a, b, h, t) != 0.0f ? (float)sum : 0.0f;
    }
}

// dq and dk: the heads of a group summed
template <typename IO>
__global__ __launch_bounds__(64) void group_kernel(DeltaArgs a, Ws w) {
    const long long row = blockIdx.x;
    const int bk = (int)(row / a.T), b = bk / a.Hk, hk = bk % a.Hk, r = a.H / a.Hk;
    const long long t = row % a.T;
    const bool live = t < tokens(a, b);
    for (int c = threadIdx.x; c < a.dk; c += 64) {
        float q = 0.0f, k = 0.0f;
        for (int i = 0; i < r && live; ++i) {
            const size_t at = (((size_t)b * a.H + hk * r + i) * a.T + t) * a.dk + c;
            q += w.gq[at];
            k += w.gk[at];
        }
        ((IO *)a.dq)[b * a.sdq.s0 + hk * a.sdq.s1 + t * a.sdq.s2 + c] = from_f<IO>(q);
        ((IO *)a.dkk)[b * a.sdk.s0 + hk * a.sdk.s1 + t * a.sdk.s2 + c] = from_f<IO>(k);
    }
}

template <typename IO>
hipError_t launch_fwd_t(const DeltaArgs &a, hipStream_t s) {
    column_kernel<IO, false><<<dim3((unsigned)(a.B * a.H * ((a.dv + BV - 1) / BV))), 256, 0, s>>>(a, Ws{});
    return hipGetLastError();
}

template <typename IO>
hipError_t launch_bwd_t(const DeltaArgs &a, hipStream_t s) {
    const Ws w = make_ws(a);
    const unsigned cols = (unsigned)(a.B * a.H * ((a.dv + BV - 1) / BV)), cells = (unsigned)(a.B * a.H);
    column_kernel<IO, false><<<dim3(cols), 256, 0, s>>>(a, w);
    column_kernel<IO, true><<<dim3(cols), 256, 0, s>>>(a, w);
    row_kernel<IO, false><<<dim3(cells * a.dk), 64, 0, s>>>(a, w);
    row_kernel<IO, true><<<dim3(cells * a.dk), 64, 0, s>>>(a, w);
    token_kernel<IO><<<dim3(cells * a.T), 64, 0, s>>>(a, w);
    decay_kernel<<<dim3(cells), 64, 0, s>>>(a, w);
    group_kernel<IO><<<dim3((unsigned)(a.B * a.Hk) * a.T), 64, 0, s>>>(a, w);
    return hipGetLastError();
}

}  // namespace

size_t deltarule_workspace_floats(int B, int Hk, int H, int T, int dk, int dv, int io_bf16, int backward) {
    (void)Hk, (void)io_bf16;
    if (!backward) return 0;
    const size_t n = (size_t)B * H;
    return n * T * (2 * (size_t)dv + 2 * (size_t)dk + 1) + n * dk * dv;
}

hipError_t launch_deltarule_fwd(const DeltaArgs &a, int io_bf16, hipStream_t s) {
    return io_bf16 ? launch_fwd_t<bf16>(a, s) : launch_fwd_t<float>(a, s);
}
hipError_t launch_deltarule_bwd(const DeltaArgs &a, int io_bf16, hipStream_t s) {
    return io_bf16 ? launch_bwd_t<bf16>(a, s) : launch_bwd_t<float>(a, s);
}

}  // namespace mlstm
