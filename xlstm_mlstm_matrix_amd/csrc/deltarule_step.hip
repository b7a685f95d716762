// deltarule_step.hip -- one token of the gated delta rule (decode):
// x = v - e^g S^T k, S <- e^g S + beta k x^T, o = scale * S^T q.
//
// The state is read and written once (8 d_qk d_v bytes a head) and nothing else is
// large: the step is bound by HBM.  Both products with the old state are taken
// while it is read, o = scale (e^g S^T q + beta (q . k) x), and a thread keeps what
// it read in registers until x is known.  A workgroup owns a block of value
// columns with all their rows, so one launch and no workspace do.
#include "ops.hpp"

namespace mlstm {

namespace {

// Workgroup: 256 threads = 16 column threads (4 columns, 16 bytes each) x 16 row
// groups; thread (rg, ct) holds rows rg, rg + 16, ... (NR of them).
template <typename IO, int NR>
__global__ __launch_bounds__(256) void deltarule_step_kernel(DeltaStepArgs a, int ntile) {
    constexpr int CT = 16, RG = 16;
    __shared__ float qs[256], ks[256];
    __shared__ f32x4 red[4][2][CT];
    __shared__ float dot[4];
    const int tile = blockIdx.x % ntile, bh = blockIdx.x / ntile;
    const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const int tid = threadIdx.x, ct = tid % CT, rg = tid / CT, wave = tid >> 6;
    const int col = (tile * CT + ct) * 4;
    const bool ok = col < a.dv;
    const IO *q = (const IO *)a.q + b * a.sq.s0 + hk * a.sq.s1;
    const IO *k = (const IO *)a.k + b * a.sk.s0 + hk * a.sk.s1;
    const IO *v = (const IO *)a.v + b * a.sv.s0 + h * a.sv.s1;
    const float gam = __builtin_amdgcn_exp2f(decay_log2(a.g[b * a.sg.s0 + h * a.sg.s1]));
    const float beta = a.beta[b * a.sb.s0 + h * a.sb.s1];
    if (tid < a.dk) {
        qs[tid] = to_f(q[tid]);
        ks[tid] = to_f(k[tid]);
    }
    const size_t base = (size_t)bh * a.dk * a.dv + col;
    f32x4 S[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = rg + RG * i;
        S[i] = f32x4{0, 0, 0, 0};
        if (ok && a.S_in && r < a.dk) S[i] = gam * *(const f32x4 *)(a.S_in + base + (size_t)r * a.dv);
    }
    __syncthreads();
    f32x4 kS = {0, 0, 0, 0}, qS = kS;
    float qk = 0.0f;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = rg + RG * i;
        if (r < a.dk) {
            kS += ks[r] * S[i];
            qS += qs[r] * S[i];
            qk += qs[r] * ks[r];
        }
    }
#pragma unroll
    for (int m = 16; m < 64; m <<= 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            kS[e] += __shfl_xor(kS[e], m);
            qS[e] += __shfl_xor(qS[e], m);
        }
        qk += __shfl_xor(qk, m);
    }
    if ((tid & 63) < CT) {
        red[wave][0][ct] = kS;
        red[wave][1][ct] = qS;
        if (ct == 0) dot[wave] = qk;
    }
    __syncthreads();
    kS = (red[0][0][ct] + red[1][0][ct]) + (red[2][0][ct] + red[3][0][ct]);
    if (!ok) return;
    const f32x4 vv = {to_f(v[col]), to_f(v[col + 1]), to_f(v[col + 2]), to_f(v[col + 3])};
    const f32x4 u = (vv - kS) * beta;
    float *So = a.S_out + base;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = rg + RG * i;
        if (r < a.dk) *(f32x4 *)(So + (size_t)r * a.dv) = S[i] + ks[r] * u;
    }
    if (rg == 0) {
        IO *o = (IO *)a.o + b * a.so.s0 + h * a.so.s1 + col;
        qS = (red[0][1][ct] + red[1][1][ct]) + (red[2][1][ct] + red[3][1][ct]);
        const f32x4 y = (qS + ((dot[0] + dot[1]) + (dot[2] + dot[3])) * u) * a.scale;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = from_f<IO>(y[e]);
    }
}

template <typename IO>
hipError_t launch_t(const DeltaStepArgs &a, hipStream_t s) {
    const int ntile = (a.dv + 63) / 64;
    const dim3 grid((unsigned)(a.B * a.H * ntile));
    if (a.dk <= 64)
        deltarule_step_kernel<IO, 4><<<grid, 256, 0, s>>>(a, ntile);
    else if (a.dk <= 128)
        deltarule_step_kernel<IO, 8><<<grid, 256, 0, s>>>(a, ntile);
    else
        deltarule_step_kernel<IO, 16><<<grid, 256, 0, s>>>(a, ntile);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_deltarule_step(const DeltaStepArgs &a, int io_bf16, hipStream_t s) {
    return io_bf16 ? launch_t<bf16>(a, s) : launch_t<float>(a, s);
}

}  // namespace mlstm
