// linattn_step.hip -- one token of linear attention with a decay for each
// head (decode): S <- e^g S + k v^T, o = scale * q^T S.
//
// The state is read and written once (8 d_qk d_v bytes a head) and nothing
// else is large: the step is bound by HBM.  Each workgroup owns a block of
// value columns of one head with all its rows, so the read-out needs no
// second launch and no workspace.
#include "ops.hpp"

namespace mlstm {

namespace {

// Workgroup: 256 threads = CT column threads (4 columns, 16 bytes each) x
// 256 / CT row groups; thread (rg, ct) walks rows rg, rg + RG, ...
template <typename IO, int CT>
__global__ __launch_bounds__(256) void linattn_step_kernel(LinStepArgs a, int ntile) {
    constexpr int RG = 256 / CT;
    __shared__ float qs[256], ks[256];
    __shared__ f32x4 red[RG][CT];
    const int tile = blockIdx.x % ntile, bh = blockIdx.x / ntile;
    const int b = bh / a.H, h = bh % a.H;
    const int ct = threadIdx.x % CT, rg = threadIdx.x / CT;
    const int col = (tile * CT + ct) * 4;
    const bool ok = col < a.dv;
    const IO *q = (const IO *)a.q + b * a.sq.s0 + h * a.sq.s1;
    const IO *k = (const IO *)a.k + b * a.sk.s0 + h * a.sk.s1;
    const IO *v = (const IO *)a.v + b * a.sv.s0 + h * a.sv.s1;
    const float gam = __builtin_amdgcn_exp2f(decay_log2(a.g[h]));
    if ((int)threadIdx.x < a.dk) {
        qs[threadIdx.x] = to_f(q[threadIdx.x]);
        ks[threadIdx.x] = to_f(k[threadIdx.x]);
    }
    __syncthreads();
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    if (ok) {
        const f32x4 vv = {to_f(v[col]), to_f(v[col + 1]), to_f(v[col + 2]), to_f(v[col + 3])};
        const size_t base = (size_t)bh * a.dk * a.dv + col;
        const float *S = a.S_in ? a.S_in + base : nullptr;
        float *So = a.S_out + base;
#pragma unroll 8
        for (int r = rg; r < a.dk; r += RG) {
            f32x4 x = vv * ks[r];
            if (S) x += gam * *(const f32x4 *)(S + (size_t)r * a.dv);
            acc += qs[r] * x;
            *(f32x4 *)(So + (size_t)r * a.dv) = x;
        }
    }
    red[rg][ct] = acc;
    __syncthreads();
    for (int m = RG / 2; m > 0; m >>= 1) {
        if (rg < m) red[rg][ct] += red[rg + m][ct];
        __syncthreads();
    }
    if (rg == 0 && ok) {
        IO *o = (IO *)a.o + b * a.so.s0 + h * a.so.s1 + col;
        const f32x4 r = red[0][ct] * a.scale;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = from_f<IO>(r[i]);
    }
}

template <typename IO>
hipError_t launch_t(const LinStepArgs &a, hipStream_t s) {
    const int quads = a.dv / 4;
    const int ct = quads >= 32 ? 32 : 16;
    const int ntile = (quads + ct - 1) / ct;
    const dim3 grid((unsigned)(a.B * a.H * ntile));
    if (ct == 32)
        linattn_step_kernel<IO, 32><<<grid, 256, 0, s>>>(a, ntile);
    else
        linattn_step_kernel<IO, 16><<<grid, 256, 0, s>>>(a, ntile);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linattn_step(const LinStepArgs &a, int io_bf16, hipStream_t s) {
    return io_bf16 ? launch_t<bf16>(a, s) : launch_t<float>(a, s);
}

}  // namespace mlstm
