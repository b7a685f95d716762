// linattn.hip -- linear attention with a decay for each head.
#include "ops.hpp"

namespace mlstm {

namespace {

constexpr int kCols = 16;  // state columns of a workgroup

// The recurrence token by token.  One workgroup owns 16 state columns of one
// (job, b, h): X [dk][16] in LDS, thread (rg, c) updates rows rg, rg + 16, ...
template <typename IO>
__global__ __launch_bounds__(256) void linattn_rec_kernel(LinArgs a, int ntile) {
    extern __shared__ float lds[];
    const int tile = blockIdx.x % ntile;
    const int bh = (blockIdx.x / ntile) % (a.B * a.H);
    const LinJob &j = a.job[blockIdx.x / ntile / (a.B * a.H)];
    const int c0 = tile * kCols;
    if (c0 >= j.dv) return;
    const int b = bh / a.H, h = bh % a.H;
    const int n = a.lengths ? max(0, min(a.lengths[b], a.T)) : a.T;
    const int c = threadIdx.x & 15, rg = threadIdx.x >> 4, dk = j.dk;
    const int col = c0 + c;
    const bool ok = col < j.dv;
    float *X = lds, *qs = X + dk * kCols, *ks = qs + dk, *red = ks + dk;
    const float gl = decay_log2(a.g[h]);
    const float gam = __builtin_amdgcn_exp2f(gl);
    const size_t st = (size_t)bh * dk * j.dv;
    for (int r = rg; r < dk; r += 16)
        X[r * kCols + c] = (ok && j.X0) ? j.X0[st + r * j.rs + col * j.cs] : 0.0f;
    const IO *q = (const IO *)j.q + b * j.sq.s0 + h * j.sq.s1;
    const IO *k = (const IO *)j.k + b * j.sk.s0 + h * j.sk.s1;
    const IO *v = (const IO *)j.v + b * j.sv.s0 + h * j.sv.s1;
    IO *o = (IO *)j.o + b * j.so.s0 + h * j.so.s1;
    for (int tau = 0; tau < n; ++tau) {
        const long long t = j.reverse ? n - 1 - tau : tau;
        __syncthreads();
        for (int r = threadIdx.x; r < dk; r += 256) {
            qs[r] = to_f(q[t * j.sq.s2 + r]);
            ks[r] = to_f(k[t * j.sk.s2 + r]);
        }
        __syncthreads();
        const float vv = ok ? to_f(v[t * j.sv.s2 + col]) : 0.0f;
        // carried part and this token's part apart: they have their own scales
        const float fade = j.shift ? 1.0f : gam;
        float inter = 0.0f, dot = 0.0f;
        for (int r = rg; r < dk; r += 16) {
            const float x = X[r * kCols + c];
            inter += qs[r] * x;
            dot += qs[r] * ks[r];
            X[r * kCols + c] = gam * x + (j.shift ? gam : 1.0f) * j.up_scale * ks[r] * vv;
        }
        red[threadIdx.x] = inter * fade * j.in_scale + dot * j.p_scale * vv;
        __syncthreads();
        if (rg == 0 && ok) {
            float x = 0.0f;
            for (int i = 0; i < 16; ++i) x += red[c + 16 * i];
            o[t * j.so.s2 + col] = from_f<IO>(x);
        }
    }
    if (ok)
        for (long long t = n + rg; t < a.T; t += 16) o[t * j.so.s2 + col] = from_f<IO>(0.0f);
    if (ok && j.Xn)
        for (int r = rg; r < dk; r += 16) j.Xn[st + r * j.rs + col * j.cs] = X[r * kCols + c];
}

}  // namespace

size_t linattn_workspace_floats(int, int, int, int, int, int, int) { return 0; }

hipError_t launch_linattn(const LinArgs &a, int io_bf16, hipStream_t s) {
    int dv = 0, dk = 0;
    for (int i = 0; i < a.njob; ++i) {
        dv = a.job[i].dv > dv ? a.job[i].dv : dv;
        dk = a.job[i].dk > dk ? a.job[i].dk : dk;
    }
    const int ntile = (dv + kCols - 1) / kCols;
    const size_t lds = ((size_t)dk * kCols + 2 * dk + 256) * 4;
    const dim3 grid((unsigned)(a.njob * a.B * a.H * ntile));
    if (io_bf16)
        linattn_rec_kernel<bf16><<<grid, 256, lds, s>>>(a, ntile);
    else
        linattn_rec_kernel<float><<<grid, 256, lds, s>>>(a, ntile);
    return hipGetLastError();
}

}  // namespace mlstm
