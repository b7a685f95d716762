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

constexpr long long kStreamBytes = 320ll << 20;  // a quarter more than the Infinity Cache

// 16 bytes of state, past the caches' replacement order when STREAM
template <bool STREAM>
__device__ __forceinline__ f32x4 load(const float *p) {
    if constexpr (STREAM) return __builtin_nontemporal_load((const f32x4 *)p);
    return *(const f32x4 *)p;
}
template <bool STREAM>
__device__ __forceinline__ void store(float *p, f32x4 x) {
    if constexpr (STREAM)
        __builtin_nontemporal_store(x, (f32x4 *)p);
    else
        *(f32x4 *)p = x;
}

// Workgroup: CT column threads (4 columns, 16 bytes each) x 16 row groups; thread
// (rg, ct) holds rows rg, rg + 16, ... (NR of them).
template <typename IO, int NR, int CT, bool STREAM>
__global__ __launch_bounds__(16 * CT) void deltarule_step_kernel(DeltaStepArgs a, int ntile) {
    constexpr int RG = 16, NW = CT / 4;
    __shared__ float qs[256], ks[256];
    __shared__ f32x4 red[NW][2][CT];
    __shared__ float dot[NW];
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
    // d_qk is a multiple of 16: a thread's rows past it are the same for all threads.  They
    // load the last row again and count as zeros, without a branch.
    const int nr = a.dk / RG;
    for (int i = tid; i < RG * NR; i += RG * CT) {
        const int r = min(i, a.dk - 1);
        qs[i] = i < a.dk ? to_f(q[r]) : 0.0f;
        ks[i] = i < a.dk ? to_f(k[r]) : 0.0f;
    }
    const int c = ok ? col : 0;
    const size_t base = (size_t)bh * a.dk * a.dv + c;
    f32x4 S[NR];
    if (a.S_in) {
#pragma unroll
        for (int i = 0; i < NR; ++i) S[i] = load<STREAM>(a.S_in + base + (size_t)(rg + RG * min(i, nr - 1)) * a.dv);
    } else {
#pragma unroll
        for (int i = 0; i < NR; ++i) S[i] = f32x4{0, 0, 0, 0};
    }
    __syncthreads();
    f32x4 kS = {0, 0, 0, 0}, qS = kS;
    float qk = 0.0f;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const float kr = ks[rg + RG * i], qr = qs[rg + RG * i];
        S[i] *= i < nr ? gam : 0.0f;
        kS += kr * S[i];
        qS += qr * S[i];
        qk += qr * kr;
    }
#pragma unroll
    for (int m = CT; m < 64; m <<= 1) {
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
    kS = red[0][0][ct];
#pragma unroll
    for (int w = 1; w < NW; ++w) kS += red[w][0][ct];
    if (!ok) return;
    const f32x4 vv = {to_f(v[col]), to_f(v[col + 1]), to_f(v[col + 2]), to_f(v[col + 3])};
    const f32x4 u = (vv - kS) * beta;
    float *So = a.S_out + base;
#pragma unroll
    for (int i = 0; i < NR; ++i)
        if (i < nr) store<STREAM>(So + (size_t)(rg + RG * i) * a.dv, S[i] + ks[rg + RG * i] * u);
    if (rg == 0) {
        IO *o = (IO *)a.o + b * a.so.s0 + h * a.so.s1 + col;
        qS = red[0][1][ct];
        qk = dot[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            qS += red[w][1][ct];
            qk += dot[w];
        }
        const f32x4 y = (qS + qk * u) * a.scale;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = from_f<IO>(y[e]);
    }
}

template <typename IO, int CT, bool STREAM>
hipError_t launch_ct(const DeltaStepArgs &a, hipStream_t s) {
    const int ntile = (a.dv + 4 * CT - 1) / (4 * CT);
    const dim3 grid((unsigned)(a.B * a.H * ntile));
    if (a.dk <= 64)
        deltarule_step_kernel<IO, 4, CT, STREAM><<<grid, 16 * CT, 0, s>>>(a, ntile);
    else if (a.dk <= 128)
        deltarule_step_kernel<IO, 8, CT, STREAM><<<grid, 16 * CT, 0, s>>>(a, ntile);
    else
        deltarule_step_kernel<IO, 16, CT, STREAM><<<grid, 16 * CT, 0, s>>>(a, ntile);
    return hipGetLastError();
}

template <typename IO>
hipError_t launch_t(const DeltaStepArgs &a, hipStream_t s) {
    const long long cells = (long long)a.B * a.H;
    const int quads = a.dv / 4;
    // States that the cache cannot hold from one step to the next are streamed past it, by
    // the bytes touched: once in place, twice from one tensor into another.  128 columns a
    // workgroup, 256 x 512: 1 GB in place 384 us, streamed 372; 128 MB 80 us, streamed 103.  With
    // 64 columns they take 439 and 83.
    const bool once = !a.S_in || a.S_in == a.S_out;
    if (cells * a.dk * a.dv * (once ? 4 : 8) > kStreamBytes && quads >= 32) return launch_ct<IO, 32, true>(a, s);
    // narrower ones for two workgroups a compute unit
    auto wgs = [&](int ct) { return cells * ((quads + ct - 1) / ct); };
    if (quads >= 32 && wgs(32) >= 512) return launch_ct<IO, 32, false>(a, s);
    if (quads >= 16 && wgs(16) >= 512) return launch_ct<IO, 16, false>(a, s);
    return launch_ct<IO, 8, false>(a, s);
}

}  // namespace

hipError_t launch_deltarule_step(const DeltaStepArgs &a, int io_bf16, hipStream_t s) {
    return io_bf16 ? launch_t<bf16>(a, s) : launch_t<float>(a, s);
}

}  // namespace mlstm
