// linattn_step.hip -- one token of linear attention with a decay for each
// head (decode): S <- e^g S + k v^T, o = scale * q^T S.
//
// The state is read and written once (8 d_qk d_v bytes a head) and nothing
// else is large: the step is bound by HBM.  Each workgroup owns a block of
// value columns of one head with all its rows, so the read-out needs no
// second launch and no workspace.  2048 heads of 256 x 512: 386 us, 5.6 TB/s.
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

// Workgroup: 256 threads = CT column threads (4 columns, 16 bytes each) x
// 256 / CT row groups; thread (rg, ct) walks rows rg, rg + RG, ...
template <typename IO, int CT, bool STREAM>
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
        constexpr int UNROLL = STREAM ? 16 : 8;  // rows in flight
#pragma unroll UNROLL
        for (int r = rg; r < a.dk; r += RG) {
            f32x4 x = vv * ks[r];
            if (S) x += gam * load<STREAM>(S + (size_t)r * a.dv);
            acc += qs[r] * x;
            store<STREAM>(So + (size_t)r * a.dv, x);
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

template <typename IO, int CT, bool STREAM>
hipError_t launch_ct(const LinStepArgs &a, hipStream_t s) {
    const int ntile = (a.dv / 4 + CT - 1) / CT;
    linattn_step_kernel<IO, CT, STREAM><<<dim3((unsigned)(a.B * a.H * ntile)), 256, 0, s>>>(a, ntile);
    return hipGetLastError();
}

template <typename IO>
hipError_t launch_t(const LinStepArgs &a, hipStream_t s) {
    const long long cells = (long long)a.B * a.H;
    const int quads = a.dv / 4;
    // States that the cache cannot hold from one step to the next are streamed past
    // it.  What counts are the bytes touched, once in place and twice from one tensor
    // into another.  In place, 256 x 512: 144 MB 46.8 us (streamed 72.1), 256 MB 94
    // (97), 320 MB 129 (141), 384 MB 152 (152), 512 MB 209 (195), 2 GB 411 (386);
    // 128 x 128: 224 MB 70 (85), 320 MB 124 (119), 512 MB 208 (189).  Into another
    // tensor, states of 144 MB 53 (65), 160 MB 59 (66), 192 MB 80 (74).  Rows too
    // short for it are not streamed (1 GB of 64 x 64: 186 us, streamed 202).
    const bool once = !a.S_in || a.S_in == a.S_out;
    if (cells * a.dk * a.dv * (once ? 4 : 8) > kStreamBytes) {
        if (quads >= 64) return launch_ct<IO, 64, true>(a, s);
        if (quads >= 32) return launch_ct<IO, 32, true>(a, s);
    }
    // Two workgroups a compute unit where the columns allow it: those 64 heads
    // take 17.2 us with blocks of 128 columns throughout.
    auto wgs = [&](int ct) { return cells * ((quads + ct - 1) / ct); };
    if (quads >= 32 && wgs(32) >= 512) return launch_ct<IO, 32, false>(a, s);
    if (quads >= 16 && wgs(16) >= 512) return launch_ct<IO, 16, false>(a, s);
    return launch_ct<IO, 8, false>(a, s);
}

}  // namespace

hipError_t launch_linattn_step(const LinStepArgs &a, int io_bf16, hipStream_t s) {
    return io_bf16 ? launch_t<bf16>(a, s) : launch_t<float>(a, s);
}

}  // namespace mlstm
