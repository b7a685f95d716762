// groupnorm.hip -- group norm with an activation, channels last, forward and
// backward.
//
//   xh = (x - mean) rstd,  z = w xh + b,  y = act(z);
//   dz = dy act'(z),  u = dz w,  dx = rstd (u - mean(u) - xh mean(u xh)),
//   dw = sum dz xh,  db = sum dz        (sums over samples and positions).
//
// All of it is bound by memory: x read and y written once (forward), x and dy
// read and dx written once (backward).  Measured over tokens, bfloat16,
// 32768 rows of 8 heads of 512: 110 us (4.9 TB/s) forward, 194 us (4.15 TB/s)
// backward; a large copy runs at 4.8.  Over long sequences x, and dy, are read
// twice: 43 us forward and 59 backward at 15000 positions of 1280 channels (GELU).
//
// Over tokens a group is D contiguous channels: gn_row_kernel holds it in the
// registers of a few lanes.  Over sequences, and for rows too long for that,
// the work is split over positions: gn_channel_kernel reduces a block of
// positions to two numbers for each channel, gn_combine_kernel joins those
// into the group's statistics (or the backward's two means), and
// gn_apply_kernel writes the result.  Every sum has a fixed order.
//
// A mean is formed in two steps: the sum over n, then that plus the mean of the
// distances from it (in the pass that sums their squares).  So it is good to its
// last bit: a constant group has exactly its value as its mean and its bias as its
// result.  (A sum of n equal floats is rounded: divided by n it can be a step off,
// which 1 / sqrt(eps) turns into 0.3 for a row of 48 times 12345.678.)  bfloat16
// groups held in registers, and bfloat16 blocks of positions, take the first step
// only: sums of up to 2^16 equal values of 8 bits are exact, and the second costs
// rows of 16 x 128 (SiLU) 5%: 26.7 -> 28 us, and float32 ones 47.3 -> 49 us.
#include "ops.hpp"

namespace mlstm {

namespace {

// Phi(z), the normal distribution function, and e = e^{-z^2/2}, which the
// derivative needs too.  Phi(-x) = t P(t) e^{-x^2/2} with t = 1 / (1 + 0.28 x): P
// is of degree 8, fitted to the smallest relative error over x = 0 .. 14.5 (6e-8;
// 3.4e-7 in float32).  So the tail keeps its relative precision: Phi is off by
// (16 + 1.3 z^2) 2^-24 of itself, most of it from the exponent.  Over 15000
// positions of 1280 channels, bfloat16, the forward takes 43 us with it, 36 with
// SiLU, 35 with neither, the backward 59, 52 and 50.
__device__ __forceinline__ float phi(float z, float *e) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.28f, fabsf(z), 1.0f));
    *e = exp_e(-0.5f * z * z);
    float q = 0.0230575129f;
    q = fmaf(q, t, -0.0846737176f);
    q = fmaf(q, t, 0.0725154057f);
    q = fmaf(q, t, 0.017673118f);
    q = fmaf(q, t, 0.0554796606f);
    q = fmaf(q, t, 0.0911203101f);
    q = fmaf(q, t, 0.10117884f);
    q = fmaf(q, t, 0.111959532f);
    q = fmaf(q, t, 0.111689366f);
    q *= t * *e;
    return z < 0.0f ? q : 1.0f - q;
}
template <int ACT>
__device__ __forceinline__ float act_f(float z) {
    if constexpr (ACT == 1) return z * __builtin_amdgcn_rcpf(1.0f + exp_e(-z));
    if constexpr (ACT == 2) {
        float e;
        return z * phi(z, &e);
    }
    return z;
}
template <int ACT>
__device__ __forceinline__ float act_d(float z) {
    if constexpr (ACT == 1) {
        const float sg = __builtin_amdgcn_rcpf(1.0f + exp_e(-z));
        return sg * (1.0f + z * (1.0f - sg));
    }
    if constexpr (ACT == 2) {
        float e;
        const float p = phi(z, &e);
        return p + z * 0.39894228f * e;
    }
    return 1.0f;
}

// Sum over aligned groups of n lanes (n a power of two), in every lane of them.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane_sum(float v, int n) {
    if (n >= 2) v = dpp_add<0xb1>(v);    // quad_perm 1,0,3,2
    if (n >= 4) v = dpp_add<0x4e>(v);    // quad_perm 2,3,0,1
    if (n >= 8) v = dpp_add<0x141>(v);   // row_half_mirror
    if (n >= 16) v = dpp_add<0x140>(v);  // row_mirror
    if (n >= 32) v += __shfl_xor(v, 16, 64);
    if (n >= 64) v += __shfl_xor(v, 32, 64);
    return v;
}

// V consecutive elements, V * sizeof(IO) = 16 bytes or one element.
template <typename IO, int V>
__device__ __forceinline__ void load_v(const IO *p, float *x) {
    if constexpr (V == 1) {
        x[0] = to_f(p[0]);
    } else {
        typedef IO vec __attribute__((ext_vector_type(V)));
        const vec t = *(const vec *)p;
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = to_f(t[i]);
    }
}
template <typename IO, int V>
__device__ __forceinline__ void store_v(IO *p, const float *x) {
    if constexpr (V == 1) {
        p[0] = from_f<IO>(x[0]);
    } else {
        typedef IO vec __attribute__((ext_vector_type(V)));
        vec t;
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = from_f<IO>(x[i]);
        *(vec *)p = t;
    }
}

// V weights from p (16-byte aligned where V > 1), or `other` without one
template <int V>
__device__ __forceinline__ void load_w(const float *p, size_t at, bool ok, float other, float *w) {
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = other;
    if (!p || !ok) return;
    if constexpr (V == 1) {
        w[0] = p[at];
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const f32x4 t = *(const f32x4 *)(p + at + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i + j] = t[j];
        }
    }
}

// Variance from the mean square distance from a point `off` below the mean.
// off is a few roundings of the mean's first step, so nothing cancels.
__device__ __forceinline__ float variance(float sq, float off) {
    const float v = sq - off * off;
    return v < 0.0f ? 0.0f : v;  // NaN stays
}

// ---- over tokens, D <= 64 V K: lanes of a row
//
// A wavefront is cut into subgroups of `lpr` lanes, each holding one group's D
// channels (K vectors a lane).  `gp` neighbouring subgroups take neighbouring
// groups of one position (contiguous memory in token-major tensors), the rest
// take further positions.  A workgroup stays with its groups, so weights are
// loaded once and the weight gradients add up in registers.
struct RowGeom {
    int lpr, gp;              // log2 of the lanes per row, of the groups side by side
    int gblk, rblk;           // blocks of groups, blocks of positions
    unsigned long long div;   // ceil(2^64 / S): r / S is the upper half of r * div
};

template <typename IO, int V, int K, int ACT, bool BWD>
__global__ __launch_bounds__(256) void gn_row_kernel(GnArgs a, RowGeom q, int block0) {
    constexpr bool TWO = sizeof(IO) == 4;  // steps of a mean
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lpr = 1 << q.lpr, sub = lane >> q.lpr, ln = lane & (lpr - 1);
    const int rpi = 64 >> (q.lpr + q.gp);  // positions side by side in a wavefront
    const int block = block0 + blockIdx.x, gb = block % q.gblk, rb = block / q.gblk;
    const int g = (gb << q.gp) + (sub & ((1 << q.gp) - 1)), rsub = sub >> q.gp;
    const int D = a.D, nrow = a.N * a.S;
    const IO *x = (const IO *)a.x + g * a.sx.s2;
    const IO *dy = BWD ? (const IO *)a.dy + g * a.sdy.s2 : nullptr;
    IO *y = (IO *)a.y + g * a.sy.s2;
    bool ok[K];
    int d[K];
    float w[K][V], bb[K][V], aw[K][V], ab[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        d[k] = (k * lpr + ln) * V;
        ok[k] = d[k] < D;
        load_w<V>(a.w, (size_t)g * D + d[k], ok[k], 1.0f, w[k]);
        load_w<V>(a.b, (size_t)g * D + d[k], ok[k], 0.0f, bb[k]);
#pragma unroll
        for (int i = 0; i < V; ++i) aw[k][i] = ab[k][i] = 0.0f;
    }
    const float inv = 1.0f / (float)D;
    for (long long r0 = (long long)(rb * 4 + wave) * rpi; r0 < nrow; r0 += (long long)q.rblk * 4 * rpi) {
        const bool rok = r0 + rsub < nrow;
        const int r = rok ? (int)r0 + rsub : 0;
        const int n = a.S == 1 ? r : (int)__umul64hi((unsigned long long)r, q.div), s = r - n * a.S;
        const size_t si = ((size_t)n * a.S + s) * a.G + g;
        // lanes without a position or channel hold zeros: they add nothing to any sum
        float v[K][V], u[BWD ? K : 1][V];
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[k][i] = 0.0f;
                if constexpr (BWD) u[k][i] = 0.0f;
            }
            if (rok && ok[k]) {
                load_v<IO, V>(x + n * a.sx.s0 + s * a.sx.s1 + d[k], v[k]);
                if constexpr (BWD) load_v<IO, V>(dy + n * a.sdy.s0 + s * a.sdy.s1 + d[k], u[k]);
            }
        }
        if constexpr (!BWD) {
            float t = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) t += v[k][i];
            const float m0 = lane_sum(t, lpr) / (float)D;
            float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float c = v[k][i] - m0;
                    if constexpr (TWO) t1 += ok[k] ? c : 0.0f;
                    t2 += ok[k] ? c * c : 0.0f;
                }
            float mu = m0, var = lane_sum(t2, lpr) * inv;
            if constexpr (TWO) {
                const float off = lane_sum(t1, lpr) * inv;
                mu += off;
                var = variance(var, off);
            }
            const float rs = rsqrtf(var + a.eps);
            if (a.mean && rok && ln == 0) {
                a.mean[si] = mu;
                a.rstd[si] = rs;
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[k][i] = act_f<ACT>((v[k][i] - mu) * rs * w[k][i] + bb[k][i]);
                if (rok && ok[k]) store_v<IO, V>(y + n * a.sy.s0 + s * a.sy.s1 + d[k], v[k]);
            }
        } else {
            const float mu = rok ? a.mean[si] : 0.0f, rs = rok ? a.rstd[si] : 0.0f;
            float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = (v[k][i] - mu) * rs;
                    const float dz = u[k][i] * act_d<ACT>(xh * w[k][i] + bb[k][i]);
                    ab[k][i] += dz;
                    aw[k][i] += dz * xh;
                    v[k][i] = xh;
                    u[k][i] = dz * w[k][i];
                    c1 += u[k][i];
                    c2 += u[k][i] * xh;
                }
            c1 = lane_sum(c1, lpr) * inv;
            c2 = lane_sum(c2, lpr) * inv;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int i = 0; i < V; ++i) u[k][i] = rs * (u[k][i] - c1 - v[k][i] * c2);
                if (rok && ok[k]) store_v<IO, V>(y + n * a.sy.s0 + s * a.sy.s1 + d[k], u[k]);
            }
        }
    }
    if constexpr (BWD) {
        if (!a.dw && !a.db) return;
        // the positions that the lanes of one channel took: over the
        // wavefront's subgroups, then over the wavefronts
        __shared__ float red[2][4][64];
        const int span = lpr << q.gp;
        float *ws = a.ws + (size_t)rb * 2 * a.G * D;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float pw = aw[k][i], pb = ab[k][i];
                for (int m = span; m < 64; m <<= 1) {
                    pw += __shfl_xor(pw, m, 64);
                    pb += __shfl_xor(pb, m, 64);
                }
                __syncthreads();
                red[0][wave][lane] = pw;
                red[1][wave][lane] = pb;
                __syncthreads();
                if (wave < 2 && lane < span && ok[k]) {
                    const float t = (red[wave][0][lane] + red[wave][1][lane]) +
                                    (red[wave][2][lane] + red[wave][3][lane]);
                    ws[(size_t)wave * a.G * D + (size_t)g * D + d[k] + i] = t;
                }
            }
    }
}

// Sums over a workgroup of up to 1024 threads, in every thread; red [32] for two
__device__ __forceinline__ void gn_block_sum2(float &x, float &y, float *red) {
    x = lane_sum(x, 64);
    y = lane_sum(y, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        red[threadIdx.x >> 6] = x;
        red[16 + (threadIdx.x >> 6)] = y;
    }
    __syncthreads();
    x = y = 0.0f;
    for (int i = 0; i < (int)blockDim.x >> 6; ++i) {
        x += red[i];
        y += red[16 + i];
    }
}
__device__ __forceinline__ float gn_block_sum(float v, float *red) {
    v = lane_sum(v, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.0f;
    for (int i = 0; i < (int)blockDim.x >> 6; ++i) t += red[i];
    return t;
}

// ---- over tokens, rows too long for the registers: a workgroup for each row,
// which later passes over the row find in the caches.  The weight gradients
// come from gn_channel_kernel.
template <typename IO, int V, int ACT, bool BWD>
__global__ __launch_bounds__(256) void gn_long_row_kernel(GnArgs a, long long rows) {
    __shared__ float red[32];
    const float inv = 1.0f / (float)a.D;
    for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
        const int g = (int)(r % a.G), ns = (int)(r / a.G);
        const int n = ns / a.S, p = ns % a.S;
        const IO *x = (const IO *)a.x + n * a.sx.s0 + p * a.sx.s1 + g * a.sx.s2;
        const IO *dy = BWD ? (const IO *)a.dy + n * a.sdy.s0 + p * a.sdy.s1 + g * a.sdy.s2 : nullptr;
        IO *y = (IO *)a.y + n * a.sy.s0 + p * a.sy.s1 + g * a.sy.s2;
        const float *w = a.w ? a.w + (size_t)g * a.D : nullptr, *b = a.b ? a.b + (size_t)g * a.D : nullptr;
        float mu, rs, s0 = 0.0f, s1 = 0.0f, s2 = 0.0f;
        float v[V], u[V];
        if constexpr (!BWD) {
            for (int d = threadIdx.x * V; d < a.D; d += 256 * V) {
                load_v<IO, V>(x + d, v);
#pragma unroll
                for (int i = 0; i < V; ++i) s0 += v[i];
            }
            const float m0 = gn_block_sum(s0, red) / (float)a.D;
            for (int d = threadIdx.x * V; d < a.D; d += 256 * V) {
                load_v<IO, V>(x + d, v);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s1 += v[i] - m0;
                    s2 += (v[i] - m0) * (v[i] - m0);
                }
            }
            gn_block_sum2(s1, s2, red);
            mu = m0 + s1 * inv;
            rs = rsqrtf(variance(s2 * inv, s1 * inv) + a.eps);
            if (a.mean && threadIdx.x == 0) {
                a.mean[r] = mu;
                a.rstd[r] = rs;
            }
        } else {
            mu = a.mean[r];
            rs = a.rstd[r];
            for (int d = threadIdx.x * V; d < a.D; d += 256 * V) {
                load_v<IO, V>(x + d, v);
                load_v<IO, V>(dy + d, u);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = (v[i] - mu) * rs, ww = w ? w[d + i] : 1.0f;
                    const float t = u[i] * act_d<ACT>(xh * ww + (b ? b[d + i] : 0.0f)) * ww;
                    s0 += t;
                    s1 += t * xh;
                }
            }
            s0 = gn_block_sum(s0, red) * inv;
            s1 = gn_block_sum(s1, red) * inv;
        }
        for (int d = threadIdx.x * V; d < a.D; d += 256 * V) {
            load_v<IO, V>(x + d, v);
            if constexpr (BWD) load_v<IO, V>(dy + d, u);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xh = (v[i] - mu) * rs, ww = w ? w[d + i] : 1.0f;
                const float z = xh * ww + (b ? b[d + i] : 0.0f);
                if constexpr (BWD)
                    v[i] = rs * (u[i] * act_d<ACT>(z) * ww - s0 - xh * s1);
                else
                    v[i] = act_f<ACT>(z);
            }
            store_v<IO, V>(y + d, v);
        }
    }
}

// ---- over sequences, groups of up to 16384 values: a workgroup holds a
// group in registers (NE values a thread), one launch instead of three.
template <typename IO, int V, int NE, int ACT>
__global__ __launch_bounds__(1024) void gn_group_kernel(GnArgs a, int block0) {
    constexpr int NV = NE / V;
    __shared__ float red[32];
    // neighbouring groups, which share cache lines, on one XCD (workgroups go round the 8)
    const int nwg = gridDim.x, xq = nwg >> 3, xr = nwg & 7, xcd = blockIdx.x & 7;
    const int id = block0 + xcd * xq + min(xcd, xr) + (blockIdx.x >> 3);
    const int g = id % a.G, n = id / a.G;
    const int rv = a.D / V, total = a.S * rv;  // vectors of a position, of the group
    const IO *x = (const IO *)a.x + n * a.sx.s0 + g * a.sx.s2;
    // e / rv for e < 2^15 and rv <= 2^14: the upper half of e * ceil(2^32 / rv)
    const unsigned magic = 0xffffffffu / (unsigned)rv + 1;  // 0 for rv = 1
    auto position = [&](int e) { return rv == 1 ? e : (int)__umulhi((unsigned)e, magic); };
    float v[NV][V], t = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = threadIdx.x + i * blockDim.x;
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = 0.0f;
        const int p = position(e);
        if (e < total) load_v<IO, V>(x + p * a.sx.s1 + (e - p * rv) * V, v[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) t += v[i][j];
    const float inv = 1.0f / ((float)a.S * (float)a.D);
    const float m0 = gn_block_sum(t, red) / ((float)a.S * (float)a.D);
    float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float c = (int)(threadIdx.x + i * blockDim.x) < total ? v[i][j] - m0 : 0.0f;
            t1 += c;
            t2 += c * c;
        }
    if constexpr (sizeof(IO) == 4) {
        gn_block_sum2(t1, t2, red);
    } else {
        t1 = 0.0f;
        t2 = gn_block_sum(t2, red);
    }
    const float off = t1 * inv, mu = m0 + off;
    const float rs = rsqrtf(variance(t2 * inv, off) + a.eps);
    if (a.mean && threadIdx.x == 0) {
        a.mean[id] = mu;
        a.rstd[id] = rs;
    }
    IO *y = (IO *)a.y + n * a.sy.s0 + g * a.sy.s2;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = threadIdx.x + i * blockDim.x;
        if (e >= total) break;
        const int p = position(e), d = (e - p * rv) * V;
        float w[V], b[V];
        load_w<V>(a.w, (size_t)g * a.D + d, true, 1.0f, w);
        load_w<V>(a.b, (size_t)g * a.D + d, true, 0.0f, b);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = act_f<ACT>((v[i][j] - mu) * rs * w[j] + b[j]);
        store_v<IO, V>(y + p * a.sy.s1 + d, v[i]);
    }
}

// ---- split over positions
//
// The S positions of a sample are cut into pblk blocks of plen.  A workgroup is
// tx channel vectors x 256 / tx positions.  Partials: ws [N][pblk][2][C].
struct PosGeom {
    int tx, cblk;    // channel vectors of a workgroup, blocks of them
    int plen, pblk;  // positions of a block, blocks
};

// offset of channel c of sample n's first position
__device__ __forceinline__ long long gn_at(const Strides &st, int D, int n, int c) {
    const int g = c / D;
    return n * st.s0 + g * st.s2 + (c - g * D);
}

// Two values of each of V channels' groups (p0, p1 [.][G], `at` the first group's)
template <int V>
__device__ __forceinline__ void load_groups(const float *p0, const float *p1, size_t at, int c, int D, float *x0, float *x1) {
    if (D % V == 0) {  // one group for the whole vector
        const float a = p0[at + c / D], b = p1[at + c / D];
#pragma unroll
        for (int i = 0; i < V; ++i) x0[i] = a, x1[i] = b;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int g = (c + i) / D;
            x0[i] = p0[at + g];
            x1[i] = p1[at + g];
        }
    }
}

// sum over the rows ty of a workgroup, for V channels of each tx
template <int V>
__device__ __forceinline__ void gn_reduce(float *red, float *t, int tx, int TX, int ty, int TY) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        __syncthreads();
        red[threadIdx.x] = t[i];
        __syncthreads();
        for (int m = TY >> 1; m > 0; m >>= 1) {
            if (ty < m) red[threadIdx.x] += red[threadIdx.x + m * TX];
            __syncthreads();
        }
        t[i] = red[tx];
    }
}
// ... of two sets of values at once; red [512]
template <int V>
__device__ __forceinline__ void gn_reduce2(float *red, float *t, float *u, int tx, int TX, int ty, int TY) {
    float *red1 = red + 256;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        __syncthreads();
        red[threadIdx.x] = t[i];
        red1[threadIdx.x] = u[i];
        __syncthreads();
        for (int m = TY >> 1; m > 0; m >>= 1) {
            if (ty < m) {
                red[threadIdx.x] += red[threadIdx.x + m * TX];
                red1[threadIdx.x] += red1[threadIdx.x + m * TX];
            }
            __syncthreads();
        }
        t[i] = red[tx];
        u[i] = red1[tx];
    }
}

// BWD false: mean and centred sum of squares of each channel of the block;
// true: sum dz and sum dz xh.
template <typename IO, int V, int ACT, bool BWD>
__global__ __launch_bounds__(256) void gn_channel_kernel(GnArgs a, PosGeom q, int block0) {
    __shared__ float red[!BWD && sizeof(IO) == 4 ? 512 : 256];
    const int C = a.G * a.D;
    const int tx = threadIdx.x % q.tx, ty = threadIdx.x / q.tx, TY = 256 / q.tx;
    const int block = block0 + blockIdx.x, cb = block % q.cblk;
    const int pb = block / q.cblk % q.pblk, o = block / q.cblk / q.pblk;
    const int c = (cb * q.tx + tx) * V;
    const bool ok = c < C;
    const int p0 = pb * q.plen, p1 = min(p0 + q.plen, a.S);
    float t[2][V];
#pragma unroll
    for (int i = 0; i < V; ++i) t[0][i] = t[1][i] = 0.0f;
    float mu[V], rs[V], w[V], bb[V], cnt = 0.0f;
    if (ok) {
        const IO *x = (const IO *)a.x + gn_at(a.sx, a.D, o, c);
        if constexpr (!BWD) {
            // Running mean and centred sum (Welford): sums of x - c and its square
            // cancel for any c that may be an outlier, by 5% of the variance for one
            // of 10^5 deviations as the first of 4096 positions.
#pragma unroll 4
            for (int p = p0 + ty; p < p1; p += TY) {
                float v[V];
                load_v<IO, V>(x + p * a.sx.s1, v);
                cnt += 1.0f;
                const float part = __builtin_amdgcn_rcpf(cnt);  // 1 exactly for the first
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = v[i] - t[0][i];
                    t[0][i] += d * part;
                    t[1][i] += d * (v[i] - t[0][i]);
                }
            }
        } else {
            const IO *dy = (const IO *)a.dy + gn_at(a.sdy, a.D, o, c);
            if (a.seq) load_groups<V>(a.mean, a.rstd, (size_t)o * a.G, c, a.D, mu, rs);
            load_w<V>(a.w, c, true, 1.0f, w);
            load_w<V>(a.b, c, true, 0.0f, bb);
#pragma unroll 2
            for (int p = p0 + ty; p < p1; p += TY) {
                float v[V], u[V];
                load_v<IO, V>(x + p * a.sx.s1, v);
                load_v<IO, V>(dy + p * a.sdy.s1, u);
                // each position has its own statistics
                if (!a.seq) load_groups<V>(a.mean, a.rstd, ((size_t)o * a.S + p) * a.G, c, a.D, mu, rs);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = (v[i] - mu[i]) * rs[i];
                    const float dz = u[i] * act_d<ACT>(xh * w[i] + bb[i]);
                    t[0][i] += dz;
                    t[1][i] += dz * xh;
                }
            }
        }
    }
    if constexpr (BWD) {
        gn_reduce<V>(red, t[0], tx, q.tx, ty, TY);
        gn_reduce<V>(red, t[1], tx, q.tx, ty, TY);
    } else {
        // the rows' means joined, then their centred sums about that, and how far
        // the rows' means still lie from it
        float m[V], off[V];
#pragma unroll
        for (int i = 0; i < V; ++i) m[i] = cnt * t[0][i];
        gn_reduce<V>(red, m, tx, q.tx, ty, TY);
        const float n = (float)(p1 - p0);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            m[i] /= n;
            const float d = t[0][i] - m[i];
            off[i] = cnt * d;
            t[1][i] += cnt * d * d;
        }
        if constexpr (sizeof(IO) == 4) {
            gn_reduce2<V>(red, t[1], off, tx, q.tx, ty, TY);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                off[i] /= n;
                t[0][i] = m[i] + off[i];
                t[1][i] = n * variance(t[1][i] / n, off[i]);
            }
        } else {
            gn_reduce<V>(red, t[1], tx, q.tx, ty, TY);
#pragma unroll
            for (int i = 0; i < V; ++i) t[0][i] = m[i];
        }
    }
    if (ty == 0 && ok) {
        float *ws = a.ws + ((size_t)o * q.pblk + pb) * 2 * C + c;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (BWD) {
                ws[C + i] = t[0][i];   // [0] is dw's sum, [1] db's, as in the row kernel
                ws[i] = t[1][i];
            } else {
                ws[i] = t[0][i];
                ws[C + i] = t[1][i];
            }
        }
    }
}

// Sum over r of channel c's two partials: 16 channels x TY rows of a workgroup.
template <int TY>
__device__ __forceinline__ void gn_wsum(const float *ws, float *dw, float *db, int C, int rblk, int cblk, int which) {
    __shared__ float red[TY][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int c = cblk * 16 + tx;
    float *out = which ? db : dw;
    if (!out) return;
    float t = 0.0f;
    if (c < C)
#pragma unroll 4
        for (int r = ty; r < rblk; r += TY) t += ws[((size_t)r * 2 + which) * C + c];
    red[ty][tx] = t;
    __syncthreads();
    for (int m = TY / 2; m > 0; m >>= 1) {
        if (ty < m) red[ty][tx] += red[ty + m][tx];
        __syncthreads();
    }
    if (ty == 0 && c < C) out[c] = red[0][tx];
}

// dw, db: sums of the partials [rblk][2][C] in ws over rblk; blockIdx.y is 0 for dw.
__global__ __launch_bounds__(1024) void gn_wsum_kernel(const float *ws, float *dw, float *db, int C, int rblk, int block0) {
    gn_wsum<64>(ws, dw, db, C, rblk, block0 + blockIdx.x, blockIdx.y);
}

// One workgroup per (sample, group).  Forward: mean and rstd from the channels'
// means and centred sums.  Backward: mean(u) and mean(u xh).  Written to
// out0, out1 [N][G].  The workgroups past those sum dw and db.
// Threads: tx channels x 1024 / tx blocks of positions.
template <bool BWD>
__global__ __launch_bounds__(1024) void gn_combine_kernel(GnArgs a, PosGeom q, float *out0, float *out1, int block0) {
    __shared__ float red[32];
    const int C = a.G * a.D;
    const int block = block0 + blockIdx.x;
    if (BWD && block >= a.N * a.G) {
        const int i = block - a.N * a.G;
        gn_wsum<64>(a.ws, a.dw, a.db, C, a.N * q.pblk, i >> 1, i & 1);
        return;
    }
    const int g = block % a.G, o = block / a.G;
    const int sh = a.D >= 64 ? 6 : a.D >= 16 ? 4 : 2;  // log2 of the channels side by side
    const int tx = threadIdx.x & ((1 << sh) - 1), ty = threadIdx.x >> sh, TY = 1024 >> sh;
    const float *ws = a.ws + (size_t)o * q.pblk * 2 * C + (size_t)g * a.D;
    const float total = (float)a.D * (float)a.S;
    auto rows = [&](int pb) { return (float)(min(a.S, (pb + 1) * q.plen) - pb * q.plen); };
    float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f;
    for (int d = tx; d < a.D; d += 1 << sh) {
        const float w = BWD && a.w ? a.w[g * a.D + d] : 1.0f;
#pragma unroll 4
        for (int pb = ty; pb < q.pblk; pb += TY) {
            const float *r = ws + (size_t)pb * 2 * C + d;
            if constexpr (BWD) {
                s0 += w * r[C];
                s1 += w * r[0];
            } else {
                s0 += r[0] * rows(pb);
            }
        }
    }
    const float m0 = gn_block_sum(s0, red) / total;
    if constexpr (!BWD) {
        for (int d = tx; d < a.D; d += 1 << sh)
#pragma unroll 4
            for (int pb = ty; pb < q.pblk; pb += TY) {
                const float *r = ws + (size_t)pb * 2 * C + d;
                const float c = r[0] - m0;
                s1 += r[C] + c * c * rows(pb);
                s2 += c * rows(pb);
            }
        gn_block_sum2(s1, s2, red);
        if (threadIdx.x == 0) {
            out0[block] = m0 + s2 / total;
            out1[block] = rsqrtf(variance(s1 / total, s2 / total) + a.eps);
        }
    } else {
        const float m1 = gn_block_sum(s1, red) / total;
        if (threadIdx.x == 0) {
            out0[block] = m0;
            out1[block] = m1;
        }
    }
}

template <typename IO, int V, int ACT, bool BWD>
__global__ __launch_bounds__(256) void gn_apply_kernel(GnArgs a, PosGeom q, const float *in0, const float *in1, int block0) {
    const int C = a.G * a.D;
    const int tx = threadIdx.x % q.tx, ty = threadIdx.x / q.tx, TY = 256 / q.tx;
    const int block = block0 + blockIdx.x, cb = block % q.cblk;
    const int pb = block / q.cblk % q.pblk, o = block / q.cblk / q.pblk;
    const int c = (cb * q.tx + tx) * V;
    if (c >= C) return;
    const int p0 = pb * q.plen, p1 = min(p0 + q.plen, a.S);
    float mu[V], rs[V], w[V], bb[V], c1[V], c2[V];
    if constexpr (BWD) {
        load_groups<V>(a.mean, a.rstd, (size_t)o * a.G, c, a.D, mu, rs);
        load_groups<V>(in0, in1, (size_t)o * a.G, c, a.D, c1, c2);
    } else {
        load_groups<V>(in0, in1, (size_t)o * a.G, c, a.D, mu, rs);
    }
    load_w<V>(a.w, c, true, 1.0f, w);
    load_w<V>(a.b, c, true, 0.0f, bb);
    const IO *x = (const IO *)a.x + gn_at(a.sx, a.D, o, c);
    const IO *dy = BWD ? (const IO *)a.dy + gn_at(a.sdy, a.D, o, c) : nullptr;
    IO *y = (IO *)a.y + gn_at(a.sy, a.D, o, c);
#pragma unroll 4
    for (int p = p0 + ty; p < p1; p += TY) {
        float v[V], u[V];
        load_v<IO, V>(x + p * a.sx.s1, v);
        if constexpr (BWD) load_v<IO, V>(dy + p * a.sdy.s1, u);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float xh = (v[i] - mu[i]) * rs[i], z = xh * w[i] + bb[i];
            if constexpr (BWD)
                v[i] = rs[i] * (u[i] * act_d<ACT>(z) * w[i] - c1[i] - xh * c2[i]);
            else
                v[i] = act_f<ACT>(z);
        }
        store_v<IO, V>(y + p * a.sy.s1, v);
    }
}

// ---- plans

// HIP takes fewer than 2^32 threads a launch: launch(workgroups, first one) for
// runs of at most 2^31 threads, until one fails.
template <typename F>
hipError_t in_runs(long long blocks, int threads, F launch) {
    const long long run = (1ll << 31) / threads;
    for (long long first = 0; first < blocks; first += run) {
        launch((unsigned)(blocks - first < run ? blocks - first : run), (int)first);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

int pow2_at_least(int x) {
    int p = 1;
    while (p < x) p <<= 1;
    return p;
}

int log2_at_least(int x) {
    int p = 0;
    while ((1 << p) < x) ++p;
    return p;
}

// lanes' vectors of a row held in registers: 1, 4 or 0 (the row is too long)
int row_vectors(int D, int V) {
    const int k = (D + 64 * V - 1) / (64 * V);
    return k <= 1 ? 1 : k <= 4 ? 4 : 0;
}

// element count of a 16-byte vector if every row of channels starts aligned
// and no vector crosses a group boundary that memory does not continue over
bool vec_ok(const GnArgs &a, int V) {
    const Strides *st[] = {&a.sx, &a.sy, &a.sdy};
    const int n = a.dy ? 3 : 2;
    for (int i = 0; i < n; ++i) {
        const bool flat = st[i]->s2 == a.D || a.G == 1;
        if (!(a.D % V == 0 || (a.seq && flat && ((long long)a.G * a.D) % V == 0))) return false;
        if ((a.N > 1 && st[i]->s0 % V) || (a.S > 1 && st[i]->s1 % V)) return false;
        if (a.D % V == 0 && a.G > 1 && st[i]->s2 % V) return false;
    }
    return true;
}

RowGeom row_geom(int N, int S, int G, int D, int V, int K, bool token_major, bool bwd) {
    RowGeom q;
    const int vecs = (D + V - 1) / V;
    q.lpr = K > 1 ? 6 : log2_at_least(vecs);
    // neighbouring groups side by side where they are neighbours in memory
    q.gp = 0;
    while (token_major && q.gp + 1 + q.lpr <= 6 && G % (2 << q.gp) == 0) ++q.gp;
    q.gblk = G >> q.gp;
    q.div = ~0ull / (unsigned)S + 1;  // 0 for S = 1, which does not use it
    const long long rows = (long long)N * S;
    const long long per = 4 * (64 >> (q.lpr + q.gp));
    long long want = (rows + per - 1) / per;
    // A workgroup loads its weights once, so it should not be too short, and the
    // backward leaves one set of partials for each block of positions.  32768
    // rows of 8 heads of 512, bfloat16: 8192 workgroups 115 us, 1024 take 148;
    // the backward with 1024 194 us, 2048 take 203.
    const long long cap = ((bwd ? 1024 : 8192) + q.gblk - 1) / q.gblk;
    if (want > cap) want = cap;
    q.rblk = (int)want;
    return q;
}

PosGeom pos_geom(int N, int S, int C, int V) {
    PosGeom q;
    const int cv = (C + V - 1) / V;
    const int p = pow2_at_least(cv);
    q.tx = p > 64 ? 64 : p;
    // narrower where an eighth of the threads would have no channels
    while (q.tx > 16 && ((cv + q.tx - 1) / q.tx * q.tx - cv) * 8 > cv) q.tx >>= 1;
    q.cblk = (cv + q.tx - 1) / q.tx;
    // About four workgroups a compute unit, at least 32 positions a block: the
    // backward of 8192 positions of 2048 channels 42 us and of 320 channels 21;
    // eight workgroups of at least 16 positions take 50 and 25.
    const long long per = (long long)N * q.cblk;
    long long want = (1024 + per - 1) / per;
    const long long most = (S + 31) / 32;
    if (want > most) want = most;
    q.plen = (int)((S + want - 1) / want);
    q.pblk = (S + q.plen - 1) / q.plen;
    return q;
}

// Groups that a workgroup's registers hold need one launch for the forward: 8 x 32
// groups of 1024 x 10 take 14.5 us, over blocks of positions 19.6.
bool group_fits(int S, int D) { return (long long)S * D <= 16384; }

template <typename IO, int V, int ACT>
hipError_t launch_group(const GnArgs &a, hipStream_t s) {
    const int n = a.S * a.D;
    const long long groups = (long long)a.N * a.G;
    // 8 values a thread, 16 where 1024 threads need it
    if (n > 8192)
        return in_runs(groups, 1024, [&](unsigned grid, int first) {
            gn_group_kernel<IO, V, 16, ACT><<<grid, 1024, 0, s>>>(a, first);
        });
    const int th = ((n + 7) / 8 + 63) / 64 * 64;
    return in_runs(groups, th, [&](unsigned grid, int first) {
        gn_group_kernel<IO, V, 8, ACT><<<grid, th, 0, s>>>(a, first);
    });
}

// the channels' sums over each block of positions
template <typename IO, int V, int ACT, bool BWD>
hipError_t launch_channel(const GnArgs &a, const PosGeom &q, hipStream_t s) {
    return in_runs((long long)q.cblk * q.pblk * a.N, 256, [&](unsigned grid, int first) {
        gn_channel_kernel<IO, V, ACT, BWD><<<grid, 256, 0, s>>>(a, q, first);
    });
}

// dw and db from rblk sets of partials
hipError_t launch_wsum(const GnArgs &a, int rblk, hipStream_t s) {
    const int C = a.G * a.D;
    return in_runs((C + 15) / 16, 2 * 1024, [&](unsigned grid, int first) {
        gn_wsum_kernel<<<dim3(grid, 2), 1024, 0, s>>>(a.ws, a.dw, a.db, C, rblk, first);
    });
}

template <typename IO, int V, int ACT, bool BWD>
hipError_t launch_blocks(const GnArgs &a, const PosGeom &q, float *m0, float *m1, hipStream_t s) {
    hipError_t e = launch_channel<IO, V, ACT, BWD>(a, q, s);
    if (e != hipSuccess) return e;
    const long long sums = a.dw || a.db ? (a.G * a.D + 15) / 16 * 2 : 0;
    e = in_runs((long long)a.N * a.G + sums, 1024, [&](unsigned grid, int first) {
        gn_combine_kernel<BWD><<<grid, 1024, 0, s>>>(a, q, m0, m1, first);
    });
    if (e != hipSuccess) return e;
    return in_runs((long long)q.cblk * q.pblk * a.N, 256, [&](unsigned grid, int first) {
        gn_apply_kernel<IO, V, ACT, BWD><<<grid, 256, 0, s>>>(a, q, m0, m1, first);
    });
}

template <typename IO, int V, int ACT>
hipError_t launch_seq(const GnArgs &a, hipStream_t s) {
    const int C = a.G * a.D;
    const PosGeom q = pos_geom(a.N, a.S, C, V);
    float *m0 = a.ws + (size_t)a.N * q.pblk * 2 * C, *m1 = m0 + (size_t)a.N * a.G;
    if (a.dy) return launch_blocks<IO, V, ACT, true>(a, q, m0, m1, s);
    if (group_fits(a.S, a.D)) {
        // vectors only where none crosses into the next group
        if (V == 1 || a.D % V == 0) return launch_group<IO, V, ACT>(a, s);
        return launch_group<IO, 1, ACT>(a, s);
    }
    return launch_blocks<IO, V, ACT, false>(a, q, a.mean ? a.mean : m0, a.mean ? a.rstd : m1, s);
}

template <typename IO, int V, int ACT>
hipError_t launch_long_row(const GnArgs &a, hipStream_t s) {
    const long long rows = (long long)a.N * a.S * a.G;
    const dim3 grid((unsigned)(rows < 16384 ? rows : 16384));
    if (!a.dy)
        gn_long_row_kernel<IO, V, ACT, false><<<grid, 256, 0, s>>>(a, rows);
    else
        gn_long_row_kernel<IO, V, ACT, true><<<grid, 256, 0, s>>>(a, rows);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !(a.dw || a.db)) return e;
    const PosGeom q = pos_geom(a.N, a.S, a.G * a.D, V);
    e = launch_channel<IO, V, ACT, true>(a, q, s);
    return e != hipSuccess ? e : launch_wsum(a, a.N * q.pblk, s);
}

template <typename IO, int V, int K, int ACT>
hipError_t launch_row(const GnArgs &a, hipStream_t s) {
    const RowGeom q = row_geom(a.N, a.S, a.G, a.D, V, K, a.sx.s2 < a.sx.s1, a.dy != nullptr);
    const hipError_t e = in_runs((long long)q.gblk * q.rblk, 256, [&](unsigned grid, int first) {
        if (!a.dy)
            gn_row_kernel<IO, V, K, ACT, false><<<grid, 256, 0, s>>>(a, q, first);
        else
            gn_row_kernel<IO, V, K, ACT, true><<<grid, 256, 0, s>>>(a, q, first);
    });
    if (e != hipSuccess || !(a.dw || a.db)) return e;
    return launch_wsum(a, q.rblk, s);
}

template <typename IO, int ACT>
hipError_t launch_io(const GnArgs &a, hipStream_t s) {
    constexpr int VV = 16 / (int)sizeof(IO);
    const bool vec = vec_ok(a, VV);
    if (!a.seq) {
        const int k = row_vectors(a.D, vec ? VV : 1);
        if (vec && k == 1) return launch_row<IO, VV, 1, ACT>(a, s);
        if (vec && k == 4) return launch_row<IO, VV, 4, ACT>(a, s);
        if (!vec && k == 1) return launch_row<IO, 1, 1, ACT>(a, s);
        if (!vec && k == 4) return launch_row<IO, 1, 4, ACT>(a, s);
        return vec ? launch_long_row<IO, VV, ACT>(a, s) : launch_long_row<IO, 1, ACT>(a, s);
    }
    return vec ? launch_seq<IO, VV, ACT>(a, s) : launch_seq<IO, 1, ACT>(a, s);
}

template <typename IO>
hipError_t launch_act(const GnArgs &a, hipStream_t s) {
    if (a.act == 1) return launch_io<IO, 1>(a, s);
    if (a.act == 2) return launch_io<IO, 2>(a, s);
    return launch_io<IO, 0>(a, s);
}

}  // namespace

// Enough for either vector width and either order of the strides, which the query does not know.
size_t groupnorm_workspace_floats(int N, int S, int G, int D, int seq, int io_bf16, int bwd) {
    size_t need = 0;
    const int C = G * D;
    for (int V : {io_bf16 ? 8 : 4, 1}) {
        const int k = seq ? 0 : row_vectors(D, V);
        size_t f = 0;
        if (k) {
            if (bwd)
                for (bool tm : {false, true}) {
                    const size_t r = (size_t)row_geom(N, S, G, D, V, k, tm, true).rblk;
                    f = r * 2 * C > f ? r * 2 * C : f;
                }
        } else if (bwd || (seq && !group_fits(S, D))) {
            const PosGeom q = pos_geom(N, S, C, V);
            f = (size_t)N * q.pblk * 2 * C + (seq ? 2 * (size_t)N * G : 0);
        }
        need = f > need ? f : need;
    }
    return need;
}

hipError_t launch_groupnorm(const GnArgs &a, int io_bf16, hipStream_t s) {
    return io_bf16 ? launch_act<bf16>(a, s) : launch_act<float>(a, s);
}

}  // namespace mlstm
