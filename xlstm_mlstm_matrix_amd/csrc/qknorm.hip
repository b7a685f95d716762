// qknorm.hip -- norm of each head's queries and keys and their rotation by the
// token's position, forward and backward.
//
// A row x of d channels: r = 1 / sqrt(mean x^2 + eps) (or of the sum, or 1),
// z = w x r, and channels a, b of each pair turned by the angle position * freq:
// y = A (z_a c - z_b s, z_b c + z_a s).  Backward, with u the row dy turned back:
// dw = sum over rows of u x r, dx = r (u w - (x r) (r sum u w x) / n).
//
// Each row is read once and written once, nothing else is large: the pass is
// bound by HBM (2 x 134 MB of 128 bfloat16 channels: 43 us, 6.2 TB/s with the inputs
// partly in the cache, 58 us cold; gradients with rotation, 252 MB: 47 us, 5.4 TB/s).  A
// row belongs to a few lanes of a wavefront; a lane holds both channels of its pairs, so that rotating costs no exchange, and the row's sums are
// the only thing that crosses lanes.  The heads of a token are walked by the
// same lanes, which keep the token's sines and cosines in registers.
#include "ops.hpp"

namespace mlstm {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 1024;  // of a backward: rows of partial weight gradients
constexpr int kMaxGrid = 1 << 22;  // of any call: HIP takes fewer than 2^32 threads a launch

struct QkPlan {
    int lpr;            // lanes of a row, a power of two
    int units, rot_units;
    int per[2];         // heads of a tensor that a group of lanes walks for one token
    int nblk_heads[2];  // groups of heads
    long long items[2];
    int blocks;         // workgroups for each tensor
};

template <typename IO, int V>
struct Raw {
    typedef IO type __attribute__((ext_vector_type(V)));
};
template <typename IO>
struct Raw<IO, 1> {
    typedef IO type;
};
template <typename IO, int V>
__device__ __forceinline__ typename Raw<IO, V>::type load_row(const IO *p, bool ok) {
    typename Raw<IO, V>::type v = {};
    if (ok) v = *(const typename Raw<IO, V>::type *)p;
    return v;
}
template <typename IO, int V>
__device__ __forceinline__ void unpack(const typename Raw<IO, V>::type &v, float *x) {
    if constexpr (V == 1) {
        x[0] = to_f(v);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = to_f((IO)v[j]);
    }
}
template <typename IO, int V>
__device__ __forceinline__ void store_row(IO *p, bool ok, const float *x) {
    if (!ok) return;
    if constexpr (V == 1) {
        *p = from_f<IO>(x[0]);
    } else {
        typedef IO vec __attribute__((ext_vector_type(V)));
        vec v;
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = from_f<IO>(x[j]);
        *(vec *)p = v;
    }
}

// Cosine and sine of position * freq.  The angle is a double product, good to
// 2^-52 of itself, and only its distance from a whole turn goes on in float32: half a turn
// to 2^-25, 1e-7 radians, as much as the sine's own rounding (sines of the double
// angle would leave outputs at 6.4e-8 of a float32 row where these are 7.4e-8).
__device__ __forceinline__ void turn(int pos, float freq, float amp, float &c, float &s) {
    const double t = (double)pos * (double)freq * 0.15915494309189533577;  // 1 / (2 pi)
    const float half = (float)(2.0 * (t - rint(t)));
    sincospif(half, &s, &c);
    c *= amp;
    s *= amp;
}

// V channels of a vector, UPL units (two vectors) of a row for each lane.  Queries and keys
// are workgroups of their own (blockIdx.y): one tensor's weights and sums at a
// time are in registers.
template <typename IO, int V, int UPL, bool PAIRS, bool BWD>
__global__ __launch_bounds__(kThreads) void qk_kernel(QkArgs a, QkPlan p) {
    constexpr int W = 2 * V;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int sub = lane & (p.lpr - 1);
    const int d = a.d, nf = a.nf;
    int off[UPL][2];
    bool ok[UPL][2], rot[UPL];
#pragma unroll
    for (int i = 0; i < UPL; ++i) {
        const int u = sub + i * p.lpr;
        rot[i] = u < p.rot_units;
        if (rot[i]) {
            off[i][0] = PAIRS ? u * W : u * V;
            off[i][1] = PAIRS ? u * W + V : nf + u * V;
        } else {
            off[i][0] = 2 * nf + (u - p.rot_units) * W;
            off[i][1] = off[i][0] + V;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) ok[i][k] = u < p.units && off[i][k] < d;
    }
    // the pair (ia(j), ib(j)) of a unit's W channels.  Channels that are not rotated are left alone, not
    // turned by 0: 0 times an infinite neighbour is a NaN.
    const auto ia = [](int j) { return PAIRS ? 2 * j : j; };
    const auto ib = [](int j) { return PAIRS ? 2 * j + 1 : V + j; };
    const int ti = blockIdx.y;
    float dw[UPL][W], w[UPL][W];
#pragma unroll
    for (int i = 0; i < UPL; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) {
            dw[i][j] = 0.0f;
            w[i][j] = a.w[ti] && ok[i][j / V] ? a.w[ti][off[i][j / V] + j % V] : 1.0f;
        }
    const float count = a.norm == 1 ? (float)d : 1.0f;
    const int groups = kThreads / p.lpr;  // of lanes in a workgroup
    for (long long item = (long long)blockIdx.x * groups + threadIdx.x / p.lpr; item < p.items[ti];
         item += (long long)gridDim.x * groups) {
        const int n = (int)(item / p.nblk_heads[ti]), hb = (int)(item % p.nblk_heads[ti]);
        const int b = n / a.T, t = n % a.T;
        float c[UPL][V], s[UPL][V];
#pragma unroll
        for (int i = 0; i < UPL; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) c[i][j] = 1.0f, s[i][j] = 0.0f;
        if (nf > 0) {
            const int pos = a.pos ? a.pos[n] : t;
#pragma unroll
            for (int i = 0; i < UPL; ++i)
                if (rot[i])
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        turn(pos, a.freq[(sub + i * p.lpr) * V + j], a.amp, c[i][j], s[i][j]);
        }
        const int first = hb * p.per[ti], last = min(first + p.per[ti], a.H[ti]);
        {
            const IO *xr = (const IO *)a.x[ti] + b * a.sx[ti].s0 + t * a.sx[ti].s2;
            const IO *gr = BWD ? (const IO *)a.dy[ti] + b * a.sdy[ti].s0 + t * a.sdy[ti].s2 : nullptr;
            IO *yr = (IO *)a.y[ti] + b * a.sy[ti].s0 + t * a.sy[ti].s2;
            // a head's row is on its way while the one before is computed
            typename Raw<IO, V>::type xn[UPL][2], gn[UPL][2];
            const auto fetch = [&](int h) {
#pragma unroll
                for (int i = 0; i < UPL; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        xn[i][k] = load_row<IO, V>(xr + h * a.sx[ti].s1 + off[i][k], ok[i][k]);
                        if constexpr (BWD) gn[i][k] = load_row<IO, V>(gr + h * a.sdy[ti].s1 + off[i][k], ok[i][k]);
                    }
            };
            fetch(first);
            for (int h = first; h < last; ++h) {
                float x[UPL][W], g[UPL][W];
                float ss = 0.0f, dot = 0.0f;
#pragma unroll
                for (int i = 0; i < UPL; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        unpack<IO, V>(xn[i][k], x[i] + k * V);
                        if constexpr (BWD) unpack<IO, V>(gn[i][k], g[i] + k * V);
                    }
                if (h + 1 < last) fetch(h + 1);
                if constexpr (BWD) {
#pragma unroll
                    for (int i = 0; i < UPL; ++i)
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float ya = g[i][ia(j)], yb = g[i][ib(j)];
                            g[i][ia(j)] = rot[i] ? c[i][j] * ya + s[i][j] * yb : ya;
                            g[i][ib(j)] = rot[i] ? c[i][j] * yb - s[i][j] * ya : yb;
                        }
                }
#pragma unroll
                for (int i = 0; i < UPL; ++i)
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        ss += x[i][j] * x[i][j];
                        if constexpr (BWD) dot += g[i][j] * w[i][j] * x[i][j];
                    }
                float r = 1.0f;
                if (a.norm != 0) {
                    for (int m = p.lpr >> 1; m > 0; m >>= 1) {
                        ss += __shfl_xor(ss, m);
                        if constexpr (BWD) dot += __shfl_xor(dot, m);
                    }
                    r = 1.0f / sqrtf(ss / count + a.eps);
                }
                // factors r one by one beside their x or u: r^3 alone leaves float32's range for rows
                // of 10^13 or of 10^-13
                const float back = dot * r / count;
#pragma unroll
                for (int i = 0; i < UPL; ++i) {
                    if constexpr (BWD) {
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            const float z = x[i][j] * r;
                            dw[i][j] += g[i][j] * z;
                            const float u = g[i][j] * w[i][j];
                            x[i][j] = a.norm != 0 ? r * (u - z * back) : u;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < W; ++j) x[i][j] = x[i][j] * r * w[i][j];
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float za = x[i][ia(j)], zb = x[i][ib(j)];
                            x[i][ia(j)] = rot[i] ? za * c[i][j] - zb * s[i][j] : za;
                            x[i][ib(j)] = rot[i] ? zb * c[i][j] + za * s[i][j] : zb;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        store_row<IO, V>(yr + h * a.sy[ti].s1 + off[i][k], ok[i][k], x[i] + k * V);
                }
            }
        }
    }
    if constexpr (BWD) {
        if (!a.dw[ti]) return;
        // rows of the workgroup together: its wavefronts in turn, in a fixed order
        __shared__ float sum[4][512];
#pragma unroll
        for (int i = 0; i < UPL; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float x = dw[i][j];
                for (int m = p.lpr; m < 64; m <<= 1) x += __shfl_xor(x, m);
                if (lane < p.lpr && ok[i][j / V]) sum[wave][off[i][j / V] + j % V] = x;
            }
        __syncthreads();
        for (int ch = threadIdx.x; ch < d; ch += kThreads)
            a.ws[((size_t)ti * gridDim.x + blockIdx.x) * d + ch] =
                (sum[0][ch] + sum[1][ch]) + (sum[2][ch] + sum[3][ch]);
    }
}

// partial weight gradients [tensor][block][d] -> dw: 16 channels a workgroup, 16
// threads a channel
__global__ __launch_bounds__(kThreads) void qk_weight_kernel(QkArgs a, int blocks) {
    __shared__ float sum[16][17];
    const int ti = blockIdx.y, ch = blockIdx.x * 16 + (threadIdx.x & 15), part = threadIdx.x >> 4;
    if (!a.dw[ti]) return;
    float x = 0.0f;
    if (ch < a.d) {
        const float *p = a.ws + (size_t)ti * blocks * a.d + ch;
        int r = part;
        // eight loads in flight: one at a time 1024 rows take 17 us
        for (; r + 16 * 7 < blocks; r += 16 * 8) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = p[(size_t)(r + 16 * i) * a.d];
#pragma unroll
            for (int i = 0; i < 8; ++i) x += y[i];
        }
        for (; r < blocks; r += 16) x += p[(size_t)r * a.d];
    }
    sum[part][threadIdx.x & 15] = x;
    __syncthreads();
    if (part == 0 && ch < a.d) {
#pragma unroll
        for (int m = 1; m < 16; ++m) x += sum[m][threadIdx.x & 15];
        a.dw[ti][ch] = x;
    }
}

int pow2_at_least(int x) {
    int p = 1;
    while (p < x) p <<= 1;
    return p;
}

template <typename IO, int V, int UPL, bool BWD>
hipError_t launch_v(const QkArgs &a, hipStream_t s) {
    QkPlan p{};
    p.rot_units = a.nf / V;
    p.units = p.rot_units + (a.d - 2 * a.nf + 2 * V - 1) / (2 * V);
    p.lpr = pow2_at_least((p.units + UPL - 1) / UPL);
    const long long tokens = (long long)a.B * a.T;
    // Heads of a token for one group of lanes: all of them where the tokens make enough
    // wavefronts, else fewer.  One wavefront a SIMD is enough for up to 48 MB: a token's turns are made
    // once and the next head's row hides the loads (cold inputs, 8 wavefronts / 1: 4096 tokens of 16 + 4
    // heads of 128, bfloat16, 21 MB, 22 / 15 us, backward 38 / 25; 1024 tokens 9.2 / 7.7 and 20 / 15).  More are in
    // flight from HBM with 8 (16384 tokens of 16 + 16 heads, 134 MB, no rotation: 58 / 76, backward 98 / 112;
    // 2 x 8192 tokens of 32 + 8 heads of 64, float32, 168 MB, rotated 72 / 82, backward 105 / 128), with 2
    // where bfloat16 rows are rotated (the same in bfloat16, 84 MB, 8 / 2 / 1: 42 / 39 / 48, backward
    // 73 / 64 / 72).  48 MB lies between what was measured.
    const long long bytes = tokens * (a.H[0] + a.H[1]) * a.d * (long long)sizeof(IO);
    const int waves = bytes <= 48ll << 20 ? 1 : a.nf > 0 && sizeof(IO) == 2 ? 2 : 8;
    const long long groups = waves * 1024ll * 64 / p.lpr;
    const long long split = tokens >= groups ? 1 : (groups + tokens - 1) / tokens;
    long long most = 0;
    for (int i = 0; i < 2; ++i) {
        const int heads = a.H[i];
        p.per[i] = (int)(split >= heads ? 1 : (heads + split - 1) / split);
        p.nblk_heads[i] = (heads + p.per[i] - 1) / p.per[i];
        p.items[i] = tokens * p.nblk_heads[i];
        most = p.items[i] > most ? p.items[i] : most;
    }
    const long long blocks = (most * p.lpr + kThreads - 1) / kThreads;
    const int limit = BWD ? kMaxBlocks : kMaxGrid;
    p.blocks = (int)(blocks > limit ? limit : blocks);
    const dim3 grid((unsigned)p.blocks, a.H[1] > 0 ? 2 : 1);
    if (a.pairs)
        qk_kernel<IO, V, UPL, true, BWD><<<grid, kThreads, 0, s>>>(a, p);
    else
        qk_kernel<IO, V, UPL, false, BWD><<<grid, kThreads, 0, s>>>(a, p);
    if (BWD && (a.dw[0] || a.dw[1]))
        qk_weight_kernel<<<dim3((unsigned)((a.d + 15) / 16), 2), kThreads, 0, s>>>(a, p.blocks);
    return hipGetLastError();
}

template <typename IO, bool BWD>
hipError_t launch_io(const QkArgs &a, hipStream_t s) {
    constexpr int V = 16 / (int)sizeof(IO);
    // whole vectors: pairs and the rest begin and end on 16 bytes, and so do all rows; else single
    // channels (bfloat16, 4 x 4096 tokens of 16 + 4 heads: 96 channels with 36 pairs 49 us, 2.6 TB/s, backward
    // 76; 128 with 64 pairs by vectors 35, 4.8 TB/s, backward 56)
    bool vec = a.d % V == 0 && a.nf % V == 0;
    for (int i = 0; i < 2; ++i) {
        if (a.H[i] == 0) continue;
        const void *ptr[3] = {a.x[i], a.y[i], BWD ? a.dy[i] : nullptr};
        const Strides *st[3] = {&a.sx[i], &a.sy[i], &a.sdy[i]};
        for (int j = 0; j < (BWD ? 3 : 2); ++j)
            vec = vec && (uintptr_t)ptr[j] % 16 == 0 && st[j]->s0 % V == 0 && st[j]->s1 % V == 0 && st[j]->s2 % V == 0;
    }
    if (vec) return launch_v<IO, V, 1, BWD>(a, s);
    return launch_v<IO, 1, 4, BWD>(a, s);
}

}  // namespace

size_t qknorm_workspace_floats(int B, int H, int Hk, int T, int d) {
    // a workgroup holds at least one (token, head) item
    const long long rows = (long long)B * T * (H + Hk);
    return (size_t)2 * (size_t)(rows < kMaxBlocks ? rows : kMaxBlocks) * d;
}

hipError_t launch_qknorm(const QkArgs &a, int io_bf16, hipStream_t s) {
    if (a.dy[0]) return io_bf16 ? launch_io<bf16, true>(a, s) : launch_io<float, true>(a, s);
    return io_bf16 ? launch_io<bf16, false>(a, s) : launch_io<float, false>(a, s);
}

}  // namespace mlstm
