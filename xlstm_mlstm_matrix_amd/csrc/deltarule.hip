// deltarule.hip -- the gated delta rule over whole sequences, in chunks of L = 32
// tokens on the matrix cores.
//
// In a chunk that starts from the state S, with G the running sum of its log
// decays, M_ij = e^{G_i - G_j} (j <= i), N = M o (K K^T) below the diagonal and
// P = scale M o (Q K^T) up to it:
//   X = T' (V - e^G o (K S)),  T' = (I + N beta)^-1,  U = beta o X,
//   O = scale e^G o (Q S) + P U,
//   S <- e^{G_L} S + K^T (e^{G_L - G} o U),
// X the values that were missing from the memory and U what is written.  What does not
// need S is computed first, for all chunks at once (prep_kernel: T', P, the decays, laid
// out as the operands that they become).  Then a workgroup owns a block of value
// columns of one head, which never mix, and walks its chunks; a wavefront holds
// all d_qk rows of 16 NCT columns of S in registers (float32, accumulator layout).
//
// Each product's result is, lane by lane, an operand of the next one: K S has a
// lane's column and the tokens 16 t + 4 g4 + r, which are the inner index of T'
// (V - ...); its result those of P U, taken as U^T P^T, and of the update.
//
// Exponents are differences of running sums, which lose what two large sums
// share; so the sums are taken in 64 bits and kept as a multiple of 2^-6, whose
// differences are exact, and a float32 rest.  -inf is an ordinary value.
//
// Roundings (bfloat16 I/O), as in linattn.hip: the copy of S that meets Q has two
// parts (8 + 8 bits), and so have P and the U that meets it: each is off by 2^-16
// where the output's own rounding is off by 2^-8.  Where the state is handed out,
// all that leads to it has three parts (24 bits): the copy of S that meets K, T', its
// right side, the update's e^{G_L - G} U; else two.  S itself, decays and sums
// are float32.  float32 I/O runs on the float32 MFMA without further rounding.
#include <type_traits>

#include "chunk_tiles.hpp"

namespace mlstm {

namespace {

// ---- records: what a chunk knows without the state

// Operand fragments: tile t holds rows 16 t + l16, slot e of lane group g4 is
// token 16 (e / 4) + 4 g4 + e % 4.  Then float vectors over the tokens: e^{G_i},
// e^{G_L - G_i}, beta_i.
template <typename IO>
struct Rec {
    typedef typename Types<IO>::Frag Frag;
    static constexpr int TP = sizeof(IO) == 2 ? 3 : 1, PP = sizeof(IO) == 2 ? 2 : 1;  // parts of T' and P
    static constexpr int FRAG = 64 * (int)sizeof(Frag);                              // bytes of a tile's part
    static constexpr int P = 2 * TP * FRAG, VEC = P + 2 * PP * FRAG, EG = 0, REST = 1, BETA = 2;
    static constexpr int BYTES = (VEC + 3 * L * 4 + 1023) / 1024 * 1024;
};

__host__ __device__ __forceinline__ long long chunks(int T) { return ((long long)T + L - 1) / L; }

__device__ __forceinline__ int tokens(const DeltaArgs &a, int b) {
    return a.lengths ? max(0, min(a.lengths[b], a.T)) : a.T;
}

// Log decay of a token in base 2; below -1024 (e^g is 0 in any case) it stays there, so
// that a chunk's sum stays below 2^15.  NaN stays.
__device__ __forceinline__ float gate_log2(float g) {
    const float x = g * 1.4426950408889634f;
    return x < -1024.0f ? -1024.0f : x;
}

template <int PARTS>
__device__ __forceinline__ void split8(const float *x, bf16x8 *f) {
#pragma unroll
    for (int p = 0; p < 4; ++p) split2<PARTS, false>(x[2 * p], x[2 * p + 1], f, p);
}
template <int PARTS>
__device__ __forceinline__ void split8(const float *x, f32x8 *f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[0][e] = x[e];
}

// 8 elements of a row at p (zeros where not ok)
__device__ __forceinline__ bf16x8 row8(const bf16 *p, bool ok) {
    bf16x8 v = {};
    if (ok) v = *(const bf16x8 *)p;
    return v;
}
__device__ __forceinline__ f32x8 row8(const float *p, bool ok) {
    f32x8 v = {};
    if (ok) {
        const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
    }
    return v;
}

constexpr int kPrepWaves = 4, kLd = 36;  // wavefronts of a workgroup, row of a matrix in LDS

// One wavefront a chunk.  The inverse goes by blocks of 16 x 16: those on the diagonal
// row by row (a lane a column), which no cancellation hurts where keys are alike,
// then T'_21 = -T'_22 (N beta)_21 T'_11 on the float32 MFMA.
template <typename IO>
__global__ __launch_bounds__(64 * kPrepWaves) void prep_kernel(DeltaArgs a, char *rec, long long total) {
    using R = Rec<IO>;
    using Frag = typename Types<IO>::Frag;
    __shared__ __attribute__((aligned(16))) float mats[kPrepWaves][2][L * kLd];
    __shared__ __attribute__((aligned(16))) float vecs[kPrepWaves][3][L];
    const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float *A = mats[wave][0], *X = mats[wave][1], *hi = vecs[wave][0], *lo = vecs[wave][1], *be = vecs[wave][2];
    const long long ci = (long long)blockIdx.x * kPrepWaves + wave;
    const long long nch = chunks(a.T);
    const long long cell = ci < total ? ci / nch : 0, c = ci < total ? ci % nch : 0;
    const int b = (int)(cell / a.H), h = (int)(cell % a.H), hk = h / (a.H / a.Hk);
    const long long s = c * L;
    const int nc = ci < total ? (int)max(0ll, min((long long)L, tokens(a, b) - s)) : 0;
    char *out = rec + ci * R::BYTES;

    // ---- gates: lane = token (twice over)
    const int tok = lane & 31;
    double G = 0.0;
    float beta = 0.0f;
    if (tok < nc) {
        G = gate_log2(a.g[b * a.sg.s0 + h * a.sg.s1 + (s + tok) * a.sg.s2]);
        beta = a.beta[b * a.sb.s0 + h * a.sb.s1 + (s + tok) * a.sb.s2];
    }
#pragma unroll
    for (int m = 1; m < L; m <<= 1) {
        const double x = __shfl_up(G, m, 32);
        if (tok >= m) G += x;
    }
    {
        const double GL = __shfl(G, 31, 32);
        const double top = rint(G * 64.0) / 64.0;
        if (lane < L) {
            hi[tok] = (float)top;
            lo[tok] = (float)(G - top);
            be[tok] = beta;
            if (nc > 0) {
                float *v = (float *)(out + R::VEC);
                v[R::EG * L + tok] = __builtin_amdgcn_exp2f((float)G);
                v[R::REST * L + tok] = __builtin_amdgcn_exp2f((float)(GL - G));
                v[R::BETA * L + tok] = beta;
            }
        }
    }
    // ---- scores: lane column j = l16 (+ 16), rows i = 4 g4 + r (+ 16)
    f32x4 kk[3] = {}, qk[3] = {};  // tiles (0, 0), (1, 0), (1, 1)
    const IO *kp = (const IO *)a.k + b * a.sk.s0 + hk * a.sk.s1 + s * a.sk.s2;
    const IO *qp = (const IO *)a.q + b * a.sq.s0 + hk * a.sq.s1 + s * a.sq.s2;
    for (int col = 8 * g4; col < (a.dk + 31) / 32 * 32; col += 32) {
        Frag k[2], q[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int r = 16 * t + l16;
            const bool ok = r < nc && col < a.dk;
            k[t] = row8(kp + r * a.sk.s2 + col, ok);
            q[t] = row8(qp + r * a.sq.s2 + col, ok);
        }
        kk[0] = mfma(k[0], k[0], kk[0]);
        kk[1] = mfma(k[1], k[0], kk[1]);
        kk[2] = mfma(k[1], k[1], kk[2]);
        qk[0] = mfma(q[0], k[0], qk[0]);
        qk[1] = mfma(q[1], k[0], qk[1]);
        qk[2] = mfma(q[1], k[1], qk[2]);
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        const int i0 = (t > 0 ? 16 : 0) + 4 * g4, j = (t == 2 ? 16 : 0) + l16;
        const float hj = hi[j], lj = lo[j];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = i0 + r;
            const float M = __builtin_amdgcn_exp2f((hi[i] - hj) + (lo[i] - lj));
            A[i * kLd + j] = j < i ? kk[t][r] * M : 0.0f;
            X[i * kLd + j] = j <= i ? a.scale * (qk[t][r] * M) : 0.0f;
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) A[(4 * g4 + r) * kLd + 16 + l16] = X[(4 * g4 + r) * kLd + 16 + l16] = 0.0f;
    __syncthreads();
    // two rows' slots of a matrix in LDS
    const auto slots = [&](const float *m, int t, float *x) {
        const f32x4 u = *(const f32x4 *)(m + (16 * t + l16) * kLd + 4 * g4);
        const f32x4 v = *(const f32x4 *)(m + (16 * t + l16) * kLd + 16 + 4 * g4);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = u[e], x[4 + e] = v[e];
    };
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float x[8];
        Frag f[R::PP];
        slots(X, t, x);
        split8<R::PP>(x, f);
        if (nc > 0)
#pragma unroll
            for (int p = 0; p < R::PP; ++p) *(Frag *)(out + R::P + (t * R::PP + p) * R::FRAG + lane * sizeof(Frag)) = f[p];
    }
    __syncthreads();
    // ---- the inverse
    if (lane < L) {
        const int o = 16 * (lane >> 4);  // block on the diagonal; column l16 of it
        float x[16], y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float sum = 0.0f;
#pragma unroll
            for (int m = 0; m < i; ++m) sum += A[(o + i) * kLd + o + m] * y[m];
            x[i] = (i == l16 ? 1.0f : 0.0f) - sum;
            y[i] = x[i] * be[o + i];
            X[(o + i) * kLd + o + l16] = x[i];
        }
    }
    __syncthreads();
    {
        f32x4 Y = {}, Z = {};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            Y = __builtin_amdgcn_mfma_f32_16x16x4f32(A[(16 + l16) * kLd + 4 * g4 + e] * be[4 * g4 + e],
                                                     X[(4 * g4 + e) * kLd + l16], Y, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            Z = __builtin_amdgcn_mfma_f32_16x16x4f32(X[(16 + l16) * kLd + 16 + 4 * g4 + e], Y[e], Z, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            X[(16 + 4 * g4 + r) * kLd + l16] = -Z[r];
            X[(4 * g4 + r) * kLd + 16 + l16] = 0.0f;
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float x[8];
        Frag f[R::TP];
        slots(X, t, x);
        const float bi = be[16 * t + l16];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= bi;
        split8<R::TP>(x, f);
        if (nc > 0)
#pragma unroll
            for (int p = 0; p < R::TP; ++p) *(Frag *)(out + (t * R::TP + p) * R::FRAG + lane * sizeof(Frag)) = f[p];
    }
}

// ---- the walk over the chunks

template <typename IO, int DKP_, int NCT_, int NW_>
struct Cfg {
    static constexpr int DKP = DKP_, NCT = NCT_, NW = NW_, NTH = 64 * NW_;
    static constexpr int BV = 16 * NCT * NW;               // value columns of a workgroup
    static constexpr int NAT = DKP / 16, NKS = DKP / 32;   // 16-row tiles of S, inner steps over d_qk
    static constexpr int EPG = Types<IO>::EPG;
    static constexpr int QG = DKP / EPG, VG = 16 * NCT / EPG, WG = BV / EPG;  // granules of a row
    // float32: V in one buffer a wavefront, whose columns are its own
    static constexpr bool VOWN = sizeof(IO) == 4;
    static constexpr int TROW = 2 * DKP + (VOWN ? 0 : BV);  // elements of a tile for each token
    static constexpr int REC = Rec<IO>::BYTES / (int)sizeof(IO);  // elements of a record
    static constexpr size_t TILE = ((size_t)L * TROW + REC) * sizeof(IO), VTILE = VOWN ? (size_t)L * BV * sizeof(IO) : 0;
    static constexpr int NBUF = 2 * TILE + VTILE <= kLds ? 2 : 1;
    static constexpr int PER_CU = 2 * (NBUF * TILE + VTILE) <= kLds && NW == 4 ? 2 : 1;  // workgroups of a compute unit
    static_assert(QG >= 8, "swizzle");
    static_assert(TILE + VTILE <= kLds, "LDS");
};

// acc + the products of two operands' parts whose joint order stays below ORD
template <int ORD, typename Frag>
__device__ __forceinline__ f32x4 mfma_parts(const Frag *x, const Frag *y, f32x4 acc) {
#pragma unroll
    for (int o = ORD - 1; o >= 0; --o)  // the smallest first
#pragma unroll
        for (int p = 0; p <= o; ++p) acc = mfma(x[p], y[o - p], acc);
    return acc;
}

// SP: parts of what leads to the state
template <typename IO, int DKP, int NCT, int NW, int SP>
__global__ __launch_bounds__(64 * NW, (Cfg<IO, DKP, NCT, NW>::PER_CU * NW / 4)) void delta_kernel(DeltaArgs a, const char *rec) {
    using C = Cfg<IO, DKP, NCT, NW>;
    using R = Rec<IO>;
    using Frag = typename Types<IO>::Frag;
    constexpr int NAT = C::NAT, NKS = C::NKS, QG = C::QG, VG = C::VG, BV = C::BV, NBUF = C::NBUF;
    constexpr int OP = Types<IO>::XPARTS;  // parts of what leads to the output
    constexpr int ES = (int)sizeof(IO);
    __shared__ __attribute__((aligned(16))) IO tile0[L * C::TROW + C::REC];
    __shared__ __attribute__((aligned(16))) IO tile1[NBUF == 2 ? L * C::TROW + C::REC : 16];
    __shared__ __attribute__((aligned(16))) IO vtiles[NW][C::VOWN ? L * 16 * NCT : 8];

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the column blocks of a head on one XCD: each XCD has a contiguous run of them
    const int nwg = gridDim.x, xq = nwg >> 3, xr = nwg & 7, xcd = blockIdx.x & 7;
    const int logical = xcd * xq + min(xcd, xr) + (blockIdx.x >> 3);
    const int ntile = (a.dv + BV - 1) / BV;
    const int tile = logical % ntile, bh = logical / ntile;
    const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const int dk = a.dk, dv = a.dv, n = tokens(a, b), col0 = tile * BV;
    const int ldq = (int)a.sq.s2, ldk = (int)a.sk.s2, ldv = (int)a.sv.s2, ldo = (int)a.so.s2;
    const IO *qg = (const IO *)a.q + b * a.sq.s0 + hk * a.sq.s1;
    const IO *kg = (const IO *)a.k + b * a.sk.s0 + hk * a.sk.s1;
    const IO *vg = (const IO *)a.v + b * a.sv.s0 + h * a.sv.s1 + col0;
    IO *og = (IO *)a.o + b * a.so.s0 + h * a.so.s1 + col0;
    const char *rg = rec + (long long)bh * chunks(a.T) * R::BYTES;

    // ---- state.  Lane (l16, g4) of tile (at, bt) holds rows krow(at) + r of column vcol + 4 bt
    const int vq = NCT == 2 ? 8 : 4;
    const int vc0 = wave * 16 * NCT;
    const int vcol = vc0 + vq * (l16 >> 2) + (l16 & 3);
    auto krow = [&](int at) { return 32 * (at >> 1) + 8 * g4 + 4 * (at & 1); };
    f32x4 X[NAT][NCT];
    const size_t cell = (size_t)bh * dk * dv;
    auto state_at = [&](int at, int bt) {
        return krow(at) < dk && col0 + vcol + 4 * bt < dv ? (unsigned)((krow(at) * dv + col0 + vcol + 4 * bt) * 4) : kOut;
    };
#pragma unroll
    for (int at = 0; at < NAT; ++at)
#pragma unroll
        for (int bt = 0; bt < NCT; ++bt) X[at][bt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (a.S0) {
        const auto xs = __builtin_amdgcn_make_buffer_rsrc((void *)(a.S0 + cell), 0, dk * dv * 4, kBuf);
#pragma unroll
        for (int at = 0; at < NAT; ++at)
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) {
                const unsigned off = state_at(at, bt);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    X[at][bt][r] = __uint_as_float(
                        __builtin_amdgcn_raw_buffer_load_b32(xs, off == kOut ? kOut : off + r * dv * 4, 0, 0));
            }
    }

    // ---- chunks.  Rows past a chunk's tokens are out of their descriptor's range:
    // they read as zero and are not written.
    const int nch = (n + L - 1) / L;
    auto count = [&](int c) -> int { return max(0, min(L, n - c * L)); };
    auto copy_offsets = [&](unsigned *off, int ld, int ncol, auto gpr_c) {
        constexpr int GPR = decltype(gpr_c)::value, RPI = C::NTH / GPR;
        static_assert(L * GPR % C::NTH == 0, "whole instructions");
#pragma unroll
        for (int i = 0; i < (RPI >= 16 ? 1 : 16 / RPI); ++i) {
            const int gi = i * C::NTH + tid, row = gi / GPR, col = ((gi % GPR) ^ swz<GPR>(row)) * C::EPG;
            off[i] = col < ncol ? (unsigned)((row * ld + col) * ES) : kOut;
        }
    };
    auto copy = [&](IO *dst, const IO *src, int ld, const unsigned *off, auto gpr_c, int c) {
        constexpr int GPR = decltype(gpr_c)::value, RPI = C::NTH / GPR, PER = RPI >= 16 ? 1 : 16 / RPI;
        const int bytes = count(c) * ld * ES;
        const auto rs = __builtin_amdgcn_make_buffer_rsrc((void *)(src + (size_t)c * L * ld), 0,
                                                          __builtin_amdgcn_readfirstlane(bytes), kBuf);
        const unsigned step = (unsigned)(RPI * ld * ES);
#pragma unroll
        for (int i = 0; i < L * GPR / C::NTH; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr *)(dst + (i * NW + wave) * 64 * C::EPG), 16,
                                                     off[i % PER] + i / PER * PER * step, 0, 0, 0);
    };
    using QGc = std::integral_constant<int, QG>;
    using WGc = std::integral_constant<int, C::WG>;
    constexpr int QPER = 16 * QG > C::NTH ? 16 * QG / C::NTH : 1, WPER = 16 * C::WG > C::NTH ? 16 * C::WG / C::NTH : 1;
    unsigned qoff[QPER], koff[QPER], voff[WPER], ownoff = kOut;
    copy_offsets(qoff, ldq, dk, QGc{});
    copy_offsets(koff, ldk, dk, QGc{});
    constexpr int VI = L * VG / 64;  // own tile: 64 / VG rows an instruction
    if constexpr (C::VOWN) {
        const int col = vc0 + lane % VG * C::EPG;
        ownoff = col0 + col < dv ? (unsigned)((lane / VG * ldv + col) * ES) : kOut;
    } else {
        copy_offsets(voff, ldv, dv - col0, WGc{});
    }
    constexpr int NREC = R::BYTES / 1024;
    auto load = [&](IO *t, int c) {
        copy(t, qg, ldq, qoff, QGc{}, c);
        copy(t + L * DKP, kg, ldk, koff, QGc{}, c);
        if constexpr (!C::VOWN) copy(t + 2 * L * DKP, vg, ldv, voff, WGc{}, c);
        const int bytes = count(c) > 0 ? R::BYTES : 0;
        const auto rs = __builtin_amdgcn_make_buffer_rsrc((void *)(rg + (long long)c * R::BYTES), 0,
                                                          __builtin_amdgcn_readfirstlane(bytes), kBuf);
#pragma unroll
        for (int i = 0; i < (NREC + NW - 1) / NW; ++i)
            if (i * NW + wave < NREC)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rs, (lds_ptr *)((char *)(t + L * C::TROW) + (i * NW + wave) * 1024), 16,
                    (unsigned)((i * NW + wave) * 1024 + lane * 16), 0, 0, 0);
    };
    IO *own = vtiles[wave];
    auto load_v = [&](int c) {
        const int bytes = count(c) * ldv * ES;
        const auto rs = __builtin_amdgcn_make_buffer_rsrc((void *)(vg + (size_t)c * L * ldv), 0,
                                                          __builtin_amdgcn_readfirstlane(bytes), kBuf);
#pragma unroll
        for (int i = 0; i < VI; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr *)(own + i * 64 * C::EPG), 16,
                                                     ownoff + i * (unsigned)(64 / VG * ldv * ES), 0, 0, 0);
    };

    Rows<QG> rows;
    Cols<QG> cols;
    rows.init((const IO *)nullptr, l16, g4);
    cols.init((const IO *)nullptr, l16, g4);
    // this lane's outputs: tokens l16 and 16 + l16, columns vc0 + vq g4 + (0 .. 4 NCT - 1)
    const int ocol = vc0 + vq * g4;
    const bool ook = col0 + ocol < dv;
    constexpr int NST = 2 * (ES == 4 ? NCT : 1);  // stores of a chunk, issued after the next one's copies
    auto body = [&](IO *cur, IO *next, int c) {
        if (NBUF == 1) {
            __syncthreads();
            load(cur, c);
            wait_vm<0>();
        } else if (c == 0) {
            wait_vm<0>();
        } else {
            wait_vm<NST>();  // this wavefront's copies have landed
        }
        __syncthreads();
        if (NBUF == 2) load(next, c + 1);
        const int nc = count(c);
        const IO *Qs = cur, *Ks = Qs + L * DKP;
        const char *rc = (const char *)(cur + L * C::TROW);
        const float *vec = (const float *)(rc + R::VEC);
        Frag vf[NCT];
#pragma unroll
        for (int bt = 0; bt < NCT; ++bt)
            vf[bt] = C::VOWN ? v_frag<16 * NCT>((const IO *)own, 4 * bt, vq, l16, g4)
                             : v_frag<BV>(cur + 2 * L * DKP, vc0 + 4 * bt, vq, l16, g4);
        // K S (lane: column, tokens 16 t + 4 g4 + r) and S^T Q^T (lane: token, columns)
        f32x4 KS[2][NCT], O[2][NCT];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) KS[t][bt] = O[t][bt] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < NKS; ++kk) {
            Frag q[2], k[2], xf[NCT][SP];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                q[t] = rows.get(Qs, t, kk);
                k[t] = rows.get(Ks, t, kk);
            }
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = X[2 * kk + (e >> 2)][bt][e & 3];
                split8<SP>(x, xf[bt]);
            }
#pragma unroll
            for (int p = SP - 1; p >= 0; --p)
#pragma unroll
                for (int bt = 0; bt < NCT; ++bt)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        KS[t][bt] = mfma(k[t], xf[bt][p], KS[t][bt]);
                        if (p < OP) O[t][bt] = mfma(xf[bt][p], q[t], O[t][bt]);
                    }
        }
        if constexpr (C::VOWN) {
            // V's next rows over this chunk's, whose reads have returned
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) asm volatile("" : "+v"(vf[bt]));
            __builtin_amdgcn_sched_barrier(0);
            load_v(c + 1);
        }
        Frag tf[2][R::TP], pf[2][R::PP];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int p = 0; p < SP; ++p) tf[t][p] = *(const Frag *)(rc + (t * R::TP + p) * R::FRAG + lane * sizeof(Frag));
#pragma unroll
            for (int p = 0; p < R::PP; ++p) pf[t][p] = *(const Frag *)(rc + R::P + (t * R::PP + p) * R::FRAG + lane * sizeof(Frag));
        }
        f32x4 eg[2], rest[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            eg[t] = *(const f32x4 *)(vec + R::EG * L + 16 * t + 4 * g4);
            rest[t] = *(const f32x4 *)(vec + R::REST * L + 16 * t + 4 * g4);
        }
        Frag uf[NCT][OP], wf[NCT][SP];
#pragma unroll
        for (int bt = 0; bt < NCT; ++bt) {
            float x[8];
            Frag rf[SP];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (float)vf[bt][e] - eg[e >> 2][e & 3] * KS[e >> 2][bt][e & 3];
            split8<SP>(x, rf);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const f32x4 u = mfma_parts<SP>(tf[t], rf, f32x4{0, 0, 0, 0});
#pragma unroll
                for (int r = 0; r < 4; ++r) x[4 * t + r] = u[r];
            }
            split8<OP>(x, uf[bt]);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= rest[e >> 2][e & 3];
            split8<SP>(x, wf[bt]);
        }
        // output
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float fade = vec[R::EG * L + 16 * t + l16] * a.scale;
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) O[t][bt] = mfma_parts<OP>(uf[bt], pf[t], O[t][bt] * fade);
        }
        // state update
        const float decay = vec[R::EG * L + L - 1];
#pragma unroll
        for (int kk = 0; kk < NKS; ++kk)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const Frag kf = cols.get(Ks, kk, t);
#pragma unroll
                for (int bt = 0; bt < NCT; ++bt) {
                    f32x4 x = X[2 * kk + t][bt] * decay;
#pragma unroll
                    for (int p = SP - 1; p >= 0; --p) x = mfma(kf, wf[bt][p], x);
                    X[2 * kk + t][bt] = x;
                }
            }
        const auto os = __builtin_amdgcn_make_buffer_rsrc((void *)(og + (size_t)c * L * ldo), 0,
                                                          __builtin_amdgcn_readfirstlane(nc * ldo * ES), kBuf);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const unsigned at = ook ? (unsigned)(((16 * t + l16) * ldo + ocol) * ES) : kOut;
            if constexpr (ES == 4) {
#pragma unroll
                for (int i = 0; i < NCT; ++i)
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[t][i]), os, at + 16 * i, 0, 0);
            } else {
                const f32x4 a0 = O[t][0], a1 = O[t][NCT - 1];
                const float y[8] = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
                bf16x8 o8;
                pack(y, o8);
                const u32x4 u = __builtin_bit_cast(u32x4, o8);
                if constexpr (NCT == 2)
                    __builtin_amdgcn_raw_buffer_store_b128(u, os, at, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b64(u32x2{u[0], u[1]}, os, at, 0, 0);
            }
        }
    };
    if (nch > 0) {
        if (NBUF == 2) load(tile0, 0);
        if constexpr (C::VOWN) load_v(0);
    }
    for (int c = 0; c < nch; c += 2) {
        body(tile0, tile1, c);
        if (c + 1 < nch) body(NBUF == 2 ? tile1 : tile0, tile0, c + 1);
    }
    wait_vm<0>();  // no copy may still be on its way into LDS when the workgroup ends

    if (a.S_T) {
        const auto xs = __builtin_amdgcn_make_buffer_rsrc((void *)(a.S_T + cell), 0, dk * dv * 4, kBuf);
#pragma unroll
        for (int at = 0; at < NAT; ++at)
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) {
                const unsigned off = state_at(at, bt);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(X[at][bt][r]), xs,
                                                          off == kOut ? kOut : off + r * dv * 4, 0, 0);
            }
    }
    // rows behind the sequence's length
    constexpr int QPR = BV / 4;  // quads of a row
    const long long quads = (long long)(a.T - n) * QPR;
    for (long long e = tid; e < quads; e += C::NTH) {
        const long long t = n + e / QPR;
        const int cc = (int)(e % QPR) * 4;
        if (col0 + cc < dv) {
            if constexpr (ES == 4)
                *(f32x4 *)(og + t * ldo + cc) = f32x4{0, 0, 0, 0};
            else
                *(u32x2 *)(og + t * ldo + cc) = u32x2{0, 0};
        }
    }
}

// ---- gradients, token by token

constexpr int kBV = 64;  // value columns of a workgroup

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
    __shared__ float ks[256], qs[256], red[2][4][kBV];
    const int ntile = (a.dv + kBV - 1) / kBV;
    const int tile = blockIdx.x % ntile, bh = blockIdx.x / ntile, b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const int tid = threadIdx.x, c = tid & 63, rg = tid >> 6, col = tile * kBV + c;
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


template <typename IO, int DKP, int NCT, int NW>
hipError_t launch_shape(const DeltaArgs &a, const char *rec, hipStream_t s) {
    const dim3 grid((unsigned)(a.B * a.H * ((a.dv + 16 * NCT * NW - 1) / (16 * NCT * NW))));
    if constexpr (sizeof(IO) == 4)
        delta_kernel<IO, DKP, NCT, NW, 1><<<grid, 64 * NW, 0, s>>>(a, rec);
    else if (a.S_T)
        delta_kernel<IO, DKP, NCT, NW, 3><<<grid, 64 * NW, 0, s>>>(a, rec);
    else
        delta_kernel<IO, DKP, NCT, NW, 2><<<grid, 64 * NW, 0, s>>>(a, rec);
    return hipGetLastError();
}

template <typename IO>
hipError_t launch_fwd_t(const DeltaArgs &a, hipStream_t s) {
    constexpr bool BF = sizeof(IO) == 2;
    char *rec = (char *)a.ws;
    const long long cells = (long long)a.B * a.H, total = cells * chunks(a.T);
    prep_kernel<IO><<<dim3((unsigned)((total + kPrepWaves - 1) / kPrepWaves)), 64 * kPrepWaves, 0, s>>>(a, rec, total);
    const bool wide = cells * ((a.dv + 127) / 128) >= 256;
    if (a.dk <= 64)
        return wide ? launch_shape<IO, 64, 2, 4>(a, rec, s) : launch_shape<IO, 64, 1, 4>(a, rec, s);
    if (a.dk <= 128)
        return wide ? launch_shape<IO, 128, 2, 4>(a, rec, s) : launch_shape<IO, 128, 1, 4>(a, rec, s);
    return wide ? launch_shape<IO, 256, BF ? 2 : 1, BF ? 4 : 8>(a, rec, s) : launch_shape<IO, 256, 1, 4>(a, rec, s);
}

template <typename IO>
hipError_t launch_bwd_t(const DeltaArgs &a, hipStream_t s) {
    const Ws w = make_ws(a);
    const unsigned cols = (unsigned)(a.B * a.H * ((a.dv + kBV - 1) / kBV)), cells = (unsigned)(a.B * a.H);
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
    (void)Hk;
    const size_t n = (size_t)B * H;
    if (!backward) return n * chunks(T) * (io_bf16 ? Rec<bf16>::BYTES : Rec<float>::BYTES) / 4;
    return n * T * (2 * (size_t)dv + 2 * (size_t)dk + 1) + n * dk * dv;
}

hipError_t launch_deltarule_fwd(const DeltaArgs &a, int io_bf16, hipStream_t s) {
    return io_bf16 ? launch_fwd_t<bf16>(a, s) : launch_fwd_t<float>(a, s);
}
hipError_t launch_deltarule_bwd(const DeltaArgs &a, int io_bf16, hipStream_t s) {
    return io_bf16 ? launch_bwd_t<bf16>(a, s) : launch_bwd_t<float>(a, s);
}

}  // namespace mlstm
