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
// at most where the output's own rounding is off by 2^-8.  Of two split operands the
// product of the last parts is left out: of P U 2^-14 at most, 2^-17 on average.  Where the
// state is handed out, all that leads to it has three parts (24 bits, products of 2^-21 at
// most left out): the copy of S that meets K, T', its right side, the update's
// e^{G_L - G} U; else two.  S itself, decays and sums
// are float32.  float32 I/O runs on the float32 MFMA without further rounding.
#include <type_traits>

#include "chunk_tiles.hpp"

namespace mlstm {

namespace {

// ---- the three walks over a sequence's chunks

enum Walk {
    FORWARD,  // o and the final state
    STATES,   // the backward's first: X of every token, the state at every block's start
    BACK      // dU and the state's gradient, from the last chunk to the first
};

// ---- records: what a chunk knows without the state

// Operand fragments: tile t holds rows 16 t + l16, slot e of lane group g4 is
// token 16 (e / 4) + 4 g4 + e % 4.  An inverse (FORWARD: beta T', STATES: T', BACK: T^T with
// T = (I + beta N)^-1), scores (FORWARD: P, BACK: P^T), then float vectors over the
// tokens: e^{G_i}, e^{G_L - G_i}, beta_i.
template <typename IO, Walk W>
struct Rec {
    typedef typename Types<IO>::Frag Frag;
    static constexpr bool BF = sizeof(IO) == 2;
    static constexpr int TP = BF ? 3 : 1;                                       // parts of the inverse
    static constexpr int PP = W == STATES ? 0 : !BF ? 1 : W == FORWARD ? 2 : 3;  // parts of the scores
    static constexpr int FRAG = 64 * (int)sizeof(Frag);                         // bytes of a tile's part
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

// 8 floats as a sum of PARTS bfloat16 operands.  All but the last part are cut, not
// rounded: the upper halves of two floats by one byte permutation, the rest by a mask
// and a subtraction.  Three parts hold a float's 24 bits, so the third is cut too and the
// sum is exact; of two the second is rounded, 2^-16 at most.  (A conversion is half as fast as those, and
// v_dot2c_f32_bf16 in place of the subtraction does not run beside the MFMA.)
template <int PARTS>
__device__ __forceinline__ void split8(const float *x, bf16x8 *f) {
    unsigned y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(x[e]);
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
        u32x4 w;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            unsigned &y0 = y[2 * p], &y1 = y[2 * p + 1];
            if (q == PARTS - 1 && PARTS < 3) {
                const bf16x2 h = __builtin_convertvector((f32x2{__uint_as_float(y0), __uint_as_float(y1)}), bf16x2);
                w[p] = __builtin_bit_cast(unsigned, h);
            } else {
                w[p] = __builtin_amdgcn_perm(y1, y0, 0x07060302u);
            }
            if (q + 1 < PARTS) {
                y0 = __float_as_uint(__uint_as_float(y0) - __uint_as_float(y0 & 0xffff0000u));
                y1 = __float_as_uint(__uint_as_float(y1) - __uint_as_float(y1 & 0xffff0000u));
            }
        }
        f[q] = __builtin_bit_cast(bf16x8, w);
    }
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
// Bound by HBM where there are many chunks: 64 heads of 256 x 512, 4096 tokens, bfloat16 71 us for
// 394 MB (5.5 TB/s; 137 MB read and 157 written for the backward at d_qk = 128: 63 us); a
// call of two chunks takes 8 us, the inverse's rows one after another.
template <typename IO, int DKP, bool BWD>
__global__ __launch_bounds__(64 * kPrepWaves) void prep_kernel(DeltaArgs a, char *rec, char *rec_back, long long total) {
    using R = Rec<IO, BWD ? STATES : FORWARD>;
    using RB = Rec<IO, BACK>;
    using Frag = typename Types<IO>::Frag;
    __shared__ __attribute__((aligned(16))) float mats[kPrepWaves][BWD ? 3 : 2][L * kLd];
    __shared__ __attribute__((aligned(16))) float vecs[kPrepWaves][3][L];
    const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // N, T', T; the scores go where T' will be
    float *A = mats[wave][0], *X = mats[wave][1], *Xb = mats[wave][BWD ? 2 : 1];
    float *hi = vecs[wave][0], *lo = vecs[wave][1], *be = vecs[wave][2];
    const long long ci = (long long)blockIdx.x * kPrepWaves + wave;
    const long long nch = chunks(a.T);
    const long long cell = ci < total ? ci / nch : 0, c = ci < total ? ci % nch : 0;
    const int b = (int)(cell / a.H), h = (int)(cell % a.H), hk = h / (a.H / a.Hk);
    const long long s = c * L;
    const int nc = ci < total ? (int)max(0ll, min((long long)L, tokens(a, b) - s)) : 0;
    char *out = rec + ci * R::BYTES, *outb = BWD ? rec_back + ci * RB::BYTES : nullptr;

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
        }
        float *v = (float *)(lane < L ? out + R::VEC : outb + RB::VEC);
        if (nc > 0 && (lane < L || BWD)) {
            v[R::EG * L + tok] = __builtin_amdgcn_exp2f((float)G);
            v[R::REST * L + tok] = __builtin_amdgcn_exp2f((float)(GL - G));
            v[R::BETA * L + tok] = beta;
        }
    }
    // ---- scores: lane column j = l16 (+ 16), rows i = 4 g4 + r (+ 16)
    f32x4 kk[3] = {}, qk[3] = {};  // tiles (0, 0), (1, 0), (1, 1)
    const IO *kp = (const IO *)a.k + b * a.sk.s0 + hk * a.sk.s1 + s * a.sk.s2;
    const IO *qp = (const IO *)a.q + b * a.sq.s0 + hk * a.sq.s1 + s * a.sq.s2;
    // loads of AHEAD steps in flight: one at a time the wavefront waits for each
    constexpr int NKS = DKP / 32, AHEAD = sizeof(IO) == 2 ? (NKS < 4 ? NKS : 4) : 2;
#pragma unroll
    for (int k0 = 0; k0 < NKS; k0 += AHEAD) {
        Frag k[AHEAD][2], q[AHEAD][2];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int r = 16 * t + l16, col = 32 * (k0 + i) + 8 * g4;
                const bool ok = r < nc && col < a.dk;
                k[i][t] = row8(kp + r * a.sk.s2 + col, ok);
                q[i][t] = row8(qp + r * a.sq.s2 + col, ok);
            }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            kk[0] = mfma(k[i][0], k[i][0], kk[0]);
            kk[1] = mfma(k[i][1], k[i][0], kk[1]);
            kk[2] = mfma(k[i][1], k[i][1], kk[2]);
            qk[0] = mfma(q[i][0], k[i][0], qk[0]);
            qk[1] = mfma(q[i][1], k[i][0], qk[1]);
            qk[2] = mfma(q[i][1], k[i][1], qk[2]);
        }
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
    // the slots of row 16 t + l16 of a matrix in LDS, or of its transpose
    const auto slots = [&](const float *m, int t, float *x) {
        const f32x4 u = *(const f32x4 *)(m + (16 * t + l16) * kLd + 4 * g4);
        const f32x4 v = *(const f32x4 *)(m + (16 * t + l16) * kLd + 16 + 4 * g4);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = u[e], x[4 + e] = v[e];
    };
    const auto columns = [&](const float *m, int t, float *x) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = m[(16 * (e >> 2) + 4 * g4 + (e & 3)) * kLd + 16 * t + l16];
    };
    const auto put = [&](char *to, int t, const float *x, auto parts_c) {
        constexpr int PARTS = decltype(parts_c)::value;
        Frag f[PARTS];
        split8<PARTS>(x, f);
        if (nc > 0)
#pragma unroll
            for (int p = 0; p < PARTS; ++p) *(Frag *)(to + (t * PARTS + p) * R::FRAG + lane * sizeof(Frag)) = f[p];
    };
    using TPc = std::integral_constant<int, R::TP>;
    using PPc = std::integral_constant<int, BWD ? RB::PP : R::PP>;
    using TBc = std::integral_constant<int, RB::TP>;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float x[8];
        if constexpr (BWD)
            columns(X, t, x);
        else
            slots(X, t, x);
        put(BWD ? outb + RB::P : out + R::P, t, x, PPc{});
    }
    __syncthreads();
    // ---- the inverses: of I + N beta by the first half of the wavefront, of I + beta N
    // by the second
    if (lane < L || BWD) {
        const int o = lane & 16;  // block on the diagonal; column l16 of it
        const bool second = lane >= L;
        float *to = second ? Xb : X;
        float x[16], y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float bi = be[o + i];
            float sum = 0.0f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const f32x4 n4 = *(const f32x4 *)(A + (o + i) * kLd + o + m);  // zeros from column i on
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m + e < i) sum += n4[e] * y[m + e];
            }
            x[i] = (i == l16 ? 1.0f : 0.0f) - (second ? sum * bi : sum);
            y[i] = second ? x[i] : x[i] * bi;
            to[(o + i) * kLd + o + l16] = x[i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < (BWD ? 2 : 1); ++w) {
        float *M = w ? Xb : X;
        const float bi = be[16 + l16];
        f32x4 Y = {}, Z = {};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            Y = __builtin_amdgcn_mfma_f32_16x16x4f32(A[(16 + l16) * kLd + 4 * g4 + e] * (w ? bi : be[4 * g4 + e]),
                                                     M[(4 * g4 + e) * kLd + l16], Y, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            Z = __builtin_amdgcn_mfma_f32_16x16x4f32(M[(16 + l16) * kLd + 16 + 4 * g4 + e], Y[e], Z, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            M[(16 + 4 * g4 + r) * kLd + l16] = -Z[r];
            M[(4 * g4 + r) * kLd + 16 + l16] = 0.0f;
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float x[8];
        slots(X, t, x);
        if constexpr (!BWD) {
            const float bi = be[16 * t + l16];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= bi;
        }
        put(out, t, x, TPc{});
        if constexpr (BWD) {
            columns(Xb, t, x);
            put(outb, t, x, TBc{});
        }
    }
}

// ---- the walk over the chunks

// Tokens between the states that the backward keeps, each a block of its last kernel.
template <typename IO>
constexpr int kBlock = sizeof(IO) == 2 ? 64 : 32;

// What the walks of the backward write: X or dU of every token, float32
// [cell][T][dv], and the state (its gradient) at each block's start (end), float32 in the
// order of operands [cell][block][32 columns][16 rows][lane][8]: slot e of lane group
// g4 is column 8 g4 + e, lane l16 of tile 2 kk + u row 32 kk + 8 (l16 / 4) + 4 u + l16 % 4.
struct WalkOut {
    float *rows;
    char *states;
};

// Segments of a sequence where few heads would leave most of the card idle.  A segment
// of `len` chunks maps the state before it linearly, S -> M S + b, M [dk x dk] the
// product of its tokens' e^g (I - beta k k^T).  A first walk (SO, state only) makes b from the zero
// state and M as dk more columns, those of the unit matrix with v = 0; scan_kernel
// runs through the segments, and a second walk starts each from its own state.
// Backwards D -> M^T D + c.
struct Segs {
    int count, len;   // count = 1: none
    float *local;     // [cell][segment][dk][dv + dk]: b and M (the BACK walk: c, [dk][dv])
    float *state;     // [cell][segment][dk][dv]: the state before (BACK: D behind) a segment
};

template <typename IO, int DKP_, int NCT_, int NW_, Walk W, bool SO = false>
struct Cfg {
    static constexpr int DKP = DKP_, NCT = NCT_, NW = NW_, NTH = 64 * NW_;
    static constexpr int BV = 16 * NCT * NW;               // value columns of a workgroup
    static constexpr int NAT = DKP / 16, NKS = DKP / 32;   // 16-row tiles of S, inner steps over d_qk
    static constexpr int EPG = Types<IO>::EPG;
    static constexpr int QG = DKP / EPG, VG = 16 * NCT / EPG, WG = BV / EPG;  // granules of a row
    // float32: V in one buffer a wavefront, whose columns are its own
    static constexpr bool VOWN = sizeof(IO) == 4;
    static constexpr bool HASQ = W == BACK || (W == FORWARD && !SO);
    static constexpr int KOFF = HASQ ? DKP : 0;             // Q, K, V
    static constexpr int TROW = KOFF + DKP + (VOWN ? 0 : BV);  // elements of a tile for each token
    static constexpr int REC = Rec<IO, W>::BYTES / (int)sizeof(IO);  // elements of a record
    static constexpr int ELEMS = L * TROW + REC, VELEMS = VOWN ? L * 16 * NCT : 8;
    static constexpr size_t TILE = (size_t)ELEMS * sizeof(IO), VTILE = VOWN ? (size_t)L * BV * sizeof(IO) : 0;
    static constexpr int PER_CU = 2 * (2 * TILE + VTILE) <= kLds && NW == 4 ? 2 : 1;  // workgroups of a compute unit
    static_assert(QG >= 8, "swizzle");
    static_assert(2 * TILE + VTILE <= kLds, "two chunks' tiles in LDS");
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

// SP: parts of what leads to the state.  BACK is called with do, dS_T and dS0 in the
// places of v, S0 and S_T:
//   dU = T^T (P^T do + e^{G_L - G} o (K D)),  dV = beta o dU,
//   D <- e^{G_L} D + Q^T (scale e^G o do) - K^T (e^G o dV).
// Workgroup `wg` of `nwg`.  The tiles are two arrays of the kernel, and a loop goes over pairs of
// chunks: the compiler waits for a copy in flight before any LDS read that may alias it.
//
// Bound by vector and matrix instructions that one or two wavefronts a SIMD overlap little (d_qk = 128,
// three parts: 82 MFMA and some 380 vector instructions a chunk and wavefront, half of these the
// split of S): 64 heads of 256 x 512, 4096 tokens, bfloat16 626 us (5 us a chunk; from one call to the
// next 572 to 783, as the clock moves under load), 128 x 128
// 1.75 us a chunk.  Half of the rows for each of two wavefronts, their sums joined in LDS, was
// slower (1.75 -> 2.05 us): the small products are then done twice.
template <typename IO, int DKP, int NCT, int NW, int SP, Walk W, bool SO>
__device__ __forceinline__ void walk(const DeltaArgs &a, const char *rec, WalkOut to, Segs sg, int wg, int nwg, IO *tile0,
                                     IO *tile1, IO *vtiles) {
    using C = Cfg<IO, DKP, NCT, NW, W, SO>;
    using R = Rec<IO, W>;
    using Frag = typename Types<IO>::Frag;
    constexpr int NAT = C::NAT, NKS = C::NKS, QG = C::QG, VG = C::VG, BV = C::BV;
    constexpr int OP = Types<IO>::XPARTS;  // parts of what leads to the output
    constexpr int ES = (int)sizeof(IO);
    constexpr bool OUT = W == FORWARD && !SO;  // makes o

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the column blocks of a head on one XCD: each XCD has a contiguous run of them
    const int xq = nwg >> 3, xr = nwg & 7, xcd = wg & 7;
    const int logical = xcd * xq + min(xcd, xr) + (wg >> 3);
    const int vtile = (a.dv + BV - 1) / BV, ntile = vtile + (SO && W != BACK ? (a.dk + BV - 1) / BV : 0);
    const int tile = logical % ntile, seg = logical / ntile % sg.count, bh = logical / ntile / sg.count;
    const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const bool unit_cols = SO && tile >= vtile;  // columns of M: those of the unit matrix, v = 0
    const int dk = a.dk, dv = unit_cols ? dk : a.dv, n = tokens(a, b), col0 = (unit_cols ? tile - vtile : tile) * BV;
    const int ldq = (int)a.sq.s2, ldk = (int)a.sk.s2, ldv = (int)a.sv.s2, ldo = (int)a.so.s2;
    const IO *qg = (const IO *)a.q + b * a.sq.s0 + hk * a.sq.s1;
    const IO *kg = (const IO *)a.k + b * a.sk.s0 + hk * a.sk.s1;
    const IO *vg = (const IO *)a.v + b * a.sv.s0 + h * a.sv.s1 + col0;
    IO *og = OUT ? (IO *)a.o + b * a.so.s0 + h * a.so.s1 + col0 : nullptr;
    const char *rg = rec + (long long)bh * chunks(a.T) * R::BYTES;

    // ---- state.  Lane (l16, g4) of tile (at, bt) holds rows krow(at) + r of column vcol + 4 bt
    // A wavefront of 16 columns has every other quad of 32 that it shares with its neighbour.
    const int vc0 = NCT == 2 ? wave * 32 : 32 * (wave >> 1) + 4 * (wave & 1);
    const int vcol = vc0 + 8 * (l16 >> 2) + (l16 & 3);
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
    const int nch = (n + L - 1) / L, c0 = seg * sg.len, c1 = min(c0 + sg.len, nch);  // this segment's chunks
    // The state before the first token of this walk.  With segments all but an empty sequence's
    // come from the scan's buffer, the first one too: S_T may be S0, which the last segment's
    // workgroups write while the first one's may not have read it.
    const float *start = SO ? nullptr : W == BACK ? (c1 == nch ? a.S0 : nullptr) : (seg == 0 ? a.S0 : nullptr);
    if (!SO && sg.count > 1 && c0 < nch && (W == BACK ? c1 < nch : seg > 0 || a.S0))
        start = sg.state + ((size_t)bh * (sg.count - 1) + seg) * dk * dv;  // + cell below
    if (start) {
        const auto xs = __builtin_amdgcn_make_buffer_rsrc((void *)(start + cell), 0, dk * dv * 4, kBuf);
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
    if (unit_cols) {
#pragma unroll
        for (int at = 0; at < NAT; ++at)
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt)
#pragma unroll
                for (int r = 0; r < 4; ++r) X[at][bt][r] = krow(at) + r == col0 + vcol + 4 * bt ? 1.0f : 0.0f;
    }

    // ---- chunks.  Rows past a chunk's tokens are out of their descriptor's range:
    // they read as zero and are not written.
    const int ncb = (dv + 31) >> 5;  // blocks of 32 columns
    const long long nblk = (chunks(a.T) * L + kBlock<IO> - 1) / kBlock<IO>;
    auto count = [&](int c) -> int { return c < 0 ? 0 : max(0, min(L, n - c * L)); };
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
    if constexpr (C::HASQ) copy_offsets(qoff, ldq, dk, QGc{});
    copy_offsets(koff, ldk, dk, QGc{});
    constexpr int VI = L * VG / 64;  // own tile: 64 / VG rows an instruction
    if constexpr (C::VOWN) {
        const int col = NCT == 2 ? vc0 + lane % VG * 4 : vc0 + lane % VG * 8;
        ownoff = !unit_cols && col0 + col < dv ? (unsigned)((lane / VG * ldv + col) * ES) : kOut;
    } else {
        copy_offsets(voff, ldv, unit_cols ? 0 : dv - col0, WGc{});
    }
    constexpr int NREC = R::BYTES / 1024;
    auto load = [&](IO *t, int c) {
        if constexpr (C::HASQ) copy(t, qg, ldq, qoff, QGc{}, c);
        copy(t + L * C::KOFF, kg, ldk, koff, QGc{}, c);
        if constexpr (!C::VOWN) copy(t + L * (C::KOFF + DKP), vg, ldv, voff, WGc{}, c);  // reads nothing for unit columns
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
    IO *own = vtiles + wave * C::VELEMS;
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
    // this lane's outputs: tokens l16 and 16 + l16, columns vc0 + 8 g4 + (0 .. 4 NCT - 1)
    const int ocol = vc0 + 8 * g4;
    const bool ook = col0 + ocol < dv;
    // memory operations of a chunk issued after the next one's copies, 15 of them at most
    constexpr int NST = SO ? 0 : W == FORWARD ? 2 * (ES == 4 ? NCT : 1) : 8 * NCT < 15 ? 8 * NCT : 15;
    constexpr int STEP = W == BACK ? -1 : 1, PER = kBlock<IO> / L;  // chunks of a block
    auto body = [&](IO *cur, IO *next, int c, bool first) {
        if (first) {
            wait_vm<0>();
        } else {
            wait_vm<NST>();  // this wavefront's copies have landed
        }
        __syncthreads();
        const int nc = count(c);
        const IO *Qs = cur, *Ks = Qs + L * C::KOFF;
        const char *rc = (const char *)(cur + L * C::TROW);
        const float *vec = (const float *)(rc + R::VEC);
        // Each step's LDS reads are issued a step ahead of the products that use them, and
        // so are the parts of S; sched_barrier keeps the steps apart.  V is read before the
        // next copies begin: the compiler waits for those ahead of this read.
        Frag vf[NCT], q[2][2], k[2][2], xf[2][NCT][SP];
        auto parts = [&](int kk) {
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = X[2 * kk + (e >> 2)][bt][e & 3];
                split8<SP>(x, xf[kk & 1][bt]);
            }
        };
#pragma unroll
        for (int bt = 0; bt < NCT; ++bt)
            vf[bt] = C::VOWN ? v_frag<16 * NCT>((const IO *)own, 4 * bt, 4 * NCT, l16, g4)
                             : v_frag<BV>(cur + L * (C::KOFF + DKP), vc0 + 4 * bt, 8, l16, g4);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if constexpr (OUT) q[0][t] = rows.get(Qs, t, 0);
            k[0][t] = rows.get(Ks, t, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        load(next, c + STEP);
        parts(0);
        __builtin_amdgcn_sched_barrier(0);
        // the state is kept: X[dk][dv] of the accumulators, transposed by the unit matrix
        const bool keep = SO ? false : W == STATES ? c % PER == 0 : W == BACK ? c % PER == PER - 1 || c == nch - 1 : false;
        char *kept = W == FORWARD || SO ? nullptr
                                  : to.states + ((((size_t)bh * nblk + c / PER) * ncb + ((col0 + vc0) >> 5)) * NAT) * 2048;
        // K S (lane: column, tokens 16 t + 4 g4 + r) and S^T Q^T (lane: token, columns)
        f32x4 KS[2][NCT], O[2][NCT];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) KS[t][bt] = O[t][bt] = f32x4{0, 0, 0, 0};
        Frag tf[2][R::TP], pf[2][R::PP > 0 ? R::PP : 1], kf[2][2], qf[2][2];
        f32x4 eg[2], rest[2], be[2];
#pragma unroll
        for (int kk = 0; kk < NKS; ++kk) {
            const int u = kk & 1;
            __builtin_amdgcn_sched_barrier(0);
            if (kk + 1 < NKS) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if constexpr (OUT) q[u ^ 1][t] = rows.get(Qs, t, kk + 1);
                    k[u ^ 1][t] = rows.get(Ks, t, kk + 1);
                }
                parts(kk + 1);
            } else {
                // the inverse, the scores of BACK, the tokens' factors
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    eg[t] = *(const f32x4 *)(vec + R::EG * L + 16 * t + 4 * g4);
                    rest[t] = *(const f32x4 *)(vec + R::REST * L + 16 * t + 4 * g4);
                    be[t] = *(const f32x4 *)(vec + R::BETA * L + 16 * t + 4 * g4);
                    if constexpr (W == BACK)
#pragma unroll
                        for (int p = 0; p < SP; ++p)
                            pf[t][p] = *(const Frag *)(rc + R::P + (t * R::PP + p) * R::FRAG + lane * sizeof(Frag));
#pragma unroll
                    for (int p = 0; p < SP; ++p) tf[t][p] = *(const Frag *)(rc + (t * R::TP + p) * R::FRAG + lane * sizeof(Frag));
                }
            }
#pragma unroll
            for (int p = SP - 1; p >= 0; --p)
#pragma unroll
                for (int bt = 0; bt < NCT; ++bt)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        KS[t][bt] = mfma(k[u][t], xf[u][bt][p], KS[t][bt]);
                        if (OUT && p < OP) O[t][bt] = mfma(xf[u][bt][p], q[u][t], O[t][bt]);
                    }
            if (W != FORWARD && !SO && keep && col0 + (vc0 & ~31) < dv)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int u2 = kk & 1;
                    Frag unit = {};
#pragma unroll
                    for (int e = 0; e < 8; ++e) unit[e] = (IO)(8 * g4 + e == 8 * (l16 >> 2) + 4 * u + (l16 & 3) ? 1.0f : 0.0f);
                    char *at = kept + (2 * kk + u) * 2048 + lane * 32;
#pragma unroll
                    for (int bt = 0; bt < NCT; ++bt) {
                        f32x4 y = {0, 0, 0, 0};  // the parts' sum is exact
#pragma unroll
                        for (int p = SP - 1; p >= 0; --p) y = mfma(xf[u2][bt][p], unit, y);
                        *(f32x4 *)(at + (NCT == 2 ? 16 * bt : 16 * (wave & 1))) = y;
                    }
                }
        }
        if constexpr (C::VOWN) {
            // V's next rows over this chunk's, whose reads have returned
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) asm volatile("" : "+v"(vf[bt]));
            __builtin_amdgcn_sched_barrier(0);
            load_v(c + STEP);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if constexpr (OUT)
#pragma unroll
                for (int p = 0; p < R::PP; ++p)
                    pf[t][p] = *(const Frag *)(rc + R::P + (t * R::PP + p) * R::FRAG + lane * sizeof(Frag));
            kf[0][t] = cols.get(Ks, 0, t);
            if constexpr (W == BACK) qf[0][t] = cols.get(Qs, 0, t);
        }
        const auto own_rows = __builtin_amdgcn_make_buffer_rsrc(
            (void *)(to.rows + ((size_t)bh * a.T + (size_t)c * L) * dv), 0,
            __builtin_amdgcn_readfirstlane(W == FORWARD || SO ? 0 : nc * dv * 4), kBuf);
        Frag uf[NCT][OP], wf[NCT][SP], gf[NCT][SP];
#pragma unroll
        for (int bt = 0; bt < NCT; ++bt) {
            float x[8];
            Frag rf[SP];
            if constexpr (W == BACK) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    f32x4 y = KS[t][bt] * rest[t];
#pragma unroll
                    for (int p = SP - 1; p >= 0; --p) y = mfma(pf[t][p], vf[bt], y);
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[4 * t + r] = y[r];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = (float)vf[bt][e] - eg[e >> 2][e & 3] * KS[e >> 2][bt][e & 3];
            }
            split8<SP>(x, rf);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const f32x4 u = mfma_parts<SP>(tf[t], rf, f32x4{0, 0, 0, 0});
#pragma unroll
                for (int r = 0; r < 4; ++r) x[4 * t + r] = u[r];
            }
            if constexpr (OUT) split8<OP>(x, uf[bt]);
            if constexpr (W != FORWARD) {
                const bool ok = col0 + vcol + 4 * bt < dv;
                if constexpr (!SO)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = 16 * (e >> 2) + 4 * g4 + (e & 3);
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[e]), own_rows,
                                                          ok ? (unsigned)((i * dv + col0 + vcol + 4 * bt) * 4) : kOut, 0, 0);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= be[e >> 2][e & 3];
            }
            if constexpr (W == BACK) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] = (float)vf[bt][e] * (eg[e >> 2][e & 3] * a.scale);
                    x[e] *= -eg[e >> 2][e & 3];
                }
                split8<SP>(y, gf[bt]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= rest[e >> 2][e & 3];
            }
            split8<SP>(x, wf[bt]);
        }
        // output
        if constexpr (OUT) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float fade = vec[R::EG * L + 16 * t + l16] * a.scale;
#pragma unroll
                for (int bt = 0; bt < NCT; ++bt) O[t][bt] = mfma_parts<OP>(uf[bt], pf[t], O[t][bt] * fade);
            }
        }
        // state update
        const float decay = vec[R::EG * L + L - 1];
#pragma unroll
        for (int kk = 0; kk < NKS; ++kk) {
            const int u = kk & 1;
            __builtin_amdgcn_sched_barrier(0);
            if (kk + 1 < NKS)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    kf[u ^ 1][t] = cols.get(Ks, kk + 1, t);
                    if constexpr (W == BACK) qf[u ^ 1][t] = cols.get(Qs, kk + 1, t);
                }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int bt = 0; bt < NCT; ++bt) X[2 * kk + t][bt] *= decay;
#pragma unroll
            for (int p = SP - 1; p >= 0; --p)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int bt = 0; bt < NCT; ++bt) {
                        f32x4 &x = X[2 * kk + t][bt];
                        x = mfma(kf[u][t], wf[bt][p], x);
                        if constexpr (W == BACK) x = mfma(qf[u][t], gf[bt][p], x);
                    }
        }
        if constexpr (OUT) {
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
        }
    };
    const int nloc = c1 - c0, first = W == BACK ? c1 - 1 : c0;
    if (nloc > 0) {
        load(tile0, first);
        if constexpr (C::VOWN) load_v(first);
    }
    for (int i = 0; i < nloc; i += 2) {
        body(tile0, tile1, first + STEP * i, i == 0);
        if (i + 1 < nloc) body(tile1, tile0, first + STEP * (i + 1), false);
    }
    wait_vm<0>();  // no copy may still be on its way into LDS when the workgroup ends

    // the state where it ends: the sequence's, or for the scan this segment's b or column of M
    const int width = SO && W != BACK ? a.dv + dk : dv;
    const int last = nch > 0 ? (nch - 1) / sg.len : 0;
    float *end = SO ? sg.local + ((size_t)bh * sg.count + seg) * dk * width + (unit_cols ? a.dv : 0)
                    : a.S_T && (W == BACK ? seg == 0 : seg == last) ? a.S_T + cell : nullptr;
    if (end) {
        const auto xs = __builtin_amdgcn_make_buffer_rsrc((void *)end, 0, (dk - 1) * width * 4 + dv * 4, kBuf);
#pragma unroll
        for (int at = 0; at < NAT; ++at)
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) {
                const int col = col0 + vcol + 4 * bt;
                const unsigned off = krow(at) < dk && col < dv ? (unsigned)((krow(at) * width + col) * 4) : kOut;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(X[at][bt][r]), xs,
                                                          off == kOut ? kOut : off + r * width * 4, 0, 0);
            }
    }
    if constexpr (OUT) {
        // rows behind the sequence's length, of this segment's tokens
        const long long z0 = max((long long)n, (long long)c0 * L);
        const long long z1 = seg == sg.count - 1 ? a.T : min((long long)a.T, (long long)(c0 + sg.len) * L);
        constexpr int QPR = BV / 4;  // quads of a row
        const long long quads = max(z1 - z0, 0ll) * QPR;
        for (long long e = tid; e < quads; e += C::NTH) {
            const long long t = z0 + e / QPR;
            const int cc = (int)(e % QPR) * 4;
            if (col0 + cc < dv) {
                if constexpr (ES == 4)
                    *(f32x4 *)(og + t * ldo + cc) = f32x4{0, 0, 0, 0};
                else
                    *(u32x2 *)(og + t * ldo + cc) = u32x2{0, 0};
            }
        }
    }
}

template <typename IO, int DKP, int NCT, int NW, int SP, bool SO>
__global__ __launch_bounds__(64 * NW, (Cfg<IO, DKP, NCT, NW, FORWARD, SO>::PER_CU * NW / 4)) void forward_kernel(DeltaArgs a, const char *rec,
                                                                                                            Segs sg) {
    using C = Cfg<IO, DKP, NCT, NW, FORWARD, SO>;
    __shared__ __attribute__((aligned(16))) IO tile0[C::ELEMS];
    __shared__ __attribute__((aligned(16))) IO tile1[C::ELEMS];
    __shared__ __attribute__((aligned(16))) IO vtiles[NW * C::VELEMS];
    walk<IO, DKP, NCT, NW, SP, FORWARD, SO>(a, rec, WalkOut{}, sg, blockIdx.x, gridDim.x, tile0, tile1, vtiles);
}

// Both walks of the backward, which do not need one another: the first `nback` workgroups are
// BACK's, the longer one (64 heads of 128 x 128, 4096 tokens, bfloat16: 365 us, 2.9 us a chunk, with
// 0.8 GB of X, dU and kept states written).
struct BackArgs {
    DeltaArgs a;              // do, dS_T and dS0 in the places of v, S0 and S_T
    const char *rec, *rec_back;
    WalkOut to, to_back;
    Segs sg, sg_back;
    int nback;
    const void *v;            // what the first walk has there
    Strides sv;
    const float *S0;
};
template <typename IO, int DKP, int NCT, int NW, bool SO>
__global__ __launch_bounds__(64 * NW, (Cfg<IO, DKP, NCT, NW, BACK, SO>::PER_CU * NW / 4)) void back_kernel(BackArgs w) {
    using C = Cfg<IO, DKP, NCT, NW, BACK, SO>;
    using S = Cfg<IO, DKP, NCT, NW, STATES, SO>;
    constexpr int SP = sizeof(IO) == 2 ? 3 : 1, ELEMS = C::ELEMS > S::ELEMS ? C::ELEMS : S::ELEMS;
    __shared__ __attribute__((aligned(16))) IO tile0[ELEMS];
    __shared__ __attribute__((aligned(16))) IO tile1[ELEMS];
    __shared__ __attribute__((aligned(16))) IO vtiles[NW * C::VELEMS];
    if ((int)blockIdx.x < w.nback) {
        walk<IO, DKP, NCT, NW, SP, BACK, SO>(w.a, w.rec_back, w.to_back, w.sg_back, blockIdx.x, w.nback, tile0, tile1, vtiles);
    } else {
        DeltaArgs a = w.a;
        a.v = w.v;
        a.sv = w.sv;
        a.S0 = w.S0;
        a.S_T = nullptr;
        walk<IO, DKP, NCT, NW, SP, STATES, SO>(a, w.rec, w.to, w.sg, blockIdx.x - w.nback, gridDim.x - w.nback, tile0, tile1, vtiles);
    }
}

// The states between segments: S_{s+1} = M_s S_s + b_s, or from the last segment back
// D_{s-1} = M_s^T D_s + c_s, for 16 columns of a head and a wavefront for each 16 rows;
// float32 MFMA.  A step is bound by latency: a step's M and b are loaded while the one
// before is computed, ahead of its stores, whose end a later load's wait includes (8 heads of 128 x 128,
// 32 segments: 160 us with loads where they are used, 81 with them behind the
// step's products).
constexpr int kScanLd = 17;
template <int DKP, bool REV>
__device__ __forceinline__ void scan(const DeltaArgs &a, const float *start, Segs fwd, Segs sg, int wg, float (*S)[DKP * kScanLd]) {
    constexpr int NK = DKP / 16, PK = NK < 8 ? NK : 8;  // 16-row tiles; those of a part of M
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ncol = a.dv / 16, col0 = wg % ncol * 16, bh = wg / ncol, b = bh / a.H;
    const int dk = a.dk, dv = a.dv;  // both multiples of 16
    const int nch = (tokens(a, b) + L - 1) / L, nseg = (nch + fwd.len - 1) / fwd.len;
    const int ld = dv + dk, lda = REV ? dv : ld;
    // Tiles past d_qk read the last one again, against rows of S that stay zero: branches around
    // the loads would make the compiler wait for them at once.
    const bool live = 16 * wave < dk;
    const int row = live ? 16 * wave : dk - 16;
    for (int i = tid; i < DKP * 16; i += 64 * NK) {
        const int r = i / 16, c = i % 16;
        const float x = start && r < dk ? start[((size_t)bh * dk + r) * dv + col0 + c] : 0.0f;
        S[0][r * kScanLd + c] = x;
        S[1][r * kScanLd + c] = 0.0f;
        if (!REV && r < dk) sg.state[((size_t)bh * sg.count * dk + r) * dv + col0 + c] = x;
    }
    // part p of M's columns (all of them up to 128, else 128 each) of a step, and b; one lane
    // address each, the rest of it the same for the wavefront (addresses in pairs of registers
    // for every load spill: one head of 256 x 512, 32 segments, backwards 511 us, so 236)
    const unsigned vm = (unsigned)((REV ? 4 * g4 * ld + row + l16 : (row + l16) * ld + 4 * g4) * 4);
    const unsigned va = (unsigned)(((row + 4 * g4) * lda + l16) * 4);
    auto fetch = [&](int step, int p, f32x4 *m, f32x4 &add) {
        const int s = max(0, min(nseg - 1, REV ? nseg - 1 - step : step));
        const float *M = fwd.local + ((size_t)bh * fwd.count + s) * dk * ld;  // b's columns first
        const float *A = REV ? sg.local + ((size_t)bh * sg.count + s) * dk * dv : M;
        const auto ms = __builtin_amdgcn_make_buffer_rsrc((void *)M, 0, dk * ld * 4, kBuf);
        const auto as = __builtin_amdgcn_make_buffer_rsrc((void *)A, 0, dk * lda * 4, kBuf);
        if (p == 0)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                add[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(as, va, (r * lda + col0) * 4, 0));
#pragma unroll
        for (int k = 0; k < PK; ++k) {
            const int k0 = min(16 * (p * PK + k), dk - 16);
            if constexpr (REV) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    m[k][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ms, vm, ((k0 + e) * ld + dv) * 4, 0));
            } else {
                m[k] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(ms, vm, (k0 + dv) * 4, 0));
            }
        }
        __builtin_amdgcn_sched_barrier(0);  // the loads stay in front of the products
    };
    f32x4 acc[2];
    auto multiply = [&](const float *from, int p, const f32x4 *m) {
#pragma unroll
        for (int k = 0; k < PK; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[e & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(m[k][e], from[(16 * (p * PK + k) + 4 * g4 + e) * kScanLd + l16],
                                                                 acc[e & 1], 0, 0, 0);
    };
    auto finish = [&](int step, float *to) {
        float *out = sg.state + ((size_t)bh * sg.count + (REV ? nseg - 2 - step : step + 1)) * dk * dv + col0 + l16;
        acc[0] += acc[1];
        if (live)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                to[(row + 4 * g4 + r) * kScanLd + l16] = acc[0][r];
                out[(row + 4 * g4 + r) * dv] = acc[0][r];
            }
        __syncthreads();
    };
    f32x4 m0[PK], m1[PK], a0, a1;
    if (nseg > 1) fetch(0, 0, m0, a0);
    __syncthreads();
    for (int step = 0; step + 1 < nseg; ++step) {
        const float *from = S[step & 1];
        acc[0] = a0;
        acc[1] = f32x4{0, 0, 0, 0};
        if constexpr (NK > PK) {
            fetch(step, 1, m1, a1);
            multiply(from, 0, m0);
            fetch(step + 1, 0, m0, a0);
            multiply(from, 1, m1);
            finish(step, S[(step & 1) ^ 1]);
        } else {
            // two steps a turn, M in turn in m0 and m1
            fetch(step + 1, 0, m1, a1);
            multiply(from, 0, m0);
            finish(step, S[(step & 1) ^ 1]);
            if (++step + 1 >= nseg) break;
            acc[0] = a1;
            acc[1] = f32x4{0, 0, 0, 0};
            fetch(step + 1, 0, m0, a0);
            multiply(S[step & 1], 0, m1);
            finish(step, S[(step & 1) ^ 1]);
        }
    }
}
// workgroups from `nfwd` on run backwards
template <int DKP>
__global__ __launch_bounds__(4 * DKP) void scan_kernel(DeltaArgs a, const float *start, Segs fwd, const float *start_back,
                                                               Segs back, int nfwd) {
    __shared__ float S[2][DKP * kScanLd];
    if ((int)blockIdx.x < nfwd)
        scan<DKP, false>(a, start, fwd, fwd, blockIdx.x, S);
    else
        scan<DKP, true>(a, start_back, fwd, back, blockIdx.x - nfwd, S);
}

// ---- the gradients of a block, all blocks at once

// From the state S at a block's start, its gradient D at the block's end, and X and dU
// of its tokens (U = beta o X, dV = beta o dU; G now runs from the block's start):
//   E1_ij = scale M_ij (do_i . U_j)  (j <= i),  E2_ij = M_ij (dV_i . U_j)  (j < i),
//   dQ = scale e^G o (do S^T) + E1 K,
//   dK = e^{G_L - G} o (U D^T) - e^G o (dV S^T) + E1^T Q - E2 K - E2^T K,
//   dbeta_i = dU_i . X_i,
//   dg_i = sum_{j >= i} (do.o - dV.v)_j + <D, S_L>,
//   (do.o)_i = scale e^{G_i} q_i . (S do_i) + sum_j E1_ij (q_i . k_j),
//   <D, S_L> = e^{G_L} <D, S> + sum_j k_j . (e^{G_L - G} o (U D^T))_j.
// The last sum is the decays' share of everything behind a token: it is exact, and
// starts anew at each block, so that its roundings do not add up over a sequence.
//
// Roundings (bfloat16 I/O): dq and dk are rounded once at the end, and what makes them
// has two parts, as in the forward (of dV S^T and E2 the first two of three cut parts' products
// leave out 2^-13 at most of their terms); dbeta and dlog_decay are float32, and so what makes
// them (X and dU themselves, three parts of S, D and X) has 24 bits.
//
// A workgroup has a block of kBlock tokens of one head of q and k and walks the
// heads of v that share it (SHARED: more than one).  A wavefront owns 16 RTW columns of
// d_qk for all tokens: S and D come to it in operand order straight from memory; do, X
// and dU are split once, by the wavefront of their 16 tokens, and shared through LDS.
// Everything is computed transposed (lane: token, rows: d_qk), so that rows leave in
// whole vectors.  Bound by HBM and what it feeds: 64 heads of 128 x 128, 4096 tokens, bfloat16
// 315 us for 1.17 GB read and 0.22 written (4.4 TB/s); float32, 16 heads of 64 x 64, 1024 tokens 19 us.
struct GradIn {
    const float *x, *du;
    const char *s, *d;
};

template <typename IO, int DKP_, int NW_>
struct GCfg {
    static constexpr int DKP = DKP_, NW = NW_, NTH = 64 * NW_;
    static constexpr int SC = kBlock<IO>, NT = SC / 16, NAT = DKP / 16, RTW = NAT / NW;  // tokens and their tiles; tiles of d_qk
    static constexpr int CB = NW / NT;                                         // 32-column blocks of a stage, one a wavefront
    static constexpr int OP = Types<IO>::XPARTS, SP = sizeof(IO) == 2 ? 3 : 1, NM = 1 + SP + OP;
    static constexpr int EPG = Types<IO>::EPG, QG = DKP / EPG, EG = SC / EPG;  // granules of a row of K, of E
    static constexpr int OPS = CB * NT * NM * 512, ES = 2 * OP * SC * SC;      // elements of a stage, of E1 and E2
    static constexpr int POOL = OPS > ES ? OPS : ES;
    static_assert(CB >= 1 && EG >= 8 && RTW >= 1, "layout");
};

// slots of row `row` of a swizzled [SC][SC] matrix in the 32 columns of block jb
template <int EGR>
__device__ __forceinline__ bf16x8 e_row(const bf16 *m, int row, int jb, int g4) {
    const int s = swz<EGR>(row & 15);
    const bf16 *p = m + row * EGR * 8;
    const int c0 = 32 * jb + 4 * g4, c1 = c0 + 16;
    const bf16x4 x = *(const bf16x4 *)(p + (((c0 >> 3) ^ s) << 3) + (c0 & 7));
    const bf16x4 y = *(const bf16x4 *)(p + (((c1 >> 3) ^ s) << 3) + (c1 & 7));
    return bf16x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
}
template <int EGR>
__device__ __forceinline__ f32x8 e_row(const float *m, int row, int jb, int g4) {
    const int s = swz<EGR>(row & 15);
    const float *p = m + row * EGR * 4;
    const int c0 = 32 * jb + 4 * g4, c1 = c0 + 16;
    const f32x4 x = *(const f32x4 *)(p + (((c0 >> 2) ^ s) << 2)), y = *(const f32x4 *)(p + (((c1 >> 2) ^ s) << 2));
    return f32x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
}
// column c0 + l16 of the 32 rows of block ib, tokens as slots
template <int EGR>
__device__ __forceinline__ bf16x8 e_col(const bf16 *m, int ib, int c0, int l16, int g4) {
    return v_frag<EGR * 8>(m + ib * 32 * EGR * 8, c0, 4, l16, g4);
}
template <int EGR>
__device__ __forceinline__ f32x8 e_col(const float *m, int ib, int c0, int l16, int g4) {
    f32x8 f;
    const int c = c0 + l16;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int r = 32 * ib + 16 * (e >> 2) + 4 * g4 + (e & 3);
        f[e] = m[r * EGR * 4 + (((c >> 2) ^ swz<EGR>(r & 15)) << 2) + (c & 3)];
    }
    return f;
}

// four consecutive elements of a row
template <typename IO>
__device__ __forceinline__ void store4(IO *p, const float *x) {
    typedef IO vec __attribute__((ext_vector_type(4)));
    vec v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = from_f<IO>(x[e]);
    *(vec *)p = v;
}

template <typename IO, int DKP, int NW, bool SHARED>
__global__ __launch_bounds__(64 * NW, SHARED && NW == 4 ? 1 : 2) void grad_kernel(DeltaArgs a, GradIn in) {
    using C = GCfg<IO, DKP, NW>;
    using Frag = typename Types<IO>::Frag;
    constexpr int SC = C::SC, NT = C::NT, NAT = C::NAT, RTW = C::RTW, CB = C::CB, OP = C::OP, SP = C::SP, NM = C::NM;
    constexpr int QG = C::QG, EPG = C::EPG;
    __shared__ __attribute__((aligned(16))) IO kt[SC * DKP], qt[SC * DKP];
    __shared__ __attribute__((aligned(16))) IO pool[C::POOL];
    __shared__ __attribute__((aligned(16))) float hi[SC], lo[SC], be[SC], eg[SC], rest[SC];
    __shared__ float dbs[CB][SC], dgs[CB][SC], eqk[SC], part[2][NW][SC], dots[NW];

    const int tid = threadIdx.x, lane0 = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const long long nblk = (chunks(a.T) * L + SC - 1) / SC;
    const int blk = (int)(blockIdx.x % nblk), bk = (int)(blockIdx.x / nblk), b = bk / a.Hk, hk = bk % a.Hk;
    const int per = a.H / a.Hk, dk = a.dk, dv = a.dv, ncb = (dv + 31) >> 5;
    const long long s0 = (long long)blk * SC;
    const int n = (int)min((long long)SC, tokens(a, b) - s0);     // of the block's tokens, may be <= 0
    const int rows = (int)min((long long)SC, a.T - s0);           // that the tensors have
    IO *dqg = (IO *)a.dq + b * a.sdq.s0 + hk * a.sdq.s1 + s0 * a.sdq.s2;
    IO *dkg = (IO *)a.dkk + b * a.sdk.s0 + hk * a.sdk.s1 + s0 * a.sdk.s2;
    const float zero4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n <= 0) {  // behind the sequence
        for (int i = tid; i < rows * (dk / 4); i += C::NTH) {
            const int t = i / (dk / 4), c = i % (dk / 4) * 4;
            store4(dqg + t * a.sdq.s2 + c, zero4);
            store4(dkg + t * a.sdk.s2 + c, zero4);
        }
        for (int h = hk * per; h < (hk + 1) * per; ++h) {
            IO *dvg = (IO *)a.dvv + b * a.sdv.s0 + h * a.sdv.s1 + s0 * a.sdv.s2;
            for (int i = tid; i < rows * (dv / 4); i += C::NTH) store4(dvg + i / (dv / 4) * a.sdv.s2 + i % (dv / 4) * 4, zero4);
            if (tid < rows) {
                a.dg[b * a.sdg.s0 + h * a.sdg.s1 + (s0 + tid) * a.sdg.s2] = 0.0f;
                a.db[b * a.sdb.s0 + h * a.sdb.s1 + (s0 + tid) * a.sdb.s2] = 0.0f;
            }
        }
        return;
    }
    // ---- K and Q
    {
        const IO *kp = (const IO *)a.k + b * a.sk.s0 + hk * a.sk.s1 + s0 * a.sk.s2;
        const IO *qp = (const IO *)a.q + b * a.sq.s0 + hk * a.sq.s1 + s0 * a.sq.s2;
        for (int i = tid; i < SC * QG; i += C::NTH) {
            const int r = i / QG, g = i % QG, c = g * EPG, at = (r * QG + (g ^ swz<QG>(r & 15))) * EPG;
            u32x4 x = {0, 0, 0, 0}, y = x;
            if (r < n && c < dk) {
                x = *(const u32x4 *)(kp + r * a.sk.s2 + c);
                y = *(const u32x4 *)(qp + r * a.sq.s2 + c);
            }
            *(u32x4 *)(kt + at) = x;
            *(u32x4 *)(qt + at) = y;
        }
    }
    f32x4 tq[SHARED ? RTW : 1][SHARED ? NT : 1], tk[SHARED ? RTW : 1][SHARED ? NT : 1];
    if constexpr (SHARED)
#pragma unroll
        for (int i = 0; i < RTW; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) tq[i][t] = tk[i][t] = f32x4{0, 0, 0, 0};
    // this wavefront's 16 tokens and block of a stage's columns where it splits, and whether
    // it makes E1 or E2 of those tokens (both if no other has the same tokens)
    const int rt = wave % NT, gq = wave / NT;
    const bool mine1 = gq == 0, mine2 = gq == (CB > 1 ? 1 : 0);
    auto put_rows = [&](int t, int x, f32x4 q, f32x4 k) {
        const int id = wave * RTW + x, c = 32 * (id >> 1) + 8 * (lane0 >> 4) + 4 * (id & 1), i = 16 * t + (lane0 & 15);
        if (i < rows && c < dk) {
            // rows behind the sequence's length are zeros, also where their zeros met a NaN of its own
            const bool own = i < n;
            float u[4], v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) u[r] = own ? q[r] : 0.0f, v[r] = own ? k[r] : 0.0f;
            store4(dqg + i * a.sdq.s2 + c, u);
            store4(dkg + i * a.sdk.s2 + c, v);
        }
    };

    for (int h = hk * per, end = SHARED ? h + per : h + 1; h < end; ++h) {
        const size_t cell = (size_t)b * a.H + h;
        // `fresh`: the addresses made from it are not kept over the heads
        const int lane = SHARED ? fresh(lane0) : lane0, l16 = lane & 15, g4 = lane >> 4;
        Cols<QG> cols;
        Rows<QG> krows;
        cols.init((const IO *)nullptr, l16, g4);
        krows.init((const IO *)nullptr, l16, g4);
        // element (token 16 t + l16, columns of tile x) of K and Q in LDS
        auto at_row = [&](int t, int x) {
            const int id = wave * RTW + x, c = 32 * (id >> 1) + 8 * g4 + 4 * (id & 1);
            return ((16 * t + l16) * QG + ((c / EPG) ^ swz<QG>(l16))) * EPG + c % EPG;
        };
        __syncthreads();
        if (tid < 64) {
            // gates of the block's tokens
            double G = 0.0;
            float beta = 0.0f;
            if (lane < n) {
                G = gate_log2(a.g[b * a.sg.s0 + h * a.sg.s1 + (s0 + lane) * a.sg.s2]);
                beta = a.beta[b * a.sb.s0 + h * a.sb.s1 + (s0 + lane) * a.sb.s2];
            }
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double x = __shfl_up(G, m);
                if (lane >= m) G += x;
            }
            const double GL = __shfl(G, 63), top = rint(G * 64.0) / 64.0;
            if (lane < SC) {
                hi[lane] = (float)top;
                lo[lane] = (float)(G - top);
                be[lane] = beta;
                eg[lane] = __builtin_amdgcn_exp2f((float)G);
                rest[lane] = __builtin_amdgcn_exp2f((float)(GL - G));
            }
        }
        __syncthreads();
        f32x4 aq[RTW][NT], ak1[RTW][NT], ak2[RTW][NT], e1[NT], e2[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            e1[t] = e2[t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < RTW; ++i) aq[i][t] = ak1[i][t] = ak2[i][t] = f32x4{0, 0, 0, 0};
        }
        const int tok = 16 * rt + l16;
        // uniform bases, 32-bit offsets of this lane's row (a block spans less than 2^30 bytes)
        const float *xr = in.x + (cell * a.T + s0) * dv, *ur = in.du + (cell * a.T + s0) * dv;
        const IO *gr = (const IO *)a.d_o + b * a.sdo.s0 + h * a.sdo.s1 + s0 * a.sdo.s2;
        const IO *ir = (const IO *)a.v + b * a.sv.s0 + h * a.sv.s1 + s0 * a.sv.s2;
        IO *vr = (IO *)a.dvv + b * a.sdv.s0 + h * a.sdv.s1 + s0 * a.sdv.s2;
        const unsigned xo = tok * dv, gof = tok * (int)a.sdo.s2, io = tok * (int)a.sv.s2, vo = tok * (int)a.sdv.s2;
        const float *sp = (const float *)in.s + (cell * nblk + blk) * ncb * NAT * 512 + wave * RTW * 512;
        const float *dp = (const float *)in.d + (cell * nblk + blk) * ncb * NAT * 512 + wave * RTW * 512;
        const float bt = be[tok];
        float dot = 0.0f, xu = 0.0f, vu = 0.0f;
        // rows of this wavefront's tokens in the next stage's block of columns
        Frag go, vi;
        f32x8 xn, un;
        auto fetch = [&](int base) {
            const unsigned c0 = 32 * (base + gq) + 8 * g4;
            const bool ok = tok < n && (int)c0 < dv;
            go = row8(gr + (gof + c0), ok);
            vi = row8(ir + (io + c0), ok);
            xn = row8(xr + (xo + c0), ok);
            un = row8(ur + (xo + c0), ok);
        };
        fetch(0);
        for (int base = 0; base < ncb; base += CB) {
            // S and D of this stage's first block are on their way while the rows are split
            f32x8 sn[RTW], dn[RTW];
            auto fetch_states = [&](int cb) {
#pragma unroll
                for (int i = 0; i < RTW; ++i) {
                    sn[i] = row8(sp + cb * NAT * 512 + i * 512 + lane * 8, true);
                    dn[i] = row8(dp + cb * NAT * 512 + i * 512 + lane * 8, true);
                }
            };
            fetch_states(base);
            if (base > 0) __syncthreads();
            if (base + gq < ncb) {
                const unsigned c0 = 32 * (base + gq) + 8 * g4;
                float y[8], z[8], w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] = xn[e];
                    z[e] = un[e];
                    w[e] = un[e] * bt;
                    xu += un[e] * xn[e];
                    vu += w[e] * (float)vi[e];
                }
                Frag *to = (Frag *)pool + (size_t)(gq * NT + rt) * NM * 64 + lane;
                Frag fx[SP], fu[OP];
                split8<SP>(y, fx);
                split8<OP>(z, fu);
                to[0] = go;
#pragma unroll
                for (int p = 0; p < SP; ++p) to[(1 + p) * 64] = fx[p];
#pragma unroll
                for (int p = 0; p < OP; ++p) to[(1 + SP + p) * 64] = fu[p];
                if (tok < rows && (int)c0 < dv) {
                    store4(vr + (vo + c0), w);
                    store4(vr + (vo + c0 + 4), w + 4);
                }
            }
            __syncthreads();
            if (base + CB < ncb) fetch(base + CB);
            for (int cbl = 0; cbl < CB && base + cbl < ncb; ++cbl) {
                const Frag *op = (const Frag *)pool + (size_t)cbl * NT * NM * 64 + lane;
                if (cbl > 0) fetch_states(base + cbl);
                // first all products with S and the scores, then those with D: the parts of one in
                // registers at a time
                Frag f[RTW][SP];
#pragma unroll
                for (int i = 0; i < RTW; ++i) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] = sn[i][e];
                        dot += sn[i][e] * dn[i][e];
                    }
                    split8<SP>(x, f[i]);
                }
                // scores of this wavefront's tokens i (lanes) with all tokens j <= i (rows)
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (t <= rt) {
                        __builtin_amdgcn_sched_barrier(0);  // keeps the operands of one tile in registers, not of all
                        if (mine1) {
                            const Frag g = op[rt * NM * 64];
#pragma unroll
                            for (int p = SP - 1; p >= 0; --p) e1[t] = mfma(op[(t * NM + 1 + p) * 64], g, e1[t]);
                        }
                        if (mine2) {
                            Frag fx[OP], fu[OP];
#pragma unroll
                            for (int p = 0; p < OP; ++p) {
                                fx[p] = op[(t * NM + 1 + p) * 64];
                                fu[p] = op[(rt * NM + 1 + SP + p) * 64];
                            }
                            e2[t] = mfma_parts<OP>(fx, fu, e2[t]);
                        }
                    }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    __builtin_amdgcn_sched_barrier(0);
                    const Frag g = op[t * NM * 64];
                    Frag fu[OP];
#pragma unroll
                    for (int p = 0; p < OP; ++p) fu[p] = op[(t * NM + 1 + SP + p) * 64];
#pragma unroll
                    for (int i = 0; i < RTW; ++i) {
#pragma unroll
                        for (int p = SP - 1; p >= 0; --p) aq[i][t] = mfma(f[i][p], g, aq[i][t]);
                        ak2[i][t] = mfma_parts<OP>(f[i], fu, ak2[i][t]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < RTW; ++i) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = dn[i][e];
                    split8<SP>(x, f[i]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    __builtin_amdgcn_sched_barrier(0);
                    Frag fx[SP];
#pragma unroll
                    for (int p = 0; p < SP; ++p) fx[p] = op[(t * NM + 1 + p) * 64];
#pragma unroll
                    for (int i = 0; i < RTW; ++i) ak1[i][t] = mfma_parts<SP>(f[i], fx, ak1[i][t]);
                }
            }
        }
        // the rows' own products: dbeta, and dV.v
        xu += __shfl_xor(xu, 16);
        vu += __shfl_xor(vu, 16);
        xu += __shfl_xor(xu, 32);
        vu += __shfl_xor(vu, 32);
        if (g4 == 0) {
            dbs[gq][tok] = xu;
            dgs[gq][tok] = -vu;
        }
        __syncthreads();
        // ---- E1 and -E2, decayed, to LDS over the operands; E1's part of do.o on the way
        IO *E1 = pool, *E2 = pool + OP * SC * SC;
        {
            const int i = tok;
            const float hii = hi[i], loi = lo[i];
            float qke = 0.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float x[4], y[4];
                const f32x4 hj = *(const f32x4 *)(hi + 16 * t + 4 * g4), lj = *(const f32x4 *)(lo + 16 * t + 4 * g4);
                const f32x4 bj = *(const f32x4 *)(be + 16 * t + 4 * g4);
                f32x4 qk = {0, 0, 0, 0};
                __builtin_amdgcn_sched_barrier(0);
                if (mine1 && t <= rt)
#pragma unroll
                    for (int kk = 0; kk < DKP / 32; ++kk)
                        qk = mfma(krows.get(kt + (t >> 1) * 32 * DKP, t & 1, kk), krows.get(qt + (rt >> 1) * 32 * DKP, rt & 1, kk), qk);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 16 * t + 4 * g4 + r;
                    const float M = j <= i ? __builtin_amdgcn_exp2f((hii - hj[r]) + (loi - lj[r])) * bj[r] : 0.0f;
                    x[r] = e1[t][r] * (M * a.scale);
                    y[r] = j < i ? -e2[t][r] * (M * bt) : 0.0f;
                    qke += x[r] * qk[r];
                }
                const int c = 16 * t + 4 * g4, at = i * SC + (((c / EPG) ^ swz<C::EG>(l16)) * EPG) + c % EPG;
#pragma unroll
                for (int p = 0; p < OP; ++p) {
                    float v[4], w[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const IO m = from_f<IO>(x[r]), o = from_f<IO>(y[r]);
                        v[r] = to_f(m);
                        w[r] = to_f(o);
                        x[r] -= v[r];
                        y[r] -= w[r];
                    }
                    if (mine1) store4(E1 + p * SC * SC + at, v);
                    if (mine2) store4(E2 + p * SC * SC + at, w);
                }
            }
            qke += __shfl_xor(qke, 16);
            qke += __shfl_xor(qke, 32);
            if (mine1 && g4 == 0) eqk[i] = qke;
        }
        // ---- the products with the state, scaled; their part of do.o and of <D, S_L>
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int i = 16 * t + l16;
            const float ei = eg[i], bi = be[i], ri = rest[i];
            float kd = 0.0f, qo = 0.0f;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int x = 0; x < RTW; ++x) {
                const int at = at_row(t, x);
                ak1[x][t] *= bi * ri;
                aq[x][t] *= a.scale * ei;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    kd += to_f(kt[at + r]) * ak1[x][t][r];
                    qo += to_f(qt[at + r]) * aq[x][t][r];
                }
                ak1[x][t] -= ak2[x][t] * (bi * ei);
            }
            kd += __shfl_xor(kd, 16);
            qo += __shfl_xor(qo, 16);
            kd += __shfl_xor(kd, 32);
            qo += __shfl_xor(qo, 32);
            if (g4 == 0) {
                part[0][wave][i] = qo;
                part[1][wave][i] = kd;
            }
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) dot += __shfl_xor(dot, m);
        if (lane == 0) dots[wave] = dot;
        __syncthreads();
        if (tid < 64) {
            // dlog_decay: sums from each token to the block's end, and what is behind it
            float x = 0.0f, y = 0.0f, z = 0.0f, tail = 0.0f;
            const bool ok = lane < n;
            if (ok) {
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    x += part[0][w][lane];
                    y += part[1][w][lane];
                }
                x += eqk[lane];
#pragma unroll
                for (int w = 0; w < CB; ++w) {
                    x += dgs[w][lane];
                    z += dbs[w][lane];
                }
            }
#pragma unroll
            for (int w = 0; w < NW; ++w) tail += dots[w];
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const float u = __shfl_down(x, m);
                if (lane + m < 64) x += u;
                y += __shfl_xor(y, m);
            }
            x += eg[SC - 1] * tail + y;
            if (lane < rows) {
                const float g = ok ? a.g[b * a.sg.s0 + h * a.sg.s1 + (s0 + lane) * a.sg.s2] : 0.0f;
                const bool gone = __builtin_amdgcn_exp2f(gate_log2(g)) == 0.0f;
                a.dg[b * a.sdg.s0 + h * a.sdg.s1 + (s0 + lane) * a.sdg.s2] = ok && !gone ? x : 0.0f;
                a.db[b * a.sdb.s0 + h * a.sdb.s1 + (s0 + lane) * a.sdb.s2] = ok ? z : 0.0f;
            }
        }
        // ---- the products within the block
#pragma unroll
        for (int ib = 0; ib < SC / 32; ++ib) {
            Frag kf[RTW], qf[RTW];
#pragma unroll
            for (int x = 0; x < RTW; ++x) {
                const int id = wave * RTW + x;
                kf[x] = cols.get(kt + ib * 32 * DKP, id >> 1, id & 1);
                qf[x] = cols.get(qt + ib * 32 * DKP, id >> 1, id & 1);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int p = OP - 1; p >= 0; --p) {
                    const IO *m1 = E1 + p * SC * SC, *m2 = E2 + p * SC * SC;
                    __builtin_amdgcn_sched_barrier(0);
                    if (ib <= t / 2) {
                        const Frag r1 = e_row<C::EG>(m1, 16 * t + l16, ib, g4), r2 = e_row<C::EG>(m2, 16 * t + l16, ib, g4);
#pragma unroll
                        for (int x = 0; x < RTW; ++x) {
                            aq[x][t] = mfma(kf[x], r1, aq[x][t]);
                            ak1[x][t] = mfma(kf[x], r2, ak1[x][t]);
                        }
                    }
                    if (ib >= t / 2) {
                        const Frag c1 = e_col<C::EG>(m1, ib, 16 * t, l16, g4), c2 = e_col<C::EG>(m2, ib, 16 * t, l16, g4);
#pragma unroll
                        for (int x = 0; x < RTW; ++x) {
                            ak1[x][t] = mfma(qf[x], c1, ak1[x][t]);
                            ak1[x][t] = mfma(kf[x], c2, ak1[x][t]);
                        }
                    }
                }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < RTW; ++x) {
                if constexpr (SHARED) {
                    tq[x][t] += aq[x][t];
                    tk[x][t] += ak1[x][t];
                } else {
                    put_rows(t, x, aq[x][t], ak1[x][t]);
                }
            }
    }
    if constexpr (SHARED)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < RTW; ++x) put_rows(t, x, tq[x][t], tk[x][t]);
}

// ---- launches

// Columns of a workgroup, and segments.  128 columns where that gives every compute unit a
// workgroup, else 64 (64 / 128 columns, bfloat16: 4096 tokens, 64 heads of 128 x 128 245 / 376 us, 192 heads
// 460 / 464, 64 heads of 256 x 512 867 / 638, backward 3663 / 3187; 256 heads of 128 x 128, 2048 tokens
// 283 / 292, 512 heads, 1024 tokens 290 / 269; 128 heads of 256 x 256, 1024 tokens 246 / 188, backward 1039 / 891;
// float32, 256 heads of 128 x 128, 1024 tokens 361 / 330, backward 1255 / 1212).  It counts blocks and not how
// full the last one is, and the backward's two walks as one, so it misses some calls: 256 heads of
// 64 x 64, 2048 tokens 165 / 221 (float32, 1024 tokens 147 / 200, backward 447 / 544), 256 heads of 128 x 192, 1024
// tokens 194 / 210; 32 heads of 256 x 512 backward, which stay with 64, 1868 / 1682.
//
// Segments where up to a quarter of the units would have a workgroup: they cost a second
// walk, of twice the columns (d_v and d_qk of them) where d_qk is as large as d_v, and the scan's
// steps, each longer than a chunk; so as many as make a workgroup a unit, and as
// sqrt(4 chunks), of at least 4 chunks.  Without / with, 4096 tokens of 128 x 128: 32 heads (64
// workgroups) 221 / 166 us, 48 heads 233 / 270; 8 heads of 256 x 512 (64) 354 / 248, 16 heads 363 / 425.  Where
// d_qk is the larger the first walk has more columns than d_v counts: 32 heads of 256 x 64 381 / 313, but 64
// heads (64 workgroups) 447 / 520.
// The backward's two walks run side by side and count both: 16 heads of 8192 tokens (2 x 32) 743 / 500 us,
// 32 heads of 4096 (2 x 64) 494 / 504, 8 heads of 256 x 512 (2 x 64) 719 / 840.
struct Plan {
    bool wide;
    int nseg, len;
};
Plan make_plan(size_t cells, int T, int dv, int walks) {
    Plan p;
    p.wide = cells * ((dv + 127) / 128) >= 256;
    const long long wgs = (long long)cells * ((dv + 63) / 64), nch = chunks(T);
    long long want = wgs * walks > 64 ? 1 : 256 / wgs;
    while (want > 1 && (want * want > 4 * nch || want * 4 > nch)) --want;
    p.len = (int)((nch + want - 1) / want + 1) / 2 * 2;  // whole blocks of the backward
    p.nseg = (int)((nch + p.len - 1) / p.len);
    return p;
}

// the walk's shape: f(DKP, NCT, NW) as constants
template <typename IO, typename F>
hipError_t with_shape(int dk, bool wide, F f) {
    using std::integral_constant;
    constexpr integral_constant<int, 1> one{};
    constexpr integral_constant<int, 2> two{};
    constexpr integral_constant<int, 4> four{};
    if (dk <= 64) return wide ? f(integral_constant<int, 64>{}, two, four) : f(integral_constant<int, 64>{}, one, four);
    if (dk <= 128) return wide ? f(integral_constant<int, 128>{}, two, four) : f(integral_constant<int, 128>{}, one, four);
    // two wavefronts a SIMD: one of 32 columns each does its vector and matrix instructions by
    // turns (64 heads of 256 x 512, 4096 tokens: 713 us, with four wavefronts of 32 columns 802)
    if constexpr (sizeof(IO) == 2)
        if (wide) return f(integral_constant<int, 256>{}, one, integral_constant<int, 8>{});
    return f(integral_constant<int, 256>{}, one, four);
}

template <typename IO, bool BWD>
void launch_prep(const DeltaArgs &a, char *rec, char *back, long long total, hipStream_t s) {
    const dim3 grid((unsigned)((total + kPrepWaves - 1) / kPrepWaves));
    if (a.dk <= 64)
        prep_kernel<IO, 64, BWD><<<grid, 64 * kPrepWaves, 0, s>>>(a, rec, back, total);
    else if (a.dk <= 128)
        prep_kernel<IO, 128, BWD><<<grid, 64 * kPrepWaves, 0, s>>>(a, rec, back, total);
    else
        prep_kernel<IO, 256, BWD><<<grid, 64 * kPrepWaves, 0, s>>>(a, rec, back, total);
}

// Workspace of the forward, floats from its start.
struct FwdWs {
    size_t rec, local, state, total;
};
FwdWs fwd_ws(size_t cells, int T, int dk, int dv, int io_bf16) {
    const Plan p = make_plan(cells, T, dv, 1);
    FwdWs w;
    w.rec = 0;
    w.local = w.rec + cells * (size_t)chunks(T) * (io_bf16 ? Rec<bf16, FORWARD>::BYTES : Rec<float, FORWARD>::BYTES) / 4;
    w.state = w.local + (p.nseg > 1 ? cells * p.nseg * dk * (dv + dk) : 0);
    w.total = w.state + (p.nseg > 1 ? cells * p.nseg * dk * dv : 0);
    return w;
}

template <typename IO>
hipError_t launch_fwd_t(const DeltaArgs &a, hipStream_t s) {
    constexpr bool BF = sizeof(IO) == 2;
    const size_t cells = (size_t)a.B * a.H;
    const FwdWs w = fwd_ws(cells, a.T, a.dk, a.dv, BF);
    const Plan p = make_plan(cells, a.T, a.dv, 1);
    char *rec = (char *)(a.ws + w.rec);
    const long long total = (long long)cells * chunks(a.T);
    launch_prep<IO, false>(a, rec, nullptr, total, s);
    const Segs sg{p.nseg, p.len, a.ws + w.local, a.ws + w.state};
    return with_shape<IO>(a.dk, p.wide, [&](auto dkp, auto nct, auto nw) {
        constexpr int DKP = decltype(dkp)::value, NCT = decltype(nct)::value, NW = decltype(nw)::value, BV = 16 * NCT * NW;
        const int vt = (a.dv + BV - 1) / BV, kt = (a.dk + BV - 1) / BV;
        const auto run = [&](auto parts) {
            constexpr int SP = decltype(parts)::value;
            if constexpr (NCT == 1 && NW == 4)
                if (p.nseg > 1) {
                    forward_kernel<IO, DKP, NCT, NW, SP, true><<<dim3((unsigned)(cells * p.nseg * (vt + kt))), 64 * NW, 0, s>>>(a, rec, sg);
                    const unsigned n = (unsigned)(cells * (a.dv / 16));
                    scan_kernel<DKP><<<dim3(n), 4 * DKP, 0, s>>>(a, a.S0, sg, nullptr, Segs{}, (int)n);
                }
            forward_kernel<IO, DKP, NCT, NW, SP, false><<<dim3((unsigned)(cells * p.nseg * vt)), 64 * NW, 0, s>>>(a, rec, sg);
        };
        if constexpr (!BF)
            run(std::integral_constant<int, 1>{});
        else if (a.S_T)
            run(std::integral_constant<int, 3>{});
        else
            run(std::integral_constant<int, 2>{});
        return hipGetLastError();
    });
}

// Workspace of the backward, bytes from its start; every part is a multiple of 16.
struct BwdWs {
    size_t rec, rec_back, x, du, s, d, local, state, local_back, state_back, total;
};
template <typename IO>
BwdWs bwd_ws(size_t cells, int T, int dk, int dv) {
    const size_t nch = (size_t)chunks(T), nblk = (nch * L + kBlock<IO> - 1) / kBlock<IO>;
    const int dkp = dk <= 64 ? 64 : dk <= 128 ? 128 : 256;
    const size_t states = cells * nblk * ((dv + 31) / 32) * (dkp / 16) * 2048;
    BwdWs w;
    w.rec = 0;
    w.rec_back = w.rec + cells * nch * Rec<IO, STATES>::BYTES;
    w.x = w.rec_back + cells * nch * Rec<IO, BACK>::BYTES;
    w.du = w.x + cells * T * dv * 4;
    w.s = w.du + cells * T * dv * 4;
    w.d = w.s + states;
    const Plan p = make_plan(cells, T, dv, 2);
    const size_t one = p.nseg > 1 ? cells * p.nseg * dk * 4 : 0;  // bytes of a column of all segments
    w.local = w.d + states;
    w.state = w.local + one * (dv + dk);
    w.local_back = w.state + one * dv;
    w.state_back = w.local_back + one * dv;
    w.total = w.state_back + one * dv;
    return w;
}

template <typename IO, bool SHARED>
hipError_t launch_grad(const DeltaArgs &a, const GradIn &in, dim3 grid, hipStream_t s) {
    if (a.dk <= 64)
        grad_kernel<IO, 64, 4, SHARED><<<grid, 256, 0, s>>>(a, in);
    else if (a.dk <= 128)
        grad_kernel<IO, 128, 4, SHARED><<<grid, 256, 0, s>>>(a, in);
    else
        grad_kernel<IO, 256, 8, SHARED><<<grid, 512, 0, s>>>(a, in);
    return hipGetLastError();
}

template <typename IO>
hipError_t launch_bwd_t(const DeltaArgs &a, hipStream_t s) {
    char *ws = (char *)a.ws;
    const size_t cells = (size_t)a.B * a.H;
    const BwdWs w = bwd_ws<IO>(cells, a.T, a.dk, a.dv);
    const long long total = (long long)cells * chunks(a.T);
    const Plan p = make_plan(cells, a.T, a.dv, 2);
    launch_prep<IO, true>(a, ws + w.rec, ws + w.rec_back, total, s);
    BackArgs k{};
    k.a = a;
    k.a.v = a.d_o;
    k.a.sv = a.sdo;
    k.a.S0 = a.dS_T;
    k.a.S_T = a.dS0;
    k.v = a.v;
    k.sv = a.sv;
    k.S0 = a.S0;
    k.rec = ws + w.rec;
    k.rec_back = ws + w.rec_back;
    k.to = WalkOut{(float *)(ws + w.x), ws + w.s};
    k.to_back = WalkOut{(float *)(ws + w.du), ws + w.d};
    k.sg = Segs{p.nseg, p.len, (float *)(ws + w.local), (float *)(ws + w.state)};
    k.sg_back = Segs{p.nseg, p.len, (float *)(ws + w.local_back), (float *)(ws + w.state_back)};
    const hipError_t e = with_shape<IO>(a.dk, p.wide, [&](auto dkp, auto nct, auto nw) {
        constexpr int DKP = decltype(dkp)::value, NCT = decltype(nct)::value, NW = decltype(nw)::value, BV = 16 * NCT * NW;
        const int vt = (a.dv + BV - 1) / BV, kt = (a.dk + BV - 1) / BV;
        k.nback = (int)(cells * p.nseg * vt);
        if constexpr (NCT == 1 && NW == 4)
            if (p.nseg > 1) {
                back_kernel<IO, DKP, NCT, NW, true><<<dim3((unsigned)(cells * p.nseg * (2 * vt + kt))), 64 * NW, 0, s>>>(k);
                const unsigned n = (unsigned)(cells * (a.dv / 16));
                scan_kernel<DKP><<<dim3(2 * n), 4 * DKP, 0, s>>>(a, a.S0, k.sg, a.dS_T, k.sg_back, (int)n);
            }
        back_kernel<IO, DKP, NCT, NW, false><<<dim3((unsigned)(2 * cells * p.nseg * vt)), 64 * NW, 0, s>>>(k);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    const GradIn in{(const float *)(ws + w.x), (const float *)(ws + w.du), ws + w.s, ws + w.d};
    const long long nblk = (chunks(a.T) * L + kBlock<IO> - 1) / kBlock<IO>;
    const dim3 grid((unsigned)((long long)a.B * a.Hk * nblk));
    return a.H == a.Hk ? launch_grad<IO, false>(a, in, grid, s) : launch_grad<IO, true>(a, in, grid, s);
}

}  // namespace

size_t deltarule_workspace_floats(int B, int H, int T, int dk, int dv, int io_bf16, int backward) {
    const size_t n = (size_t)B * H;
    if (!backward) return fwd_ws(n, T, dk, dv, io_bf16).total;
    return (io_bf16 ? bwd_ws<bf16>(n, T, dk, dv).total : bwd_ws<float>(n, T, dk, dv).total) / 4;
}

hipError_t launch_deltarule_fwd(const DeltaArgs &a, int io_bf16, hipStream_t s) {
    return io_bf16 ? launch_fwd_t<bf16>(a, s) : launch_fwd_t<float>(a, s);
}
hipError_t launch_deltarule_bwd(const DeltaArgs &a, int io_bf16, hipStream_t s) {
    return io_bf16 ? launch_bwd_t<bf16>(a, s) : launch_bwd_t<float>(a, s);
}

}  // namespace mlstm
