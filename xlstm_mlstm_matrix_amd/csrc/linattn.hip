// linattn.hip -- linear attention with a decay for each head, in chunks of
// L = 32 tokens on the matrix cores (forward, and the three passes of the
// backward).
//
// A pass (LinJob) carries a state X [dk x dv] through local tokens tau.  With
// tokens i, j of a chunk and n of them:
//   o_i = in_scale e^{g (i + 1 - shift)} X^T q_i
//         + sum_{j <= i} e^{g (i - j)} p_scale (q_i . k_j) v_j,
//   X  <- e^{g n} X + up_scale sum_j e^{g (n - 1 + shift - j)} k_j v_j^T.
// Every exponent is a number of steps times g <= 0, never a difference of
// large ones, so no decay overflows and -inf is an ordinary value.
//
// A workgroup owns a block of value columns of one (b, h) and segment and walks
// its chunks in order; a wavefront owns NCT tiles of 16 columns with all dk rows
// of X in registers (float32, accumulator layout).  Nothing is exchanged
// between wavefronts but the Q, K and V tiles in LDS: each computes the
// chunk's scores for itself (32 x 32 of them, a small part of its products),
// which saves a second barrier and a trip through LDS.
//
// Everything is computed transposed, so that each product's result is, lane by
// lane, the operand of the next one:
//   scores^T = K Q^T, lane: token i = l16, rows j           (accumulators)
//   o^T = X^T Q^T + V^T P^T, lane: token i = l16, value rows (P^T straight from the scores)
//   X += K^T (w V), lane: column l16, rows dk                (X^T straight from X)
// The MFMA's inner index may be permuted if both operands agree: slot e of
// lane group g4 stands for d_qk index 32 kk + 8 g4 + e, and for token
// 16 (e / 4) + 4 g4 + e % 4.
//
// Roundings (bfloat16 I/O).  The outputs are float32 work rounded once: the
// read-out's copy of X goes in two parts (8 + 8 bits), and so does P, each off by
// 2^-16 where the output's own rounding is off by 2^-8.  One part of X adds to
// the output as much as its rounding does (2.2e-3 root mean square instead of
// 1.7e-3), and far more where the products cancel; it is up to 19% faster (64 heads of
// 256 x 512 340 us instead of 418, 256 heads of 128 x 128 238 instead of 277).
// w_j v_j enters the state in three parts (8 + 8 + 8 bits of its 24) where the
// state is handed out: two parts would leave its float32 values 3e-6 off, three
// leave what float32 sums do.  Where nobody sees the state but the read-out,
// whose copy has 16 bits, two parts do.  X itself, every decay and every sum are
// float32.  float32 I/O runs on the float32 MFMA without further rounding.
//
// Measured (bfloat16, 4096 tokens, state handed out): 256 heads of 128 x 128 277
// us, 3.9 TB/s, where a large copy has 4.8; 64 heads of 256 x 512 418 us, 2.0
// TB/s.  There 256 workgroups leave a SIMD one wavefront, and its 879 vector
// instructions a chunk, 192 of them MFMA, overlap little.
#include "ops.hpp"

namespace mlstm {

namespace {

typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_ptr;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int L = 32;           // tokens of a chunk
constexpr int kBuf = 0x00020000; // word 3 of a raw, range-checked buffer descriptor
// An offset past any range: reads zero, writes nothing.  A chunk's range and the
// steps added to an offset are at most 2^29 bytes (32 rows of 2^22 floats), so it
// stays past the range, and below 2^32, whatever is added or taken away.
constexpr unsigned kOut = 0x80000000u;
constexpr size_t kLds = 160 * 1024;
constexpr long long kCUs = 256;  // compute units of an MI355X
constexpr float kRenorm = 9.094947e-13f;  // sigma's least value, 2^-40

struct KArgs {
    LinJob job[3];
    int tiles[3];       // column blocks of each job
    int njob, tiles_all;
    const float *g;
    const int *lengths;
    int B, H, T, nseg, seg_len;
    // incoming states of the segments: state (job, bh, seg) at
    // ws + ws_job[job] + (bh * nseg + seg) * tiles * block, in the register layout
    float *ws;
    size_t ws_job[3];
};

template <typename IO>
struct Types;
template <>
struct Types<bf16> {
    typedef bf16x8 Frag;
    static constexpr int EPG = 8;  // elements of a 16-byte granule
    static constexpr int PPARTS = 2, XPARTS = 2;  // parts of P, of the read-out's copy of X
};
template <>
struct Types<float> {
    typedef f32x8 Frag;
    static constexpr int EPG = 4;
    static constexpr int PPARTS = 1, XPARTS = 1;
};

__device__ __forceinline__ f32x4 mfma(const bf16x8 &a, const bf16x8 &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(const f32x8 &a, const f32x8 &b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

// 8 floats as one operand (rounded to nearest even for bfloat16)
__device__ __forceinline__ void pack(const float *x, bf16x8 &f) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const bf16x2 h = __builtin_convertvector((f32x2{x[2 * p], x[2 * p + 1]}), bf16x2);
        f[2 * p] = h[0];
        f[2 * p + 1] = h[1];
    }
}

// Two floats as a sum of PARTS roundings, elements 2 p and 2 p + 1 of PARTS
// operands: each part is the rounded rest of the one before.  `here` keeps the
// work in place: the compiler would move it behind the next branch.
template <int PARTS, bool HERE>
__device__ __forceinline__ void split2(float x0, float x1, bf16x8 *f, int p) {
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
        const bf16x2 h = __builtin_convertvector((f32x2{x0, x1}), bf16x2);
        unsigned b = __builtin_bit_cast(unsigned, h);
        if constexpr (HERE) asm volatile("" : "+v"(b));
        u32x4 w = __builtin_bit_cast(u32x4, f[q]);
        w[p] = b;
        f[q] = __builtin_bit_cast(bf16x8, w);
        x0 -= __uint_as_float(b << 16);
        x1 -= __uint_as_float(b & 0xffff0000u);
    }
}
template <int PARTS, bool HERE>
__device__ __forceinline__ void split2(float x0, float x1, f32x8 *f, int p) {
    f[0][2 * p] = x0;
    f[0][2 * p + 1] = x1;
}

// Granule swizzle of a tile with GPR granules a row: a row's granule p is
// stored at p ^ swz(row).  Rows are read whole-granule, 16 rows at a time at one
// granule (scores, read-out), and transposed, four rows 4 g + (0..3) at four
// neighbouring granules (state update, V); both then spread over the banks.
template <int GPR>
__device__ __forceinline__ int swz(int r) {
    if constexpr (GPR >= 16) return ((r & 3) << 2) | ((r >> 2) & 3);
    const int x = (r >> 1) & 7;
    return ((x & 1) << 2) | (x & 2) | ((x >> 2) & 1);
}


__device__ __forceinline__ s16x4 tr_read(const bf16 *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
}

// a value that is the same in all lanes, in a scalar register
__device__ __forceinline__ float uniform(float x) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// Wait until at most N of this wavefront's memory operations are outstanding
// (they complete in order).
template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N < 16, "four bits here");
    __builtin_amdgcn_s_waitcnt(0x0f70 | N);
}

// Whole-granule reads of a row: d_qk index 32 kk + 8 g4 + (0..7) of rows
// l16 and 16 + l16.  The swizzle touches the low four bits of the granule
// number at most, so one address per lane, some constant bits of it flipped, and
// constant offsets serve all kk.  `fresh` stops the compiler from keeping
// the flipped addresses in registers over the chunk loop.
__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}
template <int GPR>
struct Rows {
    static constexpr int M = GPR >= 16 ? 4 : 2;  // low parts of the granule number, in steps of 4
    int off;
    __device__ __forceinline__ void init(const bf16 *, int l16, int g4) {
        off = l16 * GPR * 8 + ((g4 ^ swz<GPR>(l16)) << 3);
    }
    __device__ __forceinline__ void init(const float *, int l16, int g4) {
        off = l16 * GPR * 4 + (((2 * g4) ^ swz<GPR>(l16)) << 2);
    }
    __device__ __forceinline__ bf16x8 get(const bf16 *t, int half, int kk) const {
        return *reinterpret_cast<const bf16x8 *>(t + (off ^ (32 * (kk % M))) + half * 16 * GPR * 8 + kk / M * M * 32);
    }
    __device__ __forceinline__ f32x8 get(const float *t, int half, int kk) const {
        f32x8 f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 x = *reinterpret_cast<const f32x4 *>(t + (off ^ (32 * (kk & 1) + 4 * h)) + half * 16 * GPR * 4 +
                                                             (kk >> 1) * 64);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * h + e] = x[e];
        }
        return f;
    }
};

// Transposed reads of all d_qk columns for the state update: columns
// 32 kk + 4 u + 8 a + (0..3) of quad a, tokens as in v_frag.
template <int GPR>
struct Cols {
    static constexpr int M = GPR >= 16 ? 4 : 2;
    int off, l16, g4;
    __device__ __forceinline__ void init(const bf16 *, int l, int g) {
        const int r0 = 4 * g + (l >> 2);
        off = r0 * GPR * 8 + (((l & 3) ^ swz<GPR>(r0)) << 3);
    }
    __device__ __forceinline__ void init(const float *, int l, int g) { off = 0, l16 = l, g4 = g; }
    __device__ __forceinline__ bf16x8 get(const bf16 *t, int kk, int u) const;
    __device__ __forceinline__ f32x8 get(const float *t, int kk, int u) const;
};

// Column l16 of 16 columns, tokens 16 (e / 4) + 4 g4 + e % 4 of the chunk.  The
// columns come in quads of 4 consecutive elements; quad a starts at element
// c0 + step * a (multiples of 4).
__device__ __forceinline__ bf16x8 tr_pair(const bf16 *p, int rows16) {
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const s16x4 a = tr_read(p), b = tr_read(p + rows16);
    const s16x8 r = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return __builtin_bit_cast(bf16x8, r);
}
// ... of a shared, swizzled V tile (rows of W elements)
template <int W>
__device__ __forceinline__ bf16x8 v_frag(const bf16 *t, int c0, int step, int l16, int g4) {
    const int r0 = 4 * g4 + (l16 >> 2), c = c0 + step * (l16 & 3);
    return tr_pair(t + r0 * W + (((c >> 3) ^ swz<W / 8>(r0)) << 3) + (c & 4), 16 * W);
}
// ... of a wavefront's own V tile (not swizzled)
template <int W>
__device__ __forceinline__ f32x8 v_frag(const float *t, int c0, int step, int l16, int g4) {
    const int c = c0 + step * (l16 >> 2) + (l16 & 3);
    f32x8 f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = t[(16 * (e >> 2) + 4 * g4 + (e & 3)) * W + c];
    return f;
}
// ... of a swizzled K tile
template <int GPR>
__device__ __forceinline__ bf16x8 Cols<GPR>::get(const bf16 *t, int kk, int u) const {
    return tr_pair(t + (off ^ (32 * (kk % M))) + kk / M * M * 32 + 4 * u, 16 * GPR * 8);
}
template <int GPR>
__device__ __forceinline__ f32x8 Cols<GPR>::get(const float *t, int kk, int u) const {
    const int c = 32 * kk + 4 * u + 8 * (l16 >> 2) + (l16 & 3);
    f32x8 f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int r = 16 * (e >> 2) + 4 * g4 + (e & 3);
        f[e] = t[r * GPR * 4 + (((c >> 2) ^ swz<GPR>(r)) << 2) + (c & 3)];
    }
    return f;
}

template <typename IO, int DKP_, int NCT_, int NW_>
struct Cfg {
    static constexpr int DKP = DKP_, NCT = NCT_, NW = NW_, NTH = 64 * NW_;
    static constexpr int BV = 16 * NCT * NW;               // value columns of a workgroup
    static constexpr int NAT = DKP / 16, NKS = DKP / 32;   // 16-row tiles of X, inner steps over d_qk
    static constexpr int EPG = Types<IO>::EPG;
    static constexpr int QG = DKP / EPG, VG = 16 * NCT / EPG, WG = BV / EPG;  // granules of a row: Q and K; a wavefront's V; V
    // V: with Q and K in the double-buffered tile; for float32, where that leaves no
    // room for a second workgroup, in one buffer a wavefront (its columns are
    // its own and go to registers at the start of the chunk).  The shared tile
    // moves whole rows: 10% faster for 64 bfloat16 columns.
    static constexpr bool VOWN = sizeof(IO) == 4;
    static constexpr int TROW = 2 * DKP + (VOWN ? 0 : BV);  // elements of a tile for each token
    static constexpr size_t TILE = (size_t)L * TROW * sizeof(IO), VTILE = VOWN ? (size_t)L * BV * sizeof(IO) : 0;
    static constexpr int NBUF = 2 * TILE + VTILE <= kLds ? 2 : 1;
    static constexpr bool EARLY = NCT == 1 || DKP < 256;  // else the registers do not suffice
    static constexpr int PER_CU = 2 * (NBUF * TILE + VTILE) <= kLds && NW == 4 ? 2 : 1;  // workgroups of a compute unit
    static constexpr int BLOCK = DKP * BV;                 // floats of a stored state block
    static_assert(QG >= 8, "swizzle");
    static_assert(TILE + VTILE <= kLds, "LDS");
};

// SO (state only): the first pass over segments, each from the zero state.
// PARTS: parts of w v (1 for float32).
template <typename IO, int DKP, int NCT, int NW, int PARTS, bool SO>
__global__ __launch_bounds__(64 * NW, (Cfg<IO, DKP, NCT, NW>::PER_CU * NW / 4)) void linattn_kernel(KArgs a) {
    using C = Cfg<IO, DKP, NCT, NW>;
    using Frag = typename Types<IO>::Frag;
    constexpr int NAT = C::NAT, NKS = C::NKS, QG = C::QG, VG = C::VG, BV = C::BV, NBUF = C::NBUF;
    constexpr int PPARTS = Types<IO>::PPARTS, XPARTS = Types<IO>::XPARTS;
    constexpr int ES = (int)sizeof(IO);
    // Q and K tiles of a chunk, double buffered where two fit.  Two arrays and
    // a loop over pairs of chunks, not one array indexed by parity: the compiler
    // waits for a copy in flight before any LDS read that may alias it.
    __shared__ __attribute__((aligned(16))) IO tile0[L * C::TROW];
    __shared__ __attribute__((aligned(16))) IO tile1[NBUF == 2 ? L * C::TROW : 16];
    __shared__ __attribute__((aligned(16))) IO vtiles[NW][C::VOWN ? L * 16 * NCT : 8];

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // consecutive workgroups go round the 8 XCDs: give each XCD a contiguous
    // run, so that the column blocks of one (b, h) share its L2
    const int nwg = gridDim.x, xq = nwg >> 3, xr = nwg & 7, xcd = blockIdx.x & 7;
    const int logical = xcd * xq + min(xcd, xr) + (blockIdx.x >> 3);
    const int gseg = SO ? a.nseg - 1 : a.nseg;
    int tile = logical % a.tiles_all, ji = 0;
    while (tile >= a.tiles[ji]) tile -= a.tiles[ji++];
    const int seg = logical / a.tiles_all % gseg, bh = logical / a.tiles_all / gseg;
    const LinJob &job = a.job[ji];
    const int b = bh / a.H, h = bh % a.H;
    const int dk = job.dk, dv = job.dv, T = a.T;
    const int n = a.lengths ? max(0, min(a.lengths[b], T)) : T;
    const int tau0 = seg * a.seg_len, tau1 = min(tau0 + a.seg_len, n);
    if (SO && tau0 + a.seg_len >= n) return;  // no later segment
    const int col0 = tile * BV;
    const int ldq = (int)job.sq.s2, ldk = (int)job.sk.s2, ldv = (int)job.sv.s2, ldo = (int)job.so.s2;
    const IO *qg = (const IO *)job.q + b * job.sq.s0 + h * job.sq.s1;
    const IO *kg = (const IO *)job.k + b * job.sk.s0 + h * job.sk.s1;
    const IO *vg = (const IO *)job.v + b * job.sv.s0 + h * job.sv.s1 + col0;
    IO *og = (IO *)job.o + b * job.so.s0 + h * job.so.s1 + col0;
    const bool rev = job.reverse;

    // ---- decays
    const float gl = decay_log2(a.g[h]);
    const auto gpow = [&](int steps) { return __builtin_amdgcn_exp2f(gl * (float)steps); };
    // Weights are products of a lane's own power and powers common to the
    // workgroup (scalar registers), all with exponents >= 0.
    // P of the score tile below the diagonal: e^{g (16 + l16 - 4 g4 - r)}
    const float below = gpow(13 + l16 - 4 * g4) * job.p_scale;
    // token 16 (e / 4) + 4 g4 + e % 4 in the state update: a chunk of nc < L tokens
    // fills its last rows, behind rows of zeros, so the weights are always these
    const float wlane = gpow(12 - 4 * g4 + job.shift) * job.up_scale;
    float upow[8];  // e^{g (19 - 16 (e / 4) - e % 4)}: the upper four are e^{g (3 - r)}
#pragma unroll
    for (int e = 0; e < 8; ++e) upow[e] = uniform(gpow(19 - 16 * (e >> 2) - (e & 3)));

    // ---- state.  Lane (l16, g4) of tile (at, bt) holds rows krow(at) + r
    // of column vcol(bt)
    const int vq = NCT == 2 ? 8 : 4;  // distance of a wavefront's column quads
    const int vc0 = wave * 16 * NCT;
    const int vcol = vc0 + vq * (l16 >> 2) + (l16 & 3);  // + 4 bt
    auto krow = [&](int at) { return 32 * (at >> 1) + 8 * g4 + 4 * (at & 1); };
    f32x4 X[NAT][NCT];
    const size_t cell = (size_t)bh * dk * dv;
    // byte offset of row krow(at), column vcol + 4 bt in one (b, h)'s state as the caller has it
    const int rs = (int)job.rs * 4, cs = (int)job.cs * 4;
    auto state_at = [&](int at, int bt) {
        return krow(at) < dk && col0 + vcol + 4 * bt < dv ? (unsigned)(krow(at) * rs + (col0 + vcol + 4 * bt) * cs)
                                                          : kOut;
    };
    float *slot = a.ws ? a.ws + a.ws_job[ji] + ((size_t)(bh * a.nseg + seg) * a.tiles[ji] + tile) * C::BLOCK +
                             (size_t)wave * NAT * NCT * 256 + lane * 4
                       : nullptr;
    if (!SO && a.nseg > 1 && (tau0 == 0 || tau0 < n)) {
#pragma unroll
        for (int at = 0; at < NAT; ++at)
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) X[at][bt] = *(const f32x4 *)(slot + (at * NCT + bt) * 256);
    } else if (!SO && a.nseg == 1 && job.X0) {
        const auto xs = __builtin_amdgcn_make_buffer_rsrc((void *)(job.X0 + cell), 0, dk * dv * 4, kBuf);
#pragma unroll
        for (int at = 0; at < NAT; ++at)
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) {
                const unsigned off = state_at(at, bt);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    X[at][bt][r] = __uint_as_float(
                        __builtin_amdgcn_raw_buffer_load_b32(xs, off == kOut ? kOut : off + r * rs, 0, 0));
            }
    } else {
#pragma unroll
        for (int at = 0; at < NAT; ++at)
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) X[at][bt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // ---- chunks.  Chunk c has tokens tau0 + c L ..., nc of them, the lowest in
    // memory is lo; row r of its tiles is local token r - (L - nc).
    const int nch = tau1 > tau0 ? (tau1 - tau0 + L - 1) / L : 0;
    auto chunk = [&](int c, int &nc, int &lo) {
        const int s = tau0 + c * L;
        nc = max(0, min(L, tau1 - s));  // 0 past the last chunk: its copies read nothing
        lo = rev ? n - s - nc : s;
    };
    // Byte offset of (row, element col) from token lo: rows run up or down in
    // memory.  Rows in front of a short chunk come out below zero or past
    // nc rows: either way out of the descriptor's range, so they read as zero
    // and are not written.
    auto row_off = [&](int row, int ld, int col) { return (unsigned)(((rev ? L - 1 - row : row) * ld + col) * ES); };
    auto short_by = [&](int nc, int ld) { return rev ? 0u : (unsigned)((L - nc) * ld * ES); };
    // Tile copies: 64 granules of LDS per wavefront and instruction, the swizzle
    // is in the source address; columns past the tensor's read as zero.  The
    // swizzle repeats every 16 rows, so a few per-lane offsets serve all instructions.
    auto copy_offsets = [&](unsigned *off, int ld, int ncol, auto gpr_c) {
        constexpr int GPR = decltype(gpr_c)::value, RPI = C::NTH / GPR;
        static_assert(L * GPR % C::NTH == 0, "whole instructions");
#pragma unroll
        for (int i = 0; i < (RPI >= 16 ? 1 : 16 / RPI); ++i) {
            const int gi = i * C::NTH + tid, row = gi / GPR, col = ((gi % GPR) ^ swz<GPR>(row)) * C::EPG;
            off[i] = col < ncol ? row_off(row, ld, col) : kOut;
        }
    };
    // instructions [i0, i1) of a tile's copy
    auto copy = [&](IO *dst, const IO *src, int ld, const unsigned *off, auto gpr_c, int lo, int nc, int i0, int i1) {
        constexpr int GPR = decltype(gpr_c)::value, RPI = C::NTH / GPR, PER = RPI >= 16 ? 1 : 16 / RPI;
        const auto rs = __builtin_amdgcn_make_buffer_rsrc((void *)(src + (size_t)lo * ld), 0,
                                                          __builtin_amdgcn_readfirstlane(nc * ld * ES), kBuf);
        const unsigned sb = short_by(nc, ld), step = (unsigned)((rev ? -RPI : RPI) * ld * ES);
#pragma unroll
        for (int i = i0; i < i1; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr *)(dst + (i * NW + wave) * 64 * C::EPG), 16,
                                                     off[i % PER] + (i / PER * PER * step - sb), 0, 0, 0);
    };
    using QGc = std::integral_constant<int, QG>;
    using WGc = std::integral_constant<int, C::WG>;
    constexpr int NI = L * QG / C::NTH, NIV = L * C::WG / C::NTH;
    constexpr int QPER = 16 * QG > C::NTH ? 16 * QG / C::NTH : 1, WPER = 16 * C::WG > C::NTH ? 16 * C::WG / C::NTH : 1;
    unsigned qoff[QPER], koff[QPER], voff[WPER], ownoff = kOut;
    if constexpr (!SO) copy_offsets(qoff, ldq, dk, QGc{});
    copy_offsets(koff, ldk, dk, QGc{});
    constexpr int VI = L * VG / 64;  // own tile: 64 / VG rows an instruction
    if constexpr (C::VOWN) {
        const int col = vc0 + lane % VG * C::EPG;
        ownoff = col0 + col < dv ? row_off(lane / VG, ldv, col) : kOut;
    } else {
        copy_offsets(voff, ldv, dv - col0, WGc{});
    }
    // part p of np of the copies of chunk c's shared tile
    auto load = [&](IO *t, int c, int p, int np) {
        int nc, lo;
        chunk(c, nc, lo);
        if constexpr (!SO) copy(t, qg, ldq, qoff, QGc{}, lo, nc, p * NI / np, (p + 1) * NI / np);
        copy(t + L * DKP, kg, ldk, koff, QGc{}, lo, nc, p * NI / np, (p + 1) * NI / np);
        if constexpr (!C::VOWN) copy(t + 2 * L * DKP, vg, ldv, voff, WGc{}, lo, nc, p * NIV / np, (p + 1) * NIV / np);
    };
    // this wavefront's own V tile
    IO *own = vtiles[wave];
    auto load_v = [&](int c) {
        int nc, lo;
        chunk(c, nc, lo);
        const auto rs = __builtin_amdgcn_make_buffer_rsrc((void *)(vg + (size_t)lo * ldv), 0,
                                                          __builtin_amdgcn_readfirstlane(nc * ldv * ES), kBuf);
        const unsigned sb = short_by(nc, ldv), step = (unsigned)((rev ? -64 / VG : 64 / VG) * ldv * ES);
#pragma unroll
        for (int i = 0; i < VI; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr *)(own + i * 64 * C::EPG), 16,
                                                     ownoff + (i * step - sb), 0, 0, 0);
    };

    Rows<QG> rows0;
    Cols<QG> cols0;
    rows0.init((const IO *)nullptr, l16, g4);
    cols0.init((const IO *)nullptr, l16, g4);
    // this lane's outputs: tokens l16 and 16 + l16, columns vc0 + vq g4 + (0 .. 4 NCT - 1)
    const int ocol = vc0 + vq * g4;
    const bool ook = col0 + ocol < dv;
    int held = 0;  // X is held divided by sigma = e^{g held}
    float sigma = 1.0f;
    // memory operations of a chunk issued after its copies of the next one: the stores of o
    constexpr int NST = SO ? 0 : 2 * (ES == 4 ? NCT : 1);
    // w v among the read-out's products, where the registers allow it
    constexpr bool EARLY = !SO && C::EARLY;
    // Copies in front of the read-out; among its steps for 512 rows only (backward
    // of 32 heads of 256 x 512 689 us instead of 715, no difference for fewer rows).
    constexpr bool SPREAD = !SO && NKS > 8;
    // Order of a chunk's work: each step's LDS reads are issued a step ahead of
    // the products that use them, and the elementwise work (w v, P, the
    // output) sits between products that do not depend on it.  sched_barrier
    // keeps the steps apart; within one the compiler orders freely.
    auto body = [&](IO *cur, IO *next, int c) {
        if (NBUF == 1) {
            __syncthreads();
            load(cur, c, 0, 1);
            wait_vm<0>();
        } else if (c == 0) {
            wait_vm<0>();
        } else {
            wait_vm<NST>();  // this wavefront's copies have landed
        }
        __syncthreads();
        int nc, lo;
        chunk(c, nc, lo);
        const IO *Qs = cur, *Ks = Qs + L * DKP;
        Rows<QG> rows = rows0;
        Cols<QG> cols = cols0;
        if constexpr (!C::EARLY) {
            rows.off = fresh(rows.off);
            cols.off = fresh(cols.off);
        }
        Frag vf[NCT], vw[NCT][PARTS], kf[2][2], q[2][2], k[2][2];
#pragma unroll
        for (int bt = 0; bt < NCT; ++bt) vf[bt] = C::VOWN ? v_frag<16 * NCT>((const IO *)own, 4 * bt, vq, l16, g4)
                             : v_frag<BV>(cur + 2 * L * DKP, vc0 + 4 * bt, vq, l16, g4);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if constexpr (SO) {
                kf[0][t] = cols.get(Ks, 0, t);
            } else {
                q[0][t] = rows.get(Qs, t, 0);
                k[0][t] = rows.get(Ks, t, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (NBUF == 2 && !SPREAD) load(next, c + 1, 0, 1);
        __builtin_amdgcn_sched_barrier(0);
        // The decay of X costs nothing while sigma carries it, and no rounded
        // factor is applied again and again; below kRenorm it is folded in.
        const float fade = sigma * job.in_scale;
        held += nc;
        sigma = gpow(held);
        const bool renorm = !(sigma >= kRenorm && sigma <= 1.0f / kRenorm);
        const float fold = sigma;
        if (renorm) {
            held = 0;
            sigma = 1.0f;
        }
        const float inv = gpow(-held);

        // parts of w v: elements 2 p and 2 p + 1 of tile bt
        const float winv = wlane * inv;
        auto weigh = [&](int bt, int p) {
            split2<PARTS, EARLY>((float)vf[bt][2 * p] * (upow[2 * p] * winv), (float)vf[bt][2 * p + 1] * (upow[2 * p + 1] * winv),
                   vw[bt], p);
        };
        f32x4 O[2][NCT], S00 = {0, 0, 0, 0}, S10 = S00, S11 = S00;
        if constexpr (!SO) {
            // read-out of the carried state and scores, one pass over d_qk
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int bt = 0; bt < NCT; ++bt) O[t][bt] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int kk = 0; kk < NKS; ++kk) {
                if constexpr (NBUF == 2 && SPREAD) load(next, c + 1, kk, NKS);
                __builtin_amdgcn_sched_barrier(0);
                const int u = kk & 1;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (kk + 1 < NKS) {
                        q[u ^ 1][t] = rows.get(Qs, t, kk + 1);
                        k[u ^ 1][t] = rows.get(Ks, t, kk + 1);
                    } else {
                        kf[0][t] = cols.get(Ks, 0, t);
                    }
                }
                Frag xf[NCT][XPARTS];
#pragma unroll
                for (int bt = 0; bt < NCT; ++bt) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = X[2 * kk + (e >> 2)][bt][e & 3];
#pragma unroll
                    for (int p = 0; p < 4; ++p) split2<XPARTS, false>(x[2 * p], x[2 * p + 1], xf[bt], p);
                }
                S00 = mfma(k[u][0], q[u][0], S00);
                S10 = mfma(k[u][0], q[u][1], S10);
                S11 = mfma(k[u][1], q[u][1], S11);
#pragma unroll
                for (int r = 0; r < XPARTS; ++r)
#pragma unroll
                    for (int bt = 0; bt < NCT; ++bt)
#pragma unroll
                        for (int t = 0; t < 2; ++t) O[t][bt] = mfma(xf[bt][r], q[u][t], O[t][bt]);
#pragma unroll
                for (int i = 0; i < 4 * NCT; ++i)
                    if (EARLY && i * NKS / (4 * NCT) == kk) weigh(i >> 2, i & 3);
            }
        }
        if constexpr (!EARLY) {
#pragma unroll
            for (int i = 0; i < 4 * NCT; ++i) weigh(i >> 2, i & 3);
        }
        if constexpr (C::VOWN) {
            // V's next rows over this chunk's, whose reads have returned
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) asm volatile("" : "+v"(vf[bt]));
            __builtin_amdgcn_sched_barrier(0);
            load_v(c + 1);
        }
        if (renorm) {
#pragma unroll
            for (int at = 0; at < NAT; ++at)
#pragma unroll
                for (int bt = 0; bt < NCT; ++bt) X[at][bt] *= fold;
        }

        // the output, in three pieces that the state update's steps take along
        Frag P[2][PPARTS];
        auto scores = [&]() {
            float p0[8], p1[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = l16 - 4 * g4 - r;  // token j <= i: d >= 0
                const float diag = gpow(max(d, 0)) * job.p_scale;
                p0[r] = d >= 0 ? S00[r] * diag : 0.0f;
                p0[4 + r] = 0.0f;
                p1[r] = S10[r] * (upow[4 + r] * below);
                p1[4 + r] = d >= 0 ? S11[r] * diag : 0.0f;
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                split2<PPARTS, false>(p0[2 * p], p0[2 * p + 1], P[0], p);
                split2<PPARTS, false>(p1[2 * p], p1[2 * p + 1], P[1], p);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                // steps since the state was carried in; rows in front of a short chunk are not tokens
                const float f = gpow(max(16 * t + l16 + 1 - job.shift - (L - nc), 0)) * fade;
#pragma unroll
                for (int bt = 0; bt < NCT; ++bt) O[t][bt] *= f;
            }
        };
        auto values = [&]() {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int bt = 0; bt < NCT; ++bt)
#pragma unroll
                    for (int q = 0; q < PPARTS; ++q) O[t][bt] = mfma(vf[bt], P[t][q], O[t][bt]);
        };
        auto output = [&]() {
            const auto os = __builtin_amdgcn_make_buffer_rsrc((void *)(og + (size_t)lo * ldo), 0,
                                                              __builtin_amdgcn_readfirstlane(nc * ldo * ES), kBuf);
            const unsigned sb = short_by(nc, ldo);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const unsigned at = ook ? row_off(16 * t + l16, ldo, ocol) - sb : kOut;
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
        // state update
#pragma unroll
        for (int kk = 0; kk < NKS; ++kk) {
            __builtin_amdgcn_sched_barrier(0);
            if (kk + 1 < NKS) {
#pragma unroll
                for (int t = 0; t < 2; ++t) kf[(kk + 1) & 1][t] = cols.get(Ks, kk + 1, t);
            }
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int bt = 0; bt < NCT; ++bt)
                        X[2 * kk + t][bt] = mfma(kf[kk & 1][t], vw[bt][q], X[2 * kk + t][bt]);
            if constexpr (!SO) {
                if (kk == 0) scores();
                if (kk == 1) values();
                if (kk == 2) output();
            }
        }
        if constexpr (!SO && NKS == 2) output();
    };
    if (nch > 0) {
        if (NBUF == 2) load(tile0, 0, 0, 1);
        if constexpr (C::VOWN) load_v(0);
    }
    for (int c = 0; c < nch; c += 2) {
        body(tile0, tile1, c);
        if (c + 1 < nch) body(NBUF == 2 ? tile1 : tile0, tile0, c + 1);
    }
    wait_vm<0>();  // no copy may still be on its way into LDS when the workgroup ends

    // ---- state out
#pragma unroll
    for (int at = 0; at < NAT; ++at)
#pragma unroll
        for (int bt = 0; bt < NCT; ++bt) X[at][bt] *= sigma;
    if constexpr (SO) {
        // the segment's own sum goes where the next one's incoming state will be
        float *next = slot + (size_t)a.tiles[ji] * C::BLOCK;
#pragma unroll
        for (int at = 0; at < NAT; ++at)
#pragma unroll
            for (int bt = 0; bt < NCT; ++bt) *(f32x4 *)(next + (at * NCT + bt) * 256) = X[at][bt];
    } else {
        const int last = n > 0 ? (n - 1) / a.seg_len : 0;
        if (job.Xn && seg == last) {
            const auto xs = __builtin_amdgcn_make_buffer_rsrc((void *)(job.Xn + cell), 0, dk * dv * 4, kBuf);
#pragma unroll
            for (int at = 0; at < NAT; ++at)
#pragma unroll
                for (int bt = 0; bt < NCT; ++bt) {
                    const unsigned off = state_at(at, bt);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(X[at][bt][r]), xs,
                                                              off == kOut ? kOut : off + r * rs, 0, 0);
                }
        }
        // rows behind the sequence's length
        const int z1 = min(tau0 + a.seg_len, T);
        constexpr int QPR = BV / 4;  // quads of a row
        const long long quads = (long long)max(z1 - max(n, tau0), 0) * QPR;
        for (long long e = tid; e < quads; e += C::NTH) {
            const long long t = max(n, tau0) + e / QPR;
            const int c = (int)(e % QPR) * 4;
            if (col0 + c < dv) {
                if constexpr (ES == 4)
                    *(f32x4 *)(og + t * ldo + c) = f32x4{0, 0, 0, 0};
                else
                    *(u32x2 *)(og + t * ldo + c) = u32x2{0, 0};
            }
        }
    }
}

// Segments' own sums -> their incoming states: in_0 = X0, in_{s+1} = e^{g
// seg_len} in_s + own_s, in place, elementwise; one thread for 4 rows of a column.
template <int DKP, int NCT, int NW>
__global__ __launch_bounds__(256) void linattn_scan_kernel(KArgs a) {
    constexpr int BV = 16 * NCT * NW, BLOCK = DKP * BV, NAT = DKP / 16;
    const int e = blockIdx.x * 256 + threadIdx.x;  // quad of the state's blocks
    const int bh = blockIdx.y, ji = blockIdx.z;
    const LinJob &job = a.job[ji];
    if (e >= a.tiles[ji] * (BLOCK / 4)) return;
    const int b = bh / a.H, h = bh % a.H;
    const int n = a.lengths ? max(0, min(a.lengths[b], a.T)) : a.T;
    const int tile = e / (BLOCK / 4), x = e % (BLOCK / 4);
    const int lane = x & 63, l16 = lane & 15, g4 = lane >> 4;
    const int bt = (x >> 6) % NCT, at = (x >> 6) / NCT % NAT, wave = x / (64 * NCT * NAT);
    const int row = 32 * (at >> 1) + 8 * g4 + 4 * (at & 1);
    const int col = tile * BV + wave * 16 * NCT + (NCT == 2 ? 8 : 4) * (l16 >> 2) + (l16 & 3) + 4 * bt;
    // e^{g seg_len} in two parts: a rounded factor just below 1, applied once a
    // segment, would pull the state 1.5e-5 off over 511 of them
    const double fd = exp2((double)decay_log2(a.g[h]) * (double)a.seg_len);
    const float f = (float)fd, fl = (float)(fd - (double)f);
    f32x4 run = {0, 0, 0, 0};
    if (job.X0)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (row + r < job.dk && col < job.dv)
                run[r] = job.X0[(size_t)bh * job.dk * job.dv + (row + r) * job.rs + col * job.cs];
    const size_t step = (size_t)a.tiles[ji] * BLOCK;
    float *s = a.ws + a.ws_job[ji] + (size_t)bh * a.nseg * step + (size_t)e * 4;
    *(f32x4 *)s = run;
    // eight segments' loads in flight: one at a time the chain of 64 segments is
    // bound by their latency (24 us where this takes 15)
    constexpr int AHEAD = 8;
    const int count = n > 0 ? (n - 1) / a.seg_len : 0;  // segments after the first
    for (int i = 0; i < count; i += AHEAD) {
        f32x4 own[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (i + j < count) own[j] = *(const f32x4 *)(s + (size_t)(i + j + 1) * step);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (i + j < count) {
                run = run * f + (run * fl + own[j]);
                *(f32x4 *)(s + (size_t)(i + j + 1) * step) = run;
            }
    }
}

// ---- plans

// One launch: the jobs of a call whose rows are padded to the same width.
struct Group {
    int dkp, bv;              // rows padded to 64, 128, 256 or 512; columns of a workgroup
    int njob, job[3], tiles[3], tiles_all;
    int nseg, seg_len;
    size_t ws_job[3];         // floats from the workspace's start
};
struct Plan {
    int ngroup;
    Group group[3];
    size_t floats;            // of workspace
};

// Columns of a workgroup and segments of a sequence, for enough workgroups to
// fill the 256 compute units.  128 columns move Q and K through LDS half as
// often as 64 do; segments cost a second reading of K and V and the states'
// way through memory; so: 128 if that gives a workgroup each, else 64 if that
// does, else 128 and segments for two each (of at least four chunks).  Measured
// (bfloat16, 4096 tokens): backward of 64 heads of 128 x 128 238 us with 64
// columns, 241 with 128 and segments; of 32 heads of 256 x 512 689 against 758.
// Segments for two workgroups a unit against one: forward of 128 heads of
// 64 x 64 88 us against 113, of 64 heads of 128 x 128 101 against 106.
Plan make_plan(int B, int H, int T, int dk, int dv, int io_bf16, int backward) {
    Plan p{};
    const int dims[3][2] = {{backward ? dv : dk, backward ? dk : dv}, {dk, dv}, {dv, dk}};
    const long long cells = (long long)B * H;
    for (int j = 0; j < (backward ? 3 : 1); ++j) {
        const int r = dims[j][0], dkp = r <= 64 ? 64 : r <= 128 ? 128 : r <= 256 ? 256 : 512;
        int i = 0;
        while (i < p.ngroup && p.group[i].dkp != dkp) ++i;
        if (i == p.ngroup) p.group[p.ngroup++].dkp = dkp;
        Group &g = p.group[i];
        g.job[g.njob++] = j;
    }
    for (int i = 0; i < p.ngroup; ++i) {
        Group &g = p.group[i];
        long long n64 = 0, n128 = 0;
        bool wide = false;
        for (int k = 0; k < g.njob; ++k) {
            const int c = dims[g.job[k]][1];
            n64 += cells * ((c + 63) / 64);
            n128 += cells * ((c + 127) / 128);
            wide |= c > 64;
        }
        // 512 float32 rows: the tiles fill LDS
        if (g.dkp == 512 && !io_bf16) wide = false;
        g.bv = wide && (n128 >= kCUs || n64 < kCUs) ? 128 : 64;
        const long long wgs = g.bv == 128 ? n128 : n64;
        const int nch = (T + L - 1) / L;
        long long want = wgs >= kCUs ? 1 : (2 * kCUs + wgs - 1) / wgs;
        if (want > nch / 4) want = nch / 4;
        if (want < 1) want = 1;
        g.seg_len = (int)((nch + want - 1) / want) * L;
        g.nseg = (T + g.seg_len - 1) / g.seg_len;
        for (int k = 0; k < g.njob; ++k) {
            g.tiles[k] = (dims[g.job[k]][1] + g.bv - 1) / g.bv;
            g.tiles_all += g.tiles[k];
            g.ws_job[k] = p.floats;
            if (g.nseg > 1) p.floats += (size_t)cells * g.nseg * g.tiles[k] * g.dkp * g.bv;
        }
    }
    return p;
}

template <typename IO, int DKP, int NCT, int NW, int PARTS>
hipError_t launch_parts(const KArgs &a, hipStream_t s) {
    const int cells = a.B * a.H;
    if (a.nseg > 1) {
        linattn_kernel<IO, DKP, NCT, NW, PARTS, true><<<dim3((unsigned)(cells * (a.nseg - 1) * a.tiles_all)), 64 * NW, 0, s>>>(a);
        int most = 0;
        for (int i = 0; i < a.njob; ++i) most = a.tiles[i] > most ? a.tiles[i] : most;
        const int quads = most * DKP * 4 * NCT * NW;
        linattn_scan_kernel<DKP, NCT, NW><<<dim3((unsigned)((quads + 255) / 256), (unsigned)cells, (unsigned)a.njob), 256, 0, s>>>(a);
    }
    linattn_kernel<IO, DKP, NCT, NW, PARTS, false><<<dim3((unsigned)(cells * a.nseg * a.tiles_all)), 64 * NW, 0, s>>>(a);
    return hipGetLastError();
}

template <typename IO, int DKP, int NCT, int NW>
hipError_t launch_shape(const KArgs &a, hipStream_t s) {
    if constexpr (sizeof(IO) == 4) {
        return launch_parts<IO, DKP, NCT, NW, 1>(a, s);
    } else {
        bool state = false;
        for (int i = 0; i < a.njob; ++i) state |= a.job[i].Xn != nullptr;
        return state ? launch_parts<IO, DKP, NCT, NW, 3>(a, s) : launch_parts<IO, DKP, NCT, NW, 2>(a, s);
    }
}

template <typename IO>
hipError_t launch_io(const LinArgs &in, hipStream_t s) {
    constexpr bool BF = sizeof(IO) == 2;
    const LinJob &whole = in.job[in.njob > 1 ? 1 : 0];  // the job of d_qk rows and d_v columns
    const Plan p = make_plan(in.B, in.H, in.T, whole.dk, whole.dv, BF, in.njob > 1);
    for (int i = 0; i < p.ngroup; ++i) {
        const Group &g = p.group[i];
        KArgs a{};
        a.g = in.g;
        a.lengths = in.lengths;
        a.B = in.B, a.H = in.H, a.T = in.T;
        a.nseg = g.nseg, a.seg_len = g.seg_len;
        a.njob = g.njob, a.tiles_all = g.tiles_all;
        a.ws = g.nseg > 1 ? in.ws : nullptr;
        for (int k = 0; k < g.njob; ++k) {
            a.job[k] = in.job[g.job[k]];
            a.tiles[k] = g.tiles[k];
            a.ws_job[k] = g.ws_job[k];
        }
        hipError_t e;
        // 32 columns a wavefront where its registers hold the state and two
        // wavefronts a SIMD, else 16
        if (g.dkp == 64)
            e = g.bv == 64 ? launch_shape<IO, 64, 1, 4>(a, s) : launch_shape<IO, 64, 2, 4>(a, s);
        else if (g.dkp == 128)
            e = g.bv == 64 ? launch_shape<IO, 128, 1, 4>(a, s) : launch_shape<IO, 128, 2, 4>(a, s);
        else if (g.dkp == 256)
            e = g.bv == 64 ? launch_shape<IO, 256, 1, 4>(a, s) : launch_shape<IO, 256, BF ? 2 : 1, BF ? 4 : 8>(a, s);
        else if constexpr (BF)
            e = g.bv == 64 ? launch_shape<IO, 512, 1, 4>(a, s) : launch_shape<IO, 512, 1, 8>(a, s);
        else
            e = launch_shape<IO, 512, 1, 4>(a, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

size_t linattn_workspace_floats(int B, int H, int T, int dk, int dv, int io_bf16, int backward) {
    return make_plan(B, H, T, dk, dv, io_bf16, backward).floats;
}

hipError_t launch_linattn(const LinArgs &a, int io_bf16, hipStream_t s) {
    return io_bf16 ? launch_io<bf16>(a, s) : launch_io<float>(a, s);
}

}  // namespace mlstm
