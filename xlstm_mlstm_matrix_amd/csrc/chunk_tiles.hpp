// chunk_tiles.hpp -- tiles of 32-token chunks: LDS swizzles and their operand reads,
// splits of float32 into bfloat16 parts, the matrix instructions.  Shared by the
// kernels that walk sequences in chunks (linattn.hip, deltarule.hip).
//
// The MFMA's inner index may be permuted if both operands agree: slot e of
// lane group g4 stands for d_qk index 32 kk + 8 g4 + e, and for token
// 16 (e / 4) + 4 g4 + e % 4.
#pragma once

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

}  // namespace

}  // namespace mlstm
