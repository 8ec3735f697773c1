// Microscaled 4-bit floating point (ssd.h, ssd_mx4_*): argument blocks and
// device helpers.  A row's columns are cut into blocks of 32, each with a
// power-of-two scale 2^(byte - 127); a value is an e2m1 code times that.
#pragma once

#include "ssd_norm.hpp"

namespace ssd {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct Mx4QuantArgs {
    const void *x;       // [rows][columns] io dtype, xs bytes between rows
    int64_t xs;
    uint8_t *q;          // [rows][128 kblocks / 2]
    uint32_t *scales;    // [kblocks][rows], four blocks of 32 columns a word
    void *y;             // the way back: [rows][columns]
    int64_t rows;
    int columns, kblocks;   // kblocks: 128-column blocks of a row
};

struct Mx4ProductArgs {
    const void *x;              // few tokens: [m][columns] io dtype, or null
    int64_t xs;
    const uint8_t *a;           // [m][64 kblocks], where x is null
    const uint32_t *as;         // [kblocks][m]
    const uint8_t *w;           // [n][64 kblocks]
    const uint32_t *ws;         // [kblocks][n]
    const float *bias;          // [n], nullable
    void *y;                    // [m][n]
    int64_t m;
    int n, columns, kblocks;
    int cus;
};

// The scale byte of a block from the largest |x| in it, as fp32 bits: the
// largest value lands in [4, 8) and saturates at 6.  255 (NaN) for a block with
// an infinity or a NaN.
__device__ inline uint32_t mx4_scale_byte(uint32_t most) {
    const uint32_t e = most >> 23;
    return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// The scale itself; 2^-127 is subnormal, and byte 255 gives a NaN.
__device__ inline float mx4_scale(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7fc00000u : byte ? byte << 23 : 0x00400000u);
}

__device__ inline uint32_t quad_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));   // lane ^ 1
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));   // lane ^ 2
}

// Sixteen bytes of a row, aligned to its columns only: accesses of global memory
// may start anywhere (16384 x 2563 bf16: 19.8 us to 4 bits, 19.4 back;
// column by column 46.4 and 73.2).
template <typename IO>
using mx4_piece = uint32_t __attribute__((ext_vector_type(4), aligned(sizeof(IO)), may_alias));

// Eight consecutive columns of a row; 0 past the last one.
template <typename IO>
__device__ inline Pack<IO, 8> mx4_load8(const char *row, int c, int columns) {
    Pack<IO, 8> r;
    if (c + 8 <= columns) {
        constexpr int N = 16 / sizeof(IO);
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) {
            const mx4_piece<IO> t = *(const mx4_piece<IO> *)(row + (c + i * N) * (int64_t)sizeof(IO));
            *(Pack<IO, N> *)&r.v[i * N] = __builtin_bit_cast(Pack<IO, N>, t);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = c + i < columns ? ((const IO *)row)[c + i] : (IO)0.f;
    }
    return r;
}

template <typename IO>
__device__ inline uint32_t mx4_most(const Pack<IO, 8> &p) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits((float)p.v[i]));
    return m;
}

// The codes of eight columns, the first in the low bits; rounded to nearest
// even and saturated by the conversion.
template <typename IO>
__device__ inline uint32_t mx4_codes(const Pack<IO, 8> &p, float scale) {
    uint32_t r = 0;
    if constexpr (sizeof(IO) == 2) {
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, bf16x2{p.v[0], p.v[1]}, scale, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, bf16x2{p.v[2], p.v[3]}, scale, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, bf16x2{p.v[4], p.v[5]}, scale, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, bf16x2{p.v[6], p.v[7]}, scale, 3);
    } else {
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, p.v[0], p.v[1], scale, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, p.v[2], p.v[3], scale, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, p.v[4], p.v[5], scale, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, p.v[6], p.v[7], scale, 3);
    }
    return r;
}

// The matrix instructions take 4-bit operands in the first half of eight
// registers.
__device__ inline i32x8 mx4_operand(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

}  // namespace ssd
