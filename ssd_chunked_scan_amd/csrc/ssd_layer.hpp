// Shared definitions of the layer operators around the scan (gated linear
// recurrence, causal depthwise convolution, root-mean-square norm): argument
// blocks, vector loads and stores of 1 to 8 elements, and the gate's maps.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd_common.hpp"

namespace ssd {

// ---------------------------------------------------------------- arguments
// Strides are in bytes between tokens (rows).

struct GlrArgs {
    const void *x, *g, *z, *dy;     // io dtype; z nullable; dy backward only
    int64_t xs, gs, zs, dys;
    const float *A, *bias;          // [channels]; bias nullable
    const int32_t *seq_idx;         // nullable
    const float *init;              // [batch][channels], nullable
    void *y;                        // forward
    float *final_states;            // nullable
    const float *dfinal;            // backward, nullable
    void *dx, *dg, *dz;             // backward; dz with z
    float *dA, *dbias, *dinit;      // backward; dbias, dinit nullable
    // Per (row, block, channel): the block's decay product, its end state from
    // a zero start, and (backward) the adjoint it passes on from a zero one.
    // The block scan replaces the latter two by the entering values.  Unused
    // for a row of one block.
    float *ws_p, *ws_h, *ws_e;      // [batch][nblk][channels]
    float *part;                    // [batch * nblk][2][channels]: dA, dbias of each block
    int batch, seqlen, channels;
    int nblk, blk_len;              // blocks (splits) per row and their tokens
    int normalize;
    int cus;                        // forward: compute units
    int whole;                      // forward: units that run as one workgroup, the others as two
    int once;                       // backward: whether the gradients are stored as kOnce
};

struct GlrStepArgs {
    const void *x, *g, *z;          // [batch] tokens; z nullable
    int64_t xs, gs, zs;
    const float *A, *bias;
    float *state;
    void *y;
    int batch, channels, normalize;
};

struct ConvArgs {
    const void *x, *dy;
    int64_t xs, dys;
    const float *weight, *bias;     // bias nullable
    const int32_t *seq_idx;         // nullable
    const void *init;               // nullable
    void *y, *final_states;         // forward; final_states nullable
    const float *dfinal;            // nullable
    void *dx;
    float *dinit;                   // nullable
    float *part;                    // [parts][channels * (width + 1)]: dweight, dbias of each part
    void *state;                    // step
    int batch, seqlen, channels, width, silu;
};

struct NormArgs {
    const void *x, *z, *residual, *dy, *dresidual;
    int64_t xs, zs, rs, dys, drs;
    const float *weight;            // nullable
    void *y, *residual_out;         // y: io dtype, or e4m3 bytes when scales is set
    float *scales;
    void *dx, *dz;
    float *part;                    // [parts][columns], nullable
    float eps;
    int quant_block;                // 0: the whole group
    int64_t rows;
    int columns, ngroups, width;    // width = columns / ngroups
    int cus;                        // compute units
    int parts;                      // backward: workgroups along the rows
};

// ------------------------------------------------------------ vector access

template <typename IO, int V>
struct alignas(sizeof(IO) * V) Pack {
    IO v[V];
};

template <typename IO, int V>
__device__ inline Pack<IO, V> load_pack(const void *p) {
    return *(const Pack<IO, V> *)p;
}

template <typename IO, int V>
__device__ inline void store_pack(void *p, const float (&f)[V]) {
    Pack<IO, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.v[i] = (IO)f[i];
    *(Pack<IO, V> *)p = o;
}

// The same kept as one machine word or vector of words, so that what waits in
// registers takes V * sizeof(IO) bytes; at(r, v) is element v.
template <int BYTES>
struct Words;
template <>
struct Words<2> { typedef uint16_t type; };
template <>
struct Words<4> { typedef uint32_t type; };
template <>
struct Words<8> { typedef uint32_t type __attribute__((ext_vector_type(2))); };
template <>
struct Words<16> { typedef uint32_t type __attribute__((ext_vector_type(4))); };

template <typename IO, int V>
struct Raw {
    typedef typename Words<sizeof(IO) * V>::type type;
    static __device__ inline uint32_t word(type r, int i) {
        if constexpr (sizeof(IO) * V <= 4) return r;
        else return r[i];
    }
    static __device__ inline float at(type r, int v) {
        if constexpr (sizeof(IO) == 4) return __uint_as_float(word(r, v));
        else if constexpr (V == 1) return __uint_as_float((uint32_t)r << 16);
        else return __uint_as_float(v % 2 ? word(r, v / 2) & 0xffff0000u : word(r, v / 2) << 16);
    }
};

// Loads and stores through a buffer descriptor: the run's base in scalar
// registers, a 32-bit offset per lane and a scalar one per token, so that no
// lane forms a 64-bit address.  Every offset is kept inside the tensor by the
// caller; the descriptor's own bound is not used.
__device__ inline __amdgpu_buffer_rsrc_t buffer_of(const void *base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, 0xffffffff, 0x00027000);
}

template <typename R>
__device__ inline R buffer_load(__amdgpu_buffer_rsrc_t b, uint32_t lane, uint32_t token) {
    if constexpr (sizeof(R) == 2) return __builtin_amdgcn_raw_buffer_load_b16(b, lane, token, 0);
    else if constexpr (sizeof(R) == 4) return __builtin_amdgcn_raw_buffer_load_b32(b, lane, token, 0);
    else if constexpr (sizeof(R) == 8) return __builtin_amdgcn_raw_buffer_load_b64(b, lane, token, 0);
    else return __builtin_amdgcn_raw_buffer_load_b128(b, lane, token, 0);
}

// A store's cache policy: kOnce marks data that should not push other lines out
// of the caches (non-temporal).
enum : int { kKeep = 0, kOnce = 2 };

template <typename IO, int V, int AUX = kKeep>
__device__ inline void buffer_store(__amdgpu_buffer_rsrc_t b, uint32_t lane, uint32_t token, const float (&f)[V]) {
    typedef typename Words<sizeof(IO) * V>::type R;
    typedef float fv __attribute__((ext_vector_type(V)));
    typedef IO iv __attribute__((ext_vector_type(V)));
    const R r = __builtin_bit_cast(R, __builtin_convertvector(__builtin_bit_cast(fv, f), iv));
    if constexpr (sizeof(R) == 2) __builtin_amdgcn_raw_buffer_store_b16(r, b, lane, token, AUX);
    else if constexpr (sizeof(R) == 4) __builtin_amdgcn_raw_buffer_store_b32(r, b, lane, token, AUX);
    else if constexpr (sizeof(R) == 8) __builtin_amdgcn_raw_buffer_store_b64(r, b, lane, token, AUX);
    else __builtin_amdgcn_raw_buffer_store_b128(r, b, lane, token, AUX);
}

// ------------------------------------------------------------------- maps

constexpr float kLn2 = 0.6931471805599453f;

// The gate's softplus in base-2 units: softplus2(v) = log2(1 + exp(v)) =
// max(w, 0) + log2(1 + e) with w = v log2(e), e = 2^-|w| in [0, 1].  1 + e is
// rounded to o and loses c = e - (o - 1), so log2(1 + e) = log2(o) + c log2(e)
// / o up to c^2; 1 / o is only needed to a few bits there, and 1 - e / 2
// equals it at both ends.  Keeps the relative accuracy for very negative v,
// where the decay's distance from 1 is all that matters.  e and o are handed
// out for the derivative 1 / (1 + exp(-v)) = (v >= 0 ? 1 : e) / o.
__device__ inline float softplus2(float v, float &e, float &o) {
    const float w = kLog2e * v;
    e = __builtin_amdgcn_exp2f(-fabsf(w));
    o = 1.f + e;
    const float c = e - (o - 1.f);
    return fmaxf(w, 0.f) + fmaf(c, fmaf(-0.5f * kLog2e, e, kLog2e), __builtin_amdgcn_logf(o));
}

// 1 - a^2 for a = 2^l, l <= 0: by the series of 1 - exp(-q), q = -2 ln(2) l,
// where a^2 is near 1 (six terms, below 5e-8 relative at q = 1/4), else
// directly (no more than 2.3 roundings of a^2 lost there).
__device__ inline float one_minus_square(float a, float l) {
    constexpr double s = -2.0 * 0.69314718055994530942;
    float p = fmaf(l, (float)(-s * s * s * s * s * s / 720.), (float)(s * s * s * s * s / 120.));
    p = fmaf(l, p, (float)(-s * s * s * s / 24.));
    p = fmaf(l, p, (float)(s * s * s / 6.));
    p = fmaf(l, p, (float)(-s * s / 2.));
    p = fmaf(l, p, (float)s);
    return l > (float)(0.25 / s) ? l * p : fmaf(-a, a, 1.f);
}

// Decay and input factor of one element.
template <bool NORM>
__device__ inline void gate_map(float v, float A, float &a, float &k) {
    float e, o;
    const float l = A * softplus2(v, e, o);
    a = __builtin_amdgcn_exp2f(l);
    k = NORM ? __builtin_amdgcn_sqrtf(one_minus_square(a, l)) : 1.f;
}

__device__ inline float sigmoid_f32(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

// Sums `parts` rows of `planes` (0: taps + 1) planes of n columns in a fixed
// order: plane j < taps of column c into out0[c * taps + j], plane taps into
// out1[c] (nullable).
void launch_part_sum(const float *in, int64_t parts, int n, int taps, float *out0, float *out1, hipStream_t stream,
                     int planes = 0);

}  // namespace ssd
