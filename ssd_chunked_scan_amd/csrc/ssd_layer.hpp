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
    // The block scan replaces the latter two by the entering values.
    float *ws_p, *ws_h, *ws_e;      // [batch][nblk][channels]
    float *part;                    // [batch * nblk][2][channels]: dA, dbias of each block
    int batch, seqlen, channels;
    int nblk, blk_len;              // blocks (splits) per row and their tokens
    int normalize;
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

// ------------------------------------------------------------------- maps

constexpr float kLn2 = 0.6931471805599453f;

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|) in [0, 1].  1 + e is
// rounded to w and loses c = e - (w - 1), so log(1 + e) = log(w) + c / w up
// to c^2; 1 / w is only needed to a few bits there, and 1 - e / 2 equals it
// at both ends.  Keeps the relative accuracy for very negative v, where the
// decay's distance from 1 is all that matters.  e and w are handed out for
// the derivative 1 / (1 + exp(-v)) = (v >= 0 ? 1 : e) / w.
__device__ inline float softplus_precise(float v, float &e, float &w) {
    e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(v));
    w = 1.f + e;
    const float c = e - (w - 1.f);
    return fmaxf(v, 0.f) + fmaf(__builtin_amdgcn_logf(w), kLn2, c * fmaf(-0.5f, e, 1.f));
}

// 1 - a^2 for a = exp(la), la <= 0: by the series of 1 - exp(-q), q = -2 la,
// where a^2 is near 1 (six terms, below 5e-8 relative at q = 1/4), else
// directly (no more than 2.3 roundings of a^2 lost there).
__device__ inline float one_minus_square(float a, float la) {
    const float q = -2.f * la;
    float p = fmaf(q, -1.f / 720.f, 1.f / 120.f);
    p = fmaf(q, p, -1.f / 24.f);
    p = fmaf(q, p, 1.f / 6.f);
    p = fmaf(q, p, -0.5f);
    p = fmaf(q, p, 1.f);
    return q < 0.25f ? q * p : fmaf(-a, a, 1.f);
}

// Decay and input factor of one element.
template <bool NORM>
__device__ inline void gate_map(float v, float A, float &a, float &k) {
    float e, w;
    const float la = A * softplus_precise(v, e, w);
    a = __builtin_amdgcn_exp2f(kLog2e * la);
    k = NORM ? __builtin_amdgcn_sqrtf(one_minus_square(a, la)) : 1.f;
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
