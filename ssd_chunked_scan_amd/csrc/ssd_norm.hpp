// What the kernels that norm rows share: sums and maxima over a row's threads,
// the packs a thread holds and the 8-bit store.
#pragma once

#include <type_traits>

#include "ssd_layer.hpp"

namespace ssd {

// Sum over the 64 lanes, in every lane, by row shifts and broadcasts.
__device__ inline float wave_sum(float v) {
    auto dpp = [](float x, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    v += dpp(v, std::integral_constant<int, 0xB1>{});    // lane ^ 1
    v += dpp(v, std::integral_constant<int, 0x4E>{});    // lane ^ 2
    v += dpp(v, std::integral_constant<int, 0x141>{});   // the other half of 8
    v += dpp(v, std::integral_constant<int, 0x140>{});   // the other half of the row of 16
    const float a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
    const float b = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16));
    const float c = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32));
    const float d = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
    return (a + b) + (c + d);
}

template <bool WAVE>
__device__ inline float group_sum(float v, float *lds) {
    v = wave_sum(v);
    if constexpr (!WAVE) {
        if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
        __syncthreads();
        v = 0.f;
        for (int i = 0; i < (int)blockDim.x / 64; ++i) v += lds[i];
        __syncthreads();
    }
    return v;
}

// Both sums at once: one pair of barriers.
template <bool WAVE>
__device__ inline void group_sum2(float &u, float &v, float *lds) {
    u = wave_sum(u);
    v = wave_sum(v);
    if constexpr (!WAVE) {
        if (threadIdx.x % 64 == 0) {
            lds[threadIdx.x / 64] = u;
            lds[16 + threadIdx.x / 64] = v;
        }
        __syncthreads();
        u = v = 0.f;
        for (int i = 0; i < (int)blockDim.x / 64; ++i) {
            u += lds[i];
            v += lds[16 + i];
        }
        __syncthreads();
    }
}

// |v| as an integer that orders like it, with NaN above infinity: a maximum
// over these carries a NaN along.
__device__ inline uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

constexpr uint32_t kMinMost = 0x2b8cbcccu;   // 1e-12f

template <int LANES>
__device__ inline uint32_t lanes_max(uint32_t v) {
    auto dpp = [](uint32_t x, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xf, 0xf, true);
    };
    v = max(v, dpp(v, std::integral_constant<int, 0xB1>{}));
    v = max(v, dpp(v, std::integral_constant<int, 0x4E>{}));
    v = max(v, dpp(v, std::integral_constant<int, 0x141>{}));
    v = max(v, dpp(v, std::integral_constant<int, 0x140>{}));
    if constexpr (LANES >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    if constexpr (LANES >= 64) v = max(v, (uint32_t)__shfl_xor((int)v, 32, 64));
    return v;
}

// The pack a thread holds as its k-th: along the row, nthr at a time; single
// elements in runs of 128 per wave (two k), so that a block of 128 columns
// stays within a wave.
template <int V>
__device__ inline int pack_at(int k, int tid, int nthr) {
    if constexpr (V == 1)
        return ((k / 2) * (nthr / 64) + tid / 64) * 128 + (k % 2) * 64 + tid % 64;
    else
        return k * nthr + tid;
}

template <bool WAVE>
__device__ inline uint32_t group_max(uint32_t v, uint32_t *lds) {
    v = lanes_max<64>(v);
    if constexpr (!WAVE) {
        if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
        __syncthreads();
        for (int i = 0; i < (int)blockDim.x / 64; ++i) v = max(v, lds[i]);
        __syncthreads();
    }
    return v;
}

// V fp32 values as e4m3 bytes, each times inv, rounded to nearest even.  The
// clamp only catches the last rounding of y * (448 / max |y|) and leaves a NaN
// as it is.
template <int V>
__device__ inline void store_e4m3(uint8_t *p, const float (&y)[V], float inv) {
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s[v] = y[v] * inv;
        s[v] = s[v] > 448.f ? 448.f : s[v];
        s[v] = s[v] < -448.f ? -448.f : s[v];
    }
    if constexpr (V == 1) {
        *p = (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[0], 0, false) & 0xff);
    } else {
        uint32_t w[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            int r = __builtin_amdgcn_cvt_pk_fp8_f32(s[4 * i], s[4 * i + 1], 0, false);
            r = __builtin_amdgcn_cvt_pk_fp8_f32(s[4 * i + 2], s[4 * i + 3], r, true);
            w[i] = (uint32_t)r;
        }
        Pack<uint32_t, V / 4> o;
#pragma unroll
        for (int i = 0; i < V / 4; ++i) o.v[i] = w[i];
        *(Pack<uint32_t, V / 4> *)p = o;
    }
}

// Threads of a workgroup that holds npack packs, K to a thread, in whole waves.
inline int norm_threads(int npack, int K) { return ((npack + K - 1) / K + 63) / 64 * 64; }

}  // namespace ssd
