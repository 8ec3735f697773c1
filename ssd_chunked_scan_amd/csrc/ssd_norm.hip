// Root-mean-square norm (ssd.h, ssd_norm_*), with the residual's addition or
// the silu gate before it, a bf16/fp32 or an 8-bit output, and its gradient:
//
//   y = v rstd w     rstd = 1 / sqrt(mean(v^2) + eps)
//   dv = rstd (w dy - n mean(w dy n)),  n = v rstd     dw = sum_rows dy n
//
// Memory-bound: one pass over the data, a row's group held in registers
// between its sum and its output, up to K packs of V elements per thread.  A
// (row, group) belongs to a wave where one can hold it, so that no barrier
// stands between a row's loads and its stores, else to a workgroup of as many
// waves as it takes.
#include <algorithm>
#include <type_traits>

#include "ssd_layer.hpp"

namespace ssd {

enum NormInput : int { kNormPlain = 0, kNormResidual = 1, kNormGate = 2 };

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

// As many workgroups as are resident take the rows in turn, the weights in
// registers and the next row loading while this one is summed and stored:
// 73 us for 16384 rows of 2560 with the residual (4.6 TB/s; without the row
// ahead 74 us, a wave per row and five packs a lane 86 us).
template <typename IO, int V, bool WAVE, int K, int MODE, bool QUANT>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_fwd_kernel(NormArgs a) {
    constexpr int RPB = WAVE ? 4 : 1;   // rows a workgroup takes at a time
    __shared__ float lds[16];
    const int tid = WAVE ? threadIdx.x % 64 : threadIdx.x, nthr = WAVE ? 64 : blockDim.x;
    const int g = blockIdx.y;
    const int npack = a.width / V;
    const int col0 = g * a.width;
    const float inv_n = 1.f / (float)a.width;
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + (WAVE ? threadIdx.x / 64 : 0);
    Pack<IO, V> xr[K], other[K], xn[K], on[K];
    auto load = [&](int64_t r, Pack<IO, V> (&x)[K], Pack<IO, V> (&o)[K]) {
        const char *xb = (const char *)a.x + r * a.xs + col0 * (int)sizeof(IO);
        const char *ob = MODE == kNormResidual ? (const char *)a.residual + r * a.rs + col0 * (int)sizeof(IO)
                         : MODE == kNormGate   ? (const char *)a.z + r * a.zs + col0 * (int)sizeof(IO)
                                               : nullptr;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = pack_at<V>(k, tid, nthr);
            if (p < npack) {
                x[k] = load_pack<IO, V>(xb + p * (V * (int)sizeof(IO)));
                if (MODE != kNormPlain) o[k] = load_pack<IO, V>(ob + p * (V * (int)sizeof(IO)));
            }
        }
    };
    if (row < a.rows) load(row, xr, other);
    constexpr bool HOLD = K * V <= 8;   // as in the backward kernel
    float wr[HOLD ? K : 1][HOLD ? V : 1];
    if constexpr (HOLD) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = pack_at<V>(k, tid, nthr);
#pragma unroll
            for (int v = 0; v < V; ++v) wr[k][v] = p < npack && a.weight ? a.weight[col0 + p * V + v] : 1.f;
        }
    }
    auto weight = [&](int k, int p, int v) {
        if constexpr (HOLD) return wr[k][v];
        else return a.weight ? a.weight[col0 + p * V + v] : 1.f;
    };
    for (; row < a.rows; row += step) {
        if (row + step < a.rows) load(row + step, xn, on);
        float val[K][V], ss = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = pack_at<V>(k, tid, nthr);
            if (p < npack) {
                Pack<IO, V> st;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float f = (float)xr[k].v[v];
                    if (MODE == kNormResidual) {
                        // the stream is kept in the io type, and the norm is
                        // of what it holds, which is what backward reads
                        st.v[v] = (IO)(f + (float)other[k].v[v]);
                        f = (float)st.v[v];
                    } else if (MODE == kNormGate) {
                        const float z = (float)other[k].v[v];
                        f *= z * sigmoid_f32(z);
                    }
                    val[k][v] = f;
                    ss = fmaf(f, f, ss);
                }
                if (MODE == kNormResidual)
                    *(Pack<IO, V> *)((IO *)a.residual_out + row * a.columns + col0 + p * V) = st;
            }
        }
        ss = group_sum<WAVE>(ss, lds);
        const float rstd = 1.f / __builtin_sqrtf(fmaf(ss, inv_n, a.eps));
        uint32_t most[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = pack_at<V>(k, tid, nthr);
            most[k] = 0;
            if (p < npack) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    val[k][v] = val[k][v] * rstd * weight(k, p, v);
                    if (QUANT) most[k] = max(most[k], abs_bits(val[k][v]));
                }
                if (!QUANT) store_pack<IO, V>((IO *)a.y + row * a.columns + col0 + p * V, val[k]);
            }
        }
        if constexpr (QUANT) {
            uint8_t *qb = (uint8_t *)a.y + row * a.columns + col0;
            const int nb = a.quant_block ? (a.width + 127) / 128 : 1;
            float *sc = a.scales + (row * a.ngroups + g) * nb;
            if (a.quant_block == 0) {
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < K; ++k) m = max(m, most[k]);
                const float mx = __uint_as_float(max(group_max<WAVE>(m, (uint32_t *)lds), kMinMost));
                if (tid == 0) *sc = mx / 448.f;
                const float inv = 448.f / mx;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int p = pack_at<V>(k, tid, nthr);
                    if (p < npack) store_e4m3<V>(qb + p * V, val[k], inv);
                }
            } else {
                // 128 columns are 16 or 32 lanes of one k, or both packs of a
                // wave's pair of k (V = 1)
                constexpr int PER = V == 1 ? 2 : 1, LANES = V == 1 ? 64 : 128 / V;
#pragma unroll
                for (int k = 0; k < K; k += PER) {
                    const uint32_t m = PER == 2 ? max(most[k], most[k + PER - 1]) : most[k];
                    const float mx = __uint_as_float(max(lanes_max<LANES>(m), kMinMost));
                    const float inv = 448.f / mx;
                    const int p0 = pack_at<V>(k, tid, nthr);
                    if (tid % LANES == 0 && p0 < npack) sc[p0 * V / 128] = mx / 448.f;
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const int p = pack_at<V>(k + j, tid, nthr);
                        if (p < npack) store_e4m3<V>(qb + p * V, val[k + j], inv);
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xr[k] = xn[k];
            other[k] = on[k];
        }
    }
}

// Backward: a.parts workgroups per group take the rows in turn and keep their
// columns' dweight sums in registers; each leaves one row of parts.  Bound by
// registers before memory: at most 8 columns a thread (up to 8192 a group),
// so that two workgroups of ten waves fit a compute unit at 5120 columns
// (195 us for 16384 gated rows, 4.3 TB/s; 16 columns a thread in half the
// threads spills: 403 us; loading a row ahead costs one of the two: 199 us).
// Odd groups of over 8192 columns have no other way than 16 single columns a
// thread, here up to 236 bytes of scratch a thread and forward 224: 16384 fp32
// rows of 8195 with the residual take 880 us, floor 438.
template <typename IO, int V, bool WAVE, int K, bool GATE>
__global__ __launch_bounds__(WAVE ? 256 : 1024, K * V <= 8 ? 5 : 4) void norm_bwd_kernel(NormArgs a) {
    constexpr int RPB = WAVE ? 4 : 1;
    __shared__ float lds[32];
    __shared__ float red[WAVE ? 4 : 1][WAVE ? 64 * K * V : 1];
    const int tid = WAVE ? threadIdx.x % 64 : threadIdx.x, nthr = WAVE ? 64 : blockDim.x;
    const int wave = threadIdx.x / 64;
    const int g = blockIdx.y;
    const int npack = a.width / V;
    const int col0 = g * a.width;
    const float inv_n = 1.f / (float)a.width;
    // the weights in registers too, unless the columns' sums take them all
    constexpr bool HOLD = K * V <= 8;
    float wr[HOLD ? K : 1][HOLD ? V : 1], dw[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int p = pack_at<V>(k, tid, nthr);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (HOLD) wr[k][v] = p < npack && a.weight ? a.weight[col0 + p * V + v] : 1.f;
            dw[k][v] = 0.f;
        }
    }
    auto weight = [&](int k, int p, int v) {
        if constexpr (HOLD) return wr[k][v];
        else return a.weight ? a.weight[col0 + p * V + v] : 1.f;
    };
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + (WAVE ? wave : 0);
    // third: z with the gate, dresidual without
    const void *third = GATE ? a.z : a.dresidual;
    const int64_t ts = GATE ? a.zs : a.drs;
    Pack<IO, V> xr[K], dr[K], tr[K];
    auto load = [&](int64_t r) {
        const char *xb = (const char *)a.x + r * a.xs + col0 * (int)sizeof(IO);
        const char *db = (const char *)a.dy + r * a.dys + col0 * (int)sizeof(IO);
        const char *tb = (const char *)third + r * ts + col0 * (int)sizeof(IO);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = pack_at<V>(k, tid, nthr);
            if (p < npack) {
                const int off = p * (V * (int)sizeof(IO));
                xr[k] = load_pack<IO, V>(xb + off);
                dr[k] = load_pack<IO, V>(db + off);
                if (third) tr[k] = load_pack<IO, V>(tb + off);
            }
        }
    };
    if (row < a.rows) load(row);
    for (; row < a.rows; row += step) {
        float val[K][V], ss = 0.f, sd = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = pack_at<V>(k, tid, nthr);
            if (p < npack) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float f = (float)xr[k].v[v];
                    if (GATE) {
                        const float z = (float)tr[k].v[v];
                        f *= z * sigmoid_f32(z);
                    }
                    val[k][v] = f;
                    ss = fmaf(f, f, ss);
                    sd = fmaf(weight(k, p, v) * (float)dr[k].v[v], f, sd);
                }
            }
        }
        group_sum2<WAVE>(ss, sd, lds);
        const float rstd = 1.f / __builtin_sqrtf(fmaf(ss, inv_n, a.eps));
        const float mean = sd * rstd * inv_n;   // of w dy n
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = pack_at<V>(k, tid, nthr);
            if (p < npack) {
                float dx[V], dz[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float n = val[k][v] * rstd, d = (float)dr[k].v[v];
                    dw[k][v] = fmaf(d, n, dw[k][v]);
                    float dv = rstd * fmaf(-n, mean, weight(k, p, v) * d);
                    if (!GATE && a.dresidual) dv += (float)tr[k].v[v];
                    dx[v] = dv;
                    if (GATE) {
                        const float z = (float)tr[k].v[v], s = sigmoid_f32(z);
                        dx[v] = dv * (z * s);
                        dz[v] = dv * (float)xr[k].v[v] * (s * fmaf(z, 1.f - s, 1.f));
                    }
                }
                const int64_t at = row * a.columns + col0 + p * V;
                store_pack<IO, V>((IO *)a.dx + at, dx);
                if (GATE) store_pack<IO, V>((IO *)a.dz + at, dz);
            }
        }
        if (row + step < a.rows) load(row + step);
    }
    if (!a.part) return;
    float *out = a.part + (int64_t)blockIdx.x * a.columns + col0;
    if constexpr (WAVE) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) red[wave][pack_at<V>(k, tid, nthr) * V + v] = dw[k][v];
        __syncthreads();
        for (int c = threadIdx.x; c < a.width; c += 256) out[c] = ((red[0][c] + red[1][c]) + red[2][c]) + red[3][c];
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = pack_at<V>(k, tid, nthr);
            if (p < npack) {
#pragma unroll
                for (int v = 0; v < V; ++v) out[p * V + v] = dw[k][v];
            }
        }
    }
}

template <typename IO, int V, bool WAVE, int K>
static void norm_fwd_launch(const NormArgs &a, hipStream_t stream, int nthr) {
    const int64_t rows = WAVE ? (a.rows + 3) / 4 : a.rows;
    const int64_t fit = std::max<int64_t>(1, (int64_t)a.cus * (2048 / nthr) / a.ngroups);
    const dim3 grid((unsigned)std::min(rows, fit), (unsigned)a.ngroups);
    const int mode = a.residual ? kNormResidual : a.z ? kNormGate : kNormPlain;
#define SSD_NORM_FWD(M)                                                                                        \
    if (mode == M) {                                                                                           \
        if (a.scales)                                                                                          \
            hipLaunchKernelGGL((norm_fwd_kernel<IO, V, WAVE, K, M, true>), grid, dim3(nthr), 0, stream, a);    \
        else                                                                                                   \
            hipLaunchKernelGGL((norm_fwd_kernel<IO, V, WAVE, K, M, false>), grid, dim3(nthr), 0, stream, a);   \
    }
    SSD_NORM_FWD(kNormPlain)
    SSD_NORM_FWD(kNormResidual)
    SSD_NORM_FWD(kNormGate)
#undef SSD_NORM_FWD
}

template <typename IO, int V, bool WAVE, int K>
static void norm_bwd_launch(const NormArgs &a, hipStream_t stream, int nthr) {
    const dim3 grid((unsigned)a.parts, (unsigned)a.ngroups);
    if (a.z)
        hipLaunchKernelGGL((norm_bwd_kernel<IO, V, WAVE, K, true>), grid, dim3(nthr), 0, stream, a);
    else
        hipLaunchKernelGGL((norm_bwd_kernel<IO, V, WAVE, K, false>), grid, dim3(nthr), 0, stream, a);
}

// Threads of a workgroup that holds npack packs, K to a thread, in whole waves.
static int norm_threads(int npack, int K) { return ((npack + K - 1) / K + 63) / 64 * 64; }

// A wave per row and group where it can hold KW packs a lane; a workgroup of
// KB packs a thread while 1024 threads can hold the group, else of KX.
template <typename IO, int V, int KW, int KB, int KX>
static void norm_fwd_shape(const NormArgs &a, hipStream_t stream) {
    const int npack = a.width / V;
    if (npack <= 64 * KW)
        norm_fwd_launch<IO, V, true, KW>(a, stream, 256);
    else if (npack <= 1024 * KB)
        norm_fwd_launch<IO, V, false, KB>(a, stream, norm_threads(npack, KB));
    else
        norm_fwd_launch<IO, V, false, KX>(a, stream, norm_threads(npack, KX));
}

template <typename IO, int V, int KW, int KB, int KX>
static void norm_bwd_shape(const NormArgs &a, hipStream_t stream) {
    const int npack = a.width / V;
    if (npack <= 64 * KW)
        norm_bwd_launch<IO, V, true, KW>(a, stream, 256);
    else if (npack <= 1024 * KB)
        norm_bwd_launch<IO, V, false, KB>(a, stream, norm_threads(npack, KB));
    else
        norm_bwd_launch<IO, V, false, KX>(a, stream, norm_threads(npack, KX));
}

void launch_norm_fwd(bool bf16_io, bool wide, const NormArgs &a, hipStream_t stream) {
    if (bf16_io)
        wide ? norm_fwd_shape<bf16, 8, 1, 1, 2>(a, stream) : norm_fwd_shape<bf16, 1, 8, 8, 16>(a, stream);
    else
        wide ? norm_fwd_shape<float, 4, 2, 2, 4>(a, stream) : norm_fwd_shape<float, 1, 8, 8, 16>(a, stream);
}

void launch_norm_bwd(bool bf16_io, bool wide, const NormArgs &a, float *dweight, hipStream_t stream) {
    if (bf16_io)
        wide ? norm_bwd_shape<bf16, 8, 1, 1, 2>(a, stream) : norm_bwd_shape<bf16, 1, 4, 4, 16>(a, stream);
    else
        wide ? norm_bwd_shape<float, 4, 2, 2, 4>(a, stream) : norm_bwd_shape<float, 1, 4, 4, 16>(a, stream);
    if (dweight) launch_part_sum(a.part, a.parts, a.columns, 1, dweight, nullptr, stream, 1);
}

}  // namespace ssd
