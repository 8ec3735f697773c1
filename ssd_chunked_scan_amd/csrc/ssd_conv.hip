// Causal depthwise convolution of width 2 to 4 (ssd.h, ssd_conv_*):
//
//   p_t = bias + sum_{j < W} w[W-1-j] x_{t-j}     y_t = p_t or silu(p_t)
//
// with x zero across a document start.  Tap j of token t is live when no
// document starts in (t - j, t].  Memory-bound: x in, y out; the W multiplies
// and the sigmoid are about 25 vector instructions an element.
#include <type_traits>

#include "ssd_layer.hpp"

namespace ssd {

constexpr int kConvTokens = 16;   // tokens a thread holds at a time

// Document starts around token t0: bit i for token t0 - (W-1) + i, i < N <= 32,
// of the row's L; one lane looks at each.  Called by whole waves.
template <int W, int N>
__device__ inline uint32_t conv_cuts(const int32_t *seq, int t0, int L) {
    const int t = t0 - (W - 1) + (int)(threadIdx.x % 64);
    const bool cut = seq[min(max(t, 0), L - 1)] != seq[min(max(t - 1, 0), L - 1)];
    return (uint32_t)__ballot(cut) & (uint32_t)((1ull << N) - 1);
}

// Whether tap j reaches back from the token with bit `at` (compile-time j, at).
__device__ inline bool conv_live(uint32_t cuts, int at, int j) {
    return j == 0 || ((cuts >> (at - j + 1)) & ((1u << j) - 1u)) == 0u;
}

// Whether a document starts in (t, L - 1].
__device__ inline bool conv_cut_after(const int32_t *seq, int t, int L) {
    bool cut = false;
    for (int s = max(t + 1, 1); s < L; ++s) cut |= seq[s] != seq[s - 1];
    return cut;
}

// V channels of token t of row b, from the window before the row for t < 0.
template <typename IO, int V, int W>
__device__ inline Pack<IO, V> conv_x(const ConvArgs &a, int64_t b, int t, int c) {
    if (t >= 0) return load_pack<IO, V>((const char *)a.x + (b * a.seqlen + t) * a.xs + c * (int64_t)sizeof(IO));
    if (a.init) return load_pack<IO, V>((const IO *)a.init + (b * (W - 1) + t + W - 1) * a.channels + c);
    Pack<IO, V> r;
#pragma unroll
    for (int v = 0; v < V; ++v) r.v[v] = (IO)0.f;
    return r;
}

template <int V, int W>
__device__ inline void conv_weights(const ConvArgs &a, int c, float (&w)[W][V], float (&bias)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][v] = a.weight[(int64_t)(c + v) * W + j];
        bias[v] = a.bias ? a.bias[c + v] : 0.f;
    }
}

// A wave's unit of work: 64 V channels (the last strip of a token may be short)
// of T tokens of one row.
struct ConvUnit {
    int strip, chunk;
    int64_t b;
};

__device__ inline ConvUnit conv_unit(uint32_t u, int nstrip, int nchunk) {
    ConvUnit r;
    r.strip = __builtin_amdgcn_readfirstlane(u % nstrip);
    const uint32_t q = u / nstrip;
    r.chunk = __builtin_amdgcn_readfirstlane(q % nchunk);
    r.b = __builtin_amdgcn_readfirstlane(q / nchunk);
    return r;
}

// Consecutive workgroups on one XCD, so that the W - 1 tokens before a chunk
// come from L2; the rows' offsets in scalar registers.  74 us for 8 x 2048 x
// 5376 in bf16 (4.8 TB/s).  Two channels a lane were chosen when that took 79
// us: four took 86 and eight 98, whose registers leave half and a third of the
// waves, and 24 tokens instead of 16 took 78.
template <typename IO, int V, int W, bool PACKED, bool SILU>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a) {
    constexpr int T = kConvTokens;
    typedef Raw<IO, V> RW;
    typedef typename RW::type R;
    const int D = a.channels, L = a.seqlen, nchunk = (L + T - 1) / T, nstrip = (D + 64 * V - 1) / (64 * V);
    const uint32_t unit = (uint32_t)xcd_contiguous(blockIdx.x, gridDim.x) * 4 + threadIdx.x / 64;
    if (unit >= (uint32_t)((int64_t)a.batch * nchunk * nstrip)) return;
    const ConvUnit u = conv_unit(unit, nstrip, nchunk);
    const int c0 = (u.strip * 64 + threadIdx.x % 64) * V;
    const int c = min(c0, D - V);   // lanes past the last channel repeat it, and store nothing
    const int t0 = u.chunk * T;
    const int32_t *seq = PACKED ? a.seq_idx + u.b * L : nullptr;
    const uint32_t cb = (uint32_t)c * (uint32_t)sizeof(IO);
    const uint32_t cuts = PACKED ? conv_cuts<W, T + W - 1>(seq, t0, L) : 0u;
    const __amdgpu_buffer_rsrc_t yb = buffer_of((IO *)a.y + (u.b * L + t0) * D);
    float w[W][V], bias[V];
    conv_weights<V, W>(a, c, w, bias);
    // INNER: a whole chunk inside a row, no document start in it, whole strip
    auto chunk = [&](auto inner) {
        constexpr bool INNER = decltype(inner)::value;
        R xr[T + W - 1];
        if (INNER) {
            const __amdgpu_buffer_rsrc_t xb = buffer_of((const char *)a.x + (u.b * L + t0 - (W - 1)) * a.xs);
#pragma unroll
            for (int i = 0; i < T + W - 1; ++i) xr[i] = buffer_load<R>(xb, cb, (uint32_t)(i * a.xs));
        } else {
            const __amdgpu_buffer_rsrc_t xb = buffer_of((const char *)a.x + (u.b * L + t0) * a.xs);
#pragma unroll
            for (int i = 0; i < T; ++i) xr[W - 1 + i] = buffer_load<R>(xb, cb, (uint32_t)(min(i, L - 1 - t0) * a.xs));
#pragma unroll
            for (int i = 0; i < W - 1; ++i)
                xr[i] = __builtin_bit_cast(R, conv_x<IO, V, W>(a, u.b, t0 - (W - 1) + i, c));
        }
#pragma unroll
        for (int i = 0; i < T; ++i) {
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float p = bias[v];
#pragma unroll
                for (int j = W - 1; j >= 0; --j) {
                    const float x = RW::at(xr[W - 1 + i - j], v);
                    p = fmaf(w[W - 1 - j][v], INNER || !PACKED || conv_live(cuts, W - 1 + i, j) ? x : 0.f, p);
                }
                o[v] = SILU ? p * sigmoid_f32(p) : p;
            }
            if (INNER || (t0 + i < L && c0 < D))
                buffer_store<IO, V>(yb, cb, (uint32_t)i * (uint32_t)D * (uint32_t)sizeof(IO), o);
        }
    };
    if (t0 > 0 && t0 + T <= L && !cuts && (u.strip + 1) * 64 * V <= D)
        chunk(std::true_type{});
    else
        chunk(std::false_type{});
    if (a.final_states && t0 + T >= L && c0 < D) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int t = L - (W - 1) + j;
            Pack<IO, V> f = conv_x<IO, V, W>(a, u.b, t, c);
            if (PACKED && conv_cut_after(seq, t, L)) {
#pragma unroll
                for (int v = 0; v < V; ++v) f.v[v] = (IO)0.f;
            }
            *(Pack<IO, V> *)((IO *)a.final_states + (u.b * (W - 1) + j) * D + c) = f;
        }
    }
}

// Backward: one workgroup per (row, run of tokens, strip of 64 V channels), a
// wave per quarter of the run, 16 tokens at a time.  ds = dy silu'(p) is
// formed for the chunk's tokens and the W - 1 after them (p recomputed);
// dx_t = sum_j w[W-1-j] ds_{t+j} over the live taps, and the weight's sums stay in
// registers over the run, joined over the four waves in order and written as
// one part per workgroup.  The chunks inside a row without a document start
// are taken first, in a loop without a mask or a bound; the others after
// them, in a loop of their own, so that neither's registers add to the
// other's.
template <typename IO, int V, int W, bool PACKED, bool SILU>
__global__ __launch_bounds__(256, sizeof(IO) == 2 ? 4 : 1) void conv_bwd_kernel(ConvArgs a, int run) {
    constexpr int T = kConvTokens, N = T + W - 1;
    typedef Raw<IO, V> RW;
    typedef typename RW::type R;
    __shared__ float red[W + 1][4][64 * V];
    const int D = a.channels, L = a.seqlen;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int nstrip = (D + 64 * V - 1) / (64 * V), nrun = (L + run - 1) / run;
    const uint32_t u = xcd_contiguous(blockIdx.x, gridDim.x);
    const int strip = __builtin_amdgcn_readfirstlane(u % nstrip), part = __builtin_amdgcn_readfirstlane(u / nstrip);
    const int64_t b = part / nrun;
    const int c0 = (strip * 64 + lane) * V;
    const bool cok = c0 < D;
    const int c = cok ? c0 : D - V;
    const uint32_t cb = (uint32_t)c * (uint32_t)sizeof(IO);
    const int begin = __builtin_amdgcn_readfirstlane((part % nrun) * run + wave * (run / 4));
    const int end = min(L, begin + run / 4);
    const int32_t *seq = PACKED ? a.seq_idx + b * L : nullptr;
    const bool whole = (strip + 1) * 64 * V <= D;
    float w[W][V], bias[V], dw[W][V], db[V];
    conv_weights<V, W>(a, c, w, bias);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
    }
    auto cuts_at = [&](int t0) { return PACKED ? conv_cuts<W, N + W - 1>(seq, t0, L) : 0u; };
    auto is_inner = [&](int t0, uint32_t cuts) { return t0 > 0 && t0 + N <= L && !cuts && whole; };
    auto chunk = [&](int t0, uint32_t cuts, auto inner) {
        constexpr bool INNER = decltype(inner)::value;
        constexpr bool MASKED = PACKED && !INNER;
        R xr[N + W - 1], dr[N];
        const __amdgpu_buffer_rsrc_t gb = buffer_of((const char *)a.dy + (b * L + t0) * a.dys);
        if (INNER) {
            const __amdgpu_buffer_rsrc_t xb = buffer_of((const char *)a.x + (b * L + t0 - (W - 1)) * a.xs);
#pragma unroll
            for (int i = 0; i < N + W - 1; ++i) xr[i] = buffer_load<R>(xb, cb, (uint32_t)(i * a.xs));
#pragma unroll
            for (int i = 0; i < N; ++i) dr[i] = buffer_load<R>(gb, cb, (uint32_t)(i * a.dys));
        } else {
            const __amdgpu_buffer_rsrc_t xb = buffer_of((const char *)a.x + (b * L + t0) * a.xs);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int k = min(i, L - 1 - t0);
                xr[W - 1 + i] = buffer_load<R>(xb, cb, (uint32_t)(k * a.xs));
                dr[i] = buffer_load<R>(gb, cb, (uint32_t)(k * a.dys));
            }
#pragma unroll
            for (int i = 0; i < W - 1; ++i) xr[i] = __builtin_bit_cast(R, conv_x<IO, V, W>(a, b, t0 - (W - 1) + i, c));
        }
        const __amdgpu_buffer_rsrc_t ob = buffer_of((IO *)a.dx + (b * L + t0) * D);
        float ds[N][V];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool in = INNER || t0 + i < L;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float xl[W], p = bias[v];
#pragma unroll
                for (int j = W - 1; j >= 0; --j) {
                    const float x = RW::at(xr[W - 1 + i - j], v);
                    xl[j] = !MASKED || conv_live(cuts, W - 1 + i, j) ? x : 0.f;
                    p = fmaf(w[W - 1 - j][v], xl[j], p);
                }
                float d = RW::at(dr[i], v);
                if (SILU) {
                    const float s = sigmoid_f32(p);
                    d *= s * fmaf(p, 1.f - s, 1.f);
                }
                d = in ? d : 0.f;
                ds[i][v] = d;
                if (i < T && in) {
                    db[v] += d;
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[W - 1 - j][v] = fmaf(d, xl[j], dw[W - 1 - j][v]);
                }
            }
            const int o = i - (W - 1);   // this token's gradient is complete
            if (o >= 0) {
                float dx[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float s = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        const float d = !MASKED || conv_live(cuts, W - 1 + o + j, j) ? ds[o + j][v] : 0.f;
                        s = fmaf(w[W - 1 - j][v], d, s);
                    }
                    dx[v] = s;
                }
                const int t = t0 + o;
                // (an inner chunk ends before the tokens of the final window)
                if (!INNER && a.dfinal && t < L && t >= L - (W - 1) && !(PACKED && conv_cut_after(seq, t, L))) {
#pragma unroll
                    for (int v = 0; v < V; ++v) dx[v] += a.dfinal[(b * (W - 1) + t - (L - (W - 1))) * D + c + v];
                }
                if (INNER || (t < L && cok))
                    buffer_store<IO, V>(ob, cb, (uint32_t)o * (uint32_t)D * (uint32_t)sizeof(IO), dx);
            }
        }
        if (!INNER && a.dinit && t0 == 0 && cok) {
            // the window before the row: tokens -(W-1) .. -1
#pragma unroll
            for (int q = 0; q < W - 1; ++q) {
                const int t = q - (W - 1);
                const bool out = a.dfinal && t >= L - (W - 1) && !(PACKED && conv_cut_after(seq, t, L));
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float s = 0.f;
#pragma unroll
                    for (int j = 1; j < W; ++j)
                        if (t + j >= 0) {
                            const float d = !MASKED || conv_live(cuts, W - 1 + t + j, j) ? ds[t + j >= 0 ? t + j : 0][v] : 0.f;
                            s = fmaf(w[W - 1 - j][v], d, s);
                        }
                    if (out) s += a.dfinal[(b * (W - 1) + t - (L - (W - 1))) * D + c + v];
                    a.dinit[(b * (W - 1) + q) * D + c + v] = s;
                }
            }
        }
    };
    for (int t0 = begin; t0 < end; t0 += T) {
        const uint32_t cuts = cuts_at(t0);
        if (is_inner(t0, cuts)) chunk(t0, cuts, std::true_type{});
    }
    for (int t0 = begin; t0 < end; t0 += T) {
        const uint32_t cuts = cuts_at(t0);
        if (!is_inner(t0, cuts)) chunk(t0, cuts, std::false_type{});
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) red[j][wave][lane * V + v] = dw[j][v];
        red[W][wave][lane * V + v] = db[v];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 64 * V; i += 256) {
        const int j = i / (64 * V), k = i % (64 * V);
        const int ch = strip * 64 * V + k;
        if (ch < D)
            a.part[((int64_t)part * (W + 1) + j) * D + ch] = ((red[j][0][k] + red[j][1][k]) + red[j][2][k]) + red[j][3][k];
    }
}

// One token: the window's W - 1 inputs and the new one; the window is shifted.
template <typename IO, int V, int W>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a) {
    const int D = a.channels, per = D / V;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)a.batch * per) return;
    const int64_t b = i / per;
    const int c = (int)(i % per) * V;
    float w[W][V], bias[V], o[V];
    Pack<IO, V> x[W];
    IO *st = (IO *)a.state + b * (W - 1) * D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) x[j] = load_pack<IO, V>(st + (int64_t)j * D);
    x[W - 1] = load_pack<IO, V>((const char *)a.x + b * a.xs + c * (int64_t)sizeof(IO));
    conv_weights<V, W>(a, c, w, bias);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float p = bias[v];
#pragma unroll
        for (int j = 0; j < W; ++j) p = fmaf(w[j][v], (float)x[j].v[v], p);
        o[v] = a.silu ? p * sigmoid_f32(p) : p;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) *(Pack<IO, V> *)(st + (int64_t)j * D) = x[j + 1];
    store_pack<IO, V>((IO *)a.y + b * D + c, o);
}

// Channels of a wave's strip.
int conv_strip(bool pair) { return 64 * (pair ? 2 : 1); }

template <typename IO, int V, int W, bool PACKED>
static void conv_fwd_launch_docs(const ConvArgs &a, unsigned grid, hipStream_t stream) {
    if (a.silu)
        hipLaunchKernelGGL((conv_fwd_kernel<IO, V, W, PACKED, true>), dim3(grid), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((conv_fwd_kernel<IO, V, W, PACKED, false>), dim3(grid), dim3(256), 0, stream, a);
}

template <typename IO, int V, int W>
static void conv_fwd_launch(const ConvArgs &a, unsigned grid, hipStream_t stream) {
    a.seq_idx ? conv_fwd_launch_docs<IO, V, W, true>(a, grid, stream) : conv_fwd_launch_docs<IO, V, W, false>(a, grid, stream);
}

template <typename IO, int V, int W, bool PACKED>
static void conv_bwd_launch_docs(const ConvArgs &a, int run, unsigned grid, hipStream_t stream) {
    if (a.silu)
        hipLaunchKernelGGL((conv_bwd_kernel<IO, V, W, PACKED, true>), dim3(grid), dim3(256), 0, stream, a, run);
    else
        hipLaunchKernelGGL((conv_bwd_kernel<IO, V, W, PACKED, false>), dim3(grid), dim3(256), 0, stream, a, run);
}

template <typename IO, int V, int W>
static void conv_bwd_launch(const ConvArgs &a, int run, unsigned grid, hipStream_t stream) {
    a.seq_idx ? conv_bwd_launch_docs<IO, V, W, true>(a, run, grid, stream)
              : conv_bwd_launch_docs<IO, V, W, false>(a, run, grid, stream);
}

template <typename IO, int V, int W>
static void conv_step_launch(const ConvArgs &a, unsigned grid, hipStream_t stream) {
    hipLaunchKernelGGL((conv_step_kernel<IO, V, W>), dim3(grid), dim3(256), 0, stream, a);
}

#define SSD_CONV_BY_WIDTH(launch, IO, V, ...)                \
    switch (a.width) {                                       \
    case 2: launch<IO, V, 2>(a, __VA_ARGS__, stream); break; \
    case 3: launch<IO, V, 3>(a, __VA_ARGS__, stream); break; \
    default: launch<IO, V, 4>(a, __VA_ARGS__, stream);       \
    }

#define SSD_CONV_BY_TYPE(launch, ...)                                                                              \
    if (bf16_io) {                                                                                                 \
        if (pair) { SSD_CONV_BY_WIDTH(launch, bf16, 2, __VA_ARGS__) } else { SSD_CONV_BY_WIDTH(launch, bf16, 1, __VA_ARGS__) }   \
    } else {                                                                                                       \
        if (pair) { SSD_CONV_BY_WIDTH(launch, float, 2, __VA_ARGS__) } else { SSD_CONV_BY_WIDTH(launch, float, 1, __VA_ARGS__) } \
    }

void launch_conv_fwd(bool bf16_io, bool pair, const ConvArgs &a, hipStream_t stream) {
    const int strip = conv_strip(pair);
    const int64_t units = a.batch * (int64_t)((a.seqlen + kConvTokens - 1) / kConvTokens) * ((a.channels + strip - 1) / strip);
    const unsigned grid = (unsigned)((units + 3) / 4);
    SSD_CONV_BY_TYPE(conv_fwd_launch, grid)
}

void launch_conv_bwd(bool bf16_io, bool pair, const ConvArgs &a, int run, float *dweight, float *dbias,
                     hipStream_t stream) {
    const int strip = conv_strip(pair);
    const int64_t parts = (int64_t)a.batch * ((a.seqlen + run - 1) / run);
    const unsigned grid = (unsigned)(parts * ((a.channels + strip - 1) / strip));
    SSD_CONV_BY_TYPE(conv_bwd_launch, run, grid)
    launch_part_sum(a.part, parts, a.channels, a.width, dweight, dbias, stream);
}

void launch_conv_step(bool bf16_io, bool pair, const ConvArgs &a, hipStream_t stream) {
    const unsigned grid = (unsigned)(((int64_t)a.batch * (a.channels / (pair ? 2 : 1)) + 255) / 256);
    SSD_CONV_BY_TYPE(conv_step_launch, grid)
}

}  // namespace ssd
