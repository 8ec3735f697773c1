// Causal depthwise convolution of width 2 to 4 (ssd.h, ssd_conv_*):
//
//   p_t = bias + sum_{j < W} w[W-1-j] x_{t-j}     y_t = p_t or silu(p_t)
//
// with x zero across a document start.  Tap j of token t is live when no
// document starts in (t - j, t].  Memory-bound: x in, y out; the W multiplies
// and the sigmoid are about 25 vector instructions an element.
#include "ssd_layer.hpp"

namespace ssd {

constexpr int kConvTokens = 16;   // tokens a thread holds at a time

// Document starts around token t0: bit i for token t0 - (W-1) + i, i < N.
template <int W, int N>
__device__ inline uint32_t conv_cuts(const int32_t *seq, int t0, int L) {
    uint32_t bits = 0;
    int p = seq[min(max(t0 - W, 0), L - 1)];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int q = seq[min(max(t0 - (W - 1) + i, 0), L - 1)];
        bits |= (q != p ? 1u : 0u) << i;
        p = q;
    }
    return bits;
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

// One thread: V channels x 16 tokens, the threads of a workgroup side by side
// along the channels (no idle lanes at the end of a token's row), consecutive
// workgroups on one XCD so that the W - 1 tokens before a chunk come from L2.
template <typename IO, int V, int W, bool PACKED>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a) {
    constexpr int T = kConvTokens;
    const int D = a.channels, L = a.seqlen, per = D / V, nch = (L + T - 1) / T;
    const int64_t first = (int64_t)xcd_contiguous(blockIdx.x, gridDim.x) * 256;
    const uint32_t r = (uint32_t)(first % per) + threadIdx.x;
    const int64_t q = first / per + r / (uint32_t)per;   // (row, chunk)
    if (q >= (int64_t)a.batch * nch) return;
    const int c = (int)(r % (uint32_t)per) * V;
    const int64_t b = q / nch;
    const int t0 = (int)(q % nch) * T;
    Pack<IO, V> xr[T + W - 1];
    const char *xb = (const char *)a.x + (b * L + t0) * a.xs + c * (int64_t)sizeof(IO);
#pragma unroll
    for (int i = 0; i < T; ++i) xr[W - 1 + i] = load_pack<IO, V>(xb + min(i, L - 1 - t0) * a.xs);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) xr[i] = conv_x<IO, V, W>(a, b, t0 - (W - 1) + i, c);
    float w[W][V], bias[V];
    conv_weights<V, W>(a, c, w, bias);
    const uint32_t cuts = PACKED ? conv_cuts<W, T + W - 1>(a.seq_idx + b * L, t0, L) : 0u;
    IO *yb = (IO *)a.y + (b * L + t0) * D + c;
#pragma unroll
    for (int i = 0; i < T; ++i) {
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float p = bias[v];
#pragma unroll
            for (int j = W - 1; j >= 0; --j) {
                const float x = (float)xr[W - 1 + i - j].v[v];
                p = fmaf(w[W - 1 - j][v], !PACKED || conv_live(cuts, W - 1 + i, j) ? x : 0.f, p);
            }
            o[v] = a.silu ? p * sigmoid_f32(p) : p;
        }
        if (t0 + i < L) store_pack<IO, V>(yb + (int64_t)i * D, o);
    }
    if (a.final_states && t0 + T >= L) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int t = L - (W - 1) + j;
            Pack<IO, V> f = conv_x<IO, V, W>(a, b, t, c);
            if (PACKED && conv_cut_after(a.seq_idx + b * L, t, L)) {
#pragma unroll
                for (int v = 0; v < V; ++v) f.v[v] = (IO)0.f;
            }
            *(Pack<IO, V> *)((IO *)a.final_states + (b * (W - 1) + j) * D + c) = f;
        }
    }
}

// Backward: one workgroup per (row, run of tokens, strip of 64 V channels), a
// wave per quarter of the run, 16 tokens at a time.  ds = dy silu'(p) is
// formed for the chunk's tokens and the W - 1 after them (p recomputed);
// dx_t = sum_j w[W-1-j] ds_{t+j} over the live taps, and the weight's sums stay in
// registers over the run, joined over the four waves in order and written as
// one part per workgroup.
template <typename IO, int V, int W, bool PACKED>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvArgs a, int run) {
    constexpr int T = kConvTokens, N = T + W - 1;
    __shared__ float red[W + 1][4][64 * V];
    const int D = a.channels, L = a.seqlen;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int nstrip = (D + 64 * V - 1) / (64 * V), nrun = (L + run - 1) / run;
    const int u = xcd_contiguous(blockIdx.x, gridDim.x);
    const int strip = u % nstrip, part = u / nstrip;
    const int64_t b = part / nrun;
    const int c0 = (strip * 64 + lane) * V;
    const bool cok = c0 < D;
    const int c = cok ? c0 : D - V;
    const int begin = (part % nrun) * run + wave * (run / 4);
    const int end = min(L, begin + run / 4);
    const int32_t *seq = PACKED ? a.seq_idx + b * L : nullptr;
    float w[W][V], bias[V], dw[W][V], db[V];
    conv_weights<V, W>(a, c, w, bias);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
    }
    for (int t0 = begin; t0 < end; t0 += T) {
        Pack<IO, V> xr[N + W - 1], dr[N];
        const char *xb = (const char *)a.x + (b * L + t0) * a.xs + c * (int64_t)sizeof(IO);
        const char *db_ = (const char *)a.dy + (b * L + t0) * a.dys + c * (int64_t)sizeof(IO);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int k = min(i, L - 1 - t0);
            xr[W - 1 + i] = load_pack<IO, V>(xb + k * a.xs);
            dr[i] = load_pack<IO, V>(db_ + k * a.dys);
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) xr[i] = conv_x<IO, V, W>(a, b, t0 - (W - 1) + i, c);
        const uint32_t cuts = PACKED ? conv_cuts<W, N + W - 1>(seq, t0, L) : 0u;
        float ds[N][V];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool in = t0 + i < L;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float xl[W], p = bias[v];
#pragma unroll
                for (int j = W - 1; j >= 0; --j) {
                    const float x = (float)xr[W - 1 + i - j].v[v];
                    xl[j] = !PACKED || conv_live(cuts, W - 1 + i, j) ? x : 0.f;
                    p = fmaf(w[W - 1 - j][v], xl[j], p);
                }
                float d = (float)dr[i].v[v];
                if (a.silu) {
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
                        const float d = !PACKED || conv_live(cuts, W - 1 + o + j, j) ? ds[o + j][v] : 0.f;
                        s = fmaf(w[W - 1 - j][v], d, s);
                    }
                    dx[v] = s;
                }
                const int t = t0 + o;
                if (t < L) {
                    if (a.dfinal && t >= L - (W - 1) && !(PACKED && conv_cut_after(seq, t, L))) {
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            dx[v] += a.dfinal[(b * (W - 1) + t - (L - (W - 1))) * D + c + v];
                    }
                    if (cok) store_pack<IO, V>((IO *)a.dx + (b * L + t) * D + c, dx);
                }
            }
        }
        if (a.dinit && t0 == 0 && cok) {
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
                            const float d = !PACKED || conv_live(cuts, W - 1 + t + j, j) ? ds[t + j >= 0 ? t + j : 0][v] : 0.f;
                            s = fmaf(w[W - 1 - j][v], d, s);
                        }
                    if (out) s += a.dfinal[(b * (W - 1) + t - (L - (W - 1))) * D + c + v];
                    a.dinit[(b * (W - 1) + q) * D + c + v] = s;
                }
            }
        }
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

int conv_strip(bool bf16_io, bool wide) { return 64 * (wide ? 4 : 1); }

template <typename IO, int V, int W>
static void conv_fwd_launch(const ConvArgs &a, unsigned grid, hipStream_t stream) {
    if (a.seq_idx)
        hipLaunchKernelGGL((conv_fwd_kernel<IO, V, W, true>), dim3(grid), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((conv_fwd_kernel<IO, V, W, false>), dim3(grid), dim3(256), 0, stream, a);
}

template <typename IO, int V, int W>
static void conv_bwd_launch(const ConvArgs &a, int run, unsigned grid, hipStream_t stream) {
    if (a.seq_idx)
        hipLaunchKernelGGL((conv_bwd_kernel<IO, V, W, true>), dim3(grid), dim3(256), 0, stream, a, run);
    else
        hipLaunchKernelGGL((conv_bwd_kernel<IO, V, W, false>), dim3(grid), dim3(256), 0, stream, a, run);
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

// Elements per access of the forward pass: 16 bytes when all is aligned for it.
int conv_fwd_vec(bool bf16_io, bool wide) { return wide ? (bf16_io ? 8 : 4) : 1; }

void launch_conv_fwd(bool bf16_io, bool wide, const ConvArgs &a, hipStream_t stream) {
    const int64_t chunks = (a.seqlen + kConvTokens - 1) / kConvTokens;
    const int64_t threads = a.batch * chunks * (a.channels / conv_fwd_vec(bf16_io, wide));
    const unsigned grid = (unsigned)((threads + 255) / 256);
    if (bf16_io) {
        if (wide) { SSD_CONV_BY_WIDTH(conv_fwd_launch, bf16, 8, grid) } else { SSD_CONV_BY_WIDTH(conv_fwd_launch, bf16, 1, grid) }
    } else {
        if (wide) { SSD_CONV_BY_WIDTH(conv_fwd_launch, float, 4, grid) } else { SSD_CONV_BY_WIDTH(conv_fwd_launch, float, 1, grid) }
    }
}

void launch_conv_bwd(bool bf16_io, bool wide, const ConvArgs &a, int run, float *dweight, float *dbias,
                     hipStream_t stream) {
    const int strip = conv_strip(bf16_io, wide);
    const int64_t parts = (int64_t)a.batch * ((a.seqlen + run - 1) / run);
    const unsigned grid = (unsigned)(parts * ((a.channels + strip - 1) / strip));
    if (bf16_io) {
        if (wide) { SSD_CONV_BY_WIDTH(conv_bwd_launch, bf16, 4, run, grid) } else { SSD_CONV_BY_WIDTH(conv_bwd_launch, bf16, 1, run, grid) }
    } else {
        if (wide) { SSD_CONV_BY_WIDTH(conv_bwd_launch, float, 4, run, grid) } else { SSD_CONV_BY_WIDTH(conv_bwd_launch, float, 1, run, grid) }
    }
    launch_part_sum(a.part, parts, a.channels, a.width, dweight, dbias, stream);
}

void launch_conv_step(bool bf16_io, bool pair, const ConvArgs &a, hipStream_t stream) {
    const unsigned grid = (unsigned)(((int64_t)a.batch * (a.channels / (pair ? 2 : 1)) + 255) / 256);
    if (bf16_io) {
        if (pair) { SSD_CONV_BY_WIDTH(conv_step_launch, bf16, 2, grid) } else { SSD_CONV_BY_WIDTH(conv_step_launch, bf16, 1, grid) }
    } else {
        if (pair) { SSD_CONV_BY_WIDTH(conv_step_launch, float, 2, grid) } else { SSD_CONV_BY_WIDTH(conv_step_launch, float, 1, grid) }
    }
}

}  // namespace ssd
