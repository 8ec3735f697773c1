// The gated linear recurrence's kernels for fp32 activations, and those that
// do not depend on the activations' type: the scan over the blocks' maps and
// the sum over per-block parts.
#include "ssd_glr.hpp"

namespace ssd {

SSD_GLR_INSTANTIATE(float)

// Joins the blocks of a row, 64 channels per workgroup: 16 threads per channel
// take a run of blocks each, so that a long row (65536 tokens: 1024 blocks of
// the backward pass) is 64 dependent steps twice and not 1024.  ws_h becomes the state entering each
// block, ws_e the adjoint entering it from behind; the adjoint leaving the
// first block is the gradient of init.
template <bool PACKED>
__global__ __launch_bounds__(1024) void glr_block_scan_kernel(GlrArgs a) {
    constexpr int B = 8;   // blocks loaded at a time, before their chain
    __shared__ float sp[16][64], sh[16][64], se[16][64];
    const int lane = threadIdx.x % 64, run = threadIdx.x / 64;
    const int D = a.channels;
    const int nct = (D + 63) / 64;
    const int b = blockIdx.x / nct, c = (blockIdx.x % nct) * 64 + lane;
    const int cc = min(c, D - 1);
    const int per = (a.nblk + 15) / 16;
    const int k0 = min(run * per, a.nblk), k1 = min(k0 + per, a.nblk);
    const int64_t base = (int64_t)b * a.nblk * D + cc;
    float p = 1.f, h = 0.f, e = 0.f;
    float pk[B], hk[B], ek[B];
    auto load = [&](int k) {
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int64_t at = base + (int64_t)min(max(k + j, k0), k1 - 1) * D;
            pk[j] = a.ws_p[at];
            hk[j] = a.ws_h[at];
            ek[j] = a.ws_e[at];
        }
    };
    for (int k = k0; k < k1; k += B) {
        load(k);
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (k + j < k1) {
                e = glr_apply<PACKED>(p, ek[j], e);
                h = glr_apply<PACKED>(pk[j], h, hk[j]);
                p = glr_join<PACKED>(p, pk[j]);
            }
    }
    sp[run][lane] = p;
    sh[run][lane] = h;
    se[run][lane] = e;
    __syncthreads();
    h = a.init ? a.init[(int64_t)b * D + cc] : 0.f;
    for (int r = 0; r < run; ++r) h = glr_apply<PACKED>(sp[r][lane], h, sh[r][lane]);
    e = a.dfinal ? a.dfinal[(int64_t)b * D + cc] : 0.f;
    for (int r = 15; r > run; --r) e = glr_apply<PACKED>(sp[r][lane], e, se[r][lane]);
    if (c >= D) return;
    for (int k = k0; k < k1; k += B) {
        load(k);
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (k + j < k1) {
                a.ws_h[base + (int64_t)(k + j) * D] = h;
                h = glr_apply<PACKED>(pk[j], h, hk[j]);
            }
    }
    for (int k = k1 - B; k > k0 - B; k -= B) {
        load(k);
#pragma unroll
        for (int j = B - 1; j >= 0; --j)
            if (k + j >= k0) {
                a.ws_e[base + (int64_t)(k + j) * D] = e;
                e = glr_apply<PACKED>(pk[j], e, ek[j]);
            }
    }
    if (run == 0 && a.dinit) a.dinit[(int64_t)b * D + c] = e;
}

void launch_glr_block_scan(const GlrArgs &a, hipStream_t stream) {
    const unsigned grid = (unsigned)((int64_t)a.batch * ((a.channels + 63) / 64));
    if (a.seq_idx)
        hipLaunchKernelGGL(glr_block_scan_kernel<true>, dim3(grid), dim3(1024), 0, stream, a);
    else
        hipLaunchKernelGGL(glr_block_scan_kernel<false>, dim3(grid), dim3(1024), 0, stream, a);
}

// One token for every (row, channel): bound by the launch, then by reading and
// writing the state.
template <typename IO, int V, bool NORM>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrStepArgs a) {
    const int per = a.channels / V;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)a.batch * per) return;
    const int64_t b = i / per;
    const int c = (int)(i % per) * V;
    const int cb = c * (int)sizeof(IO);
    const Pack<IO, V> x = load_pack<IO, V>((const char *)a.x + b * a.xs + cb);
    const Pack<IO, V> g = load_pack<IO, V>((const char *)a.g + b * a.gs + cb);
    float *st = a.state + b * a.channels + c;
    float o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float p, k;
        gate_map<NORM>((float)g.v[v] + (a.bias ? a.bias[c + v] : 0.f), a.A[c + v], p, k);
        o[v] = fmaf(p, st[v], k * (float)x.v[v]);
        st[v] = o[v];
    }
    if (a.z) {
        const Pack<IO, V> z = load_pack<IO, V>((const char *)a.z + b * a.zs + cb);
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] *= (float)z.v[v] * sigmoid_f32((float)z.v[v]);
    }
    store_pack<IO, V>((IO *)a.y + b * a.channels + c, o);
}

template <typename IO, int V>
static void launch_step(const GlrStepArgs &a, hipStream_t stream) {
    const unsigned grid = (unsigned)(((int64_t)a.batch * (a.channels / V) + 255) / 256);
    if (a.normalize)
        hipLaunchKernelGGL((glr_step_kernel<IO, V, true>), dim3(grid), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((glr_step_kernel<IO, V, false>), dim3(grid), dim3(256), 0, stream, a);
}

void launch_glr_step(bool bf16_io, bool pair, const GlrStepArgs &a, hipStream_t stream) {
    if (bf16_io)
        pair ? launch_step<bf16, 2>(a, stream) : launch_step<bf16, 1>(a, stream);
    else
        pair ? launch_step<float, 2>(a, stream) : launch_step<float, 1>(a, stream);
}

void launch_glr_fwd(bool bf16_io, bool pair, const GlrArgs &a, hipStream_t stream) {
    bf16_io ? launch_glr_fwd_io<bf16>(pair, a, stream) : launch_glr_fwd_io<float>(pair, a, stream);
}

void launch_glr_bwd(bool bf16_io, bool pair, const GlrArgs &a, hipStream_t stream) {
    bf16_io ? launch_glr_bwd_io<bf16>(pair, a, stream) : launch_glr_bwd_io<float>(pair, a, stream);
    launch_part_sum(a.part, (int64_t)a.batch * a.nblk, a.channels, 1, a.dA, a.dbias, stream);
}

// Sums over parts: in holds `parts` rows of (taps + 1) planes (or `taps`, when
// out1 is null and nothing was written there) of n columns; plane j < taps of
// column c goes to out0[c * taps + j], the last plane to out1[c].  64 columns
// per workgroup, 16 threads per column over runs of rows, joined in order.
__global__ __launch_bounds__(1024) void part_sum_kernel(const float *in, int64_t parts, int n, int planes, int taps,
                                                        float *out0, float *out1) {
    __shared__ float s[16][64];
    const int lane = threadIdx.x % 64, run = threadIdx.x / 64;
    const int ncol = (n + 63) / 64;
    const int j = blockIdx.x / ncol, c = (blockIdx.x % ncol) * 64 + lane;
    const int64_t per = (parts + 15) / 16;
    const int64_t k0 = min((int64_t)run * per, parts), k1 = min(k0 + per, parts);
    const float *p = in + (int64_t)j * n + min(c, n - 1);
    const int64_t pitch = (int64_t)planes * n;
    float acc = 0.f;
#pragma unroll 8
    for (int64_t k = k0; k < k1; ++k) acc += p[k * pitch];
    s[run][lane] = acc;
    __syncthreads();
    if (run == 0 && c < n) {
        for (int r = 1; r < 16; ++r) acc += s[r][lane];
        if (j < taps)
            out0[(int64_t)c * taps + j] = acc;
        else if (out1)
            out1[c] = acc;
    }
}

void launch_part_sum(const float *in, int64_t parts, int n, int taps, float *out0, float *out1, hipStream_t stream,
                     int planes) {
    if (!planes) planes = taps + 1;
    const int run = out1 ? planes : taps;
    hipLaunchKernelGGL(part_sum_kernel, dim3((unsigned)((n + 63) / 64 * run)), dim3(1024), 0, stream, in, parts, n,
                       planes, taps, out0, out1);
}

}  // namespace ssd
