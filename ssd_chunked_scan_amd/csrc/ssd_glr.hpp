// Gated linear recurrence over channels (ssd.h, ssd_glr_*):
//
//   s = softplus(g + bias)   a = exp(A s)   k = sqrt(1 - a^2) or 1
//   h_t = r_t a_t h_{t-1} + k_t x_t         y_t = h_t [silu(z_t)]
//
// Each step is the affine map h -> p h + q (p = r a, q = k x); runs of tokens
// compose to one such map, (p2, q2) after (p1, q1) being (p2 p1, p2 q1 + q2),
// so a row is cut into segments whose maps are formed independently and
// joined in order.  Every p is a product of decays in [0, 1]: nothing is
// divided and no exponential of a positive sum is taken.
//
// A document start (r = 0) is kept apart from a decay that happens to be 0: it
// is a p with its sign bit set, which selects q instead of multiplying h by 0,
// so that an infinity or a NaN stays in its document.
//
// A workgroup owns a strip of CT channels and takes RT tokens at a time: lane
// l of a wave holds V adjacent channels and T consecutive tokens, its segment
// of the round, in registers.
#pragma once

#include "ssd_layer.hpp"

namespace ssd {

// V channels per lane, CL lanes along the channels, T tokens per lane, W waves.
template <int V_, int CL_, int T_, int W_>
struct GlrTile {
    static constexpr int V = V_, CL = CL_, T = T_, W = W_;
    static constexpr int TL = 64 / CL;       // segments per wave
    static constexpr int SEG = W * TL;       // segments per round
    static constexpr int RT = SEG * T;       // tokens per round
    static constexpr int CT = CL * V;        // channels per workgroup
};

// Pairs of channels: a token's strip is 64 (bf16) or 128 (fp32) bytes, so that
// the strips of a narrow layer still fill the device (5120 channels x 8 rows:
// 1280 workgroups).  The single-channel tile is for odd widths and strides and
// for pointers that do not allow pairs.  Both take RT = 128 tokens a round.
typedef GlrTile<2, 16, 8, 4> GlrPair;
typedef GlrTile<1, 32, 16, 4> GlrSingle;
constexpr int kGlrRound = 128;
static_assert(GlrPair::RT == kGlrRound && GlrSingle::RT == kGlrRound, "one round length");

constexpr float kGlrReset = -0.f;
__device__ inline bool glr_is_reset(float p) { return __float_as_int(p) < 0; }

// The decay of a token: a reset, or a with any sign of a NaN taken off.
template <bool PACKED>
__device__ inline float glr_mark(float a, bool cut) {
    return PACKED ? (cut ? kGlrReset : fabsf(a)) : a;
}

// q + p h.
template <bool PACKED>
__device__ inline float glr_apply(float p, float h, float q) {
    const float f = fmaf(p, h, q);
    return PACKED && glr_is_reset(p) ? q : f;
}

// p of two maps in a row: a reset when either is one.
template <bool PACKED>
__device__ inline float glr_join(float p, float p2) {
    const float m = p * p2;
    if (!PACKED) return m;
    return __int_as_float((__float_as_int(m) & 0x7fffffff) |
                          ((__float_as_int(p) | __float_as_int(p2)) & (int)0x80000000));
}

struct GlrUnit {
    int ct, blk, b;
};

template <typename TL>
__device__ inline GlrUnit glr_unit(const GlrArgs &a, int nblk) {
    // neighbouring strips share 128-byte lines: keep them on one XCD's L2
    const int nct = (a.channels + TL::CT - 1) / TL::CT;
    const int u = xcd_contiguous(blockIdx.x, gridDim.x);
    GlrUnit r;
    r.ct = u % nct;
    r.blk = (u / nct) % nblk;
    r.b = u / nct / nblk;
    return r;
}

// A lane's T tokens of a round, token strip `base` (token 0 of the round, byte
// offset `cb` of its channels); tokens from `valid` on repeat the last one.
template <typename IO, int V, int T>
__device__ inline void glr_load(Pack<IO, V> (&r)[T], const char *base, int64_t stride, int m, int cb, int valid) {
    if (m + T <= valid) {
        const uint32_t off = (uint32_t)m * (uint32_t)stride + (uint32_t)cb;
#pragma unroll
        for (int i = 0; i < T; ++i) r[i] = load_pack<IO, V>(base + i * stride + off);
    } else {
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const uint32_t tok = (uint32_t)min(m + i, valid - 1);
            r[i] = load_pack<IO, V>(base + (tok * (uint32_t)stride + (uint32_t)cb));
        }
    }
}

// Bit i set where a document starts at token t + i of the row (never at its
// first token), for tokens before `L`.
template <int T>
__device__ inline uint32_t glr_resets(const int32_t *seq, int t, int L) {
    uint32_t bits = 0;
    int p = seq[min(max(t - 1, 0), L - 1)];
#pragma unroll
    for (int i = 0; i < T; ++i) {
        const int q = seq[min(t + i, L - 1)];
        bits |= (q != p ? 1u : 0u) << i;
        p = q;
    }
    return bits;
}

// The forward walk: one workgroup per (row, split, strip), round after round
// with the strip's state carried through LDS.  Per round each lane forms the
// maps of its tokens, publishes its segment's map, and after one barrier
// composes the segments before its own.  x and g of the next round are loaded
// meanwhile.
template <typename IO, typename TL, bool NORM, bool PACKED>
__global__ __launch_bounds__(TL::W * 64) void glr_fwd_kernel(GlrArgs a) {
    constexpr int V = TL::V, T = TL::T, SEG = TL::SEG, CT = TL::CT;
    __shared__ float2 seg_map[2][SEG][CT];
    __shared__ float carry[2][CT];
    const GlrUnit u = glr_unit<TL>(a, a.nblk);
    const int tid = threadIdx.x, cg = tid % TL::CL, seg = tid / TL::CL, m = seg * T;
    const int D = a.channels, L = a.seqlen;
    const int c = u.ct * CT + cg * V;
    const bool cok = c < D;
    const int cc = cok ? c : D - V;
    const int t0 = u.blk * a.blk_len, t1 = min(L, t0 + a.blk_len);
    float A[V], bias[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = a.A[cc + v];
        bias[v] = a.bias ? a.bias[cc + v] : 0.f;
    }
    if (seg == SEG - 1) {
        // the state entering this split: the maps of the splits before it
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float h = a.init ? a.init[(int64_t)u.b * D + cc + v] : 0.f;
            const int64_t at = (int64_t)u.b * a.nblk * D + cc + v;
            for (int q = 0; q < u.blk; ++q) 
                h = glr_apply<PACKED>(a.ws_p[at + (int64_t)q * D], h, a.ws_h[at + (int64_t)q * D]);
            carry[0][cg * V + v] = h;
        }
    }
    const int cb = cc * (int)sizeof(IO);
    const int64_t row = (int64_t)u.b * L;
    const char *xb = (const char *)a.x + row * a.xs;
    const char *gb = (const char *)a.g + row * a.gs;
    const char *zb = (const char *)a.z + row * a.zs;
    IO *yb = (IO *)a.y + row * D;
    Pack<IO, V> xr[T], gr[T], xn[T], gn[T], zr[T];
    glr_load<IO, V, T>(xr, xb + t0 * a.xs, a.xs, m, cb, L - t0);
    glr_load<IO, V, T>(gr, gb + t0 * a.gs, a.gs, m, cb, L - t0);
    int buf = 0;
    for (int t = t0; t < t1; t += TL::RT, buf ^= 1) {
        if (a.z) glr_load<IO, V, T>(zr, zb + t * a.zs, a.zs, m, cb, L - t);
        if (t + TL::RT < t1) {
            glr_load<IO, V, T>(xn, xb + (t + TL::RT) * a.xs, a.xs, m, cb, L - t - TL::RT);
            glr_load<IO, V, T>(gn, gb + (t + TL::RT) * a.gs, a.gs, m, cb, L - t - TL::RT);
        }
        float p[T][V], q[T][V];
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float k;
                gate_map<NORM>((float)gr[i].v[v] + bias[v], A[v], p[i][v], k);
                q[i][v] = k * (float)xr[i].v[v];
            }
        if (PACKED) {
            const uint32_t cut = glr_resets<T>(a.seq_idx + row, t + m, L);
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) p[i][v] = glr_mark<PACKED>(p[i][v], (cut >> i) & 1);
        }
        if (t + m + T > L) {
            // past the row's end: the identity map
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const bool ok = t + m + i < L;
                    p[i][v] = ok ? p[i][v] : 1.f;
                    q[i][v] = ok ? q[i][v] : 0.f;
                }
        }
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float ps = p[0][v], qs = q[0][v];
#pragma unroll
            for (int i = 1; i < T; ++i) {
                ps = glr_join<PACKED>(ps, p[i][v]);
                qs = glr_apply<PACKED>(p[i][v], qs, q[i][v]);
            }
            seg_map[buf][seg][cg * V + v] = make_float2(ps, qs);
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = carry[buf][cg * V + v];
        for (int s = 0; s < seg; ++s)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float2 f = seg_map[buf][s][cg * V + v];
                h[v] = glr_apply<PACKED>(f.x, h[v], f.y);
            }
#pragma unroll
        for (int i = 0; i < T; ++i) {
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[v] = glr_apply<PACKED>(p[i][v], h[v], q[i][v]);
                o[v] = h[v];
            }
            if (a.z) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float z = (float)zr[i].v[v];
                    o[v] *= z * sigmoid_f32(z);
                }
            }
            if (cok && t + m + i < L) store_pack<IO, V>(yb + (int64_t)(t + m + i) * D + cc, o);
        }
        if (seg == SEG - 1) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                carry[buf ^ 1][cg * V + v] = h[v];
                if (t + TL::RT >= L && a.final_states && cok) a.final_states[(int64_t)u.b * D + cc + v] = h[v];
            }
        }
#pragma unroll
        for (int i = 0; i < T; ++i) {
            xr[i] = xn[i];
            gr[i] = gn[i];
        }
    }
}

// The map of each block of blk_len tokens (ws_p, ws_h), and with BWD the
// adjoint a block passes to the tokens before it when none enters from behind:
// with G_t = e_t + c_t and c_{t-1} = p_t G_t, c before the block is
// sum_t (p_first .. p_t) e_t.  Each lane walks its segment of blk_len / SEG
// tokens; the segments are joined at the end.
template <typename IO, typename TL, bool NORM, bool PACKED, bool BWD>
__global__ __launch_bounds__(TL::W * 64) void glr_block_kernel(GlrArgs a, int nblk) {
    constexpr int V = TL::V, T = TL::T, SEG = TL::SEG, CT = TL::CT;
    __shared__ float2 seg_map[SEG][CT];
    __shared__ float seg_e[BWD ? SEG : 1][CT];
    const GlrUnit u = glr_unit<TL>(a, nblk);
    const int tid = threadIdx.x, cg = tid % TL::CL, seg = tid / TL::CL;
    const int D = a.channels, L = a.seqlen;
    const int c = u.ct * CT + cg * V;
    const bool cok = c < D;
    const int cc = cok ? c : D - V, cb = cc * (int)sizeof(IO);
    const int per = a.blk_len / SEG;
    const int t0 = u.blk * a.blk_len;
    const int64_t row = (int64_t)u.b * L;
    const char *xb = (const char *)a.x + row * a.xs;
    const char *gb = (const char *)a.g + row * a.gs;
    const char *zb = (const char *)a.z + row * a.zs;
    const char *db = (const char *)a.dy + row * a.dys;
    float A[V], bias[V], ps[V], qs[V], es[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = a.A[cc + v];
        bias[v] = a.bias ? a.bias[cc + v] : 0.f;
        ps[v] = 1.f;
        qs[v] = es[v] = 0.f;
    }
    for (int j = 0; j < per; j += T) {
        // this lane's first token: 64-bit row offsets, since a split's tokens
        // times the stride can pass 32 bits
        const int t = t0 + seg * per + j;
        if (t >= L) break;   // no barrier inside the loop
        Pack<IO, V> xr[T], gr[T], zr[T], dr[T];
        glr_load<IO, V, T>(xr, xb + t * a.xs, a.xs, 0, cb, L - t);
        glr_load<IO, V, T>(gr, gb + t * a.gs, a.gs, 0, cb, L - t);
        if (BWD) glr_load<IO, V, T>(dr, db + t * a.dys, a.dys, 0, cb, L - t);
        if (BWD && a.z) glr_load<IO, V, T>(zr, zb + t * a.zs, a.zs, 0, cb, L - t);
        const uint32_t cut = PACKED ? glr_resets<T>(a.seq_idx + row, t, L) : 0u;
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const bool ok = t + i < L;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float p, k;
                gate_map<NORM>((float)gr[i].v[v] + bias[v], A[v], p, k);
                const float q = ok ? k * (float)xr[i].v[v] : 0.f;
                p = ok ? glr_mark<PACKED>(p, (cut >> i) & 1) : 1.f;
                qs[v] = glr_apply<PACKED>(p, qs[v], q);
                ps[v] = glr_join<PACKED>(ps[v], p);
                if (BWD) {
                    float e = (float)dr[i].v[v];
                    if (a.z) {
                        const float z = (float)zr[i].v[v];
                        e *= z * sigmoid_f32(z);
                    }
                    es[v] = glr_apply<PACKED>(ps[v], ok ? e : 0.f, es[v]);
                }
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        seg_map[seg][cg * V + v] = make_float2(ps[v], qs[v]);
        if (BWD) seg_e[seg][cg * V + v] = es[v];
    }
    __syncthreads();
    if (tid < CT && u.ct * CT + tid < D) {
        float p = 1.f, q = 0.f, e = 0.f;
        for (int s = 0; s < SEG; ++s) {
            const float2 f = seg_map[s][tid];
            if (BWD) e = glr_apply<PACKED>(p, seg_e[s][tid], e);
            q = glr_apply<PACKED>(f.x, q, f.y);
            p = glr_join<PACKED>(p, f.x);
        }
        const int64_t at = ((int64_t)u.b * a.nblk + u.blk) * D + u.ct * CT + tid;
        a.ws_p[at] = p;
        a.ws_h[at] = q;
        if (BWD) a.ws_e[at] = e;
    }
}

// Backward, one workgroup per (row, block of RT tokens, strip), with the state
// entering the block from the left (ws_h) and the adjoint from the right
// (ws_e) already known:
//   G_t = e_t + c_t,  c_{t-1} = p_t G_t,  e = dy [silu(z)]
//   dx = k G     dla = c_{t-1} h_{t-1} + G x dk/dla,  dk/dla = -a^2 / k
//   dg = A dla sigmoid(g + bias)   dA = sum s dla   dbias = sum dg
//   dz = dy h silu'(z)
template <typename IO, typename TL, bool NORM, bool PACKED>
__global__ __launch_bounds__(TL::W * 64) void glr_bwd_kernel(GlrArgs a) {
    constexpr int V = TL::V, T = TL::T, SEG = TL::SEG, CT = TL::CT;
    __shared__ float2 seg_map[SEG][CT];
    __shared__ float seg_e[SEG][CT];
    const GlrUnit u = glr_unit<TL>(a, a.nblk);
    const int tid = threadIdx.x, cg = tid % TL::CL, seg = tid / TL::CL, m = seg * T;
    const int D = a.channels, L = a.seqlen;
    const int c = u.ct * CT + cg * V;
    const bool cok = c < D;
    const int cc = cok ? c : D - V, cb = cc * (int)sizeof(IO);
    const int t = u.blk * TL::RT;
    const int64_t row = (int64_t)u.b * L;
    const int64_t wsat = ((int64_t)u.b * a.nblk + u.blk) * D + cc;
    Pack<IO, V> xr[T], gr[T], zr[T], dr[T];
    glr_load<IO, V, T>(gr, (const char *)a.g + (row + t) * a.gs, a.gs, m, cb, L - t);
    glr_load<IO, V, T>(xr, (const char *)a.x + (row + t) * a.xs, a.xs, m, cb, L - t);
    glr_load<IO, V, T>(dr, (const char *)a.dy + (row + t) * a.dys, a.dys, m, cb, L - t);
    if (a.z) glr_load<IO, V, T>(zr, (const char *)a.z + (row + t) * a.zs, a.zs, m, cb, L - t);
    const uint32_t cut = PACKED ? glr_resets<T>(a.seq_idx + row, t + m, L) : 0u;
    float A[V], bias[V], hin[V], cin[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = a.A[cc + v];
        bias[v] = a.bias ? a.bias[cc + v] : 0.f;
        hin[v] = a.ws_h[wsat + v];
        cin[v] = a.ws_e[wsat + v];
    }
    float al[T][V], k[T][V], sp[T][V], sg[T][V], sz[T][V];
#pragma unroll
    for (int i = 0; i < T; ++i) {
        const bool ok = t + m + i < L;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float gv = (float)gr[i].v[v] + bias[v];
            float e, w;
            const float s = softplus_precise(gv, e, w), la = A[v] * s;
            const float av = __builtin_amdgcn_exp2f(kLog2e * la);
            al[i][v] = ok ? av : 1.f;
            k[i][v] = ok ? (NORM ? __builtin_amdgcn_sqrtf(one_minus_square(av, la)) : 1.f) : 0.f;
            sp[i][v] = ok ? s : 0.f;
            sg[i][v] = ok ? (gv >= 0.f ? 1.f : e) * __builtin_amdgcn_rcpf(w) : 0.f;
            sz[i][v] = a.z ? sigmoid_f32((float)zr[i].v[v]) : 0.f;
        }
    }
    auto p_of = [&](int i, int v) { return glr_mark<PACKED>(al[i][v], (cut >> i) & 1); };
    auto e_of = [&](int i, int v) {
        const float d = (float)dr[i].v[v];
        const float e = a.z ? d * ((float)zr[i].v[v] * sz[i][v]) : d;
        return t + m + i < L ? e : 0.f;
    };
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float ps = 1.f, qs = 0.f, es = 0.f;
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const float p = p_of(i, v);
            qs = glr_apply<PACKED>(p, qs, k[i][v] * (float)xr[i].v[v]);
            ps = glr_join<PACKED>(ps, p);
            es = glr_apply<PACKED>(ps, e_of(i, v), es);
        }
        seg_map[seg][cg * V + v] = make_float2(ps, qs);
        seg_e[seg][cg * V + v] = es;
    }
    __syncthreads();
    for (int s = 0; s < seg; ++s)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float2 f = seg_map[s][cg * V + v];
            hin[v] = glr_apply<PACKED>(f.x, hin[v], f.y);
        }
    for (int s = SEG - 1; s > seg; --s)
#pragma unroll
        for (int v = 0; v < V; ++v) 
            cin[v] = glr_apply<PACKED>(seg_map[s][cg * V + v].x, cin[v], seg_e[s][cg * V + v]);
    float h[T][V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float hv = hin[v];
#pragma unroll
        for (int i = 0; i < T; ++i) {
            hv = glr_apply<PACKED>(p_of(i, v), hv, k[i][v] * (float)xr[i].v[v]);
            h[i][v] = hv;
        }
    }
    float dA[V], dbias[V];
#pragma unroll
    for (int v = 0; v < V; ++v) dA[v] = dbias[v] = 0.f;
#pragma unroll
    for (int i = T - 1; i >= 0; --i) {
        float dx[V], dg[V], dz[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float G = e_of(i, v) + cin[v];
            const float x = (float)xr[i].v[v];
            const bool reset = PACKED && ((cut >> i) & 1);
            cin[v] = reset ? 0.f : al[i][v] * G;
            dx[v] = k[i][v] * G;
            float dla = reset ? 0.f : cin[v] * (i > 0 ? h[i > 0 ? i - 1 : 0][v] : hin[v]);
            if (NORM) {
                const float rk = k[i][v] > 0.f ? __builtin_amdgcn_rcpf(k[i][v]) : 0.f;
                dla = fmaf(-G * x, al[i][v] * al[i][v] * rk, dla);
            }
            dg[v] = A[v] * dla * sg[i][v];
            dA[v] = fmaf(sp[i][v], dla, dA[v]);
            dbias[v] += dg[v];
            const float z = (float)zr[i].v[v];
            dz[v] = a.z ? (float)dr[i].v[v] * h[i][v] * (sz[i][v] * fmaf(z, 1.f - sz[i][v], 1.f)) : 0.f;
        }
        if (cok && t + m + i < L) {
            const int64_t at = (row + t + m + i) * D + cc;
            store_pack<IO, V>((IO *)a.dx + at, dx);
            store_pack<IO, V>((IO *)a.dg + at, dg);
            if (a.z) store_pack<IO, V>((IO *)a.dz + at, dz);
        }
    }
    // dA and dbias of the block: the lanes' sums over their tokens, joined in
    // segment order
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) seg_map[seg][cg * V + v] = make_float2(dA[v], dbias[v]);
    __syncthreads();
    if (tid < CT && u.ct * CT + tid < D) {
        float2 s = make_float2(0.f, 0.f);
        for (int j = 0; j < SEG; ++j) {
            s.x += seg_map[j][tid].x;
            s.y += seg_map[j][tid].y;
        }
        float *out = a.part + ((int64_t)u.b * a.nblk + u.blk) * 2 * D + u.ct * CT + tid;
        out[0] = s.x;
        out[D] = s.y;
    }
}

template <typename IO>
void launch_glr_fwd_io(bool pair, const GlrArgs &a, hipStream_t stream);
template <typename IO>
void launch_glr_bwd_io(bool pair, const GlrArgs &a, hipStream_t stream);

template <typename TL>
inline dim3 glr_grid(const GlrArgs &a, int nblk) {
    return dim3((unsigned)((int64_t)a.batch * nblk * ((a.channels + TL::CT - 1) / TL::CT)));
}

template <typename IO, typename TL, bool NORM, bool PACKED>
void launch_glr_fwd_docs(const GlrArgs &a, hipStream_t stream) {
    if (a.nblk > 1)
        hipLaunchKernelGGL((glr_block_kernel<IO, TL, NORM, PACKED, false>), glr_grid<TL>(a, a.nblk - 1),
                           dim3(TL::W * 64), 0, stream, a, a.nblk - 1);
    hipLaunchKernelGGL((glr_fwd_kernel<IO, TL, NORM, PACKED>), glr_grid<TL>(a, a.nblk), dim3(TL::W * 64), 0, stream, a);
}

template <typename IO, typename TL, bool NORM>
void launch_glr_fwd_tile(const GlrArgs &a, hipStream_t stream) {
    a.seq_idx ? launch_glr_fwd_docs<IO, TL, NORM, true>(a, stream) : launch_glr_fwd_docs<IO, TL, NORM, false>(a, stream);
}

void launch_glr_block_scan(const GlrArgs &a, hipStream_t stream);

template <typename IO, typename TL, bool NORM, bool PACKED>
void launch_glr_bwd_docs(const GlrArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL((glr_block_kernel<IO, TL, NORM, PACKED, true>), glr_grid<TL>(a, a.nblk), dim3(TL::W * 64), 0,
                       stream, a, a.nblk);
    launch_glr_block_scan(a, stream);
    hipLaunchKernelGGL((glr_bwd_kernel<IO, TL, NORM, PACKED>), glr_grid<TL>(a, a.nblk), dim3(TL::W * 64), 0, stream, a);
}

template <typename IO, typename TL, bool NORM>
void launch_glr_bwd_tile(const GlrArgs &a, hipStream_t stream) {
    a.seq_idx ? launch_glr_bwd_docs<IO, TL, NORM, true>(a, stream) : launch_glr_bwd_docs<IO, TL, NORM, false>(a, stream);
}

#define SSD_GLR_INSTANTIATE(IO)                                                                      \
    template <>                                                                                      \
    void launch_glr_fwd_io<IO>(bool pair, const GlrArgs &a, hipStream_t stream) {                    \
        if (pair)                                                                                    \
            a.normalize ? launch_glr_fwd_tile<IO, GlrPair, true>(a, stream)                          \
                        : launch_glr_fwd_tile<IO, GlrPair, false>(a, stream);                        \
        else                                                                                         \
            a.normalize ? launch_glr_fwd_tile<IO, GlrSingle, true>(a, stream)                        \
                        : launch_glr_fwd_tile<IO, GlrSingle, false>(a, stream);                      \
    }                                                                                                \
    template <>                                                                                      \
    void launch_glr_bwd_io<IO>(bool pair, const GlrArgs &a, hipStream_t stream) {                    \
        if (pair)                                                                                    \
            a.normalize ? launch_glr_bwd_tile<IO, GlrPair, true>(a, stream)                          \
                        : launch_glr_bwd_tile<IO, GlrPair, false>(a, stream);                        \
        else                                                                                         \
            a.normalize ? launch_glr_bwd_tile<IO, GlrSingle, true>(a, stream)                        \
                        : launch_glr_bwd_tile<IO, GlrSingle, false>(a, stream);                      \
    }

}  // namespace ssd
