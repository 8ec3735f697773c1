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

#include <type_traits>

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

// Pairs of channels, 32 lanes of them: a token's strip is a 128-byte line in
// bf16 (with 64 bytes the forward walk over 8 x 2048 x 5120 took 168 us
// instead of 155).  The single-channel tiles are for odd widths and strides
// and for pointers that do not allow pairs.  The backward tiles hold half as
// many tokens a lane, since seven values of each stay in registers.
typedef GlrTile<2, 32, 8, 8> GlrFwdPair;
typedef GlrTile<2, 16, 4, 8> GlrFwdHalf;   // half a strip for the last, partial round of workgroups
typedef GlrTile<1, 32, 16, 4> GlrFwdSingle;
typedef GlrTile<2, 32, 4, 8> GlrBwdPair;
typedef GlrTile<1, 32, 8, 4> GlrBwdSingle;
typedef GlrTile<2, 32, 8, 4> GlrBlockPair;   // the backward blocks' maps: nothing stays
// Rows of at most 16 tokens, where the long tiles' waves would mostly be past
// the row's end (256 x 16 x 4096 forward 105 -> 27 us, backward 267 -> 62).
constexpr int kGlrShort = 16;
typedef GlrTile<2, 32, 8, 1> GlrFwdPairShort;
typedef GlrTile<1, 32, 8, 1> GlrFwdSingleShort;
typedef GlrTile<2, 32, 4, 2> GlrBwdPairShort;
typedef GlrTile<1, 32, 8, 1> GlrBwdSingleShort;
static_assert(GlrFwdPairShort::RT == kGlrShort && GlrFwdSingleShort::RT == kGlrShort, "");
static_assert(GlrBwdPairShort::RT == kGlrShort && GlrBwdSingleShort::RT == kGlrShort, "");
constexpr int kGlrFwdRound = 128, kGlrBwdBlock = 64;   // tokens a forward round, a backward block
static_assert(GlrFwdHalf::CT * 2 == GlrFwdPair::CT && GlrFwdHalf::W == GlrFwdPair::W, "");
static_assert(GlrFwdHalf::RT == kGlrFwdRound && GlrFwdPair::RT == kGlrFwdRound && GlrFwdSingle::RT == kGlrFwdRound, "");
static_assert(GlrBwdPair::RT == kGlrBwdBlock && GlrBwdSingle::RT == kGlrBwdBlock && GlrBlockPair::RT == kGlrBwdBlock, "");

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

template <typename TL, bool REVERSED = false>
__device__ inline GlrUnit glr_unit(const GlrArgs &a, int nblk) {
    // neighbouring strips share 128-byte lines: keep them on one XCD's L2
    const int nct = (a.channels + TL::CT - 1) / TL::CT;
    int u = xcd_contiguous(blockIdx.x, gridDim.x);
    if (REVERSED) u = (int)gridDim.x - 1 - u;
    GlrUnit r;
    r.ct = u % nct;
    r.blk = (u / nct) % nblk;
    r.b = u / nct / nblk;
    return r;
}

// A lane's T tokens from token m of a run on: `base` is the run's token 0, the
// same for the whole workgroup, cb the byte offset of the lane's channels.
// Tokens from `valid` on repeat the last one (not FULL).
template <bool FULL, typename R, int T>
__device__ inline void glr_load(R (&r)[T], const char *base, int64_t stride, int m, int cb, int valid) {
    const __amdgpu_buffer_rsrc_t b = buffer_of(base);
    const uint32_t st = (uint32_t)stride;
    if (FULL) {
        const uint32_t off = (uint32_t)m * st + (uint32_t)cb;
#pragma unroll
        for (int i = 0; i < T; ++i) r[i] = buffer_load<R>(b, off, i * st);
    } else {
#pragma unroll
        for (int i = 0; i < T; ++i) r[i] = buffer_load<R>(b, (uint32_t)min(m + i, valid - 1) * st + (uint32_t)cb, 0);
    }
}

// The same from the lane's own first token on, `valid` of them.
template <typename R, int T>
__device__ inline void glr_load_lane(R (&r)[T], const char *p, int64_t stride, int valid) {
    if (valid >= T) {
#pragma unroll
        for (int i = 0; i < T; ++i, p += stride) r[i] = *(const R *)p;
    } else {
#pragma unroll
        for (int i = 0; i < T; ++i) r[i] = *(const R *)(p + min(i, valid - 1) * stride);
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

// The same for a lane whose wave's segments follow each other from token t of
// the row on, one lane looking at each token.  Called by whole waves.
template <typename TL>
__device__ inline uint32_t glr_wave_resets(const int32_t *seq, int t, int L) {
    static_assert(TL::TL * TL::T <= 64, "a lane per token");
    const int k = t + (int)(threadIdx.x % 64);
    const bool cut = seq[min(k, L - 1)] != seq[min(max(k - 1, 0), L - 1)];
    const uint64_t bits = __ballot(cut);
    return (uint32_t)(bits >> (threadIdx.x % 64 / TL::CL * TL::T)) & ((1u << TL::T) - 1u);
}

// h after the maps of the segments before `seg` (wave `wave`'s are TL::TL in a
// row): whole waves first, so that their maps are read together.
template <bool PACKED, typename TL>
__device__ inline void glr_enter(float (&h)[TL::V], const float2 (&maps)[TL::SEG][TL::CT], int ch, int seg) {
    const int wave = __builtin_amdgcn_readfirstlane(seg / TL::TL), mine = seg % TL::TL;
#pragma unroll 4
    for (int s = 0; s < wave * TL::TL; ++s) {
        float2 f[TL::V];
#pragma unroll
        for (int v = 0; v < TL::V; ++v) f[v] = maps[s][ch + v];
#pragma unroll
        for (int v = 0; v < TL::V; ++v) h[v] = glr_apply<PACKED>(f[v].x, h[v], f[v].y);
    }
#pragma unroll
    for (int j = 0; j < TL::TL - 1; ++j)
#pragma unroll
        for (int v = 0; v < TL::V; ++v) {
            const float2 f = maps[wave * TL::TL + j][ch + v];
            const float n = glr_apply<PACKED>(f.x, h[v], f.y);
            h[v] = j < mine ? n : h[v];
        }
}

// The forward walk: one workgroup per (row, split, strip), round after round
// with the strip's state carried through LDS.  Per round each lane forms the
// maps of its tokens, publishes its segment's map, and after one barrier
// composes the segments before its own.  x and g of the next round are loaded
// as soon as this round's are used up.
//
// Bound by vector instructions and memory alike: 44 issue slots an element for
// the map (of them 16 in exp2, log2, exp2 and the root), 12 for the gate, 5
// for the two passes over the tokens, in all about 133 us for 8 x 2048 x 5120
// against 137 for its 671 MB at a large copy's rate; it takes 155 (4.3 TB/s).
template <typename IO, typename TL, bool NORM, bool PACKED, bool GATE>
__device__ inline void glr_fwd_walk(const GlrArgs &a, const GlrUnit u) {
    constexpr int V = TL::V, T = TL::T, SEG = TL::SEG, CT = TL::CT;
    typedef Raw<IO, V> RW;
    typedef typename RW::type R;
    __shared__ float2 seg_map[2][SEG][CT];
    __shared__ float carry[2][CT];
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
    // The state entering this split: the maps of the splits before it.  Every
    // lane forms it: under a divergent branch the scalar row offsets would be
    // merged into vector registers, and every address with them.
    {
        float h[V];
        const int64_t at = (int64_t)u.b * a.nblk * D + cc;
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = a.init ? a.init[(int64_t)u.b * D + cc + v] : 0.f;
        for (int s = 0; s < u.blk; s += 8) {
            float p[8][V], q[8][V];   // eight at a time: one wait for their loads
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int64_t k = at + (int64_t)min(s + j, u.blk - 1) * D + v;
                    p[j][v] = a.ws_p[k];
                    q[j][v] = a.ws_h[k];
                }
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (s + j < u.blk) h[v] = glr_apply<PACKED>(p[j][v], h[v], q[j][v]);
        }
        if (seg == SEG - 1)
#pragma unroll
            for (int v = 0; v < V; ++v) carry[0][cg * V + v] = h[v];
    }
    const int cb = cc * (int)sizeof(IO);
    const int64_t row = (int64_t)u.b * L;
    const char *xb = (const char *)a.x + row * a.xs;
    const char *gb = (const char *)a.g + row * a.gs;
    const char *zb = (const char *)a.z + row * a.zs;
    char *yb = (char *)a.y + row * D * (int)sizeof(IO);
    const int64_t ys = (int64_t)D * (int)sizeof(IO);
    R xr[T], gr[T], zr[T];
    auto load = [&](int t) {
        if (t + TL::RT <= L) {
            glr_load<true>(xr, xb + t * a.xs, a.xs, m, cb, 0);
            glr_load<true>(gr, gb + t * a.gs, a.gs, m, cb, 0);
        } else {
            glr_load<false>(xr, xb + t * a.xs, a.xs, m, cb, L - t);
            glr_load<false>(gr, gb + t * a.gs, a.gs, m, cb, L - t);
        }
    };
    auto round = [&](int t, int buf, auto full) {
        constexpr bool FULL = decltype(full)::value;
        // whether the wave has a token before the row's end at all: short rows
        // leave most waves of a round without one
        const bool any = FULL || t + __builtin_amdgcn_readfirstlane(tid / 64) * (TL::TL * T) < L;
        const uint32_t cut = PACKED ? glr_wave_resets<TL>(a.seq_idx + row, t + tid / 64 * (TL::TL * T), L) : 0u;
        float p[T][V], q[T][V];
        if (any) {
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float k;
                    gate_map<NORM>(RW::at(gr[i], v) + bias[v], A[v], p[i][v], k);
                    p[i][v] = glr_mark<PACKED>(p[i][v], (cut >> i) & 1);
                    q[i][v] = k * RW::at(xr[i], v);
                    if (!FULL) {
                        // past the row's end: the identity map
                        const bool ok = t + m + i < L;
                        p[i][v] = ok ? p[i][v] : 1.f;
                        q[i][v] = ok ? q[i][v] : 0.f;
                    }
                }
        } else {
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    p[i][v] = 1.f;
                    q[i][v] = 0.f;
                }
        }
        // the maps are formed here, before the next loads take the registers of
        // the words they came from, and not sunk to their use behind them
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) asm volatile("" : "+v"(p[i][v]), "+v"(q[i][v]));
        // (z in front of them: waiting for it does not wait for them)
        if (GATE && any) glr_load<FULL>(zr, zb + t * a.zs, a.zs, m, cb, L - t);
        if (t + TL::RT < t1) load(t + TL::RT);
        float h[V];
        // (most waves see no document start: their maps go without the marks)
        auto chain = [&](auto marked) {
            constexpr bool MARKED = decltype(marked)::value;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float ps = p[0][v], qs = q[0][v];
#pragma unroll
                for (int i = 1; i < T; ++i) {
                    ps = glr_join<MARKED>(ps, p[i][v]);
                    qs = glr_apply<MARKED>(p[i][v], qs, q[i][v]);
                }
                seg_map[buf][seg][cg * V + v] = make_float2(ps, qs);
            }
        };
        if (PACKED && __any(cut != 0))
            chain(std::true_type{});
        else
            chain(std::false_type{});
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = carry[buf][cg * V + v];
        glr_enter<PACKED, TL>(h, seg_map[buf], cg * V, seg);
        const __amdgpu_buffer_rsrc_t yt = buffer_of(yb + t * ys);
        const uint32_t off = (uint32_t)m * (uint32_t)ys + (uint32_t)cb;
        if (any) {
#pragma unroll
            for (int i = 0; i < T; ++i) {
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    h[v] = glr_apply<PACKED>(p[i][v], h[v], q[i][v]);
                    o[v] = h[v];
                    if (GATE) {
                        const float z = RW::at(zr[i], v);
                        o[v] *= z * sigmoid_f32(z);
                    }
                }
                if (FULL || (cok && t + m + i < L)) buffer_store<IO, V>(yt, off, (uint32_t)(i * ys), o);
            }
        }
        if (seg == SEG - 1) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                carry[buf ^ 1][cg * V + v] = h[v];
                if (t + TL::RT >= L && a.final_states && cok) a.final_states[(int64_t)u.b * D + cc + v] = h[v];
            }
        }
    };
    load(t0);
    // whole rounds of a whole strip in a loop of their own: the guarded form
    // beside them would take half as many registers again
    int buf = 0, t = t0;
    if ((u.ct + 1) * CT <= D)
        for (; t < t1 && t + TL::RT <= L; t += TL::RT, buf ^= 1) round(t, buf, std::true_type{});
    for (; t < t1; t += TL::RT, buf ^= 1) round(t, buf, std::false_type{});
}

// A compute unit's vector unit is what its workgroups wait for, so their count
// per compute unit should be even: with a little over one workgroup for each,
// those left over run as two of half a strip (4 x 2048 x 5120, 320 units on 256
// compute units: 108 -> 85 us).  Not from two for each on, where two already
// overlap and the half strips' 64-byte rows cost more than the balance gains
// (8 x 2048 x 5120, 640 units: 155 us whole, 160 with 128 of them halved).
template <typename IO, typename TL, typename HALF, bool NORM, bool PACKED, bool GATE>
__global__ __launch_bounds__(TL::W * 64) void glr_fwd_kernel(GlrArgs a) {
    const int blk = blockIdx.x;
    int unit;
    if (blk < a.whole)
        unit = xcd_contiguous(blk, a.whole);
    else
        unit = a.whole * 2 + xcd_contiguous(blk - a.whole, gridDim.x - a.whole);
    const int half = blk < a.whole ? 0 : unit & 1;
    if (blk >= a.whole) unit = (unit >> 1);
    const int nct = (a.channels + TL::CT - 1) / TL::CT;
    GlrUnit u;
    u.ct = unit % nct;
    u.blk = (unit / nct) % a.nblk;
    u.b = unit / nct / a.nblk;
    if constexpr (!std::is_same<TL, HALF>::value) {
        if (blk >= a.whole) {
            u.ct = 2 * u.ct + half;
            if (u.ct * HALF::CT < a.channels) glr_fwd_walk<IO, HALF, NORM, PACKED, GATE>(a, u);
            return;
        }
    }
    glr_fwd_walk<IO, TL, NORM, PACKED, GATE>(a, u);
}

// The map of each block of blk_len tokens (ws_p, ws_h), and with BWD the
// adjoint a block passes to the tokens before it when none enters from behind:
// with G_t = e_t + c_t and c_{t-1} = p_t G_t, c before the block is
// sum_t (p_first .. p_t) e_t.  Each lane walks its segment of blk_len / SEG
// tokens; the segments are joined at the end.
template <typename IO, typename TL, bool NORM, bool PACKED, bool BWD, bool GATE>
__global__ __launch_bounds__(TL::W * 64) void glr_block_kernel(GlrArgs a, int nblk) {
    constexpr int V = TL::V, T = TL::T, SEG = TL::SEG, CT = TL::CT;
    typedef Raw<IO, V> RW;
    typedef typename RW::type R;
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
    uint32_t seen = 0;
    for (int j = 0; j < per; j += T) {
        // this lane's first token: 64-bit row offsets, since a split's tokens
        // times the stride can pass 32 bits
        const int t = t0 + seg * per + j;
        if (t >= L) break;   // no barrier inside the loop
        R xr[T], gr[T], zr[T], dr[T];
        glr_load_lane(xr, xb + t * a.xs + cb, a.xs, L - t);
        glr_load_lane(gr, gb + t * a.gs + cb, a.gs, L - t);
        if (BWD) glr_load_lane(dr, db + t * a.dys + cb, a.dys, L - t);
        if (BWD && GATE) glr_load_lane(zr, zb + t * a.zs + cb, a.zs, L - t);
        const uint32_t cut = PACKED ? glr_resets<T>(a.seq_idx + row, t, L) : 0u;
        // marks only from the wave's first document start on
        seen |= cut;
        auto tokens = [&](auto marked) {
            constexpr bool MARKED = decltype(marked)::value;
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const bool ok = t + i < L;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float p, k;
                    gate_map<NORM>(RW::at(gr[i], v) + bias[v], A[v], p, k);
                    const float q = ok ? k * RW::at(xr[i], v) : 0.f;
                    p = ok ? glr_mark<PACKED>(p, MARKED && ((cut >> i) & 1)) : 1.f;
                    qs[v] = glr_apply<MARKED>(p, qs[v], q);
                    ps[v] = glr_join<MARKED>(ps[v], p);
                    if (BWD) {
                        float e = RW::at(dr[i], v);
                        if (GATE) {
                            const float z = RW::at(zr[i], v);
                            e *= z * sigmoid_f32(z);
                        }
                        es[v] = glr_apply<MARKED>(ps[v], ok ? e : 0.f, es[v]);
                    }
                }
            }
        };
        if (PACKED && __any(seen != 0))
            tokens(std::true_type{});
        else
            tokens(std::false_type{});
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

// Backward.  The states are recomputed: first the map of every block and the
// adjoint it passes on (glr_block_kernel: x, g, dy, z read once, 8 bytes an
// element in bf16), joined over the row by glr_block_scan_kernel, then this
// kernel with the same inputs again and the gradients out (14 bytes).  At 8 x
// 2048 x 5120 with a gate 408 us (136 + 13 + 271 by the profiler), at four
// fifths of the vector unit.
// Taking the rows in groups that stay in the Infinity Cache between the passes
// was slower (468 us in halves, 521 row by row, for 452 at that time): the
// launches' ends cost what the second reading gains.  What gains is to take
// the blocks here in the opposite order, the last ones read first, and to
// store the gradients without displacing the inputs still cached: 437 us
// without either, 432 with the order alone, 420 with the stores alone, 408 with
// both; a convolution, this recurrence and a gated norm with their backward
// passes 959 -> 943 us, at 2 x 2048 290 -> 289, at 1 x 512 91 -> 89.  Such stores
// need whole strips that start on 64 bytes (5118 channels: 554 us with them, 477
// without, 490 before).  The forward passes keep ordinary stores: 151 us for
// 155 alone, but the next kernel then reads y from memory (2 x 2048, the same
// three operators: 107 us for 102).
//
// One workgroup per (row, block of RT tokens, strip), with the state
// entering the block from the left (ws_h) and the adjoint from the right
// (ws_e) already known:
//   G_t = e_t + c_t,  c_{t-1} = p_t G_t,  e = dy [silu(z)]
//   dx = k G     dla = c_{t-1} h_{t-1} + G x dk/dla,  dk/dla = -a^2 / k
//   dg = A dla sigmoid(g + bias)   dA = sum s dla   dbias = sum dg
//   dz = dy h silu'(z)
template <typename IO, typename TL, bool NORM, bool PACKED, bool GATE>
__global__ __launch_bounds__(TL::W * 64, TL::V == 2 && !(sizeof(IO) == 4 && PACKED && GATE) ? 4 : 1) void glr_bwd_kernel(GlrArgs a) {
    constexpr int V = TL::V, T = TL::T, SEG = TL::SEG, CT = TL::CT;
    typedef Raw<IO, V> RW;
    typedef typename RW::type R;
    __shared__ float2 seg_map[SEG][CT];
    __shared__ float seg_e[SEG][CT], seg_h[SEG][CT];
    const GlrUnit u = glr_unit<TL, true>(a, a.nblk);
    const int tid = threadIdx.x, cg = tid % TL::CL, seg = tid / TL::CL, m = seg * T;
    const int D = a.channels, L = a.seqlen;
    const int c = u.ct * CT + cg * V;
    const bool cok = c < D;
    const int cc = cok ? c : D - V, cb = cc * (int)sizeof(IO);
    const int t = u.blk * TL::RT;
    const int64_t row = (int64_t)u.b * L;
    const int64_t ys = (int64_t)D * (int)sizeof(IO);
    const char *gb = (const char *)a.g + (row + t) * a.gs, *xb = (const char *)a.x + (row + t) * a.xs;
    const char *db = (const char *)a.dy + (row + t) * a.dys, *zb = (const char *)a.z + (row + t) * a.zs;
    float dA[V], dbias[V];
    auto block = [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        const bool any = FULL || t + __builtin_amdgcn_readfirstlane(tid / 64) * (TL::TL * T) < L;
        R xr[T], gr[T], zr[T], dr[T];
        if (any) {
            glr_load<FULL>(gr, gb, a.gs, m, cb, L - t);
            glr_load<FULL>(xr, xb, a.xs, m, cb, L - t);
            glr_load<FULL>(dr, db, a.dys, m, cb, L - t);
            if (GATE) glr_load<FULL>(zr, zb, a.zs, m, cb, L - t);
        } else {
#pragma unroll
            for (int i = 0; i < T; ++i) xr[i] = gr[i] = zr[i] = dr[i] = R{};
        }
        const uint32_t cut = PACKED ? glr_wave_resets<TL>(a.seq_idx + row, t + tid / 64 * (TL::TL * T), L) : 0u;
        float A[V], bias[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = a.A[cc + v];
            bias[v] = a.bias ? a.bias[cc + v] : 0.f;
        }
        auto ok = [&](int i) { return FULL || t + m + i < L; };
        // decay, input factor, softplus (base 2) and its derivative, the
        // gate's sigmoid; past the row's end the identity
        float al[T][V], k[T][V], sp[T][V], sg[T][V], sz[T][V];
        if (any) {
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float gv = RW::at(gr[i], v) + bias[v];
                    float e, o;
                    const float s = softplus2(gv, e, o), l = A[v] * s;
                    const float av = __builtin_amdgcn_exp2f(l);
                    al[i][v] = ok(i) ? av : 1.f;
                    k[i][v] = ok(i) ? (NORM ? __builtin_amdgcn_sqrtf(one_minus_square(av, l)) : 1.f) : 0.f;
                    sp[i][v] = ok(i) ? s : 0.f;
                    sg[i][v] = ok(i) ? (gv >= 0.f ? 1.f : e) * __builtin_amdgcn_rcpf(o) : 0.f;
                    if (GATE) sz[i][v] = sigmoid_f32(RW::at(zr[i], v));
                }
        } else {
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    al[i][v] = 1.f;
                    k[i][v] = sp[i][v] = sg[i][v] = sz[i][v] = 0.f;
                }
        }
        auto p_of = [&](int i, int v) { return glr_mark<PACKED>(al[i][v], (cut >> i) & 1); };
        // (a select: past the row's end x repeats the last token's, and 0 times an
        // infinity or a NaN would not be 0)
        auto q_of = [&](int i, int v) { return ok(i) ? k[i][v] * RW::at(xr[i], v) : 0.f; };
        auto e_of = [&](int i, int v) {
            const float d = RW::at(dr[i], v);
            const float e = GATE ? d * (RW::at(zr[i], v) * sz[i][v]) : d;
            return ok(i) ? e : 0.f;
        };
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float ps = 1.f, qs = 0.f, es = 0.f;
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const float p = p_of(i, v);
                qs = glr_apply<PACKED>(p, qs, q_of(i, v));
                ps = glr_join<PACKED>(ps, p);
                es = glr_apply<PACKED>(ps, e_of(i, v), es);
            }
            seg_map[seg][cg * V + v] = make_float2(ps, qs);
            seg_e[seg][cg * V + v] = es;
        }
        __syncthreads();
        // the segments are joined by a thread per channel and direction, which
        // costs a barrier and spares each lane the maps on both its sides; a row
        // of one block starts from init and dfinal
        static_assert(2 * CT <= TL::W * 64, "a thread per channel and direction");
        if (tid < 2 * CT && u.ct * CT + tid % CT < D) {
            const int ch = tid % CT;
            const int64_t at = ((int64_t)u.b * a.nblk + u.blk) * D + u.ct * CT + ch;
            const float *h0 = a.nblk > 1 ? a.ws_h : a.init, *e0 = a.nblk > 1 ? a.ws_e : a.dfinal;
            if (tid < CT) {
                float hv = h0 ? h0[at] : 0.f;
#pragma unroll 4
                for (int s = 0; s < SEG; ++s) {
                    const float2 f = seg_map[s][ch];
                    seg_h[s][ch] = hv;
                    hv = glr_apply<PACKED>(f.x, hv, f.y);
                }
            } else {
                float ev = e0 ? e0[at] : 0.f;
#pragma unroll 4
                for (int s = SEG - 1; s >= 0; --s) {
                    const float p = seg_map[s][ch].x, own = seg_e[s][ch];
                    seg_e[s][ch] = ev;
                    ev = glr_apply<PACKED>(p, ev, own);
                }
                if (a.nblk == 1 && a.dinit) a.dinit[at] = ev;
            }
        }
        __syncthreads();
        float hin[V], cin[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            hin[v] = seg_h[seg][cg * V + v];
            cin[v] = seg_e[seg][cg * V + v];
        }
        float h[T][V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float hv = hin[v];
#pragma unroll
            for (int i = 0; i < T; ++i) {
                hv = glr_apply<PACKED>(p_of(i, v), hv, q_of(i, v));
                h[i][v] = hv;
            }
            dA[v] = dbias[v] = 0.f;
        }
        const __amdgpu_buffer_rsrc_t ox = buffer_of((char *)a.dx + (row + t) * ys);
        const __amdgpu_buffer_rsrc_t og = buffer_of((char *)a.dg + (row + t) * ys);
        const __amdgpu_buffer_rsrc_t oz = buffer_of((char *)a.dz + (row + t) * ys);
        const uint32_t off = (uint32_t)m * (uint32_t)ys + (uint32_t)cb;
        auto grads = [&](auto aux) {
            constexpr int AUX = decltype(aux)::value;
#pragma unroll
            for (int i = T - 1; i >= 0; --i) {
                float dx[V], dg[V], dz[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float G = e_of(i, v) + cin[v];
                    const float x = RW::at(xr[i], v);
                    const bool reset = PACKED && ((cut >> i) & 1);
                    cin[v] = reset ? 0.f : al[i][v] * G;
                    dx[v] = k[i][v] * G;
                    float dla = reset ? 0.f : cin[v] * (i > 0 ? h[i > 0 ? i - 1 : 0][v] : hin[v]);
                    if (NORM) {
                        const float rk = k[i][v] > 0.f ? __builtin_amdgcn_rcpf(k[i][v]) : 0.f;
                        dla = fmaf(-G * x, al[i][v] * al[i][v] * rk, dla);
                    }
                    // (dfinal times a last state that is not finite is no token's)
                    dla = ok(i) ? dla : 0.f;
                    dg[v] = A[v] * dla * sg[i][v];
                    dA[v] = fmaf(sp[i][v], dla, dA[v]);
                    dbias[v] += dg[v];
                    if (GATE) {
                        const float z = RW::at(zr[i], v);
                        dz[v] = RW::at(dr[i], v) * h[i][v] * (sz[i][v] * fmaf(z, 1.f - sz[i][v], 1.f));
                    }
                }
                if (FULL || (cok && ok(i))) {
                    buffer_store<IO, V, AUX>(ox, off, (uint32_t)(i * ys), dx);
                    buffer_store<IO, V, AUX>(og, off, (uint32_t)(i * ys), dg);
                    if (GATE) buffer_store<IO, V, AUX>(oz, off, (uint32_t)(i * ys), dz);
                }
            }
        };
        if (FULL && V == 2 && a.once)
            grads(std::integral_constant<int, V == 2 ? kOnce : kKeep>{});
        else if (any)
            grads(std::integral_constant<int, kKeep>{});
    };
    if ((u.ct + 1) * CT <= D && t + TL::RT <= L)
        block(std::true_type{});
    else
        block(std::false_type{});
    // dA and dbias of the block: the lanes' sums over their tokens, joined in
    // segment order
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) seg_map[seg][cg * V + v] = make_float2(dA[v] * kLn2, dbias[v]);
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
void launch_glr_fwd_docs(GlrArgs a, hipStream_t stream) {
    typedef typename std::conditional<std::is_same<TL, GlrFwdPair>::value, GlrFwdHalf, TL>::type HALF;
    const dim3 block(TL::W * 64);
    if (a.nblk > 1)
        hipLaunchKernelGGL((glr_block_kernel<IO, TL, NORM, PACKED, false, false>), glr_grid<TL>(a, a.nblk - 1), block,
                           0, stream, a, a.nblk - 1);
    const int units = (int)glr_grid<TL>(a, a.nblk).x;
    a.whole = units;
    if (!std::is_same<TL, HALF>::value && units > a.cus && 2 * units <= 3 * a.cus) a.whole = a.cus;
    const dim3 grid((unsigned)(a.whole + 2 * (units - a.whole)));
    if (a.z)
        hipLaunchKernelGGL((glr_fwd_kernel<IO, TL, HALF, NORM, PACKED, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((glr_fwd_kernel<IO, TL, HALF, NORM, PACKED, false>), grid, block, 0, stream, a);
}

template <typename IO, typename TL, bool NORM>
void launch_glr_fwd_tile(const GlrArgs &a, hipStream_t stream) {
    a.seq_idx ? launch_glr_fwd_docs<IO, TL, NORM, true>(a, stream) : launch_glr_fwd_docs<IO, TL, NORM, false>(a, stream);
}

void launch_glr_block_scan(const GlrArgs &a, hipStream_t stream);

template <typename IO, typename TL, bool NORM, bool PACKED, bool GATE>
void launch_glr_bwd_gate(const GlrArgs &a, hipStream_t stream) {
    typedef typename std::conditional<TL::V == 2, GlrBlockPair, GlrBwdSingle>::type BL;
    if (a.nblk > 1) {
        hipLaunchKernelGGL((glr_block_kernel<IO, BL, NORM, PACKED, true, GATE>), glr_grid<BL>(a, a.nblk),
                           dim3(BL::W * 64), 0, stream, a, a.nblk);
        launch_glr_block_scan(a, stream);
    }
    hipLaunchKernelGGL((glr_bwd_kernel<IO, TL, NORM, PACKED, GATE>), glr_grid<TL>(a, a.nblk), dim3(TL::W * 64), 0,
                       stream, a);
}

template <typename IO, typename TL, bool NORM, bool PACKED>
void launch_glr_bwd_docs(const GlrArgs &a, hipStream_t stream) {
    a.z ? launch_glr_bwd_gate<IO, TL, NORM, PACKED, true>(a, stream)
        : launch_glr_bwd_gate<IO, TL, NORM, PACKED, false>(a, stream);
}

template <typename IO, typename TL, bool NORM>
void launch_glr_bwd_tile(const GlrArgs &a, hipStream_t stream) {
    a.seq_idx ? launch_glr_bwd_docs<IO, TL, NORM, true>(a, stream) : launch_glr_bwd_docs<IO, TL, NORM, false>(a, stream);
}

template <typename IO, bool NORM>
void launch_glr_fwd_len(bool pair, const GlrArgs &a, hipStream_t stream) {
    const bool brief = a.seqlen <= kGlrShort;
    if (pair)
        brief ? launch_glr_fwd_tile<IO, GlrFwdPairShort, NORM>(a, stream) : launch_glr_fwd_tile<IO, GlrFwdPair, NORM>(a, stream);
    else
        brief ? launch_glr_fwd_tile<IO, GlrFwdSingleShort, NORM>(a, stream)
              : launch_glr_fwd_tile<IO, GlrFwdSingle, NORM>(a, stream);
}

template <typename IO, bool NORM>
void launch_glr_bwd_len(bool pair, const GlrArgs &a, hipStream_t stream) {
    const bool brief = a.seqlen <= kGlrShort;
    if (pair)
        brief ? launch_glr_bwd_tile<IO, GlrBwdPairShort, NORM>(a, stream) : launch_glr_bwd_tile<IO, GlrBwdPair, NORM>(a, stream);
    else
        brief ? launch_glr_bwd_tile<IO, GlrBwdSingleShort, NORM>(a, stream)
              : launch_glr_bwd_tile<IO, GlrBwdSingle, NORM>(a, stream);
}

#define SSD_GLR_INSTANTIATE(IO)                                                                                     \
    template <>                                                                                                     \
    void launch_glr_fwd_io<IO>(bool pair, const GlrArgs &a, hipStream_t stream) {                                   \
        a.normalize ? launch_glr_fwd_len<IO, true>(pair, a, stream) : launch_glr_fwd_len<IO, false>(pair, a, stream); \
    }                                                                                                               \
    template <>                                                                                                     \
    void launch_glr_bwd_io<IO>(bool pair, const GlrArgs &a, hipStream_t stream) {                                   \
        a.normalize ? launch_glr_bwd_len<IO, true>(pair, a, stream) : launch_glr_bwd_len<IO, false>(pair, a, stream); \
    }

}  // namespace ssd
