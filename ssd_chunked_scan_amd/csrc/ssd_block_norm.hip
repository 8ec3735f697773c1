// The seam between two blocks of a residual stream (ssd.h, ssd_block_norm_*):
//
//   n1 = x rstd1      b = scale post n1 silu(z)      s = alpha residual + b
//   n2 = s rstd2      y = n2 pre                     rstd = 1 / sqrt(mean(.^2) + eps)
//
// and its gradient, with c = scale post and dsn the gradient of s from its other
// uses:
//
//   g = pre dy        ds = rstd2 (g - n2 mean(g n2)) + dsn     dresidual = alpha ds
//   h = ds c silu(z)  dx = rstd1 (h - n1 mean(h n1))           dz = ds c n1 silu'(z)
//   dpre = sum_rows dy n2     m = sum_rows ds silu(z) n1       dpost = scale m
//                                                              dscale = post m
//
// Memory-bound: each input read once and each output written once, a row held
// in registers between its sums (the layout of ssd_norm.hpp).  Two sums of a
// row depend on each other, forward s on x's and backward h on s's; the next row's
// loads are under way meanwhile.  The gradients of the two factors of c are the
// same column sum m, so that two sums a column are carried and not three.
//
// With checkpoints (CKPT) x, z and s are also written as e4m3 with a scale
// per 128 columns, and backward reads those instead: 13 bytes a column
// instead of 16 in bf16, and 3 kept instead of 6.
//
// Measured, 16384 x 2560 bf16 with the gate (a copy reaches 4.8 TB/s): forward 89
// us, 4.7 TB/s, and 121 with checkpoints, 4.5; backward 143, 4.7, and 126 from
// checkpoints, 4.3.  4096 x 12288: 106, 151, 186 and 170.  fp32 5000 x 5001: 107,
// 131, 162 and 154.  Odd bf16 rows, and codes of odd rows backward, go column by
// column: 30000 x 1003 70, 132, 110 and 111 (3.0 to 4.4 TB/s), 5000 x 5001 62, 128,
// 128 and 145 (2.2 to 4.0), and past 8192 columns with up to 83 registers spilled:
// 4096 x 12289 196, 334, 570 and 525, fp32 from checkpoints 457.
#include <algorithm>

#include "ssd_block.hpp"
#include "ssd_norm.hpp"

namespace ssd {

// Sums of N values over a row's threads, in every one of them.  One barrier: the
// caller alternates between two places in LDS, so that a place is written again
// only after a later sum's barrier.
template <bool WAVE, int N>
__device__ inline void row_sums(float (&v)[N], float *lds) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (!WAVE) {
        if (threadIdx.x % 64 == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) lds[threadIdx.x / 64 * N + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
        for (int w = 0; w < (int)blockDim.x / 64; ++w) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += lds[w * N + i];
        }
    }
}

// A row of a tensor through a buffer descriptor that ends with its last column:
// what lies past it is read as 0 and not written, so that no lane needs a
// branch, and a tensor that is not given (bytes 0) reads as 0 throughout.  That
// goes by 4-byte words, and wide accesses need no more alignment than a word: rows
// whose bytes are not a multiple of 16 take them too.
__device__ inline __amdgpu_buffer_rsrc_t row_of(const void *base, int64_t row, int64_t stride, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((char *)const_cast<void *>(base) + row * stride, 0, bytes, 0x00027000);
}

// A row's values as e4m3 with a scale per 128 columns.  WORDS: rows of codes begin
// at 4-byte words; elsewhere stores go by the address, which may be any.
template <int V, int K, bool WORDS>
__device__ inline void store_checkpoint(const BlockArgs &a, uint8_t *codes, float *scales, int64_t row, const float (&val)[K][V],
                                        int tid, int nthr) {
    const int nscale = (a.columns + 127) / 128;
    const __amdgpu_buffer_rsrc_t q = row_of(codes, row, a.columns, a.columns), sc = row_of(scales, row, nscale * 4, nscale * 4);
    constexpr int PER = V == 1 ? 2 : 1, LANES = V == 1 ? 64 : 128 / V;
#pragma unroll
    for (int k = 0; k < K; k += PER) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) m = max(m, abs_bits(val[k + j][v]));
        const float mx = __uint_as_float(max(lanes_max<LANES>(m), kMinMost));
        const float inv = 448.f / mx;
        const int p0 = pack_at<V>(k, tid, nthr);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(mx / 448.f), sc,
                                              tid % LANES == 0 ? (uint32_t)(p0 * V / 128) * 4u : 0xffffffffu, 0, 0);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint32_t at = (uint32_t)(pack_at<V>(k + j, tid, nthr) * V);
            uint8_t code[V];
            store_e4m3<V>(code, val[k + j], inv);
            if constexpr (V == 1) {
                __builtin_amdgcn_raw_buffer_store_b8(code[0], q, at, 0, 0);
            } else if constexpr (WORDS && V == 4) {
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(Pack<uint32_t, 1>, code).v[0], q, at, 0, 0);
            } else if constexpr (WORDS) {
                __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(Words<8>::type, code), q, at, 0, 0);
            } else if ((int)at + V <= a.columns) {
                typedef uint32_t __attribute__((ext_vector_type(V / 4), aligned(1), may_alias)) piece;
                *(piece *)(codes + row * a.columns + at) = __builtin_bit_cast(piece, code);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) __builtin_amdgcn_raw_buffer_store_b8(code[v], q, at + v, 0, 0);
            }
        }
    }
}

// V values of a checkpoint as they wait in registers.
template <int V>
struct Kept {
    uint32_t w[V == 8 ? 2 : 1];
    float scale;
};

template <int V>
__device__ inline Kept<V> load_kept(__amdgpu_buffer_rsrc_t q, __amdgpu_buffer_rsrc_t sc, int p) {
    Kept<V> r;
    const uint32_t at = (uint32_t)(p * V);
    if constexpr (V == 8) {
        const Words<8>::type t = __builtin_amdgcn_raw_buffer_load_b64(q, at, 0, 0);
        r.w[0] = t[0];
        r.w[1] = t[1];
    } else if constexpr (V == 4) {
        r.w[0] = __builtin_amdgcn_raw_buffer_load_b32(q, at, 0, 0);
    } else {
        r.w[0] = __builtin_amdgcn_raw_buffer_load_b8(q, at, 0, 0);
    }
    r.scale = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sc, at / 128u * 4u, 0, 0));
    return r;
}

template <int V>
__device__ inline void kept_values(const Kept<V> &r, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = __builtin_amdgcn_cvt_f32_fp8((int)r.w[0], 0) * r.scale;
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)r.w[i], false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)r.w[i], true);
            f[4 * i] = lo[0] * r.scale;
            f[4 * i + 1] = lo[1] * r.scale;
            f[4 * i + 2] = hi[0] * r.scale;
            f[4 * i + 3] = hi[1] * r.scale;
        }
    }
}

// The weights of a thread's columns: post * scale and pre, 1 where not given.
// With AGAIN they are loaded where they are used and not held for all rows: the
// compiler is kept from seeing that they are the same every time.
template <int V, bool AGAIN>
__device__ inline void block_weights(const BlockArgs &a, int p, float (&w1)[V], float (&w2)[V]) {
    auto load = [&](const float *from, float (&f)[V]) {
        const bool given = from != nullptr;
        const int bytes = given ? a.columns * 4 : 0;
        if constexpr (AGAIN) asm volatile("" : "+s"(from));
        const __amdgpu_buffer_rsrc_t rs = row_of(from, 0, 0, bytes);
        if constexpr (V == 1) {
            const float t = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, p * 4, 0, 0));
            f[0] = given ? t : 1.f;
        } else {
#pragma unroll
            for (int v = 0; v < V; v += 4) {
                const auto t = __builtin_amdgcn_raw_buffer_load_b128(rs, (p * V + v) * 4, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[v + i] = given ? __uint_as_float(t[i]) : 1.f;
            }
        }
    };
    float scale[V];
    load(a.post, w1);
    load(a.scale, scale);
    load(a.pre, w2);
#pragma unroll
    for (int v = 0; v < V; ++v) w1[v] *= scale[v];
}

// CKPT: 1 with checkpoints, 2 with ones whose rows of codes are not whole words.
template <typename IO, int V, bool WAVE, int K, bool GATE, int CKPT>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void block_fwd_kernel(BlockArgs a) {
    typedef Raw<IO, V> RW;
    typedef typename RW::type R;
    constexpr int RPB = WAVE ? 4 : 1;   // rows a workgroup takes at a time
    constexpr int E = (int)sizeof(IO);
    __shared__ float lds[2][16];
    const int tid = WAVE ? threadIdx.x % 64 : threadIdx.x, nthr = WAVE ? 64 : blockDim.x;
    const int bytes = a.columns * E, dense = bytes;
    const float inv_n = 1.f / (float)a.columns;
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + (WAVE ? __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : 0);
    if (row >= a.rows) return;   // (without WAVE a workgroup has a row)
    // Up to 8 columns a thread the weights stay in registers, and so does the
    // next row on its way; more columns leave room for neither, and the next row
    // is loaded as soon as this one's registers are free.
    constexpr bool HOLD = K * V <= 8;
    R xr[K], rr[K], zr[K], xn[HOLD ? K : 1], rn[HOLD ? K : 1], zn[HOLD ? K : 1];
    auto load = [&](int64_t r, R (&x)[K], R (&s)[K], R (&z)[K]) {
        const __amdgpu_buffer_rsrc_t xb = row_of(a.x, r, a.xs, bytes), sb = row_of(a.residual, r, a.rs, bytes);
        const __amdgpu_buffer_rsrc_t zb = row_of(a.z, r, a.zs, bytes);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t at = (uint32_t)(pack_at<V>(k, tid, nthr) * (V * E));
            x[k] = buffer_load<R>(xb, at, 0);
            s[k] = buffer_load<R>(sb, at, 0);
            if (GATE) z[k] = buffer_load<R>(zb, at, 0);
        }
    };
    load(row, xr, rr, zr);
    float w1[HOLD ? K : 1][V], w2[HOLD ? K : 1][V];
    if constexpr (HOLD) {
#pragma unroll
        for (int k = 0; k < K; ++k) block_weights<V, false>(a, pack_at<V>(k, tid, nthr), w1[k], w2[k]);
    }
    for (; row < a.rows; row += step) {
        if constexpr (HOLD) load(min(row + step, a.rows - 1), xn, rn, zn);
        float val[K][V], sum[1] = {0.f};
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                val[k][v] = RW::at(xr[k], v);
                sum[0] = fmaf(val[k][v], val[k][v], sum[0]);
            }
        if constexpr (CKPT != 0)
            store_checkpoint<V, K, CKPT == 1>(a, a.xq, a.xsc, row, val, tid, nthr);
        row_sums<WAVE, 1>(sum, lds[0]);
        const float rstd1 = 1.f / __builtin_sqrtf(fmaf(sum[0], inv_n, a.eps));
        if constexpr (CKPT != 0 && GATE) {
            float z[K][V];
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) z[k][v] = RW::at(zr[k], v);
            store_checkpoint<V, K, CKPT == 1>(a, a.zq, a.zsc, row, z, tid, nthr);
        }
        sum[0] = 0.f;
        const __amdgpu_buffer_rsrc_t ro = row_of(a.residual_out, row, dense, bytes);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = pack_at<V>(k, tid, nthr);
            if constexpr (!HOLD) block_weights<V, true>(a, p, w1[0], w2[0]);
            float st[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float b = val[k][v] * rstd1 * w1[HOLD ? k : 0][v];
                if (GATE) {
                    const float z = RW::at(zr[k], v);
                    b *= z * sigmoid_f32(z);
                }
                // the stream is kept in the io type, and the second norm is of
                // what it holds, which is what backward reads
                st[v] = (float)(IO)fmaf(a.alpha, RW::at(rr[k], v), b);
                val[k][v] = st[v];
                sum[0] = fmaf(st[v], st[v], sum[0]);
            }
            buffer_store<IO, V>(ro, (uint32_t)(p * (V * E)), 0, st);
        }
        if constexpr (CKPT != 0)
            store_checkpoint<V, K, CKPT == 1>(a, a.sq, a.ssc, row, val, tid, nthr);
        if constexpr (!HOLD) load(min(row + step, a.rows - 1), xr, rr, zr);
        row_sums<WAVE, 1>(sum, lds[1]);
        const float rstd2 = 1.f / __builtin_sqrtf(fmaf(sum[0], inv_n, a.eps));
        const __amdgpu_buffer_rsrc_t yb = row_of(a.y, row, dense, bytes);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = pack_at<V>(k, tid, nthr);
            if constexpr (!HOLD) block_weights<V, true>(a, p, w1[0], w2[0]);
#pragma unroll
            for (int v = 0; v < V; ++v) val[k][v] = val[k][v] * rstd2 * w2[HOLD ? k : 0][v];
            buffer_store<IO, V>(yb, (uint32_t)(p * (V * E)), 0, val[k]);
        }
        if constexpr (HOLD) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                xr[k] = xn[k];
                rr[k] = rn[k];
                zr[k] = zn[k];
            }
        }
    }
}

// A thread's column sums: in registers for few columns, else in LDS, each
// thread's own places, 16 bytes side by side.
template <int V, int K, bool REGISTERS>
struct ColumnSums {
    float r[REGISTERS ? K : 1][V];
    float *lds;
    static constexpr int kFloats = REGISTERS ? 1 : 1024 * K * V;

    __device__ inline void clear() {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float zero[V] = {};
            put(k, zero);
        }
    }
    __device__ inline void get(int k, float (&f)[V]) const {
        if constexpr (REGISTERS) {
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = r[k][v];
        } else if constexpr (V == 1) {
            f[0] = lds[k * 1024 + threadIdx.x];
        } else {
#pragma unroll
            for (int v = 0; v < V; v += 4) {
                const f32x4 t = *(const f32x4 *)(lds + ((k * V + v) / 4 * 1024 + threadIdx.x) * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[v + i] = t[i];
            }
        }
    }
    __device__ inline void put(int k, const float (&f)[V]) {
        if constexpr (REGISTERS) {
#pragma unroll
            for (int v = 0; v < V; ++v) r[k][v] = f[v];
        } else if constexpr (V == 1) {
            lds[k * 1024 + threadIdx.x] = f[0];
        } else {
#pragma unroll
            for (int v = 0; v < V; v += 4)
                *(f32x4 *)(lds + ((k * V + v) / 4 * 1024 + threadIdx.x) * 4) = f32x4{f[v], f[v + 1], f[v + 2], f[v + 3]};
        }
    }
};

// Single columns take more registers, for their addresses.
constexpr bool block_bwd_holds(int K, int V) { return K * V <= (V == 1 ? 4 : 8); }

// Backward: a.parts workgroups take the rows in turn and keep their columns'
// two sums; each leaves a row of parts [2][pitch]: m, dpre.
template <typename IO, int V, bool WAVE, int K, bool GATE, bool CKPT>
__global__ __launch_bounds__(WAVE ? 256 : 1024, block_bwd_holds(K, V) ? 4 : 1) void block_bwd_kernel(BlockArgs a) {
    typedef Raw<IO, V> RW;
    typedef typename RW::type R;
    constexpr int RPB = WAVE ? 4 : 1;
    constexpr int E = (int)sizeof(IO);
    __shared__ float lds[2][48];
    __shared__ float red[WAVE ? 4 : 1][WAVE ? 64 * K * V : 1];
    const int tid = WAVE ? threadIdx.x % 64 : threadIdx.x, nthr = WAVE ? 64 : blockDim.x;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int nscale = (a.columns + 127) / 128, bytes = a.columns * E, dense = bytes;
    const float inv_n = 1.f / (float)a.columns;
    constexpr bool HOLD = block_bwd_holds(K, V);   // weights and sums in registers
    float w1[HOLD ? K : 1][V], w2[HOLD ? K : 1][V];
    // Sixteen single columns leave no registers for the next row before this one is done.
    constexpr bool LATE = V == 1 && K > 8;
    typedef ColumnSums<V, K, HOLD> CS;
    __shared__ __attribute__((aligned(16))) float column_sums[2][CS::kFloats];
    CS dm, dp;
    dm.lds = column_sums[0];
    dp.lds = column_sums[1];
    dm.clear();
    dp.clear();
    if constexpr (HOLD) {
#pragma unroll
        for (int k = 0; k < K; ++k) block_weights<V, false>(a, pack_at<V>(k, tid, nthr), w1[k], w2[k]);
    }
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + (WAVE ? wave : 0);
    R yr[K], gr[K], xr[CKPT ? 1 : K], sr[CKPT ? 1 : K], zr[CKPT ? 1 : K];
    Kept<V> xk[CKPT ? K : 1], sk[CKPT ? K : 1], zk[CKPT ? K : 1];
    auto load = [&](int64_t r) {
        const __amdgpu_buffer_rsrc_t yb = row_of(a.dy, r, a.dys, bytes);
        const __amdgpu_buffer_rsrc_t gb = row_of(a.dresidual_out, r, a.drs, a.dresidual_out ? bytes : 0);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t at = (uint32_t)(pack_at<V>(k, tid, nthr) * (V * E));
            yr[k] = buffer_load<R>(yb, at, 0);
            gr[k] = buffer_load<R>(gb, at, 0);
        }
        if constexpr (CKPT) {
            auto kept = [&](Kept<V> (&to)[K], const uint8_t *q, const float *sc) {
                const __amdgpu_buffer_rsrc_t qb = row_of(q, r, a.columns, a.columns);
                const __amdgpu_buffer_rsrc_t cb = row_of(sc, r, nscale * 4, nscale * 4);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    to[k] = load_kept<V>(qb, cb, pack_at<V>(k, tid, nthr));
                    if (V == 1 && k % 2 == 1) to[k].scale = to[k - 1].scale;   // of one block
                }
            };
            kept(xk, a.xq, a.xsc);
            kept(sk, a.sq, a.ssc);
            if (GATE) kept(zk, a.zq, a.zsc);
        } else {
            auto whole = [&](R (&to)[K], const void *p, int64_t stride) {
                const __amdgpu_buffer_rsrc_t pb = row_of(p, r, stride, bytes);
#pragma unroll
                for (int k = 0; k < K; ++k)
                    to[k] = buffer_load<R>(pb, (uint32_t)(pack_at<V>(k, tid, nthr) * (V * E)), 0);
            };
            whole(xr, a.x, a.xs);
            whole(sr, a.residual, a.rs);
            if (GATE) whole(zr, a.z, a.zs);
        }
    };
    auto value = [&](const auto &raw, const auto &kept, int k, float (&f)[V]) {
        if constexpr (CKPT) {
            kept_values<V>(kept[k], f);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = RW::at(raw[k], v);
        }
    };
    if (row < a.rows) load(row);
    for (; row < a.rows; row += step) {
        float sums[3] = {0.f, 0.f, 0.f};   // of x^2, s^2, g s
        float n1[K][V], h[K][V];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (!HOLD) block_weights<V, true>(a, pack_at<V>(k, tid, nthr), w1[0], w2[0]);
            float s[V];
            value(xr, xk, k, n1[k]);
            value(sr, sk, k, s);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                sums[0] = fmaf(n1[k][v], n1[k][v], sums[0]);
                sums[1] = fmaf(s[v], s[v], sums[1]);
                sums[2] = fmaf(w2[HOLD ? k : 0][v] * RW::at(yr[k], v), s[v], sums[2]);
            }
        }
        row_sums<WAVE, 3>(sums, lds[0]);
        const float rstd1 = 1.f / __builtin_sqrtf(fmaf(sums[0], inv_n, a.eps));
        const float rstd2 = 1.f / __builtin_sqrtf(fmaf(sums[1], inv_n, a.eps));
        const float mean2 = sums[2] * rstd2 * inv_n;   // of g n2
        float sum[1] = {0.f};
        const __amdgpu_buffer_rsrc_t rb = row_of(a.dresidual, row, dense, bytes), zb = row_of(a.dz, row, dense, bytes);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = pack_at<V>(k, tid, nthr);
            if constexpr (!HOLD) block_weights<V, true>(a, p, w1[0], w2[0]);
            float s[V], z[V], dr[V], dz[V], m[V], q[V];
            dm.get(k, m);
            dp.get(k, q);
            value(sr, sk, k, s);
            if (GATE) value(zr, zk, k, z);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float c = w1[HOLD ? k : 0][v], w = w2[HOLD ? k : 0][v];
                const float dy = RW::at(yr[k], v), n2 = s[v] * rstd2;
                q[v] = fmaf(dy, n2, q[v]);
                const float ds = fmaf(rstd2, fmaf(-n2, mean2, w * dy), RW::at(gr[k], v));
                dr[v] = a.alpha * ds;
                n1[k][v] *= rstd1;
                float t = ds;
                if (GATE) {
                    const float sig = sigmoid_f32(z[v]);
                    dz[v] = ds * c * n1[k][v] * (sig * fmaf(z[v], 1.f - sig, 1.f));
                    t = ds * (z[v] * sig);
                }
                m[v] = fmaf(t, n1[k][v], m[v]);
                h[k][v] = t * c;
                sum[0] = fmaf(h[k][v], n1[k][v], sum[0]);
            }
            dm.put(k, m);
            dp.put(k, q);
            buffer_store<IO, V>(rb, (uint32_t)(p * (V * E)), 0, dr);
            if (GATE) buffer_store<IO, V>(zb, (uint32_t)(p * (V * E)), 0, dz);
        }
        if constexpr (!LATE) load(min(row + step, a.rows - 1));
        row_sums<WAVE, 1>(sum, lds[1]);
        const float mean1 = sum[0] * inv_n;
        const __amdgpu_buffer_rsrc_t xb = row_of(a.dx, row, dense, bytes);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float dx[V];
#pragma unroll
            for (int v = 0; v < V; ++v) dx[v] = rstd1 * fmaf(-n1[k][v], mean1, h[k][v]);
            buffer_store<IO, V>(xb, (uint32_t)(pack_at<V>(k, tid, nthr) * (V * E)), 0, dx);
        }
        if constexpr (LATE) load(min(row + step, a.rows - 1));
    }
    if (!a.part) return;
    float *out = a.part + (int64_t)blockIdx.x * 2 * a.pitch;
    if constexpr (WAVE) {
        auto join = [&](const float (&d)[K][V], float *to) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) red[wave][pack_at<V>(k, tid, nthr) * V + v] = d[k][v];
            __syncthreads();
            for (int c = threadIdx.x; c < a.columns; c += 256)
                to[c] = ((red[0][c] + red[1][c]) + red[2][c]) + red[3][c];
            __syncthreads();
        };
        join(dm.r, out);
        join(dp.r, out + a.pitch);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = pack_at<V>(k, tid, nthr);
            float m[V], q[V];
            dm.get(k, m);
            dp.get(k, q);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (p * V < a.columns) {
                    out[p * V + v] = m[v];
                    out[a.pitch + p * V + v] = q[v];
                }
        }
    }
}

// Sums the parts in a fixed order: 32 columns of one plane a workgroup, 32
// threads a column over runs of parts, joined in order.
constexpr int kFinish = 32;

__global__ __launch_bounds__(1024) void block_finish_kernel(BlockArgs a) {
    __shared__ float s[kFinish][kFinish + 1];
    const int lane = threadIdx.x % kFinish, run = threadIdx.x / kFinish, n = a.columns;
    const int ncol = (n + kFinish - 1) / kFinish, plane = blockIdx.x / ncol, c = blockIdx.x % ncol * kFinish + lane;
    const int per = (a.parts + kFinish - 1) / kFinish, k0 = min(run * per, a.parts), k1 = min(k0 + per, a.parts);
    const float *p = a.part + (int64_t)plane * a.pitch + min(c, n - 1);
    float acc = 0.f;
#pragma unroll 8
    for (int k = k0; k < k1; ++k) acc += p[(int64_t)k * 2 * a.pitch];
    s[run][lane] = acc;
    __syncthreads();
    if (run == 0 && c < n) {
        for (int r = 1; r < kFinish; ++r) acc += s[r][lane];
        if (plane == 1) {
            if (a.dpre) a.dpre[c] = acc;
        } else {
            if (a.dpost) a.dpost[c] = a.scale ? acc * a.scale[c] : acc;
            if (a.dscale) a.dscale[c] = a.post ? acc * a.post[c] : acc;
        }
    }
}

template <typename IO, int V, bool WAVE, int K>
static void block_fwd_launch(const BlockArgs &a, hipStream_t stream, int nthr) {
    // 28 waves a compute unit, for which bf16 rows in packs of 8 of up to 8192
    // columns have the registers (16384 x 2560 with checkpoints 122 us, 128 with
    // 32, 123 with 24; 8192 x 5120 87 without them, 89 with 32).  Other variants
    // have them for less, 16 to 24 waves: single columns, codes that are not whole
    // words, and most of fp32 and of more than 8192 columns with a gate or
    // checkpoints.  Their last workgroups start when the first ones end.
    const int64_t rows = WAVE ? (a.rows + 3) / 4 : a.rows;
    const int64_t fit = (int64_t)a.cus * std::max(1, 28 / (nthr / 64));
    const dim3 grid((unsigned)std::min(rows, fit));
    const int ckpt = !a.xq ? 0 : V == 1 || a.code_words ? 1 : 2;
#define SSD_BLOCK_FWD(G, C)                                                                                  \
    if (!a.z == !G && ckpt == C)                                                                             \
        hipLaunchKernelGGL((block_fwd_kernel<IO, V, WAVE, K, G, C>), grid, dim3(nthr), 0, stream, a);
    SSD_BLOCK_FWD(false, 0)
    SSD_BLOCK_FWD(false, 1)
    SSD_BLOCK_FWD(true, 0)
    SSD_BLOCK_FWD(true, 1)
    if constexpr (V > 1) {
        SSD_BLOCK_FWD(false, 2)
        SSD_BLOCK_FWD(true, 2)
    }
#undef SSD_BLOCK_FWD
}

template <typename IO, int V, bool WAVE, int K>
static void block_bwd_launch(const BlockArgs &a, hipStream_t stream, int nthr) {
    const dim3 grid((unsigned)a.parts);
#define SSD_BLOCK_BWD(G, C)                                                                                  \
    if (!a.dz == !G && !a.xq == !C)                                                                          \
        hipLaunchKernelGGL((block_bwd_kernel<IO, V, WAVE, K, G, C>), grid, dim3(nthr), 0, stream, a);
    // (whole fp32 rows of more than 4096 columns always go in packs)
    if constexpr (sizeof(IO) == 2 || V > 1 || K <= 4) {
        SSD_BLOCK_BWD(false, false)
        SSD_BLOCK_BWD(true, false)
    }
    SSD_BLOCK_BWD(false, true)
    SSD_BLOCK_BWD(true, true)
#undef SSD_BLOCK_BWD
}

// As the norm's kernels: a wave per row where it can hold KW packs a lane, else a
// workgroup of KB, KM or KX packs a thread, the first with which 1024 threads can
// hold the row.
#define SSD_BLOCK_SHAPE(launch)                                        \
    const int npack = (a.columns + V - 1) / V;                         \
    if (npack <= 64 * KW)                                              \
        launch<IO, V, true, KW>(a, stream, 256);                       \
    else if (npack <= 1024 * KB)                                       \
        launch<IO, V, false, KB>(a, stream, norm_threads(npack, KB));  \
    else if (npack <= 1024 * KM)                                       \
        launch<IO, V, false, KM>(a, stream, norm_threads(npack, KM));  \
    else                                                               \
        launch<IO, V, false, KX>(a, stream, norm_threads(npack, KX));

template <typename IO, int V, int KW, int KB, int KM, int KX>
static void block_fwd_shape(const BlockArgs &a, hipStream_t stream) { SSD_BLOCK_SHAPE(block_fwd_launch) }

template <typename IO, int V, int KW, int KB, int KM, int KX>
static void block_bwd_shape(const BlockArgs &a, hipStream_t stream) { SSD_BLOCK_SHAPE(block_bwd_launch) }

void launch_block_fwd(bool bf16_io, bool wide, const BlockArgs &a, hipStream_t stream) {
    if (bf16_io)
        wide ? block_fwd_shape<bf16, 8, 1, 1, 1, 2>(a, stream) : block_fwd_shape<bf16, 1, 8, 8, 8, 16>(a, stream);
    else   // (fp32 rows are whole words)
        block_fwd_shape<float, 4, 2, 2, 2, 4>(a, stream);
}

void launch_block_bwd(bool bf16_io, bool wide, const BlockArgs &a, hipStream_t stream) {
    if (bf16_io)
        wide ? block_bwd_shape<bf16, 8, 1, 1, 1, 2>(a, stream) : block_bwd_shape<bf16, 1, 4, 4, 8, 16>(a, stream);
    else
        wide ? block_bwd_shape<float, 4, 2, 2, 2, 4>(a, stream) : block_bwd_shape<float, 1, 4, 4, 8, 16>(a, stream);
    if (a.part) hipLaunchKernelGGL(block_finish_kernel, dim3((a.columns + kFinish - 1) / kFinish * 2), dim3(1024), 0, stream, a);
}

}  // namespace ssd
