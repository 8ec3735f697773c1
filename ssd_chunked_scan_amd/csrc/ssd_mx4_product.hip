// Products of 4-bit microscaled operands (ssd.h, ssd_mx4_matmul,
// ssd_mx4_linear): y[t][n] = sum_k a[t][k] w[n][k] + bias[n] on the scaled matrix
// instructions, which multiply 32 columns of e2m1 codes by both blocks' scales
// and sum in fp32.  The weights are the instruction's first operand, so that a
// lane's results are neighbouring columns of one token.
#include "ssd_mx4.hpp"
#include "ssd_tiles.hpp"

namespace ssd {

// ------------------------------------------------------------- few tokens
//
// Up to 16 MT tokens: bound by the weights, 17/32 byte each.  A workgroup owns
// 16 NT outputs and its eight waves take the 128-column blocks in turn; the
// parts are joined through LDS in a fixed order.  16x16x128: lane l brings row l % 16
// and the 32 columns 32 (l / 16) .. of either operand, 16 bytes and a scale byte;
// that is also where a lane can quantise 32 activations by itself, without
// exchanging anything (IN, up to 16 tokens).

constexpr int kFewWaves = 8;

template <typename IN>
struct Mx4Tokens {
    static constexpr bool kQuantised = false;
};
template <>
struct Mx4Tokens<uint8_t> {
    static constexpr bool kQuantised = true;
};

template <typename OUT>
__device__ inline void mx4_store4(const Mx4ProductArgs &a, int64_t t, int n, const float (&v)[4], bool wide) {
    OUT *y = (OUT *)a.y + t * a.n + n;
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = v[i] + (a.bias && n + i < a.n ? a.bias[n + i] : 0.f);
    if (wide) {
        store_pack<OUT, 4>(y, o);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < a.n) y[i] = (OUT)o[i];
    }
}

template <typename IN, typename OUT, int MT, int NT, bool WIDE>
__global__ __launch_bounds__(64 * kFewWaves) void mx4_few_kernel(Mx4ProductArgs a) {
    constexpr bool PRE = Mx4Tokens<IN>::kQuantised;
    __shared__ float red[kFewWaves][NT * MT][64][4];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int r = lane % 16, g = lane / 16;
    const int n0 = blockIdx.x * 16 * NT;
    const int m = (int)a.m;
    f32x4 acc[NT][MT] = {};
    const uint8_t *wp[NT];
    const uint8_t *wsp[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t n = min(n0 + j * 16 + r, a.n - 1);
        wp[j] = a.w + n * a.kblocks * 64 + g * 16;
        wsp[j] = (const uint8_t *)a.ws + n * 4 + g;
    }
    for (int kb = wave; kb < a.kblocks; kb += kFewWaves) {
        i32x4 w[NT], t[MT];
        int ws[NT], ts[MT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            w[j] = *(const i32x4 *)(wp[j] + kb * 64);
            ws[j] = wsp[j][(int64_t)kb * a.n * 4];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int tok = min(i * 16 + r, m - 1);
            if constexpr (PRE) {
                t[i] = *(const i32x4 *)(a.a + ((int64_t)tok * a.kblocks + kb) * 64 + g * 16);
                ts[i] = ((const uint8_t *)a.as)[((int64_t)kb * m + tok) * 4 + g];
            } else {
                const char *row = (const char *)a.x + tok * a.xs;
                Pack<IN, 8> v[4];
                uint32_t most = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = mx4_load8<IN, WIDE>(row, kb * 128 + g * 32 + q * 8, a.columns);
#pragma unroll
                for (int q = 0; q < 4; ++q) most = max(most, mx4_most<IN>(v[q]));
                const uint32_t byte = mx4_scale_byte(most);
                const float scale = mx4_scale(byte);
#pragma unroll
                for (int q = 0; q < 4; ++q) t[i][q] = (int)mx4_codes<IN>(v[q], scale);
                ts[i] = (int)byte;
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx4_operand(w[j]), mx4_operand(t[i]), acc[j][i],
                                                                             4, 4, 0, ws[j], 0, ts[i]);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) *(f32x4 *)red[wave][j * MT + i][lane] = acc[j][i];
    __syncthreads();
    for (int e = threadIdx.x; e < NT * MT * 64; e += 64 * kFewWaves) {
        const int tile = e / 64, l = e % 64;
        f32x4 s = *(const f32x4 *)red[0][tile][l];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) s += *(const f32x4 *)red[w][tile][l];
        const int t = tile % MT * 16 + l % 16, n = n0 + tile / MT * 16 + l / 16 * 4;
        const float o[4] = {s[0], s[1], s[2], s[3]};
        if (t < m && n < a.n)
            mx4_store4<OUT>(a, t, n, o, a.n % 4 == 0 && (uintptr_t)a.y % (4 * sizeof(OUT)) == 0);
    }
}

// ------------------------------------------------------------- many tokens
//
// A workgroup of four waves owns BM tokens x BN outputs and walks the columns
// 128 at a time: the codes and scales of three such steps are in LDS, loaded
// there directly, two steps ahead.  32x32x64: lane l brings row l % 32 and one
// block of 32 columns of either operand; which block goes into which of a step's two
// instructions is free as long as both operands agree, so lanes 32 .. 63 take
// blocks 2 and 3 and a lane's operands are 32 consecutive bytes and two
// neighbouring scale bytes.  Rows of 64 bytes hold their 16-byte pieces at
// piece ^ (row / 2 % 4), so that eight consecutive rows at one piece meet eight
// different bank groups.

template <int BM, int BN>
struct Mx4Stage {
    static constexpr int kCodes = (BM + BN) * 64;          // tokens, then weights
    static constexpr int kScales = (BM + BN) * 4;
    static constexpr int kBytes = kCodes + kScales;
    static constexpr int kCodeLoads = (BM + BN) / 16 / 4;  // 1 KB each, of each wave
    static constexpr int kScaleParts = (BM + BN) / 64;     // 64 words each
    static constexpr int kScaleLoads = (kScaleParts + 3) / 4;
    static constexpr int kLoads = kCodeLoads + kScaleLoads;
};

template <typename OUT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(256, 2) void mx4_tile_kernel(Mx4ProductArgs a, int tiles_m, int tiles_n, int group) {
    typedef Mx4Stage<BM, BN> ST;
    constexpr int TM = WM / 32, TN = WN / 32;
    static_assert((BM / WM) * (BN / WN) == 4, "four waves");
    constexpr int kEpilogue = 4 * 32 * (WN * (int)sizeof(OUT) + 16);
    constexpr int kLds = 3 * ST::kBytes > kEpilogue ? 3 * ST::kBytes : kEpilogue;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = wave % (BM / WM), wn = wave / (BM / WM);
    // `group` rows of tiles at a time, column by column
    int tm, tn;
    {
        const int id = xcd_contiguous(blockIdx.x, gridDim.x);
        const int per = group * tiles_n, first = id / per * group;
        const int rows = min(group, tiles_m - first), in = id % per;
        tm = first + in % rows;
        tn = in / rows;
    }
    const int64_t m0 = (int64_t)tm * BM;
    const int n0 = tn * BN;
    const int mleft = (int)min((int64_t)BM, a.m - m0), nleft = min(BN, a.n - n0);
    const int pitch = a.kblocks * 64;
    const uint8_t *ab = a.a + m0 * pitch, *wb = a.w + (int64_t)n0 * pitch;
    const uint32_t *asb = a.as + m0, *wsb = a.ws + n0;
    // each load's place in its operand: rows past the last repeat it
    uint32_t code_off[ST::kCodeLoads];
    uint32_t scale_off[ST::kScaleLoads];
#pragma unroll
    for (int i = 0; i < ST::kCodeLoads; ++i) {
        const int blk = i * 4 + wave;   // 16 rows
        const bool tok = blk < BM / 16;
        const int row = (tok ? blk : blk - BM / 16) * 16 + lane / 4;
        const int piece = (lane % 4) ^ (row / 2 % 4);
        code_off[i] = (uint32_t)min(row, (tok ? mleft : nleft) - 1) * (uint32_t)pitch + piece * 16;
    }
#pragma unroll
    for (int i = 0; i < ST::kScaleLoads; ++i) {
        const int part = (i * 4 + wave) % ST::kScaleParts;   // the surplus repeats earlier parts
        const bool tok = part < BM / 64;
        const int row = (tok ? part : part - BM / 64) * 64 + lane;
        scale_off[i] = (uint32_t)min(row, (tok ? mleft : nleft) - 1) * 4u;
    }
    auto issue = [&](int kb, int buf) {
        uint8_t *to = lds + buf * ST::kBytes;
#pragma unroll
        for (int i = 0; i < ST::kCodeLoads; ++i) {
            const int blk = i * 4 + wave;
            const uint8_t *from = (blk < BM / 16 ? ab : wb) + kb * 64;
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(from + code_off[i]),
                                             (__attribute__((address_space(3))) void *)(to + blk * 1024), 16, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < ST::kScaleLoads; ++i) {
            const int part = (i * 4 + wave) % ST::kScaleParts;
            const uint8_t *from = part < BM / 64 ? (const uint8_t *)(asb + (int64_t)kb * a.m)
                                                 : (const uint8_t *)(wsb + (int64_t)kb * a.n);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(from + scale_off[i]),
                                             (__attribute__((address_space(3))) void *)(to + ST::kCodes + part * 256), 4, 0, 0);
        }
    };
    const int r = lane % 32, g = lane / 32;
    // where the lane's operands lie in a step's LDS
    uint32_t tok_at[2], wgt_at[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int piece = (2 * g + s) ^ (r / 2 % 4);
        tok_at[s] = (wm * WM + r) * 64 + piece * 16;
        wgt_at[s] = (BM + wn * WN + r) * 64 + piece * 16;
    }
    const uint32_t tok_scale = ST::kCodes + (wm * WM + r) * 4, wgt_scale = ST::kCodes + (BM + wn * WN + r) * 4;
    // the sums start at the bias: a lane holds outputs 32 j + 8 q + 4 g + e
    f32x16 acc[TN][TM] = {};
    const int nb = n0 + wn * WN;
    if (a.bias) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float b = a.bias[min(nb + 32 * j + 8 * (e / 4) + 4 * g + e % 4, a.n - 1)];
#pragma unroll
                for (int i = 0; i < TM; ++i) acc[j][i][e] = b;
            }
    }
    auto compute = [&](int buf) {
        const uint8_t *at = lds + buf * ST::kBytes;
        int ts[TM], wsc[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) ts[i] = (int)(*(const uint32_t *)(at + tok_scale + i * 128) >> (16 * g));
#pragma unroll
        for (int j = 0; j < TN; ++j) wsc[j] = (int)(*(const uint32_t *)(at + wgt_scale + j * 128) >> (16 * g));
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            i32x4 t[TM], w[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) w[j] = *(const i32x4 *)(at + wgt_at[s] + j * 2048);
#pragma unroll
            for (int i = 0; i < TM; ++i) t[i] = *(const i32x4 *)(at + tok_at[s] + i * 2048);
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    if (s == 0)
                        acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx4_operand(w[j]), mx4_operand(t[i]),
                                                                                    acc[j][i], 4, 4, 0, wsc[j], 0, ts[i]);
                    else
                        acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx4_operand(w[j]), mx4_operand(t[i]),
                                                                                    acc[j][i], 4, 4, 1, wsc[j], 1, ts[i]);
                }
        }
    };
    const int last = a.kblocks - 1;
    issue(0, 0);
    issue(min(1, last), 1);
    vmem_lds_sync_lookahead<ST::kLoads, 0>();
    int buf = 0, ahead = 2;
    for (int kb = 0; kb <= last; ++kb) {
        issue(min(kb + 2, last), ahead);   // (past the end: the last step again, into a buffer nothing reads)
        compute(buf);
        vmem_lds_sync_lookahead<ST::kLoads, 1>();
        buf = buf == 2 ? 0 : buf + 1;
        ahead = ahead == 2 ? 0 : ahead + 1;
    }
    vmem_lds_sync();
    // 32 tokens at a time through the wave's own part of LDS, so that a row of
    // the wave's WN outputs is stored in one piece.
    constexpr int kRow = WN * (int)sizeof(OUT) + 16;
    uint8_t *mine = lds + wave * 32 * kRow;
    constexpr int V = 16 / (int)sizeof(OUT), PER = WN / V;   // 16-byte pieces of a row
    const bool wide = a.n % V == 0 && (uintptr_t)a.y % 16 == 0;
    const int col = lane % PER * V;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float o[4] = {acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]};
                store_pack<OUT, 4>(mine + r * kRow + (32 * j + 8 * q + 4 * g) * (int)sizeof(OUT), o);
            }
        lds_sync();
#pragma unroll
        for (int p = 0; p < 32 * PER / 64; ++p) {
            const int row = p * (64 / PER) + lane / PER;
            const int64_t t = m0 + wm * WM + i * 32 + row;
            const Pack<OUT, V> v = *(const Pack<OUT, V> *)(mine + row * kRow + col * (int)sizeof(OUT));
            if (t < a.m) {
                OUT *y = (OUT *)a.y + t * a.n + nb + col;
                if (wide && nb + col + V <= a.n) {
                    *(Pack<OUT, V> *)y = v;
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (nb + col + e < a.n) y[e] = v.v[e];
                }
            }
        }
        lds_sync();
    }
}

// ---------------------------------------------------------------- launches

template <typename IN, typename OUT, int MT, bool WIDE>
static void mx4_few_launch(const Mx4ProductArgs &a, hipStream_t stream) {
    // Two tiles of 16 outputs share a workgroup's activations where that still
    // gives every compute unit one.
    if ((a.n + 31) / 32 >= a.cus)
        hipLaunchKernelGGL((mx4_few_kernel<IN, OUT, MT, 2, WIDE>), dim3((a.n + 31) / 32), dim3(64 * kFewWaves), 0, stream, a);
    else
        hipLaunchKernelGGL((mx4_few_kernel<IN, OUT, MT, 1, WIDE>), dim3((a.n + 15) / 16), dim3(64 * kFewWaves), 0, stream, a);
}

template <typename OUT>
static void mx4_few_out(bool wide, const Mx4ProductArgs &a, hipStream_t stream) {
    if (a.x) {
        wide ? mx4_few_launch<OUT, OUT, 1, true>(a, stream) : mx4_few_launch<OUT, OUT, 1, false>(a, stream);
    } else {
        switch ((a.m + 15) / 16) {
        case 1: mx4_few_launch<uint8_t, OUT, 1, true>(a, stream); break;
        case 2: mx4_few_launch<uint8_t, OUT, 2, true>(a, stream); break;
        default: mx4_few_launch<uint8_t, OUT, 4, true>(a, stream);
        }
    }
}

template <typename OUT, int BM, int BN, int WM, int WN>
static void mx4_tile_launch(const Mx4ProductArgs &a, hipStream_t stream) {
    const int tm = (int)((a.m + BM - 1) / BM), tn = (a.n + BN - 1) / BN;
    hipLaunchKernelGGL((mx4_tile_kernel<OUT, BM, BN, WM, WN>), dim3((unsigned)((int64_t)tm * tn)), dim3(256), 0, stream, a, tm,
                       tn, 8);
}

template <typename OUT>
static void mx4_tile_out(const Mx4ProductArgs &a, hipStream_t stream) {
    const auto tiles = [&](int bm, int bn) { return ((a.m + bm - 1) / bm) * ((a.n + bn - 1) / bn); };
    if (tiles(256, 128) >= 2 * (int64_t)a.cus)
        mx4_tile_launch<OUT, 256, 128, 128, 64>(a, stream);
    else if (tiles(128, 128) >= 2 * (int64_t)a.cus)
        mx4_tile_launch<OUT, 128, 128, 64, 64>(a, stream);
    else
        mx4_tile_launch<OUT, 64, 64, 32, 32>(a, stream);
}

void launch_mx4_product(bool bf16_out, bool wide, bool few, const Mx4ProductArgs &a, hipStream_t stream) {
    if (few)
        bf16_out ? mx4_few_out<bf16>(wide, a, stream) : mx4_few_out<float>(wide, a, stream);
    else
        bf16_out ? mx4_tile_out<bf16>(a, stream) : mx4_tile_out<float>(a, stream);
}

}  // namespace ssd
