// Products of 4-bit microscaled operands (ssd.h, ssd_mx4_matmul,
// ssd_mx4_linear): y[t][n] = sum_k a[t][k] w[n][k] + bias[n] on the scaled matrix
// instructions, which multiply 32 columns of e2m1 codes by both blocks' scales
// and sum in fp32.  The weights are the instruction's first operand, so that a
// lane's results are neighbouring columns of one token.
#include <algorithm>
#include <type_traits>

#include "ssd_mx4.hpp"
#include "ssd_tiles.hpp"

namespace ssd {

// LDS accesses of any type.
typedef i32x4 __attribute__((may_alias)) any_i32x4;
typedef uint32_t __attribute__((may_alias)) any_u32;

// Between a wave's LDS writes and its lanes' reads of one another's: the hardware
// keeps a wave's LDS accesses in order, the compiler is told to.
__device__ inline void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// ------------------------------------------------------------- few tokens
//
// Up to 16 MT tokens: bound by the weights, 17/32 byte each.  A workgroup owns
// 16 NT outputs and its W waves take the 128-column blocks in turn; the parts are
// joined through LDS in a fixed order.  16x16x128: lane l brings row l % 16 and the
// 32 columns 32 (l / 16) .. of either operand, 16 bytes and a scale byte.
// Activations that are not in 4 bits yet (IN, up to 16 tokens) are quantised while
// the weights come, so they are loaded first (loads complete in order): 16
// lanes take 128 columns of a row, as ssd_mx4_quant's do, and the wave's codes
// change lanes through LDS (a lane that quantised the 32 columns it brings
// would read 64 separate pieces a load: 8 x 2560 x 5120 8.2 us, 16 x 2560 x 8192
// fp32 20.4).

template <typename OUT>
__device__ inline void mx4_store4(const Mx4ProductArgs &a, int64_t t, int n, const float (&v)[4]) {
    OUT *y = (OUT *)a.y + t * a.n + n;
    Pack<OUT, 4> o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = (OUT)(v[i] + (a.bias && n + i < a.n ? a.bias[n + i] : 0.f));
    if (n + 4 <= a.n) {
        typedef uint32_t __attribute__((ext_vector_type(sizeof(OUT)), aligned(sizeof(OUT)), may_alias)) four;
        *(four *)y = __builtin_bit_cast(four, o);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < a.n) y[i] = o.v[i];
    }
}

template <typename IN, typename OUT, int MT, int NT, int W>
__global__ __launch_bounds__(64 * W) void mx4_few_kernel(Mx4ProductArgs a) {
    constexpr bool PRE = std::is_same_v<IN, uint8_t>;   // the activations come in 4 bits
    static_assert(PRE || MT == 1, "quantised on the way: up to 16 tokens");
    typedef std::conditional_t<PRE, float, IN> X;
    __shared__ float red[W][NT * MT][64][4];
    __shared__ __attribute__((aligned(16))) uint8_t codes[PRE ? 1 : W][1024 + 64];   // 16 rows, then their scale bytes
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
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
    for (int kb = wave; kb < a.kblocks; kb += W) {
        i32x4 w[NT], t[MT];
        int ws[NT], ts[MT];
        Pack<X, 8> v[PRE ? 1 : 4];
        if constexpr (PRE) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int tok = min(i * 16 + r, m - 1);
                t[i] = *(const i32x4 *)(a.a + ((int64_t)tok * a.kblocks + kb) * 64 + g * 16);
                ts[i] = ((const uint8_t *)a.as)[((int64_t)kb * m + tok) * 4 + g];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * i < m)
                    v[i] = mx4_load8<X>((const char *)a.x + min(4 * i + g, m - 1) * a.xs, kb * 128 + r * 8, a.columns);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            w[j] = *(const i32x4 *)(wp[j] + kb * 64);
            ws[j] = wsp[j][(int64_t)kb * a.n * 4];
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!PRE) {
            uint8_t *mine = codes[wave];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * i < m) {
                    const uint32_t byte = mx4_scale_byte(quad_max(mx4_most<X>(v[i])));
                    *(any_u32 *)(mine + (4 * i + g) * 64 + r * 4) = byte == 255u ? 0u : mx4_codes<X>(v[i], mx4_scale(byte));
                    if (r % 4 == 0) mine[1024 + (4 * i + g) * 4 + r / 4] = (uint8_t)byte;
                }
            wave_lds_fence();
            const int tok = min(r, m - 1);
            t[0] = *(const any_i32x4 *)(mine + tok * 64 + g * 16);
            ts[0] = mine[1024 + tok * 4 + g];
            wave_lds_fence();
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx4_operand(w[j]), mx4_operand(t[i]), acc[j][i], 4,
                                                                             4, 0, ws[j], 0, ts[i]);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) *(f32x4 *)red[wave][j * MT + i][lane] = acc[j][i];
    __syncthreads();
    for (int e = threadIdx.x; e < NT * MT * 64; e += 64 * W) {
        const int tile = e / 64, l = e % 64;
        f32x4 s = *(const f32x4 *)red[0][tile][l];
#pragma unroll
        for (int w = 1; w < W; ++w) s += *(const f32x4 *)red[w][tile][l];
        const int t = tile % MT * 16 + l % 16, n = n0 + tile / MT * 16 + l / 16 * 4;
        const float o[4] = {s[0], s[1], s[2], s[3]};
        if (t < m && n < a.n) mx4_store4<OUT>(a, t, n, o);
    }
}

// ------------------------------------------------------------- many tokens
//
// 32x32x64: lane l brings row l % 32 and one block of 32 columns of either
// operand; which block goes into which instruction is free as long as both
// operands agree.  Operands go through LDS, loaded there directly, in rows of
// SEG bytes whose 16-byte pieces lie at piece ^ (row / (16 / pieces) % pieces):
// 16 consecutive rows at one piece meet 16 different bank groups.

template <typename OUT>
__device__ inline void put4(uint8_t *to, const float (&f)[4]) {
    if constexpr (sizeof(OUT) == 4) {
        *(any_i32x4 *)to = i32x4{__float_as_int(f[0]), __float_as_int(f[1]), __float_as_int(f[2]), __float_as_int(f[3])};
    } else {
        typedef uint32_t any_u32x2 __attribute__((ext_vector_type(2), may_alias));
        typedef float f4 __attribute__((ext_vector_type(4)));
        *(any_u32x2 *)to = __builtin_bit_cast(any_u32x2, __builtin_convertvector(f4{f[0], f[1], f[2], f[3]}, bf16x4));
    }
}

// Rows of y from an output on.
struct Mx4Rows {
    __amdgpu_buffer_rsrc_t rs;   // ends with the last row
    uint8_t *base;
    int rows;
};

// A 16-byte piece `at` bytes on in a row of y, `left` outputs before the row's end;
// a lane past the last row or output stores nothing (its offset is outside the
// descriptor).  Pieces of fp32 are aligned to 4 bytes at least, which is all that
// a buffer's store asks for; those of bf16 that are not (WIDE) go by the address,
// which may be any (4096 x 2561 x 2560 bf16: 28 us, output by output 47.5).
template <typename OUT, bool WIDE>
__device__ inline void store_piece(const Mx4Rows &y, int row, uint32_t at, int left, i32x4 v) {
    constexpr int V = 16 / (int)sizeof(OUT);
    if constexpr (WIDE) {
        __builtin_amdgcn_raw_buffer_store_b128(v, y.rs, left > 0 ? at : 0xffffffffu, 0, 0);
        return;
    }
    if constexpr (sizeof(OUT) == 4) {
        __builtin_amdgcn_raw_buffer_store_b128(v, y.rs, left >= V ? at : 0xffffffffu, 0, 0);
    } else if (left >= V && row < y.rows) {
        *(mx4_piece<OUT> *)(y.base + at) = __builtin_bit_cast(mx4_piece<OUT>, v);
    }
    if (left > 0 && left < V) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const uint32_t ok = left > e ? at + e * (uint32_t)sizeof(OUT) : 0xffffffffu;
            if constexpr (sizeof(OUT) == 4) __builtin_amdgcn_raw_buffer_store_b32(v[e], y.rs, ok, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)((uint32_t)v[e / 2] >> (16 * (e % 2))), y.rs, ok, 0, 0);
        }
    }
}

// A descriptor whose bound is used: rows past an operand's last are read as 0.
__device__ inline __amdgpu_buffer_rsrc_t bounded(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 0x00027000);
}

// A wave's sums of a 32 x 32 tile: lane l holds token l % 32 and outputs
// 8 q + 4 (l / 32) + e.  On their way out they are put into LDS in chunks of 32
// tokens x 64 bytes (all of the tile's outputs in bf16, a half in fp32), 16-byte
// pieces at piece ^ (token / 4 % 4), and read back in whole rows.
constexpr int kChunk = 2048;

template <typename OUT, bool WIDE>
struct Mx4Chunk {
    static constexpr int kGroups = sizeof(OUT) == 2 ? 4 : 2;   // of 8 outputs
    static constexpr int kPerTile = 4 / kGroups;
    static constexpr int V = 16 / (int)sizeof(OUT);            // outputs of a piece

    static __device__ inline void put(uint8_t *to, const f32x16 &s, int part) {
        const int r = threadIdx.x % 32, g = threadIdx.x / 32 % 2;
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
            const int e = 4 * (part * kGroups + q), byte = (8 * q + 4 * g) * (int)sizeof(OUT);
            put4<OUT>(to + r * 64 + ((byte / 16) ^ (r / 4 % 4)) * 16 + byte % 16, {s[e], s[e + 1], s[e + 2], s[e + 3]});
        }
    }

    // To y's rows from ys on; `row` the chunk's first one, n0 its tile's first
    // output and `left` what is left of the row from there.
    static __device__ inline void get(const uint8_t *from, const Mx4Rows &y, int pitch, int row, int n0, int left,
                                      int part) {
        const int lane = threadIdx.x % 64;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int t = p * 16 + lane / 4, n = part * kGroups * 8 + lane % 4 * V;
            const i32x4 v = *(const any_i32x4 *)(from + t * 64 + ((lane % 4) ^ (t / 4 % 4)) * 16);
            const uint32_t at = ((uint32_t)(row + t) * (uint32_t)pitch + (uint32_t)(n0 + n)) * (uint32_t)sizeof(OUT);
            store_piece<OUT, WIDE>(y, row + t, at, left - n, v);
        }
    }
};

// y's rows from t0 on, `rows` of them (none if negative), from output n0 on.
template <typename OUT>
__device__ inline Mx4Rows rows_of_y(const Mx4ProductArgs &a, int64_t t0, int rows, int n0) {
    OUT *base = (OUT *)a.y + t0 * a.n + n0;
    return {bounded(base, rows > 0 ? ((uint32_t)rows * (uint32_t)a.n - (uint32_t)n0) * (uint32_t)sizeof(OUT) : 0u),
            (uint8_t *)base, rows};
}

// Problems of few tiles, whose time is the latency of their loads: a workgroup of
// four waves owns 64 tokens x 64 outputs, and kRing - 1 stages of 256 columns
// are on their way while one is multiplied (512 x 1024 x 1536: 4.2 us, 5.4 with
// one on its way; 128 x 2560 x 5120: 8.0 and 10.4).  An empty kernel takes 1.6.
constexpr int kRing = 4;

// vmem_lds_sync_lookahead in a loop around a ring of tiles: the KEEP newest
// operations are the direct-to-LDS loads of several later tiles, issued in earlier
// rounds of the loop or before it.  The build check follows every path back
// from the wait.
template <int KEEP>
__device__ inline void vmem_lds_sync_ring() {
    static_assert(KEEP > 0 && KEEP < 64, "vmcnt range");
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    asm volatile("; ssd ring wait" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(KEEP));
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

template <typename OUT, bool WIDE>
__global__ __launch_bounds__(256) void mx4_ring_kernel(Mx4ProductArgs a, int tiles_n) {
    constexpr int ROWS = 128, CODES = ROWS * 128, STAGE = CODES + ROWS * 8, LOADS = 5;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing * STAGE];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int id = xcd_contiguous(blockIdx.x, gridDim.x);
    const int64_t m0 = (int64_t)(id / tiles_n) * 64;
    const int n0 = id % tiles_n * 64, pitch = a.kblocks * 64, last = (a.kblocks - 1) / 2;
    const int mleft = (int)min((int64_t)64, a.m - m0), nleft = min(64, a.n - n0);
    const __amdgpu_buffer_rsrc_t as = bounded(a.a + m0 * pitch, (uint32_t)mleft * (uint32_t)pitch);
    const __amdgpu_buffer_rsrc_t ws = bounded(a.w + (int64_t)n0 * pitch, (uint32_t)nleft * (uint32_t)pitch);
    const int lrow = wave * 8 + lane / 8;
    const uint32_t code_at = (uint32_t)lrow * (uint32_t)pitch + ((lane % 8) ^ (lrow / 2 % 8)) * 16;
    // 8 rows of codes four times, 64 words of scales once.  The second half of
    // an odd last stage brings other codes and scale bytes of 0: products below
    // 2^-240, which fp32 sums round away.
    const bool tok = wave % 2 == 0;
    const uint32_t *scales = tok ? a.as + m0 : a.ws + n0;
    const int64_t scale_pitch = tok ? a.m : a.n;
    const uint32_t scale_bytes = (uint32_t)(tok ? mleft : nleft) * 4u;
    auto load = [&](int st, int buf) {
        uint8_t *to = lds + buf * STAGE;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                i < 2 ? as : ws, (__attribute__((address_space(3))) void *)(to + (i * 4 + wave) * 1024), 16,
                code_at + (uint32_t)(i % 2 * 32 * pitch + st * 128), 0, 0, 0);
        const int kb = 2 * st + wave / 2;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(bounded(scales + kb * scale_pitch, kb < a.kblocks ? scale_bytes : 0u),
                                                 (__attribute__((address_space(3))) void *)(to + CODES + wave * 256), 4,
                                                 lane * 4, 0, 0, 0);
    };
    const int wm = wave % 2, wn = wave / 2, r = lane % 32, g = lane / 32;
    f32x16 acc = {};
    if (a.bias) {
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = a.bias[min(n0 + 32 * wn + 8 * (e / 4) + 4 * g + e % 4, a.n - 1)];
    }
    // (past the end: the last stage again, which nothing reads)
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) load(min(i, last), i);
    for (int st = 0, buf = 0; st <= last; ++st) {
        vmem_lds_sync_ring<(kRing - 2) * LOADS>();
        load(min(st + kRing - 1, last), buf == 0 ? kRing - 1 : buf - 1);
        const uint8_t *at = lds + buf * STAGE;
        // scales: [block][tokens, weights]
        const int ts = *(const int *)(at + CODES + g * 512 + (wm * 32 + r) * 4);
        const int wsc = *(const int *)(at + CODES + g * 512 + 256 + (wn * 32 + r) * 4);
        i32x4 t[4], w[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int piece = ((4 * g + s) ^ (r / 2 % 8)) * 16;
            t[s] = *(const i32x4 *)(at + (wm * 32 + r) * 128 + piece);
            w[s] = *(const i32x4 *)(at + (64 + wn * 32 + r) * 128 + piece);
        }
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx4_operand(w[0]), mx4_operand(t[0]), acc, 4, 4, 0, wsc, 0, ts);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx4_operand(w[1]), mx4_operand(t[1]), acc, 4, 4, 1, wsc, 1, ts);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx4_operand(w[2]), mx4_operand(t[2]), acc, 4, 4, 2, wsc, 2, ts);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx4_operand(w[3]), mx4_operand(t[3]), acc, 4, 4, 3, wsc, 3, ts);
        buf = buf == kRing - 1 ? 0 : buf + 1;
    }
    vmem_lds_sync();
    typedef Mx4Chunk<OUT, WIDE> CH;
    uint8_t *mine = lds + wave * kChunk;
    const Mx4Rows ys = rows_of_y<OUT>(a, m0, mleft, n0);
#pragma unroll
    for (int part = 0; part < CH::kPerTile; ++part) {
        CH::put(mine, acc, part);
        wave_lds_fence();
        CH::get(mine, ys, a.n, wm * 32, wn * 32, nleft - wn * 32, part);
    }
}

// Problems of many tiles: a workgroup owns BM tokens x BN outputs at a time and walks
// them 256 columns a stage, then goes on to its next tile without a pause: one
// stage is in LDS, the next one on its way.  What shapes it, measured for 16384 x
// 10576 x 2560 (a 16384^3 bf16 product of the library reaches 1.6 PFLOP/s here):
//  - The matrix units draw so much power on random operands that they alone
//    reach 6.5 PFLOP/s (136 us), 8.9 on constant ones.
//  - L2 is read in lines of 128 bytes: rows of 64 bytes a stage take 137 us to
//    bring 256 x 256 tiles into LDS, rows of 128 bytes 87 us; 128 x 128 tiles 145.
//  - A wave that waits to issue a load issues no matrix instruction, and what
//    the compiler moves across a barrier overlaps nothing.  So one matrix
//    instruction, one operand read and at most a few loads follow each other
//    in the order written (299 us without that, 189 with, no result stored).
//  - Loads and stores of a wave complete in order, and all tiles end at about the
//    same time: waves that store must not load.  The first half of the waves
//    loads every stage, the other half stores every result, its partner's
//    chunk by chunk through LDS (293 us before, 262 after).
//  - `group` rows of tiles column by column, four of them: neighbouring pieces
//    of y's rows meet in one XCD's L2 (230 us with four, 237 with eight, 233 with
//    two, 250 with one; 8192 x 8192 x 8192 221, 223, 225, 235; 16384 x 2560 x 5120
//    98 to 99 with any).  Each such group begins at another column: y's rows below
//    each other lie a multiple of large powers of two apart, and side by side the
//    XCDs would write to few of the memory's channels.  That is seen behind the
//    quantisation of x (252 us before, 247 after; 8192 rows 131 and 125; 8192 x 8192
//    x 8192 263 and 255), not in the product alone.
// The stage of an odd last 128 columns is the last 256 once more with the scales
// of the first half, which has been taken, at 2^-127: a product below 2^-240 in
// place of each, which fp32 sums round away.
template <int BM, int BN>
struct Mx4Stage {
    static constexpr int kRows = BM + BN;
    static constexpr int kCodes = kRows * 128;
    static constexpr int kBytes = kCodes + kRows * 8;   // codes, then two words of scales a row, block by block
};

struct Mx4Tile {
    const uint8_t *a, *w;
    const uint32_t *as, *ws;
    int m, n;      // rows of either operand, at most BM and BN
    int64_t m0;
    int n0;
};

template <typename OUT, int BM, int BN, int WM, int WN, int PERCU, bool WIDE>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN), PERCU * (BM / WM) * (BN / WN) / 4)
void mx4_tile_kernel(Mx4ProductArgs a, int tiles_m, int tiles_n, int group) {
    typedef Mx4Stage<BM, BN> ST;
    typedef Mx4Chunk<OUT, WIDE> CH;
    constexpr int W = (BM / WM) * (BN / WN), LW = W / 2;   // waves, and those of them that load
    constexpr int TM = WM / 32, TN = WN / 32, N = TN * TM, READS = TN + TM;
    constexpr int LA = BM / 8 / LW, LB = BN / 8 / LW, PARTS = ST::kRows / 64, LS = 2 * PARTS / LW, LOADS = LA + LB + LS;
    static_assert(LA * 8 * LW == BM && LB * 8 * LW == BN && LS * LW == 2 * PARTS, "whole loads");
    // Loads after the barrier that frees their buffer, and before the next one
    // that waits for them; reads and loads after each matrix instruction.
    constexpr int RP = (READS + N - 1) / N, LP = (LOADS * 6 / 10 + N - 1) / N, FIRST = LP * N < LOADS ? LP * N : LOADS,
                  LQ = (LOADS - FIRST + N - 1) / N;
    constexpr int CHUNKS = N * CH::kPerTile;
    // chunks on their way out: two of each loading wave, one of each storing one
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * ST::kBytes + 3 * LW * kChunk];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = wave % (BM / WM), wn = wave / (BM / WM);
    const int pitch = a.kblocks * 64, stages = (a.kblocks + 1) / 2;   // stages >= 2
    // each XCD a range of the tiles by its share of the workgroups, dealt to them in turn
    const int xcd = blockIdx.x % 8, each = gridDim.x / 8, more = gridDim.x % 8, nlocal = each + (xcd < more);
    const int64_t tiles = (int64_t)tiles_m * tiles_n;
    auto before = [&](int x) { return (int)(tiles * (x * each + min(x, more)) / (int)gridDim.x); };
    const int begin = before(xcd) + blockIdx.x / 8, end = before(xcd + 1);
    if (begin >= end) return;
    auto place = [&](int id) {
        const int per = group * tiles_n, first = id / per * group;
        const int rows = min(group, tiles_m - first), in = id % per;
        Mx4Tile t;
        t.m0 = (int64_t)(first + in % rows) * BM;
        const int col = in / rows + (int)((int64_t)first * tiles_n / tiles_m);
        t.n0 = (col < tiles_n ? col : col - tiles_n) * BN;
        t.m = (int)min((int64_t)BM, a.m - t.m0);
        t.n = min(BN, a.n - t.n0);
        t.a = a.a + t.m0 * pitch;
        t.w = a.w + (int64_t)t.n0 * pitch;
        t.as = a.as + t.m0;
        t.ws = a.ws + t.n0;
        return t;
    };
    // ---- loads: 8 rows of codes, or 64 words of scales, each
    const int lrow = wave * 8 + lane / 8;
    const uint32_t code_at = (uint32_t)lrow * (uint32_t)pitch + ((lane % 8) ^ (lrow / 2 % 8)) * 16;
    auto load = [&](int i, const Mx4Tile &t, int st, int buf) {
        uint8_t *to = lds + buf * ST::kBytes;
        const int byte0 = min(st * 128, pitch - 128);
        if (i < LA + LB) {
            const bool tok = i < LA;
            const int k = tok ? i : i - LA;
            const __amdgpu_buffer_rsrc_t rs = bounded(tok ? t.a : t.w, (uint32_t)(tok ? t.m : t.n) * (uint32_t)pitch);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rs, (__attribute__((address_space(3))) void *)(to + (i * LW + wave) * 1024), 16,
                code_at + (uint32_t)(k * LW * 8 * pitch + byte0), 0, 0, 0);
        } else {
            const int p = (i - LA - LB) * LW + wave, h = p / PARTS, part = p % PARTS;
            const bool tok = part < BM / 64;
            const int kb = byte0 / 64 + h;
            const uint32_t *from = tok ? t.as + (int64_t)kb * a.m : t.ws + (int64_t)kb * a.n;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                bounded(from, (uint32_t)(tok ? t.m : t.n) * 4u),
                (__attribute__((address_space(3))) void *)(to + ST::kCodes + h * ST::kRows * 4 + part * 256), 4,
                (uint32_t)((tok ? part : part - BM / 64) * 64 + lane) * 4u, 0, 0, 0);
        }
    };
    // ---- operands: lanes 0 .. 31 take the stage's first 128 columns, lanes 32 ..
    // 63 the others; step s of four multiplies each one's block s
    const int r = lane % 32, g = lane / 32;
    uint32_t tok_at[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) tok_at[s] = (wm * WM + r) * 128 + ((4 * g + s) ^ (r / 2 % 8)) * 16;
    const int to_weights = (BM + wn * WN - wm * WM) * 128;
    const uint32_t tok_scale = ST::kCodes + (g * ST::kRows + wm * WM + r) * 4;
    const uint32_t wgt_scale = ST::kCodes + (g * ST::kRows + BM + wn * WN + r) * 4;
    i32x4 t[2][TM], w[2][TN];
    int ts[TM], ws[TN], ts_next[TM], ws_next[TN];
    auto read = [&](int i, int buf, int step, int set) {
        const uint8_t *at = lds + buf * ST::kBytes + tok_at[step];
        if (i < TN) w[set][i] = *(const i32x4 *)(at + to_weights + i * 4096);
        else if (i < READS) t[set][i - TN] = *(const i32x4 *)(at + (i - TN) * 4096);
    };
    auto read_scale = [&](int i, int buf) {
        const uint8_t *at = lds + buf * ST::kBytes;
        if (i < TN) ws_next[i] = *(const int *)(at + wgt_scale + i * 128);
        else if (i < READS) ts_next[i - TN] = *(const int *)(at + tok_scale + (i - TN) * 128);
    };
    auto scales_of = [&](int st) {
        const bool taken = g == 0 && 2 * st + 1 == a.kblocks;
#pragma unroll
        for (int i = 0; i < TM; ++i) ts[i] = taken ? 0 : ts_next[i];
#pragma unroll
        for (int j = 0; j < TN; ++j) ws[j] = taken ? 0 : ws_next[j];
    };
    f32x16 acc[TN][TM];
    auto multiply = [&](auto step, int set, auto &&between) {
        constexpr int S = decltype(step)::value;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int j = k / TM, i = k % TM;
            acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx4_operand(w[set][j]), mx4_operand(t[set][i]),
                                                                        acc[j][i], 4, 4, S, ws[j], S, ts[i]);
            between(k);
            __builtin_amdgcn_sched_barrier(0x6);   // only arithmetic moves across
        }
    };
    auto walk = [&](auto role) {
        constexpr bool LOADER = decltype(role)::value;
        Mx4Tile cur = place(begin);
        if (LOADER) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) load(i, cur, 0, 0);
            vmem_lds_sync();
#pragma unroll
            for (int i = 0; i < FIRST; ++i) load(i, cur, 1, 1);
        } else {
            lds_sync();
        }
        int buf = 0;
#pragma unroll
        for (int i = 0; i < READS; ++i) {
            read(i, 0, 0, 0);
            read_scale(i, 0);
        }
        scales_of(0);
        for (int tile = begin; tile < end; tile += nlocal) {
            const Mx4Tile next = place(tile + nlocal < end ? tile + nlocal : tile);
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i) acc[j][i] = f32x16{};
            if (a.bias) {
                // lane: outputs 32 j + 8 q + 4 g + e
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float b = a.bias[min(cur.n0 + wn * WN + 32 * j + 8 * (e / 4) + 4 * g + e % 4, a.n - 1)];
#pragma unroll
                        for (int i = 0; i < TM; ++i) acc[j][i][e] += b;
                    }
            }
            for (int st = 0; st < stages; ++st) {
                auto reads = [&](int k, int step, int set) {
#pragma unroll
                    for (int q = 0; q < RP; ++q) read(k * RP + q, buf, step, set);
                };
                // The stage whose last loads begin before this one's barrier and
                // the one whose first loads begin after it: of this tile or, in
                // its place at the end of the walk this tile again, the next.
                auto ahead = [&](int n, int &of) {
                    const bool over = st + n >= stages;
                    of = over ? st + n - stages : st + n;
                    return Mx4Tile{over ? next.a : cur.a, over ? next.w : cur.w, over ? next.as : cur.as,
                                   over ? next.ws : cur.ws, over ? next.m : cur.m, over ? next.n : cur.n, 0, 0};
                };
                int s1, s2;
                const Mx4Tile t1 = ahead(1, s1), t2 = ahead(2, s2);
                __builtin_amdgcn_sched_barrier(0);
                multiply(std::integral_constant<int, 0>{}, 0, [&](int k) {
                    reads(k, 1, 1);
#pragma unroll
                    for (int q = 0; q < LQ; ++q)
                        if (LOADER && FIRST + k * LQ + q < LOADS) load(FIRST + k * LQ + q, t1, s1, buf ^ 1);
                });
                multiply(std::integral_constant<int, 1>{}, 1, [&](int k) { reads(k, 2, 0); });
                multiply(std::integral_constant<int, 2>{}, 0, [&](int k) { reads(k, 3, 1); });
                // every wave has read this stage, and the next one has landed
                if (LOADER) vmem_lds_sync();
                else lds_sync();
                __builtin_amdgcn_sched_barrier(0);
                buf ^= 1;
                multiply(std::integral_constant<int, 3>{}, 1, [&](int k) {
                    reads(k, 0, 0);
#pragma unroll
                    for (int q = 0; q < RP; ++q) read_scale(k * RP + q, buf);
#pragma unroll
                    for (int q = 0; q < LP; ++q)
                        if (LOADER && k * LP + q < FIRST) load(k * LP + q, t2, s2, buf ^ 1);
                });
                scales_of(st + 1 < stages ? st + 1 : 0);
            }
            // ---- out, both of a pair's chunks by the storing wave: a chunk of the
            // loading one is written again two barriers on
            uint8_t *out = lds + 2 * ST::kBytes;
            auto store = [&](int c, const uint8_t *from, int of) {
                const int i = c / CH::kPerTile / TN, j = c / CH::kPerTile % TN;
                const int om = of % (BM / WM) * WM, on = of / (BM / WM) * WN + 32 * j;
                CH::get(from, rows_of_y<OUT>(a, cur.m0 + om, min(WM, cur.m - om), cur.n0), a.n, 32 * i, on, cur.n - on,
                        c % CH::kPerTile);
            };
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                const int i = c / CH::kPerTile / TN, j = c / CH::kPerTile % TN, part = c % CH::kPerTile;
                if (LOADER) {
                    CH::put(out + (wave * 2 + c % 2) * kChunk, acc[j][i], part);
                    lds_sync();
                } else {
                    uint8_t *mine = out + (LW + wave) * kChunk;
                    CH::put(mine, acc[j][i], part);
                    wave_lds_fence();
                    store(c, mine, wave);
                    lds_sync();
                    store(c, out + ((wave - LW) * 2 + c % 2) * kChunk, wave - LW);
                }
            }
            cur = next;
        }
        // what was loaded for a tile that does not follow
        if (LOADER) __builtin_amdgcn_s_waitcnt(wait_vm(0));
    };
    if (wave < LW) walk(std::true_type{});
    else walk(std::false_type{});
}

// ---------------------------------------------------------------- launches

template <typename IN, typename OUT, int MT>
static void mx4_few_launch(const Mx4ProductArgs &a, hipStream_t stream) {
    // Up to four tiles of 16 outputs share a workgroup's activations where that
    // leaves 5/8 of the compute units one: 16 x 10576 x 2560 6.9 us with four, 7.6
    // with two, 8.3 with one; 8 x 2560 x 5120 8.5, 5.8 and 5.6.  Fewer outputs than
    // that are bound by latency, and more waves take their blocks where they also
    // quantise: 8 x 2560 x 5120 4.7 us with sixteen, 5.6 with eight; quantised
    // before, 4.5 and 4.3.
    const auto fits = [&](int nt) { return 8 * (int64_t)((a.n + 16 * nt - 1) / (16 * nt)) >= 5 * (int64_t)a.cus; };
    const auto launch = [&](auto nt, auto waves) {
        constexpr int NT = decltype(nt)::value, W = decltype(waves)::value;
        hipLaunchKernelGGL((mx4_few_kernel<IN, OUT, MT, NT, W>), dim3((a.n + 16 * NT - 1) / (16 * NT)), dim3(64 * W), 0,
                           stream, a);
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 8> eight;
    if constexpr (MT == 1) {   // (more tokens come this way with few outputs only)
        if (fits(4)) return launch(std::integral_constant<int, 4>{}, eight);
    }
    if (fits(2)) return launch(two, eight);
    if constexpr (!std::is_same_v<IN, uint8_t>) {
        if (a.kblocks > 8) return launch(one, std::integral_constant<int, 16>{});
    }
    launch(one, eight);
}

template <typename OUT>
static void mx4_few_out(const Mx4ProductArgs &a, hipStream_t stream) {
    if (a.x) {
        mx4_few_launch<OUT, OUT, 1>(a, stream);
    } else {
        a.m <= 16 ? mx4_few_launch<uint8_t, OUT, 1>(a, stream) : mx4_few_launch<uint8_t, OUT, 2>(a, stream);
    }
}

template <typename OUT, int BM, int BN, int WM, int WN, int PERCU, bool WIDE>
static void mx4_tile_launch(const Mx4ProductArgs &a, hipStream_t stream) {
    const int tm = (int)((a.m + BM - 1) / BM), tn = (a.n + BN - 1) / BN;
    const int64_t grid = std::min((int64_t)tm * tn, (int64_t)PERCU * a.cus);
    hipLaunchKernelGGL((mx4_tile_kernel<OUT, BM, BN, WM, WN, PERCU, WIDE>), dim3((unsigned)grid), dim3(64 * (BM / WM) * (BN / WN)), 0,
                       stream, a, tm, tn, 4);
}

// By tiles, in us with tiles of 256 / 128 / 64: m x 2560 x 5120, m = 4096: 33 41
// 57; 2048: 30 24 34; 1024: 29 17 19; 512: 26 15 15; 256: 26 15 8; m x 10576 x
// 2560, m = 4096: 60 70 117; 2048: 41 40 74; 1024: 23 24 40; 512: 18 15 23; 256:
// 17 11 13; 128: 17 10 8; m x 4096 x 512, m = 2048: 11 9 12; 512: 9 6 4.  So 64
// while two a compute unit hold them all, 256 from 5/8 of the compute units on.
// fp32 results, and bf16 ones in pieces that are not aligned, leave the 256 tiles
// too few registers on their way out, which long rows make up for: 256 / 128 for
// fp32 16384 x 10576 x 2560 344 340, 8192 x 4096 x 1024 53 44, 16384 x 2560 x
// 5120 141 164, 8192 x 8192 x 8192 278 335; bf16 8192 x 4097 x 1024 46 34, 4096 x
// 2561 x 2560 28 26, 16384 x 10577 x 2560 287 307, 16384 x 2561 x 5120 142 157.
template <typename OUT, bool WIDE>
static void mx4_tile_out(const Mx4ProductArgs &a, hipStream_t stream) {
    const auto tiles = [&](int b) { return ((a.m + b - 1) / b) * ((a.n + b - 1) / b); };
    if (a.kblocks <= 2 || tiles(64) <= 2 * (int64_t)a.cus)
        hipLaunchKernelGGL((mx4_ring_kernel<OUT, WIDE>), dim3((unsigned)tiles(64)), dim3(256), 0, stream, a, (a.n + 63) / 64);
    else if (8 * tiles(256) >= 5 * (int64_t)a.cus && a.kblocks > (sizeof(OUT) == 4 ? 32 : WIDE ? 0 : 16))
        mx4_tile_launch<OUT, 256, 256, 128, 64, 1, WIDE>(a, stream);
    else
        mx4_tile_launch<OUT, 128, 128, 64, 64, 2, WIDE>(a, stream);
}

// Up to 16 tokens are quantised on the way or share the weights' reading with
// nothing else; up to 32 go the same way where 64 outputs a workgroup would
// leave half of the compute units idle (32 x 2560 x 5120: 6.3 us, 8.0 in tiles; 32 x
// 10576 x 2560: 7.6 and 5.3).
static bool mx4_few(const Mx4ProductArgs &a) {
    return a.m <= 16 || (a.m <= 32 && (a.n + 63) / 64 <= a.cus / 2);
}

void launch_mx4_product(bool bf16_out, const Mx4ProductArgs &a, hipStream_t stream) {
    const int size = bf16_out ? 2 : 4;
    const bool wide = (uintptr_t)a.y % 16 == 0 && (int64_t)a.n * size % 16 == 0;   // every 16-byte piece of y aligned
    if (mx4_few(a))
        bf16_out ? mx4_few_out<bf16>(a, stream) : mx4_few_out<float>(a, stream);
    else if (wide)
        bf16_out ? mx4_tile_out<bf16, true>(a, stream) : mx4_tile_out<float, true>(a, stream);
    else
        bf16_out ? mx4_tile_out<bf16, false>(a, stream) : mx4_tile_out<float, false>(a, stream);
}

}  // namespace ssd
