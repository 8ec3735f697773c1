// Microscaled 4-bit floating point: to 4 bits and back (ssd.h, ssd_mx4_quant,
// ssd_mx4_dequant).  Memory-bound: 16384 x 5120 bf16 40 us, 5.3 TB/s, and 43 back;
// 10576 x 2560, which the caches hold in part, 12 and 12.  Sixteen lanes take
// 128 columns of a row, eight each: a block of 32 is a quad of lanes, its maximum
// two lane exchanges, and the four scale bytes of the 128 columns are joined into
// one word.
#include <type_traits>

#include "ssd_mx4.hpp"

namespace ssd {

constexpr int kMx4Rows = 16, kMx4Blocks = 4;   // a workgroup's rows and 128-column blocks

template <typename IO>
__global__ __launch_bounds__(256) void mx4_quant_kernel(Mx4QuantArgs a) {
    const uint32_t ncol = (a.kblocks + kMx4Blocks - 1) / kMx4Blocks;
    const int kb0 = (int)(blockIdx.x % ncol) * kMx4Blocks, lane = threadIdx.x % 16;
    const int64_t r = (int64_t)(blockIdx.x / ncol) * kMx4Rows + threadIdx.x / 16;
    const char *row = (const char *)a.x + min(r, a.rows - 1) * a.xs;
    Pack<IO, 8> v[kMx4Blocks];
#pragma unroll
    for (int b = 0; b < kMx4Blocks; ++b) v[b] = mx4_load8<IO>(row, (kb0 + b) * 128 + lane * 8, a.columns);
#pragma unroll
    for (int b = 0; b < kMx4Blocks; ++b) {
        const uint32_t byte = mx4_scale_byte(quad_max(mx4_most<IO>(v[b])));
        const uint32_t code = byte == 255u ? 0u : mx4_codes<IO>(v[b], mx4_scale(byte));
        uint32_t word = byte << (8 * (lane / 4));
        word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)word, 0x141, 0xf, 0xf, true);   // the other half of 8
        word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)word, 0x140, 0xf, 0xf, true);   // the other half of 16
        const int kb = kb0 + b;
        if (r < a.rows && kb < a.kblocks) {
            *(uint32_t *)(a.q + (r * a.kblocks + kb) * 64 + lane * 4) = code;
            if (lane == 0) a.scales[kb * a.rows + r] = word;
        }
    }
}

// The way back: a lane takes the columns of one 16-byte piece of y, 8 bf16 or 4
// fp32, and rows a half of the workgroup's apart in fp32, so that stores lie side
// by side (16384 x 5120 fp32 83 us, 8 columns a lane 101).
template <typename IO>
__global__ __launch_bounds__(256) void mx4_dequant_kernel(Mx4QuantArgs a) {
    constexpr int V = 16 / (int)sizeof(IO), LANES = 128 / V, ROWS = 256 / LANES, H = kMx4Rows / ROWS;
    typedef std::conditional_t<V == 8, uint32_t, uint16_t> Codes;
    const uint32_t ncol = (a.kblocks + kMx4Blocks - 1) / kMx4Blocks;
    const int kb0 = (int)(blockIdx.x % ncol) * kMx4Blocks, lane = threadIdx.x % LANES;
    const int64_t row0 = (int64_t)(blockIdx.x / ncol) * kMx4Rows + threadIdx.x / LANES;
    uint32_t code[H][kMx4Blocks], word[H][kMx4Blocks];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int b = 0; b < kMx4Blocks; ++b) {
            const int64_t row = min(row0 + h * ROWS, a.rows - 1);
            const int kb = min(kb0 + b, a.kblocks - 1);
            code[h][b] = *(const Codes *)(a.q + (row * a.kblocks + kb) * 64 + lane * (V / 2));
            word[h][b] = a.scales[kb * a.rows + row];
        }
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int64_t row = row0 + h * ROWS;
        if (row >= a.rows) break;
#pragma unroll
        for (int b = 0; b < kMx4Blocks; ++b) {
            const uint32_t byte = (word[h][b] >> (8 * (lane * V / 32))) & 255u;
            const float scale = mx4_scale(byte);
            float f[V];
            const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[h][b], scale, 0);
            const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[h][b], scale, 1);
            f[0] = v0[0], f[1] = v0[1], f[2] = v1[0], f[3] = v1[1];
            if constexpr (V == 8) {
                const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[h][b], scale, 2);
                const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[h][b], scale, 3);
                f[4] = v2[0], f[5] = v2[1], f[6] = v3[0], f[7] = v3[1];
            }
            Pack<IO, V> out;
#pragma unroll
            for (int i = 0; i < V; ++i) out.v[i] = (IO)(byte == 255u ? scale : f[i]);
            const int c = (kb0 + b) * 128 + lane * V;
            IO *y = (IO *)a.y + row * a.columns + c;
            if (c + V <= a.columns) {
                *(mx4_piece<IO> *)y = __builtin_bit_cast(mx4_piece<IO>, out);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (c + i < a.columns) y[i] = out.v[i];
            }
        }
    }
}

static unsigned mx4_grid(const Mx4QuantArgs &a) {
    return (unsigned)((a.rows + kMx4Rows - 1) / kMx4Rows * ((a.kblocks + kMx4Blocks - 1) / kMx4Blocks));
}

#define SSD_MX4_BY_TYPE(kernel)                                                                    \
    if (bf16_io) hipLaunchKernelGGL((kernel<bf16>), dim3(mx4_grid(a)), dim3(256), 0, stream, a);   \
    else hipLaunchKernelGGL((kernel<float>), dim3(mx4_grid(a)), dim3(256), 0, stream, a);

void launch_mx4_quant(bool bf16_io, const Mx4QuantArgs &a, hipStream_t stream) { SSD_MX4_BY_TYPE(mx4_quant_kernel) }

void launch_mx4_dequant(bool bf16_io, const Mx4QuantArgs &a, hipStream_t stream) { SSD_MX4_BY_TYPE(mx4_dequant_kernel) }

}  // namespace ssd
