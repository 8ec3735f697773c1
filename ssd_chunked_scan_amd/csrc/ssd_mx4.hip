// Microscaled 4-bit floating point: to 4 bits and back (ssd.h, ssd_mx4_quant,
// ssd_mx4_dequant).  Memory-bound: 16384 x 5120 bf16 39 us, 5.5 TB/s, and 41 back;
// 10576 x 2560, which the caches hold in part, 11.8 and 11.8.  Sixteen lanes take
// 128 columns of a row, eight each: a block of 32 is a quad of lanes, its maximum
// two lane exchanges, and the four scale bytes of the 128 columns are joined into
// one word.
#include "ssd_mx4.hpp"

namespace ssd {

constexpr int kMx4Rows = 16, kMx4Blocks = 4;   // a workgroup's rows and 128-column blocks

struct Mx4Place {
    int64_t row;
    int kb;   // first 128-column block
    bool ok;
};

__device__ inline Mx4Place mx4_place(const Mx4QuantArgs &a) {
    const uint32_t ncol = (a.kblocks + kMx4Blocks - 1) / kMx4Blocks;
    Mx4Place p;
    p.kb = (int)(blockIdx.x % ncol) * kMx4Blocks;
    p.row = (int64_t)(blockIdx.x / ncol) * kMx4Rows + threadIdx.x / 16;
    p.ok = p.row < a.rows;
    return p;
}

template <typename IO>
__global__ __launch_bounds__(256) void mx4_quant_kernel(Mx4QuantArgs a) {
    const Mx4Place p = mx4_place(a);
    const int lane = threadIdx.x % 16;
    const char *row = (const char *)a.x + min(p.row, a.rows - 1) * a.xs;
    Pack<IO, 8> v[kMx4Blocks];
#pragma unroll
    for (int b = 0; b < kMx4Blocks; ++b) v[b] = mx4_load8<IO>(row, (p.kb + b) * 128 + lane * 8, a.columns);
#pragma unroll
    for (int b = 0; b < kMx4Blocks; ++b) {
        const uint32_t byte = mx4_scale_byte(quad_max(mx4_most<IO>(v[b])));
        const uint32_t code = byte == 255u ? 0u : mx4_codes<IO>(v[b], mx4_scale(byte));
        uint32_t word = byte << (8 * (lane / 4));
        word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)word, 0x141, 0xf, 0xf, true);   // the other half of 8
        word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)word, 0x140, 0xf, 0xf, true);   // the other half of 16
        const int kb = p.kb + b;
        if (p.ok && kb < a.kblocks) {
            *(uint32_t *)(a.q + (p.row * a.kblocks + kb) * 64 + lane * 4) = code;
            if (lane == 0) a.scales[kb * a.rows + p.row] = word;
        }
    }
}

template <typename IO>
__global__ __launch_bounds__(256) void mx4_dequant_kernel(Mx4QuantArgs a) {
    const Mx4Place p = mx4_place(a);
    if (!p.ok) return;
    const int lane = threadIdx.x % 16;
    char *row = (char *)a.y + p.row * a.columns * (int64_t)sizeof(IO);
    uint32_t code[kMx4Blocks], word[kMx4Blocks];
#pragma unroll
    for (int b = 0; b < kMx4Blocks; ++b) {
        const int kb = min(p.kb + b, a.kblocks - 1);
        code[b] = *(const uint32_t *)(a.q + (p.row * a.kblocks + kb) * 64 + lane * 4);
        word[b] = a.scales[kb * a.rows + p.row];
    }
#pragma unroll
    for (int b = 0; b < kMx4Blocks; ++b) {
        const uint32_t byte = (word[b] >> (8 * (lane / 4))) & 255u;
        const float scale = mx4_scale(byte);
        float f[8];
        const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[b], scale, 0);
        const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[b], scale, 1);
        const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[b], scale, 2);
        const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[b], scale, 3);
        f[0] = v0[0], f[1] = v0[1], f[2] = v1[0], f[3] = v1[1];
        f[4] = v2[0], f[5] = v2[1], f[6] = v3[0], f[7] = v3[1];
        if (byte == 255u) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = scale;
        }
        const int c = (p.kb + b) * 128 + lane * 8;
        if (c + 8 <= a.columns) {
            constexpr int N = 16 / sizeof(IO);
#pragma unroll
            for (int i = 0; i < 8 / N; ++i) {
                Pack<IO, N> part;
#pragma unroll
                for (int j = 0; j < N; ++j) part.v[j] = (IO)f[i * N + j];
                *(mx4_piece<IO> *)(row + (c + i * N) * (int64_t)sizeof(IO)) = __builtin_bit_cast(mx4_piece<IO>, part);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < a.columns) ((IO *)row)[c + i] = (IO)f[i];
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
