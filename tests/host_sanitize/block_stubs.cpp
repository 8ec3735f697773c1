// Host stand-ins for the launchers of the operators between the layers, for the
// sanitizer build of ssd_block_api.cpp: each reads and writes every byte its
// kernels would, with the extents derived from the launch arguments the way
// the kernels index them.
#include <cstdint>
#include <cstring>
#include <string>

#include "ssd_block.hpp"
#include "ssd_mx4.hpp"

namespace {

volatile uint64_t g_sink;
std::string g_error;

void rd(const void *p, size_t n) {
    if (!p) return;
    const unsigned char *c = (const unsigned char *)p;
    uint64_t s = 0;
    for (size_t k = 0; k < n; ++k) s += c[k];
    g_sink = g_sink + s;
}

void wr(void *p, size_t n) {
    if (p) memset(p, 0x5a, n);
}

void rd_rows(const void *p, size_t rows, size_t stride, size_t bytes) {
    for (size_t t = 0; p && t < rows; ++t) rd((const char *)p + t * stride, bytes);
}

}  // namespace

extern "C" {
uint64_t g_block_launches;
const char *block_error(void) { return g_error.c_str(); }
hipError_t hipGetLastError(void) { return hipSuccess; }
const char *hipGetErrorString(hipError_t) { return "none"; }
}

namespace ssd {

void set_last_error(const char *msg) { g_error = msg; }
int compute_units(hipStream_t) { return 256; }

static void block_common(bool bf16_io, bool wide, const BlockArgs &a) {
    ++g_block_launches;
    const size_t e = bf16_io ? 2 : 4, D = a.columns;
    if (a.cus <= 0 || (wide && D * e % 4 != 0)) __builtin_trap();
    rd_rows(a.x, a.rows, a.xs, D * e);
    rd_rows(a.z, a.rows, a.zs, D * e);
    rd_rows(a.residual, a.rows, a.rs, D * e);
    rd(a.post, 4 * D);
    rd(a.pre, 4 * D);
    rd(a.scale, 4 * D);
}

void launch_block_fwd(bool bf16_io, bool wide, const BlockArgs &a, hipStream_t) {
    block_common(bf16_io, wide, a);
    const size_t e = bf16_io ? 2 : 4, D = a.columns, nb = (D + 127) / 128;
    wr(a.residual_out, a.rows * D * e);
    wr(a.y, a.rows * D * e);
    wr(a.xq, a.rows * D);
    wr(a.zq, a.rows * D);
    wr(a.sq, a.rows * D);
    wr(a.xsc, 4 * a.rows * nb);
    wr(a.zsc, 4 * a.rows * nb);
    wr(a.ssc, 4 * a.rows * nb);
}

void launch_block_bwd(bool bf16_io, bool wide, const BlockArgs &a, hipStream_t) {
    block_common(bf16_io, wide, a);
    const size_t e = bf16_io ? 2 : 4, D = a.columns, nb = (D + 127) / 128;
    if (a.parts < 1 || a.parts > a.rows) __builtin_trap();
    rd(a.xq, a.rows * D);
    rd(a.zq, a.rows * D);
    rd(a.sq, a.rows * D);
    rd(a.xsc, 4 * a.rows * nb);
    rd(a.zsc, 4 * a.rows * nb);
    rd(a.ssc, 4 * a.rows * nb);
    rd_rows(a.dy, a.rows, a.dys, D * e);
    rd_rows(a.dresidual_out, a.rows, a.drs, D * e);
    wr(a.part, 4 * (size_t)a.parts * 2 * ((D + 7) / 8 * 8));
    wr(a.dx, a.rows * D * e);
    wr(a.dz, a.rows * D * e);
    wr(a.dresidual, a.rows * D * e);
    wr(a.dpost, 4 * D);
    wr(a.dpre, 4 * D);
    wr(a.dscale, 4 * D);
}

void launch_mx4_quant(bool bf16_io, const Mx4QuantArgs &a, hipStream_t) {
    ++g_block_launches;
    rd_rows(a.x, a.rows, a.xs, (size_t)a.columns * (bf16_io ? 2 : 4));
    wr(a.q, (size_t)a.rows * a.kblocks * 64);
    wr(a.scales, (size_t)a.rows * a.kblocks * 4);
}

void launch_mx4_dequant(bool bf16_io, const Mx4QuantArgs &a, hipStream_t) {
    ++g_block_launches;
    rd(a.q, (size_t)a.rows * a.kblocks * 64);
    rd(a.scales, (size_t)a.rows * a.kblocks * 4);
    wr(a.y, (size_t)a.rows * a.columns * (bf16_io ? 2 : 4));
}

void launch_mx4_product(bool bf16_out, const Mx4ProductArgs &a, hipStream_t) {
    ++g_block_launches;
    if (a.cus <= 0 || !a.x == !a.a || (a.x && a.m > 16)) __builtin_trap();
    if (a.x) {
        rd_rows(a.x, a.m, a.xs, (size_t)a.columns * (bf16_out ? 2 : 4));
    } else {
        rd(a.a, (size_t)a.m * a.kblocks * 64);
        rd(a.as, (size_t)a.m * a.kblocks * 4);
    }
    rd(a.w, (size_t)a.n * a.kblocks * 64);
    rd(a.ws, (size_t)a.n * a.kblocks * 4);
    rd(a.bias, 4 * (size_t)a.n);
    wr(a.y, (size_t)a.m * a.n * (bf16_out ? 2 : 4));
}

}  // namespace ssd
