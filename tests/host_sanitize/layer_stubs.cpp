// Host stand-ins for the launchers of the layer operators, for the sanitizer
// build of ssd_layer_api.cpp: each reads and writes every byte its kernels
// would, with the extents derived from the launch arguments the way the
// kernels index them, so that AddressSanitizer reports any launch whose
// arguments reach outside a caller's buffer of the documented size.
#include <cstdint>
#include <cstring>
#include <string>

#include "ssd_layer.hpp"

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

// `tokens` tokens of `bytes` bytes, `stride` bytes apart
void rd_tokens(const void *p, size_t tokens, size_t stride, size_t bytes) {
    for (size_t t = 0; p && t < tokens; ++t) rd((const char *)p + t * stride, bytes);
}

}  // namespace

extern "C" {
uint64_t g_layer_launches;
int g_layer_fast;   // the last launch's vector width was the wide one
const char *layer_error(void) { return g_error.c_str(); }
hipError_t hipGetLastError(void) { return hipSuccess; }
const char *hipGetErrorString(hipError_t) { return "none"; }
}

namespace ssd {

void set_last_error(const char *msg) { g_error = msg; }
int compute_units(hipStream_t) { return 256; }

static void glr_inputs(bool bf16_io, bool pair, const GlrArgs &a) {
    ++g_layer_launches;
    g_layer_fast = pair;
    const size_t e = bf16_io ? 2 : 4, n = (size_t)a.batch * a.seqlen, D = a.channels;
    rd_tokens(a.x, n, a.xs, D * e);
    rd_tokens(a.g, n, a.gs, D * e);
    rd_tokens(a.z, n, a.zs, D * e);
    rd(a.A, 4 * D);
    rd(a.bias, 4 * D);
    rd(a.seq_idx, 4 * n);
    rd(a.init, 4 * D * a.batch);
}

void launch_glr_fwd(bool bf16_io, bool pair, const GlrArgs &a, hipStream_t) {
    glr_inputs(bf16_io, pair, a);
    const size_t e = bf16_io ? 2 : 4, D = a.channels, blocks = (size_t)a.batch * a.nblk * D;
    if (a.nblk < 1 || (int64_t)a.nblk * a.blk_len < a.seqlen || (int64_t)(a.nblk - 1) * a.blk_len >= a.seqlen)
        __builtin_trap();
    if (a.nblk > 1) {
        wr(a.ws_p, 4 * blocks);
        wr(a.ws_h, 4 * blocks);
        if (a.ws_p < a.ws_h + blocks && a.ws_h < a.ws_p + blocks) __builtin_trap();
    }
    wr(a.y, (size_t)a.batch * a.seqlen * D * e);
    wr(a.final_states, 4 * D * a.batch);
}

void launch_glr_bwd(bool bf16_io, bool pair, const GlrArgs &a, hipStream_t) {
    glr_inputs(bf16_io, pair, a);
    const size_t e = bf16_io ? 2 : 4, D = a.channels, n = (size_t)a.batch * a.seqlen, blocks = (size_t)a.batch * a.nblk * D;
    if ((int64_t)a.nblk * a.blk_len < a.seqlen || (int64_t)(a.nblk - 1) * a.blk_len >= a.seqlen) __builtin_trap();
    rd_tokens(a.dy, n, a.dys, D * e);
    rd(a.dfinal, 4 * D * a.batch);
    float *part[4] = {a.ws_p, a.ws_h, a.ws_e, a.part};
    for (int i = 0; i < 4; ++i) {
        wr(part[i], (i == 3 ? 8 : 4) * blocks);
        if (i && part[i - 1] + blocks > part[i]) __builtin_trap();
    }
    wr(a.dx, n * D * e);
    wr(a.dg, n * D * e);
    wr(a.dz, n * D * e);
    wr(a.dA, 4 * D);
    wr(a.dbias, 4 * D);
    wr(a.dinit, 4 * D * a.batch);
}

void launch_glr_step(bool bf16_io, bool pair, const GlrStepArgs &a, hipStream_t) {
    ++g_layer_launches;
    g_layer_fast = pair;
    const size_t e = bf16_io ? 2 : 4, D = a.channels;
    rd_tokens(a.x, a.batch, a.xs, D * e);
    rd_tokens(a.g, a.batch, a.gs, D * e);
    rd_tokens(a.z, a.batch, a.zs, D * e);
    rd(a.A, 4 * D);
    rd(a.bias, 4 * D);
    rd(a.state, 4 * D * a.batch);
    wr(a.state, 4 * D * a.batch);
    wr(a.y, a.batch * D * e);
}

int conv_strip(bool pair) { return 64 * (pair ? 2 : 1); }

static void conv_inputs(bool bf16_io, bool pair, const ConvArgs &a) {
    ++g_layer_launches;
    g_layer_fast = pair;
    const size_t e = bf16_io ? 2 : 4, n = (size_t)a.batch * a.seqlen, D = a.channels;
    rd_tokens(a.x, n, a.xs, D * e);
    rd(a.weight, 4 * D * a.width);
    rd(a.bias, 4 * D);
    rd(a.seq_idx, 4 * n);
    rd(a.init, e * D * a.batch * (a.width - 1));
}

void launch_conv_fwd(bool bf16_io, bool pair, const ConvArgs &a, hipStream_t) {
    conv_inputs(bf16_io, pair, a);
    const size_t e = bf16_io ? 2 : 4, n = (size_t)a.batch * a.seqlen, D = a.channels;
    wr(a.y, n * D * e);
    wr(a.final_states, e * D * a.batch * (a.width - 1));
}

void launch_conv_bwd(bool bf16_io, bool pair, const ConvArgs &a, int run, float *dweight, float *dbias, hipStream_t) {
    conv_inputs(bf16_io, pair, a);
    const size_t e = bf16_io ? 2 : 4, n = (size_t)a.batch * a.seqlen, D = a.channels;
    if (run % 64 != 0) __builtin_trap();   // four waves of whole 16-token chunks
    const size_t parts = (size_t)a.batch * ((a.seqlen + run - 1) / run);
    rd_tokens(a.dy, n, a.dys, D * e);
    rd(a.dfinal, 4 * D * a.batch * (a.width - 1));
    wr(a.part, 4 * parts * D * (a.width + 1));
    wr(a.dx, n * D * e);
    wr(a.dinit, 4 * D * a.batch * (a.width - 1));
    wr(dweight, 4 * D * a.width);
    wr(dbias, 4 * D);
}

void launch_conv_step(bool bf16_io, bool pair, const ConvArgs &a, hipStream_t) {
    conv_inputs(bf16_io, pair, a);
    const size_t e = bf16_io ? 2 : 4, D = a.channels;
    rd(a.state, e * D * a.batch * (a.width - 1));
    wr(a.state, e * D * a.batch * (a.width - 1));
    wr(a.y, a.batch * D * e);
}

void launch_norm_fwd(bool bf16_io, bool wide, const NormArgs &a, hipStream_t) {
    ++g_layer_launches;
    g_layer_fast = wide;
    const size_t e = bf16_io ? 2 : 4, D = a.columns;
    if (a.width * a.ngroups != a.columns || a.cus <= 0) __builtin_trap();
    rd_tokens(a.x, a.rows, a.xs, D * e);
    rd_tokens(a.z, a.rows, a.zs, D * e);
    rd_tokens(a.residual, a.rows, a.rs, D * e);
    rd(a.weight, 4 * D);
    wr(a.residual_out, a.rows * D * e);
    wr(a.y, a.rows * D * (a.scales ? 1 : e));
    wr(a.scales, 4 * a.rows * a.ngroups * (a.quant_block ? (a.width + 127) / 128 : 1));
}

void launch_norm_bwd(bool bf16_io, bool wide, const NormArgs &a, float *dweight, hipStream_t) {
    ++g_layer_launches;
    g_layer_fast = wide;
    const size_t e = bf16_io ? 2 : 4, D = a.columns;
    if (a.parts < 1 || a.parts > a.rows || !a.part != !dweight) __builtin_trap();
    rd_tokens(a.x, a.rows, a.xs, D * e);
    rd_tokens(a.z, a.rows, a.zs, D * e);
    rd_tokens(a.dy, a.rows, a.dys, D * e);
    rd_tokens(a.dresidual, a.rows, a.drs, D * e);
    rd(a.weight, 4 * D);
    wr(a.part, 4 * (size_t)a.parts * D);
    wr(a.dx, a.rows * D * e);
    wr(a.dz, a.rows * D * e);
    wr(dweight, 4 * D);
}

}  // namespace ssd
