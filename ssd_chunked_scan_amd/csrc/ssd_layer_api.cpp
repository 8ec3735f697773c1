// Host side of the layer operators declared in include/ssd.h (ssd_glr_*,
// ssd_conv_*, ssd_norm_*): argument validation, the choice of vector width and
// sequence splits, the workspace layout and the launches.
#include "ssd_host.hpp"
#include "ssd_layer.hpp"

namespace ssd {
void launch_glr_fwd(bool bf16_io, bool pair, const GlrArgs &a, hipStream_t stream);
void launch_glr_bwd(bool bf16_io, bool pair, const GlrArgs &a, hipStream_t stream);
void launch_glr_step(bool bf16_io, bool pair, const GlrStepArgs &a, hipStream_t stream);
int conv_strip(bool pair);
void launch_conv_fwd(bool bf16_io, bool pair, const ConvArgs &a, hipStream_t stream);
void launch_conv_bwd(bool bf16_io, bool pair, const ConvArgs &a, int run, float *dweight, float *dbias,
                     hipStream_t stream);
void launch_conv_step(bool bf16_io, bool pair, const ConvArgs &a, hipStream_t stream);
void launch_norm_fwd(bool bf16_io, bool wide, const NormArgs &a, hipStream_t stream);
void launch_norm_bwd(bool bf16_io, bool wide, const NormArgs &a, float *dweight, hipStream_t stream);
}  // namespace ssd

namespace {

constexpr int kRound = 128, kBlock = 64;   // tokens per round and per backward block of the recurrence

// ------------------------------------------------- gated linear recurrence

ssd_status_t check_glr(const ssd_glr_shape_t *s, ssd_dtype_t io) {
    if (!s) return fail(SSD_ERR_NULL, "shape is NULL");
    SSD_TRY(check_io(io));
    SSD_TRY(check_tokens(s->batch, s->seqlen, s->channels));
    SSD_TRY(check_stride("x", s->x_stride, s->channels, s->batch * s->seqlen, s->seqlen));
    SSD_TRY(check_stride("g", s->g_stride, s->channels, s->batch * s->seqlen, s->seqlen));
    SSD_TRY(check_stride("z", s->z_stride, s->channels, s->batch * s->seqlen, s->seqlen));
    SSD_TRY(check_stride("dy", s->dy_stride, s->channels, s->batch * s->seqlen, s->seqlen));
    if (s->normalize != 0 && s->normalize != 1)
        return fail(SSD_ERR_UNSUPPORTED, "normalize must be 0 or 1, got %lld", (long long)s->normalize);
    SSD_TRY(check_reserved(s->reserved));
    // the smallest strip is 32 channels
    const int64_t units = s->batch * ((s->seqlen + kBlock - 1) / kBlock) * ((s->channels + 31) / 32);
    // (workgroups of up to 512 threads; the block scan takes 1024 for every 64
    // channels of a row)
    if (units > kMaxThreads / 512 || s->batch * ((s->channels + 63) / 64) > kMaxThreads / 1024)
        return fail(SSD_ERR_UNSUPPORTED, "problem too large: %lld work units", (long long)units);
    return SSD_OK;
}

// Sequence splits of the forward walk: none when rows and strips of 64
// channels give every compute unit a workgroup; else as many as fill two for
// each, rounded up (1 x 65536 x 1024: 162 us, 167 with one for each and 168 with
// three; 2 x 4096 x 5120: 115 us with 4 splits, 126 with 3), and of at least two
// rounds.  A split costs a second reading of x and g.
void glr_fwd_split(const ssd_glr_shape_t *s, hipStream_t stream, int *nblk, int *blk_len) {
    const int64_t rounds = (s->seqlen + kRound - 1) / kRound;
    const int64_t units = s->batch * ((s->channels + 63) / 64);
    const int64_t cus = ssd::compute_units(stream);
    int64_t n = 1;
    if (units < cus) n = std::max<int64_t>(1, std::min<int64_t>((2 * cus + units - 1) / units, rounds / 2));
    const int64_t per = (rounds + n - 1) / n;
    *nblk = (int)((rounds + per - 1) / per);
    *blk_len = (int)(per * kRound);
}

size_t glr_fwd_bytes(const ssd_glr_shape_t *s, int nblk) {
    return nblk > 1 ? 2 * round_up(sizeof(float) * (size_t)s->batch * nblk * s->channels, 256) : 0;
}

size_t glr_bwd_bytes(const ssd_glr_shape_t *s) {
    const size_t one = sizeof(float) * (size_t)s->batch * ((s->seqlen + kBlock - 1) / kBlock) * s->channels;
    return 3 * round_up(one, 256) + round_up(2 * one, 256);
}

ssd::GlrArgs glr_args(const ssd_glr_shape_t *s, ssd_dtype_t io, const void *x, const void *g, const float *A,
                      const float *bias, const void *z, const int32_t *seq_idx, const float *init) {
    ssd::GlrArgs a = {};
    a.x = x;
    a.g = g;
    a.z = z;
    a.xs = stride_bytes(s->x_stride, s->channels, io);
    a.gs = stride_bytes(s->g_stride, s->channels, io);
    a.zs = stride_bytes(s->z_stride, s->channels, io);
    a.dys = stride_bytes(s->dy_stride, s->channels, io);
    a.A = A;
    a.bias = bias;
    a.seq_idx = seq_idx;
    a.init = init;
    a.batch = (int)s->batch;
    a.seqlen = (int)s->seqlen;
    a.channels = (int)s->channels;
    a.normalize = (int)s->normalize;
    return a;
}

// ------------------------------------------------------------- convolution

ssd_status_t check_conv(const ssd_conv_shape_t *s, ssd_dtype_t io) {
    if (!s) return fail(SSD_ERR_NULL, "shape is NULL");
    SSD_TRY(check_io(io));
    SSD_TRY(check_tokens(s->batch, s->seqlen, s->channels));
    if (s->width < 2 || s->width > 4) return fail(SSD_ERR_UNSUPPORTED, "width %lld not in {2, 3, 4}", (long long)s->width);
    SSD_TRY(check_stride("x", s->x_stride, s->channels, s->batch * s->seqlen, s->seqlen));
    SSD_TRY(check_stride("dy", s->dy_stride, s->channels, s->batch * s->seqlen, s->seqlen));
    if (s->silu != 0 && s->silu != 1) return fail(SSD_ERR_UNSUPPORTED, "silu must be 0 or 1, got %lld", (long long)s->silu);
    SSD_TRY(check_reserved(s->reserved));
    // single channels: a wave per 16 tokens x 64 channels (forward), a workgroup
    // per 64 x 64 (backward)
    const int64_t fwd = (s->batch * ((s->seqlen + 15) / 16) * ((s->channels + 63) / 64) + 3) / 4;
    const int64_t bwd = s->batch * ((s->seqlen + 63) / 64) * ((s->channels + 63) / 64);
    if (fwd > kMaxGrid || bwd > kMaxGrid) return fail(SSD_ERR_UNSUPPORTED, "problem too large");
    return SSD_OK;
}

// Tokens per backward workgroup: 256 (64 per wave), which keeps the weight
// sums' parts to a few percent of the traffic, or 64 when that would leave the
// device with less than two workgroups of four waves per compute unit.
int conv_run(const ssd_conv_shape_t *s, int strip, hipStream_t stream) {
    const int64_t units = s->batch * ((s->seqlen + 255) / 256) * ((s->channels + strip - 1) / strip);
    return units >= 2 * (int64_t)ssd::compute_units(stream) ? 256 : 64;
}

ssd::ConvArgs conv_args(const ssd_conv_shape_t *s, ssd_dtype_t io, const void *x, const float *weight,
                        const float *bias, const int32_t *seq_idx, const void *init) {
    ssd::ConvArgs a = {};
    a.x = x;
    a.xs = stride_bytes(s->x_stride, s->channels, io);
    a.dys = stride_bytes(s->dy_stride, s->channels, io);
    a.weight = weight;
    a.bias = bias;
    a.seq_idx = seq_idx;
    a.init = init;
    a.batch = (int)s->batch;
    a.seqlen = (int)s->seqlen;
    a.channels = (int)s->channels;
    a.width = (int)s->width;
    a.silu = (int)s->silu;
    return a;
}

// -------------------------------------------------------------------- norm

ssd_status_t check_norm(const ssd_norm_shape_t *s, ssd_dtype_t io, bool quant) {
    if (!s) return fail(SSD_ERR_NULL, "shape is NULL");
    SSD_TRY(check_io(io));
    SSD_TRY(check_tokens(s->rows, 1, s->columns));
    if (s->ngroups < 1 || s->columns % s->ngroups != 0)
        return fail(SSD_ERR_SHAPE, "columns (%lld) must be a multiple of ngroups (%lld)", (long long)s->columns,
                    (long long)s->ngroups);
    if (s->columns / s->ngroups > kMaxNormWidth)
        return fail(SSD_ERR_UNSUPPORTED, "a norm group has %lld columns, at most %lld are supported",
                    (long long)(s->columns / s->ngroups), (long long)kMaxNormWidth);
    if (s->ngroups > 65535) return fail(SSD_ERR_UNSUPPORTED, "ngroups %lld is too large", (long long)s->ngroups);
    SSD_TRY(check_stride("x", s->x_stride, s->columns, s->rows, 1));
    SSD_TRY(check_stride("z", s->z_stride, s->columns, s->rows, 1));
    SSD_TRY(check_stride("residual", s->residual_stride, s->columns, s->rows, 1));
    SSD_TRY(check_stride("dy", s->dy_stride, s->columns, s->rows, 1));
    SSD_TRY(check_stride("dresidual", s->dresidual_stride, s->columns, s->rows, 1));
    if (!(std::isfinite(s->eps) && s->eps > 0.f)) return fail(SSD_ERR_UNSUPPORTED, "eps must be positive and finite");
    if (s->quant_block != 0 && !(quant && s->quant_block == 128))
        return fail(SSD_ERR_UNSUPPORTED, "quant_block %d: 0 or 128, and 0 without an 8-bit output", (int)s->quant_block);
    return check_reserved(s->reserved);
}

// Workgroups along the rows of the backward kernel, each one part of the
// weight gradient: two per compute unit over all groups, at most one per row.
// That is what the registers of ten waves (5120 columns) leave room for: 195 us
// for 16384 gated rows, floor 171.  Groups of at most 512 columns run four
// single-row waves a workgroup and would have room for more: 40 groups of 128
// in the same rows take 622 us.
int norm_parts(const ssd_norm_shape_t *s, hipStream_t stream) {
    const int64_t want = (2 * (int64_t)ssd::compute_units(stream) + s->ngroups - 1) / s->ngroups;
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, s->rows));
}

size_t norm_bwd_bytes(const ssd_norm_shape_t *s, hipStream_t stream) {
    return round_up(sizeof(float) * (size_t)norm_parts(s, stream) * s->columns, 256);
}

ssd::NormArgs norm_args(const ssd_norm_shape_t *s, ssd_dtype_t io, const void *x, const float *weight, const void *z) {
    ssd::NormArgs a = {};
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.xs = stride_bytes(s->x_stride, s->columns, io);
    a.zs = stride_bytes(s->z_stride, s->columns, io);
    a.rs = stride_bytes(s->residual_stride, s->columns, io);
    a.dys = stride_bytes(s->dy_stride, s->columns, io);
    a.drs = stride_bytes(s->dresidual_stride, s->columns, io);
    a.eps = s->eps;
    a.quant_block = s->quant_block;
    a.rows = s->rows;
    a.columns = (int)s->columns;
    a.ngroups = (int)s->ngroups;
    a.width = (int)(s->columns / s->ngroups);
    return a;
}

ssd_status_t norm_fwd(const ssd_norm_shape_t *s, ssd_dtype_t io, const void *x, const float *weight,
                      const void *residual, const void *z, void *y, float *scales, void *residual_out, void *stream,
                      bool quant, const char *what) {
    SSD_TRY(check_norm(s, io, quant));
    const size_t e = io_size(io);
    SSD_TRY(need("x", x, e));
    SSD_TRY(maybe("weight", weight, 4));
    SSD_TRY(maybe("residual", residual, e));
    SSD_TRY(maybe("z", z, e));
    SSD_TRY(need(quant ? "q" : "y", y, quant ? 1 : e));
    if (quant) SSD_TRY(need("scales", scales, 4));
    SSD_TRY(maybe("residual_out", residual_out, e));
    if (residual && z) return fail(SSD_ERR_UNSUPPORTED, "residual and z exclude each other");
    if (!residual != !residual_out) return fail(SSD_ERR_NULL, "residual and residual_out are given together");
    ssd::NormArgs a = norm_args(s, io, x, weight, z);
    a.residual = residual;
    a.residual_out = residual_out;
    a.y = y;
    a.scales = quant ? scales : nullptr;
    a.cus = ssd::compute_units((hipStream_t)stream);
    const int n = wide_of(io);
    const int64_t dense = s->columns * (int64_t)e;
    Access acc(a.width % n == 0, n, io);
    acc.in(x, a.xs).in(z, a.zs).in(residual, a.rs).in(residual_out, dense);
    if (quant)
        acc.ok = acc.ok && aligned(y, n);
    else
        acc.in(y, dense);
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_norm_fwd(io == SSD_BF16, acc.ok, a, (hipStream_t)stream);
    return launched(what);
}

}  // namespace

extern "C" {

size_t ssd_glr_fwd_workspace_bytes(const ssd_glr_shape_t *shape, ssd_dtype_t io) {
    if (check_glr(shape, io) != SSD_OK) return 0;
    int nblk, len;
    glr_fwd_split(shape, nullptr, &nblk, &len);
    return glr_fwd_bytes(shape, nblk);
}

ssd_status_t ssd_glr_fwd(const ssd_glr_shape_t *shape, ssd_dtype_t io, const void *x, const void *g, const float *A,
                         const float *bias, const void *z, const int32_t *seq_idx, const float *init_states, void *y,
                         float *final_states, void *workspace, size_t workspace_bytes, void *stream) {
    SSD_TRY(check_glr(shape, io));
    const size_t e = io_size(io);
    SSD_TRY(need("x", x, e));
    SSD_TRY(need("g", g, e));
    SSD_TRY(need("A", A, 4));
    SSD_TRY(maybe("bias", bias, 4));
    SSD_TRY(maybe("z", z, e));
    SSD_TRY(maybe("seq_idx", seq_idx, 4));
    SSD_TRY(maybe("init_states", init_states, 4));
    SSD_TRY(need("y", y, e));
    SSD_TRY(maybe("final_states", final_states, 4));
    ssd::GlrArgs a = glr_args(shape, io, x, g, A, bias, z, seq_idx, init_states);
    glr_fwd_split(shape, (hipStream_t)stream, &a.nblk, &a.blk_len);
    a.cus = ssd::compute_units((hipStream_t)stream);
    const size_t bytes = glr_fwd_bytes(shape, a.nblk);
    SSD_TRY(check_workspace(workspace, workspace_bytes, bytes));
    a.y = y;
    a.final_states = final_states;
    a.ws_p = (float *)workspace;
    a.ws_h = bytes ? (float *)((char *)workspace + bytes / 2) : nullptr;
    const int64_t dense = shape->channels * (int64_t)e;
    const bool pair = Access(shape->channels % 2 == 0, 2, io).in(x, a.xs).in(g, a.gs).in(z, a.zs).in(y, dense).ok;
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_glr_fwd(io == SSD_BF16, pair, a, (hipStream_t)stream);
    return launched("ssd_glr_fwd");
}

size_t ssd_glr_bwd_workspace_bytes(const ssd_glr_shape_t *shape, ssd_dtype_t io) {
    return check_glr(shape, io) == SSD_OK ? glr_bwd_bytes(shape) : 0;
}

ssd_status_t ssd_glr_bwd(const ssd_glr_shape_t *shape, ssd_dtype_t io, const void *x, const void *g, const float *A,
                         const float *bias, const void *z, const int32_t *seq_idx, const float *init_states,
                         const void *dy, const float *dfinal, void *dx, void *dg, void *dz, float *dA, float *dbias,
                         float *dinit, void *workspace, size_t workspace_bytes, void *stream) {
    SSD_TRY(check_glr(shape, io));
    const size_t e = io_size(io);
    SSD_TRY(need("x", x, e));
    SSD_TRY(need("g", g, e));
    SSD_TRY(need("A", A, 4));
    SSD_TRY(maybe("bias", bias, 4));
    SSD_TRY(maybe("z", z, e));
    SSD_TRY(maybe("seq_idx", seq_idx, 4));
    SSD_TRY(maybe("init_states", init_states, 4));
    SSD_TRY(need("dy", dy, e));
    SSD_TRY(maybe("dfinal", dfinal, 4));
    SSD_TRY(need("dx", dx, e));
    SSD_TRY(need("dg", dg, e));
    SSD_TRY(maybe("dz", dz, e));
    SSD_TRY(need("dA", dA, 4));
    SSD_TRY(maybe("dbias", dbias, 4));
    SSD_TRY(maybe("dinit", dinit, 4));
    if (!z != !dz) return fail(SSD_ERR_NULL, "dz is given exactly when z is");
    if (!bias != !dbias) return fail(SSD_ERR_NULL, "dbias is given exactly when bias is");
    if (dinit && !init_states) return fail(SSD_ERR_NULL, "dinit needs init_states");
    const size_t bytes = glr_bwd_bytes(shape);
    SSD_TRY(check_workspace(workspace, workspace_bytes, bytes));
    ssd::GlrArgs a = glr_args(shape, io, x, g, A, bias, z, seq_idx, init_states);
    a.nblk = (int)((shape->seqlen + kBlock - 1) / kBlock);
    a.blk_len = kBlock;
    a.dy = dy;
    a.dfinal = dfinal;
    a.dx = dx;
    a.dg = dg;
    a.dz = dz;
    a.dA = dA;
    a.dbias = dbias;
    a.dinit = dinit;
    const size_t one = round_up(sizeof(float) * (size_t)shape->batch * a.nblk * shape->channels, 256);
    a.ws_p = (float *)workspace;
    a.ws_h = (float *)((char *)workspace + one);
    a.ws_e = (float *)((char *)workspace + 2 * one);
    a.part = (float *)((char *)workspace + 3 * one);
    const int64_t dense = shape->channels * (int64_t)e;
    const bool pair = Access(shape->channels % 2 == 0, 2, io).in(x, a.xs).in(g, a.gs).in(z, a.zs).in(dy, a.dys)
                          .in(dx, dense).in(dg, dense).in(dz, dense).ok;
    a.once = dense % 64 == 0 && aligned(dx, 64) && aligned(dg, 64) && aligned(dz, 64);
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_glr_bwd(io == SSD_BF16, pair, a, (hipStream_t)stream);
    return launched("ssd_glr_bwd");
}

ssd_status_t ssd_glr_step(const ssd_glr_shape_t *shape, ssd_dtype_t io, const void *x, const void *g, const float *A,
                          const float *bias, const void *z, float *state, void *y, void *stream) {
    SSD_TRY(check_glr(shape, io));
    if (shape->seqlen != 1) return fail(SSD_ERR_SHAPE, "a step takes one token, seqlen is %lld", (long long)shape->seqlen);
    const size_t e = io_size(io);
    SSD_TRY(need("x", x, e));
    SSD_TRY(need("g", g, e));
    SSD_TRY(need("A", A, 4));
    SSD_TRY(maybe("bias", bias, 4));
    SSD_TRY(maybe("z", z, e));
    SSD_TRY(need("state", state, 4));
    SSD_TRY(need("y", y, e));
    const ssd::GlrArgs s = glr_args(shape, io, x, g, A, bias, z, nullptr, nullptr);
    const ssd::GlrStepArgs a = {x, g, z, s.xs, s.gs, s.zs, A, bias, state, y, s.batch, s.channels, s.normalize};
    const int64_t dense = shape->channels * (int64_t)e;
    const bool pair = Access(shape->channels % 2 == 0, 2, io).in(x, a.xs).in(g, a.gs).in(z, a.zs).in(y, dense).ok;
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_glr_step(io == SSD_BF16, pair, a, (hipStream_t)stream);
    return launched("ssd_glr_step");
}

ssd_status_t ssd_conv_fwd(const ssd_conv_shape_t *shape, ssd_dtype_t io, const void *x, const float *weight,
                          const float *bias, const int32_t *seq_idx, const void *init_states, void *y,
                          void *final_states, void *stream) {
    SSD_TRY(check_conv(shape, io));
    const size_t e = io_size(io);
    SSD_TRY(need("x", x, e));
    SSD_TRY(need("weight", weight, 4));
    SSD_TRY(maybe("bias", bias, 4));
    SSD_TRY(maybe("seq_idx", seq_idx, 4));
    SSD_TRY(maybe("init_states", init_states, e));
    SSD_TRY(need("y", y, e));
    SSD_TRY(maybe("final_states", final_states, e));
    ssd::ConvArgs a = conv_args(shape, io, x, weight, bias, seq_idx, init_states);
    a.y = y;
    a.final_states = final_states;
    const int64_t dense = shape->channels * (int64_t)e;
    const bool pair = Access(shape->channels % 2 == 0, 2, io).in(x, a.xs).in(init_states, dense).in(y, dense)
                          .in(final_states, dense).ok;
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_conv_fwd(io == SSD_BF16, pair, a, (hipStream_t)stream);
    return launched("ssd_conv_fwd");
}

// The parts' size does not depend on the alignment that chooses the strip:
// the smaller run of tokens bounds it.
size_t ssd_conv_bwd_workspace_bytes(const ssd_conv_shape_t *shape, ssd_dtype_t io) {
    if (check_conv(shape, io) != SSD_OK) return 0;
    const size_t parts = (size_t)shape->batch * ((shape->seqlen + 63) / 64);
    return round_up(sizeof(float) * parts * (shape->width + 1) * shape->channels, 256);
}

ssd_status_t ssd_conv_bwd(const ssd_conv_shape_t *shape, ssd_dtype_t io, const void *x, const float *weight,
                          const float *bias, const int32_t *seq_idx, const void *init_states, const void *dy,
                          const float *dfinal, void *dx, float *dweight, float *dbias, float *dinit, void *workspace,
                          size_t workspace_bytes, void *stream) {
    SSD_TRY(check_conv(shape, io));
    const size_t e = io_size(io);
    SSD_TRY(need("x", x, e));
    SSD_TRY(need("weight", weight, 4));
    SSD_TRY(maybe("bias", bias, 4));
    SSD_TRY(maybe("seq_idx", seq_idx, 4));
    SSD_TRY(maybe("init_states", init_states, e));
    SSD_TRY(need("dy", dy, e));
    SSD_TRY(maybe("dfinal", dfinal, 4));
    SSD_TRY(need("dx", dx, e));
    SSD_TRY(need("dweight", dweight, 4));
    SSD_TRY(maybe("dbias", dbias, 4));
    SSD_TRY(maybe("dinit", dinit, 4));
    if (!bias != !dbias) return fail(SSD_ERR_NULL, "dbias is given exactly when bias is");
    if (dinit && !init_states) return fail(SSD_ERR_NULL, "dinit needs init_states");
    SSD_TRY(check_workspace(workspace, workspace_bytes, ssd_conv_bwd_workspace_bytes(shape, io)));
    ssd::ConvArgs a = conv_args(shape, io, x, weight, bias, seq_idx, init_states);
    a.dy = dy;
    a.dfinal = dfinal;
    a.dx = dx;
    a.dinit = dinit;
    a.part = (float *)workspace;
    const int64_t dense = shape->channels * (int64_t)e;
    const bool pair = Access(shape->channels % 2 == 0, 2, io).in(x, a.xs).in(dy, a.dys).in(init_states, dense)
                          .in(dx, dense).ok;
    const int run = conv_run(shape, ssd::conv_strip(pair), (hipStream_t)stream);
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_conv_bwd(io == SSD_BF16, pair, a, run, dweight, dbias, (hipStream_t)stream);
    return launched("ssd_conv_bwd");
}

ssd_status_t ssd_conv_step(const ssd_conv_shape_t *shape, ssd_dtype_t io, const void *x, const float *weight,
                           const float *bias, void *state, void *y, void *stream) {
    SSD_TRY(check_conv(shape, io));
    if (shape->seqlen != 1) return fail(SSD_ERR_SHAPE, "a step takes one token, seqlen is %lld", (long long)shape->seqlen);
    const size_t e = io_size(io);
    SSD_TRY(need("x", x, e));
    SSD_TRY(need("weight", weight, 4));
    SSD_TRY(maybe("bias", bias, 4));
    SSD_TRY(need("state", state, e));
    SSD_TRY(need("y", y, e));
    ssd::ConvArgs a = conv_args(shape, io, x, weight, bias, nullptr, nullptr);
    a.state = state;
    a.y = y;
    const int64_t dense = shape->channels * (int64_t)e;
    const bool pair = Access(shape->channels % 2 == 0, 2, io).in(x, a.xs).in(state, dense).in(y, dense).ok;
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_conv_step(io == SSD_BF16, pair, a, (hipStream_t)stream);
    return launched("ssd_conv_step");
}

ssd_status_t ssd_norm_fwd(const ssd_norm_shape_t *shape, ssd_dtype_t io, const void *x, const float *weight,
                          const void *residual, const void *z, void *y, void *residual_out, void *stream) {
    return norm_fwd(shape, io, x, weight, residual, z, y, nullptr, residual_out, stream, false, "ssd_norm_fwd");
}

ssd_status_t ssd_norm_quant_fwd(const ssd_norm_shape_t *shape, ssd_dtype_t io, const void *x, const float *weight,
                                const void *residual, const void *z, void *q, float *scales, void *residual_out,
                                void *stream) {
    return norm_fwd(shape, io, x, weight, residual, z, q, scales, residual_out, stream, true, "ssd_norm_quant_fwd");
}

size_t ssd_norm_bwd_workspace_bytes(const ssd_norm_shape_t *shape, ssd_dtype_t io) {
    return check_norm(shape, io, false) == SSD_OK ? norm_bwd_bytes(shape, nullptr) : 0;
}

ssd_status_t ssd_norm_bwd(const ssd_norm_shape_t *shape, ssd_dtype_t io, const void *x, const float *weight,
                          const void *z, const void *dy, const void *dresidual, void *dx, void *dz, float *dweight,
                          void *workspace, size_t workspace_bytes, void *stream) {
    SSD_TRY(check_norm(shape, io, false));
    const size_t e = io_size(io);
    SSD_TRY(need("x", x, e));
    SSD_TRY(maybe("weight", weight, 4));
    SSD_TRY(maybe("z", z, e));
    SSD_TRY(need("dy", dy, e));
    SSD_TRY(maybe("dresidual", dresidual, e));
    SSD_TRY(need("dx", dx, e));
    SSD_TRY(maybe("dz", dz, e));
    SSD_TRY(maybe("dweight", dweight, 4));
    if (!z != !dz) return fail(SSD_ERR_NULL, "dz is given exactly when z is");
    if (!weight != !dweight) return fail(SSD_ERR_NULL, "dweight is given exactly when weight is");
    if (z && dresidual) return fail(SSD_ERR_UNSUPPORTED, "z and dresidual exclude each other");
    if (weight) SSD_TRY(check_workspace(workspace, workspace_bytes, norm_bwd_bytes(shape, (hipStream_t)stream)));
    ssd::NormArgs a = norm_args(shape, io, x, weight, z);
    a.dy = dy;
    a.dresidual = dresidual;
    a.dx = dx;
    a.dz = dz;
    a.parts = norm_parts(shape, (hipStream_t)stream);
    a.part = weight ? (float *)workspace : nullptr;
    const int n = wide_of(io);
    const int64_t dense = shape->columns * (int64_t)e;
    const bool wide = Access(a.width % n == 0, n, io).in(x, a.xs).in(z, a.zs).in(dy, a.dys).in(dresidual, a.drs)
                          .in(dx, dense).in(dz, dense).ok;
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_norm_bwd(io == SSD_BF16, wide, a, dweight, (hipStream_t)stream);
    return launched("ssd_norm_bwd");
}

}  // extern "C"
