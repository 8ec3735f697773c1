// Host side of the operators between the layers declared in include/ssd.h
// (ssd_block_norm_*, ssd_mx4_*): argument validation, the choice of kernels,
// the workspace layout and the launches.
#include "ssd_block.hpp"
#include "ssd_host.hpp"
#include "ssd_mx4.hpp"

namespace ssd {
void launch_block_fwd(bool bf16_io, bool wide, const BlockArgs &a, hipStream_t stream);
void launch_block_bwd(bool bf16_io, bool wide, const BlockArgs &a, hipStream_t stream);
void launch_mx4_quant(bool bf16_io, const Mx4QuantArgs &a, hipStream_t stream);
void launch_mx4_dequant(bool bf16_io, const Mx4QuantArgs &a, hipStream_t stream);
void launch_mx4_product(bool bf16_out, const Mx4ProductArgs &a, hipStream_t stream);
}  // namespace ssd

namespace {

// -------------------------------------------------------------- block norm

ssd_status_t check_block(const ssd_block_shape_t *s, ssd_dtype_t io) {
    if (!s) return fail(SSD_ERR_NULL, "shape is NULL");
    SSD_TRY(check_io(io));
    SSD_TRY(check_tokens(s->rows, 1, s->columns));
    if (s->columns > kMaxNormWidth)
        return fail(SSD_ERR_UNSUPPORTED, "a row has %lld columns, at most %lld are supported", (long long)s->columns,
                    (long long)kMaxNormWidth);
    SSD_TRY(check_stride("x", s->x_stride, s->columns, s->rows, 1));
    SSD_TRY(check_stride("z", s->z_stride, s->columns, s->rows, 1));
    SSD_TRY(check_stride("residual", s->residual_stride, s->columns, s->rows, 1));
    SSD_TRY(check_stride("dy", s->dy_stride, s->columns, s->rows, 1));
    SSD_TRY(check_stride("dresidual", s->dresidual_stride, s->columns, s->rows, 1));
    if (!(std::isfinite(s->eps) && s->eps > 0.f)) return fail(SSD_ERR_UNSUPPORTED, "eps must be positive and finite");
    if (!std::isfinite(s->alpha)) return fail(SSD_ERR_UNSUPPORTED, "alpha must be finite");
    return check_reserved(s->reserved);
}

// Workgroups of the backward kernel, each one part of the column sums: twelve
// waves for each compute unit, and at most one workgroup for each row, or for each
// four where a wave takes a row.  More rows at once hide more latency but leave
// more parts to sum (16384 x 2560: 142 us with 2 workgroups of 5 waves for each
// compute unit, 158 with 3, 168 with 1; 8192 x 5120: 145 with 1 of 10, 158 with 2;
// 30000 x 1003: 107 with 3 of 4, 124 with 2, 116 with 4).  `wide`: 16-byte
// accesses, eight columns a thread up to 8192 columns, else four up to 4096 and
// eight up to 8192; sixteen past those.
int block_parts(const ssd_block_shape_t *s, bool wide, hipStream_t stream) {
    const int64_t per = s->columns > 8192 ? 16 : wide || s->columns > 4096 ? 8 : 4;
    const bool wave_rows = s->columns <= (wide ? 512 : 256);
    const int64_t waves = wave_rows ? 4 : (s->columns + 64 * per - 1) / (64 * per);
    return (int)std::min<int64_t>(std::max<int64_t>(1, 12 / waves) * ssd::compute_units(stream),
                                  wave_rows ? (s->rows + 3) / 4 : s->rows);
}

// For either access, which the buffers' alignment decides.
size_t block_bwd_bytes(const ssd_block_shape_t *s, hipStream_t stream) {
    const int parts = std::max(block_parts(s, true, stream), block_parts(s, false, stream));
    return round_up(sizeof(float) * 2 * (size_t)parts * round_up(s->columns, 8), 256);
}

ssd::BlockArgs block_args(const ssd_block_shape_t *s, ssd_dtype_t io, const void *x, const void *z, const void *residual,
                          const float *post, const float *pre, const float *scale, hipStream_t stream) {
    ssd::BlockArgs a = {};
    a.x = x;
    a.z = z;
    a.residual = residual;
    a.xs = stride_bytes(s->x_stride, s->columns, io);
    a.zs = stride_bytes(s->z_stride, s->columns, io);
    a.rs = stride_bytes(s->residual_stride, s->columns, io);
    a.dys = stride_bytes(s->dy_stride, s->columns, io);
    a.drs = stride_bytes(s->dresidual_stride, s->columns, io);
    a.post = post;
    a.pre = pre;
    a.scale = scale;
    a.eps = s->eps;
    a.alpha = s->alpha;
    a.rows = s->rows;
    a.columns = (int)s->columns;
    a.pitch = (int)round_up(s->columns, 8);
    a.cus = ssd::compute_units(stream);
    return a;
}

ssd_status_t check_checkpoint(const ssd_block_checkpoint_t *c, bool gate) {
    SSD_TRY(need("checkpoint x", c->x, 1));
    SSD_TRY(need("checkpoint x_scales", c->x_scales, 4));
    SSD_TRY(need("checkpoint residual", c->residual, 1));
    SSD_TRY(need("checkpoint residual_scales", c->residual_scales, 4));
    if (!c->z != !c->z_scales) return fail(SSD_ERR_NULL, "a checkpoint's z and z_scales are given together");
    if (!c->z != !gate) return fail(SSD_ERR_NULL, "a checkpoint has z exactly when there is a gate");
    return maybe("checkpoint z_scales", c->z_scales, 4);
}

void use_checkpoint(ssd::BlockArgs &a, const ssd_block_checkpoint_t *c) {
    a.xq = (uint8_t *)c->x;
    a.zq = (uint8_t *)c->z;
    a.sq = (uint8_t *)c->residual;
    a.xsc = c->x_scales;
    a.zsc = c->z_scales;
    a.ssc = c->residual_scales;
    a.code_words = a.columns % 4 == 0 && aligned(c->x, 4) && aligned(c->z, 4) && aligned(c->residual, 4);
}

// Wide accesses: of whole multiples of `bytes`, 4 at least.
Access multiples(const ssd_block_shape_t *s, ssd_dtype_t io, int bytes) {
    const int n = bytes / (int)io_size(io);
    return Access(s->columns % n == 0, n, io);
}

// --------------------------------------------------------- 4-bit operands

constexpr int64_t kFewQuantised = 16;   // tokens that the product's kernel quantises by itself

int64_t kblocks_of(const ssd_mx4_shape_t *s) { return (s->columns + 127) / 128; }

ssd_status_t check_mx4(const ssd_mx4_shape_t *s, ssd_dtype_t io, bool product) {
    if (!s) return fail(SSD_ERR_NULL, "shape is NULL");
    SSD_TRY(check_io(io));
    SSD_TRY(check_tokens(s->rows, 1, s->columns));
    if (product) {
        if (s->outputs < 1) return fail(SSD_ERR_SHAPE, "sizes must be >= 1 (%lld outputs)", (long long)s->outputs);
        if (s->outputs > kMaxChannels) return fail(SSD_ERR_UNSUPPORTED, "%lld outputs are too many", (long long)s->outputs);
        // tiles of 64 x 64, the smallest
        if ((s->rows + 63) / 64 * ((s->outputs + 63) / 64) > kMaxGrid)
            return fail(SSD_ERR_UNSUPPORTED, "problem too large: %lld rows, %lld outputs", (long long)s->rows,
                        (long long)s->outputs);
    } else if (s->outputs != 0) {
        return fail(SSD_ERR_UNSUPPORTED, "outputs must be zero without a product");
    }
    // the quantising kernel's workgroups: 16 rows, four blocks of 128 columns
    if ((s->rows + 15) / 16 * ((kblocks_of(s) + 3) / 4) > kMaxGrid)
        return fail(SSD_ERR_UNSUPPORTED, "problem too large: %lld x %lld", (long long)s->rows, (long long)s->columns);
    SSD_TRY(check_stride("x", s->x_stride, s->columns, s->rows, 1));
    return check_reserved(s->reserved);
}

ssd_status_t check_operand(const char *name, const void *q, const char *scales_name, const void *scales) {
    SSD_TRY(need(name, q, 16));
    return need(scales_name, scales, 4);
}

ssd::Mx4QuantArgs quant_args(const ssd_mx4_shape_t *s, ssd_dtype_t io) {
    ssd::Mx4QuantArgs a = {};
    a.xs = stride_bytes(s->x_stride, s->columns, io);
    a.rows = s->rows;
    a.columns = (int)s->columns;
    a.kblocks = (int)kblocks_of(s);
    return a;
}

ssd::Mx4ProductArgs product_args(const ssd_mx4_shape_t *s, const void *wq, const void *wscales, const float *bias,
                                 void *y, hipStream_t stream) {
    ssd::Mx4ProductArgs a = {};
    a.w = (const uint8_t *)wq;
    a.ws = (const uint32_t *)wscales;
    a.bias = bias;
    a.y = y;
    a.m = s->rows;
    a.n = (int)s->outputs;
    a.columns = (int)s->columns;
    a.kblocks = (int)kblocks_of(s);
    a.cus = ssd::compute_units(stream);
    return a;
}

size_t linear_codes(const ssd_mx4_shape_t *s) { return round_up((size_t)s->rows * kblocks_of(s) * 64, 256); }

size_t linear_bytes(const ssd_mx4_shape_t *s) {
    return s->rows <= kFewQuantised ? 0 : linear_codes(s) + round_up((size_t)s->rows * kblocks_of(s) * 4, 256);
}

}  // namespace

extern "C" {

ssd_status_t ssd_block_norm_fwd(const ssd_block_shape_t *shape, ssd_dtype_t io, const void *x, const void *residual,
                                const float *post_weight, const float *pre_weight, const void *z, const float *scale,
                                void *y, void *residual_out, const ssd_block_checkpoint_t *checkpoint, void *stream) {
    SSD_TRY(check_block(shape, io));
    const size_t e = io_size(io);
    SSD_TRY(need("x", x, e));
    SSD_TRY(need("residual", residual, e));
    SSD_TRY(maybe("post_weight", post_weight, 4));
    SSD_TRY(maybe("pre_weight", pre_weight, 4));
    SSD_TRY(maybe("z", z, e));
    SSD_TRY(maybe("scale", scale, 4));
    SSD_TRY(need("y", y, e));
    SSD_TRY(need("residual_out", residual_out, e));
    if (residual_out == residual && shape->rows > 1 && shape->residual_stride > shape->columns)
        return fail(SSD_ERR_UNSUPPORTED, "residual_out is dense: it cannot be a residual of stride %lld",
                    (long long)shape->residual_stride);
    if (checkpoint) SSD_TRY(check_checkpoint(checkpoint, z != nullptr));
    ssd::BlockArgs a = block_args(shape, io, x, z, residual, post_weight, pre_weight, scale, (hipStream_t)stream);
    a.y = y;
    a.residual_out = residual_out;
    if (checkpoint) use_checkpoint(a, checkpoint);
    const int64_t dense = shape->columns * (int64_t)e;
    // (with a checkpoint as without: it changes nothing in y)
    const bool wide = multiples(shape, io, 4).in(x, a.xs).in(z, a.zs).in(residual, a.rs)
                          .in(residual_out, dense).in(y, dense).ok;
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_block_fwd(io == SSD_BF16, wide, a, (hipStream_t)stream);
    return launched("ssd_block_norm_fwd");
}

size_t ssd_block_norm_bwd_workspace_bytes(const ssd_block_shape_t *shape, ssd_dtype_t io) {
    return check_block(shape, io) == SSD_OK ? block_bwd_bytes(shape, nullptr) : 0;
}

ssd_status_t ssd_block_norm_bwd(const ssd_block_shape_t *shape, ssd_dtype_t io, const void *x, const void *residual_out,
                                const float *post_weight, const float *pre_weight, const void *z, const float *scale,
                                const void *dy, const void *dresidual_out, const ssd_block_checkpoint_t *checkpoint,
                                void *dx, void *dresidual, void *dz, float *dpost_weight, float *dpre_weight,
                                float *dscale, void *workspace, size_t workspace_bytes, void *stream) {
    SSD_TRY(check_block(shape, io));
    const size_t e = io_size(io);
    if (checkpoint) {
        if (x || residual_out || z) return fail(SSD_ERR_UNSUPPORTED, "a checkpoint stands for x, residual_out and z");
        SSD_TRY(check_checkpoint(checkpoint, checkpoint->z != nullptr));
    } else {
        SSD_TRY(need("x", x, e));
        SSD_TRY(need("residual_out", residual_out, e));
        SSD_TRY(maybe("z", z, e));
    }
    const bool gate = checkpoint ? checkpoint->z != nullptr : z != nullptr;
    SSD_TRY(maybe("post_weight", post_weight, 4));
    SSD_TRY(maybe("pre_weight", pre_weight, 4));
    SSD_TRY(maybe("scale", scale, 4));
    SSD_TRY(need("dy", dy, e));
    SSD_TRY(maybe("dresidual_out", dresidual_out, e));
    SSD_TRY(need("dx", dx, e));
    SSD_TRY(need("dresidual", dresidual, e));
    SSD_TRY(maybe("dz", dz, e));
    SSD_TRY(maybe("dpost_weight", dpost_weight, 4));
    SSD_TRY(maybe("dpre_weight", dpre_weight, 4));
    SSD_TRY(maybe("dscale", dscale, 4));
    if (gate != (dz != nullptr)) return fail(SSD_ERR_NULL, "dz is given exactly when there is a gate");
    if (!post_weight != !dpost_weight) return fail(SSD_ERR_NULL, "dpost_weight is given exactly when post_weight is");
    if (!pre_weight != !dpre_weight) return fail(SSD_ERR_NULL, "dpre_weight is given exactly when pre_weight is");
    if (!scale != !dscale) return fail(SSD_ERR_NULL, "dscale is given exactly when scale is");
    const bool sums = dpost_weight || dpre_weight || dscale;
    if (sums) SSD_TRY(check_workspace(workspace, workspace_bytes, block_bwd_bytes(shape, (hipStream_t)stream)));
    ssd::BlockArgs a = block_args(shape, io, x, z, residual_out, post_weight, pre_weight, scale, (hipStream_t)stream);
    a.dy = dy;
    a.dresidual_out = dresidual_out;
    a.dx = dx;
    a.dresidual = dresidual;
    a.dz = dz;
    a.dpost = dpost_weight;
    a.dpre = dpre_weight;
    a.dscale = dscale;
    a.part = sums ? (float *)workspace : nullptr;
    if (checkpoint) use_checkpoint(a, checkpoint);
    const int64_t dense = shape->columns * (int64_t)e;
    // Rows of up to 4096 columns that are not whole 16-byte pieces go column by
    // column: more waves a row, fewer parts (1501 x 1477 fp32 20 us, 23 in pieces;
    // 30000 x 1003 205 and 219; but 5000 x 5001 189 and 165).
    const bool wide = (!checkpoint || a.code_words) &&
                      multiples(shape, io, shape->columns <= 4096 ? 16 : 4).in(x, a.xs).in(z, a.zs).in(residual_out, a.rs)
                          .in(dy, a.dys).in(dresidual_out, a.drs).in(dx, dense).in(dresidual, dense).in(dz, dense).ok;
    a.parts = block_parts(shape, wide, (hipStream_t)stream);
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_block_bwd(io == SSD_BF16, wide, a, (hipStream_t)stream);
    return launched("ssd_block_norm_bwd");
}

ssd_status_t ssd_mx4_quant(const ssd_mx4_shape_t *shape, ssd_dtype_t io, const void *x, void *q, void *scales,
                           void *stream) {
    SSD_TRY(check_mx4(shape, io, false));
    SSD_TRY(need("x", x, io_size(io)));
    SSD_TRY(check_operand("q", q, "scales", scales));
    ssd::Mx4QuantArgs a = quant_args(shape, io);
    a.x = x;
    a.q = (uint8_t *)q;
    a.scales = (uint32_t *)scales;
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_mx4_quant(io == SSD_BF16, a, (hipStream_t)stream);
    return launched("ssd_mx4_quant");
}

ssd_status_t ssd_mx4_dequant(const ssd_mx4_shape_t *shape, ssd_dtype_t io, const void *q, const void *scales, void *y,
                             void *stream) {
    SSD_TRY(check_mx4(shape, io, false));
    SSD_TRY(check_operand("q", q, "scales", scales));
    SSD_TRY(need("y", y, io_size(io)));
    if (shape->x_stride != 0) return fail(SSD_ERR_UNSUPPORTED, "x_stride must be zero: the output is dense");
    ssd::Mx4QuantArgs a = quant_args(shape, io);
    a.q = (uint8_t *)q;
    a.scales = (uint32_t *)scales;
    a.y = y;
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_mx4_dequant(io == SSD_BF16, a, (hipStream_t)stream);
    return launched("ssd_mx4_dequant");
}

ssd_status_t ssd_mx4_matmul(const ssd_mx4_shape_t *shape, ssd_dtype_t io, const void *q, const void *scales,
                            const void *wq, const void *wscales, const float *bias, void *y, void *stream) {
    SSD_TRY(check_mx4(shape, io, true));
    if (shape->x_stride != 0) return fail(SSD_ERR_UNSUPPORTED, "x_stride must be zero: 4-bit operands are dense");
    SSD_TRY(check_operand("q", q, "scales", scales));
    SSD_TRY(check_operand("wq", wq, "wscales", wscales));
    SSD_TRY(maybe("bias", bias, 4));
    SSD_TRY(need("y", y, io_size(io)));
    ssd::Mx4ProductArgs a = product_args(shape, wq, wscales, bias, y, (hipStream_t)stream);
    a.a = (const uint8_t *)q;
    a.as = (const uint32_t *)scales;
    (void)hipGetLastError();   // not an earlier call's
    ssd::launch_mx4_product(io == SSD_BF16, a, (hipStream_t)stream);
    return launched("ssd_mx4_matmul");
}

size_t ssd_mx4_linear_workspace_bytes(const ssd_mx4_shape_t *shape, ssd_dtype_t io) {
    return check_mx4(shape, io, true) == SSD_OK ? linear_bytes(shape) : 0;
}

ssd_status_t ssd_mx4_linear(const ssd_mx4_shape_t *shape, ssd_dtype_t io, const void *x, const void *wq,
                            const void *wscales, const float *bias, void *y, void *workspace, size_t workspace_bytes,
                            void *stream) {
    SSD_TRY(check_mx4(shape, io, true));
    SSD_TRY(need("x", x, io_size(io)));
    SSD_TRY(check_operand("wq", wq, "wscales", wscales));
    SSD_TRY(maybe("bias", bias, 4));
    SSD_TRY(need("y", y, io_size(io)));
    const size_t bytes = linear_bytes(shape);
    SSD_TRY(check_workspace(workspace, workspace_bytes, bytes));
    ssd::Mx4QuantArgs qa = quant_args(shape, io);
    qa.x = x;
    ssd::Mx4ProductArgs a = product_args(shape, wq, wscales, bias, y, (hipStream_t)stream);
    (void)hipGetLastError();   // not an earlier call's
    if (bytes == 0) {
        a.x = x;
        a.xs = qa.xs;
        ssd::launch_mx4_product(io == SSD_BF16, a, (hipStream_t)stream);
    } else {
        qa.q = (uint8_t *)workspace;
        qa.scales = (uint32_t *)((char *)workspace + linear_codes(shape));
        ssd::launch_mx4_quant(io == SSD_BF16, qa, (hipStream_t)stream);
        a.a = qa.q;
        a.as = qa.scales;
        ssd::launch_mx4_product(io == SSD_BF16, a, (hipStream_t)stream);
    }
    return launched("ssd_mx4_linear");
}

}  // extern "C"
