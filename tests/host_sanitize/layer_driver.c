/* Drives every entry point of ssd_layer_api.cpp (linked with layer_stubs.cpp)
 * with host buffers of exactly the documented sizes. */
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "ssd.h"

extern unsigned long long g_layer_launches;
extern int g_layer_fast;
const char *layer_error(void);

static void *keep[64];
static int kept;

static void *buf(size_t n) {
    void *p = NULL;
    if (posix_memalign(&p, 256, n ? n : 1)) abort();
    memset(p, 1, n);
    keep[kept++] = p;
    return p;
}

static void drop(void) {
    while (kept) free(keep[--kept]);
}

#define CHECK(expr)                                                                     \
    do {                                                                                \
        const unsigned long long before = g_layer_launches;                             \
        const int st_ = (int)(expr);                                                    \
        if (st_ != SSD_OK || g_layer_launches != before + 1) {                          \
            printf("line %d: status %d (%s)\n", __LINE__, st_, layer_error());          \
            return 1;                                                                   \
        }                                                                               \
    } while (0)

/* a tensor of `tokens` tokens, `stride` elements apart, that ends with its last one */
static void *act(size_t tokens, size_t channels, size_t stride, size_t e) {
    return buf(((tokens - 1) * (stride ? stride : channels) + channels) * e);
}

static int glr(int64_t b, int64_t L, int64_t D, int64_t stride, ssd_dtype_t io, int opt) {
    const size_t e = io == SSD_BF16 ? 2 : 4, n = (size_t)(b * L);
    ssd_glr_shape_t s = {b, L, D, stride, 0, stride, 0, opt, {0}};
    void *x = act(n, D, stride, e), *g = act(n, D, 0, e), *z = opt ? act(n, D, stride, e) : NULL;
    float *A = buf(4 * D), *bias = opt ? buf(4 * D) : NULL, *init = opt ? buf(4 * b * D) : NULL;
    int32_t *seq = opt ? buf(4 * n) : NULL;
    size_t ws = ssd_glr_fwd_workspace_bytes(&s, io);
    CHECK(ssd_glr_fwd(&s, io, x, g, A, bias, z, seq, init, buf(n * D * e), opt ? buf(4 * b * D) : NULL,
                      ws ? buf(ws) : NULL, ws, NULL));
    if (g_layer_fast != (D % 2 == 0 && stride % 2 == 0)) return printf("unexpected access width\n"), 1;
    ws = ssd_glr_bwd_workspace_bytes(&s, io);
    CHECK(ssd_glr_bwd(&s, io, x, g, A, bias, z, seq, init, act(n, D, 0, e), opt ? buf(4 * b * D) : NULL, buf(n * D * e),
                      buf(n * D * e), z ? buf(n * D * e) : NULL, buf(4 * D), bias ? buf(4 * D) : NULL,
                      init ? buf(4 * b * D) : NULL, buf(ws), ws, NULL));
    drop();
    s.seqlen = 1;
    CHECK(ssd_glr_step(&s, io, act(b, D, stride, e), act(b, D, 0, e), buf(4 * D), NULL, opt ? act(b, D, stride, e) : NULL,
                       buf(4 * b * D), buf(b * D * e), NULL));
    drop();
    return 0;
}

static int conv(int64_t b, int64_t L, int64_t D, int64_t W, int64_t stride, ssd_dtype_t io, int opt) {
    const size_t e = io == SSD_BF16 ? 2 : 4, n = (size_t)(b * L), win = (size_t)(b * (W - 1) * D);
    ssd_conv_shape_t s = {b, L, D, W, stride, 0, opt, {0}};
    void *x = act(n, D, stride, e), *init = opt ? buf(win * e) : NULL;
    float *w = buf(4 * D * W), *bias = opt ? buf(4 * D) : NULL;
    int32_t *seq = opt ? buf(4 * n) : NULL;
    CHECK(ssd_conv_fwd(&s, io, x, w, bias, seq, init, buf(n * D * e), opt ? buf(win * e) : NULL, NULL));
    const size_t ws = ssd_conv_bwd_workspace_bytes(&s, io);
    CHECK(ssd_conv_bwd(&s, io, x, w, bias, seq, init, act(n, D, 0, e), opt ? buf(4 * win) : NULL, buf(n * D * e),
                       buf(4 * D * W), bias ? buf(4 * D) : NULL, init ? buf(4 * win) : NULL, buf(ws), ws, NULL));
    drop();
    s.seqlen = 1;
    CHECK(ssd_conv_step(&s, io, act(b, D, stride, e), buf(4 * D * W), NULL, buf(win * e), buf(b * D * e), NULL));
    drop();
    return 0;
}

static int norm(int64_t rows, int64_t D, int64_t G, int64_t stride, ssd_dtype_t io, int kind) {
    const size_t e = io == SSD_BF16 ? 2 : 4;
    ssd_norm_shape_t s = {rows, D, G, stride, 0, stride, 0, 0, 1e-5f, 0, {0}};
    void *x = act(rows, D, stride, e), *r = kind == 1 ? act(rows, D, stride, e) : NULL;
    void *z = kind == 2 ? act(rows, D, 0, e) : NULL, *ro = r ? buf(rows * D * e) : NULL;
    float *w = kind ? buf(4 * D) : NULL;
    CHECK(ssd_norm_fwd(&s, io, x, w, r, z, buf(rows * D * e), ro, NULL));
    for (s.quant_block = 0; s.quant_block <= 128; s.quant_block += 128) {
        const size_t nb = s.quant_block ? (size_t)((D / G + 127) / 128) : 1;
        CHECK(ssd_norm_quant_fwd(&s, io, x, w, r, z, buf(rows * D), buf(4 * rows * G * nb), ro, NULL));
    }
    s.quant_block = 0;
    const size_t ws = w ? ssd_norm_bwd_workspace_bytes(&s, io) : 0;
    CHECK(ssd_norm_bwd(&s, io, x, w, z, act(rows, D, 0, e), kind == 1 ? act(rows, D, 0, e) : NULL, buf(rows * D * e),
                       z ? buf(rows * D * e) : NULL, w ? buf(4 * D) : NULL, ws ? buf(ws) : NULL, ws, NULL));
    drop();
    return 0;
}

int main(void) {
    const int64_t lens[] = {1, 2, 63, 64, 65, 129, 1000}, widths[] = {1, 2, 33, 64, 200};
    for (int t = 0; t < 2; ++t)
        for (int o = 0; o < 2; ++o)
            for (int i = 0; i < 7; ++i)
                for (int j = 0; j < 5; ++j) {
                    const ssd_dtype_t io = t ? SSD_BF16 : SSD_F32;
                    const int64_t D = widths[j];
                    if (glr(1 + i % 3, lens[i], D, 0, io, o) || glr(2, lens[i], D, D + 7, io, o)) return 1;
                    for (int64_t W = 2; W <= 4; ++W)
                        if (conv(1 + i % 3, lens[i], D, W, 0, io, o) || conv(2, lens[i], D, W, D + 2, io, o)) return 1;
                }
    for (int t = 0; t < 2; ++t)
        for (int kind = 0; kind < 3; ++kind)
            for (int j = 0; j < 5; ++j)
                for (int64_t G = 1; G <= 3; ++G) {
                    const ssd_dtype_t io = t ? SSD_BF16 : SSD_F32;
                    const int64_t D = widths[j] * G;
                    if (norm(1, D, G, 0, io, kind) || norm(700, D, G, D + 8, io, kind)) return 1;
                }
    if (norm(3, 16384, 1, 0, SSD_BF16, 1) || norm(3, 16383, 1, 0, SSD_F32, 2)) return 1;
    /* many splits, and the planner's edges */
    for (int64_t L = 255; L <= 520; L += 1)
        if (glr(1, L, 3, 0, SSD_F32, 1)) return 1;
    if (glr(1, 70000, 2, 0, SSD_F32, 1) || glr(300, 5, 64, 0, SSD_BF16, 1)) return 1;
    printf("all checks passed: %llu launches\n", g_layer_launches);
    return 0;
}
