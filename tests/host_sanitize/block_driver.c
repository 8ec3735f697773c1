/* Drives every entry point of ssd_block_api.cpp (linked with block_stubs.cpp)
 * with host buffers of exactly the documented sizes. */
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "ssd.h"

extern unsigned long long g_block_launches;
const char *block_error(void);

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

#define CHECK(expr, launches)                                                           \
    do {                                                                                \
        const unsigned long long before = g_block_launches;                             \
        const int st_ = (int)(expr);                                                    \
        if (st_ != SSD_OK || g_block_launches != before + (launches)) {                 \
            printf("line %d: status %d (%s)\n", __LINE__, st_, block_error());          \
            return 1;                                                                   \
        }                                                                               \
    } while (0)

static void *act(size_t rows, size_t columns, size_t stride, size_t e) {
    return buf(((rows - 1) * (stride ? stride : columns) + columns) * e);
}

static int block(int64_t rows, int64_t D, int64_t stride, ssd_dtype_t io, int gate, int weights, int ckpt) {
    const size_t e = io == SSD_BF16 ? 2 : 4, nb = (size_t)((D + 127) / 128), n = (size_t)(rows * D);
    ssd_block_shape_t s = {rows, D, stride, 0, stride, 0, stride, 1e-5f, 1.f, {0}};
    void *x = act(rows, D, stride, e), *r = act(rows, D, stride, e), *z = gate ? act(rows, D, 0, e) : NULL;
    float *post = weights & 1 ? buf(4 * D) : NULL, *pre = weights & 2 ? buf(4 * D) : NULL;
    float *scale = weights & 4 ? buf(4 * D) : NULL;
    ssd_block_checkpoint_t c = {buf(n), buf(4 * rows * nb), gate ? buf(n) : NULL, gate ? buf(4 * rows * nb) : NULL, buf(n),
                                buf(4 * rows * nb)};
    CHECK(ssd_block_norm_fwd(&s, io, x, r, post, pre, z, scale, buf(n * e), buf(n * e), ckpt ? &c : NULL, NULL), 1);
    const size_t ws = weights ? ssd_block_norm_bwd_workspace_bytes(&s, io) : 0;
    CHECK(ssd_block_norm_bwd(&s, io, ckpt ? NULL : x, ckpt ? NULL : r, post, pre, ckpt ? NULL : z, scale, act(rows, D, 0, e),
                             gate ? act(rows, D, stride, e) : NULL, ckpt ? &c : NULL, buf(n * e), buf(n * e),
                             gate ? buf(n * e) : NULL, post ? buf(4 * D) : NULL, pre ? buf(4 * D) : NULL,
                             scale ? buf(4 * D) : NULL, ws ? buf(ws) : NULL, ws, NULL), 1);
    drop();
    return 0;
}

static int mx4(int64_t rows, int64_t K, int64_t N, int64_t stride, ssd_dtype_t io, int bias) {
    const size_t e = io == SSD_BF16 ? 2 : 4, kb = (size_t)((K + 127) / 128);
    ssd_mx4_shape_t s = {rows, K, 0, stride, {0}};
    void *x = act(rows, K, stride, e), *q = buf(rows * kb * 64), *sc = buf(rows * kb * 4);
    CHECK(ssd_mx4_quant(&s, io, x, q, sc, NULL), 1);
    s.x_stride = 0;
    CHECK(ssd_mx4_dequant(&s, io, q, sc, buf(rows * K * e), NULL), 1);
    s.outputs = N;
    void *wq = buf(N * kb * 64), *wsc = buf(N * kb * 4), *y = buf(rows * N * e);
    float *b = bias ? buf(4 * N) : NULL;
    CHECK(ssd_mx4_matmul(&s, io, q, sc, wq, wsc, b, y, NULL), 1);
    s.x_stride = stride;
    const size_t ws = ssd_mx4_linear_workspace_bytes(&s, io);
    CHECK(ssd_mx4_linear(&s, io, x, wq, wsc, b, y, ws ? buf(ws) : NULL, ws, NULL), ws ? 2 : 1);
    drop();
    return 0;
}

int main(void) {
    const int64_t rows[] = {1, 2, 5, 700}, widths[] = {1, 8, 33, 128, 200, 1000};
    for (int t = 0; t < 2; ++t)
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 6; ++j) {
                const ssd_dtype_t io = t ? SSD_BF16 : SSD_F32;
                for (int o = 0; o < 32; ++o)
                    if (block(rows[i], widths[j], o % 3 ? 0 : widths[j] + 8, io, o & 1, (o >> 1) & 7, o >> 4)) return 1;
                for (int o = 0; o < 4; ++o)
                    if (mx4(rows[i], widths[j], 1 + 77 * o, o % 2 ? 0 : widths[j] + 3, io, o >> 1)) return 1;
            }
    for (int64_t m = 14; m < 70; ++m)
        if (mx4(m, 130, 20, 0, SSD_BF16, 0)) return 1;
    if (block(3, 16384, 0, SSD_BF16, 1, 7, 1) || block(3, 16383, 0, SSD_F32, 1, 7, 0)) return 1;
    printf("all checks passed: %llu launches\n", g_block_launches);
    return 0;
}
