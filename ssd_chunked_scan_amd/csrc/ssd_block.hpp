// Arguments of the block norm's kernels (ssd.h, ssd_block_norm_*).  Strides are
// in bytes between rows.
#pragma once

#include <stdint.h>

namespace ssd {

struct BlockArgs {
    const void *x, *z, *residual;       // forward; backward: residual is the stream s
    int64_t xs, zs, rs;
    const float *post, *pre, *scale;    // [columns], nullable
    void *y, *residual_out;             // forward
    const void *dy, *dresidual_out;     // backward; the latter nullable
    int64_t dys, drs;
    void *dx, *dz, *dresidual;          // backward
    float *dpost, *dpre, *dscale;       // backward, nullable
    float *part;                        // backward: [parts][2][pitch], null without a column sum to give
    uint8_t *xq, *zq, *sq;              // checkpoints: e4m3 [rows][columns], null without
    float *xsc, *zsc, *ssc;             // [rows][ceil(columns / 128)]
    float eps, alpha;
    int64_t rows;
    int columns, cus;
    int pitch;                          // columns up to whole packs of 8
    int parts;                          // backward: workgroups
    bool code_words;                    // a checkpoint's rows of codes are whole 4-byte words
};

}  // namespace ssd
