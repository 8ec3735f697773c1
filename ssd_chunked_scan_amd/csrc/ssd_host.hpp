// Host helpers of the layer operators' entry points: the error message, the
// checks of arguments that they share and what they derive from them.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "ssd.h"

namespace ssd {
void set_last_error(const char *msg);
int compute_units(hipStream_t stream);
}  // namespace ssd

namespace {

ssd_status_t fail(ssd_status_t st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    ssd::set_last_error(buf);
    return st;
}

constexpr int64_t kMaxTokens = ((int64_t)1 << 30) - 1;
constexpr int64_t kMaxChannels = (int64_t)1 << 20;
// Strides in elements: a round of 128 tokens is addressed with 32-bit byte
// offsets; single tokens and rows of the norm with 64-bit ones.
constexpr int64_t kMaxStride = (int64_t)1 << 22, kMaxRowStride = (int64_t)1 << 40;
constexpr int64_t kMaxSpan = (int64_t)1 << 60;
constexpr int64_t kMaxThreads = 0xffffffff;          // of one launch
constexpr int64_t kMaxGrid = kMaxThreads / 256;      // workgroups of 256 threads
constexpr int64_t kMaxNormWidth = 16384;             // columns of a norm group: held in registers

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
size_t io_size(ssd_dtype_t io) { return io == SSD_BF16 ? 2 : 4; }

ssd_status_t check_io(ssd_dtype_t io) {
    if (io != SSD_F32 && io != SSD_BF16) return fail(SSD_ERR_UNSUPPORTED, "unknown io dtype %d", (int)io);
    return SSD_OK;
}

ssd_status_t check_reserved(const int64_t (&r)[4]) {
    for (int64_t v : r)
        if (v != 0) return fail(SSD_ERR_UNSUPPORTED, "reserved shape fields must be zero");
    return SSD_OK;
}

ssd_status_t check_tokens(int64_t batch, int64_t seqlen, int64_t channels) {
    if (batch < 1 || seqlen < 1 || channels < 1)
        return fail(SSD_ERR_SHAPE, "sizes must be >= 1 (%lld x %lld tokens, %lld channels)", (long long)batch,
                    (long long)seqlen, (long long)channels);
    if (batch > kMaxTokens || seqlen > kMaxTokens || batch * seqlen > kMaxTokens || channels > kMaxChannels)
        return fail(SSD_ERR_UNSUPPORTED, "problem too large: %lld x %lld tokens, %lld channels", (long long)batch,
                    (long long)seqlen, (long long)channels);
    return SSD_OK;
}

// A token stride in elements (0: dense) of `tokens` tokens, `apart` of them in
// one row.
ssd_status_t check_stride(const char *name, int64_t stride, int64_t channels, int64_t tokens, int64_t apart) {
    if (stride != 0 && stride < channels)
        return fail(SSD_ERR_SHAPE, "%s_stride %lld is below the %lld elements of a token", name, (long long)stride,
                    (long long)channels);
    if (stride > (apart > 1 ? kMaxStride : kMaxRowStride) || stride > kMaxSpan / tokens)
        return fail(SSD_ERR_UNSUPPORTED, "%s_stride %lld is too large", name, (long long)stride);
    return SSD_OK;
}

int64_t stride_bytes(int64_t stride, int64_t channels, ssd_dtype_t io) {
    return (stride ? stride : channels) * (int64_t)io_size(io);
}

ssd_status_t need(const char *name, const void *p, size_t align) {
    if (!p) return fail(SSD_ERR_NULL, "%s is NULL", name);
    if (!aligned(p, align)) return fail(SSD_ERR_ALIGN, "%s must be %zu-byte aligned", name, align);
    return SSD_OK;
}

ssd_status_t maybe(const char *name, const void *p, size_t align) {
    return p ? need(name, p, align) : SSD_OK;
}

ssd_status_t check_workspace(const void *ws, size_t have, size_t want) {
    if (want == 0) return SSD_OK;
    if (!ws || have < want) return fail(SSD_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", want, ws ? have : 0);
    if (!aligned(ws, 16)) return fail(SSD_ERR_ALIGN, "workspace must be 16-byte aligned");
    return SSD_OK;
}

ssd_status_t launched(const char *what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(SSD_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
    return SSD_OK;
}

// Whether accesses of `n` elements of the io type are aligned in every tensor
// (a NULL one does not matter).
struct Access {
    bool ok;
    size_t bytes;
    Access(bool ok_, int n, ssd_dtype_t io) : ok(ok_), bytes(n * io_size(io)) {}
    Access &in(const void *p, int64_t stride) {
        ok = ok && (!p || (aligned(p, bytes) && stride % (int64_t)bytes == 0));
        return *this;
    }
};

// 16-byte accesses: 8 bf16 or 4 fp32 elements.
int wide_of(ssd_dtype_t io) { return io == SSD_BF16 ? 8 : 4; }

#define SSD_TRY(expr)                              \
    do {                                           \
        const ssd_status_t st_ = (expr);           \
        if (st_ != SSD_OK) return st_;             \
    } while (0)

}  // namespace
