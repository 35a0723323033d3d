// operators_api.cu - the C ABI of the operators that need no layer: routing
// from given logits (moe_route, moe_route_backward) and microscaled 4-bit rows
// and products (moe_mx_*). Argument checks, tensor maps, launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <utility>

#include "moe.h"
#include "moe_common.cuh"
#include "moe_kernels.cuh"
#include "mx_common.cuh"
#include "route_scores.cuh"

using namespace moe;

namespace {

int fail(int code, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return report_error(code, buf);
}

// Streaming multiprocessors of the current device, which has to be an sm_100
// one; looked up once per device.
int device_sms(int *sms) {
    static std::atomic<int> known[64];
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0) return fail(MOE_ERR_CUDA, "no CUDA device: %s", cudaGetErrorString(e));
    std::atomic<int> &slot = known[dev & 63];
    *sms = dev < 64 ? slot.load(std::memory_order_relaxed) : 0;
    if (*sms > 0) return MOE_OK;
    int major = 0, minor = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "device %d: %s", dev, cudaGetErrorString(e));
    if (major != 10 || minor != 0)
        return fail(MOE_ERR_CUDA, "device %d is sm_%d%d; this library is built for sm_100a", dev, major, minor);
    if (dev < 64) slot.store(*sms, std::memory_order_relaxed);
    return MOE_OK;
}

cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }
bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool overlap(const void *p, size_t np, const void *q, size_t nq) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return np && nq && a < b + nq && b < a + np;
}

// Whether two matrices of T rows of `width` bytes, lp and lq (at least `width`) apart, have a byte in common.
// Rows between those of the other matrix (columns of one buffer) are none.
bool rows_overlap(const void *p, int64_t lp, const void *q, int64_t lq, int64_t T, int64_t width) {
    using wide = __int128;
    wide a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    if (a < b) {
        std::swap(a, b);
        std::swap(lp, lq);
    }
    if (T <= 0 || a >= b + (wide)(T - 1) * lq + width) return false;
    // Row i of the matrix that begins later lies behind row j of the other one. With the same stride i = 0 speaks for all.
    for (int64_t i = 0; i < (lp == lq ? 1 : T); ++i) {
        const wide from = a + (wide)i * lp - b, j = from / lq, off = from % lq;
        if (j >= T) break;
        if (off < width || (j + 1 < T && off + width > lq)) return true;
    }
    return false;
}

int launched(cudaError_t e, const char *what) {
    return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "%s failed: %s", what, cudaGetErrorString(e));
}

}  // namespace

namespace moe {
int check_route_config(const moe_route_config_t *c) {
    if (!c) return fail(MOE_ERR_INVALID_ARG, "cfg is NULL");
    if (c->num_experts < 1) return fail(MOE_ERR_INVALID_ARG, "num_experts must be >= 1 (got %d)", c->num_experts);
    if (c->num_experts > kRouteMaxExperts)
        return fail(MOE_ERR_UNSUPPORTED, "num_experts > %d is not supported (got %d)", kRouteMaxExperts, c->num_experts);
    if (c->num_active < 1 || c->num_active > c->num_experts)
        return fail(MOE_ERR_INVALID_ARG, "num_active must be in 1..num_experts (got %d, E=%d)", c->num_active,
                    c->num_experts);
    if (c->num_active > kRouteMaxActive)
        return fail(MOE_ERR_UNSUPPORTED, "num_active > %d is not supported", kRouteMaxActive);
    if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID)
        return fail(MOE_ERR_INVALID_ARG, "unknown score %d", c->score);
    if (c->num_groups < 1 || c->num_experts % c->num_groups)
        return fail(MOE_ERR_INVALID_ARG, "num_groups must divide num_experts (got %d, E=%d)", c->num_groups,
                    c->num_experts);
    if (c->num_groups > kRouteMaxGroups)
        return fail(MOE_ERR_UNSUPPORTED, "num_groups > %d is not supported", kRouteMaxGroups);
    if (c->top_groups < 1 || c->top_groups > c->num_groups)
        return fail(MOE_ERR_INVALID_ARG, "top_groups must be in 1..num_groups (got %d of %d)", c->top_groups,
                    c->num_groups);
    if (c->group_top != 1 && c->group_top != 2)
        return fail(MOE_ERR_INVALID_ARG, "group_top must be 1 or 2 (got %d)", c->group_top);
    if (c->num_active > c->num_experts / c->num_groups * c->top_groups)
        return fail(MOE_ERR_INVALID_ARG, "num_active (%d) exceeds the experts of top_groups (%d) groups", c->num_active,
                    c->top_groups);
    if (c->renormalize != 0 && c->renormalize != 1) return fail(MOE_ERR_INVALID_ARG, "renormalize must be 0 or 1");
    if (!std::isfinite(c->scale)) return fail(MOE_ERR_INVALID_ARG, "scale must be finite");
    if (c->dtype != MOE_DTYPE_BF16 && c->dtype != MOE_DTYPE_FP32)
        return fail(MOE_ERR_INVALID_ARG, "unknown dtype %d", c->dtype);
    return MOE_OK;
}

RouteArgs route_args(const moe_route_config_t &c) {
    RouteArgs a;
    a.E = c.num_experts;
    a.k = c.num_active;
    a.sigmoid = c.score == MOE_SCORE_SIGMOID;
    a.groups = c.num_groups;
    a.top_groups = c.top_groups;
    a.group_top = c.group_top;
    a.renormalize = c.renormalize;
    a.scale = c.scale;
    return a;
}
}  // namespace moe

namespace {

int check_rows(const moe_route_config_t *c, const void *logits, int64_t ld, int32_t T, const char *name) {
    const size_t es = c->dtype == MOE_DTYPE_BF16 ? 2 : 4;
    if (T > 0 && !logits) return fail(MOE_ERR_INVALID_ARG, "%s is required when T > 0", name);
    if (!aligned(logits, es)) return fail(MOE_ERR_INVALID_ARG, "%s must be aligned to its elements", name);
    if (ld < c->num_experts) return fail(MOE_ERR_INVALID_ARG, "%s: row stride below num_experts", name);
    return MOE_OK;
}

// The kernels look up to a tile past a row or an element with 32-bit numbers.
constexpr int kMxMaxRows = INT32_MAX - 1023, kMxMaxCols = 1 << 30;

int check_mx(int format, int64_t rows, int64_t cols) {
    if (format != MOE_MX_MXFP4 && format != MOE_MX_NVFP4) return fail(MOE_ERR_INVALID_ARG, "unknown format %d", format);
    if (rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows must be >= 0 (got %lld)", (long long)rows);
    if (rows > kMxMaxRows || cols > kMxMaxCols)
        return fail(MOE_ERR_UNSUPPORTED, "%lld rows of %lld elements: at most %d of %d are supported", (long long)rows,
                    (long long)cols, kMxMaxRows, kMxMaxCols);
    if (cols < 32 || cols % 32)
        return fail(MOE_ERR_INVALID_ARG, "a row must have a positive multiple of 32 elements (got %lld)",
                    (long long)cols);
    return MOE_OK;
}

int check_exp(int e) {
    return e < -60 || e > 60 ? fail(MOE_ERR_INVALID_ARG, "scale_exp must be in -60..60 (got %d)", e) : MOE_OK;
}

int block_of(int format) { return format == MOE_MX_MXFP4 ? 32 : 16; }

// Checks a quantisation's arguments and fills the kernel's.
int quantize_args(MxQuantArgs *a, int32_t format, const void *x, int32_t dtype, int64_t ld, int32_t x_rows, int32_t cols,
                  const int32_t *row_index, int32_t rows, int32_t scale_exp, void *codes, void *scales) {
    int rc = check_mx(format, rows, cols);
    if (rc != MOE_OK) return rc;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP32) return fail(MOE_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (x_rows < 0) return fail(MOE_ERR_INVALID_ARG, "x_rows must be >= 0 (got %d)", x_rows);
    if (!row_index && rows != x_rows)
        return fail(MOE_ERR_INVALID_ARG, "without row_index, rows (%d) must equal x_rows (%d)", rows, x_rows);
    if (ld < cols) return fail(MOE_ERR_INVALID_ARG, "x: row stride below cols");
    if ((rc = check_exp(scale_exp)) != MOE_OK) return rc;
    if (rows > 0 && ((!x && x_rows > 0) || !codes || !scales))
        return fail(MOE_ERR_INVALID_ARG, "x, codes and scales (or the workspace) are required when rows > 0");
    if (!aligned(x, dtype == MOE_DTYPE_BF16 ? 2 : 4) || !aligned(row_index, 4))
        return fail(MOE_ERR_INVALID_ARG, "x and row_index must be aligned to their elements");
    if (!aligned(codes, 16) || !aligned(scales, 16))
        return fail(MOE_ERR_INVALID_ARG, "codes, scales and the workspace must be 16-byte aligned");
    a->x = x;
    a->ld = ld;
    a->x_rows = x_rows;
    a->row_index = row_index;
    a->rows = rows;
    a->cols = cols;
    a->pre = std::ldexp(1.f, -scale_exp);
    a->codes = static_cast<uint8_t *>(codes);
    a->scales = static_cast<uint8_t *>(scales);
    a->values = nullptr;
    a->values_ld = 0;
    a->post = std::ldexp(1.f, scale_exp);
    return MOE_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------ routing

moe_route_config_t moe_route_config_default(void) {
    moe_route_config_t c;
    c.num_experts = 8;
    c.num_active = 2;
    c.score = MOE_SCORE_SOFTMAX;
    c.num_groups = 1;
    c.top_groups = 1;
    c.group_top = 2;
    c.renormalize = 1;
    c.scale = 1.f;
    c.dtype = MOE_DTYPE_FP32;
    return c;
}

int moe_route(const moe_route_config_t *cfg, const void *logits, int64_t ld, int32_t T, const float *bias,
              float *weights, int32_t *topk_idx, int32_t *counts, void *stream_v) {
    report_error(MOE_OK, "");
    int rc = check_route_config(cfg);
    if (rc != MOE_OK) return rc;
    if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T must be >= 0 (got %d)", T);
    if ((rc = check_rows(cfg, logits, ld, T, "logits")) != MOE_OK) return rc;
    if (T > 0 && (!weights || !topk_idx)) return fail(MOE_ERR_INVALID_ARG, "weights and topk_idx are required");
    if (!aligned(bias, 4) || !aligned(weights, 4) || !aligned(topk_idx, 4) || !aligned(counts, 4))
        return fail(MOE_ERR_INVALID_ARG, "arrays must be 4-byte aligned");
    int sms = 0;
    if ((rc = device_sms(&sms)) != MOE_OK) return rc;
    RouteArgs a = route_args(*cfg);
    a.logits = logits;
    a.ld = ld;
    a.T = T;
    a.bias = bias;
    a.weights = weights;
    a.idx = topk_idx;
    a.counts = counts;
    return launched(launch_route(a, cfg->dtype == MOE_DTYPE_BF16, sms, as_stream(stream_v)), "moe_route");
}

int moe_route_backward(const moe_route_config_t *cfg, const float *grad_weights, const void *logits, int64_t ld,
                       const int32_t *topk_idx, int32_t T, void *grad_logits, int64_t grad_ld, void *stream_v) {
    report_error(MOE_OK, "");
    int rc = check_route_config(cfg);
    if (rc != MOE_OK) return rc;
    if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T must be >= 0 (got %d)", T);
    if ((rc = check_rows(cfg, logits, ld, T, "logits")) != MOE_OK) return rc;
    if ((rc = check_rows(cfg, grad_logits, grad_ld, T, "grad_logits")) != MOE_OK) return rc;
    if (T > 0 && (!grad_weights || !topk_idx))
        return fail(MOE_ERR_INVALID_ARG, "grad_weights and topk_idx are required");
    if (!aligned(grad_weights, 4) || !aligned(topk_idx, 4))
        return fail(MOE_ERR_INVALID_ARG, "arrays must be 4-byte aligned");
    const int64_t es = cfg->dtype == MOE_DTYPE_BF16 ? 2 : 4;
    if (rows_overlap(logits, T == 1 ? cfg->num_experts * es : ld * es, grad_logits,
                     T == 1 ? cfg->num_experts * es : grad_ld * es, T, cfg->num_experts * es))
        return fail(MOE_ERR_INVALID_ARG, "grad_logits may not overlap logits");
    int sms = 0;
    if ((rc = device_sms(&sms)) != MOE_OK) return rc;
    RouteBackwardArgs a;
    a.grad_weights = grad_weights;
    a.logits = logits;
    a.ld = ld;
    a.idx = topk_idx;
    a.T = T;
    a.E = cfg->num_experts;
    a.k = cfg->num_active;
    a.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
    a.renormalize = cfg->renormalize;
    a.scale = cfg->scale;
    a.grad_logits = grad_logits;
    a.grad_ld = grad_ld;
    return launched(launch_route_backward(a, cfg->dtype == MOE_DTYPE_BF16, sms, as_stream(stream_v)),
                    "moe_route_backward");
}

// ------------------------------------------------------------ microscaled 4-bit rows

size_t moe_mx_codes_bytes(int64_t rows, int64_t cols) {
    return rows < 0 || cols < 32 || cols % 32 ? 0 : (size_t)rows * (size_t)(cols / 2);
}

size_t moe_mx_scales_bytes(int32_t format, int64_t rows, int64_t cols) {
    if ((format != MOE_MX_MXFP4 && format != MOE_MX_NVFP4) || rows < 0 || cols < 32 || cols % 32) return 0;
    const int64_t tile_k = 4 * block_of(format);
    return (size_t)((rows + 127) / 128) * (size_t)((cols + tile_k - 1) / tile_k) * 512;
}

int moe_mx_quantize(int32_t format, const void *x, int32_t dtype, int64_t ld, int32_t x_rows, int32_t cols,
                    const int32_t *row_index, int32_t rows, int32_t scale_exp, void *codes, void *scales, void *values,
                    int64_t values_ld, void *stream_v) {
    report_error(MOE_OK, "");
    MxQuantArgs a;
    int rc = quantize_args(&a, format, x, dtype, ld, x_rows, cols, row_index, rows, scale_exp, codes, scales);
    if (rc != MOE_OK) return rc;
    if (values && values_ld < cols) return fail(MOE_ERR_INVALID_ARG, "values: row stride below cols");
    if (!aligned(values, dtype == MOE_DTYPE_BF16 ? 2 : 4))
        return fail(MOE_ERR_INVALID_ARG, "values must be aligned to its elements");
    if (rows == 0 || x_rows == 0) return MOE_OK;
    int sms = 0;
    if ((rc = device_sms(&sms)) != MOE_OK) return rc;
    a.values = values;
    a.values_ld = values_ld;
    return launched(launch_mx_quantize(a, format, dtype == MOE_DTYPE_BF16, sms, as_stream(stream_v)), "moe_mx_quantize");
}

size_t moe_mx_once_bytes(int32_t format, int64_t x_rows, int64_t cols) {
    if ((format != MOE_MX_MXFP4 && format != MOE_MX_NVFP4) || x_rows < 0 || cols < 32 || cols % 32) return 0;
    return (size_t)x_rows * (cols / 2 + 4 * mx_scale_tiles(static_cast<int>(std::min<int64_t>(cols, kMxMaxCols)), block_of(format)));
}

int moe_mx_quantize_once(int32_t format, const void *x, int32_t dtype, int64_t ld, int32_t x_rows, int32_t cols,
                         const int32_t *row_index, int32_t rows, int32_t scale_exp, void *codes, void *scales,
                         void *workspace, size_t ws_bytes, void *stream_v) {
    report_error(MOE_OK, "");
    MxQuantArgs a;
    int rc = quantize_args(&a, format, x, dtype, ld, x_rows, cols, nullptr, x_rows, scale_exp, workspace, workspace);
    if (rc != MOE_OK || (rc = check_mx(format, rows, cols)) != MOE_OK) return rc;
    if (rows > 0 && (!row_index || !codes || !scales))
        return fail(MOE_ERR_INVALID_ARG, "row_index, codes and scales are required when rows > 0");
    if (!aligned(row_index, 4)) return fail(MOE_ERR_INVALID_ARG, "row_index must be 4-byte aligned");
    if (!aligned(codes, 16) || !aligned(scales, 16))
        return fail(MOE_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
    if (ws_bytes < moe_mx_once_bytes(format, x_rows, cols))
        return fail(MOE_ERR_WORKSPACE, "workspace: %zu bytes given, %zu needed", ws_bytes,
                    moe_mx_once_bytes(format, x_rows, cols));
    const size_t used = moe_mx_once_bytes(format, x_rows, cols);
    if (overlap(workspace, used, codes, rows * (size_t)(cols / 2)) ||
        overlap(workspace, used, scales, moe_mx_scales_bytes(format, rows, cols)))
        return fail(MOE_ERR_INVALID_ARG, "the outputs may not overlap the workspace");
    if (rows == 0 || x_rows == 0) return MOE_OK;
    int sms = 0;
    if ((rc = device_sms(&sms)) != MOE_OK) return rc;
    a.scales = a.codes + (size_t)x_rows * (cols / 2);
    a.plain = true;
    rc = launched(launch_mx_quantize(a, format, dtype == MOE_DTYPE_BF16, sms, as_stream(stream_v)), "moe_mx_quantize_once");
    if (rc != MOE_OK) return rc;
    MxGatherArgs g;
    g.codes = a.codes;
    g.scales = a.scales;
    g.plain = true;
    g.src_rows = x_rows;
    g.rows = rows;
    g.cols = cols;
    g.row_index = row_index;
    g.out_codes = static_cast<uint8_t *>(codes);
    g.out_scales = static_cast<uint8_t *>(scales);
    return launched(launch_mx_gather(g, format, as_stream(stream_v)), "moe_mx_quantize_once");
}

int moe_mx_gather(int32_t format, const void *codes, const void *scales, int32_t src_rows, int32_t cols,
                  const int32_t *row_index, int32_t rows, void *out_codes, void *out_scales, void *stream_v) {
    report_error(MOE_OK, "");
    int rc = check_mx(format, rows, cols);
    if (rc != MOE_OK) return rc;
    if (src_rows < 0) return fail(MOE_ERR_INVALID_ARG, "src_rows must be >= 0 (got %d)", src_rows);
    if (rows > 0 && (!row_index || !out_codes || !out_scales || (src_rows > 0 && (!codes || !scales))))
        return fail(MOE_ERR_INVALID_ARG, "row_index, codes and scales are required when rows > 0");
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(out_codes, 16) || !aligned(out_scales, 16))
        return fail(MOE_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
    if (!aligned(row_index, 4)) return fail(MOE_ERR_INVALID_ARG, "row_index must be 4-byte aligned");
    const size_t row_bytes = cols / 2;
    if (overlap(codes, src_rows * row_bytes, out_codes, rows * row_bytes) ||
        overlap(scales, moe_mx_scales_bytes(format, src_rows, cols), out_scales, moe_mx_scales_bytes(format, rows, cols)))
        return fail(MOE_ERR_INVALID_ARG, "the outputs may not overlap the inputs");
    if (rows == 0 || src_rows == 0) return MOE_OK;
    int sms = 0;
    if ((rc = device_sms(&sms)) != MOE_OK) return rc;
    MxGatherArgs a;
    a.codes = static_cast<const uint8_t *>(codes);
    a.scales = static_cast<const uint8_t *>(scales);
    a.src_rows = src_rows;
    a.rows = rows;
    a.cols = cols;
    a.row_index = row_index;
    a.out_codes = static_cast<uint8_t *>(out_codes);
    a.out_scales = static_cast<uint8_t *>(out_scales);
    return launched(launch_mx_gather(a, format, as_stream(stream_v)), "moe_mx_gather");
}

int moe_mx_dequantize(int32_t format, const void *codes, const void *scales, int32_t rows, int32_t cols,
                      int32_t scale_exp, void *out, int32_t dtype, int64_t ld, void *stream_v) {
    report_error(MOE_OK, "");
    int rc = check_mx(format, rows, cols);
    if (rc != MOE_OK) return rc;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP32) return fail(MOE_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (ld < cols) return fail(MOE_ERR_INVALID_ARG, "out: row stride below cols");
    if ((rc = check_exp(scale_exp)) != MOE_OK) return rc;
    if (rows > 0 && (!codes || !scales || !out))
        return fail(MOE_ERR_INVALID_ARG, "codes, scales and out are required when rows > 0");
    if (!aligned(codes, 16) || !aligned(scales, 16))
        return fail(MOE_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
    if (!aligned(out, dtype == MOE_DTYPE_BF16 ? 2 : 4))
        return fail(MOE_ERR_INVALID_ARG, "out must be aligned to its elements");
    if (rows == 0) return MOE_OK;
    int sms = 0;
    if ((rc = device_sms(&sms)) != MOE_OK) return rc;
    MxDequantArgs a;
    a.codes = static_cast<const uint8_t *>(codes);
    a.scales = static_cast<const uint8_t *>(scales);
    a.rows = rows;
    a.cols = cols;
    a.post = std::ldexp(1.f, scale_exp);
    a.out = out;
    a.ld = ld;
    return launched(launch_mx_dequantize(a, format, dtype == MOE_DTYPE_BF16, as_stream(stream_v)), "moe_mx_dequantize");
}

int moe_mx_gemm(const moe_mx_gemm_t *p, void *stream_v) {
    report_error(MOE_OK, "");
    if (!p) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
    int rc = check_mx(p->format, p->rows, p->k);
    if (rc != MOE_OK) return rc;
    if (p->n < 1) return fail(MOE_ERR_INVALID_ARG, "n must be >= 1 (got %d)", p->n);
    if (p->groups < 1) return fail(MOE_ERR_INVALID_ARG, "groups must be >= 1 (got %d)", p->groups);
    if (p->groups > 1024) return fail(MOE_ERR_UNSUPPORTED, "groups > 1024 is not supported (got %d)", p->groups);
    if ((int64_t)p->groups * p->n > INT32_MAX - 1023)
        return fail(MOE_ERR_UNSUPPORTED, "groups x n must be below 2^31");
    if ((p->group_start == nullptr) != (p->group_rows == nullptr))
        return fail(MOE_ERR_INVALID_ARG, "group_start and group_rows go together");
    if (p->groups > 1 && !p->group_start) return fail(MOE_ERR_INVALID_ARG, "groups > 1 need group_start and group_rows");
    if (p->activation < MOE_ACT_NONE || p->activation > MOE_ACT_SWISH)
        return fail(MOE_ERR_INVALID_ARG, "unknown activation %d", p->activation);
    if (p->out_dtype != MOE_DTYPE_BF16 && p->out_dtype != MOE_DTYPE_FP32)
        return fail(MOE_ERR_INVALID_ARG, "unknown out_dtype %d", p->out_dtype);
    if (p->out_ld < p->n) return fail(MOE_ERR_INVALID_ARG, "out: row stride below n");
    if (p->scale_exp < -120 || p->scale_exp > 120)
        return fail(MOE_ERR_INVALID_ARG, "scale_exp must be in -120..120 (got %d)", p->scale_exp);
    if (p->rows > 0 && (!p->a_codes || !p->a_scales || !p->w_codes || !p->w_scales || !p->out))
        return fail(MOE_ERR_INVALID_ARG, "codes, scales and out are required when rows > 0");
    if (!aligned(p->a_codes, 16) || !aligned(p->a_scales, 16) || !aligned(p->w_codes, 16) || !aligned(p->w_scales, 16))
        return fail(MOE_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
    const int es = p->out_dtype == MOE_DTYPE_BF16 ? 2 : 4;
    if (!aligned(p->out, es)) return fail(MOE_ERR_INVALID_ARG, "out must be aligned to its elements");
    if (!aligned(p->group_start, 4) || !aligned(p->group_rows, 4) || !aligned(p->bias, 4) || !aligned(p->alpha, 4) ||
        !aligned(p->status, 4))
        return fail(MOE_ERR_INVALID_ARG, "group_start, group_rows, bias, alpha and status must be 4-byte aligned");
    if (p->rows == 0) return MOE_OK;
    MxGemmArgs a;
    a.group_start = p->group_start;
    a.group_rows = p->group_rows;
    a.rows = p->rows;
    a.N = p->n;
    a.K = p->k;
    a.G = p->groups;
    a.bias = p->bias;
    a.alpha = p->alpha;
    a.post = std::ldexp(1.f, p->scale_exp);
    a.act = p->activation;
    a.out = p->out;
    a.out_f32 = p->out_dtype == MOE_DTYPE_FP32;
    a.out_ld = p->out_ld;
    a.vec_ok = !a.out_f32 && aligned(p->out, 16) && p->out_ld % 8 == 0;
    a.status = p->status;
    // Rows beyond the 127 that each group's start may leave unused.
    a.filled = (int64_t)p->rows - (p->groups > 1 ? (int64_t)p->groups * 127 : 0);
    // Units are counted in 32 bits, even where (against the rule) every group claims all rows.
    const bool narrow = mx_gemm_narrow(a);
    const int64_t tiles = (int64_t)p->groups * (p->rows / (narrow ? 64 : 192) + 1);
    if (tiles * ((p->n + 127) / (narrow ? 128 : 256) + 1) > INT32_MAX - 65535)
        return fail(MOE_ERR_UNSUPPORTED, "%d rows x %d features in %d groups are too many", p->rows, p->n, p->groups);
    int sms = 0;
    if ((rc = device_sms(&sms)) != MOE_OK) return rc;
    MxMaps m;
    if (!encode_mx_maps(&m, narrow, p->format, p->a_codes, p->a_scales, p->rows, p->w_codes, p->w_scales, p->groups, p->n, p->k))
        return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed for the codes or scales");
    return launched(launch_mx_gemm(m, a, p->format, sms, as_stream(stream_v)), "moe_mx_gemm");
}

int moe_mx_status(void *stream_v) {
    report_error(MOE_OK, "");
    int sms = 0;
    int rc = device_sms(&sms);
    if (rc != MOE_OK) return rc;
    uint32_t bits = 0;
    if ((rc = launched(mx_take_status(&bits, as_stream(stream_v)), "moe_mx_status")) != MOE_OK) return rc;
    if (bits & kDevTimeout)
        return fail(MOE_ERR_TIMEOUT, "a bounded device-side wait of a product gave up (status 0x%x)", bits);
    if (bits & kDevBadGroup)
        return fail(MOE_ERR_INVALID_ARG, "a product's segment broke the bounds of its rows (status 0x%x)", bits);
    return MOE_OK;
}

}  // extern "C"
