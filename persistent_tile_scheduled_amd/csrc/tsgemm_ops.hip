// C ABI of the row operators and of the weight gradient (include/tsgemm.h):
// argument checks and launches.  Conventions as in tsgemm.hip.
#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "tsgemm.h"
#include "tsgemm_host.h"
#include "tsgemm_ops_launch.h"
#include "tsgemm_overlap.h"
#include "tsgemm_rows_kernel.h"
#include "tsgemm_wgrad_kernel.h"

namespace {

using tsg::fail;
using tsg::reset_error;

bool is_float(int dt) { return dt == TSGEMM_FP16 || dt == TSGEMM_BF16 || dt == TSGEMM_FP32; }
int bytes_of(int dt) { return dt == TSGEMM_FP32 ? 4 : 2; }
bool off(const void* p, unsigned align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1u)) != 0u; }

// rows and width of an activation; a width of 0 has no mean and no block.
int check_shape(int64_t rows, int64_t width) {
    if (rows < 0 || width < 0) return fail(TSGEMM_EINVAL, "rows and width must be >= 0");
    if (rows >= (int64_t(1) << 31) || width >= (int64_t(1) << 31)) return fail(TSGEMM_EINVAL, "rows and width must be below 2^31");
    return TSGEMM_OK;
}
int check_dtype(int dt, const char* what) {
    return is_float(dt) ? TSGEMM_OK
                        : fail(TSGEMM_EINVAL, "%s must be TSGEMM_FP16 (1), TSGEMM_BF16 (2) or TSGEMM_FP32 (4), got %d", what, dt);
}
// One matrix of floating values: given, aligned to its type, rows not overlapping.
int check_matrix(const char* name, const void* p, int64_t ld, int64_t width, int dt) {
    if (!p) return fail(TSGEMM_EINVAL, "%s is NULL", name);
    if (off(p, (unsigned)bytes_of(dt))) return fail(TSGEMM_EINVAL, "%s must be aligned to its type", name);
    if (ld < width) return fail(TSGEMM_EINVAL, "the row stride of %s (%lld) is below the width (%lld)", name, (long long)ld, (long long)width);
    return TSGEMM_OK;
}
int check_weights_dtype(int wdt, int dt) {
    if (wdt != dt && wdt != TSGEMM_FP32)
        return fail(TSGEMM_EINVAL, "the weights must be of the activation's type (%d) or TSGEMM_FP32, got %d", dt, wdt);
    return TSGEMM_OK;
}
int check_mx(int64_t width, const void* codes, const void* scales) {
    if (width % 32 != 0) return fail(TSGEMM_EINVAL, "MX blocks need a width divisible by 32, got %lld", (long long)width);
    if (!codes || !scales) return fail(TSGEMM_EINVAL, "codes or scales is NULL");
    if (off(codes, 16) || off(scales, 4)) return fail(TSGEMM_EINVAL, "codes must be 16-byte and scales 4-byte aligned");
    return TSGEMM_OK;
}
struct Named {
    const char* name;
    tsg::Region r;
    tsg::Extent e;
};
Named matrix(const char* name, const void* p, int64_t rows, int64_t width, int64_t ld, int bytes) {
    const tsg::Region r = {p, rows, width * bytes, ld * bytes};
    return {name, r, tsg::extent(r)};
}
Named stretch(const char* name, const void* p, int64_t bytes) { return matrix(name, p, 1, bytes, bytes, 1); }
// No output over an input or another output: workgroups read rows, some of them
// twice, while others already write.
int check_overlaps(std::initializer_list<Named> outputs, std::initializer_list<Named> inputs) {
    const auto clash = [](const Named& o, const Named& other) {  // nearly always the extents say no
        return o.e.from < other.e.to && other.e.from < o.e.to && tsg::overlap(o.r, other.r);
    };
    for (const Named& o : outputs) {
        for (const Named& i : inputs)
            if (clash(o, i)) return fail(TSGEMM_EINVAL, "%s overlaps %s", o.name, i.name);
        for (const Named* other = outputs.begin(); other != &o; ++other)
            if (clash(o, *other)) return fail(TSGEMM_EINVAL, "%s overlaps %s", o.name, other->name);
    }
    return TSGEMM_OK;
}
int launched(const char* what) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? TSGEMM_OK : fail(TSGEMM_EHIP, "%s launch failed: %s", what, hipGetErrorString(e));
}

uint32_t grad_pitch(int64_t width) { return (uint32_t)((width + 7) / 8 * 8); }

int check_weight_grad(int64_t rows, int64_t out, int64_t width) {
    int rc = check_shape(rows, width);
    if (rc != TSGEMM_OK) return rc;
    if (out < 0 || out >= (int64_t(1) << 31)) return fail(TSGEMM_EINVAL, "out must be in [0, 2^31)");
    if (width % 32 != 0) return fail(TSGEMM_EINVAL, "MX blocks need a width divisible by 32, got %lld", (long long)width);
    if (out % 8 != 0) return fail(TSGEMM_EINVAL, "out must be divisible by 8 (16-byte rows of dy), got %lld", (long long)out);
    if (width >= (int64_t(1) << 24) || out >= (int64_t(1) << 24))
        return fail(TSGEMM_EUNSUPPORTED, "out and width must be below 2^24 (32-bit offsets in a slab of 64 rows)");
    return TSGEMM_OK;
}

}  // namespace

extern "C" {

int tsgemm_layer_norm(int64_t rows, int64_t width, int dtype, int weight_dtype, const void* x, int64_t ldx, const void* gamma,
                      const void* beta, float eps, void* y, int64_t ldy, float* mean, float* rstd, void* codes, void* scales,
                      void* stream) {
    reset_error();
    int rc = check_shape(rows, width);
    if (rc == TSGEMM_OK) rc = check_dtype(dtype, "dtype");
    if (rc == TSGEMM_OK) rc = check_weights_dtype(weight_dtype, dtype);
    if (rc != TSGEMM_OK) return rc;
    if (width < 1) return fail(TSGEMM_EINVAL, "layer norm needs a width of at least 1");
    if (!(eps >= 0.0f) || std::isinf(eps)) return fail(TSGEMM_EINVAL, "eps must be finite and >= 0");
    if (rows == 0) return TSGEMM_OK;
    rc = check_matrix("x", x, ldx, width, dtype);
    if (rc != TSGEMM_OK) return rc;
    if (!y && !codes && !scales) return fail(TSGEMM_EINVAL, "no output: y, or codes and scales, must be given");
    if (y) rc = check_matrix("y", y, ldy, width, dtype);
    if (rc == TSGEMM_OK && (codes || scales)) rc = check_mx(width, codes, scales);
    if (rc != TSGEMM_OK) return rc;
    if (!mean != !rstd) return fail(TSGEMM_EINVAL, "mean and rstd are given together or not at all");
    if (off(mean, 4) || off(rstd, 4) || off(gamma, (unsigned)bytes_of(weight_dtype)) || off(beta, (unsigned)bytes_of(weight_dtype)))
        return fail(TSGEMM_EINVAL, "gamma, beta, mean and rstd must be aligned to their types");
    const int e = bytes_of(dtype), we = bytes_of(weight_dtype);
    rc = check_overlaps({matrix("y", y, rows, width, ldy, e), stretch("mean", mean, 4 * rows), stretch("rstd", rstd, 4 * rows),
                         stretch("codes", codes, rows * width), stretch("scales", scales, rows * (width / 32))},
                        {matrix("x", x, rows, width, ldx, e), stretch("gamma", gamma, we * width), stretch("beta", beta, we * width)});
    if (rc != TSGEMM_OK) return rc;
    tsg::LnArgs a = {};
    a.x = x; a.gamma = gamma; a.beta = beta; a.y = y; a.mean = mean; a.rstd = rstd;
    a.codes = static_cast<uint8_t*>(codes); a.scales = static_cast<uint8_t*>(scales);
    a.rows = rows; a.ldx = ldx; a.ldy = ldy; a.width = (uint32_t)width; a.wdt = weight_dtype;
    a.eps = eps; a.inv_n = 1.0 / (double)width;
    (void)hipGetLastError();
    tsg::launch_layer_norm(dtype, a, static_cast<hipStream_t>(stream));
    return launched("layer norm");
}

int64_t tsgemm_layer_norm_grad_workspace(int64_t rows, int64_t width) {
    reset_error();
    const int rc = check_shape(rows, width);
    if (rc != TSGEMM_OK) return rc;
    if (width < 1) return fail(TSGEMM_EINVAL, "layer norm needs a width of at least 1");
    // fp32 rows take as many workgroups as 16-bit ones or fewer
    return (int64_t)tsg::layer_norm_grad_groups(TSGEMM_BF16, rows, (uint32_t)width) * 2 * grad_pitch(width) * (int64_t)sizeof(float);
}

int tsgemm_layer_norm_grad(int64_t rows, int64_t width, int dtype, int weight_dtype, const void* dy, int64_t lddy, const void* x,
                           int64_t ldx, const void* gamma, const float* mean, const float* rstd, void* dx, int64_t lddx,
                           void* dgamma, void* dbeta, void* workspace, int64_t workspace_bytes, void* stream) {
    const int64_t need = tsgemm_layer_norm_grad_workspace(rows, width);
    if (need < 0) return (int)need;
    int rc = check_dtype(dtype, "dtype");
    if (rc == TSGEMM_OK) rc = check_weights_dtype(weight_dtype, dtype);
    if (rc != TSGEMM_OK) return rc;
    if (off(gamma, (unsigned)bytes_of(weight_dtype)) || off(dgamma, (unsigned)bytes_of(weight_dtype)) ||
        off(dbeta, (unsigned)bytes_of(weight_dtype)))
        return fail(TSGEMM_EINVAL, "gamma, dgamma and dbeta must be aligned to their type");
    const bool sums = dgamma || dbeta;
    if (rows > 0) {
        rc = check_matrix("dy", dy, lddy, width, dtype);
        if (rc == TSGEMM_OK) rc = check_matrix("x", x, ldx, width, dtype);
        if (rc == TSGEMM_OK) rc = check_matrix("dx", dx, lddx, width, dtype);
        if (rc != TSGEMM_OK) return rc;
        if (!mean || !rstd || off(mean, 4) || off(rstd, 4)) return fail(TSGEMM_EINVAL, "mean and rstd must be given, 4-byte aligned");
        if (sums && (!workspace || off(workspace, 16) || workspace_bytes < need))
            return fail(TSGEMM_EINVAL, "dgamma and dbeta need a 16-byte aligned workspace of %lld bytes", (long long)need);
    }
    const int e = bytes_of(dtype), we = bytes_of(weight_dtype);
    rc = check_overlaps({matrix("dx", dx, rows, width, lddx, e), stretch("dgamma", dgamma, we * width),
                         stretch("dbeta", dbeta, we * width), stretch("workspace", sums ? workspace : nullptr, need)},
                        {matrix("dy", dy, rows, width, lddy, e), matrix("x", x, rows, width, ldx, e),
                         stretch("gamma", gamma, we * width), stretch("mean", mean, 4 * rows), stretch("rstd", rstd, 4 * rows)});
    if (rc != TSGEMM_OK) return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool small = rows > 0 && tsg::layer_norm_grad_small(rows, (uint32_t)width);
    float* part = sums && !small ? static_cast<float*>(workspace) : nullptr;
    (void)hipGetLastError();
    if (rows > 0) {
        tsg::LnGradArgs a = {};
        a.dy = dy; a.x = x; a.gamma = gamma; a.mean = mean; a.rstd = rstd; a.dx = dx; a.part = part;
        a.rows = rows; a.lddy = lddy; a.ldx = ldx; a.lddx = lddx;
        a.width = (uint32_t)width; a.pitch = grad_pitch(width); a.wdt = weight_dtype; a.inv_n = 1.0f / (float)width;
        if (small) { a.dgamma = dgamma; a.dbeta = dbeta; }
        tsg::launch_layer_norm_grad(dtype, a, s);
        rc = launched("layer norm gradient");
        if (rc != TSGEMM_OK) return rc;
    }
    if (!sums || small) return TSGEMM_OK;
    tsg::launch_layer_norm_grad_sum(weight_dtype, part, tsg::layer_norm_grad_groups(dtype, rows, (uint32_t)width),
                                    grad_pitch(width), (uint32_t)width, dgamma, dbeta, s);
    return launched("layer norm gradient sum");
}

int tsgemm_mx_quantize(int64_t rows, int64_t width, int dtype, const void* x, int64_t ldx, void* codes, void* scales, void* stream) {
    reset_error();
    int rc = check_shape(rows, width);
    if (rc == TSGEMM_OK) rc = check_dtype(dtype, "dtype");
    if (rc != TSGEMM_OK) return rc;
    if (rows == 0 || width == 0) return TSGEMM_OK;
    rc = check_matrix("x", x, ldx, width, dtype);
    if (rc == TSGEMM_OK) rc = check_mx(width, codes, scales);
    if (rc == TSGEMM_OK)
        rc = check_overlaps({stretch("codes", codes, rows * width), stretch("scales", scales, rows * (width / 32))},
                            {matrix("x", x, rows, width, ldx, bytes_of(dtype))});
    if (rc != TSGEMM_OK) return rc;
    (void)hipGetLastError();
    tsg::launch_mx_quantize(dtype, x, ldx, rows, (uint32_t)width, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                            static_cast<hipStream_t>(stream));
    return launched("MX quantize");
}

int tsgemm_mx_dequantize(int64_t rows, int64_t width, int dtype, const void* codes, const void* scales, void* out, int64_t ldo,
                         void* stream) {
    reset_error();
    int rc = check_shape(rows, width);
    if (rc == TSGEMM_OK) rc = check_dtype(dtype, "dtype");
    if (rc != TSGEMM_OK) return rc;
    if (rows == 0 || width == 0) return TSGEMM_OK;
    rc = check_matrix("out", out, ldo, width, dtype);
    if (rc == TSGEMM_OK) rc = check_mx(width, codes, scales);
    if (rc == TSGEMM_OK)
        rc = check_overlaps({matrix("out", out, rows, width, ldo, bytes_of(dtype))},
                            {stretch("codes", codes, rows * width), stretch("scales", scales, rows * (width / 32))});
    if (rc != TSGEMM_OK) return rc;
    (void)hipGetLastError();
    tsg::launch_mx_dequantize(dtype, static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), rows, (uint32_t)width,
                              out, ldo, static_cast<hipStream_t>(stream));
    return launched("MX dequantize");
}

int64_t tsgemm_mx_weight_grad_workspace(int64_t rows, int64_t out, int64_t width) {
    reset_error();
    const int rc = check_weight_grad(rows, out, width);
    if (rc != TSGEMM_OK) return rc;
    return out == 0 || width == 0 ? 0 : tsg::wgrad_workspace(rows, out, width);
}

int tsgemm_mx_weight_grad(int64_t rows, int64_t out, int64_t width, int dtype, int grad_dtype, const void* dy, int64_t lddy,
                          const void* codes, const void* scales, void* dw, void* workspace, int64_t workspace_bytes, void* stream) {
    const int64_t need = tsgemm_mx_weight_grad_workspace(rows, out, width);
    if (need < 0) return (int)need;
    if (dtype != TSGEMM_FP16 && dtype != TSGEMM_BF16)
        return fail(TSGEMM_EINVAL, "dtype must be TSGEMM_FP16 (1) or TSGEMM_BF16 (2), got %d", dtype);
    if (grad_dtype != dtype && grad_dtype != TSGEMM_FP32)
        return fail(TSGEMM_EINVAL, "dw must be of dy's type (%d) or TSGEMM_FP32, got %d", dtype, grad_dtype);
    if (out == 0 || width == 0) return TSGEMM_OK;
    if (!dw || off(dw, 16)) return fail(TSGEMM_EINVAL, "dw must be given, 16-byte aligned");
    if (rows > 0) {
        int rc = check_matrix("dy", dy, lddy, out, dtype);
        if (rc == TSGEMM_OK) rc = check_mx(width, codes, scales);
        if (rc != TSGEMM_OK) return rc;
        if (off(dy, 16) || lddy % 8 != 0) return fail(TSGEMM_EINVAL, "dy's rows must be 16-byte aligned");
        if (lddy >= (int64_t(1) << 24)) return fail(TSGEMM_EUNSUPPORTED, "dy's row stride must be below 2^24 (32-bit offsets in a slab of 64 rows)");
        if (need > 0 && (!workspace || off(workspace, 16) || workspace_bytes < need))
            return fail(TSGEMM_EINVAL, "this shape needs a 16-byte aligned workspace of %lld bytes", (long long)need);
        rc = check_overlaps({stretch("dw", dw, out * width * bytes_of(grad_dtype)), stretch("workspace", workspace, need)},
                            {matrix("dy", dy, rows, out, lddy, 2), stretch("codes", codes, rows * width),
                             stretch("scales", scales, rows * (width / 32))});
        if (rc != TSGEMM_OK) return rc;
    }
    tsg::WgradArgs a = {};
    a.dy = static_cast<const uint16_t*>(dy); a.codes = static_cast<const uint8_t*>(codes);
    a.scales = static_cast<const uint8_t*>(scales); a.dw = dw; a.part = static_cast<float*>(workspace);
    a.rows = rows; a.lddy = lddy; a.out = (uint32_t)out; a.width = (uint32_t)width;
    (void)hipGetLastError();
    tsg::launch_wgrad(dtype, grad_dtype, a, static_cast<hipStream_t>(stream));
    return launched("weight gradient");
}

}  // extern "C"
