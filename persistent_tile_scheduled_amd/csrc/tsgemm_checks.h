// Argument checks that the C ABI's files share (tsgemm_ops.hip, tsgemm_linear.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "tsgemm.h"
#include "tsgemm_host.h"
#include "tsgemm_overlap.h"

namespace tsg {

inline bool is_float(int dt) { return dt == TSGEMM_FP16 || dt == TSGEMM_BF16 || dt == TSGEMM_FP32; }
inline int bytes_of(int dt) { return dt == TSGEMM_FP32 ? 4 : 2; }
inline bool off(const void* p, unsigned align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1u)) != 0u; }

// rows and width of an activation; a width of 0 has no mean and no block.
inline int check_shape(int64_t rows, int64_t width) {
    if (rows < 0 || width < 0) return fail(TSGEMM_EINVAL, "rows and width must be >= 0");
    if (rows >= (int64_t(1) << 31) || width >= (int64_t(1) << 31)) return fail(TSGEMM_EINVAL, "rows and width must be below 2^31");
    return TSGEMM_OK;
}
inline int check_dtype(int dt, const char* what) {
    return is_float(dt) ? TSGEMM_OK
                        : fail(TSGEMM_EINVAL, "%s must be TSGEMM_FP16 (1), TSGEMM_BF16 (2) or TSGEMM_FP32 (4), got %d", what, dt);
}
// One matrix of floating values: given, aligned to its type, rows not overlapping.
inline int check_matrix(const char* name, const void* p, int64_t ld, int64_t width, int dt) {
    if (!p) return fail(TSGEMM_EINVAL, "%s is NULL", name);
    if (off(p, (unsigned)bytes_of(dt))) return fail(TSGEMM_EINVAL, "%s must be aligned to its type", name);
    if (ld < width) return fail(TSGEMM_EINVAL, "the row stride of %s (%lld) is below the width (%lld)", name, (long long)ld, (long long)width);
    return TSGEMM_OK;
}
inline int check_weights_dtype(int wdt, int dt) {
    if (wdt != dt && wdt != TSGEMM_FP32)
        return fail(TSGEMM_EINVAL, "the weights must be of the activation's type (%d) or TSGEMM_FP32, got %d", dt, wdt);
    return TSGEMM_OK;
}
inline int check_mx(int64_t width, const void* codes, const void* scales) {
    if (width % 32 != 0) return fail(TSGEMM_EINVAL, "MX blocks need a width divisible by 32, got %lld", (long long)width);
    if (!codes || !scales) return fail(TSGEMM_EINVAL, "codes or scales is NULL");
    if (off(codes, 16) || off(scales, 4)) return fail(TSGEMM_EINVAL, "codes must be 16-byte and scales 4-byte aligned");
    return TSGEMM_OK;
}
struct Named {
    const char* name;
    Region r;
    Extent e;
};
inline Named matrix(const char* name, const void* p, int64_t rows, int64_t width, int64_t ld, int bytes) {
    const Region r = {p, rows, width * bytes, ld * bytes};
    return {name, r, extent(r)};
}
inline Named stretch(const char* name, const void* p, int64_t bytes) { return matrix(name, p, 1, bytes, bytes, 1); }
// No output over an input or another output: workgroups read rows, some of them
// twice, while others already write.
inline int check_overlaps(std::initializer_list<Named> outputs, std::initializer_list<Named> inputs) {
    const auto clash = [](const Named& o, const Named& other) {  // nearly always the extents say no
        return o.e.from < other.e.to && other.e.from < o.e.to && overlap(o.r, other.r);
    };
    for (const Named& o : outputs) {
        for (const Named& i : inputs)
            if (clash(o, i)) return fail(TSGEMM_EINVAL, "%s overlaps %s", o.name, i.name);
        for (const Named* other = outputs.begin(); other != &o; ++other)
            if (clash(o, *other)) return fail(TSGEMM_EINVAL, "%s overlaps %s", o.name, other->name);
    }
    return TSGEMM_OK;
}
inline int launched(const char* what) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? TSGEMM_OK : fail(TSGEMM_EHIP, "%s launch failed: %s", what, hipGetErrorString(e));
}

}  // namespace tsg
