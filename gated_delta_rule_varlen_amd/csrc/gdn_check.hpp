// gdn_check.hpp -- argument checks that the entry points of the operators beside the recurrence share (host code).
#pragma once

#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "gdn.h"
#include "gdn_launch.hpp"

namespace gdn {

inline bool dtype_ok(int d) { return d == GDN_F32 || d == GDN_BF16 || d == GDN_F16; }
inline long long dsize(int d) { return d == GDN_F32 ? 4 : 2; }
inline bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

inline gdn_status from_hip(hipError_t e) {
    if (e == hipSuccess) return GDN_OK;
    if (e == hipErrorInvalidConfiguration) return GDN_ERR_OVERFLOW;
    return GDN_ERR_HIP;
}

// A [rows, heads, width] tensor with free row and head strides, in elements of `es` bytes that start at multiples of
// `align` bytes; one without rows has no address to check.
inline gdn_status strided_rows(const void* p, const int64_t stride[2], long long rows, int heads, long long width_bytes,
                               long long es, long long align, HeadRows* out) {
    out->p = const_cast<void*>(p);
    out->row = stride[0];
    out->head = stride[1];
    if (rows == 0) return GDN_OK;
    if (p == nullptr) return GDN_ERR_NULL;
    if (stride[0] < 0 || stride[1] < 0) return GDN_ERR_SHAPE;
    // the last element's byte offset stays far inside 64 bits
    if (stride[0] > (LLONG_MAX / 16) / rows || stride[1] > (LLONG_MAX / 16) / heads) return GDN_ERR_OVERFLOW;
    if (reinterpret_cast<uintptr_t>(p) % align != 0 || (stride[0] * es) % align != 0 || (stride[1] * es) % align != 0 ||
        width_bytes % align != 0)
        return GDN_ERR_ALIGN;
    return GDN_OK;
}
inline gdn_status head_rows(const void* p, const int64_t stride[2], long long rows, int heads, int D, int dtype,
                            HeadRows* out) {
    return strided_rows(p, stride, rows, heads, D * dsize(dtype), dsize(dtype), 16, out);
}

constexpr long long kMaxRowBytes = 4ll << 20;  // between two rows of a cache: 32-bit offsets inside a key tile
constexpr long long kMaxFp4RowBytes = 1ll << 20;  // of a 4-bit one, of which 544 rows lie in one range

}  // namespace gdn
