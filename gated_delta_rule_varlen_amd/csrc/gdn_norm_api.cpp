// gdn_norm_api.cpp -- the extern "C" entry points of the norms before and behind a block: argument validation and
// dispatch.  Every check runs on the host before anything is queued.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>

#include "gdn.h"
#include "gdn_check.hpp"
#include "gdn_launch.hpp"

using namespace gdn;

extern "C" {

gdn_status gdn_residual_norm(const gdn_residual_norm_desc* d, const void* x, const void* residual, const float* post_weight,
                             const float* channel_scale, const float* weight, void* out, void* residual_out,
                             hipStream_t stream) {
    if (d == nullptr) return GDN_ERR_NULL;
    if (d->N < 0 || d->C < 1 || d->C > 32768 || !(d->eps >= 0.0f) || !std::isfinite(d->scale)) return GDN_ERR_SHAPE;
    if (!dtype_ok(d->dtype) || (d->residual_dtype != d->dtype && d->residual_dtype != GDN_F32)) return GDN_ERR_DTYPE;
    struct {
        const void* p;
        int64_t stride;
        int dtype;
        bool required;
    } t[4] = {{x, d->x_stride, d->dtype, true},
              {residual, d->residual_stride, d->residual_dtype, false},
              {out, d->out_stride, d->dtype, true},
              {residual_out, d->residual_out_stride, d->residual_dtype, false}};
    for (const auto& e : t) {
        if (d->N == 0 || (e.p == nullptr && !e.required)) continue;
        if (e.stride < d->C) return GDN_ERR_SHAPE;
        const int64_t stride[2] = {e.stride, 0};
        HeadRows rows;
        const gdn_status st = head_rows(e.p, stride, d->N, 1, d->C, e.dtype, &rows);
        if (st != GDN_OK) return st;
    }
    if ((d->C * dsize(d->dtype)) % 16 != 0 || misaligned(post_weight) || misaligned(channel_scale) || misaligned(weight))
        return GDN_ERR_ALIGN;
    ResidualNormLaunch a{x, residual, post_weight, channel_scale, weight, out, residual_out,
                         d->x_stride, d->residual_stride, d->out_stride, d->residual_out_stride,
                         d->N, d->C, d->dtype, d->residual_dtype, d->eps, d->scale};
    return d->N == 0 ? GDN_OK : from_hip(launch_residual_norm(a, stream));
}

gdn_status gdn_gated_norm(const gdn_gated_norm_desc* d, const void* x, const void* gate, const float* weight, void* out,
                          hipStream_t stream) {
    if (d == nullptr) return GDN_ERR_NULL;
    if (d->N < 0 || d->H < 1 || d->V < 1 || d->V > 2048 || !(d->eps >= 0.0f)) return GDN_ERR_SHAPE;
    if (!dtype_ok(d->dtype)) return GDN_ERR_DTYPE;
    if ((d->flags & ~(uint32_t)(GDN_GATE_SIGMOID | GDN_GATE_FIRST | GDN_GATE_NO_NORM)) != 0 ||
        ((d->flags & GDN_GATE_NO_NORM) && weight != nullptr))
        return GDN_ERR_UNSUPPORTED;
    if ((long long)d->N * d->H > INT_MAX - 4096) return GDN_ERR_OVERFLOW;
    GatedNormLaunch a{};
    gdn_status st;
    if ((st = head_rows(x, d->x_stride, d->N, d->H, d->V, d->dtype, &a.x)) != GDN_OK) return st;
    if ((st = head_rows(gate, d->gate_stride, d->N, d->H, d->V, d->dtype, &a.gate)) != GDN_OK) return st;
    if ((st = head_rows(out, d->out_stride, d->N, d->H, d->V, d->dtype, &a.out)) != GDN_OK) return st;
    if ((d->V * dsize(d->dtype)) % 16 != 0 || misaligned(weight)) return GDN_ERR_ALIGN;
    a.weight = weight;
    a.N = d->N;
    a.H = d->H;
    a.V = d->V;
    a.dtype = d->dtype;
    a.eps = d->eps;
    a.sigmoid = (d->flags & GDN_GATE_SIGMOID) != 0;
    a.gate_first = (d->flags & GDN_GATE_FIRST) != 0;
    a.no_norm = (d->flags & GDN_GATE_NO_NORM) != 0;
    return d->N == 0 ? GDN_OK : from_hip(launch_gated_norm(a, stream));
}

}  // extern "C"
