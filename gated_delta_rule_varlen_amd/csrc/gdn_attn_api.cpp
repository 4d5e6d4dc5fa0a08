// gdn_attn_api.cpp -- the extern "C" entry points of the softmax-attention operators: argument
// validation and dispatch.  As in gdn_api.cpp every check runs on the host before anything is queued.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "gdn.h"
#include "gdn_launch.hpp"

namespace {

constexpr long long kMaxRowBytes = 4ll << 20;  // between two rows of k or v: 32-bit offsets inside a key tile

bool dtype_ok(int d) { return d == GDN_F32 || d == GDN_BF16 || d == GDN_F16; }
long long dsize(int d) { return d == GDN_F32 ? 4 : 2; }
bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

gdn_status from_hip(hipError_t e) {
    if (e == hipSuccess) return GDN_OK;
    if (e == hipErrorInvalidConfiguration) return GDN_ERR_OVERFLOW;
    return GDN_ERR_HIP;
}

// A [rows, heads, D] tensor with free row and head strides; one without rows has no address to check.
gdn_status head_rows(const void* p, const int64_t stride[2], long long rows, int heads, int D, int dtype,
                     gdn::HeadRows* out) {
    out->p = const_cast<void*>(p);
    out->row = stride[0];
    out->head = stride[1];
    if (rows == 0) return GDN_OK;
    if (p == nullptr) return GDN_ERR_NULL;
    if (stride[0] < 0 || stride[1] < 0) return GDN_ERR_SHAPE;
    const long long es = dsize(dtype);
    // the last element's byte offset stays far inside 64 bits
    if (stride[0] > (LLONG_MAX / 16) / rows || stride[1] > (LLONG_MAX / 16) / heads) return GDN_ERR_OVERFLOW;
    if (misaligned(p) || (stride[0] * es) % 16 != 0 || (stride[1] * es) % 16 != 0 || (D * es) % 16 != 0)
        return GDN_ERR_ALIGN;
    return GDN_OK;
}

gdn_status check_sizes(int B, int N, int H, int HK, int D, int dtype) {
    if (B < 1 || N < 0 || H < 1 || HK < 1 || D < 1 || D > 256) return GDN_ERR_SHAPE;
    if (!dtype_ok(dtype)) return GDN_ERR_DTYPE;
    // an index past the last tile of rows or tokens still fits 32 bits
    if ((long long)N * H > INT_MAX - 4096 || (long long)B * H > INT_MAX) return GDN_ERR_OVERFLOW;
    return GDN_OK;
}

gdn_status check_attn_desc(const gdn_attn_desc* d, gdn::AttnLaunch* a) {
    if (d == nullptr) return GDN_ERR_NULL;
    gdn_status st = check_sizes(d->B, d->N, d->H, d->HK, d->D, d->dtype);
    if (st != GDN_OK) return st;
    if (d->H % d->HK != 0 || d->kv_rows < 0 || d->prefix_len < 0 || (d->N > 0 && d->max_q < 1)) return GDN_ERR_SHAPE;
    if (d->flags != 0) return GDN_ERR_UNSUPPORTED;
    if (std::isnan(d->scale) || std::isinf(d->scale)) return GDN_ERR_SHAPE;
    if ((d->D * dsize(d->dtype)) % 16 != 0) return GDN_ERR_ALIGN;
    // an index past the last key tile still fits 32 bits (the device checks kv_len the same way)
    if (d->kv_rows > LLONG_MAX / 16 || d->prefix_len > INT_MAX - 4096) return GDN_ERR_OVERFLOW;
    const int64_t* rows[4] = {d->k_stride, d->v_stride, d->prefix_k_stride, d->prefix_v_stride};
    for (int i = 0; i < (d->prefix_len > 0 ? 4 : 2); ++i)
        if (rows[i][0] > kMaxRowBytes / dsize(d->dtype)) return GDN_ERR_OVERFLOW;
    // the plan of a call also looks at how far apart the queries lie
    a->q = gdn::HeadRows{nullptr, d->q_stride[0], d->q_stride[1]};
    a->B = d->B;
    a->N = d->N;
    a->H = d->H;
    a->HK = d->HK;
    a->D = d->D;
    a->max_q = d->max_q < d->N ? d->max_q : d->N;
    if (a->max_q < 0) a->max_q = 0;  // N == 0 takes any
    a->prefix_len = d->prefix_len;
    a->kv_rows = d->kv_rows;
    a->dtype = d->dtype;
    a->scale = d->scale == 0.0f ? 1.0f / std::sqrt((float)d->D) : d->scale;
    return GDN_OK;
}

gdn_status attention(const gdn_attn_desc* d, const void* q, const void* pk, const void* pv, const void* k,
                     const void* v, const int32_t* offsets, const int64_t* kv_begin, const int32_t* kv_len, void* out,
                     float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status, hipStream_t stream) {
    gdn::AttnLaunch a{};
    gdn_status st = check_attn_desc(d, &a);
    if (st != GDN_OK) return st;
    if (offsets == nullptr || (kv_begin == nullptr) != (kv_len == nullptr)) return GDN_ERR_NULL;
    struct {
        const void* p;
        const int64_t* stride;
        long long rows;
        int heads;
        gdn::HeadRows* to;
    } t[6] = {{q, d->q_stride, d->N, d->H, &a.q},
              {out, d->out_stride, d->N, d->H, &a.out},
              {k, d->k_stride, d->kv_rows, d->HK, &a.k},
              {v, d->v_stride, d->kv_rows, d->HK, &a.v},
              {pk, d->prefix_k_stride, d->prefix_len, d->HK, &a.pk},
              {pv, d->prefix_v_stride, d->prefix_len, d->HK, &a.pv}};
    for (const auto& e : t)
        if ((st = head_rows(e.p, e.stride, e.rows, e.heads, d->D, d->dtype, e.to)) != GDN_OK) return st;
    if (misaligned(workspace)) return GDN_ERR_ALIGN;
    const size_t need = gdn::attention_workspace_bytes(a);
    if (need > 0 && (workspace == nullptr || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    a.offsets = offsets;
    a.kv_begin = kv_begin;
    a.kv_len = kv_len;
    a.lse = lse;
    a.workspace = workspace;
    a.dev_status = dev_status;
    return from_hip(gdn::launch_attention(a, stream));
}

}  // namespace

extern "C" {

gdn_status gdn_qk_norm_rope_varlen(const gdn_rope_desc* d, const void* q, const void* k, const void* v,
                                   const float* inv_freq, const float* q_weight, const float* k_weight,
                                   const int32_t* offsets, const int32_t* past, const int32_t* positions,
                                   const int64_t* kv_begin, void* q_out, void* k_out, void* v_out,
                                   int32_t* dev_status, hipStream_t stream) {
    if (d == nullptr || offsets == nullptr) return GDN_ERR_NULL;
    gdn_status st = check_sizes(d->B, d->N, d->H, d->HK, d->D, d->dtype);
    if (st != GDN_OK) return st;
    if (d->rot < 0 || d->rot > d->D || d->rot % 2 != 0 || d->cache_rows < 0 || !(d->eps >= 0.0f) || d->reserved != 0)
        return GDN_ERR_SHAPE;
    if ((long long)d->N * d->HK > INT_MAX) return GDN_ERR_OVERFLOW;
    if (d->flags & ~(uint32_t)GDN_ROPE_INTERLEAVED) return GDN_ERR_UNSUPPORTED;
    if (d->rot > 0 && inv_freq == nullptr) return GDN_ERR_NULL;
    if (d->N > 0 && (v == nullptr) != (v_out == nullptr)) return GDN_ERR_NULL;
    if (d->cache_rows > LLONG_MAX / 16) return GDN_ERR_OVERFLOW;
    // packed rows are token indices
    if (kv_begin == nullptr && d->cache_rows < d->N) return GDN_ERR_SHAPE;
    gdn::RopeLaunch a;
    const long long n = d->N, nv = v != nullptr ? d->N : 0;
    struct {
        const void* p;
        const int64_t* stride;
        long long rows;
        int heads;
        gdn::HeadRows* to;
    } t[6] = {{q, d->q_stride, n, d->H, &a.q},
              {k, d->k_stride, n, d->HK, &a.k},
              {v, d->v_stride, nv, d->HK, &a.v},
              {q_out, d->q_out_stride, n, d->H, &a.q_out},
              {k_out, d->k_out_stride, n > 0 ? d->cache_rows : 0, d->HK, &a.k_out},
              {v_out, d->v_out_stride, nv > 0 ? d->cache_rows : 0, d->HK, &a.v_out}};
    for (const auto& e : t)
        if ((st = head_rows(e.p, e.stride, e.rows, e.heads, d->D, d->dtype, e.to)) != GDN_OK) return st;
    if (misaligned(q_weight) || misaligned(k_weight) || misaligned(inv_freq)) return GDN_ERR_ALIGN;
    a.inv_freq = inv_freq;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.offsets = offsets;
    a.past = past;
    a.positions = positions;
    a.kv_begin = kv_begin;
    a.dev_status = dev_status;
    a.cache_rows = d->cache_rows;
    a.B = d->B;
    a.N = d->N;
    a.H = d->H;
    a.HK = d->HK;
    a.D = d->D;
    a.rot = d->rot;
    a.dtype = d->dtype;
    a.interleaved = (d->flags & GDN_ROPE_INTERLEAVED) != 0;
    a.eps = d->eps;
    return from_hip(gdn::launch_rope(a, stream));
}

gdn_status gdn_attention_varlen(const gdn_attn_desc* d, const void* q, const void* k, const void* v,
                                const int32_t* offsets, const int64_t* kv_begin, const int32_t* kv_len, void* out,
                                float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status,
                                hipStream_t stream) {
    if (d != nullptr && d->prefix_len != 0) return GDN_ERR_SHAPE;
    return attention(d, q, nullptr, nullptr, k, v, offsets, kv_begin, kv_len, out, lse, workspace, ws_bytes,
                     dev_status, stream);
}

gdn_status gdn_attention_prefix_varlen(const gdn_attn_desc* d, const void* q, const void* prefix_k,
                                       const void* prefix_v, const void* k, const void* v, const int32_t* offsets,
                                       const int64_t* kv_begin, const int32_t* kv_len, void* out, float* lse,
                                       void* workspace, size_t ws_bytes, int32_t* dev_status, hipStream_t stream) {
    return attention(d, q, prefix_k, prefix_v, k, v, offsets, kv_begin, kv_len, out, lse, workspace, ws_bytes,
                     dev_status, stream);
}

gdn_status gdn_attention_workspace_bytes(const gdn_attn_desc* d, size_t* bytes) {
    if (bytes == nullptr) return GDN_ERR_NULL;
    gdn::AttnLaunch a{};
    const gdn_status st = check_attn_desc(d, &a);
    if (st == GDN_OK) *bytes = gdn::attention_workspace_bytes(a);
    return st;
}

}  // extern "C"
