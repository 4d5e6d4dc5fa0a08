// gdn_attn_api.cpp -- the extern "C" entry points of the softmax-attention operators: argument
// validation and dispatch.  As in gdn_api.cpp every check runs on the host before anything is queued.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "gdn.h"
#include "gdn_check.hpp"
#include "gdn_launch.hpp"

namespace {

using namespace gdn;

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

// The four tensors of a 4-bit cache; one without rows has no addresses to check.
gdn_status check_cache(const gdn_fp4_cache* c, int HK, int D, gdn::Fp4Cache* to) {
    if (c == nullptr) return GDN_ERR_NULL;
    if (c->rows < 0 || D < 32 || D > 256 || D % 32 != 0) return GDN_ERR_SHAPE;
    if (c->rows > LLONG_MAX / 16) return GDN_ERR_OVERFLOW;
    to->rows = c->rows;
    struct {
        const void* p;
        const int64_t* stride;
        int width, align;
        gdn::HeadRows* to;
    } t[4] = {{c->k_codes, c->k_codes_stride, D / 2, 16, &to->k.codes},
              {c->k_scales, c->k_scales_stride, D / 32, 1, &to->k.scales},
              {c->v_codes, c->v_codes_stride, D / 2, 16, &to->v.codes},
              {c->v_scales, c->v_scales_stride, D / 32, 1, &to->v.scales}};
    for (const auto& e : t) {
        const gdn_status st = strided_rows(e.p, e.stride, c->rows, HK, e.width, 1, e.align, e.to);
        if (st != GDN_OK) return st;
        if (e.stride[0] > kMaxFp4RowBytes) return GDN_ERR_OVERFLOW;
    }
    return GDN_OK;
}

gdn_status fp4_rows(const gdn_fp4_rows_desc* d, const void* k, const void* v, const int32_t* offsets, const int32_t* past,
                    const int64_t* kv_begin, const gdn_fp4_cache* cache, bool read, int32_t* dev_status,
                    hipStream_t stream) {
    if (d == nullptr || offsets == nullptr) return GDN_ERR_NULL;
    gdn_status st = check_sizes(d->B, d->N, d->HK, d->HK, d->D, d->dtype);
    if (st != GDN_OK) return st;
    if (d->flags != 0) return GDN_ERR_UNSUPPORTED;
    gdn::Fp4RowsLaunch a{};
    if ((st = check_cache(cache, d->HK, d->D, &a.cache)) != GDN_OK) return st;
    if (d->N > (1 << 27) - 8) return GDN_ERR_OVERFLOW;  // tokens of one launch
    if ((long long)d->HK * d->D > INT_MAX - 4096) return GDN_ERR_OVERFLOW;  // pieces of a token
    if (kv_begin == nullptr && cache->rows < d->N) return GDN_ERR_SHAPE;  // rows are token indices
    if ((st = head_rows(k, d->k_stride, d->N, d->HK, d->D, d->dtype, &a.k)) != GDN_OK) return st;
    if ((st = head_rows(v, d->v_stride, d->N, d->HK, d->D, d->dtype, &a.v)) != GDN_OK) return st;
    a.offsets = offsets;
    a.past = past;
    a.kv_begin = kv_begin;
    a.dev_status = dev_status;
    a.B = d->B;
    a.N = d->N;
    a.HK = d->HK;
    a.D = d->D;
    a.dtype = d->dtype;
    a.read = read;
    return from_hip(gdn::launch_fp4_rows(a, stream));
}

// The descriptor of an attention over a 4-bit cache, without the strides that are not read.
gdn_status check_fp4_desc(const gdn_attn_desc* d, gdn::AttnLaunch* a) {
    if (d == nullptr) return GDN_ERR_NULL;
    gdn_attn_desc x = *d;
    for (int i = 0; i < 2; ++i) x.k_stride[i] = x.v_stride[i] = 0;
    if (x.prefix_len != 0) return GDN_ERR_SHAPE;
    const gdn_status st = check_attn_desc(&x, a);
    if (st != GDN_OK) return st;
    return x.D % 32 != 0 ? GDN_ERR_SHAPE : GDN_OK;
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

gdn_status gdn_cache_write_fp4_varlen(const gdn_fp4_rows_desc* d, const void* k, const void* v, const int32_t* offsets,
                                      const int32_t* past, const int64_t* kv_begin, const gdn_fp4_cache* cache,
                                      int32_t* dev_status, hipStream_t stream) {
    return fp4_rows(d, k, v, offsets, past, kv_begin, cache, false, dev_status, stream);
}

gdn_status gdn_cache_read_fp4_varlen(const gdn_fp4_rows_desc* d, const gdn_fp4_cache* cache, const int32_t* offsets,
                                     const int32_t* past, const int64_t* kv_begin, void* k_out, void* v_out,
                                     int32_t* dev_status, hipStream_t stream) {
    return fp4_rows(d, k_out, v_out, offsets, past, kv_begin, cache, true, dev_status, stream);
}

gdn_status gdn_attention_fp4_varlen(const gdn_attn_desc* d, const void* q, const gdn_fp4_cache* cache,
                                    const int32_t* offsets, const int64_t* kv_begin, const int32_t* kv_len, void* out,
                                    float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status,
                                    hipStream_t stream) {
    gdn::AttnLaunch a{};
    gdn::Fp4Cache c{};
    gdn_status st = check_fp4_desc(d, &a);
    if (st != GDN_OK) return st;
    if (offsets == nullptr || kv_begin == nullptr || kv_len == nullptr) return GDN_ERR_NULL;
    if ((st = check_cache(cache, d->HK, d->D, &c)) != GDN_OK) return st;
    if (cache->rows != d->kv_rows) return GDN_ERR_SHAPE;
    if ((st = head_rows(q, d->q_stride, d->N, d->H, d->D, d->dtype, &a.q)) != GDN_OK) return st;
    if ((st = head_rows(out, d->out_stride, d->N, d->H, d->D, d->dtype, &a.out)) != GDN_OK) return st;
    if (misaligned(workspace)) return GDN_ERR_ALIGN;
    const size_t need = gdn::attention_fp4_workspace_bytes(a);
    if (need > 0 && (workspace == nullptr || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    a.offsets = offsets;
    a.kv_begin = kv_begin;
    a.kv_len = kv_len;
    a.lse = lse;
    a.workspace = workspace;
    a.dev_status = dev_status;
    return from_hip(gdn::launch_attention_fp4(a, c, stream));
}

gdn_status gdn_attention_fp4_workspace_bytes(const gdn_attn_desc* d, size_t* bytes) {
    if (bytes == nullptr) return GDN_ERR_NULL;
    gdn::AttnLaunch a{};
    const gdn_status st = check_fp4_desc(d, &a);
    if (st == GDN_OK) *bytes = gdn::attention_fp4_workspace_bytes(a);
    return st;
}

}  // extern "C"
