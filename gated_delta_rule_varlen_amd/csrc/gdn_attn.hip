// gdn_attn.hip -- causal softmax attention of packed sequences with grouped heads, with or without a
// prefix shared by all sequences (gdn_attention_varlen, gdn_attention_prefix_varlen).
//
// One wave computes one query row (token, head) in one pass over its keys: 64 keys at a time, one
// per lane for the scores, then one element of the value row per lane for the products, with the
// running maximum m and sum l of the softmax (out = sum_j exp(s_j - m) v_j / l, rescaled by
// exp(m_old - m_new) whenever m grows).
#include <hip/hip_runtime.h>

#include <climits>

#include "gdn_device.hpp"
#include "gdn_launch.hpp"

namespace gdn {
namespace {

constexpr int NT = 64;
constexpr int MAX_D = 256;

// Offsets, lengths and key runs of the whole call; also the sequence of token t.
__device__ __forceinline__ bool attn_malformed(const AttnLaunch& a, int t, int& b) {
    int bad = 0, at_or_below = 0;
    for (int i = threadIdx.x; i <= a.B; i += NT) {
        const int o = a.offsets[i];
        if (i == 0) {
            bad |= (o != 0);
        } else {
            const int n = o - a.offsets[i - 1];
            bad |= (n < 0) | (n > a.max_q);
            if (a.kv_len != nullptr) {
                const long long len = a.kv_len[i - 1], begin = a.kv_begin[i - 1];
                bad |= (len < 0) | (begin < 0) | (begin > a.kv_rows) | (begin + len > a.kv_rows);
            } else {
                bad |= (o > a.kv_rows);
            }
        }
        if (i == a.B) bad |= (o != a.N);
        at_or_below += (o <= t);
    }
    for (int m = 1; m < 64; m <<= 1) at_or_below += __shfl_xor(at_or_below, m);
    b = at_or_below - 1;
    return __syncthreads_or(bad) != 0;
}

template <typename T>
__global__ __launch_bounds__(NT) void attn_kernel(AttnLaunch a) {
    using TS = typename T::storage;
    const int t = blockIdx.x / a.H, h = blockIdx.x - t * a.H, lane = threadIdx.x, hk = h / (a.H / a.HK);
    int b;
    const bool malformed = attn_malformed(a, t, b);
    report_status(a.dev_status, malformed);
    if (malformed || t >= a.N) return;
    const int first = a.offsets[b], T_b = a.offsets[b + 1] - first;
    const long long begin = a.kv_begin != nullptr ? a.kv_begin[b] : first;
    const int own = (a.kv_len != nullptr ? a.kv_len[b] : T_b) - T_b + (t - first) + 1;  // keys this token sees

    __shared__ float q[MAX_D];
    for (int e = lane; e < a.D; e += NT)
        q[e] = to_f32<T>(static_cast<const TS*>(a.q.p)[t * a.q.row + h * a.q.head + e]);
    __syncthreads();

    float m = -INFINITY, l = 0.0f, o[MAX_D / 64] = {0.0f, 0.0f, 0.0f, 0.0f};
    auto run = [&](const HeadRows& K, const HeadRows& V, long long row0, int n) {
        const TS* kp = static_cast<const TS*>(K.p) + row0 * K.row + hk * K.head;
        const TS* vp = static_cast<const TS*>(V.p) + row0 * V.row + hk * V.head;
        for (int j0 = 0; j0 < n; j0 += 64) {
            float s = -INFINITY;
            if (j0 + lane < n) {
                const TS* row = kp + (j0 + lane) * K.row;
                s = 0.0f;
                for (int e = 0; e < a.D; e += 4) {
                    const f32x4 x = load4<T>(row + e);
                    for (int i = 0; i < 4; ++i) s = fmaf(q[e + i], x[i], s);
                }
                s *= a.scale;
            }
            float top = s;
            for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
            const float m_new = fmaxf(m, top), ref = m_new == -INFINITY ? 0.0f : m_new;
            const float p = expf(s - ref), w = expf(m - ref);
            float sum = p;
            for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
            l = l * w + sum;
            m = m_new;
            for (int i = 0; i < MAX_D / 64; ++i) o[i] *= w;
            for (int j = 0; j < 64 && j0 + j < n; ++j) {
                const float pj = __shfl(p, j);
                for (int i = 0; i < MAX_D / 64; ++i)
                    if (lane + 64 * i < a.D) o[i] = fmaf(pj, to_f32<T>(vp[(j0 + j) * V.row + lane + 64 * i]), o[i]);
            }
        }
    };
    run(a.pk, a.pv, 0, a.prefix_len);
    run(a.k, a.v, begin, own);
    TS* out = static_cast<TS*>(a.out.p) + t * a.out.row + h * a.out.head;
    for (int i = 0; i < MAX_D / 64; ++i)
        if (lane + 64 * i < a.D) out[lane + 64 * i] = from_f32<T>(l == 0.0f ? 0.0f : o[i] / l);
    if (a.lse != nullptr && lane == 0) a.lse[t * a.H + h] = m + logf(l);
}

template <typename T>
hipError_t launch(const AttnLaunch& a, hipStream_t stream) {
    const long long blocks = a.N > 0 ? (long long)a.N * a.H : 1;
    attn_kernel<T><<<(unsigned)blocks, NT, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

size_t attention_workspace_bytes(const AttnLaunch&) { return 0; }

hipError_t launch_attention(const AttnLaunch& a, hipStream_t stream) {
    switch (a.dtype) {
        case GDN_F32: return launch<F32>(a, stream);
        case GDN_BF16: return launch<BF16>(a, stream);
        default: return launch<F16>(a, stream);
    }
}

}  // namespace gdn
