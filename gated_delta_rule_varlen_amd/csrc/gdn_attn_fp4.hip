// gdn_attn_fp4.hip -- causal attention of packed sequences over a 4-bit cache: a wave a row (one head of one token), 64
// keys at a time.
#include <hip/hip_runtime.h>

#include "gdn_attn.hpp"
#include "gdn_fp4.hpp"

namespace gdn {
namespace {

using namespace attn;

// One run of a head's cache rows.
struct Fp4Keys {
    const char *kc, *ks, *vc, *vs;
};

__device__ __forceinline__ float value_or_nan(float y, uint32_t scale_byte) {
    return scale_byte == fp4::kNotANumber ? __uint_as_float(0x7fc00000u) : y;
}

// Row q over the keys j0 .. j1 - 1: the largest score to base 2, the sum of exponentials and, four elements a lane
// (4 * lane ..), their products with the values.
struct RowSums {
    float m, sum;
    f32x4 o;
};
template <typename T>
__device__ __forceinline__ RowSums plain_row(const typename T::storage* q, const Fp4Keys& s, const Fp4Cache& c, int D, float s2,
                                             int j0, int j1) {
    const int lane = threadIdx.x & 63;
    RowSums r{kNoMax, 0.0f, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll 1
    for (; j0 < j1; j0 += 64) {
        float y = -INFINITY;
        if (j0 + lane < j1) {
            const char* codes = s.kc + (j0 + lane) * c.k.codes.row;
            const uint8_t* scales = reinterpret_cast<const uint8_t*>(s.ks + (j0 + lane) * c.k.scales.row);
            y = 0.0f;
#pragma unroll 1
            for (int b = 0; b < D / 32; ++b) {
                const u32x4 w = *reinterpret_cast<const u32x4*>(codes + 16 * b);
                const uint32_t scale = scales[b];
                float sum = 0.0f;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float k[8];
                    fp4::values(w[x], scale, k);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum = fmaf(to_f32<T>(q[32 * b + 8 * x + e]), k[e], sum);
                }
                y += value_or_nan(sum, scale);
            }
            y *= s2;
        }
        float top = y;
        for (int z = 1; z < 64; z <<= 1) top = fmaxf(top, __shfl_xor(top, z));
        const float to = fmaxf(r.m, top), w = __builtin_amdgcn_exp2f(r.m - to), p = __builtin_amdgcn_exp2f(y - to);
        r.sum = r.sum * w + group_sum<64>(p);
        r.m = to;
        r.o *= w;
#pragma unroll 1
        for (int j = 0; j < min(64, j1 - j0); ++j) {
            const float pj = __shfl(p, j);
            if (4 * lane >= D) continue;
            const uint32_t codes = *reinterpret_cast<const uint16_t*>(s.vc + (j0 + j) * c.v.codes.row + 2 * lane);
            const uint32_t scale = *reinterpret_cast<const uint8_t*>(s.vs + (j0 + j) * c.v.scales.row + lane / 8);
            float v[8];
            fp4::values(codes, scale, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) r.o[e] = fmaf(pj, value_or_nan(v[e], scale), r.o[e]);
        }
    }
    return r;
}

template <typename T>
__global__ __launch_bounds__(256) void rows_kernel(AttnLaunch c, Fp4Cache cache) {
    using TS = typename T::storage;
    const bool malformed = check<256>(c);
    report_status(c.dev_status, malformed);
    if (malformed) return;
    const int lane = threadIdx.x & 63, G = c.H / c.HK;
    const float s2 = c.scale * kLog2e;
    const long long rows = (long long)c.N * c.H;
    for (long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); row < rows; row += (long long)gridDim.x * 4) {
        const int t = (int)(row / c.H), h = (int)(row - (long long)t * c.H), hk = h / G;
        int b = 0, end = c.B;  // the last sequence that starts at t or before it
        while (end - b > 1) {
            const int mid = (b + end) / 2;
            (c.offsets[mid] <= t ? b : end) = mid;
        }
        const int first = c.offsets[b], T_ = c.offsets[b + 1] - first, n = c.kv_len[b], seen = min(max(n - T_ + 1 + t - first, 0), n);
        const long long begin = c.kv_begin[b];
        const auto at = [&](const HeadRows& x) { return static_cast<const char*>(x.p) + begin * x.row + hk * x.head; };
        const Fp4Keys keys{at(cache.k.codes), at(cache.k.scales), at(cache.v.codes), at(cache.v.scales)};
        const TS* q = static_cast<const TS*>(c.q.p) + t * c.q.row + h * c.q.head;
        const RowSums r = plain_row<T>(q, keys, cache, c.D, s2, 0, seen);
        const float inv = r.sum == 0.0f ? 0.0f : 1.0f / r.sum;
        TS* out = static_cast<TS*>(c.out.p) + t * c.out.row + h * c.out.head;
        if (4 * lane < c.D)
            for (int e = 0; e < 4; ++e) out[4 * lane + e] = from_f32<T>(r.o[e] * inv);
        if (lane == 0 && c.lse != nullptr) c.lse[row] = r.sum == 0.0f ? -INFINITY : kLn2 * (r.m + __builtin_amdgcn_logf(r.sum));
    }
}

template <typename T>
hipError_t launch(const AttnLaunch& c, const Fp4Cache& cache, hipStream_t stream) {
    const long long blocks = std::max(1ll, std::min<long long>(((long long)c.N * c.H + 3) / 4, kCUs * 64));
    rows_kernel<T><<<(unsigned)blocks, 256, 0, stream>>>(c, cache);
    return hipGetLastError();
}

}  // namespace

size_t attention_fp4_workspace_bytes(const AttnLaunch&) { return 0; }

hipError_t launch_attention_fp4(const AttnLaunch& c, const Fp4Cache& cache, hipStream_t stream) {
    switch (c.dtype) {
        case GDN_F32: return launch<F32>(c, cache, stream);
        case GDN_BF16: return launch<BF16>(c, cache, stream);
        default: return launch<F16>(c, cache, stream);
    }
}

}  // namespace gdn
