// gdn_attn_fp4.hip -- host side of the attention over a 4-bit cache: which form and tile a call takes and its workspace.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdn_attn_fp4.hpp"
#include "gdn_attn_join.hpp"

namespace gdn {
namespace {

using namespace attn;

constexpr int kShortRows = 64;

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
        const TS* q = static_cast<const TS*>(c.q.p) + t * c.q.row + h * c.q.head;
        const RowSums r = plain_row<T>(q, fp4_keys(cache, c.kv_begin[b], hk), cache, c.D, s2, 0, seen);
        const float inv = r.sum == 0.0f ? 0.0f : 1.0f / r.sum;
        TS* out = static_cast<TS*>(c.out.p) + t * c.out.row + h * c.out.head;
        if (4 * lane < c.D)
            for (int e = 0; e < 4; ++e) out[4 * lane + e] = from_f32<T>(r.o[e] * inv);
        if (lane == 0 && c.lse != nullptr) c.lse[row] = r.sum == 0.0f ? -INFINITY : kLn2 * (r.m + __builtin_amdgcn_logf(r.sum));
    }
}

struct Plan {
    Fp4Args f;
    bool is_short, join;
    int dp, rt, bm, lds;
    size_t bytes;
};

template <typename T>
Plan plan(const AttnLaunch& c) {
    Plan p{};
    Args& a = p.f.a;
    a.c = c;
    a.G = c.H / c.HK;
    a.s2 = fabsf(c.scale) * kLog2e;
    a.negate = c.scale < 0.0f;
    a.splits = 1;
    a.set_rows = (long long)c.N * c.H;
    p.dp = c.D <= 64 ? 64 : c.D <= 128 ? 128 : 256;
    const long long rows = std::max(1ll, (long long)c.max_q * a.G);
    p.is_short = rows <= kShortRows;
    if (!p.is_short) return p;
    p.rt = (int)(rows + 15) / 16;
    struct Shape {
        int bm, unit, waves, lds;
    };
    const Shape s = with_short4<T>(p.dp, p.rt, [&](auto x) {
        using C = typename decltype(x)::C;
        return Shape{C::BM, C::UNIT, C::WAVES, C::lds((int)rows)};
    });
    p.bm = s.bm;
    p.lds = s.lds;
    const int per_cu = std::max(1, std::min(s.waves, kCULds / (p.lds + 2048)));
    const long long units = c.HK * (c.kv_rows / s.unit + c.B);  // fewer blocks than that have work, bar overlapping runs
    a.workers = (int)std::max(1ll, std::min((long long)kCUs * per_cu, units));
    p.join = c.N > 0 && a.workers > 1;
    size_t at = 0;
    auto take = [&](size_t n) {
        char* r = static_cast<char*>(c.workspace) + at;
        at += (n + 255) / 256 * 256;
        return r;
    };
    if (p.join) {
        a.status = reinterpret_cast<int*>(take(4));
        if (few_rows(a)) a.row_info = reinterpret_cast<int2*>(take((size_t)c.N * c.HK * 8));
        else a.cut = reinterpret_cast<int4*>(take((size_t)a.workers * 16));
        a.slot_ml = reinterpret_cast<float2*>(take((size_t)a.workers * 2 * p.bm * 8));
        a.slot_o = reinterpret_cast<float*>(take((size_t)a.workers * 2 * p.bm * c.D * 4));
    }
    p.bytes = at;
    return p;
}

template <typename T>
hipError_t launch(const AttnLaunch& c, const Fp4Cache& cache, hipStream_t stream) {
    Plan p = plan<T>(c);
    p.f.cache = cache;
    if (p.is_short) {
        const hipError_t e = start_short4<T>(p.f, p.dp, p.rt, p.lds, stream);
        return e != hipSuccess || !p.join ? e : start_join<T>(p.f.a, p.bm, -1, stream);
    }
    const long long blocks = std::max(1ll, std::min<long long>(((long long)c.N * c.H + 3) / 4, kCUs * 64));
    rows_kernel<T><<<(unsigned)blocks, 256, 0, stream>>>(c, cache);
    return hipGetLastError();
}

}  // namespace

size_t attention_fp4_workspace_bytes(const AttnLaunch& c) {
    switch (c.dtype) {
        case GDN_F32: return plan<F32>(c).bytes;
        case GDN_BF16: return plan<BF16>(c).bytes;
        default: return plan<F16>(c).bytes;
    }
}

hipError_t launch_attention_fp4(const AttnLaunch& c, const Fp4Cache& cache, hipStream_t stream) {
    switch (c.dtype) {
        case GDN_F32: return launch<F32>(c, cache, stream);
        case GDN_BF16: return launch<BF16>(c, cache, stream);
        default: return launch<F16>(c, cache, stream);
    }
}

}  // namespace gdn
