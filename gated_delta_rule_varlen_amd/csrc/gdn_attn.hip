// gdn_attn.hip -- host side of the softmax attention: which form and tile a call takes, its workspace, and
// the kernel that joins key parts.  The tile kernels are in gdn_attn.hpp.
//
// Short form (max_q * G rows fit a tile of 32, 64 or 128): decode steps and short blocks, bound by the
// cache's bytes.  Long form: prompts, bound by the matrix cores.  A shared prefix is one more run of
// keys for the long form's tiles; for the short form a launch of its own first runs all tokens' rows
// over the prefix, reading it once for the whole batch.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdn_attn.hpp"

namespace gdn {
namespace {

using namespace attn;

constexpr int kCUs = 256;
constexpr int kShortRows = 128;

// Joins the parts of a row: pieces of a cut run (a chain of workers' slots) and sets [0, sets).  One block of
// 1 or 4 waves a row (token, head); its waves share the parts.
template <typename T, int NW>
__global__ __launch_bounds__(64 * NW) void join_kernel(Args a, int bm, int local_set) {
    using TS = typename T::storage;
    if (*a.status != 0) return;
    const long long row = blockIdx.x;
    const int t = (int)(row / a.c.H), h = (int)(row - (long long)t * a.c.H), hk = h / a.G;
    int worker = -1, pieces = 0;
    long long slot_row = 0;
    if (a.row_info != nullptr) {
        const int2 info = a.row_info[(long long)t * a.c.HK + hk];
        worker = info.x;
        if (worker >= 0) {
            pieces = info.y >> 7;
            slot_row = (info.y & 127) * a.G + (h - hk * a.G);
        } else if (a.sets == 0) {
            return;  // written whole
        }
    }
    const int sets = a.sets - (worker >= 0 && local_set >= 0 ? 1 : 0);  // a cut run left its own set (the last) unused
    const int parts = pieces + sets, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // the first piece is slot 1 of its worker, the others slot 0 of the following ones
    auto slot = [&](int p) { return ((long long)(worker + p) * 2 + (p == 0 ? 1 : 0)) * bm + slot_row; };
    auto ml_of = [&](int p) { return p < pieces ? a.slot_ml[slot(p)] : a.set_ml[(p - pieces) * a.set_rows + row]; };
    float top = kNoMax;
    for (int p = lane; p < parts; p += 64) top = fmaxf(top, ml_of(p).x);
    for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
    float l = 0.0f;
    for (int p = lane; p < parts; p += 64) {
        const float2 ml = ml_of(p);
        l += ml.y * __builtin_amdgcn_exp2f(ml.x - top);
    }
    l = group_sum<64>(l);
    f32x4 o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int e = 4 * lane;
    if (e < a.c.D) {
#pragma unroll 4
        for (int p = wave; p < parts; p += NW) {
            const float w = __builtin_amdgcn_exp2f(ml_of(p).x - top);
            const float* src = p < pieces ? a.slot_o + slot(p) * a.c.D : a.set_o + ((p - pieces) * a.set_rows + row) * a.c.D;
            o += w * *reinterpret_cast<const f32x4*>(src + e);
        }
    }
    if constexpr (NW > 1) {
        __shared__ f32x4 xo[NW][64];
        xo[wave][lane] = o;
        __syncthreads();
        if (wave != 0) return;
        for (int w = 1; w < NW; ++w) o += xo[w][lane];
    }
    if (e < a.c.D) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        TS* out = static_cast<TS*>(a.c.out.p) + t * a.c.out.row + h * a.c.out.head;
        for (int j = 0; j < 4; ++j) out[e + j] = from_f32<T>(o[j] * inv);
    }
    if (a.c.lse != nullptr && threadIdx.x == 0)
        a.c.lse[row] = l == 0.0f ? -INFINITY : kLn2 * (top + __builtin_amdgcn_logf(l));
}

template <typename T>
Shape shape(int dp, int wr) {
    return with_pick<T>(dp, wr, [](auto p) { return shape_of<typename decltype(p)::C>(); });
}

struct Plan {
    Args a;
    bool is_short, join;
    int dp, wr, bm;
    long long blocks, prefix_blocks;
    size_t bytes;
};

template <typename T>
Plan plan(const AttnLaunch& c) {
    Plan p{};
    Args& a = p.a;
    a.c = c;
    a.G = c.H / c.HK;
    a.s2 = fabsf(c.scale) * kLog2e;
    a.negate = c.scale < 0.0f;
    a.splits = 1;
    a.set_rows = (long long)c.N * c.H;
    p.dp = c.D <= 64 ? 64 : c.D <= 128 ? 128 : 256;
    const long long rows = (long long)c.max_q * a.G;
    p.is_short = rows <= kShortRows;
    p.wr = !p.is_short || rows > 64 ? 4 : rows > 32 ? 2 : 1;
    const Shape s = shape<T>(p.dp, p.wr), whole = shape<T>(p.dp, 4);
    p.bm = s.bm;
    // key parts of the long form: enough blocks for two a CU, each with a few tiles at least
    auto parts = [&](long long tiles, long long keys) {
        const long long want = (2 * kCUs + tiles - 1) / std::max(1ll, tiles), most = keys / (4 * whole.bn);
        return (int)std::max(1ll, std::min(std::min(want, most), 64ll));
    };
    const long long N = c.N, all_rows = N * a.G;
    if (p.is_short) {
        const long long units = c.HK * (c.kv_rows / s.bn + c.B);  // fewer blocks than that have work, bar overlapping runs
        a.workers = (int)std::max(1ll, std::min((long long)kCUs * s.per_cu, units));
        p.blocks = a.workers;
        if (c.prefix_len > 0 && c.N > 0) {
            const long long tiles = (all_rows + whole.bm - 1) / whole.bm;
            a.splits = parts(tiles * c.HK, c.prefix_len);
            p.prefix_blocks = tiles * c.HK * a.splits;
            a.sets = a.splits + 1;
            a.to_sets = true;
            a.set0 = a.splits;
        }
        p.join = c.N > 0 && (a.workers > 1 || a.sets > 0);
    } else {
        const long long most = (rows + whole.bm - 1) / whole.bm;  // tiles of the longest sequence
        a.splits = parts(std::min(most * c.B, all_rows / whole.bm + c.B) * c.HK, c.kv_rows + c.prefix_len);
        p.blocks = most * c.B * c.HK * a.splits;
        if (a.splits > 1) {
            a.sets = a.splits;
            a.to_sets = true;
            p.join = true;
        }
    }
    size_t at = 0;
    auto take = [&](size_t n) {
        char* r = static_cast<char*>(c.workspace) + at;
        at += (n + 255) / 256 * 256;
        return r;
    };
    if (p.join) {
        a.status = reinterpret_cast<int*>(take(4));
        if (p.is_short) {
            a.row_info = reinterpret_cast<int2*>(take(N * c.HK * 8));
            a.slot_ml = reinterpret_cast<float2*>(take((size_t)a.workers * 2 * p.bm * 8));
            a.slot_o = reinterpret_cast<float*>(take((size_t)a.workers * 2 * p.bm * c.D * 4));
        }
        if (a.sets > 0) {
            a.set_ml = reinterpret_cast<float2*>(take((size_t)a.sets * a.set_rows * 8));
            a.set_o = reinterpret_cast<float*>(take((size_t)a.sets * a.set_rows * c.D * 4));
        }
    }
    p.bytes = at;
    return p;
}

template <typename T>
hipError_t launch(const AttnLaunch& c, hipStream_t stream) {
    Plan p = plan<T>(c);
    if (p.blocks > kMaxBlocks || p.prefix_blocks > kMaxBlocks || (p.join && p.a.set_rows > kMaxBlocks))
        return hipErrorInvalidConfiguration;
    hipError_t e;
    if (p.is_short) {
        if (p.prefix_blocks > 0) {
            Args a = p.a;
            a.prefix_rows = true;
            a.set0 = 0;
            if ((e = start_long<T>(a, p.dp, p.prefix_blocks, stream)) != hipSuccess) return e;
        }
        e = start_short<T>(p.a, p.dp, p.wr, p.blocks, stream);
    } else {
        e = start_long<T>(p.a, p.dp, p.blocks, stream);
    }
    if (e != hipSuccess || !p.join) return e;
    const int local = p.is_short && p.a.sets > 0 ? p.a.set0 : -1;
    if (p.a.set_rows <= 4 * kCUs) join_kernel<T, 4><<<(unsigned)p.a.set_rows, 256, 0, stream>>>(p.a, p.bm, local);
    else join_kernel<T, 1><<<(unsigned)p.a.set_rows, 64, 0, stream>>>(p.a, p.bm, local);
    return hipGetLastError();
}

}  // namespace

size_t attention_workspace_bytes(const AttnLaunch& c) {
    switch (c.dtype) {
        case GDN_F32: return plan<F32>(c).bytes;
        case GDN_BF16: return plan<BF16>(c).bytes;
        default: return plan<F16>(c).bytes;
    }
}

hipError_t launch_attention(const AttnLaunch& c, hipStream_t stream) {
    switch (c.dtype) {
        case GDN_F32: return launch<F32>(c, stream);
        case GDN_BF16: return launch<BF16>(c, stream);
        default: return launch<F16>(c, stream);
    }
}

}  // namespace gdn
