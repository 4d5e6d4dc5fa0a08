// gdn_attn.hip -- host side of the softmax attention: which form and tile a call takes, its workspace, and
// the kernel that joins key parts.  The tile kernels are in gdn_attn.hpp.
//
// Short form (max_q * G rows are 128 at most): decode steps and short blocks, bound by the
// cache's bytes.  Long form: prompts, bound by the matrix cores.  A shared prefix is one more run of
// keys for the long form's tiles; beside the short form, blocks of the long form run all tokens' rows over
// the prefix, reading it once for the whole batch: in a launch of their own, or for small calls in the same one
// (both_kernel).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdn_attn.hpp"

namespace gdn {
namespace {

using namespace attn;

constexpr int kShortRows = 128;

// A row's result from its parts' sums: out and lse.
template <typename T>
__device__ __forceinline__ void finish(const Args& a, int t, int h, int e, f32x4 o, float top, float l, bool stats) {
    using TS = typename T::storage;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    union {
        TS s[4];
        f32x4 f;
        u32x2 u;
    } y;
    for (int j = 0; j < 4; ++j) y.s[j] = from_f32<T>(o[j] * inv);
    TS* out = static_cast<TS*>(a.c.out.p) + t * a.c.out.row + h * a.c.out.head + e;
    if constexpr (sizeof(TS) == 2) *reinterpret_cast<u32x2*>(out) = y.u;
    else *reinterpret_cast<f32x4*>(out) = y.f;
    if (stats && a.c.lse != nullptr)
        a.c.lse[(long long)t * a.c.H + h] = l == 0.0f ? -INFINITY : kLn2 * (top + __builtin_amdgcn_logf(l));
}

// The parts of row (t, h): the pieces of a cut run (a chain of workers' slots) and the first `sets` sets.
struct Parts {
    long long row, slot_row;
    int worker, pieces, all;
    __device__ __forceinline__ void find(const Args& a, int t, int h, int local_set) {
        const int hk = h / a.G;
        row = (long long)t * a.c.H + h;
        worker = -1;
        pieces = 0;
        slot_row = 0;
        if (a.row_info != nullptr) {
            const int2 info = a.row_info[(long long)t * a.c.HK + hk];
            worker = info.x;
            if (worker >= 0) {
                pieces = info.y >> 7;
                slot_row = (info.y & 127) * a.G + (h - hk * a.G);
            }
        }
        // a cut run left its own set (the last) unused; a run that was not, without sets, is written already
        all = pieces + (a.live != nullptr ? a.live[t] : a.sets) - (worker >= 0 && local_set >= 0 ? 1 : 0);
    }
    // Adds part p to the running (top, l, o) of elements e .. e + 3.
    __device__ __forceinline__ void add(const Args& a, int bm, int p, int e, float& top, float& l, f32x4& o) const {
        // the first piece is slot 1 of its worker, the others slot 0 of the following ones
        const bool piece = p < pieces;
        const long long at = piece ? ((long long)(worker + p) * 2 + (p == 0 ? 1 : 0)) * bm + slot_row : (p - pieces) * a.set_rows + row;
        const float2 ml = (piece ? a.slot_ml : a.set_ml)[at];
        const f32x4 x = *reinterpret_cast<const f32x4*>((piece ? a.slot_o : a.set_o) + at * a.c.D + (e < a.c.D ? e : 0));
        merge(top, l, o, ml.x, ml.y, x);
    }
    static __device__ __forceinline__ void merge(float& top, float& l, f32x4& o, float m, float s, f32x4 x) {
        const float to = fmaxf(top, m), w = __builtin_amdgcn_exp2f(top - to), wx = __builtin_amdgcn_exp2f(m - to);
        top = to;
        l = l * w + s * wx;
        o = o * w + x * wx;
    }
};

// Few rows, perhaps of many parts: a block a row and 64 elements of it; 16 lanes hold the elements and the 16
// groups of them share the parts.
template <typename T>
__global__ __launch_bounds__(256) void join_few_kernel(Args a, int bm, int local_set) {
    const int status = *a.status;  // asked for together with the row's information
    const int t = blockIdx.x / a.c.H, h = blockIdx.x - t * a.c.H;
    Parts parts;
    parts.find(a, t, h, local_set);
    if (parts.all == 0 || status != 0) return;
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4, e = blockIdx.y * 64 + 4 * lane;
    float top = kNoMax, l = 0.0f;
    f32x4 o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int p = group; p < parts.all; p += 16) parts.add(a, bm, p, e, top, l, o);
    __shared__ f32x4 xo[16][16];
    __shared__ float2 xm[16];
    xo[group][lane] = o;
    if (lane == 0) xm[group] = make_float2(top, l);
    __syncthreads();
    if (group != 0) return;
    for (int g = 1; g < min(parts.all, 16); ++g) Parts::merge(top, l, o, xm[g].x, xm[g].y, xo[g][lane]);
    if (e < a.c.D) finish<T>(a, t, h, e, o, top, l, e == 0);
}

// Many rows: `lanes` (16, 32 or 64) of a wave hold a row's elements, its other groups of so many share the parts.
// A block takes four rows; the grid's second axis is there for more rows than one axis counts threads for.
template <typename T, int LANES>
__global__ __launch_bounds__(256) void join_rows_kernel(Args a, int bm, int local_set) {
    const int status = *a.status;
    const long long row = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (row >= a.set_rows) return;
    const int t = (int)(row / a.c.H), h = (int)(row - (long long)t * a.c.H);
    Parts parts;
    parts.find(a, t, h, local_set);
    if (parts.all == 0 || status != 0) return;
    const int lane = threadIdx.x & (LANES - 1), group = (threadIdx.x & 63) / LANES, e = 4 * lane;
    float top = kNoMax, l = 0.0f;
    f32x4 o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int p = group; p < parts.all; p += 64 / LANES) parts.add(a, bm, p, e, top, l, o);
    for (int x = LANES; x < 64; x <<= 1) {
        const f32x4 y = f32x4{__shfl_xor(o[0], x), __shfl_xor(o[1], x), __shfl_xor(o[2], x), __shfl_xor(o[3], x)};
        const float m = __shfl_xor(top, x), s = __shfl_xor(l, x);
        Parts::merge(top, l, o, m, s, y);
    }
    if (group == 0 && e < a.c.D) finish<T>(a, t, h, e, o, top, l, lane == 0);
}

// Many rows, of which few were cut: for every worker, the run that starts there and goes on; a wave a row.
template <typename T>
__global__ __launch_bounds__(256) void join_cut_kernel(Args a, int bm) {
    const int status = *a.status;
    const int4 cut = a.cut[blockIdx.x];  // first token, tokens, key head, pieces
    if (status != 0) return;
    const int lane = threadIdx.x & 63, e = 4 * lane, r = blockIdx.y * 4 + (threadIdx.x >> 6);
    if (r >= cut.y * a.G) return;
    Parts parts{0, r, (int)blockIdx.x, cut.w, cut.w};
    float top = kNoMax, l = 0.0f;
    f32x4 o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
    for (int p = 0; p < cut.w; ++p) parts.add(a, bm, p, e, top, l, o);
    const int i = r / a.G;
    if (e < a.c.D) finish<T>(a, cut.x + i, cut.z * a.G + r - i * a.G, e, o, top, l, lane == 0);
}

struct Plan {
    Args a;
    bool is_short, join, both;
    int dp, wr, bm;
    int lds, long_lds, threads, long_threads;
    long long blocks;
    size_t bytes;
};

// Rows few enough for a block each.
bool few_rows(const Args& a) { return a.set_rows <= 8 * kCUs; }

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
    const long long rows = (long long)c.max_q * a.G, es = sizeof(typename T::storage);
    p.wr = rows <= 64 ? (int)(rows + 15) / 16 : 8;
    if (p.wr < 1) p.wr = 1;
    const Shape s = with_short<T>(p.dp, p.wr, Shape{0, 0, kMaxLds + 1, 0, 0}, [](auto x) { return shape_of<typename decltype(x)::C>(); });
    const Shape whole = with_long<T>(p.dp, [](auto x) { return shape_of<typename decltype(x)::C>(); });
    // the short form's queries lie in LDS beside the ring, and a run's span a 32-bit range
    const long long q_lds = (rows + 7) / 8 * 8 * s.row;
    const long double q_span = ((long double)c.max_q * c.q.row + (long double)a.G * c.q.head) * es;
    p.is_short = rows <= kShortRows && s.ring + q_lds <= kMaxLds && q_span < kOutside;
    p.long_lds = whole.ring;
    p.threads = p.long_threads = whole.threads;
    // Key parts of the long form: enough blocks for two a CU, each of kPartKeys keys at least.  The sequences' own
    // lengths are on the device: there a sequence takes as many of the parts as its keys fill.
    auto parts = [&](long long tiles, long long keys) {
        const long long want = (2 * kCUs + tiles - 1) / std::max(1ll, tiles), most = keys / kPartKeys;
        return (int)std::max(1ll, std::min(std::min(want, most), 64ll));
    };
    const long long N = c.N, all_rows = N * a.G;
    bool by_rows = true;
    if (p.is_short) {
        p.bm = s.bm;
        p.threads = s.threads;
        p.lds = (int)(s.ring + q_lds);
        if (c.prefix_len > 0 && c.N > 0) {
            const long long tiles = (all_rows + whole.bm - 1) / whole.bm;
            a.splits = parts(tiles * c.HK, c.prefix_len);
            a.prefix_blocks = tiles * c.HK * a.splits;
            a.sets = a.splits + 1;
            a.to_sets = true;
            a.local_set = a.splits;
        }
        const int per_cu = std::min(8, kCULds / ((p.lds + 1279) / 1280 * 1280));  // LDS is handed out in 1280 bytes
        const long long units = c.HK * (c.kv_rows / s.bn + c.B);  // fewer blocks than that have work, bar overlapping runs
        a.workers = (int)std::max(1ll, std::min((long long)kCUs * per_cu, units));
        p.blocks = a.workers;
        // Both forms in one launch where all blocks run at once (8 drafts behind 1001 shared keys: 12.4 us, in two
        // launches 18.7).  In more rounds the short form's blocks are too few on a CU beside the long form's
        // (256 sequences behind 8192 keys: 136 us, in two launches 130).
        p.both = a.prefix_blocks > 0 && a.prefix_blocks + a.workers <= 2 * kCUs && p.wr <= 4 && joint(whole.ring, p.lds);
        if (p.both) {
            p.lds = std::max(p.lds, whole.ring);
            p.threads = p.long_threads;
            p.blocks = ((a.prefix_blocks + kCUs - 1) / kCUs + (a.workers + kCUs - 1) / kCUs) * kCUs;  // whole turns
        }
        p.join = c.N > 0 && (a.workers > 1 || a.sets > 0);
        by_rows = a.sets > 0 || few_rows(a);
    } else {
        // One block for every slot that a row tile can have, however long max_q says that one sequence may be.  (With
        // blocks for each sequence as for the longest, one prompt of 8192 tokens among 63 of up to 200 took 1220 us,
        // so 557; max_q = N for eight prompts 756 and 680.  In the order of their keys 64 fp32 prompts of up to
        // 300 tokens take 275 us, as they come 326.)
        const long long most = (rows + whole.bm - 1) / whole.bm, slots = all_rows / whole.bm + c.B;
        a.splits = parts(std::min(most * c.B, slots) * c.HK, c.kv_rows + c.prefix_len);
        p.blocks = slots * c.HK * a.splits;
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
            if (by_rows) a.row_info = reinterpret_cast<int2*>(take(N * c.HK * 8));
            else a.cut = reinterpret_cast<int4*>(take((size_t)a.workers * 16));
            a.slot_ml = reinterpret_cast<float2*>(take((size_t)a.workers * 2 * p.bm * 8));
            a.slot_o = reinterpret_cast<float*>(take((size_t)a.workers * 2 * p.bm * c.D * 4));
        }
        if (a.sets > 0) {
            a.set_ml = reinterpret_cast<float2*>(take((size_t)a.sets * a.set_rows * 8));
            a.set_o = reinterpret_cast<float*>(take((size_t)a.sets * a.set_rows * c.D * 4));
            if (!p.is_short) a.live = reinterpret_cast<int*>(take(N * 4));
        }
    }
    p.bytes = at;
    return p;
}

template <typename T>
hipError_t launch(const AttnLaunch& c, hipStream_t stream) {
    Plan p = plan<T>(c);
    if (p.blocks * p.threads > kMaxThreads || p.a.prefix_blocks * p.long_threads > kMaxThreads)
        return hipErrorInvalidConfiguration;
    hipError_t e;
    if (p.is_short) {
        if (p.both) {
            e = start_both<T>(p.a, p.dp, p.wr, p.blocks, p.lds, stream);
        } else {
            if (p.a.prefix_blocks > 0 &&
                (e = start_long<T>(p.a, p.dp, p.a.prefix_blocks, p.long_lds, stream)) != hipSuccess)
                return e;
            e = start_short<T>(p.a, p.dp, p.wr, p.blocks, p.lds, stream);
        }
    } else {
        e = start_long<T>(p.a, p.dp, p.blocks, p.long_lds, stream);
    }
    if (e != hipSuccess || !p.join) return e;
    const int local = p.is_short && p.a.sets > 0 ? p.a.local_set : -1;
    const long long blocks = (p.a.set_rows + 3) / 4, most_x = kMaxThreads / 256;
    const dim3 fours((unsigned)std::min(blocks, most_x), (unsigned)((blocks + most_x - 1) / most_x));
    if (p.a.cut != nullptr) {
        const unsigned most = (unsigned)(c.max_q * p.a.G + 3) / 4;
        join_cut_kernel<T><<<dim3((unsigned)p.a.workers, most), 256, 0, stream>>>(p.a, p.bm);
    } else if (few_rows(p.a)) {
        join_few_kernel<T><<<dim3((unsigned)p.a.set_rows, (c.D + 63) / 64), 256, 0, stream>>>(p.a, p.bm, local);
    } else if (c.D <= 64) {
        join_rows_kernel<T, 16><<<fours, 256, 0, stream>>>(p.a, p.bm, local);
    } else if (c.D <= 128) {
        join_rows_kernel<T, 32><<<fours, 256, 0, stream>>>(p.a, p.bm, local);
    } else {
        join_rows_kernel<T, 64><<<fours, 256, 0, stream>>>(p.a, p.bm, local);
    }
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
