// gdn_attn_join.hpp -- the kernels that join a row's key parts, for the attentions over a plain cache and a 4-bit one.
#pragma once

#include "gdn_attn.hpp"

namespace gdn {
namespace attn {

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

// Rows few enough for a block each.
inline bool few_rows(const Args& a) { return a.set_rows <= 8 * kCUs; }

// Starts the joining kernel of a call whose parts lie in slots of bm rows and in sets; local_set as in Parts::find.
template <typename T>
hipError_t start_join(const Args& a, int bm, int local_set, hipStream_t stream) {
    const long long blocks = (a.set_rows + 3) / 4, most_x = kMaxThreads / 256;
    const dim3 fours((unsigned)std::min(blocks, most_x), (unsigned)((blocks + most_x - 1) / most_x));
    if (a.cut != nullptr) {
        const unsigned most = (unsigned)(a.c.max_q * a.G + 3) / 4;
        join_cut_kernel<T><<<dim3((unsigned)a.workers, most), 256, 0, stream>>>(a, bm);
    } else if (few_rows(a)) {
        join_few_kernel<T><<<dim3((unsigned)a.set_rows, (a.c.D + 63) / 64), 256, 0, stream>>>(a, bm, local_set);
    } else if (a.c.D <= 64) {
        join_rows_kernel<T, 16><<<fours, 256, 0, stream>>>(a, bm, local_set);
    } else if (a.c.D <= 128) {
        join_rows_kernel<T, 32><<<fours, 256, 0, stream>>>(a, bm, local_set);
    } else {
        join_rows_kernel<T, 64><<<fours, 256, 0, stream>>>(a, bm, local_set);
    }
    return hipGetLastError();
}

}  // namespace attn
}  // namespace gdn
