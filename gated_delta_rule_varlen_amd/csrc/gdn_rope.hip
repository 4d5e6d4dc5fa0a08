// gdn_rope.hip -- per-head RMS norm of q and k, rotary positions and the write of the new keys and
// values into the cache, in one pass over the packed tokens (gdn_qk_norm_rope_varlen).
//
// One row is one head of one token.  A wave takes a token (or a quarter of its rows, where tokens are few):
// 64 / L rows at a time, L lanes of two 16-byte pieces each.  The two pieces of a lane hold whole pairs --
// piece j of the low and of the high half, or two neighbouring pieces when pairs are neighbours -- so a
// rotation needs no exchange, and the sum of squares is a butterfly over L lanes.  The token's (cos, sin)
// table is computed once, a pair a lane, and read back from LDS.  Halves that are no multiple of 16
// bytes take the plain kernel at the end, one piece a lane and the pair's other element read by itself.
//
// The angle is formed and reduced to a fraction of a turn in fp64 -- position * frequency passes 2^20 turns
// on long contexts, where an fp32 product has no fraction left -- and only that fraction goes to the fp32
// sincos.  Bound by the bytes of the rows.
#include <hip/hip_runtime.h>

#include <climits>

#include "gdn_device.hpp"
#include "gdn_launch.hpp"

namespace gdn {
namespace {

constexpr int NT = 256;        // threads per block
constexpr int MAX_TPB = 8;     // tokens per block at most
constexpr int MAX_HALF = 128;  // rotated pairs at most

// Whole-call check: the offsets, and for every sequence with tokens the rows it writes.  Also counts
// the offsets at or below token t0, which gives its sequence (the last one starting there, so empty
// sequences are passed over).  Reached by all threads of the block.
__device__ __forceinline__ bool rope_malformed(const RopeLaunch& a, int t0, int& b0) {
    int bad = 0, at_or_below = 0;
    for (int i = threadIdx.x; i <= a.B; i += NT) {
        const int o = a.offsets[i];
        if (i == 0) {
            bad |= (o != 0);
        } else {
            const int prev = a.offsets[i - 1];
            bad |= (prev > o);
            if (prev < o) {
                const long long past = a.past != nullptr ? a.past[i - 1] : 0;
                bad |= (past < 0);
                if (a.kv_begin != nullptr) {
                    const long long begin = a.kv_begin[i - 1];
                    bad |= (begin < 0) | (begin > a.cache_rows) | (begin + past + ((long long)o - prev) > a.cache_rows);
                }
            }
        }
        if (i == a.B) bad |= (o != a.N);
        at_or_below += (o <= t0);
    }
    __shared__ int count;
    if (threadIdx.x == 0) count = 0;
    const bool malformed = __syncthreads_or(bad) != 0;
    if (at_or_below != 0) atomicAdd(&count, at_or_below);
    __syncthreads();
    b0 = count - 1;
    return malformed;
}

// (cos, sin) of pair j at position pos.
__device__ __forceinline__ float2 turn_of(long long pos, float freq) {
    const double turns = (double)pos * (double)freq * 0.15915494309189535;  // 1 / (2 pi)
    const float f = (float)(turns - rint(turns));                           // [-1/2, 1/2] turns
    float s, c;
    sincospif(2.0f * f, &s, &c);
    return make_float2(c, s);
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// wpt waves share a token's rows; a block takes tpb tokens.  LOG2_L: log2 of the lanes of a row.
template <typename T, int LOG2_L, bool NEIGHBOURS>
__global__ __launch_bounds__(NT) void rope_rows_kernel(RopeLaunch a, int tpb, int wpt) {
    using TS = typename T::storage;
    constexpr int VEC = 16 / sizeof(TS), L = 1 << LOG2_L, R = 64 / L, UNROLL = 4;
    __shared__ float2 turn[NT / 64][MAX_HALF];
    const int t0 = blockIdx.x * tpb, half = a.rot / 2, lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    int b;
    const bool malformed = rope_malformed(a, t0, b);
    report_status(a.dev_status, malformed);
    if (malformed) return;
    b = uniform(b);

    // the lane's two pieces
    const int j = lane & (L - 1), pairs = half / VEC;
    int e0, e1;
    if (NEIGHBOURS) {
        e0 = 2 * j * VEC;
        e1 = e0 + VEC;
    } else if (j < pairs) {
        e0 = j * VEC;
        e1 = e0 + half;
    } else {
        e0 = a.rot + 2 * (j - pairs) * VEC;
        e1 = e0 + VEC;
    }
    const bool in0 = e0 < a.D, in1 = e1 < a.D, turns = NEIGHBOURS ? e0 < a.rot : j < pairs;
    float wq[2 * VEC], wk[2 * VEC];
#pragma unroll
    for (int i = 0; i < 2 * VEC; ++i) {
        const int e = i < VEC ? e0 + i : e1 + i - VEC;
        wq[i] = a.q_weight != nullptr && e < a.D ? a.q_weight[e] : 1.0f;
        wk[i] = a.k_weight != nullptr && e < a.D ? a.k_weight[e] : 1.0f;
    }
    const int heads = a.H + a.HK + (a.v.p != nullptr ? a.HK : 0), share = wave % wpt;

    for (int t = t0 + wave / wpt; t < min(t0 + tpb, a.N); t += NT / 64 / wpt) {
        while (b + 1 < a.B && a.offsets[b + 1] <= t) ++b;
        const int i_tok = t - a.offsets[b];
        const long long past = a.past != nullptr ? a.past[b] : 0;
        const long long pos = (a.positions != nullptr ? a.positions[b] : past) + i_tok;
        const long long row = a.kv_begin != nullptr ? a.kv_begin[b] + past + i_tok : t;
        union Piece {
            u32x4 v;
            TS e[VEC];
        };
        auto place = [&](const HeadRows& r, long long at, int h) { return static_cast<TS*>(r.p) + at * r.row + h * r.head; };
        auto source = [&](int h) {
            return h < a.H ? place(a.q, t, h) : h < a.H + a.HK ? place(a.k, t, h - a.H) : place(a.v, t, h - a.H - a.HK);
        };
        auto target = [&](int h) {
            return h < a.H ? place(a.q_out, t, h)
                           : h < a.H + a.HK ? place(a.k_out, row, h - a.H) : place(a.v_out, row, h - a.H - a.HK);
        };
        // the first rows are on their way while the table is computed
        const int h0 = share * R + lane / L, step = wpt * R;
        Piece x[UNROLL][2];
        auto fetch = [&](int hb) {
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int h = hb + u * step;
                // lanes without a piece read the row's first (and count it as zero below): no load in a branch
                const TS* p = source(min(h, heads - 1));
                x[u][0].v = *reinterpret_cast<const u32x4*>(p + (in0 ? e0 : 0));
                x[u][1].v = *reinterpret_cast<const u32x4*>(p + (in1 ? e1 : 0));
            }
        };
        fetch(h0);
        for (int i = lane; i < half; i += 64) turn[wave][i] = turn_of(pos, a.inv_freq[i]);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        float2 cs[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            cs[i] = turns && e0 / (NEIGHBOURS ? 2 : 1) + i < half ? turn[wave][e0 / (NEIGHBOURS ? 2 : 1) + i] : make_float2(1.0f, 0.0f);
        for (int hb = h0; hb - lane / L < heads; hb += UNROLL * step) {
            if (hb != h0) fetch(hb);
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int h = hb + u * step;
                float y[2 * VEC], ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 2 * VEC; ++i) {
                    y[i] = to_f32<T>(x[u][i / VEC].e[i % VEC]);
                    ss = fmaf(y[i], (i < VEC ? in0 : in1) ? y[i] : 0.0f, ss);
                }
                ss = group_sum<L>(ss);
                if (h >= heads) continue;
                if (h < a.H + a.HK) {
                    const float inv = 1.0f / sqrtf(ss / (float)a.D + a.eps);
                    const bool is_q = h < a.H;
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) y[i] = y[i] * inv * (is_q ? wq[i] : wk[i]);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const int lo = NEIGHBOURS ? 2 * i : i, hi = NEIGHBOURS ? 2 * i + 1 : VEC + i;
                        const float p = y[lo], q = y[hi];
                        y[lo] = p * cs[i].x - q * cs[i].y;
                        y[hi] = p * cs[i].y + q * cs[i].x;
                    }
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) x[u][i / VEC].e[i % VEC] = from_f32<T>(y[i]);
                }
                TS* p = target(h);
                if (in0) *reinterpret_cast<u32x4*>(p + e0) = x[u][0].v;
                if (in1) *reinterpret_cast<u32x4*>(p + e1) = x[u][1].v;
            }
        }
    }
}

// Any rotated width: one piece a lane, the pair's other element read by itself.
template <typename T>
__global__ __launch_bounds__(NT) void rope_kernel(RopeLaunch a, int tpb, int log2_lanes) {
    using TS = typename T::storage;
    constexpr int VEC = 16 / sizeof(TS);
    __shared__ float2 turn[MAX_TPB * MAX_HALF];
    __shared__ int seq[MAX_TPB];
    const int t0 = blockIdx.x * tpb, nt = min(tpb, a.N - t0), half = a.rot / 2;
    int b0;
    const bool malformed = rope_malformed(a, t0, b0);
    report_status(a.dev_status, malformed);
    if (malformed || nt <= 0) return;
    if (threadIdx.x < nt) {
        int b = b0;
        while (b + 1 < a.B && a.offsets[b + 1] <= t0 + (int)threadIdx.x) ++b;
        seq[threadIdx.x] = b;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * half; i += NT) {
        const int tk = i / half, j = i - tk * half, b = seq[tk];
        const int* first = a.positions != nullptr ? a.positions : a.past;
        const long long pos = (long long)(first != nullptr ? first[b] : 0) + (t0 + tk - a.offsets[b]);
        turn[i] = turn_of(pos, a.inv_freq[j]);
    }
    __syncthreads();

    const int lanes = 1 << log2_lanes, lane = threadIdx.x & (lanes - 1), e0 = lane * VEC;
    const int heads = a.H + a.HK + (a.v.p != nullptr ? a.HK : 0);
    const bool in = e0 < a.D;
    const int rows = nt * heads, step = NT >> log2_lanes;
    // every lane of a group stays in the loop for the group sum
    for (int r = threadIdx.x >> log2_lanes; r < rows; r += step) {
        const int tk = r / heads, h = r - tk * heads, t = t0 + tk, b = seq[tk];
        const bool is_q = h < a.H, is_v = h >= a.H + a.HK;
        const int hh = is_q ? h : is_v ? h - a.H - a.HK : h - a.H;
        const HeadRows &src = is_q ? a.q : is_v ? a.v : a.k, &dst = is_q ? a.q_out : is_v ? a.v_out : a.k_out;
        long long row = t;
        if (!is_q && a.kv_begin != nullptr)
            row = a.kv_begin[b] + (a.past != nullptr ? a.past[b] : 0) + (t - a.offsets[b]);
        const TS* x = static_cast<const TS*>(src.p) + t * src.row + hh * src.head;
        TS* y = static_cast<TS*>(dst.p) + row * dst.row + hh * dst.head;
        union Chunk {
            u32x4 v;
            TS e[VEC];
        } raw;
        raw.v = in ? *reinterpret_cast<const u32x4*>(x + e0) : u32x4{0u, 0u, 0u, 0u};
        if (is_v) {
            if (in) *reinterpret_cast<u32x4*>(y + e0) = raw.v;
            continue;
        }
        float own[VEC], ss = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            own[e] = to_f32<T>(raw.e[e]);
            ss = fmaf(own[e], own[e], ss);
        }
        for (int m = 1; m < lanes; m <<= 1) ss += __shfl_xor(ss, m);
        const float inv = 1.0f / sqrtf(ss / (float)a.D + a.eps);
        const float* w = is_q ? a.q_weight : a.k_weight;
        auto normed = [&](int e, float v) { return v * inv * (w != nullptr ? w[e] : 1.0f); };
        if (in) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int e = e0 + i;
                float v = normed(e, own[i]);
                if (e < a.rot) {
                    const bool low = a.interleaved ? (i & 1) == 0 : e < half;
                    const int pair = a.interleaved ? e >> 1 : low ? e : e - half;
                    const int other = a.interleaved ? e ^ 1 : low ? e + half : e - half;
                    const float o = normed(other, to_f32<T>(x[other]));
                    const float2 cs = turn[tk * half + pair];
                    v = low ? v * cs.x - o * cs.y : o * cs.y + v * cs.x;
                }
                raw.e[i] = from_f32<T>(v);
            }
            *reinterpret_cast<u32x4*>(y + e0) = raw.v;
        }
    }
}

template <typename T>
hipError_t launch(const RopeLaunch& a, hipStream_t stream) {
    constexpr int VEC = 16 / (int)sizeof(typename T::storage);
    int log2_pieces = 0;
    while ((VEC << log2_pieces) < a.D) ++log2_pieces;
    if (!a.interleaved && a.rot / 2 % VEC != 0) {
        const int tpb = a.N > 1024 ? 4 : 1;
        const int blocks = a.N > 0 ? (a.N + tpb - 1) / tpb : 1;
        rope_kernel<T><<<blocks, NT, 0, stream>>>(a, tpb, log2_pieces);
        return hipGetLastError();
    }
    // a block's four waves share a token while that still leaves idle CUs, else take four tokens each
    const int wpt = a.N <= 1024 ? 4 : 1, tpb = a.N <= 1024 ? 1 : a.N <= 8192 ? 4 : 16;
    const int blocks = a.N > 0 ? (a.N + tpb - 1) / tpb : 1;
    auto go = [&](auto kernel) {
        kernel<<<blocks, NT, 0, stream>>>(a, tpb, wpt);
        return hipGetLastError();
    };
    // lanes of a row: its pairs' (or neighbours') two pieces each, the rest of the row two each
    const int pieces = (a.D + VEC - 1) / VEC, pairs = a.rot / 2 / VEC;
    const int lanes = a.interleaved ? (pieces + 1) / 2 : pairs + (pieces - 2 * pairs + 1) / 2;
    int l = 0;
    while ((1 << l) < lanes) ++l;
    switch (l) {
#define GDN_ROPE_CASE(n) \
    case n: return a.interleaved ? go(rope_rows_kernel<T, n, true>) : go(rope_rows_kernel<T, n, false>);
        GDN_ROPE_CASE(0)
        GDN_ROPE_CASE(1)
        GDN_ROPE_CASE(2)
        GDN_ROPE_CASE(3)
        GDN_ROPE_CASE(4)
#undef GDN_ROPE_CASE
        default: return a.interleaved ? go(rope_rows_kernel<T, 5, true>) : go(rope_rows_kernel<T, 5, false>);
    }
}

}  // namespace

hipError_t launch_rope(const RopeLaunch& a, hipStream_t stream) {
    switch (a.dtype) {
        case GDN_F32: return launch<F32>(a, stream);
        case GDN_BF16: return launch<BF16>(a, stream);
        default: return launch<F16>(a, stream);
    }
}

}  // namespace gdn
