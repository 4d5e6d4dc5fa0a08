// gdn_rope.hip -- per-head RMS norm of q and k, rotary positions and the write of the new keys and
// values into the cache, in one pass over the packed tokens (gdn_qk_norm_rope_varlen).
//
// One row is one head of one token.  A wave takes a token (or a quarter of its passes, where tokens are few), 64 / L
// rows a pass -- the queries, then the keys with the values behind them -- and L lanes of two 16-byte pieces a row.
// The two pieces of a lane hold whole pairs -- piece j of the low and of the high half, or two neighbouring pieces
// when pairs are neighbours -- so a rotation needs no exchange, and the sum of squares is a butterfly over L
// lanes.  The token's (cos, sin) table is computed once, a pair a lane, and read back from LDS.  Halves that are no
// multiple of 16 bytes take the plain kernel at the end, one piece a lane and the pair's other element read by itself.
//
// The angle is formed and reduced to a fraction of a turn in fp64 -- position * frequency passes 2^20 turns
// on long contexts, where an fp32 product has no fraction left -- and only that fraction goes to the fp32
// sincos.
//
// Large batches are bound by the bytes of the rows (24748 tokens, 608 MB, D = 128: 128 us = 4.8 TB/s), narrow heads
// by vector instructions (10277 tokens, D = 64: 18.3 us; 21.7 with values in passes of their own and more selects), a
// decode step by the latencies of one launch (64 tokens: 7.5 us).
#include <hip/hip_runtime.h>

#include <climits>

#include "gdn_device.hpp"
#include "gdn_launch.hpp"

namespace gdn {
namespace {

constexpr int NT = 256;        // threads per block
constexpr int MAX_TPB = 16;    // tokens per block at most
constexpr int MAX_HALF = 128;  // rotated pairs at most

// What the block's tokens need of their sequences.
struct Token {
    long long pos, row;
};

// Whole-call check: the offsets, and for every sequence with tokens the rows it writes.  The thread that holds a
// sequence of the block's tokens t0 .. t1 - 1 leaves their positions and rows in `tok`, so nothing of the call's
// small arrays is read a second time.  Reached by all threads of the block.
__device__ __forceinline__ bool rope_malformed(const RopeLaunch& a, int t0, int t1, Token* tok) {
    int bad = 0;
    for (int i = threadIdx.x; i < a.B; i += NT) {
        const int o = a.offsets[i], e = a.offsets[i + 1];
        const long long past = a.past != nullptr ? a.past[i] : 0;
        const long long first = a.positions != nullptr ? a.positions[i] : past;
        const long long begin = a.kv_begin != nullptr ? a.kv_begin[i] : 0;
        bad |= (i == 0 && o != 0) | (o > e) | (i == a.B - 1 && e != a.N);
        if (o < e) {
            bad |= (past < 0);
            if (a.kv_begin != nullptr)
                bad |= (begin < 0) | (begin > a.cache_rows) | (begin + past + ((long long)e - o) > a.cache_rows);
        }
        for (int t = max(o, t0); t < min(e, t1); ++t)
            tok[t - t0] = Token{first + (t - o), a.kv_begin != nullptr ? begin + past + (t - o) : t};
    }
    return any_in_block<NT>(bad != 0);
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
__device__ __forceinline__ long long uniform(long long x) {
    return ((long long)uniform((int)(x >> 32)) << 32) | (uint32_t)uniform((int)x);
}

// wpt waves share a token's rows; a block takes tpb tokens.  LOG2_L: log2 of the lanes of a row.
template <typename T, int LOG2_L, bool NEIGHBOURS>
__global__ __launch_bounds__(NT) void rope_rows_kernel(RopeLaunch a, int tpb, int wpt) {
    using TS = typename T::storage;
    constexpr int VEC = 16 / sizeof(TS), L = 1 << LOG2_L, R = 64 / L;
    __shared__ float2 turn[NT / 64][MAX_HALF];
    __shared__ Token tok[MAX_TPB];
    const int t0 = blockIdx.x * tpb, t1 = min(t0 + tpb, a.N), half = a.rot / 2;
    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), share = wave % wpt;

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
    const bool in0 = e0 < a.D, in1 = e1 < a.D;
    // lanes without a piece read the row's first (and count it as zero below): no load stands in a branch
    const int r0 = in0 ? e0 : 0, r1 = in1 ? e1 : 0;

    // A pass is R rows: of the queries, or of the keys with the values behind them, of a token.
    const int kv = a.v.p != nullptr ? 2 * a.HK : a.HK, pq = (a.H + R - 1) / R, passes = pq + (kv + R - 1) / R;
    union Piece {
        u32x4 v;
        TS e[VEC];
    };
    struct Rows {
        Piece x[2];
    };
    const TS* const qp = static_cast<const TS*>(a.q.p);
    const TS* const kp = static_cast<const TS*>(a.k.p);
    const TS* const vp = static_cast<const TS*>(a.v.p);
    auto fetch = [&](int t, int p) {
        const TS* src;
        if (p < pq) {
            src = qp + t * a.q.row + min(p * R + lane / L, a.H - 1) * a.q.head;
        } else {
            const int r = min((p - pq) * R + lane / L, kv - 1);
            src = r < a.HK ? kp + t * a.k.row + r * a.k.head : vp + t * a.v.row + (r - a.HK) * a.v.head;
        }
        Rows y;
        y.x[0].v = *reinterpret_cast<const u32x4*>(src + r0);
        y.x[1].v = *reinterpret_cast<const u32x4*>(src + r1);
        return y;
    };
    // the first rows, the weights and the frequencies are on their way while the call is checked
    int t = t0 + wave / wpt;
    Rows next;
    if (t < t1 && share < passes) next = fetch(t, share);
    float freq[MAX_HALF / 64];
#pragma unroll
    for (int i = 0; i < MAX_HALF / 64; ++i) freq[i] = lane + 64 * i < half ? a.inv_freq[lane + 64 * i] : 0.0f;
    float wq[2 * VEC], wk[2 * VEC];
#pragma unroll
    for (int i = 0; i < 2 * VEC; ++i) {
        const int e = i < VEC ? r0 + i : r1 + i - VEC;
        wq[i] = a.q_weight != nullptr ? a.q_weight[e] : 1.0f;
        wk[i] = a.k_weight != nullptr ? a.k_weight[e] : 1.0f;
    }
    // past the pairs the table turns by nothing, for the pieces of the tail
    for (int i = half + lane; i < MAX_HALF; i += 64) turn[wave][i] = make_float2(1.0f, 0.0f);
    const int pair0 = min(NEIGHBOURS ? e0 / 2 : e0, MAX_HALF - VEC);
    const bool malformed = rope_malformed(a, t0, t1, tok);
    report_status(a.dev_status, malformed);
    if (malformed) return;

    const float inv_d = 1.0f / (float)a.D;
    float2 cs[VEC];
    auto turned = [&](Rows x, const float (&w)[2 * VEC]) {
        float y[2 * VEC], s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * VEC; ++i) {
            y[i] = to_f32<T>(x.x[i / VEC].e[i % VEC]);
            (i < VEC ? s0 : s1) = fmaf(y[i], y[i], i < VEC ? s0 : s1);
        }
        const float ss = (in0 ? s0 : 0.0f) + (in1 ? s1 : 0.0f);
        const float inv = __builtin_amdgcn_rsqf(fmaf(group_sum<L>(ss), inv_d, a.eps));
#pragma unroll
        for (int i = 0; i < 2 * VEC; ++i) y[i] = y[i] * inv * w[i];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int lo = NEIGHBOURS ? 2 * i : i, hi = NEIGHBOURS ? 2 * i + 1 : VEC + i;
            const float u = y[lo], v = y[hi];
            y[lo] = u * cs[i].x - v * cs[i].y;
            y[hi] = u * cs[i].y + v * cs[i].x;
        }
#pragma unroll
        for (int i = 0; i < 2 * VEC; ++i) x.x[i / VEC].e[i % VEC] = from_f32<T>(y[i]);
        return x;
    };
    auto put = [&](TS* dst, const Rows& x) {
        if (in0) *reinterpret_cast<u32x4*>(dst + e0) = x.x[0].v;
        if (in1) *reinterpret_cast<u32x4*>(dst + e1) = x.x[1].v;
    };
    for (; t < t1; t += NT / 64 / wpt) {
        const long long pos = uniform(tok[t - t0].pos), row = uniform(tok[t - t0].row);
#pragma unroll
        for (int i = 0; i < MAX_HALF / 64; ++i)
            if (lane + 64 * i < half) turn[wave][lane + 64 * i] = turn_of(pos, freq[i]);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int i = 0; i < VEC; ++i) cs[i] = turn[wave][pair0 + i];
        __builtin_amdgcn_wave_barrier();
        // the next rows of this token, or the first of the wave's next one
        auto take = [&](int p) {
            const Rows now = next;
            if (p + wpt < passes) next = fetch(t, p + wpt);
            else if (t + NT / 64 / wpt < t1) next = fetch(t + NT / 64 / wpt, share);
            return now;
        };
        int p = share;
        for (; p < pq; p += wpt) {
            const Rows x = turned(take(p), wq);
            const int h = p * R + lane / L;
            if (h < a.H) put(static_cast<TS*>(a.q_out.p) + t * a.q_out.row + h * a.q_out.head, x);
        }
        for (; p < passes; p += wpt) {
            Rows x = take(p);
            const int first = (p - pq) * R, r = first + lane / L;
            const bool is_k = r < a.HK;
            if (first < a.HK) {
                const Rows y = turned(x, wk);
                if (is_k) x = y;
            }
            if (is_k) put(static_cast<TS*>(a.k_out.p) + row * a.k_out.row + r * a.k_out.head, x);
            else if (r < kv) put(static_cast<TS*>(a.v_out.p) + row * a.v_out.row + (r - a.HK) * a.v_out.head, x);
        }
    }
}

// Any rotated width: one piece a lane, the pair's other element read by itself.
template <typename T>
__global__ __launch_bounds__(NT) void rope_kernel(RopeLaunch a, int tpb, int log2_lanes) {
    using TS = typename T::storage;
    constexpr int VEC = 16 / sizeof(TS);
    __shared__ float2 turn[MAX_TPB * MAX_HALF];
    __shared__ Token tok[MAX_TPB];
    const int t0 = blockIdx.x * tpb, nt = min(tpb, a.N - t0), half = a.rot / 2;
    const bool malformed = rope_malformed(a, t0, t0 + nt, tok);
    report_status(a.dev_status, malformed);
    if (malformed || nt <= 0) return;
    for (int i = threadIdx.x; i < nt * half; i += NT) {
        const int tk = i / half;
        turn[i] = turn_of(tok[tk].pos, a.inv_freq[i - tk * half]);
    }
    __syncthreads();

    const int lanes = 1 << log2_lanes, lane = threadIdx.x & (lanes - 1), e0 = lane * VEC;
    const int heads = a.H + a.HK + (a.v.p != nullptr ? a.HK : 0);
    const bool in = e0 < a.D;
    const int rows = nt * heads, step = NT >> log2_lanes;
    // every lane of a group stays in the loop for the group sum
    for (int r = threadIdx.x >> log2_lanes; r < rows; r += step) {
        const int tk = r / heads, h = r - tk * heads, t = t0 + tk;
        const bool is_q = h < a.H, is_v = h >= a.H + a.HK;
        const int hh = is_q ? h : is_v ? h - a.H - a.HK : h - a.H;
        const HeadRows &src = is_q ? a.q : is_v ? a.v : a.k, &dst = is_q ? a.q_out : is_v ? a.v_out : a.k_out;
        const long long row = is_q ? t : tok[tk].row;
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
        }
        // in place: all lanes have read their partners before one writes (a row lies in one wave)
        __builtin_amdgcn_wave_barrier();
        if (in) *reinterpret_cast<u32x4*>(y + e0) = raw.v;
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
        if ((long long)blocks * NT > kMaxThreads) return hipErrorInvalidConfiguration;
        rope_kernel<T><<<blocks, NT, 0, stream>>>(a, tpb, log2_pieces);
        return hipGetLastError();
    }
    // A block's four waves share a token while that leaves CUs idle.  Else a wave takes tokens of its own: as many
    // as let all blocks run at once (10277 tokens, D = 64: 19 us at three, 24 at one), and where there are too
    // many for that, one, which evens out the last round (24748 tokens, D = 128: 131 us at one, 137 at three).
    const bool few = a.N <= 1024;
    const int wpt = few ? 4 : 1, tpb = few ? 1 : a.N <= 12288 ? 4 * ((a.N + 4095) / 4096) : 4;
    const int blocks = a.N > 0 ? (a.N + tpb - 1) / tpb : 1;
    if ((long long)blocks * NT > kMaxThreads) return hipErrorInvalidConfiguration;
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
