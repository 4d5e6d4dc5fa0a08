// gdn_rope.hip -- per-head RMS norm of q and k, rotary positions and the write of the new keys and
// values into the cache, in one pass over the packed tokens (gdn_qk_norm_rope_varlen).
//
// One row is one head of one token.  A group of lanes (16 bytes of the row each, the group a power of
// two inside a wave) loads the row, sums its squares in fp32 over the group, scales, rotates and
// stores it.  The block's tokens share a table of (cos, sin) per rotated pair: the angle is formed and
// reduced to a fraction of a turn in fp64 -- position * frequency passes 2^20 turns on long contexts,
// where an fp32 product has no fraction left -- and only that fraction goes to the fp32 sincos.
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
        const double turns = (double)pos * (double)a.inv_freq[j] * 0.15915494309189535;  // 1 / (2 pi)
        const float f = (float)(turns - rint(turns));                                    // [-1/2, 1/2] turns
        float s, c;
        sincospif(2.0f * f, &s, &c);
        turn[i] = make_float2(c, s);
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
    const int vec = 16 / (int)sizeof(typename T::storage);
    int log2_lanes = 0;
    while ((vec << log2_lanes) < a.D) ++log2_lanes;
    const int tpb = a.N > 1024 ? 4 : 1;
    const int blocks = a.N > 0 ? (a.N + tpb - 1) / tpb : 1;
    rope_kernel<T><<<blocks, NT, 0, stream>>>(a, tpb, log2_lanes);
    return hipGetLastError();
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
