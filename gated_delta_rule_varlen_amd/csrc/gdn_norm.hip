// gdn_norm.hip -- the norms before and behind a block: residual_norm over whole rows of the residual stream, gated_norm over
// the heads of a mixer's output.  Both read every input once and write every output once, and hold a row in
// registers between its sums and its results; squares, sums and roots are fp32, each output is rounded once.
//
// Both are bound by bytes where there are many rows (a 1 GiB copy reaches 5.2 TB/s): residual_norm of 24748 rows of 4096 (bf16
// beside an fp32 stream, norm of the block's output and channel scales, 1.22 GB) 244 to 248 us, 4.9 TB/s; in fp32 332, 4.9;
// 4096 rows of 32768 in bf16 220, 4.9, but beside an fp32 stream 440, 3.7, and in fp32 1003, 2.1: four and eight pieces of both
// rows, this one and the next, pass the 128 registers that 1024 threads leave (43 and 148 spilled).  gated_norm of
// 9111 x 16 heads of 64 fp16 elements (56 MB) 10.9 us, 5.1 TB/s.  With few rows they are one launch: 256 rows of 4096
// 4.2 us, 256 x 32 heads of 128 4.1 us.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "gdn_device.hpp"
#include "gdn_launch.hpp"

namespace gdn {
namespace {

constexpr int kCUs = 256;

// 16 bytes of a row of type T, as fp32.
template <typename T>
struct Piece {
    using TS = typename T::storage;
    static constexpr int VEC = 16 / sizeof(TS);
    union {
        u32x4 v;
        TS e[VEC];
    };
    __device__ __forceinline__ float get(int i) const { return to_f32<T>(e[i]); }
    __device__ __forceinline__ void set(int i, float x) { e[i] = from_f32<T>(x); }
};

// VEC consecutive elements of type R as whole pieces (VEC elements of fp32 are one or two of them).
template <typename R, int VEC>
struct Span {
    static constexpr int PV = Piece<R>::VEC, NP = VEC / PV;
    Piece<R> p[NP];
    __device__ __forceinline__ void load(const typename R::storage* at) {
#pragma unroll
        for (int i = 0; i < NP; ++i) p[i].v = *reinterpret_cast<const u32x4*>(at + i * PV);
    }
    __device__ __forceinline__ void store(typename R::storage* at) const {
#pragma unroll
        for (int i = 0; i < NP; ++i) *reinterpret_cast<u32x4*>(at + i * PV) = p[i].v;
    }
    __device__ __forceinline__ float get(int i) const { return p[i / PV].get(i % PV); }
    __device__ __forceinline__ void set(int i, float x) { p[i / PV].set(i % PV, x); }
};

// Sum over the RT threads that share a row.  Two sums follow each other in different halves of `lds`, so a wave may write
// the next one's part while another still reads this one's.
template <int RT>
__device__ __forceinline__ float row_sum(float x, float (*lds)[16], int& turn) {
    x = group_sum<64>(x);
    if constexpr (RT > 64) {
        if ((threadIdx.x & 63) == 0) lds[turn][threadIdx.x >> 6] = x;
        __syncthreads();
        x = 0.0f;
#pragma unroll
        for (int w = 0; w < RT / 64; ++w) x += lds[turn][w];
        turn ^= 1;
    }
    return x;
}

// VEC consecutive entries of a vector in fp32.
template <int VEC>
__device__ __forceinline__ void load_vector(const float* p, float* to) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(p + i);
        to[i] = x[0], to[i + 1] = x[1], to[i + 2] = x[2], to[i + 3] = x[3];
    }
}

// RT threads a row, P spans of 16 bytes of x a thread.  A block goes over rows with the next one on its way, and keeps the
// vectors in registers where they are few (P <= 2): read again for every row they are as many bytes from L2 as the row.
// (Both, and even shares of rows, against a wave a row that reads every row twice: 609 us, so 248, on the 24748 rows above.)
template <typename T, typename R, int RT, int P>
__global__ __launch_bounds__(RT < 256 ? 256 : RT) void residual_norm_kernel(ResidualNormLaunch a) {
    using TS = typename T::storage;
    using RS = typename R::storage;
    constexpr int VEC = 16 / sizeof(TS), NT = RT < 256 ? 256 : RT, ROWS = NT / RT;
    constexpr bool KEEP = P <= 2;
    __shared__ float sums[2][16];
    int turn = 0;
    const int j = threadIdx.x % RT;
    const float inv_c = 1.0f / (float)a.C;
    struct Row {
        Span<T, VEC> x[P];
        Span<R, VEC> r[P];
    };
    auto fetch = [&](long long row) {
        Row y;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * RT + j) * VEC, at = e < a.C ? e : 0;
            y.x[p].load(static_cast<const TS*>(a.x) + row * a.x_row + at);
            if (a.residual != nullptr) y.r[p].load(static_cast<const RS*>(a.residual) + row * a.residual_row + at);
        }
        return y;
    };
    float by_kept[KEEP ? P : 1][VEC], w_kept[KEEP ? P : 1][VEC];
    // scale * channel_scale * post_weight, and the weight, of a span
    auto factors = [&](int p, float* by) {
        const int e = (p * RT + j) * VEC, at = e < a.C ? e : 0;
        float x[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) by[i] = a.scale;
        for (const float* v : {a.channel_scale, a.post_weight}) {
            if (v == nullptr) continue;
            load_vector<VEC>(v + at, x);
#pragma unroll
            for (int i = 0; i < VEC; ++i) by[i] *= x[i];
        }
    };
    auto weights = [&](int p, float* w) {
        const int e = (p * RT + j) * VEC;
        if (a.weight != nullptr) {
            load_vector<VEC>(a.weight + (e < a.C ? e : 0), w);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = 1.0f;
        }
    };
    const long long step = (long long)gridDim.x * ROWS;
    long long row = (long long)blockIdx.x * ROWS + threadIdx.x / RT;
    if (row >= a.N) return;
    Row next = fetch(row);
    if constexpr (KEEP) {
#pragma unroll
        for (int p = 0; p < P; ++p) factors(p, by_kept[p]), weights(p, w_kept[p]);
    }
    for (; row < a.N; row += step) {
        Row cur = next;
        if (row + step < a.N) next = fetch(row + step);
        float inv_x = 1.0f;
        if (a.post_weight != nullptr) {
            float sum = 0.0f;
#pragma unroll
            for (int p = 0; p < P; ++p)
                if ((p * RT + j) * VEC < a.C)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) sum = fmaf(cur.x[p].get(i), cur.x[p].get(i), sum);
            inv_x = 1.0f / sqrtf(row_sum<RT>(sum, sums, turn) * inv_c + a.eps);
        }
        float h[P][VEC], sum = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float now[VEC];
            if constexpr (!KEEP) factors(p, now);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float t = cur.x[p].get(i) * inv_x, by = KEEP ? by_kept[KEEP ? p : 0][i] : now[i];
                h[p][i] = fmaf(t, by, a.residual != nullptr ? cur.r[p].get(i) : 0.0f);
            }
            if ((p * RT + j) * VEC < a.C)
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum = fmaf(h[p][i], h[p][i], sum);
        }
        const float inv = 1.0f / sqrtf(row_sum<RT>(sum, sums, turn) * inv_c + a.eps);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * RT + j) * VEC;
            if (e >= a.C) continue;
            if (a.residual_out != nullptr) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) cur.r[p].set(i, h[p][i]);
                cur.r[p].store(static_cast<RS*>(a.residual_out) + row * a.residual_out_row + e);
            }
            float now[VEC];
            if constexpr (!KEEP) weights(p, now);
#pragma unroll
            for (int i = 0; i < VEC; ++i) cur.x[p].set(i, h[p][i] * inv * (KEEP ? w_kept[KEEP ? p : 0][i] : now[i]));
            cur.x[p].store(static_cast<TS*>(a.out) + row * a.out_row + e);
        }
    }
}

// Blocks for `groups` of rows, each as many of them as any other or one less, `most` at most.
unsigned even_blocks(long long groups, long long most) {
    const long long rounds = (groups + most - 1) / most;
    return (unsigned)((groups + rounds - 1) / rounds);
}

template <typename T, typename R, int RT, int P>
hipError_t start_residual(const ResidualNormLaunch& a, hipStream_t stream) {
    constexpr int NT = RT < 256 ? 256 : RT, ROWS = NT / RT;
    residual_norm_kernel<T, R, RT, P><<<even_blocks(((long long)a.N + ROWS - 1) / ROWS, kCUs * 1024 / NT), NT, 0, stream>>>(a);
    return hipGetLastError();
}
template <typename T, typename R>
hipError_t residual_for(const ResidualNormLaunch& a, hipStream_t stream) {
    const int pieces = a.C / (16 / (int)sizeof(typename T::storage));
    if (pieces <= 64) return start_residual<T, R, 64, 1>(a, stream);
    if (pieces <= 256) return start_residual<T, R, 256, 1>(a, stream);
    if (pieces <= 512) return start_residual<T, R, 256, 2>(a, stream);
    if (pieces <= 1024) return start_residual<T, R, 512, 2>(a, stream);
    if (pieces <= 2048) return start_residual<T, R, 1024, 2>(a, stream);
    if (pieces <= 4096) return start_residual<T, R, 1024, 4>(a, stream);
    if constexpr (sizeof(typename T::storage) == 4) return start_residual<T, R, 1024, 8>(a, stream);
    return hipErrorInvalidValue;  // 32768 elements are 4096 pieces
}

// 1 / (1 + exp(-g)).  In fp32 to a few roundings for every g: the exponential's argument is exact and never positive, so it
// does not overflow, and the quotient is rounded once (9111 x 32 heads of 128, 448 MB, 88 us as before; 9111 x 16 of 64 from
// caches 19.5 instead of 17.9).  The half types take the chip's exponential and reciprocal: the
// rounded argument is off by |g| 2^-24, which for gates that do not vanish (|g| < 88) is 2^-17 relative, a sixtieth of
// fp16's own rounding; below -87 the gate is zero.
template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
    if constexpr (T::code == GDN_F32) {
        const float e = expf(-fabsf(g));
        return (g < 0.0f ? e : 1.0f) / (1.0f + e);
    } else {
        return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g));
    }
}

// A head's row: L lanes of a wave, P pieces of 16 bytes each.  A block goes over rows with the next ones on their way.
template <typename T, int L, int P>
__global__ __launch_bounds__(256) void gated_norm_kernel(GatedNormLaunch a, uint32_t h_inverse) {
    using TS = typename T::storage;
    constexpr int VEC = 16 / sizeof(TS), ROWS = 256 / L;
    const int j = threadIdx.x % L;
    const float inv_v = 1.0f / (float)a.V;
    const unsigned rows = (unsigned)a.N * a.H, step = gridDim.x * ROWS;
    struct Row {
        Piece<T> x[P], z[P];
        TS* out;
    };
    // lanes past the last row read that one, so that no load stands in a branch
    auto fetch = [&](unsigned first) {
        const unsigned row = min(first + threadIdx.x / L, rows - 1);
        unsigned t = a.H == 1 ? row : __umulhi(row, h_inverse);  // one too many at most, as h_inverse is 2^32 / H rounded up
        t -= t * a.H > row;
        const unsigned head = row - t * a.H;
        const TS* x = static_cast<const TS*>(a.x.p) + t * a.x.row + head * a.x.head;
        const TS* z = static_cast<const TS*>(a.gate.p) + t * a.gate.row + head * a.gate.head;
        Row y;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * L + j) * VEC, at = e < a.V ? e : 0;
            y.x[p].v = *reinterpret_cast<const u32x4*>(x + at);
            y.z[p].v = *reinterpret_cast<const u32x4*>(z + at);
        }
        y.out = static_cast<TS*>(a.out.p) + t * a.out.row + head * a.out.head;
        return y;
    };
    unsigned first = blockIdx.x * ROWS;
    Row next = fetch(first);
    float w[P][VEC];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int e = (p * L + j) * VEC;
        if (a.weight != nullptr) {
            load_vector<VEC>(a.weight + (e < a.V ? e : 0), w[p]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[p][i] = 1.0f;
        }
    }
    // every lane goes round as often as its wave's first, so that all take part in the sums
    for (; first < rows; first += step) {
        Row cur = next;
        const bool in = first + threadIdx.x / L < rows;
        if (first + step < rows) next = fetch(first + step);
        float y[P][VEC], act[P][VEC], sum = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const bool real = (p * L + j) * VEC < a.V;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float g = cur.z[p].get(i), s = sigmoid<T>(g);
                act[p][i] = a.sigmoid ? s : g * s;
                y[p][i] = cur.x[p].get(i);
                if (a.gate_first) y[p][i] *= act[p][i];
                sum = real ? fmaf(y[p][i], y[p][i], sum) : sum;
            }
        }
        const float inv = a.no_norm ? 1.0f : 1.0f / sqrtf(group_sum<L>(sum) * inv_v + a.eps);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * L + j) * VEC;
            if (e >= a.V || !in) continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float v = y[p][i] * inv * w[p][i];
                cur.x[p].set(i, a.gate_first ? v : v * act[p][i]);
            }
            *reinterpret_cast<u32x4*>(cur.out + e) = cur.x[p].v;
        }
    }
}

template <typename T, int L, int P>
hipError_t start_gated(const GatedNormLaunch& a, hipStream_t stream) {
    constexpr int ROWS = 256 / L;
    const uint32_t h_inverse = (uint32_t)(((1ull << 32) + a.H - 1) / a.H);
    gated_norm_kernel<T, L, P><<<even_blocks(((long long)a.N * a.H + ROWS - 1) / ROWS, kCUs * 8), 256, 0, stream>>>(a, h_inverse);
    return hipGetLastError();
}
template <typename T>
hipError_t gated_for(const GatedNormLaunch& a, hipStream_t stream) {
    const int pieces = a.V / (16 / (int)sizeof(typename T::storage));
    if (pieces <= 4) return start_gated<T, 4, 1>(a, stream);
    if (pieces <= 8) return start_gated<T, 8, 1>(a, stream);
    if (pieces <= 16) return start_gated<T, 16, 1>(a, stream);
    if (pieces <= 32) return start_gated<T, 32, 1>(a, stream);
    if (pieces <= 64) return start_gated<T, 64, 1>(a, stream);
    if (pieces <= 128) return start_gated<T, 64, 2>(a, stream);
    if (pieces <= 256) return start_gated<T, 64, 4>(a, stream);
    if constexpr (sizeof(typename T::storage) == 4) return start_gated<T, 64, 8>(a, stream);
    return hipErrorInvalidValue;  // 2048 elements are 256 pieces
}

}  // namespace

hipError_t launch_residual_norm(const ResidualNormLaunch& a, hipStream_t stream) {
    const bool wide = a.residual_dtype != a.dtype;
    switch (a.dtype) {
        case GDN_F32: return residual_for<F32, F32>(a, stream);
        case GDN_BF16: return wide ? residual_for<BF16, F32>(a, stream) : residual_for<BF16, BF16>(a, stream);
        default: return wide ? residual_for<F16, F32>(a, stream) : residual_for<F16, F16>(a, stream);
    }
}

hipError_t launch_gated_norm(const GatedNormLaunch& a, hipStream_t stream) {
    switch (a.dtype) {
        case GDN_F32: return gated_for<F32>(a, stream);
        case GDN_BF16: return gated_for<BF16>(a, stream);
        default: return gated_for<F16>(a, stream);
    }
}

}  // namespace gdn
