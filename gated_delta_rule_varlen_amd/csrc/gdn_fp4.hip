// gdn_fp4.hip -- new keys and values into the 4-bit cache, and its rows back as values.
//
// A thread takes eight elements of a head: four neighbours hold a block of 32 and find its largest element among
// themselves.  Codes of eight elements are 32 bits, so a wave's loads and stores are whole segments.
//
// e is the least with max|x| <= 6 * 2^e, from the bits of the largest element and without a logarithm; the conversion rounds
// x / 2^e to the nearest code.  Bound by bytes: 24748 tokens of 8 heads of 128 written (101 MB of bf16 to 27 MB) take 21 to 23
// us and come back in 21 to 22, 5.5 to 6 TB/s; 64 tokens 3.3 and 5.2, the check of the call and one chain of loads.
// A wave a row took 63 us there and back; loads and stores past the caches 51 against 47; two or eight tokens on their way
// instead of four, no difference.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>

#include "gdn_device.hpp"
#include "gdn_fp4.hpp"
#include "gdn_launch.hpp"

namespace gdn {
namespace {

constexpr int NT = 256;      // threads a block
constexpr int MAX_TPB = 8;   // tokens a block at most (24748 tokens written and read back from caches: 44 us, with 16 tokens 47)
constexpr int kCUs = 256;

// Whole-call check; the thread that holds a sequence of the block's tokens t0 .. t1 - 1 leaves their rows in `rows`.
// Reached by all threads of the block.
__device__ __forceinline__ bool rows_malformed(const Fp4RowsLaunch& a, int t0, int t1, long long* rows) {
    int bad = 0;
    for (int i = threadIdx.x; i < a.B; i += NT) {
        const int o = a.offsets[i], e = a.offsets[i + 1];
        const long long past = a.past != nullptr ? a.past[i] : 0;
        const long long begin = a.kv_begin != nullptr ? a.kv_begin[i] : 0;
        bad |= (i == 0 && o != 0) | (o > e) | (i == a.B - 1 && e != a.N);
        if (o < e) {
            bad |= (past < 0);
            if (a.kv_begin != nullptr) bad |= (begin < 0) | (begin > a.cache.rows) | (begin + past + ((long long)e - o) > a.cache.rows);
        }
        for (int t = max(o, t0); t < min(e, t1); ++t) rows[t - t0] = a.kv_begin != nullptr ? begin + past + (t - o) : t;
    }
    return any_in_block<NT>(bad != 0);
}

// Eight elements of type T.
template <typename T>
struct Eight {
    static constexpr int NP = sizeof(typename T::storage) / 2;
    union {
        u32x4 v[NP];
        typename T::storage e[8];
    };
    __device__ __forceinline__ void load(const typename T::storage* p) {
#pragma unroll
        for (int i = 0; i < NP; ++i) v[i] = reinterpret_cast<const u32x4*>(p)[i];
    }
    __device__ __forceinline__ void store(typename T::storage* p) const {
#pragma unroll
        for (int i = 0; i < NP; ++i) reinterpret_cast<u32x4*>(p)[i] = v[i];
    }
};

// Eight elements' values from their codes.
template <typename T>
__device__ __forceinline__ void widen(uint32_t codes, uint32_t scale, Eight<T>& y) {
    float f[8];
    fp4::values(codes, scale, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) y.e[e] = from_f32<T>(f[e]);
}

// Codes of eight elements of a block, and the scale byte that the four threads of the block find together.
template <typename T>
__device__ __forceinline__ void narrow(const Eight<T>& y, uint32_t& codes, uint32_t& scale) {
    float f[8];
    uint32_t top = 0;  // bits of the largest element: NaN above infinity above all numbers
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        f[e] = to_f32<T>(y.e[e]);
        top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
    }
    top = max(top, (uint32_t)__float_as_uint(dpp<DPP_QUAD_XOR1>(__uint_as_float(top))));
    top = max(top, (uint32_t)__float_as_uint(dpp<DPP_QUAD_XOR2>(__uint_as_float(top))));
    // top = 1.m * 2^(E - 127) is at most 6 * 2^e = 1.5 * 2^(e + 2)
    const bool finite = top < 0x7f800000u;
    int byte = (int)(top >> 23) - 2 + ((top & 0x7fffffu) > 0x400000u);
    byte = max(byte, T::code == GDN_F16 ? 127 - 23 : 1);
    byte = min(byte, T::code == GDN_F16 ? 127 + 13 : 127 + 125);  // with 4 * 2^126 a value would pass the type
    const float s = fp4::scale_of(finite ? byte : 127);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], s, 3);
    codes = finite ? w : 0u;
    scale = finite ? (uint32_t)byte : fp4::kNotANumber;
}

template <typename T, bool READ>
__global__ __launch_bounds__(NT) void fp4_rows_kernel(Fp4RowsLaunch a, int tpb) {
    using TS = typename T::storage;
    __shared__ long long rows[MAX_TPB];
    const int t0 = blockIdx.x * tpb, t1 = min(t0 + tpb, a.N);
    const bool bad = rows_malformed(a, t0, t1, rows);
    report_status(a.dev_status, bad);
    if (bad) return;
    // A thread keeps its place in the token's row and goes over tokens, UNROLL of them on their way at a time; where a row has
    // fewer places than the block has threads, several tokens at once.
    constexpr int UNROLL = 4;
    const int per_head = a.D / 8, per_half = a.HK * per_head, per_token = 2 * per_half, count = t1 - t0;
    const int groups = max(NT / per_token, 1);
    for (int x = threadIdx.x; x < (per_token < NT ? groups * per_token : per_token); x += NT) {
        const int in_token = per_token < NT ? x % per_token : x, first = per_token < NT ? x / per_token : 0;
        const bool half = in_token >= per_half;
        const int in_half = half ? in_token - per_half : in_token, head = in_half / per_head, piece = in_half - head * per_head;
        const HeadRows& tok = half ? a.v : a.k;
        const Fp4Half& to = half ? a.cache.v : a.cache.k;
        TS* const at = static_cast<TS*>(tok.p) + (long long)t0 * tok.row + head * tok.head + piece * 8;
        char* const codes = static_cast<char*>(to.codes.p) + head * to.codes.head + piece * 4;
        uint8_t* const scales = static_cast<uint8_t*>(to.scales.p) + head * to.scales.head + piece / 4;
        for (int i0 = first; i0 < count; i0 += UNROLL * groups) {
            Eight<T> y[UNROLL];
            uint32_t w[UNROLL], byte[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int i = min(i0 + u * groups, count - 1);  // past the last token that one again
                if constexpr (READ) {
                    w[u] = *reinterpret_cast<const uint32_t*>(codes + rows[i] * to.codes.row);
                    byte[u] = scales[rows[i] * to.scales.row];
                } else {
                    y[u].load(at + i * tok.row);
                }
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int i = i0 + u * groups;
                if (i >= count) break;  // four neighbours go round together
                if constexpr (READ) {
                    widen<T>(w[u], byte[u], y[u]);
                    y[u].store(at + i * tok.row);
                } else {
                    narrow<T>(y[u], w[u], byte[u]);
                    *reinterpret_cast<uint32_t*>(codes + rows[i] * to.codes.row) = w[u];
                    if (piece % 4 == 0) scales[rows[i] * to.scales.row] = (uint8_t)byte[u];
                }
            }
        }
    }
}

template <typename T>
hipError_t launch_rows(const Fp4RowsLaunch& a, hipStream_t stream) {
    // enough blocks to fill the chip, and enough tokens a block that the whole-call check is shared
    const long long per_token = 2ll * a.HK * a.D / 8;
    int tpb = 1;
    while (tpb < MAX_TPB && (tpb * per_token < NT || ((long long)a.N + tpb - 1) / tpb > 4 * kCUs)) tpb *= 2;
    const long long blocks = std::max(1ll, ((long long)a.N + tpb - 1) / tpb);
    if (blocks * NT > kMaxThreads) return hipErrorInvalidConfiguration;
    if (a.read) fp4_rows_kernel<T, true><<<(unsigned)blocks, NT, 0, stream>>>(a, tpb);
    else fp4_rows_kernel<T, false><<<(unsigned)blocks, NT, 0, stream>>>(a, tpb);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp4_rows(const Fp4RowsLaunch& a, hipStream_t stream) {
    switch (a.dtype) {
        case GDN_F32: return launch_rows<F32>(a, stream);
        case GDN_BF16: return launch_rows<BF16>(a, stream);
        default: return launch_rows<F16>(a, stream);
    }
}

}  // namespace gdn
