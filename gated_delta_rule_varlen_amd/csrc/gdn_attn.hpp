// gdn_attn.hpp -- the tile kernels of the softmax attention (instances per type in gdn_attn_<type>.hip,
// host side and the joining kernel in gdn_attn.hip).
//
// Rows.  The G = H/HK query heads of a key head and the tokens of a sequence form one list of query rows,
// row r = (token r / G, head r % G): a block's rows all read the same keys, so K and V are loaded once
// for the whole group.  A wave owns 32 rows (QT times), a block WR waves of them and WK waves along
// the keys.
//
// Products.  S^T = K Q^T and O^T = V^T P^T on 32x32 MFMA tiles: a lane's accumulators all belong to one
// query row (column lane%32), so the softmax statistics are one number a lane and rescaling O
// needs no exchange; the exponentials of S^T, rounded, are the second product's operand where they lie:
// the 16 scores of a lane are keys 8(i/4) + 4(lane/32) + i%4, and V^T is read with its keys in that
// order (a contraction may run in any order).
//
// Keys and values reach LDS by 16-byte asynchronous loads that write it directly, NS stages deep, with
// the 16-byte pieces of row r stored at place piece ^ (r % 8), which spreads a column read (K) and a
// transposing read (V) over the banks.  The buffer's range check returns zeros for rows past the
// sequence's keys and pieces past D, so nothing outside a run is read, and nothing unwritten is used.
//
// Softmax in base 2: p = 2^(s*c - ref), c = scale*log2(e).  ref follows the running maximum only when
// that has grown by more than 2^8 (P stays in range, the quotient O / l is the same), so O, which lives
// in accumulation registers, is hardly ever rescaled.
#pragma once

#include <hip/hip_runtime.h>

#include <climits>

#include "gdn_device.hpp"
#include "gdn_launch.hpp"

namespace gdn {
namespace attn {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short v4i16 __attribute__((ext_vector_type(4)));

constexpr int kRsrc = 0x00020000;     // raw buffer, range checked
constexpr int kOutside = 0x40000000;  // a byte offset past every tile's range
constexpr float kNoMax = -3.0e38f;    // running maximum before the first key: below every score
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What a launch needs beside the call's own arguments.
struct Args {
    AttnLaunch c;
    int G;          // heads per key head
    float s2;       // |scale| * log2(e); the sign goes to the queries
    bool negate;
    int splits;     // key parts of the long form
    int workers;    // blocks of the short form
    bool prefix_rows;  // the long form runs all tokens' rows over the prefix alone
    bool to_sets;   // results go to the workspace, for the joining kernel
    int set0;       // first set this launch writes
    // workspace
    int* status;
    int2* row_info;    // [N][HK]: x = worker a cut run starts in (-1: not cut), y = pieces * 128 + token in sequence
    float* slot_o;     // [workers][2][BM][D]
    float2* slot_ml;   // [workers][2][BM]
    float* set_o;      // [sets][N*H][D]
    float2* set_ml;    // [sets][N*H]
    int sets;
    long long set_rows;  // N*H
};

template <typename T>
struct Mma;
template <>
struct Mma<BF16> {
    static __device__ __forceinline__ void mul(u32x4 a, u32x4 b, f32x16& c) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y) {
        typedef __bf16 v2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, v2{(__bf16)x, (__bf16)y});
    }
};
template <>
struct Mma<F16> {
    static __device__ __forceinline__ void mul(u32x4 a, u32x4 b, f32x16& c) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y) {
        typedef _Float16 v2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, v2{(_Float16)x, (_Float16)y});
    }
};
template <>
struct Mma<F32> {
    static __device__ __forceinline__ void mul(u32x4 a, u32x4 b, f32x16& c) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[j]), __uint_as_float(b[j]), c, 0, 0, 0);
    }
};

// The sign bits of the elements (one or two in 32 bits) whose exponent is all ones.
template <typename T>
__device__ __forceinline__ uint32_t not_finite_sign(uint32_t x) {
    constexpr uint32_t E = T::code == GDN_BF16 ? 0x7f807f80u : T::code == GDN_F16 ? 0x7c007c00u : 0x7f800000u;
    constexpr uint32_t ONE = T::code == GDN_BF16 ? 0x00800080u : T::code == GDN_F16 ? 0x04000400u : 0x00800000u;
    return (x & E) + ONE;  // carries into an element's sign bit from an exponent of all ones only
}
// Waits until at most N of this wave's loads are on their way and its LDS reads have returned, then for the
// whole block.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The maximum and the sum of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float max_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A value every lane holds, as a scalar.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ long long uniform(long long x) {
    return ((long long)uniform((int)(x >> 32)) << 32) | (uint32_t)uniform((int)x);
}

// Whole-call check (offsets, lengths, key runs) with a per-sequence sum: `units(T, n)` of every sequence.
// Returns whether the call is malformed; total = the sum over all sequences, and for the sequence that
// holds unit `want` (want < total) seq = its index and base = the sum before it.  Reached by all threads.
template <int NT, typename F>
__device__ __forceinline__ bool check_and_find(const AttnLaunch& c, F units, long long* total_out) {
    __shared__ long long wave_sum[NT / 64];
    int bad = 0;
    long long sum = 0;
    for (int i = threadIdx.x; i < c.B; i += NT) {
        const int o = c.offsets[i], e = c.offsets[i + 1], t = e - o;
        bad |= (t < 0) | (t > c.max_q) | (i == 0 && o != 0) | (i == c.B - 1 && e != c.N);
        long long n;
        if (c.kv_len != nullptr) {
            n = c.kv_len[i];
            const long long begin = c.kv_begin[i];
            bad |= (n < 0) | (begin < 0) | (begin > c.kv_rows) | (begin + n > c.kv_rows);
        } else {
            n = t;
            bad |= (e > c.kv_rows);
        }
        sum += units(t, (int)n);
    }
    const bool malformed = __syncthreads_or(bad) != 0;
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    if ((threadIdx.x & 63) == 0) wave_sum[threadIdx.x >> 6] = sum;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < NT / 64; ++w) total += wave_sum[w];
    *total_out = uniform(total);
    return malformed;
}

// The sequence that holds unit `want` (in sequence order) and the units before it; all threads.
template <int NT, typename F>
__device__ __forceinline__ void find_unit(const AttnLaunch& c, F units, long long want, int* seq, long long* base) {
    __shared__ long long wave_sum[NT / 64], found_base;
    __shared__ int found;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    long long before = 0;
    for (int i0 = 0;; i0 += NT) {
        const int i = i0 + threadIdx.x;
        long long mine = 0;
        if (i < c.B) {
            const int t = c.offsets[i + 1] - c.offsets[i];
            mine = units(t, c.kv_len != nullptr ? c.kv_len[i] : t);
        }
        long long inc = mine;
        for (int m = 1; m < 64; m <<= 1) {
            const long long y = __shfl_up(inc, m);
            if (lane >= m) inc += y;
        }
        if (lane == 63) wave_sum[wave] = inc;
        if (threadIdx.x == 0) found = -1;
        __syncthreads();
        long long at = before + inc - mine, all = before;
        for (int w = 0; w < NT / 64; ++w) {
            if (w < wave) at += wave_sum[w];
            all += wave_sum[w];
        }
        if (want >= at && want < at + mine) {
            found = i;
            found_base = at;
        }
        __syncthreads();
        const int f = found;
        const long long fb = found_base;
        __syncthreads();
        if (f >= 0 || i0 + NT >= c.B) {
            *seq = uniform(f < 0 ? 0 : f);
            *base = uniform(fb);
            return;
        }
        before = all;
    }
}

template <typename T_, int DP_, int WR_, int WK_, int QT_, int KT_, int NS_, int WAVES_>
struct Cfg {
    using T = T_;
    using TS = typename T::storage;
    static constexpr int DP = DP_, WR = WR_, WK = WK_, QT = QT_, KT = KT_, NS = NS_, WAVES = WAVES_;
    static constexpr bool HALF = sizeof(TS) == 2;
    static constexpr int ES = sizeof(TS), NW = WR * WK, NT = 64 * NW, BM = 32 * QT * WR, KW = 32 * KT, BN = KW * WK;
    static constexpr int RB = DP * ES;            // bytes of a row in LDS
    static constexpr int CPR = RB / 16;           // 16-byte pieces of a row
    static constexpr int CS = RB / 32;            // operand steps of a score tile
    static constexpr int DT = DP / 32;            // 32-wide parts of the head
    static constexpr int TILE = BN * RB, STAGE = 2 * TILE;
    static constexpr int JN = TILE / (NT * 16);   // loads a wave issues for one of K, V
    static constexpr int RPI = NT / CPR;          // rows one load of the whole block covers
    static constexpr int PRE = RPI >= 8 ? 1 : 8 / RPI;
    static constexpr int XCH = (WK / 2) * WR * QT * DT * 16 * 64 * 4 + WK * WR * QT * 64 * 8;  // joining the key waves
    static constexpr int LDS = NS * STAGE > XCH ? NS * STAGE : XCH;
    static_assert(CPR >= 8 && TILE % (NT * 16) == 0 && RPI >= 1 && LDS <= 160 * 1024, "tile");
    // P of fp16 is kept 2^4 larger, away from the subnormals; with the 2^8 of lag it stays below 2^13
    static constexpr float BIAS = T::code == GDN_F16 ? 4.0f : 0.0f, LAG = 8.0f;
};

// One run of key tiles: n rows of keys at k, v (row 0 of the run, this key head).
struct Keys {
    const char* k;
    const char* v;
    int n;
};

template <typename C>
struct Block {
    using T = typename C::T;
    using TS = typename C::TS;
    static constexpr int QT = C::QT, KT = C::KT, DT = C::DT;

    const Args& a;
    char* lds;
    int lane, wave, wr, wk, col, half;
    int kstride, vstride;                   // bytes between rows of this source
    int koff[C::PRE], voff[C::PRE];
    u32x4 q[QT][C::CS];
    int vis[QT];                            // keys the lane's row sees
    int vis_lo, vis_hi;                     // over the wave's rows
    int run_n;                              // keys of the run
    bool spoiled = false;                   // the wave met values only redo() can deal with
    f32x16 o[QT][DT];
    float ref[QT], l[QT];

    __device__ __forceinline__ Block(const Args& a_, char* lds_) : a(a_), lds(lds_) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wr = wave / C::WK;
        wk = wave % C::WK;
        col = lane & 31;
        half = lane >> 5;
    }

    // byte offsets of the 16-byte pieces this lane loads, for rows `ks` and `vs` bytes apart
    __device__ __forceinline__ void set_source(long long krow, long long vrow) {
        kstride = (int)(krow * C::ES);
        vstride = (int)(vrow * C::ES);
#pragma unroll
        for (int j = 0; j < C::PRE; ++j) {
            const int p = (j * C::NW + wave) * 64 + lane, row = p / C::CPR, piece = (p % C::CPR) ^ (row & 7);
            const bool in = piece * 16 < a.c.D * C::ES;
            koff[j] = in ? row * kstride + piece * 16 : kOutside;
            voff[j] = in ? row * vstride + piece * 16 : kOutside;
        }
    }

    __device__ __forceinline__ void load_tile(const Keys& s, int tile, bool real, int stage) {
        const int k0 = tile * C::BN, left = s.n - k0, rows = left < C::BN ? left : C::BN, last = rows - 1;
        const bool any = real && rows > 0;
        const __amdgpu_buffer_rsrc_t rk = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(s.k + (long long)k0 * kstride), 0, any ? last * kstride + a.c.D * C::ES : 0, kRsrc);
        const __amdgpu_buffer_rsrc_t rv = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(s.v + (long long)k0 * vstride), 0, any ? last * vstride + a.c.D * C::ES : 0, kRsrc);
        char* to = lds + stage * C::STAGE + wave * 1024;
#pragma unroll
        for (int j = 0; j < C::JN; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rk, (__attribute__((address_space(3))) void*)(to + j * C::NW * 1024), 16,
                                                     koff[j % C::PRE], (j / C::PRE) * C::PRE * C::RPI * kstride, 0, 0);
#pragma unroll
        for (int j = 0; j < C::JN; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rv, (__attribute__((address_space(3))) void*)(to + C::TILE + j * C::NW * 1024), 16,
                voff[j % C::PRE], (j / C::PRE) * C::PRE * C::RPI * vstride, 0, 0);
    }

    // Queries of the block's rows row0 .. (of `rows` in the list); rows past the list are zeros.
    __device__ __forceinline__ void load_rows(int row0, int rows, long long first, int hk) {
        const int G = a.G;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int r = row0 + (wr * QT + t) * 32 + col, i = r / G, g = r - i * G;
            const bool in = r < rows;
            // lanes without an element read the row's first instead, so no load stands in a branch
            const TS* p = static_cast<const TS*>(a.c.q.p) + (first + (in ? i : 0)) * a.c.q.row +
                          (long long)(hk * G + (in ? g : 0)) * a.c.q.head;
            const uint32_t flip = !a.negate ? 0u : C::HALF ? 0x80008000u : 0x80000000u;
#pragma unroll
            for (int s = 0; s < C::CS; ++s) {
                const int e = (2 * s + half) * (16 / C::ES);
                q[t][s] = *reinterpret_cast<const u32x4*>(p + (e < a.c.D ? e : 0));
            }
#pragma unroll
            for (int s = 0; s < C::CS; ++s) {
                const uint32_t keep = in && (2 * s + half) * (16 / C::ES) < a.c.D ? ~0u : 0u;
                q[t][s] = (q[t][s] ^ flip) & keep;
            }
            ref[t] = kNoMax;
            l[t] = 0.0f;
            spoiled = false;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[t][d] = f32x16{};
        }
    }

    // The keys each row sees of a run of n: all, or (causal) seen0 + its token, at least 0 and at most n.
    __device__ __forceinline__ void see(int row0, int rows, bool causal, int seen0, int n) {
        run_n = n;
        const int G = a.G, lo = row0 + wr * QT * 32, hi = min(lo + QT * 32, rows) - 1;
        auto keys = [&](int r) { return causal ? min(max(seen0 + r / G, 0), n) : n; };
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int r = lo + t * 32 + col;
            vis[t] = r < rows ? keys(r) : n;
        }
        vis_lo = __builtin_amdgcn_readfirstlane(keys(lo));
        vis_hi = __builtin_amdgcn_readfirstlane(lo < rows ? keys(hi) : 0);
    }

    // A stage's keys and values against the wave's rows; key0 = index of its first key in the run.
    __device__ __forceinline__ void use_tile(int stage, int key0) {
        const int base = key0 + wk * C::KW;
        if (base >= vis_hi) return;
        const char* kt_ = lds + stage * C::STAGE + (wk * C::KW + col) * C::RB;
        f32x16 s[QT][KT];
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int t = 0; t < QT; ++t) s[t][k] = f32x16{};
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int x = 0; x < C::CS; ++x) {
                const u32x4 f = *reinterpret_cast<const u32x4*>(kt_ + k * 32 * C::RB + (((2 * x + half) ^ (lane & 7)) * 16));
#pragma unroll
                for (int t = 0; t < QT; ++t) Mma<T>::mul(f, q[t][x], s[t][k]);
            }
        if (base + C::KW > vis_lo) {
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                const int room = vis[t] - base - 4 * half;
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (32 * k + 8 * (i / 4) + i % 4 >= room) s[t][k][i] = -INFINITY;
            }
        }
        float c = a.s2;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            float top = s[t][0][0];
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][k][i]);
            top = max_halves(top) * c;
            if (__builtin_amdgcn_ballot_w64(top > ref[t] + (C::BIAS + C::LAG)) != 0) {
                const float to = fmaxf(ref[t], top - C::BIAS), w = __builtin_amdgcn_exp2f(ref[t] - to);
                ref[t] = to;
                l[t] *= w;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[t][d] *= w;
            }
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float p = __builtin_amdgcn_exp2f(fmaf(s[t][k][i], c, -ref[t]));
                    s[t][k][i] = p;
                    sum += p;
                }
            l[t] += sum;
        }
        const char* vt = lds + stage * C::STAGE + C::TILE + wk * C::KW * C::RB;
        // 0 * infinity is NaN: where rows differ in what they see, a value that is not finite would reach the
        // rows that must not see it.  Such a tile is found here and its block done again by redo().
        if (vis_lo < min(base + C::KW, run_n)) spoiled |= any_not_finite(vt);
        product(vt, s);
    }

    __device__ __forceinline__ bool any_not_finite(const char* vt) {
        uint32_t acc = 0;
#pragma unroll 1
        for (int at = lane * 16; at < C::KW * C::RB; at += 1024) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(vt + at);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc |= not_finite_sign<T>(x[j]);
        }
        return __builtin_amdgcn_ballot_w64((acc & (C::HALF ? 0x80008000u : 0x80000000u)) != 0) != 0;
    }

    // O^T += V^T P^T for the tile at vt.
    __device__ __forceinline__ void product(const char* vt, const f32x16 (&s)[QT][KT]) {
        if constexpr (C::HALF) {
            // lane x of 16 names key x/4 and elements 4(x%4) .. of the 16-wide part (lane/16)%2
            const int x = lane & 15, part = (lane >> 4) & 1, sw = 4 * half + (x >> 2);
            const char* vp = vt + sw * C::RB + (x & 1) * 8;
#pragma unroll
            for (int k = 0; k < 2 * KT; ++k) {
                u32x4 p[QT];
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[t][e] = Mma<T>::pack(s[t][k / 2][8 * (k % 2) + 2 * e], s[t][k / 2][8 * (k % 2) + 2 * e + 1]);
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const int piece = 4 * d + 2 * part + ((x >> 1) & 1);
                    const char* at = vp + 16 * k * C::RB + ((piece ^ sw) * 16);
                    union {
                        v4i16 h[2];
                        u32x4 v;
                    } f;
                    f.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16*)(at));
                    f.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16*)(at + 8 * C::RB));
#pragma unroll
                    for (int t = 0; t < QT; ++t) Mma<T>::mul(f.v, p[t], o[t][d]);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int sw = 4 * half + i % 4;
                    const char* row = vt + (32 * k + 8 * (i / 4) + sw) * C::RB + (col & 3) * 4;
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        const float v = *reinterpret_cast<const float*>(row + (((8 * d + (col >> 2)) ^ sw) * 16));
#pragma unroll
                        for (int t = 0; t < QT; ++t)
                            o[t][d] = __builtin_amdgcn_mfma_f32_32x32x2f32(v, s[t][k][i], o[t][d], 0, 0, 0);
                    }
                }
        }
    }

    // Tiles [t0, t1) of the run.  Loads run NS - 1 tiles ahead; the ones past the end are asked for with an
    // empty range, so the count of loads on their way is the same at every wait.
    __device__ __forceinline__ void run(const Keys& s, int t0, int t1) {
        // LDS addresses are worth registers inside this loop, not across a block's runs
        asm volatile("" : "+v"(lane), "+v"(col), "+v"(half));
#pragma unroll
        for (int i = 0; i < C::NS - 1; ++i) load_tile(s, t0 + i, t0 + i < t1, i);
        int stage = 0;
        for (int t = t0; t < t1; ++t) {
            wait_and_meet<(C::NS - 2) * 2 * C::JN>();
            const int next = stage == 0 ? C::NS - 1 : stage - 1;
            load_tile(s, t + C::NS - 1, t + C::NS - 1 < t1, next);
            use_tile(stage, t * C::BN);
            stage = stage == C::NS - 1 ? 0 : stage + 1;
        }
        wait_and_meet<0>();
    }

    // Joins the key waves' parts into wave wk = 0 of each row group, and the two halves' sums.
    __device__ __forceinline__ void join() {
#pragma unroll
        for (int t = 0; t < QT; ++t) l[t] = sum_halves(l[t]);
        if constexpr (C::WK > 1) {
            constexpr int OB = QT * DT * 16 * 64;  // floats of one wave's O
            float* xo = reinterpret_cast<float*>(lds);
            float2* xm = reinterpret_cast<float2*>(lds + (C::WK / 2) * C::WR * OB * 4);
#pragma unroll
            for (int step = C::WK / 2; step >= 1; step /= 2) {
                if (wk >= step && wk < 2 * step) {
                    float* to = xo + (wr * step + wk - step) * OB + lane;
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                        xm[((wr * step + wk - step) * QT + t) * 64 + lane] = make_float2(ref[t], l[t]);
#pragma unroll
                        for (int d = 0; d < DT; ++d)
#pragma unroll
                            for (int i = 0; i < 16; ++i) to[((t * DT + d) * 16 + i) * 64] = o[t][d][i];
                    }
                }
                __syncthreads();
                if (wk < step) {
                    const float* from = xo + (wr * step + wk) * OB + lane;
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                        const float2 ml = xm[((wr * step + wk) * QT + t) * 64 + lane];
                        const float top = fmaxf(ref[t], ml.x), w = __builtin_amdgcn_exp2f(ref[t] - top),
                                    wo = __builtin_amdgcn_exp2f(ml.x - top);
                        ref[t] = top;
                        l[t] = l[t] * w + ml.y * wo;
#pragma unroll
                        for (int d = 0; d < DT; ++d)
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[t][d][i] = o[t][d][i] * w + from[((t * DT + d) * 16 + i) * 64] * wo;
                    }
                }
                __syncthreads();
            }
        }
    }

    // O of the lane's row, four elements at a time.
    template <typename F>
    __device__ __forceinline__ void each4(int t, F put) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = 32 * d + 8 * i + 4 * half;
                if (e < a.c.D) put(e, f32x4{o[t][d][4 * i], o[t][d][4 * i + 1], o[t][d][4 * i + 2], o[t][d][4 * i + 3]});
            }
    }

    // Where a row's result goes: its place in the list, and out or the workspace.
    struct To {
        int row0, rows;
        long long first;
        int hk;
        int set;          // >= 0: this set of the workspace
        long long slot;   // >= 0: this slot of the workspace
    };
    // Unscaled elements e .. e+3 of row r (or, N = 1, one element), and once a row its ref and l.
    template <int N>
    __device__ __forceinline__ void put(const To& to, int r, int e, const float (&x)[N], float m, float sum, bool stats) {
        const int i = r / a.G, h = to.hk * a.G + r - i * a.G;
        const long long at = to.slot >= 0 ? to.slot * C::BM + r : (to.set >= 0 ? to.set * a.set_rows : 0) + (to.first + i) * a.c.H + h;
        if (to.slot >= 0 || to.set >= 0) {
            float* p = (to.slot >= 0 ? a.slot_o : a.set_o) + at * a.c.D + e;
            if (stats) (to.slot >= 0 ? a.slot_ml : a.set_ml)[at] = make_float2(m, sum);
            if constexpr (N == 4) *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
            else *p = x[0];
        } else {
            TS* out = static_cast<TS*>(a.c.out.p) + (to.first + i) * a.c.out.row + h * a.c.out.head + e;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            union {
                TS s[4];
                f32x4 f;
                u32x2 u;
            } y;
#pragma unroll
            for (int j = 0; j < N; ++j) y.s[j] = from_f32<T>(x[j] * inv);
            if constexpr (N == 1) *out = y.s[0];
            else if constexpr (C::HALF) *reinterpret_cast<u32x2*>(out) = y.u;
            else *reinterpret_cast<f32x4*>(out) = y.f;
            if (stats && a.c.lse != nullptr)
                a.c.lse[at] = sum == 0.0f ? -INFINITY : kLn2 * (m + __builtin_amdgcn_logf(sum));
        }
    }

    // The accumulators of the block's rows.
    __device__ __forceinline__ void store(const To& to) {
        if (wk != 0) return;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int r = to.row0 + (wr * QT + t) * 32 + col;
            if (r >= to.rows) continue;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = 32 * d + 8 * i + 4 * half;
                    const float x[4] = {o[t][d][4 * i], o[t][d][4 * i + 1], o[t][d][4 * i + 2], o[t][d][4 * i + 3]};
                    if (e < a.c.D) put(to, r, e, x, ref[t], l[t], d == 0 && i == 0 && half == 0);
                }
        }
    }

    // The block's rows again, plainly: a wave a row, 64 keys at a time, over the keys p0 .. p1 - 1 of the prefix
    // and k0 .. k1 - 1 of the run (seen0 + token of them seen).
    __device__ __forceinline__ void redo(const To& to, const Keys& prefix, int p0, int p1, const Keys& own, int k0, int k1,
                                         int seen0) {
#pragma unroll 1
        for (int r = to.row0 + wave; r < min(to.row0 + C::BM, to.rows); r += C::NW) {
            const int i = r / a.G, g = r - i * a.G;
            const TS* qp = static_cast<const TS*>(a.c.q.p) + (to.first + i) * a.c.q.row + (long long)(to.hk * a.G + g) * a.c.q.head;
            float m = kNoMax, sum = 0.0f, x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
                const Keys& s = part == 0 ? prefix : own;
                const long long ks = (part == 0 ? a.c.pk : a.c.k).row, vs = (part == 0 ? a.c.pv : a.c.v).row;
                const int j1 = part == 0 ? p1 : min(k1, seen0 + i);
#pragma unroll 1
                for (int j0 = part == 0 ? p0 : k0; j0 < j1; j0 += 64) {
                    float y = -INFINITY;
                    if (j0 + lane < j1) {
                        const TS* kp = reinterpret_cast<const TS*>(s.k) + (j0 + lane) * ks;
                        y = 0.0f;
#pragma unroll 1
                        for (int e = 0; e < a.c.D; e += 4) {
                            const f32x4 qv = load4<T>(qp + e), kv = load4<T>(kp + e);
                            for (int z = 0; z < 4; ++z) y = fmaf(qv[z], kv[z], y);
                        }
                        y *= a.negate ? -a.s2 : a.s2;
                    }
                    float top = y;
                    for (int z = 1; z < 64; z <<= 1) top = fmaxf(top, __shfl_xor(top, z));
                    const float to_m = fmaxf(m, top), w = __builtin_amdgcn_exp2f(m - to_m), p = __builtin_amdgcn_exp2f(y - to_m);
                    sum = sum * w + group_sum<64>(p);
                    m = to_m;
                    for (int z = 0; z < 4; ++z) x[z] *= w;
#pragma unroll 1
                    for (int j = 0; j < min(64, j1 - j0); ++j) {
                        const float pj = __shfl(p, j);
                        const TS* vp = reinterpret_cast<const TS*>(s.v) + (j0 + j) * vs;
                        for (int z = 0; z < 4; ++z)
                            if (lane + 64 * z < a.c.D) x[z] = fmaf(pj, to_f32<T>(vp[lane + 64 * z]), x[z]);
                    }
                }
            }
            for (int z = 0; z < 4; ++z) {
                const float one[1] = {x[z]};
                if (lane + 64 * z < a.c.D) put(to, r, lane + 64 * z, one, m, sum, z == 0 && lane == 0);
            }
        }
    }
};

__device__ __forceinline__ void report(const Args& a, bool malformed) {
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (a.c.dev_status != nullptr) *a.c.dev_status = malformed ? GDN_ERR_OFFSETS : GDN_OK;
        if (a.status != nullptr) *a.status = malformed ? 1 : 0;
    }
}

// The long form: one block per key head, sequence, tile of BM rows and key part; the last tiles of a
// sequence (which see most keys) come first.  Key heads are the fastest index, so the blocks that read
// one head's keys at a time lie on few XCDs.  With prefix_rows the rows are all tokens' and the keys
// the prefix alone.
template <typename C>
__global__ __launch_bounds__(C::NT, C::WAVES) void long_kernel(Args a) {
    extern __shared__ __align__(1024) char lds[];
    long long total;
    const bool malformed = check_and_find<C::NT>(a.c, [](int, int) { return 0ll; }, &total);
    report(a, malformed);
    if (malformed) return;
    unsigned x = blockIdx.x;
    const int hk = x % a.c.HK;
    x /= a.c.HK;
    const int B = a.prefix_rows ? 1 : a.c.B, b = x % B;
    x /= B;
    const int part = x % a.splits, back = x / a.splits;
    const int first = uniform(a.prefix_rows ? 0 : a.c.offsets[b]);
    const int T = uniform(a.prefix_rows ? a.c.N : a.c.offsets[b + 1]) - first;
    const int rows = T * a.G, tiles = (rows + C::BM - 1) / C::BM, row0 = (tiles - 1 - back) * C::BM;
    if (row0 < 0 || rows == 0) return;
    int n = 0;
    long long begin = 0;
    if (!a.prefix_rows) {
        n = a.c.kv_len != nullptr ? uniform(a.c.kv_len[b]) : T;
        begin = a.c.kv_begin != nullptr ? uniform((long long)a.c.kv_begin[b]) : first;
    }
    const int seen0 = n - T + 1;
    const int last_token = min(row0 + C::BM, rows) - 1;
    const int reach = max(0, min(n, seen0 + last_token / a.G));  // keys the last row sees
    const int ptiles = (a.c.prefix_len + C::BN - 1) / C::BN, all = ptiles + (reach + C::BN - 1) / C::BN;
    const int t0 = (int)((long long)all * part / a.splits), t1 = (int)((long long)all * (part + 1) / a.splits);

    Block<C> blk(a, lds);
    blk.load_rows(row0, rows, first, hk);
    const Keys prefix{static_cast<const char*>(a.c.pk.p) + hk * a.c.pk.head * C::ES,
                      static_cast<const char*>(a.c.pv.p) + hk * a.c.pv.head * C::ES, a.c.prefix_len};
    const Keys own{static_cast<const char*>(a.c.k.p) + (begin * a.c.k.row + hk * a.c.k.head) * C::ES,
                   static_cast<const char*>(a.c.v.p) + (begin * a.c.v.row + hk * a.c.v.head) * C::ES, n};
    const int p1 = min(t1, ptiles), k0 = max(t0, ptiles) - ptiles, k1 = t1 - ptiles;
    if (t0 < p1) {
        blk.see(row0, rows, false, 0, a.c.prefix_len);
        blk.set_source(a.c.pk.row, a.c.pv.row);
        blk.run(prefix, t0, p1);
    }
    if (k0 < k1) {
        blk.see(row0, rows, true, seen0, n);
        blk.set_source(a.c.k.row, a.c.v.row);
        blk.run(own, k0, k1);
    }
    blk.join();
    const typename Block<C>::To to{row0, rows, first, hk, a.to_sets ? a.set0 + part : -1, -1};
    blk.store(to);
    if (__syncthreads_or(blk.spoiled))
        blk.redo(to, prefix, t0 * C::BN, min(p1 * C::BN, a.c.prefix_len), own, k0 * C::BN, max(0, min(k1 * C::BN, n)), seen0);
}

// The short form (a sequence's rows fit one tile): all (sequence, key head) runs laid end to end, counted
// in key tiles, and cut into equal parts, one a block.  A run inside one block is finished there; pieces of
// a cut run go to the workspace for the joining kernel.
template <typename C>
__global__ __launch_bounds__(C::NT, C::WAVES) void short_kernel(Args a) {
    extern __shared__ __align__(1024) char lds[];
    const int HK = a.c.HK;
    // a sequence without keys still has rows to write: one (masked) tile
    auto tiles_of = [](int T, int n) { return T <= 0 ? 0 : n <= C::BN ? 1 : (n + C::BN - 1) / C::BN; };
    auto units = [&](int T, int n) { return (long long)HK * tiles_of(T, n); };
    long long total;
    const bool malformed = check_and_find<C::NT>(a.c, units, &total);
    report(a, malformed);
    if (malformed || total == 0) return;
    const long long W = total < a.workers ? total : a.workers;
    if (blockIdx.x >= W) return;
    const int w = blockIdx.x;
    long long u = w * total / W;
    const long long u1 = (w + 1ll) * total / W;
    int b;
    long long base;
    find_unit<C::NT>(a.c, units, u, &b, &base);

    Block<C> blk(a, lds);
    blk.set_source(a.c.k.row, a.c.v.row);
    int first = 0, T = 0, n = 0, nt = 0;
    long long begin = 0;
    auto open = [&] {
        first = uniform(a.c.offsets[b]);
        T = uniform(a.c.offsets[b + 1]) - first;
        n = a.c.kv_len != nullptr ? uniform(a.c.kv_len[b]) : T;
        begin = a.c.kv_begin != nullptr ? uniform((long long)a.c.kv_begin[b]) : first;
        nt = tiles_of(T, n);
    };
    open();
    const int within = (int)(u - base);
    int hk = within / nt, tile = within - hk * nt;
    while (true) {
        const int count = (int)min((long long)(nt - tile), u1 - u), rows = T * a.G;
        blk.load_rows(0, rows, first, hk);
        blk.see(0, rows, true, n - T + 1, n);
        const Keys s{static_cast<const char*>(a.c.k.p) + (begin * a.c.k.row + hk * a.c.k.head) * C::ES,
                     static_cast<const char*>(a.c.v.p) + (begin * a.c.v.row + hk * a.c.v.head) * C::ES, n};
        blk.run(s, tile, tile + count);
        blk.join();
        // a worker's slot 0: its first run, cut at the front; slot 1: a run that goes on in the next worker
        const bool whole = count == nt;
        const typename Block<C>::To to{0, rows, first, hk, whole && a.to_sets ? a.set0 : -1,
                                       whole ? -1 : w * 2ll + (tile == 0 ? 1 : 0)};
        blk.store(to);
        if (T > 1 && __syncthreads_or(blk.spoiled))
            blk.redo(to, s, 0, 0, s, tile * C::BN, min((tile + count) * C::BN, n), n - T + 1);
        if (tile == 0 && a.row_info != nullptr) {
            // the worker that holds the run's last unit
            const long long last = u + nt - 1, w_last = ((last + 1) * W - 1) / total;
            for (int i = threadIdx.x; i < T; i += C::NT)
                a.row_info[(long long)(first + i) * HK + hk] = make_int2(whole ? -1 : w, (int)(w_last - w + 1) * 128 + i);
        }
        u += count;
        if (u >= u1) break;
        tile = 0;
        if (++hk == HK) {
            hk = 0;
            do {
                ++b;
                open();
            } while (nt == 0);
        }
    }
}

// ---- which tile for which call -------------------------------------------------------------------
// Head widths are compiled for 64, 128 and 256.  A stage holds about 32 KB of keys and values, so two
// blocks of two stages fit a CU.
template <typename T, int DP, int WR>
struct Pick;
#define GDN_ATTN_PICK(T, DP, WR, WK, KT, NS, WAVES) \
    template <>                                     \
    struct Pick<T, DP, WR> {                        \
        using C = Cfg<T, DP, WR, WK, 1, KT, NS, WAVES>; \
    };
#define GDN_ATTN_PICK_HALF(T)              \
    GDN_ATTN_PICK(T, 64, 1, 4, 1, 2, 2)    \
    GDN_ATTN_PICK(T, 64, 2, 2, 2, 2, 2)    \
    GDN_ATTN_PICK(T, 64, 4, 1, 2, 2, 2)    \
    GDN_ATTN_PICK(T, 128, 1, 2, 1, 2, 1)   \
    GDN_ATTN_PICK(T, 128, 2, 2, 1, 2, 2)   \
    GDN_ATTN_PICK(T, 128, 4, 1, 2, 2, 2)   \
    GDN_ATTN_PICK(T, 256, 1, 1, 1, 2, 1)   \
    GDN_ATTN_PICK(T, 256, 2, 1, 1, 2, 1)   \
    GDN_ATTN_PICK(T, 256, 4, 1, 1, 2, 2)
GDN_ATTN_PICK_HALF(BF16)
GDN_ATTN_PICK_HALF(F16)
GDN_ATTN_PICK(F32, 64, 1, 2, 1, 2, 1)
GDN_ATTN_PICK(F32, 64, 2, 2, 1, 2, 2)
GDN_ATTN_PICK(F32, 64, 4, 1, 2, 2, 2)
GDN_ATTN_PICK(F32, 128, 1, 1, 1, 2, 1)
GDN_ATTN_PICK(F32, 128, 2, 1, 1, 2, 1)
GDN_ATTN_PICK(F32, 128, 4, 1, 1, 2, 2)
GDN_ATTN_PICK(F32, 256, 1, 1, 1, 2, 1)
GDN_ATTN_PICK(F32, 256, 2, 1, 1, 2, 1)
GDN_ATTN_PICK(F32, 256, 4, 1, 1, 2, 1)

// What the host needs to know of a configuration.
struct Shape {
    int bm, bn, per_cu;
};
template <typename C>
constexpr Shape shape_of() {
    return Shape{C::BM, C::BN, 2 * C::LDS <= 156 * 1024 ? 2 : 1};
}

template <typename C, bool LONG>
hipError_t start(const Args& a, long long blocks, hipStream_t stream) {
    if (blocks > kMaxBlocks) return hipErrorInvalidConfiguration;
    void (*f)(Args);
    if constexpr (LONG) f = &long_kernel<C>;
    else f = &short_kernel<C>;
    // more than 64 KB of LDS has to be asked for; the attribute belongs to the current device
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
    if (e != hipSuccess) return e;
    f<<<(unsigned)blocks, C::NT, C::LDS, stream>>>(a);
    return hipGetLastError();
}

// dp 64, 128 or 256; wr 1, 2 or 4.  The long form runs at wr = 4.
template <typename T, typename F>
auto with_pick(int dp, int wr, F f) {
    switch (dp * 8 + wr) {
        case 64 * 8 + 1: return f(Pick<T, 64, 1>{});
        case 64 * 8 + 2: return f(Pick<T, 64, 2>{});
        case 64 * 8 + 4: return f(Pick<T, 64, 4>{});
        case 128 * 8 + 1: return f(Pick<T, 128, 1>{});
        case 128 * 8 + 2: return f(Pick<T, 128, 2>{});
        case 128 * 8 + 4: return f(Pick<T, 128, 4>{});
        case 256 * 8 + 1: return f(Pick<T, 256, 1>{});
        case 256 * 8 + 2: return f(Pick<T, 256, 2>{});
        default: return f(Pick<T, 256, 4>{});
    }
}

// One translation unit per type holds its kernels.
template <typename T>
hipError_t start_short(const Args& a, int dp, int wr, long long blocks, hipStream_t stream);
template <typename T>
hipError_t start_long(const Args& a, int dp, long long blocks, hipStream_t stream);

#define GDN_ATTN_INSTANCES(T)                                                                                     \
    template <>                                                                                                   \
    hipError_t start_short<T>(const Args& a, int dp, int wr, long long blocks, hipStream_t stream) {              \
        return with_pick<T>(dp, wr, [&](auto p) { return start<typename decltype(p)::C, false>(a, blocks, stream); }); \
    }                                                                                                             \
    template <>                                                                                                   \
    hipError_t start_long<T>(const Args& a, int dp, long long blocks, hipStream_t stream) {                       \
        if (dp == 64) return start<typename Pick<T, 64, 4>::C, true>(a, blocks, stream);                          \
        if (dp == 128) return start<typename Pick<T, 128, 4>::C, true>(a, blocks, stream);                        \
        return start<typename Pick<T, 256, 4>::C, true>(a, blocks, stream);                                       \
    }

}  // namespace attn
}  // namespace gdn
