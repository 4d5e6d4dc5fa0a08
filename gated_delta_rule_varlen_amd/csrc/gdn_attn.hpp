// gdn_attn.hpp -- the tile kernels of the softmax attention (instances per type in gdn_attn_<type>.hip,
// host side and the joining kernel in gdn_attn.hip).
//
// Rows.  The G = H/HK query heads of a key head and the tokens of a sequence form one list of query rows,
// row r = (token r / G, head r % G): a block's rows all read the same keys, so K and V are loaded once
// for the whole group.  A wave owns M of them, M = 32 in the long form (prompts: bound by the matrix cores) and 16
// in the short form (decode and drafts: bound by the cache's bytes).
//
// Products.  S^T = K Q^T and O^T = V^T P^T on MxM MFMA tiles: a lane's accumulators all belong to one
// query row (column lane % M), so the softmax statistics are one number a lane and rescaling O
// needs no exchange; the exponentials of S^T, rounded, are the second product's operand where they lie:
// with M = 32 the 16 scores of a lane are keys 8(i/4) + 4(lane/32) + i%4, and V^T is read with its keys in that
// order (a contraction may run in any order).
//
// Keys and values reach LDS by 16-byte asynchronous loads that write it directly, NS stages deep, with
// the 16-byte pieces of a row stored at place piece ^ f(row): an LDS read serves 16 rows of one piece (K) or 4
// to 8 rows of neighbouring pieces (V) at a time, and f differs between those (without it, two thirds of the
// LDS cycles were conflicts; now none).  The buffer's range check returns zeros for rows past the
// sequence's keys and pieces past D, so nothing outside a run is read, and nothing unwritten is used.
//
// Softmax in base 2: p = 2^(s*c - ref), c = scale*log2(e).  ref follows the running maximum only when
// that has grown by more than 2^8 (P stays in range, the quotient O / l is the same), so O is hardly ever rescaled.
//
// On the MI355X, by card: a prompt of 16384 tokens (H 16, HK 2, D 256, bf16) takes 1747 to 1867 us = 1.18 to 1.26 PFLOP/s,
// the matrix cores busy in 71% of the cycles; eight prompts of 24748 tokens (H 32, HK 8, D 128) 663 to 700 us = 0.95 to
// 1.0 PFLOP/s, busy in 54%; decode of 256 sequences over 2.26 GB of cache 357 to 363 us = 6.2 to 6.3 TB/s.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

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
constexpr int kMostKeys = INT_MAX - 4096;  // of a sequence: an index past its last tile still fits
constexpr int kPartKeys = 128;  // of a key part of the long form at least
constexpr float kNoMax = -3.0e38f;    // running maximum before the first key: below every score
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What a launch needs beside the call's own arguments.
struct Args {
    AttnLaunch c;
    int G;          // heads per key head
    float s2;       // |scale| * log2(e); the sign goes to the queries
    bool negate;
    int splits;     // key parts of the long form at most: a sequence has one for every kPartKeys of its keys
    int workers;    // blocks of the short form
    bool to_sets;   // results go to the workspace, for the joining kernel
    int local_set;  // the set of a sequence's own keys, behind the prefix's key parts
    long long prefix_blocks;  // blocks of the long form that run all tokens' rows over the prefix alone
    // workspace
    int* status;
    int2* row_info;    // [N][HK]: x = worker a cut run starts in (-1: not cut), y = pieces * 128 + token in sequence
    int4* cut;         // [workers]: first token, tokens, key head, pieces of the cut run that starts there (tokens 0: none)
    float* slot_o;     // [workers][2][BM][D]
    float2* slot_ml;   // [workers][2][BM]
    float* set_o;      // [sets][N*H][D]
    float2* set_ml;    // [sets][N*H]
    int sets;
    long long set_rows;  // N*H
    int* live;         // [N]: sets that the long form wrote of a token's rows
};

// Accumulators of an M x M tile, and one step of its product: 16 bytes of each operand's rows a lane.
template <int M>
struct AccOf {
    typedef float type __attribute__((ext_vector_type(M* M / 64)));
};
template <int M>
using Acc = typename AccOf<M>::type;

template <typename T, int M>
__device__ __forceinline__ void multiply(u32x4 a, u32x4 b, Acc<M>& c) {
    if constexpr (T::code == GDN_BF16) {
        const bf16x8 x = __builtin_bit_cast(bf16x8, a), y = __builtin_bit_cast(bf16x8, b);
        if constexpr (M == 32) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, c, 0, 0, 0);
        else c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
    } else if constexpr (T::code == GDN_F16) {
        const f16x8 x = __builtin_bit_cast(f16x8, a), y = __builtin_bit_cast(f16x8, b);
        if constexpr (M == 32) c = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, y, c, 0, 0, 0);
        else c = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = __uint_as_float(a[j]), y = __uint_as_float(b[j]);
            if constexpr (M == 32) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x, y, c, 0, 0, 0);
            else c = __builtin_amdgcn_mfma_f32_16x16x4f32(x, y, c, 0, 0, 0);
        }
    }
}
template <int M>
__device__ __forceinline__ void multiply1(float x, float y, Acc<M>& c) {
    if constexpr (M == 32) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x, y, c, 0, 0, 0);
    else c = __builtin_amdgcn_mfma_f32_16x16x4f32(x, y, c, 0, 0, 0);
}

// Two values rounded to the half type T.
template <typename T>
__device__ __forceinline__ uint32_t pack(float x, float y) {
    if constexpr (T::code == GDN_BF16) {
        typedef __bf16 v2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, v2{(__bf16)x, (__bf16)y});
    } else {
        typedef _Float16 v2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, v2{(_Float16)x, (_Float16)y});
    }
}

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

// Maximum and sum over the 64 / M lanes that share a query row.
template <bool MAX>
__device__ __forceinline__ float both(uint32_t x, uint32_t y) {
    return MAX ? fmaxf(__uint_as_float(x), __uint_as_float(y)) : __uint_as_float(x) + __uint_as_float(y);
}
template <int M, bool MAX>
__device__ __forceinline__ float over_row(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = both<MAX>(r[0], r[1]);
    if constexpr (M == 16) {
        const auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = both<MAX>(q[0], q[1]);
    }
    return x;
}

// A value every lane holds, as a scalar.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ long long uniform(long long x) {
    return ((long long)uniform((int)(x >> 32)) << 32) | (uint32_t)uniform((int)x);
}

// An entry of one of the call's small arrays (nothing writes them while it runs), through the scalar cache: a
// vector load here would wait for every tile on its way.
template <typename X>
__device__ __forceinline__ X entry(const X* p, int i) {
    return ((const __attribute__((address_space(4))) X*)p)[i];
}

// 64 x 16 bytes to LDS, at `at` + 16 * lane, from base + voff + soff of a range of `bytes`; zeros past it.  No register
// waits for this load, and wait_and_meet() counts it.  (As a builtin the compiler would wait for all of them
// before every transposing LDS read.)
struct Range {
    u32x4 r;
    __device__ __forceinline__ Range(const void* base, int bytes) {
        const uint64_t b = reinterpret_cast<uint64_t>(base);
        r = u32x4{(uint32_t)b, (uint32_t)(b >> 32) & 0xffffu, (uint32_t)bytes, (uint32_t)kRsrc};
    }
};
// A statement carries the five wait states that a vector memory instruction needs behind a vector one that wrote a scalar
// register it reads (a spilled one comes back by v_readlane), as the compiler adds none ahead of assembly.  Four loads share
// them: one token over 131072 keys 54.2 us without, 55.5 with them at every load.
// STREAM: the bytes are read by this block alone (decode of 256 sequences: 357 us, without the hint 408).
#define GDN_LOAD(hint)                                                                                                 \
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen" hint " lds"                     \
                 ::"s"(at), "v"(voff), "s"(s.r), "s"(soff) : "m0", "memory")
template <bool STREAM>
__device__ __forceinline__ void load_to_lds(const Range& s, uint32_t at, int voff, int soff) {
    if constexpr (STREAM) GDN_LOAD(" nt");
    else GDN_LOAD("");
}
#undef GDN_LOAD
// Four of them, NEXT bytes apart in LDS.
#define GDN_LOAD(hint)                                                                                                 \
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %5, %6 offen" hint " lds\n\t"                 \
                 "s_add_u32 m0, %0, %10\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %5, %7 offen" hint " lds\n\t"            \
                 "s_add_u32 m0, %0, %11\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %5, %8 offen" hint " lds\n\t"            \
                 "s_add_u32 m0, %0, %12\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, %5, %9 offen" hint " lds"                \
                 ::"s"(at), "v"(voff[0]), "v"(voff[1]), "v"(voff[2]), "v"(voff[3]), "s"(s.r), "s"(soff[0]), "s"(soff[1]), \
                 "s"(soff[2]), "s"(soff[3]), "n"(NEXT), "n"(2 * NEXT), "n"(3 * NEXT) : "m0", "scc", "memory")
template <bool STREAM, int NEXT>
__device__ __forceinline__ void load_four_to_lds(const Range& s, uint32_t at, const int* voff, const int* soff) {
    if constexpr (STREAM) GDN_LOAD(" nt");
    else GDN_LOAD("");
}
#undef GDN_LOAD

// Sequence i of the call as its arrays give it, in bounds whatever they hold: what a block asks for before the
// whole call is checked lies inside the tensors.
struct Sequence {
    int first, T, n;
    long long begin;
};
__device__ __forceinline__ Sequence sequence(const AttnLaunch& c, int i) {
    Sequence s;
    s.first = min(max(uniform(entry(c.offsets, i)), 0), c.N);
    s.T = min(max(uniform(entry(c.offsets, i + 1)) - s.first, 0), min(c.max_q, c.N - s.first));
    if (c.kv_len != nullptr) {
        const long long n = max(uniform(entry(c.kv_len, i)), 0), begin = uniform((long long)entry(c.kv_begin, i));
        s.n = (int)min(n, c.kv_rows);
        s.begin = min(max(begin, 0ll), c.kv_rows - s.n);
    } else {
        s.begin = min((long long)s.first, c.kv_rows);
        s.n = (int)min((long long)s.T, c.kv_rows - s.begin);
    }
    return s;
}

// Row tiles end to end without a sum over the sequences: those of sequence b start at slot offsets[b] * G / BM + b.
// ceil(T * G / BM) is at most one more than the difference of two neighbours' quotients, so the next sequence's slots
// begin behind them, and N * G / BM + B slots hold all.
template <int BM>
__device__ __forceinline__ unsigned slot_of(const AttnLaunch& c, int G, int offset, int b) {
    return (unsigned)(min(max(offset, 0), c.N) * G) / BM + (unsigned)b;
}
// The last sequence that starts at `slot` or before it: 64 candidates a step, a sequence of the call whatever its
// offsets hold.
template <int BM>
__device__ __forceinline__ int sequence_at(const AttnLaunch& c, int G, unsigned slot) {
    int lo = 0, hi = c.B;
    while (hi - lo > 1) {
        const int step = (hi - lo - 1) / 64 + 1, i = lo + min((int)(threadIdx.x & 63), (hi - lo - 1) / step) * step;
        const uint64_t here = __builtin_amdgcn_ballot_w64(slot_of<BM>(c, G, c.offsets[i], i) <= slot);
        const int at = here == 0 ? 0 : 63 - __builtin_clzll(here);
        lo = uniform(lo + min(at, (hi - lo - 1) / step) * step);
        hi = min(hi, lo + step);
    }
    return lo;
}

// Up to 64 sequences, one a lane: their row tiles end to end without gaps, those of the one with most keys first, so that
// the last blocks are short ones.  The tile's place from the end of its sequence b; past all tiles a large number.
template <int BM>
__device__ __forceinline__ unsigned by_keys(const AttnLaunch& c, int G, unsigned slot, int* b) {
    const int lane = threadIdx.x & 63, i = min(lane, c.B - 1);
    const int o = min(max(c.offsets[i], 0), c.N), T = min(max(c.offsets[i + 1], o), c.N) - o;
    const int n = c.kv_len != nullptr ? c.kv_len[i] : T;
    const int tiles = lane < c.B ? (T * G + BM - 1) / BM : 0;
    unsigned start = 0;
    for (int j = 0; j < c.B; ++j) {
        const int other = __builtin_amdgcn_readlane(n, j), t = __builtin_amdgcn_readlane(tiles, j);
        start += (other > n) | (other == n && j < lane) ? t : 0;
    }
    const uint64_t here = __builtin_amdgcn_ballot_w64(slot - start < (unsigned)tiles);
    if (here == 0) return ~0u;
    *b = uniform((int)__builtin_ctzll(here));
    return slot - (unsigned)__builtin_amdgcn_readlane((int)start, *b);
}

// Sequence i as the arrays have it, and whether it is malformed.
struct Entry {
    int o, e, n;
    long long begin;
    __device__ __forceinline__ void read(const AttnLaunch& c, int i) {
        o = c.offsets[i];
        e = c.offsets[i + 1];
        n = c.kv_len != nullptr ? c.kv_len[i] : 0;
        begin = c.kv_begin != nullptr ? c.kv_begin[i] : 0;
    }
    __device__ __forceinline__ bool bad(const AttnLaunch& c, int i) const {
        const int t = e - o;
        const bool offsets = (t < 0) | (t > c.max_q) | (i == 0 && o != 0) | (i == c.B - 1 && e != c.N);
        if (c.kv_len == nullptr) return offsets | (e > c.kv_rows) | (t > kMostKeys);
        return offsets | (n < 0) | (n > kMostKeys) | (begin < 0) | (begin > c.kv_rows) | (begin + n > c.kv_rows);
    }
    __device__ __forceinline__ int keys(const AttnLaunch& c) const { return c.kv_len != nullptr ? n : e - o; }
};
// Whole-call check.  Reached by all threads.
template <int NT>
__device__ __forceinline__ bool check(const AttnLaunch& c) {
    int bad = 0;
    for (int i = threadIdx.x; i < c.B; i += NT) {
        Entry s;
        s.read(c, i);
        bad |= s.bad(c, i);
    }
    return __syncthreads_or(bad) != 0;
}
// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ uint32_t scan_lanes(uint32_t x) {
#define GDN_SCAN_STEP(ctrl, rows) x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, rows, 0xf, false)
    GDN_SCAN_STEP(0x111, 0xf);  // from 1, 2, 4 and 8 lanes below, in each 16
    GDN_SCAN_STEP(0x112, 0xf);
    GDN_SCAN_STEP(0x114, 0xf);
    GDN_SCAN_STEP(0x118, 0xf);
    GDN_SCAN_STEP(0x142, 0xa);  // the sum of 16 to the second and fourth 16, that of 32 to the upper half
    GDN_SCAN_STEP(0x143, 0xc);
#undef GDN_SCAN_STEP
    return x;
}

// The call's sequences with their key tiles: the whole-call check, the sum of the tiles, and the sequence that holds
// a given tile.  Every wave goes over all sequences by itself, 64 a time; the first 256 stay in its registers, so a
// decode step reads the call's arrays once.
template <int BN>
struct Tiles {
    static constexpr int KEEP = 4;
    const AttnLaunch& c;
    uint32_t upto[KEEP];  // tiles of the 64 up to and with the lane's sequence
    long long total = 0;
    bool malformed = false;

    // a sequence without keys still has rows to write: one (masked) tile
    static __device__ __forceinline__ int of(int T, int n) { return T <= 0 ? 0 : n <= BN ? 1 : (int)(((unsigned)n + BN - 1) / BN); }

    __device__ __forceinline__ explicit Tiles(const AttnLaunch& c_) : c(c_) {
        const int lane = threadIdx.x & 63;
        bool bad = false;
        Entry s[KEEP] = {};
#pragma unroll
        for (int j = 0; j < KEEP; ++j)
            if (64 * j < c.B) s[j].read(c, min(64 * j + lane, c.B - 1));  // all on their way before one is used
#pragma unroll
        for (int j = 0; j < KEEP; ++j) {
            upto[j] = 0;
            if (64 * j < c.B) {
                upto[j] = count(s[j], 64 * j + lane, &bad);
                total += (uint32_t)__builtin_amdgcn_readlane((int)upto[j], 63);
            }
        }
        for (int i0 = 64 * KEEP; i0 < c.B; i0 += 64) {
            s[0].read(c, min(i0 + lane, c.B - 1));
            total += (uint32_t)__builtin_amdgcn_readlane((int)count(s[0], i0 + lane, &bad), 63);
        }
        malformed = __builtin_amdgcn_ballot_w64(bad) != 0;
    }
    // Tiles of the lanes' sequences (lane i has entry i) up to and with each one.
    __device__ __forceinline__ uint32_t count(const Entry& s, int i, bool* bad) const {
        *bad |= s.bad(c, min(i, c.B - 1));
        return scan_lanes(i < c.B ? (uint32_t)of(s.e - s.o, s.keys(c)) : 0u);
    }
    // The sequence of tile v < total, and the tiles before that sequence.
    __device__ __forceinline__ void find(long long v, int* b, long long* before) const {
        const int lane = threadIdx.x & 63;
        long long sum = 0;
        auto here = [&](int i0, uint32_t with) {
            const uint32_t all = (uint32_t)__builtin_amdgcn_readlane((int)with, 63);
            if (v - sum >= all) {
                sum += all;
                return false;
            }
            // the first lane whose tiles go past v
            const int at = __ffsll((unsigned long long)__builtin_amdgcn_ballot_w64(with > (uint32_t)(v - sum))) - 1;
            *b = i0 + at;
            *before = sum + (at == 0 ? 0u : (uint32_t)__builtin_amdgcn_readlane((int)with, at - 1));
            return true;
        };
#pragma unroll
        for (int j = 0; j < KEEP; ++j)
            if (here(64 * j, upto[j])) return;
        for (int i0 = 64 * KEEP; i0 < c.B; i0 += 64) {
            Entry s;
            bool bad = false;
            s.read(c, min(i0 + lane, c.B - 1));
            if (here(i0, count(s, i0 + lane, &bad))) return;
        }
    }
};

// `total` units in W parts that differ by one at most: where part w starts, and which part holds unit u.
struct Cut {
    long long size, longer;  // the first `longer` parts have size + 1
    __device__ __forceinline__ Cut(long long total, int W) {
        size = total >> 31 ? total / W : (long long)((unsigned)total / (unsigned)W);
        longer = total - size * W;
    }
    __device__ __forceinline__ long long start(long long w) const { return w * size + min(w, longer); }
    __device__ __forceinline__ int part(long long u) const {
        const long long x = longer * (size + 1), a = u < x ? u : u - x, d = u < x ? size + 1 : size;
        return (int)((u < x ? 0 : longer) + (a >> 31 ? a / d : (long long)((unsigned)a / (unsigned)d)));
    }
};

template <typename T_, int M_, int DP_, int WR_, int KT_, int NS_, int WAVES_, int QL_ = 10>
struct Cfg {
    using T = T_;
    using TS = typename T::storage;
    static constexpr int M = M_, DP = DP_, KT = KT_, NS = NS_, WAVES = WAVES_;
    static constexpr bool HALF = sizeof(TS) == 2;
    static constexpr int ES = sizeof(TS), NW = WR_, NT = 64 * NW, BM = M * NW, BN = 32 * KT;
    static constexpr int NG = 64 / M;             // lanes that share a query row
    static constexpr int EA = M * M / 64;         // accumulators a lane and tile
    static constexpr int SUB = 32 / M;            // tiles that make up 32 keys
    static constexpr int RB = DP * ES;            // bytes of a row in LDS
    static constexpr int CPR = RB / 16;           // 16-byte pieces of a row
    static constexpr int CS = RB / (16 * NG);     // operand steps of a score tile
    static constexpr int DT = DP / M;             // M-wide parts of the head
    static constexpr int TILE = BN * RB;
    // Rows in LDS: 1024 bytes after 1024 bytes as they are loaded, those of the widest half-precision rows of the
    // long form PAD apart: with that the places of a row's pieces depend on one bit of its index only, and the reads
    // of a tile are a register or two and a constant each, where eight registers were spilled.
    static constexpr bool PADDED = M == 32 && RB == 512 && HALF;
    static constexpr int KB = TILE / 1024, KSTEP = 1024 + (PADDED ? 32 : 0), VSTEP = 1024 + (PADDED ? 128 : 0);
    static constexpr int KTILE = KB * KSTEP, STAGE = KTILE + KB * VSTEP;
    template <int STEP>
    static __device__ __forceinline__ constexpr int row_at(int r) {
        return STEP == 1024 ? r * RB : r / (1024 / RB) * STEP + r % (1024 / RB) * RB;
    }
    static constexpr int POW = NW >= 8 ? 8 : NW >= 4 ? 4 : NW >= 2 ? 2 : 1;
    static constexpr int LW = POW * 1024 <= TILE ? POW : TILE / 1024;  // waves that load
    static constexpr int JN = TILE / (LW * 1024);  // loads such a wave issues for one of K, V
    static constexpr int RPI = LW * 64 / CPR;      // rows one load of all of them covers
    static constexpr int PRE = RPI >= 16 ? 1 : 16 / RPI;  // after which the places of a row's pieces repeat
    // Operand steps of the queries that lie in LDS, behind the ring: at width 256 eight waves' share of the CU's
    // registers holds six (with ten in LDS a 16384-token prompt takes 1785 us, with seven and spills 2195)
    static constexpr int QL = PADDED ? QL_ : 0;
    static constexpr int RING = NS * STAGE, LDS = RING + QL * NW * 1024;
    static constexpr bool PIPE = RB <= 256;       // the registers hold two tiles' scores (long form)
    static_assert(CPR >= 8 && TILE % (LW * 1024) == 0 && RPI >= 1 && LDS <= 159 * 1024 && JN % PRE == 0, "tile");
    // Where the pieces of row r are stored: at place piece ^ this.  16 places are the 256 bytes the banks span.
    static __device__ __forceinline__ int place_k(int r) { return PADDED ? r & 1 : RB == 128 ? (r >> 1) & 7 : r & 15; }
    static __device__ __forceinline__ int place_v(int r) {
        const int b0 = r & 1, b1 = (r >> 1) & 1, b2 = (r >> 2) & 1;
        return PADDED ? b0 << 2 : RB == 128 ? b1 << 2 | b2 << 1 : b1 << 3 | b0 << 2 | b2 << 1;
    }
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
    static constexpr int M = C::M, KT = C::KT, DT = C::DT;

    const Args& a;
    char* lds;
    int lane, wave, col, grp;  // the lane's query row in the wave's tile, and its place among the lanes of that row
    uint32_t lds_base;                      // LDS address of the ring
    int row_bytes;                          // of a head
    float c;                                // scores to base 2
    int kstride, vstride;                   // bytes between rows of this source
    int koff[C::PRE], voff[C::PRE];
    u32x4 q[C::CS - C::QL];
    int vis;                                // keys the lane's row sees
    int vis_lo, vis_hi;                     // over the wave's rows
    int run_n;                              // keys of the run
    bool spoiled = false;                   // the wave met values only redo() can deal with
    Acc<M> o[DT];
    float ref, l;

    __device__ __forceinline__ Block(const Args& a_, char* lds_) : a(a_), lds(lds_) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        col = lane & (M - 1);
        grp = lane / M;
        lds_base = uniform((int)(uintptr_t)(__attribute__((address_space(3))) char*)lds);
        row_bytes = a.c.D * C::ES;
        c = a.s2;
        asm volatile("" : "+s"(c));  // a register: not read again for every tile
    }

    // byte offsets of the 16-byte pieces this lane loads, for rows `ks` and `vs` bytes apart
    __device__ __forceinline__ void set_source(long long krow, long long vrow) {
        kstride = (int)(krow * C::ES);
        vstride = (int)(vrow * C::ES);
#pragma unroll
        for (int j = 0; j < C::PRE; ++j) {
            const int p = (j * C::LW + wave) * 64 + lane, row = p / C::CPR, place = p % C::CPR;
            const int kp = (place ^ C::place_k(row)) * 16, vp = (place ^ C::place_v(row)) * 16;
            koff[j] = kp < row_bytes ? row * kstride + kp : kOutside;
            voff[j] = vp < row_bytes ? row * vstride + vp : kOutside;
        }
    }

    template <bool V>
    __device__ __forceinline__ void load_half(const Keys& s, int tile, bool real, int stage) {
        if (C::LW < C::NW && wave >= C::LW) return;
        const int k0 = tile * C::BN, left = s.n - k0, rows = left < C::BN ? left : C::BN, stride = V ? vstride : kstride;
        const Range r((V ? s.v : s.k) + (long long)k0 * stride, real && rows > 0 ? (rows - 1) * stride + row_bytes : 0);
        constexpr int STEP = V ? C::VSTEP : C::KSTEP;
        const uint32_t to = lds_base + stage * C::STAGE + (V ? C::KTILE : 0) + wave * STEP;
        constexpr int NEXT = C::LW * STEP, BY = C::JN % 4 == 0 ? 4 : 1;
#pragma unroll
        for (int j = 0; j < C::JN; j += BY) {
            int v[BY], row[BY];
#pragma unroll
            for (int i = 0; i < BY; ++i) {
                v[i] = (V ? voff : koff)[(j + i) % C::PRE];
                row[i] = (j + i) / C::PRE * C::PRE * C::RPI * stride;
            }
            if constexpr (BY == 4) load_four_to_lds<M == 16, NEXT>(r, to + j * NEXT, v, row);
            else load_to_lds<M == 16>(r, to + j * NEXT, v[0], row[0]);
        }
    }
    __device__ __forceinline__ void load_tile(const Keys& s, int tile, bool real, int stage) {
        load_half<false>(s, tile, real, stage);
        load_half<true>(s, tile, real, stage);
    }

    // Queries of the block's rows row0 .. (of `rows` in the list); rows past the list are zeros.
    __device__ __forceinline__ void load_rows(int row0, int rows, long long first, int hk) {
        const int G = a.G, r = row0 + wave * M + col, i = r / G, g = r - i * G;
        const bool in = r < rows;
        // lanes without an element read the row's first instead, so no load stands in a branch
        const TS* p = static_cast<const TS*>(a.c.q.p) + (first + (in ? i : 0)) * a.c.q.row +
                      (long long)(hk * G + (in ? g : 0)) * a.c.q.head;
        const uint32_t flip = !a.negate ? 0u : C::HALF ? 0x80008000u : 0x80000000u;
        u32x4 x[C::CS];
#pragma unroll
        for (int s = 0; s < C::CS; ++s) {
            const int e = (C::NG * s + grp) * (16 / C::ES);
            x[s] = *reinterpret_cast<const u32x4*>(p + (e < a.c.D ? e : 0));
        }
#pragma unroll
        for (int s = 0; s < C::CS; ++s) {
            const uint32_t keep = in && (C::NG * s + grp) * (16 / C::ES) < a.c.D ? ~0u : 0u;
            x[s] = (x[s] ^ flip) & keep;
            if (s < C::CS - C::QL) q[s] = x[s];
            else *query_at(s) = x[s];
        }
        clear();
    }

    __device__ __forceinline__ void clear() {
        spoiled = false;
        ref = kNoMax;
        l = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = Acc<M>{};
    }

    // Where this lane keeps operand step s of its queries in LDS, for the last QL of them.
    __device__ __forceinline__ u32x4* query_at(int s) {
        return reinterpret_cast<u32x4*>(lds + C::RING + (wave * C::QL + s - (C::CS - C::QL)) * 1024 + lane * 16);
    }

    // The short form takes queries through LDS, as rows at `at` laid out like the keys': asked for with the run's
    // first tile, long before they are needed, and read when the run begins.
    __device__ __forceinline__ void ask_rows(int at, int T, long long first, int hk) {
        if (C::LW < C::NW && wave >= C::LW) return;  // as for the tiles: only who loads those waits in order for these
        const int G = a.G, rows = T * G;
        const char* p = static_cast<const char*>(a.c.q.p) + (first * a.c.q.row + (long long)hk * G * a.c.q.head) * C::ES;
        const int bytes = (int)(((T - 1) * a.c.q.row + (G - 1) * a.c.q.head + a.c.D) * C::ES);
        const Range rq(p, bytes);
        const int padded = (rows + 7) & ~7;
        for (int x = wave * 64; x < padded * C::CPR; x += C::LW * 64) {
            const int r = (x + lane) / C::CPR, piece = ((x + lane) % C::CPR) ^ C::place_k(r), i = r / G, g = r - i * G;
            const int off = r < rows && piece * 16 < a.c.D * C::ES
                                ? (int)((i * a.c.q.row + g * a.c.q.head) * C::ES) + piece * 16 : kOutside;
            load_to_lds<false>(rq, lds_base + at + x * 16, off, 0);
        }
    }
    __device__ __forceinline__ void take_rows(const char* at, int rows) {
        const uint32_t flip = !a.negate ? 0u : C::HALF ? 0x80008000u : 0x80000000u;
        const int r = wave * M + col, have = r < rows ? r : 0;
        const uint32_t keep = r < rows ? ~0u : 0u;  // rows past the list were not loaded
        const char* p = at + have * C::RB;
#pragma unroll
        for (int s = 0; s < C::CS - C::QL; ++s)
            q[s] = (*reinterpret_cast<const u32x4*>(p + (((C::NG * s + grp) ^ C::place_k(have)) * 16)) ^ flip) & keep;
        clear();
    }

    // The keys each row sees of a run of n: all, or (causal) seen0 + its token, at least 0 and at most n.
    __device__ __forceinline__ void see(int row0, int rows, bool causal, int seen0, int n) {
        run_n = n;
        const int G = a.G, lo = row0 + wave * M, hi = min(lo + M, rows) - 1, r = lo + col;
        auto keys = [&](int x) { return causal ? min(max(seen0 + x / G, 0), n) : n; };
        vis = r < rows ? keys(r) : n;
        vis_lo = uniform(keys(lo));
        vis_hi = uniform(lo < rows ? keys(hi) : 0);
    }

    static constexpr int SN = C::SUB * C::EA;  // scores of 32 keys a lane
    using Scores = Acc<M>[KT][C::SUB];

    // The fp32 products of a score in the short form are summed in four chains: one sum of 256 after the other was off by
    // up to 2.7 times as much as one in a tree (outputs of a token over 63 keys of D 256: 7.8e-7, so 2.9e-7).  The long
    // form keeps one, as a plain product does: it has no registers for more (D 256, 8192 tokens: 2.6 ms, with four 3.2).
    static constexpr int CHAINS = C::HALF || M == 32 ? 1 : 4;
    // Scores of a stage's keys: element i of a lane's scores of 32 keys is key 4 NG (i / 4) + 4 grp + i % 4.
    template <bool GROUPED>
    __device__ __forceinline__ void scores(int stage, Scores& acc) {
        const char* kt_ = lds + stage * C::STAGE + C::template row_at<C::KSTEP>(col);
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int u = 0; u < C::SUB; ++u) acc[k][u] = Acc<M>{};
        Acc<M> more[CHAINS][KT][C::SUB] = {};  // of chains 1 to CHAINS - 1
        // operands are read in groups ahead of the products that use them
        constexpr int KG = C::CS < 8 ? C::CS : C::CS > 8 && C::WAVES > 1 ? 4 : 8;
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int x0 = 0; x0 < C::CS; x0 += KG) {
                u32x4 f[KG][C::SUB];
#pragma unroll
                for (int x = 0; x < KG; ++x)
#pragma unroll
                    for (int u = 0; u < C::SUB; ++u)
                        f[x][u] = *reinterpret_cast<const u32x4*>(kt_ + C::template row_at<C::KSTEP>(k * 32 + u * M) +
                                                                  (((C::NG * (x0 + x) + grp) ^ C::place_k(col)) * 16));
                if constexpr (GROUPED) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int x = 0; x < KG; ++x) {
                    const u32x4 y = x0 + x < C::CS - C::QL ? q[x0 + x] : *query_at(x0 + x);
#pragma unroll
                    for (int u = 0; u < C::SUB; ++u)
                        multiply<T, M>(f[x][u], y, (x0 + x) % CHAINS == 0 ? acc[k][u] : more[(x0 + x) % CHAINS][k][u]);
                }
            }
        if constexpr (CHAINS == 4) {
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int u = 0; u < C::SUB; ++u) acc[k][u] = (acc[k][u] + more[1][k][u]) + (more[2][k][u] + more[3][k][u]);
        }
    }
    // Hides the keys a row does not see; base = index of the tile's first key in the run.
    __device__ __forceinline__ void hide(Scores& s, int base) {
        const int room = vis - base - 4 * grp;
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int i = 0; i < SN; ++i)
                s[k][i / C::EA][i % C::EA] = 32 * k + 4 * C::NG * (i / 4) + i % 4 >= room ? -INFINITY : s[k][i / C::EA][i % C::EA];
    }
    // The largest score of each row, to base 2.
    __device__ __forceinline__ float largest(const Scores& s) {
        float top = s[0][0][0];
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int i = 0; i < SN; ++i) top = fmaxf(top, s[k][i / C::EA][i % C::EA]);
        return over_row<M, true>(top) * c;
    }
    __device__ __forceinline__ void follow(float top) {
        if (__builtin_amdgcn_ballot_w64(top > ref + (C::BIAS + C::LAG)) != 0) {
            const float to = fmaxf(ref, top - C::BIAS), w = __builtin_amdgcn_exp2f(ref - to);
            ref = to;
            l *= w;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= w;
        }
    }
    __device__ __forceinline__ void exponentials(Scores& s) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int i = 0; i < SN; ++i) {
                const float p = __builtin_amdgcn_exp2f(fmaf(s[k][i / C::EA][i % C::EA], c, -ref));
                s[k][i / C::EA][i % C::EA] = p;
                sum += p;
            }
        l += sum;
    }
    // 0 * infinity is NaN: where rows differ in what they see, a value that is not finite would reach the
    // rows that must not see it.  Such a tile is found here and the wave's rows are done again by redo().
    __device__ __forceinline__ void look(const char* vt, int base) {
        if (vis_lo < min(base + C::BN, run_n)) spoiled |= any_not_finite(vt);
    }

    // A stage's keys and values against the wave's rows.  The reads of values run ahead of their products, the first
    // of them ahead of the softmax: one after the other they took longer than the tile's bytes from memory.
    __device__ __forceinline__ void use_tile(int stage, int base) {
        if (base >= vis_hi) return;
        static_assert(KT == 1, "a tile of 32 keys");
        const char* vt = lds + stage * C::STAGE + C::KTILE;
        constexpr int N = C::HALF ? DT * (SN / 8) : DT * SN, AHEAD = N < 8 ? N : 8;
        using Value = std::conditional_t<C::HALF, u32x4, float>;
        Value v[N];
        auto read = [&](int x) {
            if constexpr (C::HALF) v[x] = values(vt, 0, x / DT, x % DT);
            else v[x] = value(vt, 0, x / DT, x % DT);
        };
        Scores s;
        scores<true>(stage, s);
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) read(x);
        __builtin_amdgcn_sched_barrier(0);
        if (base + C::BN > vis_lo) {
            hide(s, base);
            asm volatile("");  // keeps this a branch: most tiles hide nothing
        }
        follow(largest(s));
        exponentials(s);
        look(vt, base);
        u32x4 p;
#pragma unroll
        for (int x = 0; x < N; ++x) {
            if (C::HALF && x % DT == 0) p = packed(s, 0, x / DT);
            if (x + AHEAD < N) read(x + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (C::HALF) multiply<T, M>(v[x], p, o[x % DT]);
            else multiply1<M>(v[x], s[0][x / DT / C::EA][x / DT % C::EA], o[x % DT]);
        }
    }

    __device__ __forceinline__ bool any_not_finite(const char* vt) {
        uint32_t acc = 0;
#pragma unroll 1
        for (int i = 0; i < C::KB; ++i) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(vt + i * C::VSTEP + lane * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc |= not_finite_sign<T>(x[j]);
        }
        return __builtin_amdgcn_ballot_w64((acc & (C::HALF ? 0x80008000u : 0x80000000u)) != 0) != 0;
    }

    // Operands of the second product: eight probabilities a lane, and the values of the same keys.
    static __device__ __forceinline__ u32x4 packed(const Scores& s, int k, int z) {
        u32x4 p;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 8 * z + 2 * e;
            p[e] = pack<T>(s[k][i / C::EA][i % C::EA], s[k][(i + 1) / C::EA][(i + 1) % C::EA]);
        }
        return p;
    }
    __device__ __forceinline__ u32x4 values(const char* vt, int k, int z, int d) {
        // lane x of 16 names key x/4 of its four and elements 4(x%4) .. of a 16-wide part of the head
        const int x = lane & 15, part = M == 32 ? (lane >> 4) & 1 : 0, key = 4 * grp + (x >> 2), sw = C::place_v(key);
        const int piece = M / 8 * d + 2 * part + ((x >> 1) & 1);
        const char* at = vt + C::template row_at<C::VSTEP>(key) + (x & 1) * 8 +
                         C::template row_at<C::VSTEP>(32 * k + 8 * C::NG * z) + ((piece ^ sw) * 16);
        union {
            v4i16 h[2];
            u32x4 v;
        } f;
        f.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16*)(at));
        f.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) v4i16*)(at + C::template row_at<C::VSTEP>(4 * C::NG)));
        return f.v;
    }

    __device__ __forceinline__ float value(const char* vt, int k, int i, int d) {
        const int key = 4 * grp + i % 4, sw = C::place_v(key);
        const char* row = vt + (32 * k + 4 * C::NG * (i / 4) + key) * C::RB + (col & 3) * 4;
        return *reinterpret_cast<const float*>(row + (((M / 4 * d + (col >> 2)) ^ sw) * 16));
    }

    // O^T += V^T P^T for the tile at vt.
    __device__ __forceinline__ void product(const char* vt, const Scores& s) {
        if constexpr (C::HALF) {
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int z = 0; z < SN / 8; ++z) {  // eight scores a lane are one step: 8 NG keys
                    const u32x4 p = packed(s, k, z);
#pragma unroll
                    for (int d = 0; d < DT; ++d) multiply<T, M>(values(vt, k, z, d), p, o[d]);
                }
        } else {
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int i = 0; i < SN; ++i)
#pragma unroll
                    for (int d = 0; d < DT; ++d) multiply1<M>(value(vt, k, i, d), s[k][i / C::EA][i % C::EA], o[d]);
        }
    }

    // LDS addresses are worth registers inside a loop over tiles, not across a block's runs.
    __device__ __forceinline__ void fresh_addresses() {
        asm volatile("" : "+v"(lane));
        col = lane & (M - 1);
        grp = lane / M;
    }

    // One tile of the long form's pipeline.  While the matrix cores form the next tile's scores, the vector unit
    // takes this one's exponentials, and while they multiply those with the values, the next tile's maximum: a
    // wave has work for both at any time.  HIDE: the next tile has keys that some rows must not see.
    template <bool HIDE, bool LAST>
    __device__ __forceinline__ void step(int stage, int t, Scores& cur, Scores& next, float& top) {
        follow(top);
        const char* vt = lds + stage * C::STAGE + C::KTILE;
        if constexpr (!LAST) scores<false>(stage ^ 1, next);
        exponentials(cur);
        product(vt, cur);
        if constexpr (!LAST) {
            if constexpr (HIDE) hide(next, (t + 1) * C::BN);
            top = largest(next);
            order<QK, KREADS, KREADS + AHEAD_V, PV, VREADS, 5 * KT * SN / 2, KT * SN, KT * SN>();
        }
    }
    // The same where the registers do not hold two tiles' scores: one tile after the other, and the other wave
    // of the SIMD fills the matrix cores meanwhile.  The order is written out, as the compiler's own gives up
    // the reads ahead when registers are short.
    template <bool HIDE>
    __device__ __forceinline__ void plain_step(int stage, int t, Scores& cur) {
        const char* vt = lds + stage * C::STAGE + C::KTILE;
        if constexpr (C::HALF) {
            static_assert(KT == 1 && C::SUB == 1, "one tile of 32 keys");
            constexpr int AK = 4, AV = 4, Z = SN / 8;
            const char* kt_ = lds + stage * C::STAGE + C::template row_at<C::KSTEP>(col);
            auto key = [&](int x) { return *reinterpret_cast<const u32x4*>(kt_ + (((C::NG * x + grp) ^ C::place_k(col)) * 16)); };
            auto query = [&](int x) { return x < C::CS - C::QL ? q[x] : *query_at(x); };
            u32x4 f[C::CS], g[C::CS], v[DT * Z];
#pragma unroll
            for (int x = 0; x < AK; ++x) f[x] = key(x), g[x] = query(x);
            cur[0][0] = Acc<M>{};
#pragma unroll
            for (int x = 0; x < C::CS; ++x) {
                if (x + AK < C::CS) f[x + AK] = key(x + AK), g[x + AK] = query(x + AK);
                __builtin_amdgcn_sched_barrier(0);
                multiply<T, M>(f[x], g[x], cur[0][0]);
            }
#pragma unroll
            for (int x = 0; x < AV; ++x) v[x] = values(vt, 0, x / DT, x % DT);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (HIDE) hide(cur, t * C::BN);
            follow(largest(cur));
            float sum = 0.0f;
            auto exponential = [&](int i) {
                cur[0][0][i] = __builtin_amdgcn_exp2f(fmaf(cur[0][0][i], c, -ref));
                sum += cur[0][0][i];
            };
#pragma unroll
            for (int i = 0; i < 8; ++i) exponential(i);
            u32x4 p = packed(cur, 0, 0);
#pragma unroll
            for (int x = 0; x < DT * Z; ++x) {
                if (x + AV < DT * Z) v[x + AV] = values(vt, 0, (x + AV) / DT, (x + AV) % DT);
                __builtin_amdgcn_sched_barrier(0);
                multiply<T, M>(v[x], p, o[x % DT]);
                if (x < 8 * (Z - 1)) exponential(8 + x);
                if (x % DT == DT - 1 && x + 1 < DT * Z) p = packed(cur, 0, x / DT + 1);
            }
            l += sum;
        } else {
            scores<false>(stage, cur);
            if constexpr (HIDE) hide(cur, t * C::BN);
            const float top = largest(cur);
            order<QK, KREADS, KREADS, 0, 0, 0, 0, 0>();
            follow(top);
            exponentials(cur);
            product(vt, cur);
            order<0, 0, 0, PV, VREADS, 0, 0, 5 * KT * SN / 2>();
        }
    }
    static constexpr int QK = KT * C::SUB * C::CS * (C::HALF ? 1 : 4), PV = KT * DT * (C::HALF ? SN / 8 : SN);  // matrix instructions
    static constexpr int KREADS = KT * (C::SUB * C::CS + C::QL), VREADS = KT * DT * (C::HALF ? SN / 4 : SN);           // LDS reads
    static constexpr int AHEAD_V = C::HALF ? 8 : 4;  // reads of values before the products with them begin
    // The order of a step's instructions: reads run ahead of the products that use them, and vector work stands
    // between the products.  M1, M2: products of either kind, with D1, D2 reads (E1 of them during the first kind) and
    // V1, X1 vector instructions and exponentials during the first kind, V2 vector ones during the second.
    template <int M1, int D1, int E1, int M2, int D2, int V1, int X1, int V2>
    static __device__ __forceinline__ void order() {
        constexpr int AHEAD = 4, FIRST = M1 > 0 ? AHEAD : AHEAD_V;
        __builtin_amdgcn_sched_group_barrier(0x100, FIRST, 0);
        if constexpr (M1 > 0) spread<M1, 0, E1 - FIRST, (E1 - FIRST + M1 - 1) / M1, V1, X1>();
        if constexpr (M2 > 0) spread<M2, 0, D1 + D2 - (M1 > 0 ? E1 : FIRST), (D2 + M2 - 1) / M2, V2, 0>();
    }
    // Products I .. M - 1, with `RATE` of the D reads each while there are any, and their even share of V vector
    // instructions and X exponentials.
    template <int M_, int I, int D, int RATE, int V, int X>
    static __device__ __forceinline__ void spread() {
        if constexpr (I < M_) {
            constexpr int done = I * RATE < D ? I * RATE : D, d = D - done < RATE ? D - done : RATE, v = V * (I + 1) / M_ - V * I / M_, x = X * (I + 1) / M_ - X * I / M_;
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if constexpr (d > 0) __builtin_amdgcn_sched_group_barrier(0x100, d, 0);
            if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x002, v, 0);
            if constexpr (x > 0) __builtin_amdgcn_sched_group_barrier(0x400, x, 0);
            spread<M_, I + 1, D, RATE, V, X>();
        }
    }

    // Tiles [t0, t1) of the run; those before `full` are seen whole by all rows of the block.  Values run a tile
    // ahead, keys two; the loads past the end are asked for with an empty range.
    // `stop` is asked once they are on their way.
    template <typename F>
    __device__ __forceinline__ bool run(const Keys& s, int t0, int t1, int full, F stop) {
        fresh_addresses();
        int stage = 0, t = t0;
        if constexpr (!C::PIPE) {
            Scores cur;
            load_tile(s, t0, true, 0);
            if (stop()) return false;
            auto one = [&](auto hidden, int at) {
                wait_and_meet<0>();
                load_tile(s, t + 1, t + 1 < t1, at ^ 1);
                if (hidden.value) look(lds + at * C::STAGE + C::KTILE, t * C::BN);
                plain_step<hidden.value>(at, t, cur);
                ++t;
            };
            while (t + 1 < min(full, t1)) {
                one(std::false_type{}, 0);
                one(std::false_type{}, 1);
            }
            for (; t < t1; stage ^= 1) one(std::true_type{}, stage);
        } else {
            Scores now, next;
            float top;
            load_half<false>(s, t0, true, 0);
            load_half<true>(s, t0, true, 0);
            load_half<false>(s, t0 + 1, t0 + 1 < t1, 1);
            if (stop()) return false;
            wait_and_meet<2 * C::JN>();
            scores<true>(0, now);
            if (t0 >= full) hide(now, t0 * C::BN);
            top = largest(now);
            auto ahead = [&](int at) {
                wait_and_meet<0>();
                load_half<true>(s, t + 1, t + 1 < t1, at ^ 1);
                load_half<false>(s, t + 2, t + 2 < t1, at);
            };
            while (t + 2 < min(full, t1 - 1)) {
                ahead(0);
                step<false, false>(0, t, now, next, top);
                ++t;
                ahead(1);
                step<false, false>(1, t, next, now, top);
                ++t;
            }
            for (; t < t1 - 1; ++t) {
                ahead(stage);
                if (t >= full) look(lds + stage * C::STAGE + C::KTILE, t * C::BN);
                step<true, false>(stage, t, now, next, top);
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int u = 0; u < C::SUB; ++u) now[k][u] = next[k][u];
                stage ^= 1;
            }
            wait_and_meet<0>();
            if (t >= full) look(lds + stage * C::STAGE + C::KTILE, t * C::BN);
            step<false, true>(stage, t, now, next, top);
        }
        wait_and_meet<0>();
        return true;
    }

    // The lanes of a row summed their own keys.
    __device__ __forceinline__ void sum_rows() { l = over_row<M, false>(l); }

    // Where rows' results go: their place in the list, and out or the workspace.
    struct To {
        int row0, rows;
        long long first;
        int hk;
        int set;          // >= 0: this set of the workspace
        long long slot;   // >= 0: this slot of the workspace
    };
    // Row r of them: the destination of its elements (fp32 sums, or the finished row), and its statistics there.
    struct Row {
        float* sums;
        TS* out;
        float inv;
    };
    __device__ __forceinline__ Row row_at(const To& to, int r, float m, float sum, bool stats) {
        const int i = r / a.G, h = to.hk * a.G + r - i * a.G;
        const long long token_row = (to.first + i) * a.c.H + h;
        Row y{nullptr, nullptr, 1.0f};
        if (to.slot >= 0 || to.set >= 0) {
            const long long at = to.slot >= 0 ? to.slot * C::BM + r : to.set * a.set_rows + token_row;
            y.sums = (to.slot >= 0 ? a.slot_o : a.set_o) + at * a.c.D;
            if (stats) (to.slot >= 0 ? a.slot_ml : a.set_ml)[at] = make_float2(m, sum);
        } else {
            y.out = static_cast<TS*>(a.c.out.p) + (to.first + i) * a.c.out.row + h * a.c.out.head;
            y.inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            if (stats && a.c.lse != nullptr)
                a.c.lse[token_row] = sum == 0.0f ? -INFINITY : kLn2 * (m + __builtin_amdgcn_logf(sum));
        }
        return y;
    }

    // The accumulators of the wave's rows, unless redo() is to follow: it reads the queries, which may be where the
    // results go.
    __device__ __forceinline__ void store(const To& to) {
        const int r = to.row0 + wave * M + col;
        if (r >= to.rows || spoiled) return;
        const Row y = row_at(to, r, ref, l, grp == 0);
        if (y.sums != nullptr) {
            float* p = y.sums + 4 * grp;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < C::EA / 4; ++i) {
                    const int e = M * d + 4 * C::NG * i;
                    if (e + 4 * grp < a.c.D)
                        *reinterpret_cast<f32x4*>(p + e) = f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
                }
        } else {
            TS* p = y.out + 4 * grp;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < C::EA / 4; ++i) {
                    const int e = M * d + 4 * C::NG * i;
                    if (e + 4 * grp >= a.c.D) continue;
                    const f32x4 x = f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]} * y.inv;
                    if constexpr (C::HALF) *reinterpret_cast<u32x2*>(p + e) = u32x2{pack<T>(x[0], x[1]), pack<T>(x[2], x[3])};
                    else *reinterpret_cast<f32x4*>(p + e) = x;
                }
        }
    }

    // The wave's rows again, plainly: one after the other, 64 keys at a time, over the keys p0 .. p1 - 1 of the prefix
    // and k0 .. k1 - 1 of the run (seen0 + token of them seen).  In place of store(): where out is q, a row's queries
    // are read before its result is written, and no other row's are written.
    __device__ __forceinline__ void redo(const To& to, const Keys& prefix, int p0, int p1, const Keys& own, int k0, int k1,
                                         int seen0) {
#pragma unroll 1
        for (int x0 = 0; x0 < M; ++x0) {
            const int r = to.row0 + wave * M + x0;
            if (r >= to.rows) break;
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
            const Row y = row_at(to, r, m, sum, lane == 0);
            for (int z = 0; z < 4; ++z) {
                const int e = lane + 64 * z;
                if (e >= a.c.D) break;
                if (y.sums != nullptr) y.sums[e] = x[z];
                else y.out[e] = from_f32<T>(x[z] * y.inv);
            }
        }
    }
};

__device__ __forceinline__ void report(const Args& a, bool malformed, unsigned block) {
    if (block == 0 && threadIdx.x == 0) {
        if (a.c.dev_status != nullptr) *a.c.dev_status = malformed ? GDN_ERR_OFFSETS : GDN_OK;
        if (a.status != nullptr) *a.status = malformed ? 1 : 0;
    }
}

// The long form: one block per key head, key part and tile of BM rows.  The row tiles of all sequences lie end to
// end (a few blocks find none and end), up to 64 sequences by their keys, those of a sequence from its last, which sees
// most keys.  Key heads are the fastest index, so the blocks that read one head's keys at a time lie on few XCDs.  With
// prefix_rows the rows are all tokens' and the keys the prefix alone.
template <typename C>
__device__ __forceinline__ void long_form(const Args& a, char* lds, const unsigned block, const bool prefix_rows) {
    unsigned x = block;
    const int hk = x % a.c.HK;
    x /= a.c.HK;
    const unsigned slots = prefix_rows ? (a.c.N * a.G + C::BM - 1) / C::BM : a.c.N * a.G / C::BM + a.c.B;
    // Four parts of a tile follow one another, so that blocks go from the longest down; parts that short sequences do
    // not have come last (512 tokens in a cache of 2^20 rows, 16 parts: 34 us, with all of a tile in a row 49).
    int part = 0;
    if (a.splits > 1) {
        const int four = x / (4 * slots), of = min(4, a.splits - 4 * four);
        x -= four * 4 * slots;
        part = 4 * four + x % of;
        x /= of;
    }
    int b = 0;
    unsigned back = x;  // tiles of the sequence behind this one
    if (!prefix_rows) {
        if (a.c.B <= 64) {
            back = by_keys<C::BM>(a.c, a.G, x, &b);
        } else {
            b = sequence_at<C::BM>(a.c, a.G, x);
            back = x - slot_of<C::BM>(a.c, a.G, uniform(entry(a.c.offsets, b)), b);
        }
    }
    // Queries and the first keys are on their way while the call is checked.
    const Sequence seq = prefix_rows ? Sequence{0, a.c.N, 0, 0} : sequence(a.c, b);
    const int first = seq.first, T = seq.T, n = seq.n;
    const long long begin = seq.begin;
    auto stop = [&] {
        const bool malformed = check<C::NT>(a.c);
        report(a, malformed, block);
        if (malformed) wait_and_meet<0>();
        return malformed;
    };
    const int rows = T * a.G, tiles = (rows + C::BM - 1) / C::BM;
    const int parts = min(a.splits, max(1, (int)(((unsigned)a.c.prefix_len + (unsigned)n) / kPartKeys)));
    if (back >= (unsigned)tiles || part >= parts) {
        if (block == 0) stop();  // the block that reports
        return;
    }
    const int row0 = (tiles - 1 - (int)back) * C::BM;
    const int seen0 = n - T + 1;
    const int last_token = min(row0 + C::BM, rows) - 1;
    const int reach = uniform(max(0, min(n, seen0 + last_token / a.G)));  // keys the last row sees
    const int ptiles = (a.c.prefix_len + C::BN - 1) / C::BN, all = ptiles + (reach + C::BN - 1) / C::BN;
    const int t0 = uniform((int)((long long)all * part / parts)), t1 = uniform((int)((long long)all * (part + 1) / parts));

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
        if (!blk.run(prefix, t0, p1, a.c.prefix_len / C::BN, stop)) return;
    }
    if (k0 < k1) {
        blk.see(row0, rows, true, seen0, n);
        blk.set_source(a.c.k.row, a.c.v.row);
        const int full = uniform(max(0, min(n, seen0 + row0 / a.G)) / C::BN);
        if (!blk.run(own, k0, k1, full, [&] { return t0 < p1 ? false : stop(); })) return;
    }
    if (t0 >= p1 && k0 >= k1 && stop()) return;  // no keys at all
    if (a.live != nullptr && part == 0 && hk == 0)
        for (int i = row0 / a.G + (int)threadIdx.x; i <= last_token / a.G; i += C::NT) a.live[first + i] = parts;
    blk.sum_rows();
    const typename Block<C>::To to{row0, rows, first, hk, a.to_sets ? part : -1, -1};
    blk.store(to);
    if (blk.spoiled)
        blk.redo(to, prefix, t0 * C::BN, min(p1 * C::BN, a.c.prefix_len), own, k0 * C::BN, max(0, min(k1 * C::BN, n)), seen0);
}

// The short form (a sequence's rows fit one tile): all (sequence, key head) runs laid end to end, counted
// in key tiles, and cut into equal parts, one a block.  A run inside one block is finished there; pieces of
// a cut run go to the workspace for the joining kernel.  Loads follow the part's tiles across the ends of
// runs, so a block's stream never dries up where a new run starts.
struct Run {
    int b, hk, first, T, n, tiles;  // the run
    int t0, t1;                     // this block's tiles of it
    long long begin;
};

template <typename C>
__device__ __forceinline__ void short_form(const Args& a, char* lds, const int w) {
    const int HK = a.c.HK;
    const Tiles<C::BN> all(a.c);
    auto tiles_of = [](int T, int n) { return Tiles<C::BN>::of(T, n); };
    const long long total = uniform(all.total) * HK;
    report(a, all.malformed, w);
    const int W = (int)min(total, (long long)a.workers);
    if (all.malformed || w >= W) {
        if (a.cut != nullptr && threadIdx.x == 0) a.cut[w] = make_int4(0, 0, 0, 0);
        return;
    }
    const Cut cut(total, W);
    long long u = uniform(cut.start(w));  // first unit of the consumer's run
    const long long u1 = uniform(cut.start(w + 1));
    Run ld;  // the run whose tiles are being asked for
    long long base;
    all.find(u >> 31 ? u / HK : (unsigned)u / (unsigned)HK, &ld.b, &base);
    ld.b = uniform(ld.b);
    base = uniform(base) * HK;
    auto open = [&] {
        ld.first = uniform(entry(a.c.offsets, ld.b));
        ld.T = uniform(entry(a.c.offsets, ld.b + 1)) - ld.first;
        ld.n = a.c.kv_len != nullptr ? uniform(entry(a.c.kv_len, ld.b)) : ld.T;
        ld.begin = a.c.kv_begin != nullptr ? uniform((long long)entry(a.c.kv_begin, ld.b)) : ld.first;
        ld.tiles = tiles_of(ld.T, ld.n);
    };
    open();
    Block<C> blk(a, lds);
    blk.set_source(a.c.k.row, a.c.v.row);
    const int q_at = C::NS * C::STAGE;

    int left = (int)(u1 - u);  // tiles not asked for yet
    const int within = (int)(u - base);
    ld.hk = uniform(within / ld.tiles);
    ld.t0 = within - ld.hk * ld.tiles;
    Keys keys;
    auto enter = [&] {  // the loads go on in run ld
        ld.t1 = min(ld.tiles, ld.t0 + left);
        keys = Keys{static_cast<const char*>(a.c.k.p) + (ld.begin * a.c.k.row + ld.hk * a.c.k.head) * C::ES,
                    static_cast<const char*>(a.c.v.p) + (ld.begin * a.c.v.row + ld.hk * a.c.v.head) * C::ES, ld.n};
        blk.ask_rows(q_at, ld.T, ld.first, ld.hk);
    };
    enter();
    Run run = ld;  // the run being computed; the loads are in it or in the next one
    bool crossed = false, fresh = true;  // fresh: the run's queries are still in LDS only
    int ask = ld.t0, ahead = 0, ask_stage = 0, stage = 0, t = run.t0;
    auto fill = [&] {
        while (ahead < C::NS - 1 && left > 0) {
            if (ask == ld.t1) {
                if (crossed || fresh) return;  // the queries' place in LDS holds one run's
                if (++ld.hk == HK) {
                    ld.hk = 0;
                    do {
                        ++ld.b;
                        open();
                    } while (ld.tiles == 0);
                }
                ld.t0 = ask = 0;
                enter();
                crossed = true;
            }
            blk.load_tile(keys, ask, true, ask_stage);
            ask_stage = ask_stage == C::NS - 1 ? 0 : ask_stage + 1;
            ++ask;
            ++ahead;
            --left;
        }
    };
    fill();
    while (true) {
        // the next tile (and what was asked for before it) is there; with the ring full, NS - 2 newer ones may
        // be on their way
        if (ahead == C::NS - 1) wait_and_meet<(C::NS - 2) * 2 * C::JN>();
        else wait_and_meet<0>();
        if (t == run.t1) {
            // Results are stored here, behind the wait, so that no later wait for tiles has to sit out the stores.
            blk.sum_rows();
            const int rows = run.T * a.G;
            const bool whole = run.t1 - run.t0 == run.tiles;
            // a worker's slot 0: a run cut at the front; slot 1: a run that starts here and goes on in the next worker
            const typename Block<C>::To to{0, rows, run.first, run.hk, whole && a.to_sets ? a.local_set : -1,
                                           whole ? -1 : w * 2ll + (run.t0 == 0 ? 1 : 0)};
            blk.store(to);
            if (blk.spoiled) {
                const Keys own{static_cast<const char*>(a.c.k.p) + (run.begin * a.c.k.row + run.hk * a.c.k.head) * C::ES,
                               static_cast<const char*>(a.c.v.p) + (run.begin * a.c.v.row + run.hk * a.c.v.head) * C::ES,
                               run.n};
                blk.redo(to, own, 0, 0, own, run.t0 * C::BN, min(run.t1 * C::BN, run.n), run.n - run.T + 1);
            }
            if (run.t0 == 0) {
                const int pieces = whole ? 1 : cut.part(u + run.tiles - 1) - w + 1;
                if (a.row_info != nullptr)
                    for (int i = threadIdx.x; i < run.T; i += C::NT)
                        a.row_info[(long long)(run.first + i) * HK + run.hk] = make_int2(whole ? -1 : w, pieces * 128 + i);
                if (!whole && a.cut != nullptr && threadIdx.x == 0) a.cut[w] = make_int4(run.first, run.T, run.hk, pieces);
            }
            u += run.t1 - run.t0;
            if (u >= u1) {
                if ((whole || run.t0 != 0) && a.cut != nullptr && threadIdx.x == 0) a.cut[w] = make_int4(0, 0, 0, 0);
                return;
            }
            run = ld;
            t = run.t0;
            crossed = false;
            fresh = true;
        }
        if (fresh) {
            blk.fresh_addresses();
            blk.see(0, run.T * a.G, true, run.n - run.T + 1, run.n);
            blk.take_rows(lds + q_at, run.T * a.G);
            wait_and_meet<63>();  // all waves have read the queries: their place may be written again
            fresh = false;
        }
        --ahead;
        fill();
        blk.use_tile(stage, t * C::BN);
        stage = stage == C::NS - 1 ? 0 : stage + 1;
        ++t;
    }
}

template <typename C>
__global__ __launch_bounds__(C::NT, C::WAVES) void long_kernel(Args a) {
    extern __shared__ __align__(1024) char lds[];
    long_form<C>(a, lds, blockIdx.x, a.prefix_blocks > 0);
}
template <typename C>
__global__ __launch_bounds__(C::NT, C::WAVES) void short_kernel(Args a) {
    extern __shared__ __align__(1024) char lds[];
    short_form<C>(a, lds, blockIdx.x);
}

// A small batch behind a shared prefix, in one launch: blocks of the long form over the prefix beside blocks of the
// short form over the sequences' own keys, so that neither waits for the other's launch and latency.  They take
// turns by as many blocks as there are CUs.
constexpr int kCUs = 256;
template <typename CL, typename CS>
__global__ __launch_bounds__(CL::NT, CL::WAVES) void both_kernel(Args a) {
    static_assert(CS::NT <= CL::NT, "a block of either form");
    extern __shared__ __align__(1024) char lds[];
    const int turn = blockIdx.x / kCUs, at = blockIdx.x % kCUs;
    const int pt = (int)((a.prefix_blocks + kCUs - 1) / kCUs), st = (a.workers + kCUs - 1) / kCUs, both = min(pt, st);
    const bool over_prefix = turn < 2 * both ? turn % 2 == 0 : pt > st;
    const int block = (turn < 2 * both ? turn / 2 : turn - both) * kCUs + at;
    if (over_prefix) {
        if (block < a.prefix_blocks) long_form<CL>(a, lds, block, true);
    } else {
        // the waves a block of the short form does not have end here; barriers wait for those that are left
        if (block < a.workers && threadIdx.x < CS::NT) short_form<CS>(a, lds, block);
    }
}

constexpr int kCULds = 160 * 1024;   // of a CU
constexpr int kMaxLds = 159 * 1024;  // of a block: less the kernels' own few words

// ---- which tile for which call -------------------------------------------------------------------
// Head widths are compiled for 64, 128 and 256.
//
// Short form, 16 x 16 tiles, one wave for every 16 rows (1, 2, 3, 4 or 8 waves).  What counts is bytes on their way:
// the ring is the deepest with which two blocks and all their rows' queries fit a CU, or where none does the deepest
// with which one does, of 4 stages at most.  That is 64 to 96 KB on their way a CU, and 32 KB with eight waves at
// 512-byte rows.  (64 sequences over 613 MB, 32 rows of D 256: 120 us, with one block a CU 137; 64 rows of D 128 over
// 1.2 GB: 257 and 342.)  A depth of 0: no such call, not even the fewest rows of so many waves fit beside two stages.
template <typename T, int DP, int WR>
struct Short {
    static constexpr int WIDTH = DP;
    static constexpr int RB = DP * (int)sizeof(typename T::storage);
    static constexpr int lds(int stages, int rows) { return stages * 64 * RB + rows * RB; }
    static constexpr int depth() {
        for (int blocks = 2; blocks >= 1; --blocks)
            for (int ns = 4; ns >= 2; --ns)
                if (lds(ns, 16 * WR) <= (blocks == 2 ? kCULds / 2 : kMaxLds)) return ns;
        constexpr int fewest = WR == 8 ? 65 : 16 * (WR - 1) + 1;
        return lds(2, (fewest + 7) / 8 * 8) <= kMaxLds ? 2 : 0;
    }
    static constexpr int NS = depth();
    using C = Cfg<T, 16, DP, WR, 1, NS, 1>;
};
// Long form, 32 x 32 tiles, four waves (eight at width 256 in half precision, where they share the queries' place).
template <typename T, int DP, int QL = 10>
struct Long {
    static constexpr int WIDTH = DP;
    static constexpr int RB = DP * (int)sizeof(typename T::storage);
    using C = Cfg<T, 32, DP, RB == 512 && sizeof(typename T::storage) == 2 ? 8 : 4, RB <= 256 ? 2 : 1, 2, RB <= 512 ? 2 : 1, QL>;
};

// What the host needs to know of a configuration: tile sizes, bytes of the ring and of a row in LDS, threads.
struct Shape {
    int bm, bn, ring, row, threads;
};
template <typename C>
constexpr Shape shape_of() {
    return Shape{C::BM, C::BN, C::LDS, C::RB, C::NT};
}


// dp 64, 128 or 256; wr 1, 2, 3, 4 or 8.  `none` where there is no short form of so many rows.
template <typename T, int DP, typename R, typename F>
R with_waves(int wr, R none, F f) {
    auto go = [&](auto s) -> R {
        if constexpr (decltype(s)::NS > 0) return f(s);
        else return none;
    };
    switch (wr) {
        case 1: return go(Short<T, DP, 1>{});
        case 2: return go(Short<T, DP, 2>{});
        case 3: return go(Short<T, DP, 3>{});
        case 4: return go(Short<T, DP, 4>{});
        default: return go(Short<T, DP, 8>{});
    }
}
template <typename T, typename R, typename F>
R with_short(int dp, int wr, R none, F f) {
    return dp == 64 ? with_waves<T, 64>(wr, none, f) : dp == 128 ? with_waves<T, 128>(wr, none, f) : with_waves<T, 256>(wr, none, f);
}
template <typename T, typename F>
auto with_long(int dp, F f) {
    return dp == 64 ? f(Long<T, 64>{}) : dp == 128 ? f(Long<T, 128>{}) : f(Long<T, 256>{});
}

// Both forms in one launch: for the widths and waves whose blocks of either form fit a CU twice.
constexpr bool joint(int ring_long, int lds_short) { return std::max(ring_long, lds_short) <= 80 * 1024 - 512; }

// One translation unit per type holds its kernels.
template <typename T>
hipError_t start_short(const Args& a, int dp, int wr, long long blocks, int lds, hipStream_t stream);
template <typename T>
hipError_t start_long(const Args& a, int dp, long long blocks, int lds, hipStream_t stream);
template <typename T>
hipError_t start_both(const Args& a, int dp, int wr, long long blocks, int lds, hipStream_t stream);

// `asked`: the devices on which the kernel may have more than 64 KB of LDS already.
template <typename F, typename A>
hipError_t start_kernel(F* f, std::atomic<uint64_t>& asked, const A& a, long long blocks, int threads, int lds,
                        hipStream_t stream) {
    if (blocks * threads > kMaxThreads || lds > kMaxLds) return hipErrorInvalidConfiguration;
    if (lds > 64 * 1024) {
        int dev = 0;
        hipError_t e = hipGetDevice(&dev);
        const uint64_t bit = 1ull << (dev & 63);
        if (e == hipSuccess && (dev > 63 || !(asked.load(std::memory_order_relaxed) & bit))) {
            e = hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLds);
            if (e == hipSuccess) asked.fetch_or(bit, std::memory_order_relaxed);
        }
        if (e != hipSuccess) return e;
    }
    f<<<(unsigned)blocks, threads, lds, stream>>>(a);
    return hipGetLastError();
}
template <typename C>
hipError_t start_one_long(const Args& a, long long blocks, int lds, hipStream_t stream) {
    static std::atomic<uint64_t> asked{0};
    return start_kernel(&long_kernel<C>, asked, a, blocks, C::NT, lds, stream);
}
template <typename C>
hipError_t start_one_short(const Args& a, long long blocks, int lds, hipStream_t stream) {
    static std::atomic<uint64_t> asked{0};
    return start_kernel(&short_kernel<C>, asked, a, blocks, C::NT, lds, stream);
}
template <typename CL, typename CS>
hipError_t start_one_both(const Args& a, long long blocks, int lds, hipStream_t stream) {
    if constexpr (CS::NT <= CL::NT && joint(CL::LDS, CS::LDS)) {
        static std::atomic<uint64_t> asked{0};
        return start_kernel(&both_kernel<CL, CS>, asked, a, blocks, CL::NT, lds, stream);
    } else {
        return hipErrorInvalidConfiguration;
    }
}

#define GDN_ATTN_INSTANCES(T)                                                                                           \
    template <>                                                                                                         \
    hipError_t start_short<T>(const Args& a, int dp, int wr, long long blocks, int lds, hipStream_t stream) {           \
        return with_short<T>(dp, wr, hipErrorInvalidConfiguration, [&](auto p) { return start_one_short<typename decltype(p)::C>(a, blocks, lds, stream); }); \
    }                                                                                                                   \
    template <>                                                                                                         \
    hipError_t start_long<T>(const Args& a, int dp, long long blocks, int lds, hipStream_t stream) {                    \
        return with_long<T>(dp, [&](auto p) { return start_one_long<typename decltype(p)::C>(a, blocks, lds, stream); }); \
    }                                                                                                                   \
    template <>                                                                                                         \
    hipError_t start_both<T>(const Args& a, int dp, int wr, long long blocks, int lds, hipStream_t stream) {            \
        return with_long<T>(dp, [&](auto l) {                                                                           \
            return with_short<T>(dp, wr, hipErrorInvalidConfiguration, [&](auto p) {                                                                  \
                using L = decltype(l);                                                                                  \
                using P = decltype(p);                                                                                  \
                if constexpr (L::WIDTH == P::WIDTH) return start_one_both<typename L::C, typename P::C>(a, blocks, lds, stream); \
                else return hipErrorInvalidConfiguration;                                                               \
            });                                                                                                         \
        });                                                                                                             \
    }

}  // namespace attn
}  // namespace gdn
