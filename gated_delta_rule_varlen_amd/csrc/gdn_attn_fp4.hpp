// gdn_attn_fp4.hpp -- the kernels of the attention over a 4-bit cache (instances per type in gdn_attn_fp4_<type>.hip, host
// side in gdn_attn_fp4.hip).  Rows, products and softmax are those of gdn_attn.hpp.
//
// Short form (decode and drafts, up to 64 rows a sequence and key head): bound by the cache's bytes.  Codes and scales
// reach LDS by asynchronous loads and become matrix operands in registers, two elements an instruction, the block's
// power of two included.  A lane reads its part of a key, a block of 32 elements or half of one; a contraction may run in
// any order, so these are taken eight a step and the queries are held in the same order.  Values are needed key by key for one
// element of the head: a lane reads the same few elements of eight keys, widens them, and swaps halves of registers between
// two keys.
//
// A block's four waves take 32 keys each of every 128, each with places of its own in LDS and nothing shared until a run's
// end, where their sums are joined.  Scales are asked for two tiles at a time, as a tile's are half a load.  All runs lie
// end to end and are cut into equal parts, one a block, as in the short form there.
//
// Measured (bf16; the floor is the bytes at a 1 GiB copy's 5.2 TB/s): 256 sequences of up to 4096 keys (H 32, HK 8, D 128,
// 604 MB) 122 to 128 us of 116: its loads alone take 114.5, its work without them 90, the joining launch 5.  One token over 131072
// keys (HK 2, D 256, 71 MB) 24 to 25 of 13.7: 19 and the joining launch's 6.  Drafts of five tokens over 1000 to 8000 keys
// (64 sequences, D 256, 167 MB) 73 to 75 of 32: bound by the products and the vector work of 40 rows (matrix
// instructions busy 23% of cycles, vector ones 53%).  Tried: codes to registers without LDS 152 us on the first of
// these; loads that leave the caches as they are, without the hint, 138; a barrier a tile, no gain.
//
// fp32 takes 150 us for a batch like the first of these (floor 125, bf16 123), 52 for single tokens over 1000 to 8000 keys at D 256
// (floor 31, bf16 41) and 171 for the drafts (33, 74): every product is made three times, and the kernels for one tile of
// rows at width 256 and four at 128 spill 7 to 17 vector registers.
//
// Long form (prompts): see Long4.  24748 tokens over up to 7100 keys (H 32, HK 8, D 128) 1309 to 1446 us by card (1309 on one),
// 0.93 to 1.03 PFLOP/s of the 1.34 that a large library product reaches: matrix instructions are busy 46% of cycles, the rest
// is the vector work of the softmax and the widening (6.3 vector instructions for one of theirs), and power holds the clock.
// That kernel spills 6 vector registers, those of fp32 at widths 128 and 256 8 and 21.
#pragma once

#include "gdn_attn.hpp"
#include "gdn_fp4.hpp"

namespace gdn {
namespace attn {

struct Fp4Args {
    Args a;
    Fp4Cache cache;
    int share;           // of the call's key heads as the kernels see them, so many in a row are one of the cache's
    uint32_t g_inverse;  // floor(2^16 / G) + 1: r * g_inverse >> 16 is r / G for the short form's rows, as r * G < 2^16
};

// The kernel's argument, read again: what a loop does not need is not worth scalar registers across it.  With all of it held
// 130 of them were spilled and read back in the loop; 68 to 165 still are in the kernels that go over pieces, the more the
// wider the rows, but most come back once a piece.
__device__ __forceinline__ const Fp4Args& args_again() {
    auto p = (const __attribute__((address_space(4))) Fp4Args*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const Fp4Args*)p;
}

// One run of a head's cache rows.
struct Fp4Keys {
    const char *kc, *ks, *vc, *vs;
};
__device__ __forceinline__ Fp4Keys fp4_keys(const Fp4Cache& c, long long begin, int hk) {
    const auto at = [&](const HeadRows& x) { return static_cast<const char*>(x.p) + begin * x.row + hk * x.head; };
    return Fp4Keys{at(c.k.codes), at(c.k.scales), at(c.v.codes), at(c.v.scales)};
}

// Two elements' values as matrix operands of type OP.
template <typename OP>
__device__ __forceinline__ uint32_t widen2(uint32_t codes, float scale, int pair) {
    // the pair is part of the instruction
    switch (pair) {
#define GDN_PAIR(p)                                                                                                    \
    case p:                                                                                                            \
        if constexpr (OP::code == GDN_BF16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, p)); \
        else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, p));
        GDN_PAIR(0)
        GDN_PAIR(1)
        GDN_PAIR(2)
        default: GDN_PAIR(3)
#undef GDN_PAIR
    }
}

// Eight elements' values as the products have them: rounded to fp16 (to an infinity past its range) with fp16 queries,
// so that a row that is done again has the values it had; otherwise exact.
template <typename T>
__device__ __forceinline__ void operand_values(uint32_t codes, uint32_t scale_byte, float* y) {
    if constexpr (T::code == GDN_F16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = widen2<F16>(codes, fp4::scale_of(scale_byte), i);
            y[2 * i] = to_f32<F16>((uint16_t)w);
            y[2 * i + 1] = to_f32<F16>((uint16_t)(w >> 16));
        }
    } else {
        fp4::values(codes, scale_byte, y);
    }
}

// Row q over the keys j0 .. j1 - 1 plainly, by a wave: the largest score to base 2, the sum of exponentials and, four
// elements a lane (4 * lane ..), their products with the values.
struct RowSums {
    float m, sum;
    f32x4 o;
};
template <typename T>
__device__ __forceinline__ RowSums plain_row(const typename T::storage* q, const Fp4Keys& s, const Fp4Cache& c, int D, float s2,
                                             int j0, int j1) {
    const int lane = threadIdx.x & 63;
    RowSums r{kNoMax, 0.0f, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll 1
    for (; j0 < j1; j0 += 64) {
        float y = -INFINITY;
        if (j0 + lane < j1) {
            const char* codes = s.kc + (j0 + lane) * c.k.codes.row;
            const uint8_t* scales = reinterpret_cast<const uint8_t*>(s.ks + (j0 + lane) * c.k.scales.row);
            y = 0.0f;
#pragma unroll 1
            for (int x = 0; x < D / 8; ++x) {
                float k[8];
                operand_values<T>(reinterpret_cast<const uint32_t*>(codes)[x], scales[x / 4], k);
#pragma unroll
                for (int e = 0; e < 8; ++e) y = fmaf(to_f32<T>(q[8 * x + e]), k[e], y);
            }
            y *= s2;
        }
        float top = y;
        for (int z = 1; z < 64; z <<= 1) top = fmaxf(top, __shfl_xor(top, z));
        const float to = fmaxf(r.m, top), w = __builtin_amdgcn_exp2f(r.m - to), p = __builtin_amdgcn_exp2f(y - to);
        r.sum = r.sum * w + group_sum<64>(p);
        r.m = to;
        r.o *= w;
#pragma unroll 1
        for (int j = 0; j < min(64, j1 - j0); ++j) {
            const float pj = __shfl(p, j);
            if (4 * lane >= D) continue;
            float v[8];
            operand_values<T>(*reinterpret_cast<const uint16_t*>(s.vc + (j0 + j) * c.v.codes.row + 2 * lane),
                              *reinterpret_cast<const uint8_t*>(s.vs + (j0 + j) * c.v.scales.row + lane / 8), v);
#pragma unroll
            for (int e = 0; e < 4; ++e) r.o[e] = fmaf(pj, v[e], r.o[e]);
        }
    }
    return r;
}

// T: the type of queries and outputs.  fp16 has operands in fp16, the others in bf16, where an fp32 query or probability is
// the sum of three parts: their products with the cache's values, which are exact in bf16, are exact as well.
// WIDE: a head's scales are read as many as fit 32 bits at a time, otherwise byte by byte.
// KW x RG waves: of every 32 KW keys a wave takes 32, and of the rows the RT tiles of its group; the groups of a
// wave's keys share their places in LDS, and one asks for the keys, the other for the values.
template <typename T_, int DP_, int RT_, int KW_, int RG_, int WAVES_, bool WIDE_>
struct Cfg4 {
    using T = T_;
    using TS = typename T::storage;
    using OP = std::conditional_t<T::code == GDN_F16, F16, BF16>;
    static constexpr int DP = DP_, RT = RT_, KW = KW_, RG = RG_, WAVES = WAVES_;  // WAVES: of a SIMD
    static constexpr bool WIDE = WIDE_;
    static constexpr int PARTS = T::code == GDN_F32 ? 3 : 1;
    static constexpr int W = KW * RG, NT = 64 * W, BN = 32, UNIT = BN * KW, BM = 16 * RT * RG, NS = 2;
    static constexpr int CL = DP / 4 < 32 ? DP / 4 : 32;  // neighbouring elements a lane holds of a key
    static constexpr int KH = DP / (4 * CL);              // such pieces of a key
    static constexpr int STEPS = DP / 32, SPP = CL / 8;   // operand steps, and of a piece
    static constexpr int VD = DP / 16;                    // neighbouring elements a lane holds of a value
    static constexpr int NB = DP / 32, RB = DP / 2;       // blocks and bytes of codes of a row
    static constexpr int SB = WIDE ? (NB < 4 ? NB : 4) : 1, SLOTS = NB / SB;  // scales of a 32-bit place in LDS, places of a row
    static constexpr int CODES = BN * RB, CN = CODES / 1024, RPL = 1024 / RB; // bytes, loads, rows a load
    static constexpr int SN = SLOTS, SCALES = 256 * SN;   // loads of the scales of two tiles, and their bytes in LDS
    static constexpr int STAGE = 2 * (CODES + SCALES);    // of a wave's keys: a tile's codes, and the scales of two
    static constexpr int CODE_LOADS = 2 * CN / RG, SCALE_LOADS = 2 * SN / RG;  // of a wave
    static constexpr bool QLDS = RT * RG > 1;             // queries in LDS: read once for two products
    static constexpr int PLACES = NS * KW * STAGE, QBYTES = QLDS ? RG * RT * PARTS * STEPS * 1024 : 0;
    static constexpr int ROW = DP + 4;                    // fp32 sums of a row in LDS
    static constexpr int STATS = KW * 16 * 8 + W * 4;     // the waves' maxima and sums of a tile's rows, and who met NaN
    static constexpr int LDS = PLACES + QBYTES + STATS;
    static_assert(RG <= 2 && 16 * ROW * 4 <= NS * STAGE, "the waves' sums take the tiles' place");
    // Rows whose sums fit the second half, while the next piece's first tile is on its way to the first.
    static constexpr int EARLY = RT * RG == 1 ? STAGE / (ROW * 4) : 0;
    // The largest scale byte of which every value is a finite operand: 6 * 2^13 in fp16, 6 * 2^125 in bf16.
    static constexpr int FINITE = OP::code == GDN_F16 ? 127 + 13 : 127 + 125;
    static constexpr float BIAS = T::code == GDN_F16 ? 4.0f : 0.0f, LAG = 8.0f;
    // Codes in LDS: 16-byte pieces (a block each) of key r at place piece ^ place_k(r), so that the 16 rows that are read
    // at a time lie in different banks; values in the order of row_of, so that four groups' rows are neighbours.
    static __device__ __forceinline__ int place_k(int r) { return DP == 64 ? (r >> 3) & 1 : DP == 128 ? (r >> 2) & 3 : (r >> 1) & 7; }
    static __device__ __forceinline__ int row_of(int place) { return (place & 16) + (place & 3) * 4 + ((place >> 2) & 3); }
};

// The parts of two fp32 numbers as operands.
template <typename OP, int PARTS>
__device__ __forceinline__ void split2(float x, float y, uint32_t* to, int step) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        const uint32_t w = pack<OP>(x, y);
        to[i * step] = w;
        if (i + 1 < PARTS) {
            x -= __uint_as_float(w << 16);
            y -= __uint_as_float(w & 0xffff0000u);
        }
    }
}

// A number whose exponent is the byte at `at` of x, as the conversions look at nothing else of a scale: sign and fraction are
// bits of its neighbours.
__device__ __forceinline__ float scale_at(uint32_t x, uint32_t at) {
    return __uint_as_float(__builtin_amdgcn_alignbit(x, x, 8 * at + 9));
}

// 64 x BYTES to LDS, 32 bits a lane (zeros above) for fewer than 16 bytes, as load_to_lds of gdn_attn.hpp.
template <int BYTES>
__device__ __forceinline__ void stream_to_lds(u32x4 s, uint32_t at, int voff, int soff) {
    static_assert(BYTES == 1 || BYTES == 2 || BYTES == 4 || BYTES == 16, "bytes");
#define GDN_LOAD(op) asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\t" op " %1, %2, %3 offen nt lds" ::"s"(at), "v"(voff), "s"(s), "s"(soff) : "m0", "memory")
    if constexpr (BYTES == 16) GDN_LOAD("buffer_load_dwordx4");
    else if constexpr (BYTES == 4) GDN_LOAD("buffer_load_dword");
    else if constexpr (BYTES == 2) GDN_LOAD("buffer_load_ushort");
    else GDN_LOAD("buffer_load_ubyte");
#undef GDN_LOAD
}

template <typename C>
struct Short4 {
    using T = typename C::T;
    using TS = typename C::TS;
    using OP = typename C::OP;
    static constexpr int RT = C::RT, PARTS = C::PARTS, KH = C::KH, VD = C::VD, CN = C::CN, SN = C::SN;
    static constexpr int KO = C::RPL < 16 ? 2 : 1;  // loads after which the places of a key's pieces repeat

    char* lds;
    uint32_t lds_at;    // its LDS address
    int lane, wave, keys_of, rows_of, col, grp;  // keys_of, rows_of: the wave's part of the keys and of the rows
    int kc_off[KO], vc_off, ks_off[SN], vs_off[SN];  // byte offsets of what the lane loads of a tile
    int krow, vrow;                              // bytes between rows of codes
    uint32_t q[C::QLDS ? 1 : PARTS][C::QLDS ? 1 : C::STEPS][4];
    Acc<16> o[RT][VD];
    float ref[RT], l[RT], c;
    int vis[RT], vis_lo;
    bool spoiled;

    // One tensor of the run, from the wave's next tile on.
    struct Stream {
        u32x4 r;
        int step, tail;  // bytes to the next tile (or two), and of the rows where the run ends
        __device__ __forceinline__ void open(const HeadRows& x, long long row, int hk, int tiles, int full, int rows, int width) {
            const uint64_t at = (uint64_t)uniform((long long)(reinterpret_cast<uint64_t>(x.p) + row * x.row + hk * x.head));
            const int stride = (int)x.row;
            r = u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, (uint32_t)uniform((full - 1) * stride + width), (uint32_t)kRsrc};
            step = uniform(tiles * C::UNIT * stride);
            tail = uniform(rows > 0 ? (rows - 1) * stride + width : 0);
        }
        __device__ __forceinline__ void advance() {
            const uint64_t at = ((uint64_t)r[1] << 32 | r[0]) + (uint32_t)step;
            r[0] = (uint32_t)at;
            r[1] = (uint32_t)(at >> 32);
        }
    };
    Stream kc, ks, vc, vs;
    int left;  // rows of the run from the next tile on

    __device__ __forceinline__ explicit Short4(char* lds_) : lds(lds_) {
        const Fp4Args& f = args_again();
        lane = threadIdx.x & 63;
        wave = uniform((int)threadIdx.x >> 6);
        keys_of = C::RG == 1 ? wave : wave % C::KW;
        rows_of = C::RG == 1 ? 0 : wave / C::KW;
        col = lane & 15;
        grp = lane >> 4;
        c = f.a.s2;
        krow = (int)f.cache.k.codes.row;
        vrow = (int)f.cache.v.codes.row;
        lds_at = uniform((int)(uintptr_t)(__attribute__((address_space(3))) char*)lds);
        const int D = f.a.c.D, in_load = lane / C::NB, piece = lane % C::NB;
#pragma unroll
        for (int j = 0; j < KO; ++j) {
            const int kp = piece ^ C::place_k(j * C::RPL + in_load);
            kc_off[j] = kp * 32 < D ? in_load * krow + kp * 16 : kOutside;
        }
        vc_off = piece * 32 < D ? C::row_of(in_load) * vrow + piece * 16 : kOutside;
#pragma unroll
        for (int j = 0; j < SN; ++j) {
            const int x = j * 64 + lane, row = x / C::SLOTS % C::BN, slot = x % C::SLOTS, later = x / (C::SLOTS * C::BN) * C::UNIT;
            const bool in = slot * C::SB * 32 < D;
            ks_off[j] = in ? (later + row) * (int)f.cache.k.scales.row + slot * C::SB : kOutside;
            vs_off[j] = in ? (later + C::row_of(row)) * (int)f.cache.v.scales.row + slot * C::SB : kOutside;
        }
    }
    // Places in LDS: two halves, each the codes of a tile for every wave's keys and behind them the scales of two tiles.
    static __device__ __forceinline__ int codes_at(int half, int keys) { return half * C::KW * C::STAGE + keys * 2 * C::CODES; }
    static __device__ __forceinline__ int scales_at(int half, int keys) {
        return half * C::KW * C::STAGE + C::KW * 2 * C::CODES + keys * 2 * C::SCALES;
    }

    // The wave's tile of every unit from t0 on, of a run of n rows that begins at `begin`; nothing from unit t1 on.
    __device__ __forceinline__ void open(const Fp4Args& f, long long begin, int hk, int t0, int t1, int n) {
        const int j0 = t0 * C::UNIT + keys_of * C::BN, D = f.a.c.D;
        if (f.share > 1) hk /= f.share;
        left = uniform(min(n, t1 * C::UNIT) - j0);
        const int tail = left & (C::BN - 1);  // of the one tile that may be shorter, if it is this wave's
        kc.open(f.cache.k.codes, begin + j0, hk, 1, C::BN, tail, D / 2);
        vc.open(f.cache.v.codes, begin + j0, hk, 1, C::BN, tail, D / 2);
        // of two tiles: until the run's end where that is nearer
        const int end = left & (2 * C::UNIT - 1);
        ks.open(f.cache.k.scales, begin + j0, hk, 2, C::UNIT + C::BN, end, D / 32);
        vs.open(f.cache.v.scales, begin + j0, hk, 2, C::UNIT + C::BN, end, D / 32);
    }
    // Asks for the scales of the next two tiles.  Who read these places before is done: the wait is for its reads.
    __device__ __forceinline__ void ask_scales(int half) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (left < C::UNIT + C::BN) {
            ks.r[2] = left > 0 ? ks.tail : 0;
            vs.r[2] = left > 0 ? vs.tail : 0;
        }
        const uint32_t to = lds_at + scales_at(half, keys_of);
        if (C::RG == 1 || rows_of == 0) {
#pragma unroll
            for (int j = 0; j < SN; ++j) stream_to_lds<C::SB>(ks.r, to + j * 256, ks_off[j], 0);
            ks.advance();
        }
        if (C::RG == 1 || rows_of == 1) {
#pragma unroll
            for (int j = 0; j < SN; ++j) stream_to_lds<C::SB>(vs.r, to + C::SCALES + j * 256, vs_off[j], 0);
            vs.advance();
        }
    }
    // Asks for the codes of the next tile.
    __device__ __forceinline__ void ask_codes(int half) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (left < C::BN) {
            kc.r[2] = left > 0 ? kc.tail : 0;
            vc.r[2] = left > 0 ? vc.tail : 0;
        }
        const uint32_t to = lds_at + codes_at(half, keys_of);
        if (C::RG == 1 || rows_of == 0) {
#pragma unroll
            for (int j = 0; j < CN; ++j) stream_to_lds<16>(kc.r, to + j * 1024, kc_off[j % KO], j * C::RPL * krow);
            kc.advance();
        }
        if (C::RG == 1 || rows_of == 1) {
#pragma unroll
            for (int j = 0; j < CN; ++j) {
                // rows of 16 lie one behind the other in eights: places 8 .. 15 are two rows further
                const int rows = C::RPL >= 16 ? j * C::RPL : j / 2 * 16 + j % 2 * 2;
                stream_to_lds<16>(vc.r, to + C::CODES + j * 1024, vc_off, rows * vrow);
            }
            vc.advance();
        }
        left -= C::UNIT;
    }
    // The first tile of a piece.
    __device__ __forceinline__ void ask_first() {
        ask_scales(0);
        ask_codes(0);
    }

    // The queries of the sequence's rows, eight elements a step in the order of the keys' pieces; in LDS each wave
    // leaves a part of them.
    __device__ __forceinline__ void take_rows(const Fp4Args& f, int rows, long long first, int hk) {
        const Args& a = f.a;
        const int G = a.G;
        const uint32_t flip = a.negate ? 0x80008000u : 0u;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int r = 16 * (rows_of * RT + rt) + col, i = (int)(r * f.g_inverse >> 16), g = r - i * G;
            const bool in = r < rows;
            const TS* p = static_cast<const TS*>(a.c.q.p) + (first + (in ? i : 0)) * a.c.q.row + (long long)(hk * G + (in ? g : 0)) * a.c.q.head;
#pragma unroll
            for (int s = 0; s < C::STEPS; ++s) {
                if (C::QLDS && (rt * C::STEPS + s) % C::KW != keys_of) continue;
                const int e = s / C::SPP * 128 + C::CL * grp + s % C::SPP * 8;
                const bool real = in && e < a.c.D;
                const TS* at = p + (real ? e : 0);
                uint32_t w[PARTS][4];
                if constexpr (PARTS == 1) {
                    const u32x4 x = *reinterpret_cast<const u32x4*>(at);
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[0][j] = x[j];
                } else {
                    const f32x4 x = reinterpret_cast<const f32x4*>(at)[0], y = reinterpret_cast<const f32x4*>(at)[1];
                    const float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
                    for (int j = 0; j < 4; ++j) split2<OP, PARTS>(v[2 * j], v[2 * j + 1], &w[0][j], 4);
                }
#pragma unroll
                for (int z = 0; z < PARTS; ++z) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[z][j] = real ? w[z][j] ^ flip : 0u;
                    if constexpr (C::QLDS) {
                        *query_at(rt, z, s) = vec(w[z]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) q[z][s][j] = w[z][j];
                    }
                }
            }
            ref[rt] = kNoMax;
            l[rt] = 0.0f;
#pragma unroll
            for (int y = 0; y < VD; ++y) o[rt][y] = Acc<16>{};
        }
        spoiled = false;
    }
    __device__ __forceinline__ u32x4* query_at(int rt, int part, int step) const {
        return reinterpret_cast<u32x4*>(lds + C::PLACES + (((rows_of * RT + rt) * PARTS + part) * C::STEPS + step) * 1024 + lane * 16);
    }
    // The keys each row sees: seen0 + its token, at least 0; the last token sees all n.
    __device__ __forceinline__ void see(const Fp4Args& f, int rows, int seen0, int n) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int r = 16 * (rows_of * RT + rt) + col;
            vis[rt] = r < rows ? max(seen0 + (int)(r * f.g_inverse >> 16), 0) : n;
        }
        vis_lo = uniform(max(seen0, 0));
    }

    static __device__ __forceinline__ u32x4 vec(const uint32_t* x) { return u32x4{x[0], x[1], x[2], x[3]}; }

    // The tile of the half `codes`, with the first or second scales of the half `scales`: keys j0 .. j0 + 31 of a run of n,
    // against the first ACT tiles of the wave's rows.
    template <int ACT>
    __device__ __forceinline__ void use(int codes, int scales, int second, int j0, int n) {
        if (ACT == 0 || j0 >= n) return;
        const char* kt = lds + codes_at(codes, keys_of);
        const char* vt = kt + C::CODES;
        const uint32_t* kst = reinterpret_cast<const uint32_t*>(lds + scales_at(scales, keys_of)) + second * C::BN * C::SLOTS;
        const uint32_t* vst = kst + C::SCALES / 4;
        Acc<16> s[ACT + 1][2];
#pragma unroll
        for (int rt = 0; rt < ACT; ++rt) s[rt][0] = s[rt][1] = Acc<16>{};
#pragma unroll
        for (int h = 0; h < KH; ++h) {
            uint32_t k[2][C::CL / 8];
            float scale[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int row = 16 * u + col, block = C::CL == 32 ? grp + 4 * h : grp / 2;
                const char* at = kt + row * C::RB + ((block ^ C::place_k(row)) * 16);
                if constexpr (C::CL == 32) {
                    const u32x4 x = *reinterpret_cast<const u32x4*>(at);
#pragma unroll
                    for (int i = 0; i < 4; ++i) k[u][i] = x[i];
                } else {
                    const u32x2 x = *reinterpret_cast<const u32x2*>(at + (grp & 1) * 8);
                    k[u][0] = x[0], k[u][1] = x[1];
                }
                scale[u] = scale_at(kst[row * C::SLOTS + block / C::SB], block % C::SB);
            }
#pragma unroll
            for (int x = 0; x < C::SPP; ++x) {
                uint32_t w[2][4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int u = 0; u < 2; ++u) w[u][j] = widen2<OP>(k[u][x], scale[u], j);
#pragma unroll
                for (int rt = 0; rt < ACT; ++rt)
#pragma unroll
                    for (int z = PARTS - 1; z >= 0; --z) {
                        u32x4 y;
                        if constexpr (C::QLDS) y = *query_at(rt, z, h * C::SPP + x);
                        else y = vec(q[z][h * C::SPP + x]);
#pragma unroll
                        for (int u = 0; u < 2; ++u) multiply<OP, 16>(vec(w[u]), y, s[rt][u]);
                    }
            }
        }
        const bool masked = j0 + C::BN > vis_lo;
        if (masked) {
#pragma unroll
            for (int rt = 0; rt < ACT; ++rt) {
                const int room = vis[rt] - j0 - 4 * grp;
#pragma unroll
                for (int i = 0; i < 8; ++i) s[rt][i / 4][i % 4] = 16 * (i / 4) + i % 4 >= room ? -INFINITY : s[rt][i / 4][i % 4];
            }
            asm volatile("");  // keeps this a branch: most tiles hide nothing
        }
        uint32_t p[ACT + 1][PARTS][4];
#pragma unroll
        for (int rt = 0; rt < ACT; ++rt) {
            float top = s[rt][0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, s[rt][i / 4][i % 4]);
            top = over_row<16, true>(top) * c;
            if (__builtin_amdgcn_ballot_w64(top > ref[rt] + (C::BIAS + C::LAG)) != 0) {
                const float to = fmaxf(ref[rt], top - C::BIAS), w = __builtin_amdgcn_exp2f(ref[rt] - to);
                ref[rt] = to;
                l[rt] *= w;
#pragma unroll
                for (int y = 0; y < VD; ++y) o[rt][y] *= w;
            }
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                e[i] = __builtin_amdgcn_exp2f(fmaf(s[rt][i / 4][i % 4], c, -ref[rt]));
                l[rt] += e[i];
            }
            // Operands of the second product: in the half types one part, rounded to the type, as over a plain cache.  The rounding
            // is half a step of a probability, as the output's own is of the output; a second part would double the products.
            // The sum is of the unrounded ones.
#pragma unroll
            for (int i = 0; i < 4; ++i) split2<OP, PARTS>(e[2 * i], e[2 * i + 1], &p[rt][0][i], 4);
        }
        // Places 4 x + grp hold the lane's keys: 4 grp + x of the first 16 for x < 4, 4 grp + x - 4 of the second behind them.
        const int block = col * VD / 32;
        float scale[8];
        uint32_t v[8][VD > 8 ? 2 : 1];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int place = 4 * x;
            const char* at = vt + grp * C::RB + col * (C::RB / 16) + place * C::RB;
            if constexpr (VD == 4) v[x][0] = *reinterpret_cast<const uint16_t*>(at);
            else if constexpr (VD == 8) v[x][0] = *reinterpret_cast<const uint32_t*>(at);
            else {
                const u32x2 y = *reinterpret_cast<const u32x2*>(at);
                v[x][0] = y[0], v[x][1] = y[1];
            }
            scale[x] = scale_at(vst[(place + grp) * C::SLOTS + block / C::SB], block % C::SB);
        }
        // 0 times NaN or an infinity is NaN: where rows differ in what they see, a value that is not finite as an operand would
        // reach rows that must not see it.  Such a tile is found by its scales, and the piece's rows are done again plainly: a
        // tile whose codes are small enough for the scale to be harmless only costs that.
        if (vis_lo < min(j0 + C::BN, n)) {
            uint32_t most = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) most = max(most, __float_as_uint(scale[x]) & 0x7f800000u);
            spoiled |= __builtin_amdgcn_ballot_w64(most > (uint32_t)C::FINITE << 23) != 0;
        }
#pragma unroll
        for (int y = 0; y < VD; y += 2) {
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) w[x] = widen2<OP>(v[x][y / 8], scale[x], y % 8 / 2);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t z[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], half ? 0x07060302u : 0x05040100u);
#pragma unroll
                for (int rt = 0; rt < ACT; ++rt)
#pragma unroll
                    for (int part = PARTS - 1; part >= 0; --part) multiply<OP, 16>(vec(z), vec(p[rt][part]), o[rt][y + half]);
            }
        }
    }

    // Units t0 .. t1 - 1 of the run, the first of them asked for already: a tile on its way while another is used, and
    // scales for two.  The loads past the end have an empty range.
    template <int ACT>
    __device__ __forceinline__ void run_tiles(int t0, int t1, int n) {
        for (int t = 0; t < t1 - t0; ++t) {
            const int half = t & 1;
            // (RG = 2: both groups' loads of this tile are there, and the other half is free)
            if constexpr (C::RG > 1) wait_and_meet<0>();
            if (half) ask_scales((t >> 1 & 1) ^ 1);
            ask_codes(half ^ 1);
            if constexpr (C::RG == 1) {
                if (half) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(C::CODE_LOADS + C::SCALE_LOADS) : "memory");
                else asm volatile("s_waitcnt vmcnt(%0)" ::"n"(C::CODE_LOADS) : "memory");
            }
            use<ACT>(half, t >> 1 & 1, half, (t0 + t) * C::UNIT + keys_of * C::BN, n);
        }
    }
    // With two groups of waves the second one may have no rows, or one tile of them.
    __device__ __forceinline__ void run(int t0, int t1, int n, int rows) {
        const int mine = rows - 16 * rows_of * RT;
        if (C::RG == 1 || mine > 16) run_tiles<RT>(t0, t1, n);
        else if (mine > 0) run_tiles<1>(t0, t1, n);
        else run_tiles<0>(t0, t1, n);
        wait_and_meet<0>();  // all waves are done with their places
    }
};

// Where a piece's rows go: `slot` of the workspace, or out.
template <typename C>
__device__ __forceinline__ void put_row(const Fp4Args& f, long long first, int hk, int r, long long slot, float m, float sum, int e,
                                        f32x4 o) {
    using TS = typename C::TS;
    const Args& a = f.a;
    const int i = (int)(r * f.g_inverse >> 16), h = hk * a.G + r - i * a.G;
    if (slot >= 0) {
        const long long at = slot * C::BM + r;
        *reinterpret_cast<f32x4*>(a.slot_o + at * a.c.D + e) = o;
        if (e == 0) a.slot_ml[at] = make_float2(m, sum);
        return;
    }
    o *= sum == 0.0f ? 0.0f : 1.0f / sum;
    TS* p = static_cast<TS*>(a.c.out.p) + (first + i) * a.c.out.row + h * a.c.out.head + e;
    if constexpr (sizeof(TS) == 2) *reinterpret_cast<u32x2*>(p) = u32x2{pack<typename C::T>(o[0], o[1]), pack<typename C::T>(o[2], o[3])};
    else *reinterpret_cast<f32x4*>(p) = o;
    if (e == 0 && a.c.lse != nullptr)
        a.c.lse[(first + i) * a.c.H + h] = sum == 0.0f ? -INFINITY : kLn2 * (m + __builtin_amdgcn_logf(sum));
}

// Joins the waves' sums of a piece and stores its rows.  Reached by all threads of the block.
template <typename C>
__device__ __forceinline__ void finish_piece(Short4<C>& b, const Run& run, long long slot) {
    const Fp4Args& f = args_again();
    const Args& a = f.a;
    const int rows = run.T * a.G;
    auto ml = reinterpret_cast<float2(*)[16]>(b.lds + C::PLACES + C::QBYTES);
    int* const spoiled = reinterpret_cast<int*>(b.lds + C::PLACES + C::QBYTES + C::KW * 16 * 8);
    float* const sums = reinterpret_cast<float*>(b.lds + (rows <= C::EARLY ? Short4<C>::codes_at(1, 0) : 0));
    const int most = min(rows, 16);  // rows of a tile in LDS
    bool again = false;
#pragma unroll
    for (int tile = 0; tile < C::RT * C::RG; ++tile) {
        const int here = min(rows - 16 * tile, 16);
        const int rt = tile % C::RT;
        if (tile > 0) {
            if (here <= 0) break;
            wait_and_meet<63>();  // the last tile's sums are read
        }
        if (b.rows_of == tile / C::RT) {
            const float l = over_row<16, false>(b.l[rt]);
            if (b.col < here) {
                if (b.grp == 0) ml[b.keys_of][b.col] = make_float2(b.ref[rt], l);
                float* at = sums + (b.keys_of * most + b.col) * C::ROW;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int y = 0; y < C::VD; y += 4)
                        *reinterpret_cast<f32x4*>(at + C::VD * (4 * b.grp + i) + y) =
                            f32x4{b.o[rt][y][i], b.o[rt][y + 1][i], b.o[rt][y + 2][i], b.o[rt][y + 3][i]};
            }
        }
        if (tile == 0 && b.lane == 0) spoiled[b.wave] = b.spoiled;
        wait_and_meet<63>();
        if (tile == 0)
#pragma unroll
            for (int w = 0; w < C::W; ++w) again |= spoiled[w] != 0;
        if (again) break;
        for (int x = threadIdx.x; x < here * (C::DP / 4); x += C::NT) {
            const int r = x / (C::DP / 4), e = x % (C::DP / 4) * 4;
            if (e >= a.c.D) continue;
            float m = ml[0][r].x, sum = 0.0f;
#pragma unroll
            for (int w = 1; w < C::KW; ++w) m = fmaxf(m, ml[w][r].x);
            f32x4 o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < C::KW; ++w) {
                const float by = __builtin_amdgcn_exp2f(ml[w][r].x - m);
                sum = fmaf(ml[w][r].y, by, sum);
                o += *reinterpret_cast<const f32x4*>(sums + (w * most + r) * C::ROW + e) * by;
            }
            put_row<C>(f, run.first, run.hk, 16 * tile + r, slot, m, sum, e, o);
        }
    }
    if (again) {
        using TS = typename C::TS;
        const float s2 = a.negate ? -a.s2 : a.s2;
        const Fp4Keys keys = fp4_keys(f.cache, run.begin, run.hk / f.share);
#pragma unroll 1
        for (int r = b.wave; r < rows; r += C::W) {
            const int i = r / a.G, g = r - i * a.G, seen = min(max(run.n - run.T + 1 + i, 0), run.n);
            const TS* q = static_cast<const TS*>(a.c.q.p) + (run.first + i) * a.c.q.row + (long long)(run.hk * a.G + g) * a.c.q.head;
            const RowSums x = plain_row<typename C::T>(q, keys, f.cache, a.c.D, s2, run.t0 * C::UNIT, min(run.t1 * C::UNIT, seen));
            if (4 * b.lane < a.c.D) put_row<C>(f, run.first, run.hk, r, slot, x.m, x.sum, 4 * b.lane, x.o);
        }
    }
}

template <typename C>
__global__ __launch_bounds__(C::NT, C::WAVES) void short4_kernel(Fp4Args) {
    extern __shared__ __align__(1024) char lds[];
    const int w = blockIdx.x;
    using All = Tiles<C::UNIT>;
    Run run;
    long long u, u1, total;
    int W;
    {
        const Args& a = args_again().a;
        const All all(a.c);
        total = uniform(all.total) * a.c.HK;
        report(a, all.malformed, w);
        W = (int)min(total, (long long)a.workers);
        if (all.malformed || w >= W) {
            if (a.cut != nullptr && threadIdx.x == 0) a.cut[w] = make_int4(0, 0, 0, 0);
            return;
        }
        const Cut cut(total, W);
        u = uniform(cut.start(w));
        u1 = uniform(cut.start(w + 1));
        long long base;
        all.find(u >> 31 ? u / a.c.HK : (unsigned)u / (unsigned)a.c.HK, &run.b, &base);
        run.b = uniform(run.b);
        run.t0 = (int)(u - uniform(base) * a.c.HK);
    }
    auto look_up = [&](Run& r) {
        const AttnLaunch& c = args_again().a.c;
        r.first = uniform(entry(c.offsets, r.b));
        r.T = uniform(entry(c.offsets, r.b + 1)) - r.first;
        r.n = uniform(entry(c.kv_len, r.b));
        r.begin = uniform((long long)entry(c.kv_begin, r.b));
        r.tiles = All::of(r.T, r.n);
    };
    look_up(run);
    run.hk = uniform(run.t0 / run.tiles);
    run.t0 -= run.hk * run.tiles;
    Short4<C> b(lds);
    auto start = [&](Run& r, long long at) {  // asks for the first tile of the piece that begins at unit `at`
        r.t1 = (int)min((long long)r.tiles, r.t0 + (u1 - at));
        b.open(args_again(), r.begin, r.hk, r.t0, r.t1, r.n);
        b.ask_first();
    };
    start(run, u);
    while (true) {
        {
            const Fp4Args& f = args_again();
            const int rows = run.T * f.a.G;
            b.take_rows(f, rows, run.first, run.hk);
            b.see(f, rows, run.n - run.T + 1, run.n);
        }
        if constexpr (C::QLDS) wait_and_meet<63>();
        b.run(run.t0, run.t1, run.n, run.T * args_again().a.G);

        const Args& a = args_again().a;
        const long long next_u = u + run.t1 - run.t0;
        Run next = run;
        bool early = false;
        if (next_u < u1) {
            next.t0 = 0;
            if (++next.hk == a.c.HK) {
                next.hk = 0;
                do {
                    ++next.b;
                    look_up(next);
                } while (next.tiles == 0);
            }
            early = run.T * a.G <= C::EARLY;
            if (early) start(next, next_u);
        }
        // a worker's slot 0: a run cut at the front; slot 1: a run that starts here and goes on in the next worker
        const bool whole = run.t1 - run.t0 == run.tiles;
        finish_piece<C>(b, run, whole ? -1 : w * 2ll + (run.t0 == 0 ? 1 : 0));
        if (run.t0 == 0 && (a.row_info != nullptr || !whole)) {
            const int pieces = whole ? 1 : Cut(total, W).part(u + run.tiles - 1) - w + 1;
            if (a.row_info != nullptr)
                for (int i = threadIdx.x; i < run.T; i += C::NT)
                    a.row_info[(long long)(run.first + i) * a.c.HK + run.hk] = make_int2(whole ? -1 : w, pieces * 128 + i);
            if (!whole && a.cut != nullptr && threadIdx.x == 0) a.cut[w] = make_int4(run.first, run.T, run.hk, pieces);
        }
        if (next_u >= u1) {
            if ((whole || run.t0 != 0) && a.cut != nullptr && threadIdx.x == 0) a.cut[w] = make_int4(0, 0, 0, 0);
            return;
        }
        u = next_u;
        run = next;
        wait_and_meet<63>();  // the piece's sums are read
        if (!early) start(run, u);
    }
}

// A block a run, for short ones: nothing is cut, and no second launch joins anything.
template <typename C>
__global__ __launch_bounds__(C::NT, C::WAVES) void runs4_kernel(Fp4Args) {
    extern __shared__ __align__(1024) char lds[];
    const Fp4Args& f = args_again();
    const AttnLaunch& c = f.a.c;
    Run run;
    run.b = blockIdx.x / c.HK;
    run.hk = blockIdx.x - run.b * c.HK;
    const Sequence s = sequence(c, run.b);  // in bounds, whatever the arrays hold
    run.first = s.first, run.T = s.T, run.n = s.n, run.begin = s.begin;
    run.t0 = 0;
    run.t1 = run.tiles = Tiles<C::UNIT>::of(run.T, run.n);
    Short4<C> b(lds);
    const int rows = run.T * f.a.G;
    if (run.T > 0) {  // on their way while the call is checked
        b.open(f, run.begin, run.hk, 0, run.t1, run.n);
        b.ask_first();
        b.take_rows(f, rows, run.first, run.hk);
    }
    const bool malformed = check<C::NT>(c);
    report(f.a, malformed, blockIdx.x);
    if (malformed || run.T == 0) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        return;
    }
    b.see(f, rows, run.n - run.T + 1, run.n);
    if constexpr (C::QLDS) wait_and_meet<63>();
    b.run(0, run.t1, run.n, rows);
    finish_piece<C>(b, run, -1);
}

// Operand steps of the long form's queries in LDS at width 256: one more than over a plain cache, as codes on their way take
// registers.
constexpr int kQueriesInLds = 11;

// The long form (prompts): gdn_attn.hpp's tiles, pipeline and products, with the keys and values of a tile widened on their way
// to LDS: a thread loads the codes of a run of elements of one key and of one value, a tile ahead of their use, and writes
// them as operands where the asynchronous loads of a plain cache would have put them.
template <typename C>
struct Long4 : Block<C> {
    using B = Block<C>;
    using T = typename C::T;
    using Scores = typename B::Scores;
    using Rsrc = __amdgpu_buffer_rsrc_t;
    static constexpr int U = C::BN * C::DP / C::NT, UPR = C::DP / U;  // elements a thread, and such runs of a row
    static_assert((U == 16 || U == 32) && U * UPR == C::DP, "half a block of elements or a whole one");
    struct Half {
        uint32_t codes[U / 8], scale;
    };
    const Fp4Cache& cache;
    Half k, v;

    __device__ __forceinline__ Long4(const Fp4Args& f, char* lds) : B(f.a, lds), cache(f.cache) {}
    // What says the thread's row of a tile and its run of elements there.  At width 256 these are worked out where they are
    // needed, as there are no registers to keep them (16384 tokens 2231 us with fifty spilled, so 1940); at width 128 that
    // takes longer than keeping them (24748 tokens 1513 us and 1427).
    static __device__ __forceinline__ int thread() {
        int x = threadIdx.x;
        if constexpr (C::DP == 256) asm volatile("" : "+v"(x));
        return x;
    }
    // Thread x's row of a tile of keys or values, its run of elements there, and the order in which it writes the run's
    // pieces: piece i ^ turn at step i.  LDS takes 16 bytes of eight neighbours a cycle, over 128 bytes of banks, so these are
    // such that the places of eight neighbours differ modulo 8 (values of fp32 operands: in pairs).  With neighbours along
    // a row 40% of LDS's busy cycles were conflicts at width 128 (24748 tokens over up to 7100 keys 1372 us, so 1309; 2000
    // tokens of fp32 at width 256 831 us, so 753).
    template <bool V>
    static __device__ __forceinline__ int row_of(int x) {
        if constexpr (!C::HALF) return x >> 6 << 3 | (x & 7);
        else if constexpr (C::RB == 512) return x >> 5 << 1 | (x >> 2 & 1);
        else if constexpr (C::RB == 128) return x >> 4 << 2 | (x >> 1 & 2) | (x >> 3 & 1);
        else return V ? x >> 6 << 4 | (x >> 1 & 3) << 2 | (x >> 4 & 3) : x >> 4 << 2 | (x >> 1 & 3);
    }
    static __device__ __forceinline__ int part_of(int x) {
        if constexpr (!C::HALF) return x >> 3 & 7;
        else if constexpr (C::RB == 512) return (x >> 1 & 12) | (x & 3);
        else return C::RB == 128 ? x & 3 : (x >> 2 & 2) | (x & 1);
    }
    template <bool V>
    static __device__ __forceinline__ int turn_of(int x) {
        return V && C::HALF ? x >> 2 & 1 : 0;
    }
    static_assert(C::HALF ? U == (C::RB == 256 ? 32 : 16) && C::RB <= 512 : U == 32 && C::RB == 1024, "the threads' places");
    __device__ __forceinline__ Rsrc rows_of(const char* p, int j0, int left, long long stride, int width) const {
        const int rows = min(left, C::BN);
        return __builtin_amdgcn_make_buffer_rsrc((void*)(p + j0 * stride), 0, rows > 0 ? (rows - 1) * (int)stride + width : 0, kRsrc);
    }
    // Asks for a tile's keys or values; nothing for one that is not real.
    template <bool V>
    __device__ __forceinline__ void fetch(const Fp4Keys& s, int tile, bool real) {
        const Fp4Half& h = V ? cache.v : cache.k;
        const int j0 = real ? tile * C::BN : 0, left = real ? B::run_n - j0 : 0, D = B::a.c.D;
        const Rsrc rc = rows_of(V ? s.vc : s.kc, j0, left, h.codes.row, D / 2), rs = rows_of(V ? s.vs : s.ks, j0, left, h.scales.row, D / 32);
        const int x = thread(), row = row_of<V>(x), e = part_of(x) * U;
        const int c_off = e < D ? row * (int)h.codes.row + e / 2 : kOutside, s_off = e < D ? row * (int)h.scales.row + e / 32 : kOutside;
        Half& to = V ? v : k;
        if constexpr (U == 32) {
            const u32x4 y = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rc, c_off, 0, 0));
#pragma unroll
            for (int i = 0; i < 4; ++i) to.codes[i] = y[i];
        } else {
            const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rc, c_off, 0, 0));
            to.codes[0] = y[0], to.codes[1] = y[1];
        }
        to.scale = __builtin_amdgcn_raw_buffer_load_b8(rs, s_off, 0, 0);
    }
    // Writes them to a stage of the ring.
    template <bool V>
    __device__ __forceinline__ void put(int stage) {
        const int tid = thread(), row = row_of<V>(tid), run_at = part_of(tid), turn = turn_of<V>(tid);
        char* at = B::lds + stage * C::STAGE + (V ? C::KTILE + C::template row_at<C::VSTEP>(row) : C::template row_at<C::KSTEP>(row));
        const int sw = V ? C::place_v(row) : C::place_k(row);
        const Half& x = V ? v : k;
        const float scale = fp4::scale_of(x.scale);
        const uint32_t other = -turn;
#pragma unroll
        for (int i = 0; i < U / 8; ++i) {
            if constexpr (C::HALF) {
                u32x4 w;
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = widen2<T>((x.codes[i] & ~other) | (x.codes[i ^ 1] & other), scale, j);
                *reinterpret_cast<u32x4*>(at + (((run_at * (U / 8) + (i ^ turn)) ^ sw) * 16)) = w;
            } else {
                float y[8];
                fp4::values(x.codes[i], x.scale, y);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<f32x4*>(at + (((run_at * (U / 4) + 2 * i + j) ^ sw) * 16)) = f32x4{y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]};
            }
        }
    }

    // Tiles [t0, t1) of the run, as Block::run.  A wave without rows (`idle`) widens its share of every tile and leaves the matrix
    // cores to the others.
    template <typename F>
    __device__ __forceinline__ bool run(const Fp4Keys& s, int t0, int t1, int full, bool idle, F stop) {
        B::fresh_addresses();
        int stage = 0, t = t0;
        fetch<false>(s, t0, true);
        fetch<true>(s, t0, true);
        if (stop()) return false;
        put<false>(0);
        put<true>(0);
        fetch<false>(s, t0 + 1, t0 + 1 < t1);
        fetch<true>(s, t0 + 1, t0 + 1 < t1);
        if constexpr (!C::PIPE) {
            Scores cur;
            auto next = [&](int at) {
                wait_and_meet<63>();
                put<false>(at ^ 1);
                put<true>(at ^ 1);
                fetch<false>(s, t + 2, t + 2 < t1);
                fetch<true>(s, t + 2, t + 2 < t1);
            };
            for (; idle && t < t1; ++t, stage ^= 1) next(stage);
            auto one = [&](auto hidden, int at) {
                next(at);
                if (hidden.value) B::look(B::lds + at * C::STAGE + C::KTILE, t * C::BN);
                B::template plain_step<hidden.value>(at, t, cur);
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
            put<false>(1);
            fetch<false>(s, t0 + 2, t0 + 2 < t1);
            wait_and_meet<63>();
            // Widening stands behind the step's products: 24748 tokens over up to 7100 keys 1419 us, before them 1463.
            auto later = [&](int at) {
                put<true>(at ^ 1);
                put<false>(at);
                fetch<true>(s, t + 2, t + 2 < t1);
                fetch<false>(s, t + 3, t + 3 < t1);
            };
            if (idle) {
                for (; t < t1 - 1; ++t, stage ^= 1) {
                    wait_and_meet<63>();
                    later(stage);
                }
                wait_and_meet<63>();
                wait_and_meet<63>();
                return true;
            }
            B::template scores<true>(0, now);
            if (t0 >= full) B::hide(now, t0 * C::BN);
            top = B::largest(now);
            while (t + 2 < min(full, t1 - 1)) {
                wait_and_meet<63>();
                B::template step<false, false>(0, t, now, next, top);
                later(0);
                ++t;
                wait_and_meet<63>();
                B::template step<false, false>(1, t, next, now, top);
                later(1);
                ++t;
            }
            for (; t < t1 - 1; ++t) {
                wait_and_meet<63>();
                if (t >= full) B::look(B::lds + stage * C::STAGE + C::KTILE, t * C::BN);
                B::template step<true, false>(stage, t, now, next, top);
                later(stage);
#pragma unroll
                for (int x = 0; x < B::KT; ++x)
#pragma unroll
                    for (int u = 0; u < C::SUB; ++u) now[x][u] = next[x][u];
                stage ^= 1;
            }
            wait_and_meet<63>();
            if (t >= full) B::look(B::lds + stage * C::STAGE + C::KTILE, t * C::BN);
            B::template step<false, true>(stage, t, now, next, top);
        }
        wait_and_meet<63>();
        return true;
    }

    // The wave's rows again, plainly, in place of store(), over the keys k0 .. k1 - 1.
    __device__ __forceinline__ void redo4(const typename B::To& to, const Fp4Keys& s, int k0, int k1, int seen0) {
        const Args& a = B::a;
        const float s2 = a.negate ? -a.s2 : a.s2;
#pragma unroll 1
        for (int x0 = 0; x0 < B::M; ++x0) {
            const int r = to.row0 + B::wave * B::M + x0;
            if (r >= to.rows) break;
            const int i = r / a.G, g = r - i * a.G;
            const auto* q = static_cast<const typename C::TS*>(a.c.q.p) + (to.first + i) * a.c.q.row + (long long)(to.hk * a.G + g) * a.c.q.head;
            const RowSums x = plain_row<T>(q, s, cache, a.c.D, s2, k0, min(k1, seen0 + i));
            const auto y = B::row_at(to, r, x.m, x.sum, B::lane == 0);
            for (int z = 0; z < 4 && 4 * B::lane < a.c.D; ++z) {
                if (y.sums != nullptr) y.sums[4 * B::lane + z] = x.o[z];
                else y.out[4 * B::lane + z] = from_f32<T>(x.o[z] * y.inv);
            }
        }
    }
};

// The long form for fp32 queries up to width 128, on matrix instructions of bf16: queries and probabilities are sums of
// three parts each (short form, Cfg4), and three of those products take less than half of the fp32 one's time.
template <typename C>
struct Long4Split : Long4<C> {
    using B = Block<C>;
    using L = Long4<C>;
    using Scores = typename B::Scores;
    static constexpr int PARTS = 3;
    u32x4 parts[PARTS][C::CS];

    __device__ __forceinline__ Long4Split(const Fp4Args& f, char* lds) : L(f, lds) {}

    __device__ __forceinline__ const float* query(const typename B::To& to, int r) const {
        const Args& a = B::a;
        const int i = r / a.G, g = r - i * a.G;
        return static_cast<const float*>(a.c.q.p) + (to.first + i) * a.c.q.row + (long long)(to.hk * a.G + g) * a.c.q.head;
    }
    __device__ __forceinline__ void load_rows(int row0, int rows, long long first, int hk) {
        const int r = row0 + B::wave * B::M + B::col;
        const bool in = r < rows;
        const float* p = query(typename B::To{row0, rows, first, hk, -1, -1}, in ? r : row0);
        const uint32_t flip = B::a.negate ? 0x80008000u : 0u;
#pragma unroll
        for (int s = 0; s < C::CS; ++s) {
            const int e = (C::NG * s + B::grp) * 8;
            const bool real = in && e < B::a.c.D;
            const f32x4 x = *reinterpret_cast<const f32x4*>(p + (real ? e : 0)), y = *reinterpret_cast<const f32x4*>(p + (real ? e + 4 : 0));
            const float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[PARTS];
                split2<BF16, PARTS>(v[2 * j], v[2 * j + 1], w, 1);
#pragma unroll
                for (int z = 0; z < PARTS; ++z) parts[z][s][j] = real ? w[z] ^ flip : 0u;
            }
        }
        B::clear();
    }
    __device__ __forceinline__ void scores(int stage, Scores& acc) {
        const char* kt = B::lds + stage * C::STAGE + C::template row_at<C::KSTEP>(B::col);
#pragma unroll
        for (int k = 0; k < B::KT; ++k) {
            acc[k][0] = Acc<B::M>{};
#pragma unroll
            for (int x = 0; x < C::CS; ++x) {
                const u32x4 f = *reinterpret_cast<const u32x4*>(kt + C::template row_at<C::KSTEP>(k * 32) + (((C::NG * x + B::grp) ^ C::place_k(B::col)) * 16));
#pragma unroll
                for (int z = PARTS - 1; z >= 0; --z) multiply<BF16, B::M>(f, parts[z][x], acc[k][0]);
            }
        }
    }
    __device__ __forceinline__ void product(const char* vt, const Scores& s) {
#pragma unroll
        for (int k = 0; k < B::KT; ++k)
#pragma unroll
            for (int z = 0; z < B::SN / 8; ++z) {
                uint32_t p[PARTS][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split2<BF16, PARTS>(s[k][0][8 * z + 2 * e], s[k][0][8 * z + 2 * e + 1], &p[0][e], 4);
#pragma unroll
                for (int d = 0; d < B::DT; ++d) {
                    const u32x4 v = B::values(vt, k, z, d);
#pragma unroll
                    for (int x = PARTS - 1; x >= 0; --x) multiply<BF16, B::M>(v, u32x4{p[x][0], p[x][1], p[x][2], p[x][3]}, B::o[d]);
                }
            }
    }
    // Tiles [t0, t1) of the run, one after the other: three products take long enough for the other wave of the SIMD.
    template <typename F>
    __device__ __forceinline__ bool run(const Fp4Keys& s, int t0, int t1, int full, bool idle, F stop) {
        B::fresh_addresses();
        L::template fetch<false>(s, t0, true);
        L::template fetch<true>(s, t0, true);
        if (stop()) return false;
        L::template put<false>(0);
        L::template put<true>(0);
        L::template fetch<false>(s, t0 + 1, t0 + 1 < t1);
        L::template fetch<true>(s, t0 + 1, t0 + 1 < t1);
        Scores cur;
        for (int t = t0, stage = 0; t < t1; ++t, stage ^= 1) {
            wait_and_meet<63>();
            const char* vt = B::lds + stage * C::STAGE + C::KTILE;
            if (!idle) {
                scores(stage, cur);
                if (t >= full) {
                    B::hide(cur, t * C::BN);
                    B::look(vt, t * C::BN);
                }
                B::follow(B::largest(cur));
                B::exponentials(cur);
                product(vt, cur);
            }
            L::template put<false>(stage ^ 1);
            L::template put<true>(stage ^ 1);
            L::template fetch<false>(s, t + 2, t + 2 < t1);
            L::template fetch<true>(s, t + 2, t + 2 < t1);
        }
        return true;
    }
    // Where row r goes: fp32 sums, or fp32 outputs.
    __device__ __forceinline__ float* place(const typename B::To& to, int r, float m, float sum, bool stats, float& by) const {
        const Args& a = B::a;
        const int i = r / a.G, h = to.hk * a.G + r - i * a.G;
        const long long token_row = (to.first + i) * a.c.H + h;
        by = 1.0f;
        if (to.set >= 0) {
            const long long at = to.set * a.set_rows + token_row;
            if (stats) a.set_ml[at] = make_float2(m, sum);
            return a.set_o + at * a.c.D;
        }
        by = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (stats && a.c.lse != nullptr) a.c.lse[token_row] = sum == 0.0f ? -INFINITY : kLn2 * (m + __builtin_amdgcn_logf(sum));
        return static_cast<float*>(a.c.out.p) + (to.first + i) * a.c.out.row + h * a.c.out.head;
    }
    __device__ __forceinline__ void store(const typename B::To& to) {
        const int r = to.row0 + B::wave * B::M + B::col;
        if (r >= to.rows || B::spoiled) return;
        float by;
        float* p = place(to, r, B::ref, B::l, B::grp == 0, by) + 4 * B::grp;
#pragma unroll
        for (int d = 0; d < B::DT; ++d)
#pragma unroll
            for (int i = 0; i < C::EA / 4; ++i) {
                const int e = B::M * d + 4 * C::NG * i;
                if (e + 4 * B::grp < B::a.c.D)
                    *reinterpret_cast<f32x4*>(p + e) = f32x4{B::o[d][4 * i], B::o[d][4 * i + 1], B::o[d][4 * i + 2], B::o[d][4 * i + 3]} * by;
            }
    }
    __device__ __forceinline__ void redo4(const typename B::To& to, const Fp4Keys& s, int k0, int k1, int seen0) {
        const Args& a = B::a;
#pragma unroll 1
        for (int x0 = 0; x0 < B::M; ++x0) {
            const int r = to.row0 + B::wave * B::M + x0;
            if (r >= to.rows) break;
            const RowSums x = plain_row<F32>(query(to, r), s, L::cache, a.c.D, a.negate ? -a.s2 : a.s2, k0, min(k1, seen0 + r / a.G));
            float by;
            float* p = place(to, r, x.m, x.sum, B::lane == 0, by);
            if (4 * B::lane < a.c.D) *reinterpret_cast<f32x4*>(p + 4 * B::lane) = x.o * by;
        }
    }
};

// Which of them, and its tiles: L is the block, C its configuration.
template <typename T, int DP>
struct Long4For {
    using C = typename Long<T, DP, kQueriesInLds>::C;
    using L = Long4<C>;
};
template <>
struct Long4For<F32, 64> {
    using C = typename Long<BF16, 64>::C;
    using L = Long4Split<C>;
};
template <>
struct Long4For<F32, 128> {
    using C = typename Long<BF16, 128>::C;
    using L = Long4Split<C>;
};
template <typename T, typename F>
auto with_long4(int dp, F f) {
    return dp == 64 ? f(Long4For<T, 64>{}) : dp == 128 ? f(Long4For<T, 128>{}) : f(Long4For<T, 256>{});
}

// One block per key head, key part and tile of BM rows, as gdn_attn.hpp's long form.
template <typename X>
__global__ __launch_bounds__(X::C::NT, X::C::WAVES) void long4_kernel(Fp4Args f) {
    using C = typename X::C;
    extern __shared__ __align__(1024) char lds[];
    const Args& a = f.a;
    const unsigned block = blockIdx.x;
    unsigned x = block;
    const int hk = x % a.c.HK;
    x /= a.c.HK;
    const unsigned slots = a.c.N * a.G / C::BM + a.c.B;
    int part = 0;
    if (a.splits > 1) {
        const int four = x / (4 * slots), of = min(4, a.splits - 4 * four);
        x -= four * 4 * slots;
        part = 4 * four + x % of;
        x /= of;
    }
    int b = 0;
    unsigned back = x;  // tiles of the sequence behind this one
    if (a.c.B <= 64) {
        back = by_keys<C::BM>(a.c, a.G, x, &b);
    } else {
        b = sequence_at<C::BM>(a.c, a.G, x);
        back = x - slot_of<C::BM>(a.c, a.G, uniform(entry(a.c.offsets, b)), b);
    }
    const Sequence seq = sequence(a.c, b);
    const int first = seq.first, T = seq.T, n = seq.n;
    auto stop = [&] {
        const bool malformed = check<C::NT>(a.c);
        report(a, malformed, block);
        return malformed;
    };
    const int rows = T * a.G, tiles = (rows + C::BM - 1) / C::BM;
    const int parts = min(a.splits, max(1, (int)((unsigned)n / kPartKeys)));
    if (back >= (unsigned)tiles || part >= parts) {
        if (block == 0) stop();  // the block that reports
        return;
    }
    const int row0 = (tiles - 1 - (int)back) * C::BM;
    const int seen0 = n - T + 1;
    const int last_token = min(row0 + C::BM, rows) - 1;
    const int reach = uniform(max(0, min(n, seen0 + last_token / a.G)));  // keys the last row sees
    const int all = (reach + C::BN - 1) / C::BN;
    const int t0 = uniform((int)((long long)all * part / parts)), t1 = uniform((int)((long long)all * (part + 1) / parts));

    typename X::L blk(f, lds);
    blk.load_rows(row0, rows, first, hk);
    blk.see(row0, rows, true, seen0, n);
    const Fp4Keys keys = fp4_keys(f.cache, seq.begin, hk);
    if (t0 < t1) {
        const int full = uniform(max(0, min(n, seen0 + row0 / a.G)) / C::BN);
        if (!blk.run(keys, t0, t1, full, row0 + blk.wave * C::M >= rows, stop)) return;
    } else if (stop()) {
        return;  // no keys at all
    }
    if (a.live != nullptr && part == 0 && hk == 0)
        for (int i = row0 / a.G + (int)threadIdx.x; i <= last_token / a.G; i += C::NT) a.live[first + i] = parts;
    blk.sum_rows();
    const typename Block<C>::To to{row0, rows, first, hk, a.to_sets ? part : -1, -1};
    blk.store(to);
    if (blk.spoiled) blk.redo4(to, keys, t0 * C::BN, max(0, min(t1 * C::BN, n)), seen0);
}

// Row tiles and waves of the short form, for `tiles` tiles of 16 rows.  Up to four tiles a wave (WAVES: of a SIMD, as the
// registers leave room for); at width 256 two, and two groups of waves for more.  (40 rows over 64 caches of 1000 to 8000
// keys, D 256: 74 us, 90 with three tiles a wave and one wave a SIMD.)
template <typename T, int DP, int TILES>
struct Short4For {
    static constexpr bool F32IO = T::code == GDN_F32;
    static constexpr int RG = DP == 256 && TILES > 2 && !F32IO ? 2 : 1, RT = RG == 2 ? 2 : TILES;
    static constexpr int STATE = RT * (DP / 4 + 18) + (TILES == 1 ? DP / 8 * (F32IO ? 3 : 1) : 0) + DP / 8 + 40;
    static constexpr int WAVES = STATE <= 128 ? 4 : STATE <= 170 ? 3 : STATE <= 256 ? 2 : 1;
    template <bool WIDE>
    using C = Cfg4<T, DP, RT, 4, RG, WAVES, WIDE>;
    // a block a run: as many waves as there are registers and LDS for
    template <bool WIDE, int KW>
    using Wide = Cfg4<T, DP, RT, KW, 1, KW / 4, WIDE>;
    template <bool WIDE>
    using Whole = std::conditional_t<DP < 256 && Wide<WIDE, 16>::LDS <= kMaxLds, Wide<WIDE, 16>,
                                     std::conditional_t<Wide<WIDE, 8>::LDS <= kMaxLds, Wide<WIDE, 8>, Wide<WIDE, 4>>>;
};
// Rows of the short form at most: the three parts of more than 32 fp32 queries wider than 128 do not fit LDS beside byte by
// byte scales, nor the registers.
template <typename T>
constexpr int short_rows(int dp) {
    return T::code == GDN_F32 && dp == 256 ? 32 : 64;
}

template <typename T, int DP, typename F>
auto with_row_tiles(int tiles, F f) {
    constexpr int MOST = short_rows<T>(DP) / 16;
    switch (std::min(tiles, MOST)) {
        case 1: return f(Short4For<T, DP, 1>{});
        case 2: return f(Short4For<T, DP, 2>{});
        case 3: return f(Short4For<T, DP, std::min(3, MOST)>{});
        default: return f(Short4For<T, DP, MOST>{});
    }
}
template <typename T, typename F>
auto with_short4(int dp, int tiles, bool wide, F f) {
    auto g = [&](auto x) {
        return wide ? f(typename decltype(x)::template C<true>{}) : f(typename decltype(x)::template C<false>{});
    };
    return dp == 64 ? with_row_tiles<T, 64>(tiles, g) : dp == 128 ? with_row_tiles<T, 128>(tiles, g) : with_row_tiles<T, 256>(tiles, g);
}
// One tile of rows.
template <typename T, typename F>
auto with_whole4(int dp, bool wide, F f) {
    auto g = [&](auto x) {
        return wide ? f(typename decltype(x)::template Whole<true>{}) : f(typename decltype(x)::template Whole<false>{});
    };
    return dp == 64 ? g(Short4For<T, 64, 1>{}) : dp == 128 ? g(Short4For<T, 128, 1>{}) : g(Short4For<T, 256, 1>{});
}

template <typename T>
hipError_t start_short4(const Fp4Args& f, int dp, int tiles, bool wide, hipStream_t stream);
template <typename T>
hipError_t start_whole4(const Fp4Args& f, int dp, bool wide, hipStream_t stream);

template <typename T>
hipError_t start_long4(const Fp4Args& f, int dp, long long blocks, int lds, hipStream_t stream);

template <typename X>
hipError_t start_one_long4(const Fp4Args& f, long long blocks, int lds, hipStream_t stream) {
    static std::atomic<uint64_t> asked{0};
    return start_kernel(&long4_kernel<X>, asked, f, blocks, X::C::NT, lds, stream);
}
template <typename C>
hipError_t start_one_short4(const Fp4Args& f, hipStream_t stream) {
    static std::atomic<uint64_t> asked{0};
    return start_kernel(&short4_kernel<C>, asked, f, f.a.workers, C::NT, C::LDS, stream);
}
template <typename C>
hipError_t start_one_whole4(const Fp4Args& f, hipStream_t stream) {
    static std::atomic<uint64_t> asked{0};
    return start_kernel(&runs4_kernel<C>, asked, f, (long long)f.a.c.B * f.a.c.HK, C::NT, C::LDS, stream);
}

#define GDN_ATTN_FP4_INSTANCES(T)                                                                                      \
    template <>                                                                                                        \
    hipError_t start_short4<T>(const Fp4Args& f, int dp, int tiles, bool wide, hipStream_t stream) {                   \
        return with_short4<T>(dp, tiles, wide, [&](auto c) { return start_one_short4<decltype(c)>(f, stream); });      \
    }                                                                                                                  \
    template <>                                                                                                        \
    hipError_t start_whole4<T>(const Fp4Args& f, int dp, bool wide, hipStream_t stream) {                              \
        return with_whole4<T>(dp, wide, [&](auto c) { return start_one_whole4<decltype(c)>(f, stream); });             \
    }                                                                                                                  \
    template <>                                                                                                        \
    hipError_t start_long4<T>(const Fp4Args& f, int dp, long long blocks, int lds, hipStream_t stream) {               \
        return with_long4<T>(dp, [&](auto x) { return start_one_long4<decltype(x)>(f, blocks, lds, stream); });        \
    }

}  // namespace attn
}  // namespace gdn
