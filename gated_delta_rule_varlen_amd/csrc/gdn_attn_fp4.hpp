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
// A block's four waves take 32 keys each of every 128, each with a ring of its own and nothing shared until a run's end,
// where their sums are joined through LDS.  All runs lie end to end and are cut into equal parts, one a block, as in the
// short form there.
#pragma once

#include "gdn_attn.hpp"
#include "gdn_fp4.hpp"

namespace gdn {
namespace attn {

struct Fp4Args {
    Args a;
    Fp4Cache cache;
};

// The kernel's argument, read again: what a loop does not need is not worth scalar registers across it (with all of it
// held, 130 of them were spilled, and read back in the loop).
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
                fp4::values(reinterpret_cast<const uint32_t*>(codes)[x], scales[x / 4], k);
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
            fp4::values(*reinterpret_cast<const uint16_t*>(s.vc + (j0 + j) * c.v.codes.row + 2 * lane),
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
template <typename T_, int DP_, int RT_, int WAVES_, bool WIDE_>
struct Cfg4 {
    using T = T_;
    using TS = typename T::storage;
    using OP = std::conditional_t<T::code == GDN_F16, F16, BF16>;
    static constexpr int DP = DP_, RT = RT_, WAVES = WAVES_;  // WAVES: of a SIMD, which is blocks of a CU
    static constexpr bool WIDE = WIDE_;
    static constexpr int PARTS = T::code == GDN_F32 ? 3 : 1;
    static constexpr int W = 4, NT = 64 * W, BN = 32, UNIT = BN * W, BM = 16 * RT, NS = 2;
    static constexpr int CL = DP / 4 < 32 ? DP / 4 : 32;  // neighbouring elements a lane holds of a key
    static constexpr int KH = DP / (4 * CL);              // such pieces of a key
    static constexpr int STEPS = DP / 32, SPP = CL / 8;   // operand steps, and of a piece
    static constexpr int VD = DP / 16;                    // neighbouring elements a lane holds of a value
    static constexpr int NB = DP / 32, RB = DP / 2;       // blocks and bytes of codes of a row
    static constexpr int SB = WIDE ? (NB < 4 ? NB : 4) : 1, SLOTS = NB / SB;  // scales of a 32-bit place in LDS, places of a row
    static constexpr int CODES = BN * RB, CN = CODES / 1024, RPL = 1024 / RB; // bytes, loads, rows a load
    static constexpr int SN = (BN * SLOTS + 63) / 64, SCALES = 256 * SN;      // loads of scales, and their bytes in LDS
    static constexpr int STAGE = 2 * (CODES + SCALES), LOADS = 2 * (CN + SN);
    static constexpr bool QLDS = RT * PARTS > 1;          // queries in LDS: read once for two products
    static constexpr int RING = NS * STAGE, QBYTES = QLDS ? RT * PARTS * STEPS * 1024 : 0;
    static constexpr int ROW = DP + 4;                    // fp32 sums of a row in LDS
    static constexpr int LDS = W * RING + QBYTES;
    static_assert(W * 16 * ROW * 4 <= W * RING && LDS <= 159 * 1024, "the waves' sums take the ring's place");
    static constexpr float BIAS = T::code == GDN_F16 ? 4.0f : 0.0f, LAG = 8.0f;
    // Codes in LDS: 16-byte pieces (a block each) of key r at place piece ^ place_k(r), so that the 16 rows that are read
    // at a time lie in different banks; values in the order of row_of, so that four groups' rows are neighbours.
    static __device__ __forceinline__ int place_k(int r) { return DP == 64 ? (r >> 3) & 1 : DP == 128 ? (r >> 2) & 3 : (r >> 1) & 7; }
    static __device__ __forceinline__ int row_of(int place) { return (place & 16) + (place & 3) * 4 + ((place >> 2) & 3); }
};

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

// A number whose exponent is the byte at `at` of x, as the conversions look at nothing else of a scale (checked over all
// exponents with the other bits at random).
__device__ __forceinline__ float scale_at(uint32_t x, uint32_t at) {
    return __uint_as_float(__builtin_amdgcn_alignbit(x, x, 8 * at + 9));
}

// 64 x BYTES to LDS, 32 bits a lane (zeros above) for fewer than 16 bytes, as load_to_lds of gdn_attn.hpp.
template <int BYTES>
__device__ __forceinline__ void stream_to_lds(const Range& s, uint32_t at, int voff, int soff) {
    static_assert(BYTES == 1 || BYTES == 2 || BYTES == 4 || BYTES == 16, "bytes");
#define GDN_LOAD(op) asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\t" op " %1, %2, %3 offen nt lds" ::"s"(at), "v"(voff), "s"(s.r), "s"(soff) : "m0", "memory")
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
    char* ring;         // this wave's
    uint32_t ring_at;   // its LDS address
    int lane, wave, col, grp;
    int kc_off[KO], vc_off, ks_off[SN], vs_off[SN];  // byte offsets of what the lane loads of a tile
    int krow, vrow;                              // bytes between rows of codes
    uint32_t q[C::QLDS ? 1 : C::STEPS][4];
    Acc<16> o[RT][VD];
    float ref[RT], l[RT], c;
    int vis[RT], vis_lo, vis_hi;
    bool spoiled;

    // One tensor of the run, from the wave's next tile on.
    struct Stream {
        uint64_t at;
        int step, full, tail;  // bytes to the wave's next tile; of 32 rows; of the rows of the last, shorter tile
        __device__ __forceinline__ void open(const char* p, int j0, int rows, long long stride, int width) {
            at = (uint64_t)uniform((long long)(reinterpret_cast<uint64_t>(p) + j0 * stride));
            step = C::UNIT * (int)stride;
            full = (C::BN - 1) * (int)stride + width;
            tail = uniform(rows > 0 ? (rows - 1) * (int)stride + width : 0);
        }
        __device__ __forceinline__ Range tile(int left) {
            Range r(reinterpret_cast<const void*>(at), uniform(left >= C::BN ? full : left > 0 ? tail : 0));
            at += (uint64_t)(int64_t)step;
            return r;
        }
    };
    Stream kc, ks, vc, vs;
    int left;  // rows of the run from the next tile on

    __device__ __forceinline__ explicit Short4(char* lds_) : lds(lds_) {
        const Fp4Args& f = args_again();
        lane = threadIdx.x & 63;
        wave = uniform((int)threadIdx.x >> 6);
        col = lane & 15;
        grp = lane >> 4;
        c = f.a.s2;
        krow = (int)f.cache.k.codes.row;
        vrow = (int)f.cache.v.codes.row;
        ring = lds + wave * C::RING;
        ring_at = uniform((int)(uintptr_t)(__attribute__((address_space(3))) char*)ring);
        const int D = f.a.c.D, in_load = lane / C::NB, piece = lane % C::NB;
#pragma unroll
        for (int j = 0; j < KO; ++j) {
            const int kp = piece ^ C::place_k(j * C::RPL + in_load);
            kc_off[j] = kp * 32 < D ? in_load * krow + kp * 16 : kOutside;
        }
        vc_off = piece * 32 < D ? C::row_of(in_load) * vrow + piece * 16 : kOutside;
#pragma unroll
        for (int j = 0; j < SN; ++j) {
            const int x = j * 64 + lane, row = x / C::SLOTS, slot = x % C::SLOTS;
            const bool in = row < C::BN && slot * C::SB * 32 < D;
            ks_off[j] = in ? row * (int)f.cache.k.scales.row + slot * C::SB : kOutside;
            vs_off[j] = in ? C::row_of(row) * (int)f.cache.v.scales.row + slot * C::SB : kOutside;
        }
    }

    // The wave's tile of every unit from t0 on, of a run of n rows; nothing from unit t1 on.
    __device__ __forceinline__ void open(const Fp4Args& f, const Fp4Keys& s, int t0, int t1, int n) {
        const int j0 = t0 * C::UNIT + wave * C::BN, end = min(n, t1 * C::UNIT), D = f.a.c.D;
        left = uniform(end - j0);
        const int tail = left & (C::BN - 1);  // of the one tile that may be shorter, if it is this wave's
        kc.open(s.kc, j0, tail, f.cache.k.codes.row, D / 2);
        ks.open(s.ks, j0, tail, f.cache.k.scales.row, D / 32);
        vc.open(s.vc, j0, tail, f.cache.v.codes.row, D / 2);
        vs.open(s.vs, j0, tail, f.cache.v.scales.row, D / 32);
    }
    // Asks for the next tile.  Who read this stage before is done: the wait is for its reads.
    __device__ __forceinline__ void ask(int stage) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        const uint32_t to = ring_at + stage * C::STAGE;
        const Range rk = kc.tile(left), rks = ks.tile(left), rv = vc.tile(left), rvs = vs.tile(left);
#pragma unroll
        for (int j = 0; j < CN; ++j) stream_to_lds<16>(rk, to + j * 1024, kc_off[j % KO], j * C::RPL * krow);
#pragma unroll
        for (int j = 0; j < SN; ++j) stream_to_lds<C::SB>(rks, to + 2 * C::CODES + j * 256, ks_off[j], 0);
#pragma unroll
        for (int j = 0; j < CN; ++j) {
            // rows of 16 lie one behind the other in eights: places 8 .. 15 are two rows further
            const int rows = C::RPL >= 16 ? j * C::RPL : j / 2 * 16 + j % 2 * 2;
            stream_to_lds<16>(rv, to + C::CODES + j * 1024, vc_off, rows * vrow);
        }
#pragma unroll
        for (int j = 0; j < SN; ++j) stream_to_lds<C::SB>(rvs, to + 2 * C::CODES + C::SCALES + j * 256, vs_off[j], 0);
        left -= C::UNIT;
    }

    // The queries of the sequence's rows, eight elements a step in the order of the keys' pieces; in LDS each wave
    // leaves a part of them.
    __device__ __forceinline__ void take_rows(const Args& a, int rows, long long first, int hk) {
        const int G = a.G;
        const uint32_t flip = a.negate ? 0x80008000u : 0u;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int r = 16 * rt + col, i = r / G, g = r - i * G;
            const bool in = r < rows;
            const TS* p = static_cast<const TS*>(a.c.q.p) + (first + (in ? i : 0)) * a.c.q.row + (long long)(hk * G + (in ? g : 0)) * a.c.q.head;
#pragma unroll
            for (int s = 0; s < C::STEPS; ++s) {
                if (C::QLDS && (rt * C::STEPS + s) % C::W != wave) continue;
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
                        for (int j = 0; j < 4; ++j) q[s][j] = w[0][j];
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
        return reinterpret_cast<u32x4*>(lds + C::W * C::RING + ((rt * PARTS + part) * C::STEPS + step) * 1024 + lane * 16);
    }
    // The keys each row sees: seen0 + its token, at least 0 and at most n.
    __device__ __forceinline__ void see(int G, int rows, int seen0, int n) {
        auto keys = [&](int r) { return min(max(seen0 + r / G, 0), n); };
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) vis[rt] = 16 * rt + col < rows ? keys(16 * rt + col) : n;
        vis_lo = uniform(keys(0));
        vis_hi = uniform(keys(rows - 1));
    }

    static __device__ __forceinline__ u32x4 vec(const uint32_t* x) { return u32x4{x[0], x[1], x[2], x[3]}; }

    // The tile at `stage`, keys j0 .. j0 + 31 of a run of n, against all rows.
    __device__ __forceinline__ void use(int stage, int j0, int n) {
        if (j0 >= vis_hi) return;
        const char* kt = ring + stage * C::STAGE;
        const char* vt = kt + C::CODES;
        const uint32_t* kst = reinterpret_cast<const uint32_t*>(kt + 2 * C::CODES);
        const uint32_t* vst = reinterpret_cast<const uint32_t*>(kt + 2 * C::CODES + C::SCALES);
        Acc<16> s[RT][2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = Acc<16>{};
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
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int z = PARTS - 1; z >= 0; --z) {
                        u32x4 y;
                        if constexpr (C::QLDS) y = *query_at(rt, z, h * C::SPP + x);
                        else y = vec(q[h * C::SPP + x]);
#pragma unroll
                        for (int u = 0; u < 2; ++u) multiply<OP, 16>(vec(w[u]), y, s[rt][u]);
                    }
            }
        }
        const bool masked = j0 + C::BN > vis_lo;
        if (masked) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const int room = vis[rt] - j0 - 4 * grp;
#pragma unroll
                for (int i = 0; i < 8; ++i) s[rt][i / 4][i % 4] = 16 * (i / 4) + i % 4 >= room ? -INFINITY : s[rt][i / 4][i % 4];
            }
            asm volatile("");  // keeps this a branch: most tiles hide nothing
        }
        uint32_t p[RT][PARTS][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
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
        // 0 * NaN is NaN: where rows differ in what they see, a value without a number would reach rows that must not
        // see it.  Such a tile is found here, and the piece's rows are done again plainly.
        if (vis_lo < min(j0 + C::BN, n)) {
            uint32_t most = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) most = max(most, __float_as_uint(scale[x]) & 0x7f800000u);
            spoiled |= __builtin_amdgcn_ballot_w64(most == 0x7f800000u) != 0;
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
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int part = PARTS - 1; part >= 0; --part) multiply<OP, 16>(vec(z), vec(p[rt][part]), o[rt][y + half]);
            }
        }
    }

    // Units t0 .. t1 - 1 of the run, a tile on its way while another is used; the loads past the end have an empty range.
    __device__ __forceinline__ void run(int t0, int t1, int n) {
        int stage = 0;
        for (int t = t0; t < t1; ++t) {
            ask(stage ^ 1);
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(C::LOADS) : "memory");
            use(stage, t * C::UNIT + wave * C::BN, n);
            stage ^= 1;
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
};

// Where a piece's rows go: `slot` of the workspace, or out.
template <typename C>
__device__ __forceinline__ void put_row(const Args& a, long long first, int hk, int r, long long slot, float m, float sum, int e,
                                        f32x4 o) {
    using TS = typename C::TS;
    const int i = r / a.G, h = hk * a.G + r - i * a.G;
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
    __shared__ float2 ml[C::W][16];
    __shared__ int spoiled[C::W];
    float* const sums = reinterpret_cast<float*>(b.lds);
    const int most = min(rows, 16);  // rows of a tile in LDS
    bool again = false;
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
        const int here = min(rows - 16 * rt, 16);
        if (rt > 0) {
            if (here <= 0) break;
            __syncthreads();  // the last tile's sums are read
        }
        const float l = over_row<16, false>(b.l[rt]);
        if (b.col < here) {
            if (b.grp == 0) ml[b.wave][b.col] = make_float2(b.ref[rt], l);
            float* at = sums + (b.wave * most + b.col) * C::ROW;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int y = 0; y < C::VD; y += 4)
                    *reinterpret_cast<f32x4*>(at + C::VD * (4 * b.grp + i) + y) =
                        f32x4{b.o[rt][y][i], b.o[rt][y + 1][i], b.o[rt][y + 2][i], b.o[rt][y + 3][i]};
        }
        if (rt == 0 && b.lane == 0) spoiled[b.wave] = b.spoiled;
        __syncthreads();
        if (rt == 0)
#pragma unroll
            for (int w = 0; w < C::W; ++w) again |= spoiled[w] != 0;
        if (again) break;
        for (int x = threadIdx.x; x < here * (C::DP / 4); x += C::NT) {
            const int r = x / (C::DP / 4), e = x % (C::DP / 4) * 4;
            if (e >= a.c.D) continue;
            float m = ml[0][r].x, sum = 0.0f;
#pragma unroll
            for (int w = 1; w < C::W; ++w) m = fmaxf(m, ml[w][r].x);
            f32x4 o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < C::W; ++w) {
                const float by = __builtin_amdgcn_exp2f(ml[w][r].x - m);
                sum = fmaf(ml[w][r].y, by, sum);
                o += *reinterpret_cast<const f32x4*>(sums + (w * most + r) * C::ROW + e) * by;
            }
            put_row<C>(a, run.first, run.hk, 16 * rt + r, slot, m, sum, e, o);
        }
    }
    if (again) {
        using TS = typename C::TS;
        const float s2 = a.negate ? -a.s2 : a.s2;
        const Fp4Keys keys = fp4_keys(f.cache, run.begin, run.hk);
#pragma unroll 1
        for (int r = b.wave; r < rows; r += C::W) {
            const int i = r / a.G, g = r - i * a.G, seen = min(max(run.n - run.T + 1 + i, 0), run.n);
            const TS* q = static_cast<const TS*>(a.c.q.p) + (run.first + i) * a.c.q.row + (long long)(run.hk * a.G + g) * a.c.q.head;
            const RowSums x = plain_row<typename C::T>(q, keys, f.cache, a.c.D, s2, run.t0 * C::UNIT, min(run.t1 * C::UNIT, seen));
            if (4 * b.lane < a.c.D) put_row<C>(a, run.first, run.hk, r, slot, x.m, x.sum, 4 * b.lane, x.o);
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
    auto open = [&] {
        const AttnLaunch& c = args_again().a.c;
        run.first = uniform(entry(c.offsets, run.b));
        run.T = uniform(entry(c.offsets, run.b + 1)) - run.first;
        run.n = uniform(entry(c.kv_len, run.b));
        run.begin = uniform((long long)entry(c.kv_begin, run.b));
        run.tiles = All::of(run.T, run.n);
    };
    open();
    run.hk = uniform(run.t0 / run.tiles);
    run.t0 -= run.hk * run.tiles;
    Short4<C> b(lds);
    while (true) {
        run.t1 = (int)min((long long)run.tiles, run.t0 + (u1 - u));
        const bool whole = run.t1 - run.t0 == run.tiles;
        {
            const Fp4Args& f = args_again();
            const int rows = run.T * f.a.G;
            b.open(f, fp4_keys(f.cache, run.begin, run.hk), run.t0, run.t1, run.n);
            b.ask(0);
            b.take_rows(f.a, rows, run.first, run.hk);
            b.see(f.a.G, rows, run.n - run.T + 1, run.n);
        }
        if constexpr (C::QLDS) wait_and_meet<63>();
        b.run(run.t0, run.t1, run.n);
        wait_and_meet<63>();  // the sums take the place of all waves' rings
        // a worker's slot 0: a run cut at the front; slot 1: a run that starts here and goes on in the next worker
        finish_piece<C>(b, run, whole ? -1 : w * 2ll + (run.t0 == 0 ? 1 : 0));
        const Args& a = args_again().a;
        if (run.t0 == 0) {
            const int pieces = whole ? 1 : Cut(total, W).part(u + run.tiles - 1) - w + 1;
            if (a.row_info != nullptr)
                for (int i = threadIdx.x; i < run.T; i += C::NT)
                    a.row_info[(long long)(run.first + i) * a.c.HK + run.hk] = make_int2(whole ? -1 : w, pieces * 128 + i);
            if (!whole && a.cut != nullptr && threadIdx.x == 0) a.cut[w] = make_int4(run.first, run.T, run.hk, pieces);
        }
        u += run.t1 - run.t0;
        if (u >= u1) {
            if ((whole || run.t0 != 0) && a.cut != nullptr && threadIdx.x == 0) a.cut[w] = make_int4(0, 0, 0, 0);
            return;
        }
        run.t0 = 0;
        if (++run.hk == a.c.HK) {
            run.hk = 0;
            do {
                ++run.b;
                open();
            } while (run.tiles == 0);
        }
        __syncthreads();  // the piece's sums are read
    }
}

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
    int row, run_at;        // the thread's row of a tile and its run of elements there
    int kc_off, ks_off, vc_off, vs_off;
    Half k, v;

    __device__ __forceinline__ Long4(const Fp4Args& f, char* lds) : B(f.a, lds), cache(f.cache) {
        row = (int)threadIdx.x / UPR;
        run_at = (int)threadIdx.x % UPR;
        const int e = run_at * U;
        const bool in = e < f.a.c.D;
        kc_off = in ? row * (int)cache.k.codes.row + e / 2 : kOutside;
        ks_off = in ? row * (int)cache.k.scales.row + e / 32 : kOutside;
        vc_off = in ? row * (int)cache.v.codes.row + e / 2 : kOutside;
        vs_off = in ? row * (int)cache.v.scales.row + e / 32 : kOutside;
    }
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
        Half& to = V ? v : k;
        if constexpr (U == 32) {
            const u32x4 x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rc, V ? vc_off : kc_off, 0, 0));
#pragma unroll
            for (int i = 0; i < 4; ++i) to.codes[i] = x[i];
        } else {
            const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rc, V ? vc_off : kc_off, 0, 0));
            to.codes[0] = x[0], to.codes[1] = x[1];
        }
        to.scale = __builtin_amdgcn_raw_buffer_load_b8(rs, V ? vs_off : ks_off, 0, 0);
    }
    // Writes them to a stage of the ring.
    template <bool V>
    __device__ __forceinline__ void put(int stage) {
        char* at = B::lds + stage * C::STAGE + (V ? C::KTILE + C::template row_at<C::VSTEP>(row) : C::template row_at<C::KSTEP>(row));
        const int sw = V ? C::place_v(row) : C::place_k(row);
        const Half& x = V ? v : k;
        const float scale = fp4::scale_of(x.scale);
#pragma unroll
        for (int i = 0; i < U / 8; ++i) {
            if constexpr (C::HALF) {
                u32x4 w;
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = widen2<T>(x.codes[i], scale, j);
                *reinterpret_cast<u32x4*>(at + (((run_at * (U / 8) + i) ^ sw) * 16)) = w;
            } else {
                float y[8];
                fp4::values(x.codes[i], x.scale, y);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<f32x4*>(at + (((run_at * (U / 4) + 2 * i + j) ^ sw) * 16)) = f32x4{y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]};
            }
        }
    }

    // Tiles [t0, t1) of the run, as Block::run.
    template <typename F>
    __device__ __forceinline__ bool run(const Fp4Keys& s, int t0, int t1, int full, F stop) {
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
            auto one = [&](auto hidden, int at) {
                wait_and_meet<63>();
                put<false>(at ^ 1);
                put<true>(at ^ 1);
                fetch<false>(s, t + 2, t + 2 < t1);
                fetch<true>(s, t + 2, t + 2 < t1);
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
            B::template scores<true>(0, now);
            if (t0 >= full) B::hide(now, t0 * C::BN);
            top = B::largest(now);
            auto ahead = [&](int at) {
                wait_and_meet<63>();
                put<true>(at ^ 1);
                put<false>(at);
                fetch<true>(s, t + 2, t + 2 < t1);
                fetch<false>(s, t + 3, t + 3 < t1);
            };
            while (t + 2 < min(full, t1 - 1)) {
                ahead(0);
                B::template step<false, false>(0, t, now, next, top);
                ++t;
                ahead(1);
                B::template step<false, false>(1, t, next, now, top);
                ++t;
            }
            for (; t < t1 - 1; ++t) {
                ahead(stage);
                if (t >= full) B::look(B::lds + stage * C::STAGE + C::KTILE, t * C::BN);
                B::template step<true, false>(stage, t, now, next, top);
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

// One block per key head, key part and tile of BM rows, as gdn_attn.hpp's long form.
template <typename C>
__global__ __launch_bounds__(C::NT, C::WAVES) void long4_kernel(Fp4Args f) {
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

    Long4<C> blk(f, lds);
    blk.load_rows(row0, rows, first, hk);
    blk.see(row0, rows, true, seen0, n);
    const Fp4Keys keys = fp4_keys(f.cache, seq.begin, hk);
    if (t0 < t1) {
        const int full = uniform(max(0, min(n, seen0 + row0 / a.G)) / C::BN);
        if (!blk.run(keys, t0, t1, full, stop)) return;
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

// Waves of a SIMD that the registers of a configuration leave room for.
template <typename T, int DP, int RT>
struct Short4For {
    static constexpr int STATE = RT * (DP / 4 + 18) + (RT == 1 && T::code != GDN_F32 ? DP / 8 : 0) + DP / 8 + 40;
    static constexpr int WAVES = STATE <= 128 ? 4 : STATE <= 170 ? 3 : STATE <= 256 ? 2 : 1;
    template <bool WIDE>
    using C = Cfg4<T, DP, RT, WAVES, WIDE>;
};

template <typename T, int DP, typename F>
auto with_row_tiles(int rt, F f) {
    switch (rt) {
        case 1: return f(Short4For<T, DP, 1>{});
        case 2: return f(Short4For<T, DP, 2>{});
        case 3: return f(Short4For<T, DP, 3>{});
        default: return f(Short4For<T, DP, T::code == GDN_F32 && DP == 256 ? 3 : 4>{});
    }
}
template <typename T, typename F>
auto with_short4(int dp, int rt, bool wide, F f) {
    auto g = [&](auto x) {
        return wide ? f(typename decltype(x)::template C<true>{}) : f(typename decltype(x)::template C<false>{});
    };
    return dp == 64 ? with_row_tiles<T, 64>(rt, g) : dp == 128 ? with_row_tiles<T, 128>(rt, g) : with_row_tiles<T, 256>(rt, g);
}
// Rows of the short form at most: three row tiles of fp32 queries wider than 128 fill LDS, otherwise four.
template <typename T>
constexpr int short_rows(int dp) {
    return T::code == GDN_F32 && dp == 256 ? 48 : 64;
}

template <typename T>
hipError_t start_short4(const Fp4Args& f, int dp, int rt, bool wide, hipStream_t stream);

template <typename T>
hipError_t start_long4(const Fp4Args& f, int dp, long long blocks, int lds, hipStream_t stream);

template <typename C>
hipError_t start_one_long4(const Fp4Args& f, long long blocks, int lds, hipStream_t stream) {
    static std::atomic<uint64_t> asked{0};
    return start_kernel(&long4_kernel<C>, asked, f, blocks, C::NT, lds, stream);
}
template <typename C>
hipError_t start_one_short4(const Fp4Args& f, hipStream_t stream) {
    static std::atomic<uint64_t> asked{0};
    return start_kernel(&short4_kernel<C>, asked, f, f.a.workers, C::NT, C::LDS, stream);
}

#define GDN_ATTN_FP4_INSTANCES(T)                                                                                      \
    template <>                                                                                                        \
    hipError_t start_short4<T>(const Fp4Args& f, int dp, int rt, bool wide, hipStream_t stream) {                      \
        return with_short4<T>(dp, rt, wide, [&](auto c) { return start_one_short4<decltype(c)>(f, stream); });         \
    }                                                                                                                  \
    template <>                                                                                                        \
    hipError_t start_long4<T>(const Fp4Args& f, int dp, long long blocks, int lds, hipStream_t stream) {               \
        return with_long<T>(dp, [&](auto p) { return start_one_long4<typename decltype(p)::C>(f, blocks, lds, stream); }); \
    }

}  // namespace attn
}  // namespace gdn
