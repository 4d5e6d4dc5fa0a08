// gdn_attn_fp4.hip -- host side of the attention over a 4-bit cache: which form and tile a call takes and its workspace.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdn_attn_fp4.hpp"
#include "gdn_attn_join.hpp"

namespace gdn {
namespace {

using namespace attn;

// A block a run, without a joining launch, where a run takes a block few steps: the cache has at most kWholeSteps of them a
// sequence, and kWholeMost in all, as one sequence may hold nearly all of it.  The host knows the cache's rows only, not
// what sequences hold of them: one token over 1023 keys takes 8.6 us in a cache of that size, and 11 in one with room.  (H 32, HK 8, D 128, 512 keys a step: eight
// sequences of 500 keys 9.1 us, cut and joined 11.3, of 2000 keys 13.5 and 13.9, of 4000 19.6 and 16.7; one of 2000 12.9
// and 11.6, of 8000 27 and 13.5.  H 16, HK 2, D 256, 256 keys a step: one of 500 keys 10.3 and 12.2, of 2000 17.4 and 12.9.)
constexpr int kWholeSteps = 3, kWholeMost = 16;

// Whether a head's scales can be read several bytes at a time: as many heads' widths as there are kernels for have all
// their blocks, and then only where every row starts at a multiple of that.
bool wide_scales(const Fp4Cache& c, int D) {
    const int n = std::min(D / 32, 4);
    auto fits = [&](const HeadRows& x) { return reinterpret_cast<uintptr_t>(x.p) % n == 0 && x.row % n == 0 && x.head % n == 0; };
    return (D == 64 || D == 128 || D == 256) && fits(c.k.scales) && fits(c.v.scales);
}

struct Plan {
    Fp4Args f;
    bool is_short, whole, wide, join;  // whole: a block a run
    int dp, tiles, bm, lds;
    long long blocks;
    size_t bytes;
};

template <typename T>
Plan plan(const AttnLaunch& c, bool wide) {
    Plan p{};
    Args& a = p.f.a;
    a.c = c;
    a.G = c.H / c.HK;
    a.s2 = fabsf(c.scale) * kLog2e;
    a.negate = c.scale < 0.0f;
    a.splits = 1;
    a.set_rows = (long long)c.N * c.H;
    p.dp = c.D <= 64 ? 64 : c.D <= 128 ? 128 : 256;
    // Wider than 128, a key head's rows that are too many for the short form's registers are divided by query heads among so
    // many blocks that they are not: keys are read more than once, which bounds nothing there.  In half precision up to
    // 128 rows (20 sequences of 9 tokens over 3000 to 9000 keys, H 16, HK 2, D 256: 58 us, in the long form, whose tiles
    // have 256 rows, 80; at widths 128 and 64 it is 43 and 40, 18 and 16, 27 and 40); in fp32, whose long form runs on
    // fp32 matrix instructions, where 32 rows or fewer are left (26 of 7 tokens and 131 keys, H 32, HK 4, D 160: 24 and 149).
    p.f.share = 1;
    const long long all_rows = (long long)c.max_q * a.G, fit = short_rows<T>(p.dp);
    if (p.dp == 256 && all_rows > fit && (T::code == GDN_F32 || all_rows <= 128)) {
        int share = 1;
        while (share <= a.G && (a.G % share != 0 || (long long)c.max_q * (a.G / share) > fit)) ++share;
        if (share <= a.G) {
            p.f.share = share;
            a.G /= share;
            a.c.HK *= share;
        }
    }
    const long long rows = std::max(1ll, (long long)c.max_q * a.G);
    p.is_short = rows <= short_rows<T>(p.dp);
    p.wide = wide;
    p.f.g_inverse = 65536u / (uint32_t)a.G + 1;
    p.tiles = (int)std::min(rows + 15, 64ll) / 16;
    const long long step = with_whole4<T>(p.dp, wide, [](auto x) { return decltype(x)::UNIT; });
    p.whole = p.tiles == 1 && c.kv_rows <= step * std::min<long long>((long long)c.B * kWholeSteps, kWholeMost) && (long long)c.B * a.c.HK <= kCUs;
    if (p.whole) return p;
    if (p.is_short) {
        struct Tile {
            int bm, unit, per_cu;
        };
        const Tile s = with_short4<T>(p.dp, p.tiles, wide, [&](auto c) {
            using C = decltype(c);
            return Tile{C::BM, C::UNIT, std::max(1, std::min(C::WAVES * 4 / C::W, kCULds / (C::LDS + 1280)))};
        });
        p.bm = s.bm;
        const long long units = a.c.HK * (c.kv_rows / s.unit + c.B);  // fewer blocks than that have work, bar overlapping runs
        a.workers = (int)std::max(1ll, std::min((long long)kCUs * s.per_cu, units));
        p.join = c.N > 0 && a.workers > 1;
    } else {
        // Row tiles as for a plain cache.  As many key parts as leave room for all blocks at once, one a CU at width 256 and two
        // below: each part writes fp32 sums of its rows.  (Parts until every CU has two blocks or more, and now: 15 sequences
        // of 226 to 452 tokens, H 8, HK 2, D 160, 68 us and 36; four of 300 tokens and 4300 keys, H 16, HK 2, D 256, 163 and
        // 106; one of 2000, H 32, HK 8, D 128, 78 and 55.  One part wherever half of the CUs have a block: one of 700 there 25
        // instead of 29, but in fp32 one of 500 and 3500 keys 167 instead of 89.)
        const Shape s = with_long4<T>(p.dp, [](auto x) { return shape_of<typename decltype(x)::C>(); });
        p.bm = s.bm;
        p.lds = s.ring;
        const long long most = (rows + s.bm - 1) / s.bm, slots = (long long)c.N * a.G / s.bm + c.B;
        const long long tiles = std::min(most * c.B, slots) * a.c.HK;
        a.splits = (int)std::max(1ll, std::min({(p.dp == 256 ? 1 : 2) * kCUs / std::max(1ll, tiles), c.kv_rows / kPartKeys, 64ll}));
        p.blocks = slots * a.c.HK * a.splits;
        p.join = a.to_sets = a.splits > 1;
        a.sets = p.join ? a.splits : 0;
    }
    size_t at = 0;
    auto take = [&](size_t n) {
        char* r = static_cast<char*>(c.workspace) + at;
        at += (n + 255) / 256 * 256;
        return r;
    };
    if (p.join) a.status = reinterpret_cast<int*>(take(4));
    if (p.join && !p.is_short) {
        a.set_ml = reinterpret_cast<float2*>(take((size_t)a.sets * a.set_rows * 8));
        a.set_o = reinterpret_cast<float*>(take((size_t)a.sets * a.set_rows * c.D * 4));
        a.live = reinterpret_cast<int*>(take((size_t)c.N * 4));
    } else if (p.join) {
        if (few_rows(a)) a.row_info = reinterpret_cast<int2*>(take((size_t)c.N * a.c.HK * 8));
        else a.cut = reinterpret_cast<int4*>(take((size_t)a.workers * 16));
        a.slot_ml = reinterpret_cast<float2*>(take((size_t)a.workers * 2 * p.bm * 8));
        a.slot_o = reinterpret_cast<float*>(take((size_t)a.workers * 2 * p.bm * c.D * 4));
    }
    p.bytes = at;
    return p;
}

template <typename T>
hipError_t launch(const AttnLaunch& c, const Fp4Cache& cache, hipStream_t stream) {
    Plan p = plan<T>(c, wide_scales(cache, c.D));
    p.f.cache = cache;
    if (p.whole) return start_whole4<T>(p.f, p.dp, p.wide, stream);
    const hipError_t e = p.is_short ? start_short4<T>(p.f, p.dp, p.tiles, p.wide, stream) : start_long4<T>(p.f, p.dp, p.blocks, p.lds, stream);
    return e != hipSuccess || !p.join ? e : start_join<T>(p.f.a, p.bm, -1, stream);
}

}  // namespace

// Of the kernel for either way to read scales, as the query does not know the cache.
size_t attention_fp4_workspace_bytes(const AttnLaunch& c) {
    auto bytes = [&](bool wide) {
        switch (c.dtype) {
            case GDN_F32: return plan<F32>(c, wide).bytes;
            case GDN_BF16: return plan<BF16>(c, wide).bytes;
            default: return plan<F16>(c, wide).bytes;
        }
    };
    return std::max(bytes(false), bytes(true));
}

hipError_t launch_attention_fp4(const AttnLaunch& c, const Fp4Cache& cache, hipStream_t stream) {
    switch (c.dtype) {
        case GDN_F32: return launch<F32>(c, cache, stream);
        case GDN_BF16: return launch<BF16>(c, cache, stream);
        default: return launch<F16>(c, cache, stream);
    }
}

}  // namespace gdn
