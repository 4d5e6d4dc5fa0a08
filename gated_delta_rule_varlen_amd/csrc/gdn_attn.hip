// gdn_attn.hip -- host side of the softmax attention: which form and tile a call takes, its workspace, and
// when the parts of a row are joined.  The tile kernels are in gdn_attn.hpp, the joining ones in gdn_attn_join.hpp.
//
// Short form (max_q * G rows are 128 at most): decode steps and short blocks, bound by the
// cache's bytes.  Long form: prompts, bound by the matrix cores.  A shared prefix is one more run of
// keys for the long form's tiles; beside the short form, blocks of the long form run all tokens' rows over
// the prefix, reading it once for the whole batch: in a launch of their own, or for small calls in the same one
// (both_kernel).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdn_attn_join.hpp"

namespace gdn {
namespace {

using namespace attn;

constexpr int kShortRows = 128;

struct Plan {
    Args a;
    bool is_short, join, both;
    int dp, wr, bm;
    int lds, long_lds, threads, long_threads;
    long long blocks;
    size_t bytes;
};

template <typename T>
Plan plan(const AttnLaunch& c) {
    Plan p{};
    Args& a = p.a;
    a.c = c;
    a.G = c.H / c.HK;
    a.s2 = fabsf(c.scale) * kLog2e;
    a.negate = c.scale < 0.0f;
    a.splits = 1;
    a.set_rows = (long long)c.N * c.H;
    p.dp = c.D <= 64 ? 64 : c.D <= 128 ? 128 : 256;
    const long long rows = (long long)c.max_q * a.G, es = sizeof(typename T::storage);
    p.wr = rows <= 64 ? (int)(rows + 15) / 16 : 8;
    if (p.wr < 1) p.wr = 1;
    const Shape s = with_short<T>(p.dp, p.wr, Shape{0, 0, kMaxLds + 1, 0, 0}, [](auto x) { return shape_of<typename decltype(x)::C>(); });
    const Shape whole = with_long<T>(p.dp, [](auto x) { return shape_of<typename decltype(x)::C>(); });
    // the short form's queries lie in LDS beside the ring, and a run's span a 32-bit range
    const long long q_lds = (rows + 7) / 8 * 8 * s.row;
    const long double q_span = ((long double)c.max_q * c.q.row + (long double)a.G * c.q.head) * es;
    p.is_short = rows <= kShortRows && s.ring + q_lds <= kMaxLds && q_span < kOutside;
    p.long_lds = whole.ring;
    p.threads = p.long_threads = whole.threads;
    // Key parts of the long form: enough blocks for two a CU, each of kPartKeys keys at least.  The sequences' own
    // lengths are on the device: there a sequence takes as many of the parts as its keys fill.
    auto parts = [&](long long tiles, long long keys) {
        const long long want = (2 * kCUs + tiles - 1) / std::max(1ll, tiles), most = keys / kPartKeys;
        return (int)std::max(1ll, std::min(std::min(want, most), 64ll));
    };
    const long long N = c.N, all_rows = N * a.G;
    bool by_rows = true;
    if (p.is_short) {
        p.bm = s.bm;
        p.threads = s.threads;
        p.lds = (int)(s.ring + q_lds);
        if (c.prefix_len > 0 && c.N > 0) {
            const long long tiles = (all_rows + whole.bm - 1) / whole.bm;
            a.splits = parts(tiles * c.HK, c.prefix_len);
            a.prefix_blocks = tiles * c.HK * a.splits;
            a.sets = a.splits + 1;
            a.to_sets = true;
            a.local_set = a.splits;
        }
        const int per_cu = std::min(8, kCULds / ((p.lds + 1279) / 1280 * 1280));  // LDS is handed out in 1280 bytes
        const long long units = c.HK * (c.kv_rows / s.bn + c.B);  // fewer blocks than that have work, bar overlapping runs
        a.workers = (int)std::max(1ll, std::min((long long)kCUs * per_cu, units));
        p.blocks = a.workers;
        // Both forms in one launch where all blocks run at once (8 drafts behind 1001 shared keys: 12.4 us, in two
        // launches 18.7).  In more rounds the short form's blocks are too few on a CU beside the long form's
        // (256 sequences behind 8192 keys: 136 us, in two launches 130).
        p.both = a.prefix_blocks > 0 && a.prefix_blocks + a.workers <= 2 * kCUs && p.wr <= 4 && joint(whole.ring, p.lds);
        if (p.both) {
            p.lds = std::max(p.lds, whole.ring);
            p.threads = p.long_threads;
            p.blocks = ((a.prefix_blocks + kCUs - 1) / kCUs + (a.workers + kCUs - 1) / kCUs) * kCUs;  // whole turns
        }
        p.join = c.N > 0 && (a.workers > 1 || a.sets > 0);
        by_rows = a.sets > 0 || few_rows(a);
    } else {
        // One block for every slot that a row tile can have, however long max_q says that one sequence may be.  (With
        // blocks for each sequence as for the longest, one prompt of 8192 tokens among 63 of up to 200 took 1220 us,
        // so 557; max_q = N for eight prompts 756 and 680.  In the order of their keys 64 fp32 prompts of up to
        // 300 tokens take 275 us, as they come 326.)
        const long long most = (rows + whole.bm - 1) / whole.bm, slots = all_rows / whole.bm + c.B;
        a.splits = parts(std::min(most * c.B, slots) * c.HK, c.kv_rows + c.prefix_len);
        p.blocks = slots * c.HK * a.splits;
        if (a.splits > 1) {
            a.sets = a.splits;
            a.to_sets = true;
            p.join = true;
        }
    }
    size_t at = 0;
    auto take = [&](size_t n) {
        char* r = static_cast<char*>(c.workspace) + at;
        at += (n + 255) / 256 * 256;
        return r;
    };
    if (p.join) {
        a.status = reinterpret_cast<int*>(take(4));
        if (p.is_short) {
            if (by_rows) a.row_info = reinterpret_cast<int2*>(take(N * c.HK * 8));
            else a.cut = reinterpret_cast<int4*>(take((size_t)a.workers * 16));
            a.slot_ml = reinterpret_cast<float2*>(take((size_t)a.workers * 2 * p.bm * 8));
            a.slot_o = reinterpret_cast<float*>(take((size_t)a.workers * 2 * p.bm * c.D * 4));
        }
        if (a.sets > 0) {
            a.set_ml = reinterpret_cast<float2*>(take((size_t)a.sets * a.set_rows * 8));
            a.set_o = reinterpret_cast<float*>(take((size_t)a.sets * a.set_rows * c.D * 4));
            if (!p.is_short) a.live = reinterpret_cast<int*>(take(N * 4));
        }
    }
    p.bytes = at;
    return p;
}

template <typename T>
hipError_t launch(const AttnLaunch& c, hipStream_t stream) {
    Plan p = plan<T>(c);
    if (p.blocks * p.threads > kMaxThreads || p.a.prefix_blocks * p.long_threads > kMaxThreads)
        return hipErrorInvalidConfiguration;
    hipError_t e;
    if (p.is_short) {
        if (p.both) {
            e = start_both<T>(p.a, p.dp, p.wr, p.blocks, p.lds, stream);
        } else {
            if (p.a.prefix_blocks > 0 &&
                (e = start_long<T>(p.a, p.dp, p.a.prefix_blocks, p.long_lds, stream)) != hipSuccess)
                return e;
            e = start_short<T>(p.a, p.dp, p.wr, p.blocks, p.lds, stream);
        }
    } else {
        e = start_long<T>(p.a, p.dp, p.blocks, p.long_lds, stream);
    }
    if (e != hipSuccess || !p.join) return e;
    const int local = p.is_short && p.a.sets > 0 ? p.a.local_set : -1;
    return start_join<T>(p.a, p.bm, local, stream);
}

}  // namespace

size_t attention_workspace_bytes(const AttnLaunch& c) {
    switch (c.dtype) {
        case GDN_F32: return plan<F32>(c).bytes;
        case GDN_BF16: return plan<BF16>(c).bytes;
        default: return plan<F16>(c).bytes;
    }
}

hipError_t launch_attention(const AttnLaunch& c, hipStream_t stream) {
    switch (c.dtype) {
        case GDN_F32: return launch<F32>(c, stream);
        case GDN_BF16: return launch<BF16>(c, stream);
        default: return launch<F16>(c, stream);
    }
}

}  // namespace gdn
