// Tree attention over a prefix the batch shares, and with transformed scores:
// the work's cutting into items, shared by the kernels that compute the items
// and the kernel that joins them.
//
// Query rows of one (sequence, KV head): its g query heads x T nodes, gT rows,
// contiguous in q [B, Hq, T, D].  Two kinds of columns:
//   own     one (sequence, KV head, block of RB rows) against the sequence's
//           cached keys and its tree keys
//   shared  one (KV head, block of RB rows) against the shared keys; here a block
//           holds the rows of as many whole sequences as fit (nbb of them), so
//           that a shared key is read once for all of those
// Every column's key tiles (KT keys each) are cut into splits of about `chunk`
// tiles, one item each.  The cut follows the lengths, which only the device
// knows: a warp of every CTA reads them and works out the same Plan.  An item
// leaves (max, sum, unnormalised O) of its rows in its own part of the
// workspace; the join merges a row's items.  A row that has a single item gets
// its output from there directly.
#pragma once

#include "attention_tc.cuh"
#include "common.cuh"

namespace spec {
namespace shr {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
    int B, T, g, gT, Hq, Hkv, D, words;
    int Lshared, Lmax;                 // capacities
    int RB, KT;                        // rows of a block, keys of a tile
    int nbb, n_rbO, n_rbS, rowsO, rowsS;
    int ctas, max_extra;               // CTAs the plan fills; bound on splits beyond one per column
    float fixed;                       // cost of an item beyond its tiles, in tiles
    float scale, softcap;              // softcap 0: none
    int window;                        // 0: none
    const float* slopes;               // [Hq] or NULL
    const int32_t* prefix_len;         // [B]
    const int32_t* shared_len;         // [1]; NULL: nothing shared
    const int32_t* depth;
    const uint64_t* anc;
    tc::KvPages pg;                    // own pages; table NULL: contiguous
    const int32_t* shared_table;       // shared pages when pg.table is set
    const void *q, *kc, *vc, *ks, *vs, *kt, *vt;
    void* out;
    float* lse;
    void* ws;                          // status word, then the Plan, then cum [B + 1], then the items
    int32_t* cum;                      // splits of the sequences before b, one column each
    float4 *part_s, *part_o;           // items: [D / 4 + 1][rows] float4: (m, l, -, -), then O
};

struct Plan {
    int Ls;          // shared keys
    int sT0, nS;     // first shared tile any row sees, and how many from there
    int chunk;       // tiles of a split, at most
    int nsS;         // splits of a shared column
    int itemsS, items;
};

constexpr int kPlanOffset = 64;        // bytes into the workspace header
static_assert(kPlanOffset + sizeof(Plan) <= kWsHeader, "the plan fits in the header");

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Tiles of sequence length L that its root (the node that looks furthest back) sees.
__device__ __forceinline__ int own_first(const Params& p, int L) {
    return p.window > 0 ? max(0, L - p.window + 1) / p.KT : 0;
}
__device__ __forceinline__ int own_tiles(const Params& p, int L) {   // with the tree's
    return max(0, ceil_div(L, p.KT) - own_first(p, L)) + ceil_div(p.T, p.KT);
}
__device__ __forceinline__ int own_len(const Params& p, int b) { return min(max(p.prefix_len[b], 0), p.Lmax); }

// A whole warp works out the plan (every lane gets it).  Cost of a cut with splits of c tiles,
// W tiles in all: if it has at most one item per CTA, c + fixed; else the items are handed out
// as CTAs get free, W / ctas tiles and fixed * items / ctas beside them, and half an item at the end.
__device__ __forceinline__ Plan make_plan(const Params& p) {
    const int lane = threadIdx.x & 31;
    long long own = 0;
    int longest = 0, least = 0x7fffffff;
    for (int b = lane; b < p.B; b += 32) {
        const int L = own_len(p, b), n = own_tiles(p, L);
        own += n;
        longest = max(longest, n);
        least = min(least, L);
    }
    for (int o = 16; o > 0; o >>= 1) {
        own += __shfl_xor_sync(0xffffffffu, own, o);
        longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
        least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    }
    Plan t;
    t.Ls = p.shared_len ? min(max(*p.shared_len, 0), p.Lshared) : 0;
    t.sT0 = p.window > 0 ? max(0, t.Ls + least - p.window + 1) / p.KT : 0;
    t.nS = max(0, ceil_div(t.Ls, p.KT) - t.sT0);
    const int colsS = p.Hkv * p.n_rbS, colsO = p.Hkv * p.n_rbO;
    const long long W = static_cast<long long>(colsS) * t.nS + own * colsO;
    const long long cols = (t.nS ? colsS : 0) + static_cast<long long>(p.B) * colsO;
    longest = max(longest, t.nS);
    const int floor_c = static_cast<int>((W + p.max_extra - 1) / p.max_extra);   // bounds the items
    // 32 candidates at even distances up to the longest column
    int c = max(floor_c, static_cast<int>((static_cast<long long>(longest) * (lane + 1) + 31) / 32));
    // about W / c + cols / 2 items; the last candidate cuts nothing
    const float items = lane == 31 ? static_cast<float>(cols) : fmaxf(static_cast<float>(W) / c + 0.5f * cols, static_cast<float>(cols));
    const float n = static_cast<float>(p.ctas);
    float cost = items <= n ? c + p.fixed : (static_cast<float>(W) + p.fixed * items) / n + 0.5f * (c + p.fixed);
    for (int o = 16; o > 0; o >>= 1) {
        const float c2 = __shfl_xor_sync(0xffffffffu, cost, o);
        const int k2 = __shfl_xor_sync(0xffffffffu, c, o);
        if (c2 < cost || (c2 == cost && k2 > c)) { cost = c2; c = k2; }
    }
    t.chunk = max(c, 1);
    t.nsS = ceil_div(t.nS, t.chunk);
    t.itemsS = colsS * t.nsS;
    int ns = 0;
    for (int b = lane; b < p.B; b += 32) ns += ceil_div(own_tiles(p, own_len(p, b)), t.chunk);
    for (int o = 16; o > 0; o >>= 1) ns += __shfl_xor_sync(0xffffffffu, ns, o);
    t.items = t.itemsS + ns * colsO;
    return t;
}

// The plan and the sequences' split offsets, for the join: one warp of the grid writes them.
__device__ __forceinline__ void publish_plan(const Params& p, const Plan& t) {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        const int n = b < p.B ? ceil_div(own_tiles(p, own_len(p, b)), t.chunk) : 0;
        int at = n;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += y;
        }
        if (b < p.B) p.cum[b] = before + at - n;
        before += __shfl_sync(0xffffffffu, at, 31);
    }
    if (lane == 0) {
        p.cum[p.B] = before;
        *reinterpret_cast<Plan*>(static_cast<unsigned char*>(p.ws) + kPlanOffset) = t;
    }
}

struct Item {
    int shared;      // against the shared keys
    int b;           // sequence (of the block's first row)
    int kvh, rb;     // KV head; block of rows within the sequence's gT
    int rows;        // rows of the block, over all its sequences
    int L;           // the sequence's cached keys (own items)
    int t0, t1;      // tiles [t0, t1) of the column: own ones count from own_first, the tree's last
    int index;       // among the items of its kind
    int direct;      // the rows' only item: write their output
};

// Item number `id`; a whole warp, every lane gets it.
__device__ __forceinline__ Item find_item(const Params& p, const Plan& t, int id) {
    const int lane = threadIdx.x & 31;
    Item it;
    if (id < t.itemsS) {
        const int col = id / t.nsS, split = id - col * t.nsS;
        const int sb = col % p.n_rbS;
        it.shared = 1;
        it.kvh = col / p.n_rbS;
        it.b = p.gT >= p.RB ? sb / p.n_rbO : sb * p.nbb;
        it.rb = p.gT >= p.RB ? sb % p.n_rbO : 0;
        it.rows = p.gT >= p.RB ? min(p.RB, p.gT - it.rb * p.RB) : min(p.nbb, p.B - it.b) * p.gT;
        it.L = 0;
        it.t0 = static_cast<int>(static_cast<long long>(t.nS) * split / t.nsS);
        it.t1 = static_cast<int>(static_cast<long long>(t.nS) * (split + 1) / t.nsS);
        it.index = id;
        it.direct = 0;
        return it;
    }
    const int cols = p.Hkv * p.n_rbO;
    const int at = (id - t.itemsS) / cols;      // number of the split over all sequences, one column each
    int before = 0;
    for (int b0 = 0;; b0 += 32) {
        const int b = b0 + lane;
        const int L = b < p.B ? own_len(p, b) : 0;
        const int tiles = b < p.B ? own_tiles(p, L) : 0;
        const int n = ceil_div(tiles, t.chunk);
        int end = n;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, at < before + end);
        if (hit || b0 + 32 >= p.B) {
            const int l = hit ? __ffs(hit) - 1 : 31;
            const int first = before + __shfl_sync(0xffffffffu, end - n, l);
            const int ns = __shfl_sync(0xffffffffu, n, l), tl = __shfl_sync(0xffffffffu, tiles, l);
            // items of one sequence: (KV head, block, split); the splits of all columns of the
            // sequences before it come first
            const int r = (id - t.itemsS) - first * cols;
            const int col = r / ns, split = r - col * ns;
            it.shared = 0;
            it.b = b0 + l;
            it.L = __shfl_sync(0xffffffffu, L, l);
            it.kvh = col / p.n_rbO;
            it.rb = col % p.n_rbO;
            it.rows = min(p.RB, p.gT - it.rb * p.RB);
            it.t0 = static_cast<int>(static_cast<long long>(tl) * split / ns);
            it.t1 = static_cast<int>(static_cast<long long>(tl) * (split + 1) / ns);
            it.index = id - t.itemsS;
            it.direct = t.nsS + ns == 1;
            return it;
        }
        before += __shfl_sync(0xffffffffu, end, 31);
    }
}

// The row of q and out that row r of the item's block is.
__device__ __forceinline__ size_t row_of_q(const Params& p, const Item& it, int r) {
    const int b = it.b + (p.gT < p.RB ? r / p.gT : 0);
    const int i = p.gT < p.RB ? r % p.gT : it.rb * p.RB + r;
    return (static_cast<size_t>(b) * p.Hq + it.kvh * p.g) * p.T + i;
}

// ---------------------------------------------------------------- host

struct HostPlan {
    bool tc;
    size_t cum_off, part_s_off, part_o_off, total;
};

// Fills the shape fields of p that follow from the sizes, and the workspace layout.
HostPlan host_plan(Params& p, bool tc, bool shared, int ctas);

// The tensor-core items (bf16, D 64 or 128).
spec_status attn_shared_tc_run(const Params& p, int blocks, cudaStream_t s);

}  // namespace shr
}  // namespace spec
