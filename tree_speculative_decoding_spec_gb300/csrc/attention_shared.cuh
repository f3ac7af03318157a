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
// All columns' key tiles (64 keys each) are laid end to end, each as long as its cost, each
// column led by what an item costs beside its tiles, and the line is cut into equal
// parts, one per CTA; a column that a cut crosses is that many items more.  So the CTAs finish
// together, with one split per CTA more than there are columns (cutting every column
// into equal splits left the last round of them part empty: 306 tiles on the longest of
// 152 CTAs where the mean was 233).  The cut follows the lengths, which only the device
// knows: a warp of every CTA reads them and works out the same line.  An item leaves
// (max, sum, unnormalised O) of its rows in its own part of the workspace; the join
// merges a row's items.  A row that has a single item gets its output from there directly.
#pragma once

#include "attention_tc.cuh"
#include "common.cuh"

namespace spec {
namespace shr {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kTile = 64;       // keys of a tile
constexpr int kTcRows = 256;    // rows of a block, tensor-core items

struct Params {
    int B, T, g, gT, Hq, Hkv, D, words;
    int Lshared, Lmax;                 // capacities
    int RB;                            // rows of a block
    int nbb, n_rbO, n_rbS, rowsO, rowsS;
    int ctas;                          // parts of the line
    int per;                           // blocks of one sequence's rows a shared column may be one of (1 when it holds whole sequences)
    // a tile's cost and an item's beside its tiles: blocks with more rows behind them, the last (or only) one
    int wF, wS, wO, fixF, fixS, fixO;
    int tailF, tailO;                  // of an own column's partial tile and its tree's masks, behind its tiles
    int min_piece;                     // tiles of the shortest split
    int repS, repO;                    // copies of a row in an item (see attention_shared_tc.cu)
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
    void* ws;                          // status word and Plan, the CTAs' statuses, cum [B], the items
    int32_t* cta_status;               // [ctas]
    int32_t* cum;                      // place on the line of each sequence's first column [B]
    float4 *part_s, *part_o;           // items: [D / 4 + 1][rows] float4: (m, l, -, -), then O
};

struct Plan {
    int Ls;          // shared keys
    int sT0, nS;     // first shared tile any row sees, and how many from there
    int q;           // length of a CTA's part of the line
    int colsS;       // shared columns on the line
    int own0;        // place of the own columns
};

constexpr int kPlanOffset = 64;        // bytes into the workspace header
static_assert(kPlanOffset + sizeof(Plan) <= kWsHeader, "the plan fits in the header");

// A division is some forty instructions; the scheduling code runs once per item, cold, and its
// length is what it costs.
static __device__ __noinline__ int divide(int a, int b) { return a / b; }
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }

// Tiles of sequence length L that its root (the node that looks furthest back) sees.
__device__ __forceinline__ int own_first(const Params& p, int L) {
    return p.window > 0 ? max(0, L - p.window + 1) / kTile : 0;
}
__device__ __forceinline__ int own_tiles(const Params& p, int L) {   // with the tree's
    return max(0, tiles_of(L) - own_first(p, L)) + tiles_of(p.T);
}
__device__ __forceinline__ int own_len(const Params& p, int b) { return min(max(p.prefix_len[b], 0), p.Lmax); }

// Place of column c (of those with `per` blocks to a group of rows) relative to the first, n tiles each.
struct Place {
    int full, group;   // length of a full block's column; of a group
    int w, fix, n;     // of the last block's
    __device__ __forceinline__ Place(const Params& p, bool shared, int n_) : n(n_) {
        w = shared ? p.wS : p.wO;
        fix = shared ? p.fixS : p.fixO;
        full = n * p.wF + p.fixF + (shared ? 0 : p.tailF);
        group = ((shared ? p.per : p.n_rbO) - 1) * full + n * w + fix + (shared ? 0 : p.tailO);
    }
};

// A whole warp works out the plan (every lane gets it).
__device__ __forceinline__ Plan make_plan(const Params& p) {
    int own = 0, least = 0x7fffffff;
    for (int b = threadIdx.x & 31; b < p.B; b += 32) {
        const int L = own_len(p, b);
        own += Place(p, false, own_tiles(p, L)).group;
        least = min(least, L);
    }
    for (int o = 16; o > 0; o >>= 1) {
        own += __shfl_xor_sync(0xffffffffu, own, o);
        least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    }
    Plan t;
    t.Ls = p.shared_len ? min(max(*p.shared_len, 0), p.Lshared) : 0;
    t.sT0 = p.window > 0 ? max(0, t.Ls + least - p.window + 1) / kTile : 0;
    t.nS = max(0, tiles_of(t.Ls) - t.sT0);
    t.colsS = t.nS ? p.Hkv * p.n_rbS : 0;
    t.own0 = t.nS ? Place(p, true, t.nS).group * p.Hkv * divide(p.n_rbS, p.per) : 0;
    const int total = t.own0 + own * p.Hkv;
    t.q = max(divide(total + p.ctas - 1, p.ctas), p.fixF + p.wF * p.min_piece);
    return t;
}

// The items of column c of those with n tiles, `first` the place of column 0: the line is cut at
// multiples of q, save where less than min_piece tiles of the column would be left on one side.
// Item k belongs to CTA owner + k.
struct Cuts {
    int owner, count, base, q, w, n;
    __device__ __forceinline__ Cuts(const Params& p, int q_, const Place& pl, int first, int c, int per) : q(q_), n(pl.n) {
        const int g = per == 1 ? c : divide(c, per), r = c - g * per;
        const bool last = r == per - 1;
        w = last ? pl.w : p.wF;
        base = first + g * pl.group + r * pl.full + (last ? pl.fix : p.fixF);      // place of the column's first tile
        const int i0 = min(divide(base + p.min_piece * w + q - 1, q), p.ctas);      // first cut
        const int i1 = divide(max(base + (n - p.min_piece) * w, 0), q);             // last cut
        owner = i0 - 1;
        count = max(0, i1 - i0 + 1) + 1;
    }
    __device__ __forceinline__ int tile(int place) const { return divide(place - base, w); }
    __device__ __forceinline__ int begin(int k) const { return k == 0 ? 0 : tile((owner + k) * q); }
    __device__ __forceinline__ int end(int k) const { return k == count - 1 ? n : tile((owner + k + 1) * q); }
    // the workspace slot among `cols` columns: one per column, one per cut of the line
    __device__ __forceinline__ int slot(int col, int cols, int k) const { return k == 0 ? col : cols + owner + k; }
};

// The plan and the sequences' places, for the join: one warp of the grid writes them.
__device__ __forceinline__ void publish_plan(const Params& p, const Plan& t) {
    const int lane = threadIdx.x & 31;
    int before = t.own0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        const int n = b < p.B ? Place(p, false, own_tiles(p, own_len(p, b))).group * p.Hkv : 0;
        int at = n;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += y;
        }
        if (b < p.B) p.cum[b] = before + at - n;
        before += __shfl_sync(0xffffffffu, at, 31);
    }
    if (lane == 0) *reinterpret_cast<Plan*>(static_cast<unsigned char*>(p.ws) + kPlanOffset) = t;
}

struct Item {
    int shared;      // against the shared keys
    int b;           // sequence (of the block's first row)
    int kvh, rb;     // KV head; block of rows within the sequence's gT
    int rows;        // rows of the block, over all its sequences
    int L;           // the sequence's cached keys (own items)
    int t0, t1;      // tiles [t0, t1) of the column: own ones count from own_first, the tree's last
    int index;       // workspace slot among those of its kind
    int direct;      // the rows' only item: write their output
};

// The items of one CTA in the line's order; a whole warp, every lane gets them.
struct Walk {
    int cta, colS;             // next shared column
    int b, base, col, L, n;    // next own column: sequence, place of its first column, column, keys, tiles
    __device__ __forceinline__ Walk(const Params& p, const Plan& t, int cta_) : cta(cta_) {
        const int lane = threadIdx.x & 31;
        const int x = max(0, cta * t.q - p.fixF - p.wF * p.min_piece);   // no earlier column has an item here
        colS = t.nS ? min(divide(x, Place(p, true, t.nS).group) * p.per, t.colsS) : 0;
        b = p.B;
        base = t.own0;
        col = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int i = b0 + lane;
            const int Li = i < p.B ? own_len(p, i) : 0;
            const int ni = i < p.B ? own_tiles(p, Li) : 0;
            const int w = i < p.B ? Place(p, false, ni).group * p.Hkv : 0;
            int end = w;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end += y;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, i < p.B && x < base + end);
            if (hit) {
                const int l = __ffs(hit) - 1;
                b = b0 + l;
                base += __shfl_sync(0xffffffffu, end - w, l);
                L = __shfl_sync(0xffffffffu, Li, l);
                n = __shfl_sync(0xffffffffu, ni, l);
                col = divide(max(0, x - base), Place(p, false, n).group) * p.n_rbO;
                break;
            }
            base += __shfl_sync(0xffffffffu, end, 31);
        }
    }
    __device__ __forceinline__ bool next(const Params& p, const Plan& t, Item& it) {
        for (; colS < t.colsS;) {
            const int c = colS++;
            const Cuts k(p, t.q, Place(p, true, t.nS), 0, c, p.per);
            if (k.owner > cta) return false;
            if (k.owner + k.count <= cta) continue;
            const int i = cta - k.owner;
            it.shared = 1;
            it.kvh = divide(c, p.n_rbS);
            const int sb = c - it.kvh * p.n_rbS;
            it.b = p.gT >= p.RB ? divide(sb, p.n_rbO) : sb * p.nbb;
            it.rb = p.gT >= p.RB ? sb - it.b * p.n_rbO : 0;
            it.rows = p.gT >= p.RB ? min(p.RB, p.gT - it.rb * p.RB) : min(p.nbb, p.B - it.b) * p.gT;
            it.L = 0;
            it.t0 = k.begin(i);
            it.t1 = k.end(i);
            it.index = k.slot(c, p.Hkv * p.n_rbS, i);
            it.direct = 0;
            return true;
        }
        const int cols = p.Hkv * p.n_rbO;
        while (b < p.B) {
            if (col == cols) {
                base += p.Hkv * Place(p, false, n).group;
                col = 0;
                if (++b == p.B) break;
                L = own_len(p, b);
                n = own_tiles(p, L);
                continue;
            }
            const int c = col++;
            const Cuts k(p, t.q, Place(p, false, n), base, c, p.n_rbO);
            if (k.owner > cta) return false;
            if (k.owner + k.count <= cta) continue;
            const int i = cta - k.owner;
            it.shared = 0;
            it.b = b;
            it.L = L;
            it.kvh = divide(c, p.n_rbO);
            it.rb = c - it.kvh * p.n_rbO;
            it.rows = min(p.RB, p.gT - it.rb * p.RB);
            it.t0 = k.begin(i);
            it.t1 = k.end(i);
            it.index = k.slot(b * cols + c, p.B * cols, i);
            it.direct = t.nS == 0 && k.count == 1 && p.repO == 1;
            return true;
        }
        return false;
    }
};

// The row of q and out that row r of the item's block is.
__device__ __forceinline__ size_t row_of_q(const Params& p, const Item& it, int r) {
    const int b = it.b + (p.gT < p.RB ? r / p.gT : 0);
    const int i = p.gT < p.RB ? r % p.gT : it.rb * p.RB + r;
    return (static_cast<size_t>(b) * p.Hq + it.kvh * p.g) * p.T + i;
}

// ---------------------------------------------------------------- host

struct HostPlan {
    bool tc;
    size_t status_off, cum_off, part_s_off, part_o_off, total;
};

// Fills the shape fields of p that follow from the sizes, and the workspace layout.
HostPlan host_plan(Params& p, bool tc, bool shared, int ctas);

// The tensor-core items (bf16, D 64 or 128).
spec_status attn_shared_tc_run(const Params& p, int blocks, cudaStream_t s);

}  // namespace shr
}  // namespace spec
