// Tensor-core (tcgen05) items of the shared-prefix and scored tree attention:
// bf16, head dim 64 or 128.
//
// One persistent CTA per SM takes items of the cut that attention_shared.cuh
// describes: up to 256 query rows against a range of 64-key tiles.  Twelve warps:
//   warp 11      schedule: works out the plan and puts its CTA's items into a ring of
//                descriptors that the other roles read
//   warp 8       TMA: the item's Q rows, then its K and V tiles into a ring that runs
//                on across items
//   warps 9, 10  MMA, one thread each, thread g for softmax group g
//   warps 0-3 / 4-7: two softmax groups, one thread per query row
// Key tiles are 64 keys long where the work is cut; there are two ways through an item:
//   pair (more than 128 rows): group g owns rows 128 g .. and takes every tile, two of
//     them at a time (128 keys), so one K/V tile in shared memory serves 256 rows and L2
//     carries half the bytes that two 128-row CTAs would read.  S is M 128, N 128: a
//     product with both operands in shared memory reads A again for every 128 x N, and at
//     N 64 takes as long as at N 128 (measured: 8 products 500 cycles either way).
//   narrow (at most 128 rows, bound by memory): both groups work on the same rows and take
//     alternate 64-key tiles; each group has two score buffers, so that S of its next tile
//     runs while it works on this one, and small tiles keep more loads in flight.  At the
//     item's end the groups exchange (max, sum) and each joins half the columns of both O.
//     At most 32 rows (single tokens above all) are there four times, once for each warp's
//     TMEM lanes: warp w takes keys 16 w .. of a tile, weights of the others stay zero in
//     its lanes, and each copy leaves its own (max, sum, O).  A warp's chain per tile is
//     that of 16 scores instead of 64 with three warps idle (1900 cycles, more than a
//     tile takes to arrive).
// Per tile and group: S = Q K^T into the group's score buffer; the softmax thread reads
// its row, transforms and masks it, keeps the running maximum and sum in base 2 and 32
// bits and writes P as bf16 pairs over the first half of the buffer; O += P V with P read
// from TMEM.  P is rounded to bf16 because the product takes both operands in one type
// and V is bf16; the sum is taken before the rounding.
// A thread's MMAs run in issue order, so an S may overwrite the buffer an earlier PV
// reads.  O is rescaled only when a row's maximum grows by more than 2^8, once the
// group's previous PV is complete (in a pair S complete says so; a narrow item waits).
// V rows that no row sees (past the lengths, past the tree) are zeroed before PV reads
// them: their weight is zero, but zero times a stale infinity is not.
// The ring's stages hold K and V of one narrow tile, or K or V of one pair tile, so both
// kinds of item run through the same ring.  Barrier phases that one of the MMA threads
// skips (it has no part in a tile) are behind it by construction: landing barriers are
// used every second round of the stages, and both threads pass q_full and o_empty at every
// item.
// Waits are bounded (2 s); on expiry SPEC_ETIMEOUT goes to the status word, every
// role leaves its loops, and the CTA drains its own loads and MMAs before it
// frees TMEM.
#include <algorithm>
#include <cstring>

#include "attention_shared.cuh"
#include "tc.cuh"

namespace spec {
namespace shr {

using namespace tc;

constexpr int kRows = 128;        // query rows of a group (MMA M)
constexpr int kBlock = kTcRows;   // of a block: two groups
constexpr int kKeys = kTile;    // keys of a tile
constexpr int kThreads = 384;
constexpr int kItems = 4;         // item descriptors in flight
constexpr int kQHalf = kBlock * 128;    // bytes of a 64-column half of the Q block
constexpr int kHalf = kKeys * 128;      // of a 64-key tile; a 128-key tile's is twice that

template <int D> struct Cfg {
    static constexpr int kH = D / 64;                      // 64-column halves
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int kFull = 2 * kStages;              // landing barriers
    static constexpr int kQ = kH * kQHalf;
    static constexpr int kStage = 2 * kH * kHalf;          // K, then V of 64 keys; K or V of 128
    static constexpr int kBars = 5 + 4 + 4 + 2 + 2 + 2 + kFull + kStages + 2 * kItems;
    static constexpr int kExchange = 512 + kItems * 64;    // barriers and flags, descriptors
    static constexpr int kSmem = kQ + kStages * kStage + kExchange + 2 * kRows * 8;
};
constexpr uint32_t kTmemCols = 512;   // scores of group g at 128 g (narrow: buffer b at 128 g + 64 b); O of group g at 256 + D g
constexpr uint32_t kO = 256;

struct Maps {
    CUtensorMap q_own, q_shared, kc, vc, ks, vs, kt, vt;
};

// One lane of the warp, the same at every call, as a condition the compiler knows to be uniform:
// the issuing code around the products comes out a third shorter than behind lane == 0.
__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// What the roles need to know of an item, 64 bytes.
struct Desc {
    int valid, shared, pair, direct;
    int b, kvh, rb, rows;
    int first, n_pre, end, Ls;     // first key tile, tiles before the tree's, keys before the tree's, shared keys
    int t0, tiles, index, L;
};
static_assert(sizeof(Desc) == 64, "four descriptors");

// The tiles of an item as its way through counts them: `width` 64-key tiles at a time, none
// across the border between prefix and tree.
struct Tiles {
    int width, pre, count;   // tiles of the prefix, tiles in all
    __device__ __forceinline__ explicit Tiles(const Desc& it) {
        width = it.pair ? 2 : 1;
        const int n_pre = min(max(it.n_pre - it.t0, 0), it.tiles);
        pre = (n_pre + width - 1) / width;
        count = pre + (it.tiles - n_pre + width - 1) / width;
    }
};
struct Tile {
    bool tree;
    int k0, nvalid;          // first key (of the source's), keys that any row can see
    // in the order they are worked off: from the item's end, where a bias by distance is largest (the
    // other way a row's maximum grows, and O is rescaled, at every tile)
    __device__ __forceinline__ Tile(const Params& p, const Desc& it, const Tiles& ts, int back) {
        const int j = ts.count - 1 - back;
        tree = j >= ts.pre;
        const int first = tree ? max(it.t0 - it.n_pre, 0) + (j - ts.pre) * ts.width : it.first + it.t0 + j * ts.width;
        // a pair tile ends with the item's part of the column
        const int last = tree ? it.t0 + it.tiles - it.n_pre : it.first + min(it.t0 + it.tiles, it.n_pre);
        k0 = first * kKeys;
        nvalid = min(min(ts.width, last - first) * kKeys, (tree ? p.T : it.end) - k0);
    }
};

// Wait for a phase, bounded (2 s, or another role's abort).  The clock is read only now and then:
// most waits here are short, and reading it takes as long as they do.
static __device__ __noinline__ bool slow_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    uint64_t t0 = 0;
    for (uint32_t i = 1; !mbar_try_wait_hint(bar, parity, 20000u); ++i) {
        if ((i & 15u) == 0) {
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (*abort_flag || now - t0 > 2000000000ull) return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return mbar_try_wait(bar, parity) || slow_wait(bar, parity, abort_flag);
}
// The same by a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort_flag));
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One query row's place: position, slope (times log2 e), ancestor words.
struct Row {
    bool in;
    int pos;
    float slope2;
    const uint64_t* anc;
};

__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[16]) { tmem_ld16(addr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[32]) { tmem_ld32(addr, r); }

// 64 scores of the thread's row, from TMEM and back.
__device__ __forceinline__ void load64(uint32_t addr, float (&x)[64]) {
    uint32_t r0[32], r1[32];
    tmem_ld32(addr, r0);
    tmem_ld32(addr + 32, r1);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        x[e] = __uint_as_float(r0[e]);
        x[e + 32] = __uint_as_float(r1[e]);
    }
}
__device__ __forceinline__ void store64(uint32_t addr, const float (&x)[64]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t r[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(x[16 * q + e]);
        tmem_st16(addr + 16 * q, r);
    }
}
__device__ __forceinline__ float max64(const float (&x)[64]) {
    float m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        m[e] = fmax3(fmax3(x[e], x[e + 8], x[e + 16]), fmax3(x[e + 24], x[e + 32], x[e + 40]), fmaxf(x[e + 48], x[e + 56]));
    return fmax3(fmax3(m[0], m[1], m[2]), fmax3(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
}

__device__ __forceinline__ float absmax64(const float (&x)[64]) {
    float m[8];
    auto a = [&](int e) { return fabsf(x[e]); };
#pragma unroll
    for (int e = 0; e < 8; ++e)
        m[e] = fmax3(fmax3(a(e), a(e + 8), a(e + 16)), fmax3(a(e + 24), a(e + 32), a(e + 40)), fmaxf(a(e + 48), a(e + 56)));
    return fmax3(fmax3(m[0], m[1], m[2]), fmax3(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
}

// 2^arg(x) of 64 scores, two at a time, as bf16 pairs to TMEM; returns their sum before the rounding.
template <typename Arg>
__device__ __forceinline__ float weigh64(const float (&x)[64], uint32_t addr, Arg arg) {
    unsigned long long acc2 = pk2(0.f, 0.f);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t packed[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            const int e = 16 * q + 2 * h;
            float x0, x1;
            upk2(arg(pk2(x[e], x[e + 1])), x0, x1);
            const float a0 = ex2(x0), a1 = ex2(x1);
            acc2 = fadd2(acc2, pk2(a0, a1));
            const __nv_bfloat162 pr = __floats2bfloat162_rn(a0, a1);   // .x (lower key) low
            packed[h] = *reinterpret_cast<const uint32_t*>(&pr);
        }
        tmem_st8(addr + 8 * q, packed);
    }
    float acc0, acc1;
    upk2(acc2, acc0, acc1);
    return acc0 + acc1;
}

// cap2 tanh(s k) of raw scores s, cap2 = softcap log2 e, k = scale / softcap.  Where the whole warp's
// |s k| stay small (caps sit far above ordinary scores) by tanh(u) = u (1 + u^2 P(u^2)): P of degree 1
// up to |u| = 0.16 and of degree 4 up to 0.7, fitted by weighted least squares whose weights are
// iterated towards an even relative error, 3.5e-8 and 1.6e-8 at most; on the FMA units that the softmax
// leaves idle, and the last product is the exponent's: s (cap2 k (1 + ...)) - reference.  Else as
// cap2 (1 - 2 / (e^(2u) + 1)), two special-function operations a score, the pipe the exponentials need.
struct Cap {
    float k, cap2, scale2;
    __device__ __forceinline__ explicit Cap(const Params& p) : k(p.scale / p.softcap), cap2(p.softcap * kLog2e), scale2(p.scale * kLog2e) {}
    __device__ __forceinline__ float operator()(float s) const { return fmaf(-2.f * cap2, rcp(ex2(s * (2.f * kLog2e * k)) + 1.f), cap2); }
    // the largest |s k| of the warp's rows; what stale memory made of others must not choose the way, or
    // results would vary with it
    __device__ __forceinline__ bool below(float most, float limit, bool in) const {
        return k < 100.f && __all_sync(0xffffffffu, !in || most * k <= limit);
    }
    struct Small {
        unsigned long long p0, p1, sc;
        __device__ __forceinline__ explicit Small(const Cap& c) {
            const float z = c.k * c.k, c0 = -0.33331832037990994f * z * c.scale2, c1 = 0.13143139243852983f * z * z * c.scale2;
            p0 = pk2(c0, c0), p1 = pk2(c1, c1), sc = pk2(c.scale2, c.scale2);
        }
        __device__ __forceinline__ unsigned long long factor(unsigned long long v) const {
            const unsigned long long w = ffma2(v, v, pk2(0.f, 0.f));
            return ffma2(w, ffma2(w, p1, p0), sc);
        }
    };
    struct Middle {
        unsigned long long p0, p1, p2, p3, p4, sc;
        __device__ __forceinline__ explicit Middle(const Cap& c) {
            const float z = c.k * c.k, z2 = z * z, s = c.scale2;
            const float c0 = -0.33333189899901133f * z * s, c1 = 0.13329110734967342f * z2 * s, c2 = -0.053558861130687065f * z2 * z * s,
                        c3 = 0.02009196966007083f * z2 * z2 * s, c4 = -0.005138661857974488f * z2 * z2 * z * s;
            p0 = pk2(c0, c0), p1 = pk2(c1, c1), p2 = pk2(c2, c2), p3 = pk2(c3, c3), p4 = pk2(c4, c4), sc = pk2(s, s);
        }
        __device__ __forceinline__ unsigned long long factor(unsigned long long v) const {
            const unsigned long long w = ffma2(v, v, pk2(0.f, 0.f));
            return ffma2(w, ffma2(w, ffma2(w, ffma2(w, ffma2(w, p4, p3), p2), p1), p0), sc);
        }
    };
};

// A tile's maximum `tmax` joins the row's.  The reference moves only when it grew by more than 2^8, and
// to a whole number: what was weighed against the old one is then off by a power of two, and O and the
// `p_cols` columns of weights at p_addr (the tile's first half, not yet given to PV) are rescaled
// without rounding.  The TMEM accesses are the whole warp's, so its rows rescale together (by 1 where
// nothing grew).
// o_cols: columns of O, 0 in an item's first tile.  Its first PV overwrites what O holds until then, which
// is the last item's, and the other group may still be reading it: only PV waits for o_empty.
__device__ __forceinline__ bool grow(float tmax, bool in, float& m_used, float& l, uint32_t o_addr, int o_cols, uint32_t p_addr,
                                     int p_cols, uint64_t* pv_bar, uint32_t pv_parity, volatile int* abort_flag) {
    float m_new = m_used, alpha = 1.f;
    bool rescale = false;
    if (tmax > m_used + 8.f) {
        m_new = ceilf(tmax);
        if (m_used != -INFINITY) {
            rescale = in;   // rows past the block hold whatever memory held
            alpha = ex2(m_used - m_new);
        }
    }
    m_used = m_new;
    if (__any_sync(0xffffffffu, rescale)) {
        if (pv_bar && !warp_wait(pv_bar, pv_parity, abort_flag)) return false;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < o_cols; c += 16) {
            uint32_t o[16];
            tmem_ld16(o_addr + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(o_addr + c, o);
        }
        tmem_st_wait();
        const __nv_bfloat162 a2 = __float2bfloat162_rn(alpha);
#pragma unroll 1
        for (int c = 0; c < p_cols; c += 16) {
            uint32_t w[16];
            tmem_ld16(p_addr + c, w);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]), a2);
                w[e] = *reinterpret_cast<const uint32_t*>(&y);
            }
            tmem_st16(p_addr + c, w);
        }
        l *= alpha;
    }
    return true;
}

// One softmax thread's work on a tile of 64 * halves keys: wait for S, then 64 scores at a time
// transform, mask, running maximum (rescaling what was weighed so far where it grew) and the weights
// back as bf16 pairs over scores already read.  (A row of 128 in registers, all of it unrolled with
// its transforms, is code that the instruction cache does not hold: a first tile took 9 us, one in a
// hundred afterwards 2 us.  Transformed scores written back and read again by a second pass took
// 1200 cycles more per 128 keys.)
// first: the item's first tile.
// pv_bar: the barrier of the group's previous PV, NULL where S complete implies it.
// landed(): called once S is complete; release(h): the weights of keys 64 h .. (-1: all) are in place.
template <int D, bool kScored, typename Landed, typename Release>
__device__ __forceinline__ bool softmax_tile(const Params& p, const Desc& it, const Tile& tl, const Row& row, int halves, bool first,
                                             bool warp_in, uint32_t s_addr, uint32_t o_addr, float& m_used, float& l, uint64_t* s_bar,
                                             uint32_t s_parity, uint64_t* pv_bar, uint32_t pv_parity, volatile int* abort_flag,
                                             Landed landed, Release release) {
    uint64_t seen0 = ~0ull, seen1 = ~0ull;   // of the tree: the node's ancestors and itself
    if (tl.tree && warp_in) {
        seen0 = row.anc[tl.k0 >> 6];
        if (tl.nvalid > 64) seen1 = row.anc[(tl.k0 >> 6) + 1];
    }
    if (!warp_wait(s_bar, s_parity, abort_flag)) return false;
    tc_fence_after();
    if (!landed()) return false;
    if (!warp_in) {
        release(-1);
        return true;
    }
    const float scale2 = p.scale * kLog2e;
    const bool capped = kScored && p.softcap > 0.f, biased = kScored && p.slopes;
    const float in_scale = capped || biased ? 1.f : scale2;   // what the exponent's FFMA still multiplies by
#pragma unroll 1
    for (int h = 0; h < halves; ++h) {
        float x[64];
        load64(s_addr + 64 * h, x);
        const int nv = min(max(tl.nvalid - 64 * h, 0), 64);
        uint64_t bits = nv >= 64 ? ~0ull : (1ull << nv) - 1ull;
        bits &= h ? seen1 : seen0;
        bool masked = tl.tree || nv < 64;
        auto reach = [&](float top) {   // the half's maximum
            return grow(top, row.in, m_used, l, o_addr, first ? 0 : D, s_addr, 32 * h, pv_bar, pv_parity, abort_flag);
        };
        auto reference = [&]() {
            const float r = m_used == -INFINITY ? 0.f : -m_used;
            return pk2(r, r);
        };
        const uint32_t w_addr = s_addr + 32 * h;
        if constexpr (kScored) {
            const int k0 = tl.k0 + 64 * h;
            const int kbase = it.shared ? k0 : it.Ls + k0;      // position of the first key (not the tree's)
            const int depth = row.pos - it.Ls - it.L;           // (own items) the node's
            if (p.window > 0) {
                if (tl.tree) {
                    if (p.window <= SPEC_MAX_DEPTH)
                        for (uint64_t left = bits; left; left &= left - 1) {
                            const int e = __ffsll(static_cast<long long>(left)) - 1;
                            if (depth - p.depth[k0 + e] >= p.window) bits &= ~(1ull << e);
                        }
                } else {
                    const int lo = min(max(row.pos - p.window + 1 - kbase, 0), 64);   // first key seen
                    bits &= lo >= 64 ? 0ull : ~0ull << lo;
                    masked = masked || __any_sync(0xffffffffu, lo > 0);
                }
            }
            if (capped) {
                const Cap cap(p);
                if (!masked && !biased) {
                    // the largest |score| serves both the choice and, where it is within 2^40 of every
                    // weight's scale, the reference: half the comparisons (32K capped 270 -> 260 us)
                    const float most = absmax64(x);
                    if (cap.below(most, fminf(0.16f, 40.f / cap.cap2), row.in)) {
                        if (!reach(most * scale2)) return false;
                        const Cap::Small f(cap);
                        const unsigned long long nm2 = reference();
                        l += weigh64(x, w_addr, [&](unsigned long long v) { return ffma2(v, f.factor(v), nm2); });
                        continue;
                    }
                    if (cap.below(most, 0.7f, row.in)) {
                        if (!reach(cap(max64(x)))) return false;   // the cap keeps the order
                        const Cap::Middle f(cap);
                        const unsigned long long nm2 = reference();
                        l += weigh64(x, w_addr, [&](unsigned long long v) { return ffma2(v, f.factor(v), nm2); });
                        continue;
                    }
                }
#pragma unroll
                for (int e = 0; e < 64; ++e) x[e] = cap(x[e]);
            }
            if (biased) {
                const float f = capped ? 1.f : scale2;
                if (tl.tree) {
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (4 * q < nv) {   // the encoded tree pads its arrays to 16 bytes
                            const int4 d = *reinterpret_cast<const int4*>(p.depth + k0 + 4 * q);
                            x[4 * q] = fmaf(x[4 * q], f, -row.slope2 * static_cast<float>(depth - d.x));
                            x[4 * q + 1] = fmaf(x[4 * q + 1], f, -row.slope2 * static_cast<float>(depth - d.y));
                            x[4 * q + 2] = fmaf(x[4 * q + 2], f, -row.slope2 * static_cast<float>(depth - d.z));
                            x[4 * q + 3] = fmaf(x[4 * q + 3], f, -row.slope2 * static_cast<float>(depth - d.w));
                        }
                } else {
                    const float b0 = row.slope2 * static_cast<float>(kbase - row.pos);
                    const unsigned long long f2 = pk2(f, f), b2 = pk2(b0, b0), s2 = pk2(row.slope2, row.slope2);
#pragma unroll
                    for (int e = 0; e < 64; e += 2)
                        upk2(ffma2(pk2(x[e], x[e + 1]), f2, ffma2(s2, pk2(static_cast<float>(e), static_cast<float>(e + 1)), b2)), x[e], x[e + 1]);
                }
            }
        }
        if (masked) {
            const uint32_t w0 = static_cast<uint32_t>(bits), w1 = static_cast<uint32_t>(bits >> 32);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                if (!((w0 >> e) & 1u)) x[e] = -INFINITY;
                if (!((w1 >> e) & 1u)) x[e + 32] = -INFINITY;
            }
        }
        if (!reach(max64(x) * in_scale)) return false;
        const unsigned long long sc2 = pk2(in_scale, in_scale), nm2 = reference();
        l += weigh64(x, w_addr, [&](unsigned long long v) { return ffma2(v, sc2, nm2); });
    }
    release(-1);   // all of them
    return true;
}

// The same for a pair's 128 keys with plain scores, in a straight line: the maximum 64 scores at a
// time, then the exponentials 32 at a time with the next 32 on their way from TMEM.  (All 128 in
// registers would save the second reading and spill as much.)  The second half's exponentials
// run while the first half is in PV.
template <int D, typename Landed, typename Release>
__device__ __forceinline__ bool softmax_pair(const Params& p, const Tile& tl, const Row& row, bool warp_in, uint32_t s_addr, uint32_t o_addr,
                                             float& m_used, float& l, uint64_t* s_bar, uint32_t s_parity, volatile int* abort_flag,
                                             Landed landed, Release release) {
    if (!warp_wait(s_bar, s_parity, abort_flag)) return false;
    tc_fence_after();
    if (!landed()) return false;
    if (!warp_in) {
        release(0);
        release(1);
        return true;
    }
    float top = -INFINITY;
    if (tl.tree || tl.nvalid < 128) {
        // hidden keys become -inf, in place
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            float x[64];
            load64(s_addr + 64 * h, x);
            const int nv = min(max(tl.nvalid - 64 * h, 0), 64);
            uint64_t bits = nv >= 64 ? ~0ull : (1ull << nv) - 1ull;
            if (tl.tree && nv > 0) bits &= row.anc[(tl.k0 >> 6) + h];   // only the node's ancestors and itself
            const uint32_t w0 = static_cast<uint32_t>(bits), w1 = static_cast<uint32_t>(bits >> 32);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                if (!((w0 >> e) & 1u)) x[e] = -INFINITY;
                if (!((w1 >> e) & 1u)) x[e + 32] = -INFINITY;
            }
            store64(s_addr + 64 * h, x);
            top = fmaxf(top, max64(x));
        }
        tmem_st_wait();
    } else {
        float x[64];
        load64(s_addr, x);
        top = max64(x);
        load64(s_addr + 64, x);
        top = fmaxf(top, max64(x));
    }
    uint32_t a[32], b[32];
    tmem_ld32(s_addr, a);
    const float scale2 = p.scale * kLog2e;
    if (!grow(top * scale2, row.in, m_used, l, o_addr, D, 0, 0, nullptr, 0, abort_flag)) return false;
    const float nmref = m_used == -INFINITY ? 0.f : -m_used;
    const unsigned long long sc2 = pk2(scale2, scale2), nm2 = pk2(nmref, nmref);
    auto weigh = [&](const uint32_t (&x)[32], int c) {   // weights 32 c .. of the row, to columns 16 c ..
        uint32_t packed[16];
        unsigned long long acc2 = pk2(0.f, 0.f);
#pragma unroll
        for (int h2 = 0; h2 < 16; ++h2) {
            float x0, x1;
            upk2(ffma2(pk2(__uint_as_float(x[2 * h2]), __uint_as_float(x[2 * h2 + 1])), sc2, nm2), x0, x1);
            const float a0 = ex2(x0), a1 = ex2(x1);
            acc2 = fadd2(acc2, pk2(a0, a1));
            const __nv_bfloat162 pr = __floats2bfloat162_rn(a0, a1);   // .x (lower key) low
            packed[h2] = *reinterpret_cast<const uint32_t*>(&pr);
        }
        float acc0, acc1;
        upk2(acc2, acc0, acc1);
        l += acc0 + acc1;
        tmem_st16(s_addr + 16 * c, packed);
    };
    // (weights go where scores have been read: 0 .. 31 behind scores 0 .. 63, 32 .. 63 behind 64 .. 127)
    tmem_ld_wait();
    tmem_ld32(s_addr + 32, b);
    weigh(a, 0);
    tmem_ld_wait();
    tmem_ld32(s_addr + 64, a);
    weigh(b, 1);
    release(0);
    tmem_ld_wait();
    tmem_ld32(s_addr + 96, b);
    weigh(a, 2);
    tmem_ld_wait();
    weigh(b, 3);
    release(1);
    return true;
}

// The same for an item of at most 32 rows with the rows' four copies: this warp's 16 keys of a 64-key
// tile.  Weights of the other keys are zero in its lanes.
template <int D, bool kScored, typename Landed, typename Release>
__device__ __forceinline__ bool softmax_few(const Params& p, const Desc& it, const Tile& tl, const Row& row, int copy, uint32_t s_addr,
                                            uint32_t o_addr, float& m_used, float& l, uint64_t* s_bar, uint32_t s_parity,
                                            uint64_t* pv_bar, uint32_t pv_parity, volatile int* abort_flag, Landed landed, Release release) {
    const int e0 = 16 * copy, k0 = tl.k0 + e0;
    const int nv = min(max(tl.nvalid - e0, 0), 16);
    uint32_t bits = (1u << nv) - 1u;
    if (tl.tree) bits &= static_cast<uint32_t>(row.anc[tl.k0 >> 6] >> e0);
    const int kbase = it.shared ? k0 : it.Ls + k0;      // position of the first key (not the tree's)
    const int depth = row.pos - it.Ls - it.L;           // (own items) the node's
    float bias[16];
    if constexpr (kScored) {
        if (p.slopes) {
#pragma unroll
            for (int e = 0; e < 16; ++e) bias[e] = fmaf(row.slope2, static_cast<float>(e), row.slope2 * static_cast<float>(kbase - row.pos));
            if (tl.tree) {
#pragma unroll
                for (int e = 0; e < 16; ++e) bias[e] = e < nv ? -row.slope2 * static_cast<float>(depth - p.depth[k0 + e]) : 0.f;
            }
        }
        if (p.window > 0) {
            if (tl.tree) {
                if (p.window <= SPEC_MAX_DEPTH)
                    for (uint32_t left = bits; left; left &= left - 1) {
                        const int e = __ffs(static_cast<int>(left)) - 1;
                        if (depth - p.depth[k0 + e] >= p.window) bits &= ~(1u << e);
                    }
            } else {
                const int lo = min(max(row.pos - p.window + 1 - kbase, 0), 16);   // first key seen
                bits &= ~0u << lo;
            }
        }
    }
    if (!warp_wait(s_bar, s_parity, abort_flag)) return false;
    tc_fence_after();
    if (!landed()) return false;
    const float scale2 = p.scale * kLog2e;
    uint32_t raw[16];
    tmem_ld16(s_addr + e0, raw);
    tmem_ld_wait();
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(raw[e]) * scale2;
    if constexpr (kScored) {
        if (p.softcap > 0.f) {   // Cap's last form, for small scores too: off by some 2^-22 of the cap
            const float cap2 = p.softcap * kLog2e, k2 = 2.f / p.softcap;   // x is log2 e times the score
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = fmaf(-2.f * cap2, rcp(ex2(x[e] * k2) + 1.f), cap2);
        }
        if (p.slopes) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] += bias[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (!((bits >> e) & 1u)) x[e] = -INFINITY;
    const float top = fmax3(fmax3(fmax3(x[0], x[1], x[2]), fmax3(x[3], x[4], x[5]), fmax3(x[6], x[7], x[8])),
                            fmax3(x[9], x[10], x[11]), fmax3(fmax3(x[12], x[13], x[14]), x[15], x[15]));
    if (!grow(top, row.in, m_used, l, o_addr, D, 0, 0, pv_bar, pv_parity, abort_flag)) return false;
    const float nmref = m_used == -INFINITY ? 0.f : -m_used;
    uint32_t packed[8];
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        const float a0 = ex2(x[e] + nmref), a1 = ex2(x[e + 1] + nmref);
        sum += a0 + a1;
        const __nv_bfloat162 pr = __floats2bfloat162_rn(a0, a1);   // .x (lower key) low
        packed[e / 2] = *reinterpret_cast<const uint32_t*>(&pr);
    }
    l += sum;
    const uint32_t none[8] = {};
#pragma unroll
    for (int c = 1; c < 4; ++c) tmem_st8(s_addr + 8 * ((copy + c) & 3), none);
    tmem_st8(s_addr + 8 * copy, packed);
    release(0);
    return true;
}

template <int D, bool kScored>
__global__ void __launch_bounds__(kThreads, 1) k_attn_shared_tc(const __grid_constant__ Maps mp, const Params p, const int page_log) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((smem_u32(smem) & 1023u) != 0) {   // the swizzle counts address bits: a base elsewhere would scramble tiles
        griddep_wait();
        if (threadIdx.x == 0) p.cta_status[blockIdx.x] = SPEC_EUNSUPPORTED;
        if (blockIdx.x == 0) {             // nothing to join
            for (int b = threadIdx.x; b < p.B; b += kThreads) p.cum[b] = 0;
            if (threadIdx.x == 0) *reinterpret_cast<Plan*>(static_cast<unsigned char*>(p.ws) + kPlanOffset) = Plan{0, 0, 0, 0x3fffffff, 0, 0};
        }
        return;
    }
    uint8_t* sQ = smem;
    uint8_t* sKV = sQ + C::kQ;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + C::kStages * C::kStage);
    uint64_t* q_full = bars;
    uint64_t* q_empty = bars + 1;
    uint64_t* o_final = bars + 2;
    uint64_t* o_empty = bars + 3;
    uint64_t* drain = bars + 4;
    uint64_t* s_full = bars + 5;                  // [group][buffer]
    uint64_t* p_full = s_full + 4;                // [group][buffer]
    uint64_t* ml_full = p_full + 4;               // [group]
    uint64_t* pv_done = ml_full + 2;              // [group]
    uint64_t* turn = pv_done + 2;                 // [group]
    uint64_t* item_full = turn + 2;               // [slot]
    uint64_t* item_empty = item_full + kItems;    // [slot]
    uint64_t* kv_full = item_empty + kItems;      // [J % kFull]
    uint64_t* kv_empty = kv_full + C::kFull;      // [stage]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kv_empty + C::kStages);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* status = reinterpret_cast<int*>(tmem_slot + 2);   // of this CTA: the join takes the largest
    static_assert(C::kBars * 8 + 12 <= 512, "barriers and flags end before the descriptors");
    Desc* desc = reinterpret_cast<Desc*>(reinterpret_cast<uint8_t*>(bars) + 512);            // [slot]
    float2* ml = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(bars) + C::kExchange); // [group][row]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Plan plan{};
    if (warp == 11) {   // its look-ups run beside the set-up
        griddep_wait();
        plan = make_plan(p);
    }
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 2);
        mbar_init(o_final, 2);
        mbar_init(o_empty, 8);
        mbar_init(drain, 2);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ml_full[i], 4);
            mbar_init(&pv_done[i], 1);
            mbar_init(&turn[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], 11);   // TMA, two MMA, eight softmax warps
        }
        for (int i = 0; i < C::kFull; ++i) mbar_init(&kv_full[i], 1);
        for (int i = 0; i < C::kStages; ++i) mbar_init(&kv_empty[i], 2);
        *abort_flag = 0;
        *status = SPEC_OK;
        fence_mbar_init();
        mbar_arrive(&turn[0]);   // thread 0 has the first turn
    }
    if (warp == 0) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    griddep_launch();   // the join may start launching: it waits for the partials

    int U = 0;          // running number of stage uses, the same in every role
    int n = 0;          // running item number
    bool ok = true;
    int q_loads = 0;    // (TMA) items whose Q was requested
    // item number i's descriptor; a whole warp
    auto get_item = [&](Desc& it, int i) -> bool {
        if (!(ok = warp_wait(&item_full[i % kItems], (i / kItems) & 1, abort_flag))) return false;
        it = desc[i % kItems];
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[i % kItems]);
        return it.valid != 0;
    };

    if (warp == 11) {
        if (blockIdx.x == 0) publish_plan(p, plan);
        const int tree_tiles = tiles_of(p.T);
        Walk walk(p, plan, blockIdx.x);
        for (;; ++n) {
            Item it;
            Desc d;
            d.valid = walk.next(p, plan, it);
            if (d.valid) {
                d.shared = it.shared;
                d.pair = it.rows > kRows;
                d.direct = it.direct;
                d.b = it.b; d.kvh = it.kvh; d.rb = it.rb; d.rows = it.rows;
                d.first = it.shared ? plan.sT0 : own_first(p, it.L);
                d.n_pre = it.shared ? plan.nS : own_tiles(p, it.L) - tree_tiles;
                d.end = it.shared ? plan.Ls : it.L;
                d.Ls = plan.Ls;
                d.t0 = it.t0; d.tiles = it.t1 - it.t0; d.index = it.index; d.L = it.L;
            }
            if (n >= kItems && !(ok = warp_wait(&item_empty[n % kItems], ((n / kItems) - 1) & 1, abort_flag))) break;
            if (lane == 0) {
                desc[n % kItems] = d;
                mbar_arrive(&item_full[n % kItems]);
            }
            if (!d.valid) break;
        }
    } else if (warp == 8) {
        const bool leader = elected();
        const uint32_t q_bytes_own = static_cast<uint32_t>(p.rowsO * p.repO) * 128 * C::kH;
        const uint32_t q_bytes_shared = static_cast<uint32_t>(p.rowsS * p.repS) * 128 * C::kH;
        const bool paged = p.pg.table != nullptr;
        const int box_log = paged ? page_log : 6;             // rows of a box of the cache's maps
        int at = 0;                                           // the next use's landing barrier
        Desc it;
        for (; ok && get_item(it, n); ++n) {
            const Tiles ts(it);
            const int* table = it.shared ? p.shared_table : p.pg.table + static_cast<size_t>(it.b) * p.pg.max_blocks;
            const int pre_row = it.shared ? it.kvh * p.Lshared : (it.b * p.Hkv + it.kvh) * p.Lmax;   // contiguous
            const int tree_row = (it.b * p.Hkv + it.kvh) * p.T;
            // Q as soon as the last item's scores are done: the first uses' stages free without it
            bool q_due = true;
            auto load_q = [&](bool now) -> bool {
                if (n > 0 && !(now ? warp_wait(q_empty, (n - 1) & 1, abort_flag) : __all_sync(0xffffffffu, mbar_test(q_empty, (n - 1) & 1))))
                    return !now;
                if (leader) {
                    mbar_arrive_expect_tx(q_full, it.shared ? q_bytes_shared : q_bytes_own);
                    for (int c = 0; c < (it.shared ? p.repS : p.repO); ++c)
                        for (int h = 0; h < C::kH; ++h)
                            tma_load_4d(sQ + h * kQHalf + c * (32 * 128), it.shared ? &mp.q_shared : &mp.q_own, q_full, 64 * h,
                                        it.rb * kBlock, it.kvh, it.b);
                }
                q_loads = n + 1;
                q_due = false;
                return true;
            };
            const int half = ts.width * kHalf, uses = ts.width * ts.count;
            // the rows of 32 boxes at a time, one per lane: lane = tile * 2^plog + box (a look-up in the block
            // table and some fifty instructions for each tile on its own took 1700 cycles, more than the tile)
            const int plog = (it.pair ? 7 : 6) - box_log, batch = 32 >> plog;
            int use = 0;
            for (int j0 = 0; ok && j0 < ts.count; j0 += batch) {
                int row, meta;
                {
                    const Tile tl(p, it, ts, min(j0 + (lane >> plog), ts.count - 1));
                    const int log = tl.tree ? 6 : box_log, off = (lane & ((1 << plog) - 1)) << log;
                    row = (tl.tree ? tree_row : pre_row) + tl.k0 + off;
                    meta = ((tl.nvalid + (1 << log) - 1) >> log) + (tl.tree ? 256 : 0);   // boxes
                    if (paged && !tl.tree && off < tl.nvalid) {
                        const int x = divide(tl.k0 + off, p.pg.bs);
                        int blk = table[x];
                        if (blk < 0 || blk >= p.pg.num_blocks) {
                            atomicMax(status, SPEC_EINVAL);
                            blk = 0;
                        }
                        row = (blk * p.Hkv + it.kvh) * p.pg.bs + (tl.k0 + off - x * p.pg.bs);
                    }
                }
                const int j_end = min(j0 + batch, ts.count);
                for (int j = j0; ok && j < j_end; ++j) {
                    const int src = (j - j0) << plog;
                    const int m = __shfl_sync(0xffffffffu, meta, src), boxes = m & 255;
                    const bool tree = m > 255;
                    const int rows = tree ? min(p.T, kKeys) : 1 << box_log, log = tree ? 6 : box_log;
                    const CUtensorMap* mk = tree ? &mp.kt : it.shared && !paged ? &mp.ks : &mp.kc;
                    const CUtensorMap* mv = tree ? &mp.vt : it.shared && !paged ? &mp.vs : &mp.vc;
                    for (int part = 0; part < ts.width; ++part, ++use) {   // pair: K, then V; narrow: both at once
                        const int stage = at < C::kStages ? at : at - C::kStages;
                        uint8_t* st = sKV + stage * C::kStage;
                        uint64_t* bar = &kv_full[at];
                        if (U >= C::kStages && !(ok = warp_wait(&kv_empty[stage], at < C::kStages ? 1u : 0u, abort_flag))) break;
                        if (leader) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes * rows) * 128 * C::kH * (it.pair ? 1 : 2));
                        for (int i = 0; i < boxes; ++i) {
                            const int r = __shfl_sync(0xffffffffu, row, src + i);
                            if (leader) {
                                uint8_t* dst = st + ((i << log) * 128);
#pragma unroll
                                for (int h = 0; h < C::kH; ++h) tma_load_2d(dst + h * half, part ? mv : mk, bar, 64 * h, r);
                                if (!it.pair)
#pragma unroll
                                    for (int h = 0; h < C::kH; ++h) tma_load_2d(dst + C::kStage / 2 + h * half, mv, bar, 64 * h, r);
                            }
                        }
                        ++U;
                        if (++at == C::kFull) at = 0;
                        if (q_due && !(ok = load_q(n == 0 || use == C::kStages - 1 || use == uses - 1))) break;
                    }
                }
            }
        }
    } else if (warp == 9 || warp == 10) {
        const bool leader = elected();
        const int g = warp - 9;
        const uint32_t idesc_o = idesc_bf16_f32_bmn(kRows, D);
        uint32_t p_phase = 0, t_phase = 0;                // bit b: phase of p_full[g][b]; of turn[g]
        // S of the K tile in `stage` into column `dst`: Q block `block`; in a pair the turn goes
        // to the other thread while the last products are still running
        auto issue_s = [&](uint32_t dst, int block, int stage, int width) {
            const uint64_t qd = sdesc_k128(smem_u32(sQ) + block * (kRows * 128));
            const uint64_t kd = sdesc_k128(smem_u32(sKV + stage * C::kStage));
            const uint32_t idesc_s = idesc_bf16_f32(kRows, width * kKeys);
            const int half = width * kHalf;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                mma_bf16(dst, qd + (((k >> 2) * kQHalf + (k & 3) * 32) >> 4), kd + (((k >> 2) * half + (k & 3) * 32) >> 4), idesc_s,
                         k > 0 ? 1u : 0u);
        };
        auto pass_turn = [&]() { mbar_arrive(&turn[g ^ 1]); };
        // O += P (column `src`) V (at v, halves `half` bytes apart) for keys 64 h .. of the tile, whole steps of 16
        auto issue_pv = [&](uint32_t src, uint32_t v, int half, int h, int nvalid, bool first) {
            const uint64_t vd = sdesc_mn128(v, half, 1024) + h * (kHalf >> 4);
            const uint32_t o = tmem + kO + g * D;
            src += h * (kKeys / 2);
            nvalid -= h * kKeys;
            if (nvalid >= kKeys) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_bf16_ts(o, src + k * 8, vd + ((k * 2048) >> 4), idesc_o, (first && k == 0) ? 0u : 1u);
            } else {
#pragma unroll 1
                for (int k = 0; k * 16 < nvalid; ++k)
                    mma_bf16_ts(o, src + k * 8, vd + ((k * 2048) >> 4), idesc_o, (first && k == 0) ? 0u : 1u);
            }
        };
        // landing barrier and stage of a stage use, kept as counters: no division per tile
        struct Use {
            int at, round;
            __device__ __forceinline__ explicit Use(int u) : at(u % C::kFull), round((u / C::kFull) & 1) {}
            __device__ __forceinline__ void two_on() {
                at += 2;
                if (at >= C::kFull) {
                    at -= C::kFull;
                    round ^= 1;
                }
            }
            __device__ __forceinline__ int stage() const { return at < C::kStages ? at : at - C::kStages; }
        };
        Desc it;
        for (; ok && get_item(it, n); ++n) {
            const Tiles ts(it);
            if (leader) {
                auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = ok && bounded_wait(bar, parity, abort_flag); };
                auto wait_p = [&](int buf) {
                    const bool r = wait(&p_full[2 * g + buf], (p_phase >> buf) & 1u);
                    p_phase ^= 1u << buf;
                    return r;
                };
                auto wait_turn = [&]() {
                    const bool r = wait(&turn[g], t_phase);
                    t_phase ^= 1u;
                    return r;
                };
                wait(q_full, n & 1);
                bool o_clear = n == 0;
                auto clear_o = [&]() {                    // once in every item
                    if (!o_clear) wait(o_empty, (n - 1) & 1);
                    o_clear = true;
                    return ok;
                };
                if (it.pair) {
                    // The threads take turns, PV and the next S at a time: group 1's softmax then runs half a
                    // period behind group 0's and each batch has the tensor pipe to itself.  Without turns the
                    // batches share the pipe, both groups wait twice as long at the same time and then leave
                    // it idle at the same time (2685 cycles per 128 x 128 scores); one thread issuing for both
                    // leaves it idle in its waits and commits (1890).
                    // Stages are released by the softmax groups: a group's S of its next tile complete says
                    // that its products before it are, and a commit costs the issuing thread some 250 cycles.
                    Use k_use(U), v_use(U + 1);
                    if (wait(&kv_full[k_use.at], k_use.round) && wait_turn()) {
                        tc_fence_after();
                        issue_s(tmem + g * 128, g, k_use.stage(), 2);
                        pass_turn();
                        mma_commit(&s_full[2 * g]);
                    }
                    for (int j = 0; ok && j < ts.count; ++j) {
                        const bool more = j + 1 < ts.count;
                        if (!more) mma_commit(q_empty);
                        k_use.two_on();
                        const int nvalid = Tile(p, it, ts, j).nvalid;
                        if (!wait(&kv_full[v_use.at], v_use.round) || !clear_o()) break;
                        if (more && !wait(&kv_full[k_use.at], k_use.round)) break;
                        if (!wait_p(0) || !wait_turn()) break;
                        tc_fence_after();
                        issue_pv(tmem + g * 128, smem_u32(sKV + v_use.stage() * C::kStage), 2 * kHalf, 0, nvalid, j == 0);
                        if (!wait_p(1)) break;
                        tc_fence_after();
                        issue_pv(tmem + g * 128, smem_u32(sKV + v_use.stage() * C::kStage), 2 * kHalf, 1, nvalid, false);
                        pass_turn();
                        if (more) issue_s(tmem + g * 128, g, k_use.stage(), 2);
                        if (more) mma_commit(&s_full[2 * g]);
                        v_use.two_on();
                    }
                } else {
                    // thread g for group g: every second tile; S of the next and PV of the last, whichever is ready
                    const int cnt = (ts.count - g + 1) / 2;
                    Use s_use(U + g), v_use(U + g);
                    if (cnt == 0) mma_commit(q_empty);
                    int issued = 0, done = 0;
                    uint64_t idle_since = 0;
                    for (uint32_t idle = 1; ok && done < cnt; ++idle) {
                        const int buf = done & 1;
                        if (issued < cnt && issued - done < 2 && mbar_test(&kv_full[s_use.at], s_use.round)) {
                            tc_fence_after();
                            issue_s(tmem + g * 128 + (issued & 1) * kKeys, 0, s_use.stage(), 1);
                            mma_commit(&s_full[2 * g + (issued & 1)]);
                            s_use.two_on();
                            if (++issued == cnt) mma_commit(q_empty);
                        } else if (issued > done && mbar_test(&p_full[2 * g + buf], (p_phase >> buf) & 1u)) {
                            p_phase ^= 1u << buf;
                            if (!clear_o()) break;
                            tc_fence_after();
                            issue_pv(tmem + g * 128 + buf * kKeys, smem_u32(sKV + v_use.stage() * C::kStage + C::kStage / 2), kHalf, 0,
                                     Tile(p, it, ts, g + 2 * done).nvalid, done == 0);
                            mma_commit(&kv_empty[v_use.stage()]);
                            mma_commit(&pv_done[g]);
                            v_use.two_on();
                            ++done;
                        } else {
                            if ((idle & 1023u) == 0) {   // bounded like the other waits
                                const uint64_t now = globaltimer_ns();
                                if (idle_since == 0) idle_since = now;
                                ok = !*abort_flag && now - idle_since <= 2000000000ull;
                            }
                            continue;
                        }
                        idle = 0;
                        idle_since = 0;
                    }
                    clear_o();
                }
                if (ok) mma_commit(o_final);
            }
            U += ts.width * ts.count;
            ok = __all_sync(0xffffffffu, ok);
        }
        if (leader) mma_commit(drain);
        __syncwarp();
    } else {
        const int grp = warp >> 2;
        const int tl_row = (warp & 3) * 32 + lane;         // TMEM lane
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_base = lane_base + grp * 128, o_addr = lane_base + kO + grp * D;
        uint32_t s_phase = 0, ml_phase = 0;                // bit b: phase of s_full[grp][b]
        int narrow = 0;                                    // narrow tiles this group has finished
        // the thread's row of an item: its place in gT, node, position, slope (rows past the block repeat its last)
        struct At {
            Row row;
            int r, ib, i;
        };
        auto row_of = [&](const Desc& d) -> At {
            At at;
            at.r = (d.shared ? p.repS : p.repO) > 1 ? lane : (d.pair ? grp * kRows : 0) + tl_row;
            const int rr = min(at.r, d.rows - 1);
            at.ib = p.gT < kBlock ? rr / p.gT : 0;
            at.i = p.gT < kBlock ? rr - at.ib * p.gT : d.rb * kBlock + rr;
            const int head = at.i / p.T, node = at.i - head * p.T;
            at.row = Row{at.r < d.rows, 0, 0.f, p.anc + static_cast<size_t>(node) * p.words};
            if constexpr (kScored) {
                at.row.pos = d.Ls + (d.shared ? own_len(p, d.b + at.ib) : d.L) + p.depth[node];
                if (p.slopes) at.row.slope2 = p.slopes[d.kvh * p.g + head] * kLog2e;
            }
            return at;
        };
        // the softmax threads read descriptors where they are: their registers hold scores
        auto look_at = [&](int i) -> bool {
            ok = warp_wait(&item_full[i % kItems], (i / kItems) & 1, abort_flag);
            return ok && desc[i % kItems].valid != 0;
        };
        bool more = look_at(0);
        At at{};
        if (more) at = row_of(desc[0]);
        for (; more; ++n) {
            const Desc& it = desc[n % kItems];
            const Tiles ts(it);
            const bool few = (it.shared ? p.repS : p.repO) > 1;
            const int r = at.r;
            const bool warp_in = few || (it.pair ? grp * kRows : 0) + (warp & 3) * 32 < it.rows;
            const bool in = at.row.in;
            const Row& row = at.row;
            float m_used = -INFINITY, l = 0.f;
            for (int j = it.pair ? 0 : grp, k = 0; j < ts.count; j += it.pair ? 1 : 2, ++k) {
                const Tile tl(p, it, ts, j);
                const int buf = it.pair ? 0 : k & 1;
                uint64_t* s_bar = &s_full[2 * grp + buf];
                const uint32_t parity = (s_phase >> buf) & 1u;
                s_phase ^= 1u << buf;
                auto landed = [&]() -> bool {
                    if (it.pair && (warp & 3) == 0 && lane == 0) {
                        // the group's S of this tile and PV of the last one are complete: K and the last V may go
                        mbar_arrive(&kv_empty[(U + 2 * j) % C::kStages]);
                        if (j > 0) mbar_arrive(&kv_empty[(U + 2 * j - 1) % C::kStages]);
                    }
                    if (tl.nvalid & 15) {
                        // zero V from the last key to the end of its step of 16, once it has landed (narrow: with
                        // K); of a pair's V both groups read all of it, and each zeroes before its own PV may start
                        const int use = U + (it.pair ? 2 * j + 1 : j);
                        if (it.pair && !warp_wait(&kv_full[use % C::kFull], (use / C::kFull) & 1, abort_flag)) return false;
                        uint8_t* sv_tile = sKV + (use % C::kStages) * C::kStage + (it.pair ? 0 : C::kStage / 2);
                        const int pad = 16 - (tl.nvalid & 15);
                        for (int x = tl_row; x < pad * 8 * C::kH; x += kRows) {
                            const int v_row = tl.nvalid + x / (8 * C::kH), y = x % (8 * C::kH);
                            *reinterpret_cast<uint4*>(sv_tile + (y >> 3) * ts.width * kHalf + v_row * 128 + (y & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                    return true;
                };
                // a pair's halves go to PV one after the other: it starts while the second half is computed
                auto release = [&](int h) {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (it.pair && h < 0) mbar_arrive(&p_full[2 * grp + 1]);
                        mbar_arrive(&p_full[2 * grp + (it.pair ? max(h, 0) : buf)]);
                    }
                };
                uint64_t* pv_bar = it.pair ? nullptr : &pv_done[grp];
                const uint32_t s_addr = s_base + buf * kKeys;
                if (few)
                    ok = softmax_few<D, kScored>(p, it, tl, row, warp & 3, s_addr, o_addr, m_used, l, s_bar, parity, pv_bar,
                                                 (narrow - 1) & 1, abort_flag, landed, release);
                else if (!kScored && it.pair)
                    ok = softmax_pair<D>(p, tl, row, warp_in, s_addr, o_addr, m_used, l, s_bar, parity, abort_flag, landed, release);
                else
                    ok = softmax_tile<D, kScored>(p, it, tl, row, ts.width, k == 0, warp_in, s_addr, o_addr, m_used, l, s_bar, parity,
                                                  pv_bar, (narrow - 1) & 1, abort_flag, landed, release);
                if (!ok) break;
                if (!it.pair) {
                    // the stage's second arrival, beside PV's commit (a pair's come from both groups)
                    if ((warp & 3) == 0 && lane == 0) mbar_arrive(&kv_empty[(U + j) % C::kStages]);
                    ++narrow;
                }
            }
            if (!ok) break;
            // the next item's row, looked up while the last products run
            At next_at{};
            more = look_at(n + 1);
            if (!ok) break;
            if (more) next_at = row_of(desc[(n + 1) % kItems]);
            // the item's end: in a pair each group has its rows' whole (m, l, O); otherwise (m, l)
            // across the groups, then each joins half the columns
            if (!(ok = warp_wait(o_final, n & 1, abort_flag))) break;
            tc_fence_after();
            if (it.pair && (warp & 3) == 0 && lane == 0) mbar_arrive(&kv_empty[(U + 2 * ts.count - 1) % C::kStages]);
            float m = m_used, lsum = l, a0 = 1.f, a1 = 0.f;   // weights of the group's own O and the other's
            uint32_t from = o_addr;                           // the first of them, and whether there are both
            bool both = false;
            if (!it.pair) {
                ml[grp * kRows + tl_row] = make_float2(m_used, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(&ml_full[grp]);
                if (!(ok = warp_wait(&ml_full[grp ^ 1], ml_phase, abort_flag))) break;
                ml_phase ^= 1u;
                const float2 other = ml[(grp ^ 1) * kRows + tl_row];
                m = fmaxf(m_used, other.x);
                const float ref = m == -INFINITY ? 0.f : m;
                a0 = ex2(m_used - ref);
                a1 = ex2(other.x - ref);
                lsum = a0 * l + a1 * other.y;
                both = ts.count > 1;
                if (!both && grp == 1) {                   // a group without a tile left its O as it was
                    from = lane_base + kO;
                    a0 = a1;
                }
            }
            if (warp_in) {
                const int cap = it.shared ? p.rowsS : p.rowsO, stride = cap * (few ? 4 : 1);
                float4* part = (it.shared ? p.part_s : p.part_o) + static_cast<size_t>(it.index) * (D / 4 + 1) * stride +
                               (few ? (warp & 3) * cap : 0) + r;
                const float inv = it.direct ? 1.f / lsum : 1.f;
                const size_t q_row = (static_cast<size_t>(it.b + at.ib) * p.Hq + it.kvh * p.g) * p.T + at.i;
                if (in && (it.pair || grp == 0)) {
                    if (!it.direct) part[0] = make_float4(m, lsum, 0.f, 0.f);
                    else if (p.lse) p.lse[q_row] = (m + log2f(lsum)) * kLn2;
                }
                a0 *= inv;
                a1 *= inv;
                const int c_end = it.pair ? D : (grp + 1) * (D / 2);
                // W columns at a time.  This code runs once an item, and fetching it costs some ten cycles an
                // instruction, so 16 where the softmax's own code is long (32K capped 260 us at 32, 247 at 16);
                // with plain scores 32 (70B trees 222, at 16 228).
                constexpr int W = kScored ? 16 : 32;
#pragma unroll 1
                for (int c0 = it.pair ? 0 : grp * (D / 2); c0 < c_end; c0 += W) {
                    uint32_t o[W], o1[W];
                    float v[W];
                    tmem_ld(from + c0, o);
                    if (both) tmem_ld(lane_base + kO + (grp ^ 1) * D + c0, o1);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < W; ++e) v[e] = a0 * __uint_as_float(o[e]);
                    if (both)
#pragma unroll
                        for (int e = 0; e < W; ++e) v[e] = fmaf(a1, __uint_as_float(o1[e]), v[e]);
                    if (in && !it.direct) {
#pragma unroll
                        for (int e = 0; e < W / 4; ++e)
                            part[static_cast<size_t>(1 + c0 / 4 + e) * stride] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    } else if (in) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + q_row * D + c0);
#pragma unroll
                        for (int e = 0; e < W / 8; ++e) {
                            uint32_t w[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * e + 2 * q], v[8 * e + 2 * q + 1]);
                                w[q] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                            dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_empty);
            U += ts.width * ts.count;
            if (lane == 0) mbar_arrive(&item_empty[n % kItems]);
            at = next_at;
        }
    }
    if (!ok) {
        if (lane == 0) {
            atomicMax(status, SPEC_ETIMEOUT);
            *abort_flag = 1;
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // a wait ran out: let this CTA's own loads and MMAs land before it ends
        if (warp == 8) {
            for (int j = max(0, U - C::kFull); j < U; ++j) mbar_wait(&kv_full[j % C::kFull], (j / C::kFull) & 1, 100000000ull);
            if (q_loads > 0) mbar_wait(q_full, (q_loads - 1) & 1, 100000000ull);
        }
        if (warp == 9 || warp == 10) mbar_wait(drain, 0, 100000000ull);
    }
    __syncthreads();
    if (threadIdx.x == 0) p.cta_status[blockIdx.x] = *status;
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- host

template <int D, bool kScored>
static spec_status launch_items(const Maps& m, const Params& p, int page_log, int blocks, cudaStream_t s) {
    static_assert(Cfg<D>::kSmem <= 232448, "shared memory of one CTA");
    auto kern = k_attn_shared_tc<D, kScored>;
    SPEC_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem));
    SPEC_CUDA_TRY(launch_ex("attn_shared_tc", kern, dim3(blocks), dim3(kThreads), Cfg<D>::kSmem, s, true, m, p, page_log));
    return SPEC_OK;
}

spec_status attn_shared_tc_run(const Params& p, int blocks, cudaStream_t s) {
    Maps m;
    memset(&m, 0, sizeof(m));
    const uint64_t B = p.B, Hkv = p.Hkv, T = p.T, D = p.D;
    const uint32_t b1 = static_cast<uint32_t>(std::min(p.gT, kBlock));
    SPEC_CUDA_TRY(make_tmap_bf16_4d(&m.q_own, p.q, B, Hkv, p.gT, D, 1, b1));
    SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.kt, p.kt, B * Hkv * T, D, D, static_cast<uint32_t>(std::min(p.T, kKeys))));
    SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.vt, p.vt, B * Hkv * T, D, D, static_cast<uint32_t>(std::min(p.T, kKeys))));
    int page_log = 0;
    if (p.pg.table) {
        // a box lies inside one block and one tile: the largest power of two that divides both
        page_log = 4;
        while ((1 << page_log) < kKeys && p.pg.bs % (2 << page_log) == 0) ++page_log;
        const uint64_t rows = static_cast<uint64_t>(p.pg.num_blocks) * Hkv * p.pg.bs;
        SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.kc, p.kc, rows, D, D, 1u << page_log));
        SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.vc, p.vc, rows, D, D, 1u << page_log));
    } else {
        SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.kc, p.kc, B * Hkv * p.Lmax, D, D, kKeys));
        SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.vc, p.vc, B * Hkv * p.Lmax, D, D, kKeys));
    }
    if (p.shared_len) {
        SPEC_CUDA_TRY(make_tmap_bf16_4d(&m.q_shared, p.q, B, Hkv, p.gT, D, static_cast<uint32_t>(p.nbb), b1));
        if (!p.pg.table) {
            SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.ks, p.ks, Hkv * p.Lshared, D, D, kKeys));
            SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.vs, p.vs, Hkv * p.Lshared, D, D, kKeys));
        }
    }
    const bool scored = p.softcap > 0.f || p.window > 0 || p.slopes;
    if (p.D == 64)
        return scored ? launch_items<64, true>(m, p, page_log, blocks, s) : launch_items<64, false>(m, p, page_log, blocks, s);
    return scored ? launch_items<128, true>(m, p, page_log, blocks, s) : launch_items<128, false>(m, p, page_log, blocks, s);
}

}  // namespace shr
}  // namespace spec
