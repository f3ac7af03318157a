// Tensor-core (tcgen05) kernel of kv_weigh: bf16, head dim 64 or 128.
//
// The product is taken as S^T: keys are the rows of the MMA (M = 128 keys of a tile, one TMEM lane
// each), query rows its columns.  So a thread owns a key, and the sum over query rows that the
// operator asks for runs along its own registers: no reduction between lanes, no atomics, one
// result a thread.  lse is a value per column, read from shared memory by all lanes at once:
//   w(key) = sum over columns c of 2^(S[key, c] scale log2 e - lse_c log2 e)
//
// Two ways through, chosen on the host:
//   few   at most 256 query rows of a KV head (generated tokens, accepted paths, short chains; more in
//         several passes): a head's rows stay in shared memory while its keys stream through a ring of
//         128-key tiles.  Bound by the keys' bytes up to some 130 rows.
//   many  prompts: 256 keys stay while chunks of 128 query rows of one head stream through, each chunk
//         multiplied with both halves of the keys: with 128 keys a CTA the rows would come out of L2 at
//         9 TB/s.  Bound by the exponentials, one for each pair of row and key.
// The work, (sequence, head, key tile, chunk) in that order, is one line of chunks, cut into as
// many equal parts as there are CTAs; lengths are known on the device only, so every CTA works its part
// out itself.  A tile that is cut leaves partial sums, which kv_weigh_join adds up in order.
//
// One persistent CTA an SM:
//   two groups of 4    one thread per key.  few: alternate tiles; many: half of a tile each
//   and then           a warp for TMA (key tiles; chunks of rows), one that issues products (many: two, one
//                      for each half of a tile: issuing waits for the tensor pipe, and a single one left it idle
//                      for as long again while it looked at barriers), and two or one that gather a head's
//                      rows (few) and lse (both)
// Waits are bounded (2 s); on expiry SPEC_ETIMEOUT goes to the status word, every role leaves its
// loops, and the CTA drains its own loads and MMAs before it frees TMEM.
#include <algorithm>
#include <cstring>

#include "kv_weigh.cuh"
#include "tc.cuh"

namespace spec {
namespace weigh {

using namespace tc;

constexpr int kKeys = 128;            // keys of a product
constexpr int kChunk = 128;           // query rows of a chunk (many)
template <bool MANY> constexpr int kTile = MANY ? 2 * kKeys : kKeys;   // keys of a tile
constexpr int kMostRows = 256;        // query rows of a pass (few)
constexpr int kGroups = 2;            // of four warps
constexpr int kTcThreads = (4 * kGroups + 4) * 32;
constexpr int kMaxStages = 8;
constexpr uint32_t kTmemCols = 512;
constexpr float kL2e = 1.4426950408889634f;

struct Maps {
    CUtensorMap k, q;
};

// What a CTA leaves for the join: its first tile began before it (and whether it ends here), its last
// one goes on after it.
struct Record {
    int head, head_ends, tail, b, h, t, pad0, pad1;
};

struct TcParams {
    Params p;
    int g, nq;                        // query heads per KV head; rows of a Q stage
    int row0;                         // few: first of the head's rows that this pass takes
    int k_stages, q_stages, buffers;  // buffers of scores in TMEM
    int box;                          // keys of a load
    Record* records;                  // [CTAs] (many)
    float* parts;                     // [CTAs][2][2 * kKeys]
};

// Barriers and small arrays behind the operand stages.
struct Small {
    uint64_t k_full[kMaxStages], k_empty[kMaxStages];
    uint64_t q_full[4], q_empty[4];
    uint64_t l_full[4], l_empty[4];   // many: lse of a chunk's rows
    uint64_t s_full[4], s_empty[4];   // many: [half][turn]
    uint64_t drain;
    uint32_t tmem;
    int abort_flag, bad;
    int start[4];                     // the CTA's first tile: b, h, t, chunk of it
    long long length;                 // its chunks
    __align__(16) float nl2[4][kMostRows];   // -lse log2 e of a stage's rows, -inf: does not count
    int last[4][kMostRows];           // few: the last key that a row sees
    int odd[4][2];                    // few: whether a stage has rows that do not count although they are there (each warp's
                                      // word): such rows may hold anything, and 0 times that need not be 0
};

// The line of chunks of one sequence and head: row chunks first(t) .. C - 1 for tile t, times `mult` query heads.
struct Head {
    int tiles, C, o, mult;
    __device__ __forceinline__ long long before(int t) const {   // chunks of the tiles in front of t
        const long long s = o / 2 + 1, k = max(0ll, t - s);      // the first tile that some chunks do not see
        return (static_cast<long long>(C) * t - k * (s + t - 1 - o)) * mult;
    }
    __device__ __forceinline__ int first(int t) const { return max(0, 2 * t - o); }  // row (256 t - rows in front) / 128
    __device__ __forceinline__ int chunks(int t) const { return (C - first(t)) * mult; }
};
template <bool MANY> __device__ __forceinline__ Head head_of(const TcParams& tp, const Rows& r) {
    Head h{0, 1, 1 << 30, 1};
    if (!r.ok) return h;
    h.tiles = (r.n + kTile<MANY> - 1) / kTile<MANY>;
    if (r.count == 0 && tp.p.decay == 1.f) h.tiles = 0;          // nothing changes
    if (MANY) {
        if (r.count > 0) {
            h.C = (r.count + kChunk - 1) / kChunk;
            h.o = (r.n - r.count + kChunk - 1) / kChunk;
            h.mult = tp.g;
        }
    } else if (tp.row0 > 0 && tp.g * r.count <= tp.row0) {
        h.tiles = 0;                                             // no rows left for this pass
    }
    return h;
}

static __device__ __noinline__ bool wait_slowly(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
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
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return mbar_try_wait(bar, parity) || wait_slowly(bar, parity, abort_flag);
}
__device__ __forceinline__ bool warp_wait_for(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, wait_for(bar, parity, abort_flag));
}

// One lane of the warp, the same at every call, as a condition the compiler knows to be uniform: behind lane == 0 the
// products' descriptors went through vector registers, and issuing 16 products took twice as long as they did.
__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// The tiles of a CTA's part of the line, the same in every role.
template <bool MANY> struct Walk {
    const TcParams& tp;
    int b, h, t, c, take;             // the tile, its first chunk here, and how many are here
    long long left;
    Rows rows;
    Head head;
    bool more;
    __device__ __forceinline__ Walk(const TcParams& tp_, const Small& sm) : tp(tp_) {
        b = sm.start[0]; h = sm.start[1]; t = sm.start[2]; c = sm.start[3];
        left = sm.length;
        more = left > 0;
        if (more) {
            rows = rows_of(tp.p, b);
            head = head_of<MANY>(tp, rows);
            set();
        }
    }
    __device__ __forceinline__ void set() { take = static_cast<int>(min(static_cast<long long>(head.chunks(t) - c), left)); }
    // many: first rows of the chunks one after the other, and which of its query heads the first belongs to
    struct Chunks {
        int i0, begin, end;
        __device__ __forceinline__ void next() {
            i0 += kChunk;
            if (i0 >= end) i0 = begin;
        }
    };
    __device__ __forceinline__ Chunks chunks(int& head_at) const {
        const int m = head.C - head.first(t);
        head_at = c / m;
        const int begin = head.first(t) * kChunk;
        return {begin + (c - head_at * m) * kChunk, begin, head.C * kChunk};
    }
    __device__ __forceinline__ bool whole() const { return take == head.chunks(t); }
    // whether the next tile is of another head (or there is none)
    __device__ __forceinline__ bool column_ends() const { return left == take || t + 1 == head.tiles; }
    __device__ __forceinline__ void next() {
        left -= take;
        more = left > 0;
        c = 0;
        if (!more) return;
        if (++t == head.tiles) {
            t = 0;
            if (++h == tp.p.Hkv) {
                h = 0;
                do {                  // there is another one with tiles: chunks are left
                    if (++b == tp.p.B) {
                        more = false;
                        return;
                    }
                    rows = rows_of(tp.p, b);
                    head = head_of<MANY>(tp, rows);
                } while (head.tiles == 0);
            }
        }
        set();
    }
};

// Where this CTA's part begins and how long it is; one warp.
template <bool MANY> __device__ void plan(const TcParams& tp, Small& sm) {
    const int lane = threadIdx.x & 31;
    long long total = 0;
    auto weight = [&](int b) -> long long {
        if (b >= tp.p.B) return 0;
        const Head h = head_of<MANY>(tp, rows_of(tp.p, b));
        return h.tiles ? h.before(h.tiles) * tp.p.Hkv : 0;
    };
    long long w0 = 0;                 // of the first 32 sequences, kept for the second look
    for (int b0 = 0; b0 < tp.p.B; b0 += 32) {
        long long w = weight(b0 + lane);
        if (b0 == 0) w0 = w;
        for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
        total += w;
    }
    // as many CTAs have a part as there are chunks, the first ones: the join looks for a tile's parts side by side
    const long long ctas = min(total, static_cast<long long>(gridDim.x));
    long long from = 0, to = 0;
    if (blockIdx.x < ctas) {
        from = total * blockIdx.x / ctas;
        to = total * (blockIdx.x + 1) / ctas;
    }
    if (lane == 0) sm.length = to - from;
    if (to == from) return;
    long long base = 0;
    for (int b0 = 0; b0 < tp.p.B; b0 += 32) {
        const long long w = b0 == 0 ? w0 : weight(b0 + lane);
        long long upto = w;
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
        }
        const long long mine = base + upto - w;
        const unsigned here = __ballot_sync(0xffffffffu, from >= mine && from < mine + w);
        if (here) {
            if (lane == __ffs(here) - 1) {
                const Head hd = head_of<MANY>(tp, rows_of(tp.p, b0 + lane));
                const long long per = hd.before(hd.tiles);
                const long long in = from - mine;
                const int h = static_cast<int>(in / per);
                const long long r = in - h * per;
                int lo = 0, hi = hd.tiles - 1;       // the last tile that begins at or before r
                while (lo < hi) {
                    const int mid = (lo + hi + 1) / 2;
                    if (hd.before(mid) <= r) lo = mid; else hi = mid - 1;
                }
                sm.start[0] = b0 + lane;
                sm.start[1] = h;
                sm.start[2] = lo;
                sm.start[3] = static_cast<int>(r - hd.before(lo));
            }
            return;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
}

// A slot of a ring and how often it has come round, kept without divisions (with them, by numbers that are not known to
// the compiler, single tokens took 72 us where this takes 63, prompts 142 for 128).
struct Ring {
    int at = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next(int n) {
        if (++at == n) {
            at = 0;
            ++round;
        }
    }
    __device__ __forceinline__ uint32_t full() const { return round & 1; }            // parity of "filled" this time
    __device__ __forceinline__ uint32_t empty() const { return (round + 1) & 1; }     // of "emptied" the time before, if round > 0
};

// Whether no row of the chunk that begins at i0 sees a key of the half tile that begins at k0 (many).
__device__ __forceinline__ bool unseen(const Rows& r, int k0, int i0) {
    return k0 >= r.n || k0 > r.n - r.count + min(i0 + kChunk, r.count) - 1;
}

__device__ __forceinline__ void load_scores(uint32_t addr, uint32_t (&r)[16]) { tmem_ld16(addr, r); }
__device__ __forceinline__ void load_scores(uint32_t addr, uint32_t (&r)[32]) { tmem_ld32(addr, r); }

// -lse log2 e of N columns.  (Read before the wait for their scores: that is a barrier to the compiler, and behind it
// every step began with the latency of shared memory.)
template <int N> __device__ __forceinline__ void load_lse(const float* nl2, unsigned long long (&l)[N / 2]) {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(nl2 + e);
        l[e / 2] = x.x;
        l[e / 2 + 1] = x.y;
    }
}

// Bit i of lane k's word becomes bit k of lane i's: blocks of 16, 8, .. 1 change places across the diagonal.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x) {
    const int lane = threadIdx.x & 31;
    uint32_t low = 0x0000ffffu;       // the lower half of every block
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const uint32_t y = __shfl_xor_sync(0xffffffffu, x, d);
        x = lane & d ? (x & ~low) | ((y >> d) & low) : (x & low) | ((y << d) & ~low);
        low ^= low << (d >> 1);
    }
    return x;
}

// N columns of a key's scores: the sum of their weights.
template <int N>
__device__ __forceinline__ unsigned long long weights(const uint32_t (&s)[N], const unsigned long long (&l)[N / 2], unsigned long long c2) {
    unsigned long long sum = pk2(0.f, 0.f), sum1 = pk2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        float a, b, c, d;
        upk2(ffma2(pk2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, l[e / 2]), a, b);
        upk2(ffma2(pk2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), c2, l[e / 2 + 1]), c, d);
        sum = fadd2(sum, pk2(ex2(a), ex2(b)));
        sum1 = fadd2(sum1, pk2(ex2(c), ex2(d)));
    }
    return fadd2(sum, sum1);
}

// The same of the columns whose bit is set; the others may hold anything.
template <int N>
__device__ __forceinline__ unsigned long long masked(const uint32_t (&s)[N], const unsigned long long (&l)[N / 2], unsigned long long c2, uint32_t seen) {
    uint32_t x[N];
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = (seen >> e) & 1u ? s[e] : 0xff800000u;   // -inf: weighs nothing
    return weights(x, l, c2);
}

template <int D, bool MANY>
__global__ void __launch_bounds__(kTcThreads, 1) k_weigh_tc(const __grid_constant__ Maps mp, const TcParams tp) {
    constexpr int kH = D / 64;
    constexpr int kKHalf = kKeys * 128;                  // bytes of a 64-column half of 128 keys
    constexpr int kHalves = MANY ? 2 : 1;                // 128 keys each
    constexpr int kKStage = kHalves * kH * kKHalf;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    // the swizzle counts address bits: tiles start on 1024-byte boundaries
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const Params& p = tp.p;
    uint8_t* sK = smem;
    uint8_t* sQ = sK + tp.k_stages * kKStage;
    const int q_half = tp.nq * 128;
    Small& sm = *reinterpret_cast<Small*>(sQ + tp.q_stages * kH * q_half);
    volatile int* abort_flag = &sm.abort_flag;
    constexpr int kTma = 4 * kGroups, kMma = kTma + 1, kRowsWarp = kTma + (MANY ? 3 : 2);   // the other roles' warps
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], MANY ? 2 : 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sm.q_full[i], MANY ? 1 : 2);
            mbar_init(&sm.q_empty[i], MANY ? 2 : 9);
            mbar_init(&sm.l_full[i], 1);
            mbar_init(&sm.l_empty[i], 4 * kGroups);
            mbar_init(&sm.s_full[i], MANY ? 2 : 1);
            mbar_init(&sm.s_empty[i], 4);
        }
        mbar_init(&sm.drain, MANY ? 2 : 1);
        sm.abort_flag = 0;
        sm.bad = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&sm.tmem, kTmemCols);
    griddep_wait();                   // the stream's kernel before this one may still run: its results are behind here
    if (MANY && threadIdx.x == 0) tp.records[blockIdx.x] = Record{0, 0, 0, 0, 0, 0, 0, 0};
    if (warp == kTma) plan<MANY>(tp, sm);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const uint32_t buf_cols = kTmemCols / tp.buffers;
    griddep_launch();                 // the join may start launching: it waits for the partial sums
    bool ok = true;
    Ring k_ring, q_ring;              // key tiles; chunks of rows, or columns' rows
    Walk<MANY> w(tp, sm);

    if (warp == kTma) {
        // ------------------------------------------------ keys, and the chunks of rows
        const uint64_t policy = l2_policy_evict_first();
        for (; ok && w.more; w.next()) {
            const int stage = k_ring.at;
            if (k_ring.round > 0 && !(ok = warp_wait_for(&sm.k_empty[stage], k_ring.empty(), abort_flag))) break;
            uint8_t* dst = sK + stage * kKStage;
            const int k0 = w.t * kTile<MANY>;
            // a lane per load of `box` keys; what lies behind the length, or in a block outside the pool, is left out
            const int in = lane * tp.box, at = k0 + in;
            int64_t row = -1;
            if (in < kTile<MANY> && at < w.rows.n) row = key_row(p, w.b, w.h, at);
            const unsigned there = __ballot_sync(0xffffffffu, row >= 0);
            if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[stage], __popc(there) * tp.box * 128 * kH);
            __syncwarp();
            if (row >= 0)
                for (int hh = 0; hh < kH; ++hh) {
                    uint8_t* to = dst + ((in / kKeys) * kH + hh) * kKHalf + in % kKeys * 128;
                    // (few: read once, so first to leave the L2: what others keep there stays.  Twelve caches of 64 sequences in
                    // turn: 62.8 us a call, 63.6 without; three in turn, 1 GB in all: 56.6 and 63.1, as a part of each is still
                    // there the next time.  A prompt's keys are read again by the CTAs that have other rows of theirs)
                    if (MANY) tma_load_2d(to, &mp.k, &sm.k_full[stage], hh * 64, static_cast<int>(row));
                    else tma_load_2d_hint(to, &mp.k, &sm.k_full[stage], hh * 64, static_cast<int>(row), policy);
                }
            k_ring.next(tp.k_stages);
            if (MANY) {
                int qh;
                typename Walk<MANY>::Chunks ch = w.chunks(qh);
                for (int c = 0; c < w.take; ++c) {
                    const int qs = q_ring.at;
                    if (q_ring.round > 0 && !(ok = warp_wait_for(&sm.q_empty[qs], q_ring.empty(), abort_flag))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&sm.q_full[qs], kH * q_half);
                        for (int hh = 0; hh < kH; ++hh)
                            tma_load_2d(sQ + (qs * kH + hh) * q_half, &mp.q, &sm.q_full[qs], hh * 64, (w.b * p.Hq + w.h * tp.g + qh) * p.T + ch.i0);
                    }
                    ch.next();
                    if (ch.i0 == ch.begin) ++qh;
                    q_ring.next(tp.q_stages);
                }
            }
            __syncwarp();
        }
    } else if (warp >= kMma && warp < kRowsWarp) {
        // ------------------------------------------------ products
        const bool leader = elected();
        const int half = warp - kMma; // of the tile's keys
        const int buffers = MANY ? 2 : tp.buffers;
        Ring s_ring, l_ring;          // a score buffer for each product; many: two of each half
        for (; ok && w.more; w.next(), k_ring.next(tp.k_stages)) {
            const int ks = k_ring.at;
            if (!(ok = warp_wait_for(&sm.k_full[ks], k_ring.full(), abort_flag))) break;
            const uint64_t ka = sdesc_k128(smem_u32(sK + ks * kKStage + half * kH * kKHalf));
            const int n = MANY ? kChunk : max(16, min(tp.nq, (tp.g * w.rows.count - tp.row0 + 15) / 16 * 16));
            const uint32_t idesc = idesc_bf16_f32(kKeys, n);
            int qh;
            typename Walk<MANY>::Chunks ch{};
            if (MANY) ch = w.chunks(qh);
            for (int c = 0; c < w.take; ++c) {
                const int qs = q_ring.at;
                if (!(ok = warp_wait_for(&sm.q_full[qs], q_ring.full(), abort_flag))) break;
                if (!MANY || !unseen(w.rows, w.t * kTile<MANY> + half * kKeys, ch.i0)) {
                    const int buf = (MANY ? 2 * half : 0) + s_ring.at;
                    if (s_ring.round > 0 && !(ok = warp_wait_for(&sm.s_empty[buf], s_ring.empty(), abort_flag))) break;
                    s_ring.next(buffers);
                    if (MANY && !(ok = warp_wait_for(&sm.l_full[l_ring.at], l_ring.full(), abort_flag))) break;
                    tc_fence_after();
                    if (leader) {
                        // the rows' lse has come too: this arrival hands it on, the products' own says nothing of it.  (The
                        // weights' warps would wait 200 cycles for it in every chunk, these have the time.)
                        if (MANY) mbar_arrive(&sm.s_full[buf]);
                        const uint64_t qa = sdesc_k128(smem_u32(sQ + qs * kH * q_half));
                        // (an address is 16 bytes a unit in a descriptor)
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_bf16(tmem + buf * buf_cols, ka + (((k / 4) * kKHalf + (k % 4) * 32) >> 4),
                                     qa + static_cast<uint32_t>(((k / 4) * q_half + (k % 4) * 32) >> 4), idesc, k > 0);
                        mma_commit(&sm.s_full[buf]);
                    }
                }
                __syncwarp();
                if (!ok) break;
                if (MANY) {
                    if (leader) mma_commit(&sm.q_empty[qs]);
                    q_ring.next(tp.q_stages);
                    l_ring.next(4);
                    ch.next();
                }
            }
            if (!ok) break;
            if (leader) mma_commit(&sm.k_empty[ks]);
            if (!MANY && w.column_ends()) {
                if (leader) mma_commit(&sm.q_empty[q_ring.at]);
                q_ring.next(tp.q_stages);
            }
            __syncwarp();
        }
        if (leader) mma_commit(&sm.drain);
        __syncwarp();
    } else if (warp >= kRowsWarp) {
        // ------------------------------------------------ rows
        if constexpr (MANY) {
            // lse of a chunk's rows: four for each lane of the first warp
            int u = 0;
            if (warp == kRowsWarp)
                for (; ok && w.more; w.next()) {
                    int qh;
                    typename Walk<MANY>::Chunks ch = w.chunks(qh);
                    for (int c = 0; c < w.take; ++c, ++u) {
                        const int ls = u & 3;
                        float x[4];
                        for (int e = 0; e < 4; ++e) {
                            const int i = ch.i0 + lane * 4 + e;
                            x[e] = INFINITY;
                            if (i < w.rows.count) x[e] = p.lse[static_cast<int64_t>(w.b * p.Hq + w.h * tp.g + qh) * p.T + i];
                        }
                        if (u >= 4 && !(ok = warp_wait_for(&sm.l_empty[ls], (u / 4 - 1) & 1, abort_flag))) break;
                        for (int e = 0; e < 4; ++e) x[e] = isfinite(x[e]) ? -x[e] * kL2e : -INFINITY;
                        *reinterpret_cast<float4*>(&sm.nl2[ls][lane * 4]) = make_float4(x[0], x[1], x[2], x[3]);
                        // Rows that do not count may hold anything, and 0 times that need not be 0: zeros take their place, once
                        // they have come.  (A flag for the weights' warps to look at cost every chunk: prompts 124 us for 118.)
                        bool odd = false;
                        for (int e = 0; e < 4; ++e) odd |= x[e] == -INFINITY && ch.i0 + lane * 4 + e < w.rows.count;
                        if (__any_sync(0xffffffffu, odd)) {
                            // (the products wait for l_full, so the slot cannot be a turn further; as many slots as stages)
                            if (!(ok = warp_wait_for(&sm.q_full[q_ring.at], q_ring.full(), abort_flag))) break;
                            for (int e = 0; e < 4; ++e)
                                if (x[e] == -INFINITY)
                                    for (int i = 0; i < kH * 8; ++i)
                                        *reinterpret_cast<uint4*>(sQ + (q_ring.at * kH + i / 8) * q_half + (lane * 4 + e) * 128 + i % 8 * 16) = make_uint4(0, 0, 0, 0);
                            fence_proxy_async_smem();
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.l_full[ls]);
                        ch.next();
                        if (ch.i0 == ch.begin) ++qh;
                        q_ring.next(tp.q_stages);
                    }
                }
        } else {
            // a head's rows, 16 bytes a thread at a time, swizzled as the products read them
            bool fresh = true;        // the first tile of a column here
            for (; ok && w.more; w.next()) {
                if (fresh) {
                    const int qs = q_ring.at;
                    if (q_ring.round > 0 && !(ok = warp_wait_for(&sm.q_empty[qs], q_ring.empty(), abort_flag))) break;
                    const int total = min(tp.nq, tp.g * w.rows.count - tp.row0), padded = max(16, (total + 15) / 16 * 16);
                    const int tid = threadIdx.x - 32 * kRowsWarp;
                    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
                    const int64_t q0 = static_cast<int64_t>(w.b) * p.Hq + w.h * tp.g;
                    // lse, four rows a thread, and a path's nodes: on their way while the rows are
                    float l[4];
                    int ii[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = tid + 64 * k, rr = tp.row0 + r;
                        l[k] = INFINITY;
                        if (r < total) {
                            const int head = rr / w.rows.count;
                            ii[k] = rr - head * w.rows.count;
                            l[k] = p.lse[(q0 + head) * p.T + node_of(p, w.b, ii[k])];
                        }
                    }
                    const int node_at = p.path && lane < w.rows.count ? node_of(p, w.b, lane) : 0;
                    // Asynchronous copies, so that all of a thread's are on their way together; rows behind the last are zeros.
                    // A thread has the same 16 bytes of every 64 / (D / 8)-th row; which head's it is and which of it go in steps.  (With
                    // every row's address worked out by itself, and lse behind them, 8 sequences of 300 keys and 32 rows of 8 heads
                    // took 26 us where this takes 13)
                    constexpr int kParts = D / 8, kStep = 64 / kParts;
                    const int part = tid % kParts, count = max(w.rows.count, 1);
                    const int step_head = kStep / count, step_i = kStep - step_head * count;
                    int r = tid / kParts, gi = (tp.row0 + r) / count, i = tp.row0 + r - gi * count;
                    const int64_t head_size = static_cast<int64_t>(p.T) * D;
                    const __nv_bfloat16* from = q + (q0 + gi) * head_size + part * 8;
                    const uint32_t to = smem_u32(sQ + (qs * kH + part / 8) * q_half);
#pragma unroll 4
                    for (; r < padded; r += kStep) {
                        const int node = p.path ? __shfl_sync(0xffffffffu, node_at, i) : i;
                        const __nv_bfloat16* src = r < total ? from + node * D : q;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                                     ::"r"(to + r * 128 + ((part % 8) ^ (r & 7)) * 16), "l"(src), "r"(r < total ? 16 : 0) : "memory");
                        i += step_i;
                        from += step_head * head_size;
                        if (i >= count) {
                            i -= count;
                            from += head_size;
                        }
                    }
                    // the last key that each sees
                    bool odd = false;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int at = tid + 64 * k;
                        if (at < padded) {
                            const bool counts = isfinite(l[k]);
                            if (!counts && at < total) odd = true;
                            sm.nl2[qs][at] = counts ? -l[k] * kL2e : -INFINITY;
                            sm.last[qs][at] = counts ? w.rows.n - w.rows.count + ii[k] : -1;
                        }
                    }
                    odd = __any_sync(0xffffffffu, odd);
                    if (lane == 0) sm.odd[qs][warp - kRowsWarp] = odd;
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.q_full[qs]);
                    fresh = false;
                }
                if (w.column_ends()) {
                    fresh = true;
                    q_ring.next(tp.q_stages);
                }
            }
        }
    } else {
        // ------------------------------------------------ weights
        const int grp = warp >> 2, key = (warp & 3) * 32 + lane;
        if (blockIdx.x == 0) {
            // the status: sequences that make no sense, blocks outside the pool.  (A wait that runs out flags it
            // two seconds later.)
            int bad = 0;
            for (int b = warp; b < p.B; b += 4 * kGroups) {
                const Rows r = rows_of(p, b);
                if (!r.ok) {
                    bad = 1;
                } else if (p.table) {
                    const int used = (r.n + p.rows - 1) / p.rows;
                    for (int j = lane; j < used; j += 32) {
                        const int blk = p.table[static_cast<int64_t>(b) * p.max_blocks + j];
                        if (blk < 0 || blk >= p.num_blocks) bad = 1;
                    }
                }
            }
            if (bad) sm.bad = 1;
            asm volatile("bar.sync 1, %0;" ::"n"(128 * kGroups) : "memory");   // all of these warps come here, once, and wait for nobody else
            if (threadIdx.x == 0 && tp.row0 == 0) *static_cast<int4*>(p.ws) = make_int4(sm.bad ? SPEC_EINVAL : SPEC_OK, 0, 0, 0);
        }
        const unsigned long long c2 = pk2(p.scale * kL2e, p.scale * kL2e);
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        // column sums of key j where it lies, with what it had (`old`) on its way since the products began
        auto there = [&](int j) { return j < w.rows.n && (!p.table || key_row(p, w.b, w.h, j) >= 0); };
        auto place = [&](int j) { return (static_cast<int64_t>(w.b) * p.Hkv + w.h) * p.cap + j; };
        auto had = [&](int j) { return tp.row0 > 0 || (j < w.rows.n - w.rows.count && p.decay != 0.f) ? p.acc[place(j)] : 0.f; };
        auto store_sum = [&](int j, float old, float sum) {
            p.acc[place(j)] = tp.row0 > 0 ? old + sum : fmaf(p.decay, old, sum);
            if (j >= w.rows.n - w.rows.count && p.pos && tp.row0 == 0) p.pos[place(j)] = (p.seen ? p.seen[w.b] : w.rows.n) - w.rows.n + j;
        };
        if constexpr (MANY) {
            constexpr int W = 32;
            int u = 0;
            Ring s_ring;                                     // the half's score buffers
            for (; ok && w.more; w.next()) {
                const int k0 = w.t * kTile<MANY>, in_front = w.rows.n - w.rows.count;
                const int j = k0 + grp * kKeys + key;
                const bool mine = w.whole() && there(j);
                const float old = mine ? had(j) : 0.f;
                float sum = 0.f;
                int qh;
                typename Walk<MANY>::Chunks ch = w.chunks(qh);
                const int h0 = k0 + grp * kKeys;             // the group's half
                for (int c = 0; c < w.take; ++c, ++u, ch.next()) {
                    const int ls = u & 3;
                    // a chunk that the half does not see: its slot must not be given back for an earlier turn
                    if (unseen(w.rows, h0, ch.i0)) {
                        if (!(ok = warp_wait_for(&sm.l_full[ls], (u >> 2) & 1, abort_flag))) break;
                    } else {
                        const int buf = 2 * grp + s_ring.at;
                        const uint32_t parity = s_ring.full();
                        s_ring.next(2);
                        const float* nl2 = sm.nl2[ls];
                        const uint32_t s_addr = lane_base + buf * buf_cols;
                        unsigned long long part = pk2(0.f, 0.f);
                        uint32_t r[2][W];
                        unsigned long long l[2][W / 2];
                        if (!(ok = warp_wait_for(&sm.s_full[buf], parity, abort_flag))) break;
                        tc_fence_after();
                        load_scores(s_addr, r[0]);
                        load_lse<W>(nl2, l[0]);
                        if (w.rows.count - ch.i0 >= kChunk && h0 + kKeys - 1 <= in_front + ch.i0) {   // all see all
#pragma unroll
                            for (int x = 0; x < kChunk; x += W) {
                                const int now = x / W & 1, next = now ^ 1;
                                if (x + W < kChunk) load_lse<W>(nl2 + x + W, l[next]);
                                tmem_ld_wait();
                                if (x + W < kChunk) load_scores(s_addr + x + W, r[next]);
                                part = fadd2(part, weights(r[now], l[now], c2));
                            }
                        } else {
                            const int lo = h0 + key - in_front - ch.i0, cols = w.rows.count - ch.i0;   // columns from .. to that see this key
#pragma unroll 1
                            for (int x = 0; x < kChunk; x += W) {
                                uint32_t seen = lo <= x ? ~0u : lo >= x + W ? 0u : ~0u << (lo - x);
                                seen = cols >= x + W ? seen : cols <= x ? 0u : seen & ~(~0u << (cols - x));
                                if (x > 0) {
                                    load_scores(s_addr + x, r[0]);
                                    load_lse<W>(nl2 + x, l[0]);
                                }
                                tmem_ld_wait();
                                if (__any_sync(0xffffffffu, seen)) part = fadd2(part, masked(r[0], l[0], c2, seen));
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.s_empty[buf]);
                        float f0, f1;
                        upk2(part, f0, f1);
                        sum += f0 + f1;
                    }
                    if (lane == 0) mbar_arrive(&sm.l_empty[ls]);
                }
                if (!ok) break;
                if (w.whole()) {
                    if (mine) store_sum(j, old, sum);
                    continue;
                }
                // a tile that another CTA has a part of: the join puts them together
                const bool tail = w.c == 0;
                tp.parts[(static_cast<int64_t>(blockIdx.x) * 2 + tail) * 2 * kKeys + grp * kKeys + key] = sum;
                if (threadIdx.x == 0) {
                    Record& rec = tp.records[blockIdx.x];
                    if (tail) {
                        rec.tail = 1;
                        rec.b = w.b; rec.h = w.h; rec.t = w.t;
                    } else {
                        rec.head = 1;
                        rec.head_ends = w.c + w.take == w.head.chunks(w.t);
                    }
                }
            }
        } else {
            Ring s_ring;
            for (int u = 0; ok && w.more; w.next(), ++u, s_ring.next(tp.buffers)) {
                const int cs = q_ring.at;
                if ((u & 1) == grp) {
                    const int k0 = w.t * kTile<MANY>, j = k0 + key;
                    const bool mine = there(j);
                    const float old = mine ? had(j) : 0.f;
                    const int buf = s_ring.at;
                    if (!(ok = warp_wait_for(&sm.q_full[cs], q_ring.full(), abort_flag))) break;
                    if (!(ok = warp_wait_for(&sm.s_full[buf], s_ring.full(), abort_flag))) break;
                    tc_fence_after();
                    const uint32_t s_addr = lane_base + buf * buf_cols;
                    const float* nl2 = sm.nl2[cs];
                    const int cols = min(tp.nq, tp.g * w.rows.count - tp.row0);
                    unsigned long long part = pk2(0.f, 0.f);
                    if (cols > 0 && k0 + kKeys - 1 <= w.rows.n - w.rows.count && !(sm.odd[cs][0] | sm.odd[cs][1])) {   // all rows see all keys
                        const int steps = (cols + 15) / 16;
                        uint32_t r[2][16];
                        unsigned long long l[2][8];
                        tmem_ld16(s_addr, r[0]);
                        load_lse<16>(nl2, l[0]);
#pragma unroll 1
                        for (int x = 0; x < steps; x += 2) {
                            if (x + 1 < steps) load_lse<16>(nl2 + 16 * (x + 1), l[1]);
                            tmem_ld_wait();
                            if (x + 1 < steps) tmem_ld16(s_addr + 16 * (x + 1), r[1]);
                            part = fadd2(part, weights(r[0], l[0], c2));
                            if (x + 1 < steps) {
                                if (x + 2 < steps) load_lse<16>(nl2 + 16 * (x + 2), l[0]);
                                tmem_ld_wait();
                                if (x + 2 < steps) tmem_ld16(s_addr + 16 * (x + 2), r[0]);
                                part = fadd2(part, weights(r[1], l[1], c2));
                            }
                        }
                    } else {
#pragma unroll 1
                        for (int x = 0; x < cols; x += 16) {
                            uint32_t r[16];
                            tmem_ld16(s_addr + x, r);
                            // which of the warp's keys the column of each lane sees, turned into which columns see the lane's key
                            const int upto = x + (lane & 15) < cols ? sm.last[cs][x + (lane & 15)] - (j - lane) : -1;
                            const uint32_t seen = transpose_bits(upto >= 31 ? ~0u : upto < 0 ? 0u : (2u << upto) - 1) & 0xffffu;
                            unsigned long long l[8];
                            load_lse<16>(nl2 + x, l);
                            tmem_ld_wait();
                            part = fadd2(part, masked(r, l, c2, seen));
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.s_empty[buf]);
                    float f0, f1;
                    upk2(part, f0, f1);
                    if (mine) store_sum(j, old, f0 + f1);
                }
                if (w.column_ends()) {
                    // (a group without a tile in this column waits for its rows all the same: else it would give back a later
                    // turn of the slot in place of this one)
                    if (!(ok = warp_wait_for(&sm.q_full[cs], q_ring.full(), abort_flag))) break;
                    if (lane == 0) mbar_arrive(&sm.q_empty[cs]);
                    q_ring.next(tp.q_stages);
                }
            }
        }
    }
    if (!ok) {
        if (lane == 0) {
            flag_status(p.ws, SPEC_ETIMEOUT);
            *abort_flag = 1;
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // a wait ran out: let this CTA's own loads and MMAs land before it ends
        if (warp == kTma) {
            // every slot's last load: its barrier's phase, if it ever had one
            auto land = [&](uint64_t* full, const Ring& r, int n) {
                for (int i = 0; i < n; ++i) {
                    const uint32_t loads = r.round + (i < r.at ? 1 : 0);
                    if (loads > 0) mbar_wait(&full[i], (loads - 1) & 1, 100000000ull);
                }
            };
            land(sm.k_full, k_ring, tp.k_stages);
            if (MANY) land(sm.q_full, q_ring, tp.q_stages);
        }
    }
    // the products' last arrivals too: no CTA ends before what it has set off has come
    if (warp >= kMma && warp < kRowsWarp) mbar_wait(&sm.drain, 0, 100000000ull);
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// The tiles that were cut: the CTA in which one begins adds up its parts, in order.
__global__ void __launch_bounds__(2 * kKeys) k_weigh_join(const TcParams tp, int ctas) {
    griddep_wait();
    const Record rec = tp.records[blockIdx.x];
    if (!rec.tail) return;
    const Params& p = tp.p;
    float sum = tp.parts[(static_cast<int64_t>(blockIdx.x) * 2 + 1) * 2 * kKeys + threadIdx.x];
    int end = blockIdx.x + 1;         // one more than the CTA in which the tile ends, 32 records at a time
    for (; end < ctas; end += 32) {
        const int c = end + (threadIdx.x & 31);
        const unsigned ends = __ballot_sync(0xffffffffu, c >= ctas || tp.records[c].head_ends);
        if (ends) {
            end += __ffs(ends);
            break;
        }
    }
    end = min(end, ctas);
#pragma unroll 8
    for (int c = blockIdx.x + 1; c < end; ++c) sum += tp.parts[static_cast<int64_t>(c) * 4 * kKeys + threadIdx.x];
    const Rows rows = rows_of(p, rec.b);
    const int j = rec.t * kTile<true> + threadIdx.x;
    if (rows.ok && j < rows.n && key_row(p, rec.b, rec.h, j) >= 0) store(p, rec.b, rec.h, j, rows, sum);
}

// ---------------------------------------------------------------- host

constexpr size_t kSmem = 232448;      // of one CTA, all there is: no two share an SM's TMEM

static int few_rows(int g, int T, int P) { return g * (P ? P : T); }
// Rows of a prompt fill chunks of 128 of one query head, shorter ones go side by side, several heads in a pass.  A pass takes
// some 12 cycles for 128 keys and row, a chunk 980 however few of its rows there are.  In us, few and many: 8 sequences of 4000 keys
// and 8 heads of 8, 48 rows (two passes) 48, 68; 64 rows 57, 68; 80 rows 76, 74; of 300 keys 22, 16; 25, 16; 35, 17; in one pass, 32
// heads of one, 64 rows 16.5, 19.6; 128 rows 19.9, 19.4; 160 rows 22, 27.  So from 64 rows on, if they need more than a pass.
bool weigh_many(int g, int T, int P) { return !P && T >= 64 && static_cast<int64_t>(g) * T > kMostRows; }

size_t weigh_tc_bytes(int g, int T, int P) {
    return weigh_many(g, T, P) ? static_cast<size_t>(device_sm_count()) * (sizeof(Record) + 4 * kKeys * sizeof(float)) : 0;
}

template <int D, bool MANY>
static spec_status launch_tc(const Maps& m, TcParams& tp, cudaStream_t s) {
    constexpr size_t kStage = static_cast<size_t>(kTile<MANY>) * D * 2;
    const size_t q = static_cast<size_t>(tp.nq) * D * 2;
    tp.q_stages = MANY ? 4 : 2;       // many, D = 128: 64 KB of keys once, 32 KB of rows four times
    tp.buffers = MANY || tp.nq <= 128 ? 4 : 2;
    const size_t room = kSmem - 1024 - sizeof(Small) - tp.q_stages * q;
    tp.k_stages = static_cast<int>(std::min<size_t>(MANY ? 2 : kMaxStages, room / kStage));
    auto kern = k_weigh_tc<D, MANY>;
    SPEC_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)));
    const int ctas = device_sm_count();
    SPEC_CUDA_TRY(launch_ex("kv_weigh_tc", kern, dim3(ctas), dim3(kTcThreads), kSmem, s, true, m, tp));
    if (MANY) SPEC_CUDA_TRY(launch_ex("kv_weigh_join", k_weigh_join, dim3(ctas), dim3(2 * kKeys), 0, s, true, tp, ctas));
    return SPEC_OK;
}

spec_status weigh_tc_run(const Params& p, int D, void* scratch, cudaStream_t s) {
    Maps m;
    memset(&m, 0, sizeof(m));
    TcParams tp{};
    tp.p = p;
    tp.g = p.Hq / p.Hkv;
    tp.box = kKeys;
    if (p.table) {                    // a load lies inside one block and one tile
        tp.box = 16;
        while (tp.box < kKeys && p.rows % (2 * tp.box) == 0) tp.box *= 2;
    }
    const uint64_t k_rows = static_cast<uint64_t>(p.table ? p.num_blocks : p.B) * p.Hkv * p.rows;
    const uint64_t q_rows = static_cast<uint64_t>(p.B) * p.Hq * p.T;
    if (k_rows > 0x7fffffffull || q_rows > 0x7fffffffull) return fail(SPEC_EINVAL, "more than 2^31 rows of keys or queries");
    SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.k, p.k, k_rows, D, D, tp.box));
    SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.q, p.q, q_rows, D, D, kChunk));
    if (weigh_many(tp.g, p.T, p.path ? p.P : 0)) {
        tp.nq = kChunk;
        tp.records = static_cast<Record*>(scratch);
        tp.parts = reinterpret_cast<float*>(tp.records + device_sm_count());
        return D == 64 ? launch_tc<64, true>(m, tp, s) : launch_tc<128, true>(m, tp, s);
    }
    const int rows = few_rows(tp.g, p.T, p.path ? p.P : 0);
    tp.nq = std::min(kMostRows, (rows + 15) / 16 * 16);
    for (tp.row0 = 0; tp.row0 < rows; tp.row0 += kMostRows) {
        const spec_status st = D == 64 ? launch_tc<64, false>(m, tp, s) : launch_tc<128, false>(m, tp, s);
        if (st != SPEC_OK) return st;
    }
    return SPEC_OK;
}

}  // namespace weigh
}  // namespace spec
