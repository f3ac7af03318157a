// Eviction from the cache: every KV head of a sequence keeps `budget` keys.
//
// Kept are, in this order, the keys whose positions are protected (the first `sink` and the
// last `recent` of the sequence), then those that received the most attention weight; of equal ones the
// lower place in the cache.  The cache's order does not matter to attention over rotated keys,
// so kept keys in front of the budget stay where they are and the places of evicted ones are
// filled, in ascending order, by the kept keys behind it: a step that adds five keys to a full
// cache moves five rows, where closing the gaps would move half of the cache.
//
//   evict_pick   a CTA per (sequence, head): radix selection of the budget-th largest of
//                (protected, weight), then ordered lists of holes and of the keys that fill them;
//                moves weights and positions
//   evict_move   the rows of K and V, where the cache can hold many more rows than the budget (else
//                evict_pick's CTA moves its few itself and the second launch is saved)
// With another cache to go to, everything kept is copied there, place for place the same.
// Bound by memory, 8 bytes a key to choose and 4 rows' bytes for each that moves; a step of a full
// cache by the latency of the selection.
#include <algorithm>

#include "common.cuh"

namespace spec {
namespace evict {

constexpr int kCached = 49152;        // keys of a head whose ranks stay in shared memory
constexpr int kBins = 2048;           // of a digit of 11 bits
constexpr int kFew = 128;             // rows behind the budget that evict_pick moves itself
constexpr int kGone = 64;             // keys to evict that are looked for one by one
constexpr int kList = 512;            // candidates for them

struct Params {
    const char *k, *v;
    char *k_out, *v_out;              // the same, in place
    const float* acc;
    const int32_t* pos;
    float* acc_out;
    int32_t* pos_out;
    const int32_t *table, *out_table; // paged; out_table == table in place
    const int32_t *len, *seen;        // [B]; seen NULL: len
    int32_t* len_out;
    int B, Hkv, budget, sink, recent;
    int max_blocks, out_blocks, num_blocks;
    int rows, out_rows;               // positions of one (block, head)
    int cap, out_cap;                 // positions of one sequence (the stride of acc and pos)
    int row16;                        // 16-byte chunks of a row
    int here;                         // evict_pick moves the rows
    int in_place, cached;
    int2* moves;                      // [B * Hkv][most]: (to, from), ascending in both
    int32_t* source;                  // another cache: [B * Hkv][places], where each place's key comes from
    int32_t* count;                   // [B * Hkv]: moves, or places
    unsigned* bits;                   // longer caches than shared memory has room for: three maps of bits for each head
    int most, places;
    void* ws;
};

// Whether sequence b's length and table entries are sound, as far as thread t of N looks.
template <int N> __device__ __forceinline__ bool sound(const Params& p, int b, int t) {
    const int n = p.len[b];
    int bad = n < 0 || n > p.cap;
    if (!bad && p.table) {
        const int used = (n + p.rows - 1) / p.rows;
        for (int j = t; j < used; j += N) {
            const int blk = p.table[static_cast<size_t>(b) * p.max_blocks + j];
            if (blk < 0 || blk >= p.num_blocks) bad = 1;
        }
        if (!p.in_place) {
            const int out = (min(n, p.budget) + p.rows - 1) / p.rows;
            for (int j = t; j < out; j += N) {
                const int blk = p.out_table[static_cast<size_t>(b) * p.out_blocks + j];
                if (blk < 0 || blk >= p.num_blocks) bad = 1;
            }
        }
    }
    return !bad;
}

__device__ __forceinline__ int64_t row_at(const int32_t* table, int max_blocks, int rows, int Hkv, int b, int h, int at) {
    int64_t blk = b;
    if (table) {
        blk = table[static_cast<size_t>(b) * max_blocks + at / rows];
        at %= rows;
    }
    return (blk * Hkv + h) * rows + at;
}

__device__ __forceinline__ void move_chunk(const Params& p, int b, int h, int2 mv, int c, bool value) {
    const int64_t src = row_at(p.table, p.max_blocks, p.rows, p.Hkv, b, h, mv.y) * p.row16 + c;
    const int64_t dst = row_at(p.out_table, p.out_blocks, p.out_rows, p.Hkv, b, h, mv.x) * p.row16 + c;
    const uint4* from = reinterpret_cast<const uint4*>(value ? p.v : p.k);
    uint4* to = reinterpret_cast<uint4*>(value ? p.v_out : p.k_out);
    to[dst] = from[src];
}

// Exclusive prefix sums of two counts over the CTA; totals in t0, t1.
template <int kWarps> __device__ __forceinline__ void scan2(int (&part)[2][kWarps], int& a, int& b, int& t0, int& t1) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int x = a, y = b;
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) { x += u; y += v; }
    }
    __syncthreads();                  // an earlier scan's readers are through
    if (lane == 31) { part[0][warp] = x; part[1][warp] = y; }
    __syncthreads();
    // every warp adds up the warps' totals itself, a lane each
    int u = lane < kWarps ? part[0][lane] : 0, v = lane < kWarps ? part[1][lane] : 0;
    const int own0 = __shfl_sync(0xffffffffu, u, warp), own1 = __shfl_sync(0xffffffffu, v, warp);
    for (int o = 1; o < 32; o <<= 1) {
        const int m = __shfl_up_sync(0xffffffffu, u, o), k = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) { u += m; v += k; }
    }
    const int p0 = __shfl_sync(0xffffffffu, u, warp) - own0, p1 = __shfl_sync(0xffffffffu, v, warp) - own1;
    t0 = __shfl_sync(0xffffffffu, u, 31);
    t1 = __shfl_sync(0xffffffffu, v, 31);
    a = p0 + x - a;
    b = p1 + y - b;
}

// Few keys too many, a step's: the e = n - budget ones of the lowest (protected, weight, higher place first) are
// among the e / warps lowest of each warp's threads or below the largest of those, some tens in all, and
// are ranked by counting.  Two passes over the keys and no histogram: 24 us became 12 for 512 heads of 2065.
// Returns the moves, in s_moves, or -1 where too many keys are equal to tell them apart so.
struct Few {
    unsigned long long list[kList], gone_late;
    int2 moves[kGone];
    int gone[kGone];
    unsigned bound[32];
    int count;
};
template <int kThreads> __device__ __noinline__ int pick_few(Few& s, const Params& p, const float* acc, const int32_t* pos, int n, int64_t since) {
    constexpr int kWarps = kThreads / 32, kKeep = 8;   // keys a thread has in registers; the others are read twice
    const int e = n - p.budget, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto key = [&](int i, int at, float x) {
        const unsigned long long safe = at < p.sink || at >= since;
        return (safe << 54) | (static_cast<unsigned long long>(order_key(x)) << 22) | static_cast<unsigned>((1 << 22) - 1 - i);
    };
    int at[kKeep];
    float x[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i < n) {
            at[k] = pos[i];
            x[k] = acc[i];
        }
    }
    unsigned long long kept[kKeep];
    unsigned low = 0xffffffffu;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = threadIdx.x + k * kThreads;
        kept[k] = i < n ? key(i, at[k], x[k]) : ~0ull;
        low = min(low, static_cast<unsigned>(kept[k] >> 23));
    }
    for (int i = threadIdx.x + kKeep * kThreads; i < n; i += kThreads) low = min(low, static_cast<unsigned>(key(i, pos[i], acc[i]) >> 23));
    unsigned kth = 0;
    for (int k = 0; k < (e + kWarps - 1) / kWarps; ++k) {
        kth = __reduce_min_sync(0xffffffffu, low);
        const unsigned who = __ballot_sync(0xffffffffu, low == kth);
        if (lane == __ffs(who) - 1) low = 0xffffffffu;
    }
    if (lane == 0) s.bound[warp] = kth;
    if (threadIdx.x == 0) {
        s.count = 0;
        s.gone_late = 0;
    }
    __syncthreads();
    unsigned bound = s.bound[0];
    for (int i = 1; i < kWarps; ++i) bound = max(bound, s.bound[i]);
    auto offer = [&](unsigned long long k) {
        if (static_cast<unsigned>(k >> 23) <= bound && k != ~0ull) {
            const int at = atomicAdd(&s.count, 1);
            if (at < kList) s.list[at] = k;
        }
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k) offer(kept[k]);
    for (int i = threadIdx.x + kKeep * kThreads; i < n; i += kThreads) offer(key(i, pos[i], acc[i]));
    __syncthreads();
    const int m = s.count;
    if (m > kList) return -1;
    for (int i = threadIdx.x; i < m; i += kThreads) {
        const unsigned long long k = s.list[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < m; ++j) rank += s.list[j] < k;
        if (rank < e) {
            const int at = (1 << 22) - 1 - static_cast<int>(k & ((1 << 22) - 1));
            s.gone[rank] = at < p.budget ? at : -1;
            if (at >= p.budget) atomicOr(&s.gone_late, 1ull << (at - p.budget));
        }
    }
    __syncthreads();
    const unsigned long long late = ~s.gone_late & (e == 64 ? ~0ull : (1ull << e) - 1);   // kept ones behind the budget
    if (static_cast<int>(threadIdx.x) < e) {
        const int hole = s.gone[threadIdx.x];
        int before = 0;
        for (int j = 0; j < e; ++j) before += s.gone[j] >= 0 && s.gone[j] < hole;
        if (hole >= 0) s.moves[before].x = hole;
        if ((late >> threadIdx.x) & 1) s.moves[__popcll(late & ((1ull << threadIdx.x) - 1))].y = p.budget + threadIdx.x;
    }
    __syncthreads();
    return __popcll(late);
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) k_pick(const Params p) {
    constexpr int kWarps = kThreads / 32;
    extern __shared__ unsigned s_rank[];              // ranks of the keys, where they fit
    __shared__ int s_hist[kBins];
    __shared__ int part[2][kWarps];
    __shared__ int s_digit, s_above, s_equal;
    __shared__ unsigned s_ends[2][kWarps];
    __shared__ Few few;
    const int h = blockIdx.x, b = blockIdx.y;
    griddep_wait();                   // the stream's kernel before this one may still run: its results are behind here
    griddep_launch();
    if (h == p.Hkv) {                 // one CTA more: the status word, which no other writes
        if (b != 0) return;
        int bad = 0;
        for (int i = threadIdx.x >> 5; i < p.B; i += kWarps) bad |= !sound<32>(p, i, threadIdx.x & 31);
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *static_cast<int4*>(p.ws) = make_int4(bad ? SPEC_EINVAL : SPEC_OK, 0, 0, 0);
        return;
    }
    const int bh = b * p.Hkv + h;
    const int n = p.len[b];
    const bool ok = __syncthreads_and(sound<kThreads>(p, b, threadIdx.x));
    if (h == 0 && threadIdx.x == 0) p.len_out[b] = ok ? min(n, p.budget) : n;
    const bool all = n <= p.budget;   // nothing is evicted
    if (!ok || (all && p.in_place)) {
        if (threadIdx.x == 0) p.count[bh] = 0;
        return;
    }
    const float* acc = p.acc + static_cast<size_t>(bh) * p.cap;
    const int32_t* pos = p.pos + static_cast<size_t>(bh) * p.cap;
    float* acc_out = p.acc_out + static_cast<size_t>(bh) * p.out_cap;
    int32_t* pos_out = p.pos_out + static_cast<size_t>(bh) * p.out_cap;
    int2* moves = p.moves + static_cast<size_t>(bh) * p.most;
    const int2* found = moves;
    int count = 0;
    const int64_t since = static_cast<int64_t>(p.seen ? p.seen[b] : n) - p.recent;
    if (!all && n - p.budget <= kGone) {
        count = pick_few<kThreads>(few, p, acc, pos, n, since);
        if (count >= 0) {
            found = few.moves;
            if (!p.here && static_cast<int>(threadIdx.x) < count) moves[threadIdx.x] = few.moves[threadIdx.x];
        }
    }
    if (!all && found == moves) {
        // Ranks come to shared memory where they fit, and of each key a bit in one of three maps: protected; ranked
        // above the border; equal to it.  What follows the ranks goes by words of 32 keys: with a look at every
        // key of a thread's run instead it took 5 us more for 16384 keys.
        const bool cached = n <= p.cached;
        const int words = (n + 31) / 32;
        unsigned *safe_bits, *above_bits, *equal_bits;
        if (p.cap <= kCached) {
            safe_bits = s_rank + p.cached;
            above_bits = safe_bits + (p.cap + 31) / 32;
            equal_bits = above_bits + (p.cap + 31) / 32;
        } else {
            safe_bits = p.bits + static_cast<size_t>(bh) * 3 * ((p.cap + 31) / 32);
            above_bits = safe_bits + words;
            equal_bits = above_bits + words;
        }
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        int mine = 0;
        unsigned least = 0xffffffffu, largest = 0;       // rank of the others
        constexpr int kAhead = 8;     // words of a warp on their way together (one by one: 33 us for 16384 keys)
        for (int w0 = warp; w0 < words; w0 += kAhead * kWarps) {
            int at[kAhead];
            float x[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = (w0 + k * kWarps) * 32 + lane;
                if (i < n) at[k] = pos[i];
                if (i < n) x[k] = acc[i];
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int w = w0 + k * kWarps, i = w * 32 + lane;
                if (w >= words) break;
                const unsigned bits = __ballot_sync(0xffffffffu, i < n && (at[k] < p.sink || at[k] >= since));
                if (i < n) {
                    const unsigned r = order_key(x[k]);
                    if (cached) s_rank[i] = r;
                    if (!(bits >> lane & 1)) {
                        least = min(least, r);
                        largest = max(largest, r);
                    }
                }
                if (lane == 0) {
                    safe_bits[w] = bits;
                    mine += __popc(bits);
                }
            }
        }
        least = __reduce_min_sync(0xffffffffu, least);
        largest = __reduce_max_sync(0xffffffffu, largest);
        if (lane == 0) {
            s_ends[0][warp] = least;
            s_ends[1][warp] = largest;
        }
        int zero = 0, safe, none;
        scan2(part, mine, zero, safe, none);
        least = __reduce_min_sync(0xffffffffu, lane < kWarps ? s_ends[0][lane] : 0xffffffffu);
        largest = __reduce_max_sync(0xffffffffu, lane < kWarps ? s_ends[1][lane] : 0u);
        auto rank_at = [&](int i) { return cached ? s_rank[i] : order_key(acc[i]); };
        // all protected ones are kept and the best of the others, or the best of the protected ones
        const bool among_safe = safe > p.budget;
        const unsigned flip = among_safe ? 0u : ~0u;     // safe_bits[w] ^ flip: keys in play
        int want = among_safe ? p.budget : p.budget - safe;
        // The want-th largest rank of those in play, by digits of eleven bits.  The digits begin at the highest bit in which the
        // ranks differ from the least: the weights' exponents are much the same, and with digits of the rank itself they met
        // in a few counters (64.4 us with the copies for 128 heads of up to 16384 keys, so 62.9).  A digit that leaves no more than are wanted is the last.
        const bool choose = want > 0;
        unsigned border = 0;          // ranks from here on are above those that are kept in part
        if (choose) {
            if (among_safe) {
                least = 0;
                largest = 0xffffffffu;
            }
            const int bits = 32 - __clz(largest - least);
            int shift = max(bits - 11, 0), width = bits - shift;
            unsigned prefix = 0, mask = 0;
            for (;;) {
                const unsigned digits = (1u << width) - 1;
                for (int i = threadIdx.x; i < kBins; i += kThreads) s_hist[i] = 0;
                __syncthreads();
#pragma unroll 4
                for (int w = warp; w < words; w += kWarps) {
                    const int i = w * 32 + lane;
                    const unsigned x = (i < n ? rank_at(i) : 0) - least;
                    if (i < n && ((safe_bits[w] ^ flip) >> lane & 1) && (x & mask) == prefix) atomicAdd(&s_hist[(x >> shift) & digits], 1);
                }
                __syncthreads();
                // thread t has bins kBins - 1 - kEach t and those below, kEach in all
                constexpr int kEach = kBins / kThreads;
                int c[kEach], above = 0, all_of, skip = 0;
#pragma unroll
                for (int j = 0; j < kEach; ++j) above += c[j] = s_hist[kBins - 1 - kEach * threadIdx.x - j];
                scan2(part, above, skip, all_of, none);
#pragma unroll
                for (int j = 0; j < kEach; ++j) {
                    if (above < want && above + c[j] >= want) {
                        s_digit = kBins - 1 - kEach * threadIdx.x - j;
                        s_above = above;
                        s_equal = c[j];
                    }
                    above += c[j];
                }
                __syncthreads();
                prefix |= static_cast<unsigned>(s_digit) << shift;
                mask |= digits << shift;
                want -= s_above;      // now: how many of those equal so far are wanted
                const bool whole = want == s_equal;
                if (whole) want = 0;
                if (whole || shift == 0) {
                    border = least + prefix + (whole ? 0 : 1);
                    break;
                }
                width = min(shift, 11);
                shift -= width;
            }
#pragma unroll 4
            for (int w = warp; w < words; w += kWarps) {
                const int i = w * 32 + lane;
                const unsigned r = i < n ? rank_at(i) : 0, play = safe_bits[w] ^ flip;
                const unsigned up = __ballot_sync(0xffffffffu, i < n && r >= border) & play, eq = __ballot_sync(0xffffffffu, i < n && r == border - 1) & play;
                if (lane == 0) {
                    above_bits[w] = among_safe ? up : up | safe_bits[w];
                    equal_bits[w] = eq;   // (looked at where some of them are wanted)
                }
            }
        }
        __syncthreads();
        // a run of words per thread: the equal ones that are kept are the first `want`; then holes in front of the
        // budget and kept keys behind it
        const int run = (words + kThreads - 1) / kThreads;
        const int w0 = min(words, static_cast<int>(threadIdx.x) * run), w1 = min(words, w0 + run);
        int equal = 0, skip = 0, t0, t1;
        if (want > 0)
            for (int w = w0; w < w1; ++w) equal += __popc(equal_bits[w]);
        scan2(part, equal, skip, t0, t1);
        int holes = 0, late = 0;
        auto in_front = [&](int w) {  // keys of the word in front of the budget
            const int k = p.budget - w * 32;
            return k >= 32 ? ~0u : k <= 0 ? 0u : (1u << k) - 1;
        };
        auto inside = [&](int w) { return n - w * 32 >= 32 ? ~0u : (1u << (n - w * 32)) - 1; };
        for (int w = w0; w < w1; ++w) {
            unsigned kept = choose ? above_bits[w] : safe_bits[w];   // (nothing wanted beside the protected ones)
            if (want > 0)
                for (unsigned eq = equal_bits[w]; eq && equal < want; eq &= eq - 1, ++equal) kept |= eq & -eq;
            above_bits[w] = kept;
            holes += __popc(in_front(w) & inside(w) & ~kept);
            late += __popc(kept & ~in_front(w));
        }
        scan2(part, holes, late, t0, t1);
        count = t0;                   // as many keys come from behind the budget as there are holes in front
        for (int w = w0; w < w1; ++w) {
            for (unsigned m = in_front(w) & inside(w) & ~above_bits[w]; m; m &= m - 1) moves[holes++].x = w * 32 + __ffs(m) - 1;
            for (unsigned m = above_bits[w] & ~in_front(w); m; m &= m - 1) moves[late++].y = w * 32 + __ffs(m) - 1;
        }
        __syncthreads();
    }
    if (!p.in_place) {
        // places from their own key, those of evicted ones from behind the budget
        const int m = min(n, p.budget);
        int32_t* source = p.source + static_cast<size_t>(bh) * p.places;
        for (int i = threadIdx.x; i < m; i += kThreads) source[i] = i;
        __syncthreads();
        for (int i = threadIdx.x; i < count; i += kThreads) source[found[i].x] = found[i].y;
        __syncthreads();
        for (int i0 = threadIdx.x; i0 < m; i0 += 4 * kThreads) {
            int j[4], at[4];
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) j[k] = i0 + k * kThreads < m ? source[i0 + k * kThreads] : 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[k] = acc[j[k]];
                at[k] = pos[j[k]];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i0 + k * kThreads < m) {
                    acc_out[i0 + k * kThreads] = x[k];
                    pos_out[i0 + k * kThreads] = at[k];
                }
        }
        if (threadIdx.x == 0) p.count[bh] = m;
        return;
    }
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const int2 mv = found[i];
        acc_out[mv.x] = acc[mv.y];
        pos_out[mv.x] = pos[mv.y];
    }
    if (threadIdx.x == 0) p.count[bh] = count;
    if (p.here) {
        const int units = count * p.row16 * 2;
        for (int u = threadIdx.x; u < units; u += kThreads) {
            const int c = u % p.row16, r = u / p.row16;
            move_chunk(p, b, h, found[r >> 1], c, r & 1);
        }
    }
}

constexpr int kMoveThreads = 256;
constexpr int kBatch = 4;             // rows of K and V that a thread has under way

// Rows of K and V, a thread per 16 bytes of a row of each.
__global__ void __launch_bounds__(kMoveThreads) k_move(const Params p) {
    const int h = blockIdx.y % p.Hkv, b = blockIdx.y / p.Hkv, bh = blockIdx.y;
    const int rows = kMoveThreads / p.row16, c = threadIdx.x % p.row16, row0 = threadIdx.x / p.row16;   // row16 <= 256
    griddep_wait();
    if (row0 >= rows) return;
    const int count = p.count[bh];
    const int2* moves = p.moves + static_cast<size_t>(bh) * p.most;
    const int32_t* source = p.source + static_cast<size_t>(bh) * p.places;
    const uint4 *k = reinterpret_cast<const uint4*>(p.k), *v = reinterpret_cast<const uint4*>(p.v);
    uint4 *ko = reinterpret_cast<uint4*>(p.k_out), *vo = reinterpret_cast<uint4*>(p.v_out);
    const int step = gridDim.x * rows;
    for (int r = blockIdx.x * rows + row0; r < count; r += kBatch * step) {
        uint4 x[kBatch], y[kBatch];
        int to[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int q = r + i * step;
            if (q >= count) continue;
            const int2 mv = p.in_place ? moves[q] : make_int2(q, source[q]);
            to[i] = mv.x;
            const int64_t src = row_at(p.table, p.max_blocks, p.rows, p.Hkv, b, h, mv.y) * p.row16 + c;
            x[i] = k[src];
            y[i] = v[src];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (r + i * step >= count) continue;
            const int64_t dst = row_at(p.out_table, p.out_blocks, p.out_rows, p.Hkv, b, h, to[i]) * p.row16 + c;
            ko[dst] = x[i];
            vo[dst] = y[i];
        }
    }
}

int most_moves(int cap, int budget) { return std::max(1, std::min(budget, cap - std::min(budget, cap))); }
// (as much for a cache evicted in place as for another one)
size_t bytes_for(int B, int Hkv, int cap, int budget) {
    const size_t heads = static_cast<size_t>(B) * Hkv;
    return kWsHeader + round_up(heads * 4, 256) + round_up(heads * static_cast<size_t>(most_moves(cap, budget)) * sizeof(int2), 256) +
           round_up(heads * std::min(budget, cap) * 4, 256) + (cap > kCached ? heads * 3 * ((cap + 31) / 32) * 4 : 0);
}

spec_status check_sizes(int B, int Hkv, int64_t cap, int budget) {
    if (B < 1 || B > 65535) return fail(SPEC_EINVAL, "B = %d out of 1..65535", B);
    if (Hkv < 1 || Hkv > 1024 || static_cast<int64_t>(B) * Hkv > 65535) return fail(SPEC_EINVAL, "Hkv = %d out of 1..1024, or B * Hkv above 65535", Hkv);
    if (cap < 1 || cap > (1 << 22)) return fail(SPEC_EINVAL, "%lld positions out of 1..2^22", static_cast<long long>(cap));
    if (budget < 1 || budget > (1 << 22)) return fail(SPEC_EINVAL, "budget = %d out of 1..2^22", budget);
    return SPEC_OK;
}

bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + static_cast<uintptr_t>(bn) && y < x + static_cast<uintptr_t>(an);
}

spec_status run(Params& p, int D, spec_dtype dt, size_t ws_bytes, cudaStream_t s) {
    spec_status st = check_sizes(p.B, p.Hkv, p.cap, p.budget);
    if (st != SPEC_OK) return st;
    if (dt != SPEC_BF16 && dt != SPEC_F32) return fail(SPEC_EINVAL, "dtype %d unknown", static_cast<int>(dt));
    const int es = dt == SPEC_BF16 ? 2 : 4;
    if (D < 1 || D > 1024 || (D * es) % 16) return fail(SPEC_EINVAL, "D = %d: 1..1024 and a multiple of 16 bytes", D);
    if (p.sink < 0 || p.recent < 0 || static_cast<int64_t>(p.sink) + p.recent > p.budget)
        return fail(SPEC_EINVAL, "sink = %d, recent = %d: not negative, together at most the budget of %d", p.sink, p.recent, p.budget);
    if (!p.k || !p.v || !p.acc || !p.pos || !p.len || !p.len_out) return fail(SPEC_EINVAL, "the cache, acc, pos, prefix_len and len_out must not be NULL");
    if (!aligned16(p.k) || !aligned16(p.v) || !aligned16(p.k_out) || !aligned16(p.v_out)) return fail(SPEC_EALIGN, "the caches must be 16-byte aligned");
    const void* small[] = {p.acc, p.pos, p.acc_out, p.pos_out, p.table, p.out_table, p.len, p.seen, p.len_out};
    for (const void* x : small)
        if (!aligned4(x)) return fail(SPEC_EALIGN, "acc, pos, lengths and block tables must be 4-byte aligned");
    if (overlap(p.len_out, 4ll * p.B, p.len, 4ll * p.B) || (p.seen && overlap(p.len_out, 4ll * p.B, p.seen, 4ll * p.B)))
        return fail(SPEC_EINVAL, "len_out overlaps prefix_len or seen, which every head reads");
    const int64_t heads = static_cast<int64_t>(p.B) * p.Hkv;
    if (!p.in_place) {
        if (p.out_cap < std::min(p.budget, p.cap)) return fail(SPEC_EINVAL, "the other cache holds %d positions, fewer than are kept", p.out_cap);
        const int64_t a = heads * p.cap * 4, o = heads * p.out_cap * 4;
        const void* outs[] = {p.acc_out, p.pos_out};
        const void* ins[] = {p.acc, p.pos};
        for (const void* x : outs)
            for (const void* y : ins)
                if (overlap(x, o, y, a)) return fail(SPEC_EINVAL, "acc_out or pos_out overlaps acc or pos");
        if (overlap(p.acc_out, o, p.pos_out, o)) return fail(SPEC_EINVAL, "acc_out overlaps pos_out");
        if (!p.table) {
            const int64_t ib = heads * p.cap * D * es, ob = heads * p.out_cap * D * es;
            if (overlap(p.k_out, ob, p.k, ib) || overlap(p.k_out, ob, p.v, ib) || overlap(p.v_out, ob, p.k, ib) ||
                overlap(p.v_out, ob, p.v, ib) || overlap(p.k_out, ob, p.v_out, ob))
                return fail(SPEC_EINVAL, "the caches overlap");
        }
    }
    p.row16 = D * es / 16;
    p.most = most_moves(p.cap, p.budget);
    p.places = std::min(p.budget, p.cap);
    const size_t need = bytes_for(p.B, p.Hkv, p.cap, p.budget);
    if (!p.ws || ws_bytes < need) return fail(SPEC_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
    if (!aligned16(p.ws)) return fail(SPEC_EALIGN, "workspace must be 16-byte aligned");
    p.count = reinterpret_cast<int32_t*>(static_cast<char*>(p.ws) + kWsHeader);
    p.moves = reinterpret_cast<int2*>(static_cast<char*>(p.ws) + kWsHeader + round_up(static_cast<size_t>(heads) * 4, 256));
    p.source = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(p.moves) + round_up(static_cast<size_t>(heads) * p.most * sizeof(int2), 256));
    p.bits = reinterpret_cast<unsigned*>(reinterpret_cast<char*>(p.source) + round_up(static_cast<size_t>(heads) * p.places * 4, 256));
    p.here = p.in_place && p.most <= kFew;
    p.cached = std::min(p.cap, kCached);
    const size_t smem = static_cast<size_t>(p.cached) * 4 + (p.cap <= kCached ? 3 * ((p.cap + 31) / 32) * 4 : 0);
    // a full cache's step is a chain of short stages, which 256 threads go through fastest (8.1 us for 512 heads of 2065
    // keys, 512 threads 11.5); selections by digits, few of which share an SM anyway, get all of its threads
    const bool step = p.cap - p.budget <= kGone && p.cap <= 4096;
    auto pick = step ? k_pick<256> : k_pick<1024>;
    if (smem > 30000) SPEC_CUDA_TRY(cudaFuncSetAttribute(pick, cudaFuncAttributeMaxDynamicSharedMemorySize, kCached * 4 + kCached / 8 * 3));
    SPEC_CUDA_TRY(launch_ex("evict_pick", pick, dim3(p.Hkv + 1, p.B), dim3(step ? 256 : 1024), smem, s, true, p));
    if (!p.here) {
        const int64_t rows = kBatch * (kMoveThreads / p.row16);
        const int64_t most = ((p.in_place ? p.most : p.places) + rows - 1) / rows;
        const int64_t want = (16 * device_sm_count() + heads - 1) / heads;
        SPEC_CUDA_TRY(launch_ex("evict_move", k_move, dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min(most, want))), static_cast<unsigned>(heads)),
                                dim3(kMoveThreads), 0, s, true, p));
    }
    return SPEC_OK;
}

}  // namespace evict
}  // namespace spec

using namespace spec;

extern "C" size_t kv_evict_workspace_size(int32_t B, int32_t Hkv, int32_t Lmax, int32_t budget) {
    clear_error();
    if (evict::check_sizes(B, Hkv, Lmax, budget) != SPEC_OK) return 0;
    return evict::bytes_for(B, Hkv, Lmax, budget);
}

extern "C" spec_status kv_evict(void* k_cache, void* v_cache, const int32_t* prefix_len, const int32_t* seen, float* acc,
                                int32_t* pos, int32_t B, int32_t Hkv, int32_t Lmax, int32_t D, int32_t budget, int32_t sink,
                                int32_t recent, void* k_out, void* v_out, float* acc_out, int32_t* pos_out, int32_t Lout,
                                int32_t* len_out, spec_dtype dt, void* ws, size_t ws_bytes, spec_stream_t s) {
    clear_error();
    evict::Params p{};
    p.in_place = !k_out && !v_out && !acc_out && !pos_out;
    if (!p.in_place && (!k_out || !v_out || !acc_out || !pos_out)) return fail(SPEC_EINVAL, "k_out, v_out, acc_out and pos_out go together");
    if (!p.in_place && (Lout < 1 || Lout > (1 << 22))) return fail(SPEC_EINVAL, "Lout = %d out of 1..2^22", Lout);
    p.k = static_cast<char*>(k_cache); p.v = static_cast<char*>(v_cache); p.acc = acc; p.pos = pos;
    p.k_out = static_cast<char*>(p.in_place ? k_cache : k_out); p.v_out = static_cast<char*>(p.in_place ? v_cache : v_out);
    p.acc_out = p.in_place ? acc : acc_out; p.pos_out = p.in_place ? pos : pos_out;
    p.len = prefix_len; p.seen = seen; p.len_out = len_out;
    p.B = B; p.Hkv = Hkv; p.budget = budget; p.sink = sink; p.recent = recent;
    p.rows = p.cap = Lmax; p.out_rows = p.out_cap = p.in_place ? Lmax : Lout; p.ws = ws;
    return evict::run(p, D, dt, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}

extern "C" spec_status kv_evict_paged(void* k_pool, void* v_pool, int32_t num_blocks, const int32_t* block_table,
                                      int32_t max_blocks, int32_t block_size, const int32_t* prefix_len, const int32_t* seen,
                                      float* acc, int32_t* pos, int32_t B, int32_t Hkv, int32_t D, int32_t budget, int32_t sink,
                                      int32_t recent, const int32_t* out_table, int32_t out_blocks, float* acc_out,
                                      int32_t* pos_out, int32_t* len_out, spec_dtype dt, void* ws, size_t ws_bytes,
                                      spec_stream_t s) {
    clear_error();
    if (num_blocks < 1 || max_blocks < 1 || block_size < 1)
        return fail(SPEC_EINVAL, "num_blocks = %d, max_blocks = %d, block_size = %d must be positive", num_blocks,
                    max_blocks, block_size);
    if (static_cast<int64_t>(max_blocks) * block_size > (1 << 22))
        return fail(SPEC_EINVAL, "max_blocks * block_size = %lld positions exceed 2^22",
                    static_cast<long long>(max_blocks) * block_size);
    if (!block_table) return fail(SPEC_EINVAL, "block_table must not be NULL");
    evict::Params p{};
    p.in_place = !out_table && !acc_out && !pos_out;
    if (!p.in_place && (!out_table || !acc_out || !pos_out)) return fail(SPEC_EINVAL, "out_table, acc_out and pos_out go together");
    if (!p.in_place && (out_blocks < 1 || static_cast<int64_t>(out_blocks) * block_size > (1 << 22)))
        return fail(SPEC_EINVAL, "out_blocks = %d: 1.. and at most 2^22 positions", out_blocks);
    p.k = p.k_out = static_cast<char*>(k_pool); p.v = p.v_out = static_cast<char*>(v_pool); p.acc = acc; p.pos = pos;
    p.acc_out = p.in_place ? acc : acc_out; p.pos_out = p.in_place ? pos : pos_out;
    p.table = block_table; p.out_table = p.in_place ? block_table : out_table;
    p.max_blocks = max_blocks; p.out_blocks = p.in_place ? max_blocks : out_blocks; p.num_blocks = num_blocks;
    p.len = prefix_len; p.seen = seen; p.len_out = len_out;
    p.B = B; p.Hkv = Hkv; p.budget = budget; p.sink = sink; p.recent = recent;
    p.rows = p.out_rows = block_size; p.cap = max_blocks * block_size;
    p.out_cap = p.in_place ? p.cap : out_blocks * block_size; p.ws = ws;
    return evict::run(p, D, dt, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}
