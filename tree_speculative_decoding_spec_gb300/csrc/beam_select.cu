// Selection of a beam search: of B sequences with W beams each, the K best continuations
// over beams and vocabulary.
//
//   score(w, t) = scores[w] + x[w, t] - log sum_u exp x[w, u],   rank by score / length^alpha
//
// Bound by memory: every logit of a live beam is read once, and nothing of the
// vocabulary's size is written.  One pass over a row gives its maximum, its sum of
// exponentials and its K largest logits:
//   beam_slices  a CTA per row and slice of the vocabulary.  A row's candidates are ordered by
//                the logit alone, so they need no log-sum.  A running threshold, the K-th largest
//                logit so far, lets through some K ln(chunks) of all elements; a thread
//                compares it with the maximum of its 16 or 32 elements, which the sum needs anyway.
//   beam_join    a CTA per sequence: log-sums of the rows from their slices, then the K best of
//                W * slices * K candidates by (rank, beam, token).  Ranks are in 64 bits: at a score
//                of -20 neighbouring 32-bit numbers are 2e-6 apart, more than the logits of
//                two beams often are.
// Candidates are 64-bit keys (the logit's order, then the token, lower ones first), so that
// equal logits have one order and results do not depend on which thread came first.
#include <algorithm>

#include "common.cuh"
#include "tc.cuh"

namespace spec {
namespace beam {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVecs = 4;              // 16-byte loads of a thread and chunk
constexpr int kPerSm = 6;             // CTAs of an SM: loads in flight come from the others while one works
constexpr int kCap = 1024;            // candidates a slice holds at most
constexpr int kFound = 512;           // vectors of a stretch with candidates in them
constexpr int kMaxSlices = 32;        // one lane each in the join
constexpr int kJoinCap = 1024;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
    const void* logits;
    int64_t stride;                   // elements between rows
    const float* scores;
    const int32_t *ended, *length;    // or NULL
    int B, W, V, K, eos, slices, per; // per: 16-byte vectors of a slice
    float alpha;
    unsigned long long* cand;         // [B * W][slices][K]
    float2* sums;                     // [B * W][slices]: maximum, sum of exp(x - maximum)
    int32_t *token, *parent;
    float* score;
    int32_t *ended_out, *length_out;
    void* ws;
};

enum State { kDead = 0, kLive = 1, kEnded = 2 };
__device__ __forceinline__ State state_of(const Params& p, int row) {
    if (!isfinite(p.scores[row])) return kDead;
    return p.ended && p.ended[row] != 0 ? kEnded : kLive;
}

// 16 bytes of a row: NaN becomes -inf where they are loaded, in one instruction for a word.
template <typename T> struct Vec {
    static constexpr int E = 16 / sizeof(T);
    static __device__ __forceinline__ uint32_t& word(uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
    static __device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
    static __device__ __forceinline__ void clean(uint4& v);
    static __device__ __forceinline__ float at(const uint4& v, int e);
    static __device__ __forceinline__ float top(const uint4& v);
};
template <> __device__ __forceinline__ void Vec<float>::clean(uint4& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) word(v, i) = __float_as_uint(fmaxf(__uint_as_float(word(v, i)), -INFINITY));
}
template <> __device__ __forceinline__ float Vec<float>::at(const uint4& v, int e) { return __uint_as_float(word(v, e)); }
template <> __device__ __forceinline__ float Vec<float>::top(const uint4& v) { return fmaxf(tc::fmax3(at(v, 0), at(v, 1), at(v, 2)), at(v, 3)); }
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <> __device__ __forceinline__ void Vec<__nv_bfloat16>::clean(uint4& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) word(v, i) = max_bf16x2(word(v, i), 0xFF80FF80u);
}
template <> __device__ __forceinline__ float Vec<__nv_bfloat16>::at(const uint4& v, int e) {
    const uint32_t w = word(v, e / 2);
    return __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
}
template <> __device__ __forceinline__ float Vec<__nv_bfloat16>::top(const uint4& v) {
    const uint32_t m = max_bf16x2(max_bf16x2(v.x, v.y), max_bf16x2(v.z, v.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}
__device__ __forceinline__ unsigned long long fmul2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ unsigned long long make_key(float x, int token) {
    return (static_cast<unsigned long long>(order_key(x)) << 32) | static_cast<uint32_t>(~token);
}

struct Shared {
    __align__(16) unsigned long long cand[2][kCap];    // the list and the next one, in turn
    uint4 vec[kFound];                // vectors that hold candidates, and their first elements
    int where[kFound];
    unsigned long long best[SPEC_MAX_BEAMS];
    int found, count, kept;
    unsigned bound[kWarps];
    int part[2][kWarps];
    float fpart[kWarps];
};

// The kq-th largest of a warp's values, as order keys; 0 where it has fewer.
__device__ __forceinline__ unsigned warp_kth(unsigned mine, int kq) {
    unsigned top = 0;
#pragma unroll 1
    for (int i = 0; i < kq; ++i) {
        top = __reduce_max_sync(0xffffffffu, mine);
        const unsigned who = __ballot_sync(0xffffffffu, mine == top);
        if ((threadIdx.x & 31) == __ffs(who) - 1) mine = 0;
    }
    return top;
}

// The K largest of from[0 .. n), sorted, in to[0 ..): every thread finds its candidates' ranks.
__device__ __forceinline__ void cut(const unsigned long long* from, unsigned long long* to, int n, int K) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const unsigned long long key = from[i];
        int rank = 0, j = 0;
#pragma unroll 2
        for (; j + 4 <= n; j += 4) {
            const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(&from[j]), b = *reinterpret_cast<const ulonglong2*>(&from[j + 2]);
            rank += (a.x > key) + (a.y > key) + (b.x > key) + (b.y > key);
        }
        for (; j < n; ++j) rank += from[j] > key;
        if (rank < K) to[rank] = key;
    }
}

__device__ __forceinline__ int block_sum(Shared& sh, int v, int turn) {
    v = __reduce_add_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) sh.part[turn & 1][threadIdx.x >> 5] = v;
    __syncthreads();                  // two buffers in turn: the next call cannot overwrite what is read here
    int sum = 0;
    for (int i = 0; i < kWarps; ++i) sum += sh.part[turn & 1][i];
    return sum;
}

// A row as 16-byte vectors that start at 16-byte boundaries, the first in front of the row where that does not; of one slice.
template <typename T> struct Row {
    static constexpr int E = Vec<T>::E;
    const T* x;
    int V, head, end;                 // elements in front of the row; one more than the slice's last vector
    bool few = false;                 // less than a vector a thread
    __device__ __forceinline__ Row(const Params& p, int row)
        : x(static_cast<const T*>(p.logits) + static_cast<int64_t>(row) * p.stride), V(p.V),
          head(static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T))), end((head + p.V + E - 1) / E) {}
};

// The row's ends, element by element: i is the vector's first one.
template <typename T> __device__ __noinline__ uint4 load_end(const T* x, int V, int i) {
    constexpr int E = Vec<T>::E, P = E / 4;   // elements of a word
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int h = 0; h < P; ++h) {
            const int e = i + k * P + h;
            const float val = e >= 0 && e < V ? to_f32<T>(x[e]) : -INFINITY;
            w[k] |= P == 1 ? __float_as_uint(val) : (__float_as_uint(val) >> 16) << (16 * h);
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The first of a thread's vectors of the chunk that begins at vector c, kThreads apart.  Slices of less than a vector a
// thread go to the warps in turn: if some had none, there would be no bound (15 of 599: 32 us, so 13).
template <typename T> __device__ __forceinline__ int vector_of(const Row<T>& row, int c) {
    const int t = threadIdx.x;
    return c + (row.few ? (t & 31) * kWarps + (t >> 5) : t);
}

// A thread's vectors of the chunk that begins at vector c.
template <typename T> __device__ __forceinline__ void load_chunk(const Row<T>& row, int c, uint4 (&raw)[kVecs]) {
    constexpr int E = Vec<T>::E;
    constexpr uint32_t kNone = E == 4 ? 0xFF800000u : 0xFF80FF80u;   // -inf
    const int v0 = vector_of(row, c);
    if (c > 0 && c + kVecs * kThreads <= row.end && (c + kVecs * kThreads) * E - row.head <= row.V) {   // inside the row
        const T* at = row.x + (v0 * E - row.head);
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(raw[v].x), "=r"(raw[v].y), "=r"(raw[v].z), "=r"(raw[v].w) : "l"(at + v * kThreads * E));
        return;
    }
    bool part[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int at = v0 + v * kThreads, i = at * E - row.head;
        const bool whole = at < row.end && i >= 0 && i + E <= row.V;
        part[v] = at < row.end && !whole;
        raw[v] = make_uint4(kNone, kNone, kNone, kNone);
        if (whole)
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(raw[v].x), "=r"(raw[v].y), "=r"(raw[v].z), "=r"(raw[v].w) : "l"(row.x + i));
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
        if (part[v]) raw[v] = load_end<T>(row.x, row.V, (v0 + v * kThreads) * E - row.head);
}

// More elements pass the threshold than the list holds (rows of equal logits, logits that rise with the token): the K
// largest of cand[0 .. before), at most K, and one chunk by bisection, over the order of the logits, then of the tokens.
template <typename T>
__device__ __noinline__ float cut_chunk(Shared& sh, unsigned long long* cand, const Row<T>& row, int c, int before, int K) {
    constexpr int E = Vec<T>::E;
    uint4 raw[kVecs];                 // the chunk once more
    load_chunk(row, c, raw);
#pragma unroll
    for (int v = 0; v < kVecs; ++v) Vec<T>::clean(raw[v]);
    const int first = vector_of(row, c) * E - row.head;
    const unsigned long long mine = static_cast<int>(threadIdx.x) < before ? cand[threadIdx.x] : 0;   // before is below kThreads
    const unsigned none = order_key(-INFINITY);
    int turn = 0;
    auto count = [&](auto&& test) {
        int n = mine && test(static_cast<unsigned>(mine >> 32), static_cast<int>(~static_cast<uint32_t>(mine))) ? 1 : 0;
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const unsigned k = order_key(Vec<T>::at(raw[v], e));
                n += k > none && test(k, first + v * kThreads * E + e);
            }
        return block_sum(sh, n, turn++);
    };
    unsigned lo = none + 1, hi = 0xffffffffu;             // the largest t with K keys at least t lies in lo .. hi
    while (lo < hi) {
        const unsigned mid = lo + (hi - lo) / 2 + 1;
        if (count([&](unsigned k, int) { return k >= mid; }) >= K) lo = mid; else hi = mid - 1;
    }
    const unsigned t = lo;            // or all there are, if fewer than K
    const int need = K - count([&](unsigned k, int) { return k > t; });
    int from = 0, to = 0x7fffffff;                        // the lowest token by which `need` of the equal ones have come
    while (from < to) {
        const int mid = from + (to - from) / 2;
        if (count([&](unsigned k, int i) { return k == t && i <= mid; }) >= need) to = mid; else from = mid + 1;
    }
    __syncthreads();
    if (threadIdx.x == 0) sh.kept = 0;
    __syncthreads();
    auto keep = [&](unsigned k, int i) { return k > t || (k == t && i <= from); };
    auto add = [&](unsigned long long key) { sh.best[atomicAdd(&sh.kept, 1)] = key; };   // K in all
    if (mine && keep(static_cast<unsigned>(mine >> 32), static_cast<int>(~static_cast<uint32_t>(mine)))) add(mine);
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float x = Vec<T>::at(raw[v], e);
            if (order_key(x) > none && keep(order_key(x), first + v * kThreads * E + e)) add(make_key(x, first + v * kThreads * E + e));
        }
    __syncthreads();
    const int kept = sh.kept;
    if (static_cast<int>(threadIdx.x) < kept) cand[threadIdx.x] = sh.best[threadIdx.x];
    if (threadIdx.x == 0) sh.count = kept;
    __syncthreads();
    return kept < K ? -INFINITY : key_value(t);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kPerSm) k_slices(const Params p) {
    constexpr int E = Vec<T>::E;
    __shared__ Shared sh;
    griddep_wait();                   // in front of the trigger: the join reads the call's inputs without a wait of its own
    clear_status_then_trigger(p.ws);
    const int row_at = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Row<T> row(p, row_at);
    const int v0 = slice * p.per;
    if (slice + 1 < p.slices) row.end = min(row.end, v0 + p.per);
    row.few = row.end - v0 < kThreads;
    if (threadIdx.x == 0) sh.found = sh.count = 0;
    float m = -INFINITY, s = 0.f, least = -INFINITY;   // logits above `least` are candidates
    int before = 0, turn = 0;
    __syncthreads();
    // One chunk, then stretches as long as all before them: each lets some K candidates through, and the warps run free within it.
    constexpr int kStep = kVecs * kThreads;
    int c = v0;
#pragma unroll 1
    for (int64_t len = kStep; c < row.end; len = c - v0) {
        const int c0 = c, c1 = static_cast<int>(min(static_cast<int64_t>(row.end), c0 + len));
#pragma unroll 1
        for (; c < c1; c += kStep) {
            uint4 raw[kVecs];
            load_chunk(row, c, raw);
            if (c == v0 && state_of(p, row_at) != kLive) return;   // looked up while the first loads run
            float tops[kVecs];
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                Vec<T>::clean(raw[v]);
                tops[v] = Vec<T>::top(raw[v]);
            }
            static_assert(kVecs == 4, "the maximum of a thread's vectors");
            const float top = fmaxf(tc::fmax3(tops[0], tops[1], tops[2]), tops[3]);
            // the sum, rescaled to the larger maximum.  x - m is taken before the factor: with both in one
            // FMA the rounding of m log2(e) would shift every term the same way
            const float nm = fmaxf(m, top), ref = nm == -INFINITY ? 0.f : nm;
            const unsigned long long nref = tc::pk2(-ref, -ref), factor = tc::pk2(kLog2e, kLog2e);
            unsigned long long part[2] = {tc::pk2(s * tc::ex2((m - ref) * kLog2e), 0.f), tc::pk2(0.f, 0.f)};
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    float a, b;
                    tc::upk2(fmul2(tc::fadd2(tc::pk2(Vec<T>::at(raw[v], e), Vec<T>::at(raw[v], e + 1)), nref), factor), a, b);
                    part[(e / 2) & 1] = tc::fadd2(part[(e / 2) & 1], tc::pk2(tc::ex2(a), tc::ex2(b)));
                }
            float s0, s1;
            tc::upk2(tc::fadd2(part[0], part[1]), s0, s1);
            s = s0 + s1;
            m = nm;
            if (c == v0) {
                // the first chunk's bound: four warps have kq elements each of at least the fourth largest of the warps' kq-th
                // largest thread maxima; `least` lies one step below it
                const unsigned k = warp_kth(order_key(top), (p.K + 3) / 4);
                if (lane == 0) sh.bound[warp] = k;
                __syncthreads();
                const unsigned fourth = warp_kth(lane < kWarps ? sh.bound[lane] : 0u, 4);
                if (fourth > order_key(-INFINITY)) least = key_value(fourth - (fourth == order_key(0.f) ? 2 : 1));   // (-0 is 0)
            }
            if (!__any_sync(0xffffffffu, top > least)) continue;
            // Only the vectors: their elements are looked at when the stretch is through, one by each thread.  (Elements listed
            // here, a warp's one after the other, kept the other warps waiting: 57 us for 768 rows of 131072 where this takes 52.)
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
                if (tops[v] > least) {
                    const int at = atomicAdd(&sh.found, 1);
                    if (at < kFound) {
                        sh.vec[at] = raw[v];
                        sh.where[at] = (vector_of(row, c) + v * kThreads) * E - row.head;
                    }
                }
        }
        __syncthreads();
        const int found = sh.found;   // the same for all: nobody adds to it before the next barrier
        if (found == 0) {
            __syncthreads();          // all have seen that there are none
            continue;
        }
        unsigned long long* list = sh.cand[turn];
        int n = kCap + 1;
        if (found <= kFound) {
            for (int i = threadIdx.x; i < found * E; i += kThreads) {
                const float x = to_f32<T>(reinterpret_cast<const T*>(sh.vec)[i]);
                if (x > least) {
                    const int at = atomicAdd(&sh.count, 1);
                    if (at < kCap) list[at] = make_key(x, sh.where[i / E] + i % E);
                }
            }
            __syncthreads();
            n = sh.count;
        }
        if (n > kCap) {               // too many: chunk by chunk, each time the K best of it and of those so far
            __syncthreads();
            if (threadIdx.x == 0) {
                sh.found = 0;
                sh.count = before;
            }
            __syncthreads();
            for (int d = c0; d < c1; d += kStep) {
                least = cut_chunk<T>(sh, list, row, d, before, p.K);
                before = sh.count;
                __syncthreads();
            }
        } else {
            if (threadIdx.x == 0) sh.found = 0;        // read by all in front of the last barrier
            cut(list, sh.cand[turn ^ 1], n, p.K);
            turn ^= 1;
            __syncthreads();
            before = min(n, p.K);
            if (threadIdx.x == 0) sh.count = before;   // next used behind a barrier
            least = n >= p.K ? key_value(static_cast<unsigned>(sh.cand[turn][p.K - 1] >> 32)) : -INFINITY;
        }
    }
    const size_t out = static_cast<size_t>(row_at) * p.slices + slice;
    if (static_cast<int>(threadIdx.x) < p.K)
        p.cand[out * p.K + threadIdx.x] = static_cast<int>(threadIdx.x) < before ? sh.cand[turn][threadIdx.x] : 0ull;
    // the slice's maximum and sum
    const float wm = warp_max(m);
    if (lane == 0) sh.fpart[warp] = wm;
    __syncthreads();
    float M = sh.fpart[0];
    for (int i = 1; i < kWarps; ++i) M = fmaxf(M, sh.fpart[i]);
    __syncthreads();
    const float ws = warp_sum(M == -INFINITY ? 0.f : s * exp2f((m - M) * kLog2e));
    if (lane == 0) sh.fpart[warp] = ws;
    __syncthreads();
    if (threadIdx.x == 0) {
        float sum = 0.f;
        for (int i = 0; i < kWarps; ++i) sum += sh.fpart[i];
        p.sums[out] = make_float2(M, sum);
    }
}

// A 64-bit key that orders like the double.
__device__ __forceinline__ unsigned long long order_key64(double v) {
    if (v == 0.0) v = 0.0;
    const unsigned long long b = __double_as_longlong(v);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

struct Entry {
    unsigned long long key;
    uint32_t tie;                     // beam * V + token
    float x;                          // the logit
};

// log(x), x >= 1, to some 2^-25: logf of a mantissa near 1, where its error is that small, and the exponent's part.
__device__ __forceinline__ double log_parts(float x) {
    int e = static_cast<int>(__float_as_uint(x) >> 23) - 127;
    float f = __uint_as_float((__float_as_uint(x) & 0x7fffffu) | 0x3f800000u);
    if (f > 1.4142135f) { f *= 0.5f; ++e; }
    return e * 0.693147180559945309 + static_cast<double>(logf(f));
}

// n^-a to some 2^-40, n >= 1: n = 2^k f, log f by the series of artanh, e^r by its own; thirty 64-bit operations,
// where pow() took 8 us of the join.
__device__ __noinline__ double power(int n, float a) {
    int k = 31 - __clz(n);
    double f = static_cast<double>(n) * __longlong_as_double(static_cast<long long>(1023 - k) << 52);
    if (f > 1.4142135623730951) { f *= 0.5; ++k; }
    const double d = f + 1.0, r0 = static_cast<double>(1.f / static_cast<float>(d));
    const double s = (f - 1.0) * (r0 * fma(-d, r0, 2.0)), z = s * s;
    double l = 1.0 / 15;
#pragma unroll
    for (int i = 13; i >= 1; i -= 2) l = fma(l, z, 1.0 / i);
    constexpr double kLn2 = 0.693147180559945309;
    const double y = -static_cast<double>(a) * fma(static_cast<double>(k), kLn2, 2.0 * s * l);
    const int e = __float2int_rn(static_cast<float>(y) * kLog2e);
    const double r = fma(static_cast<double>(-e), kLn2, y);
    double c = 1.0 / 479001600, v = c;   // 1 / 12!
#pragma unroll
    for (int i = 12; i >= 1; --i) {
        c *= i;                       // 1 / (i - 1)!, at compile time
        v = fma(v, r, c);
    }
    return v * __longlong_as_double(static_cast<long long>(1023 + e) << 52);   // e >= -496: n below 2^31, a at most 16
}

// Ranks are needed in 64 bits only of those near the K-th: this GPU does two 64-bit operations a clock and SM,
// and a first pass in 32 bits leaves some tens of candidates (all of them in 64 bits: 15 us of 21
// for 8 beams of 32000 tokens).  What depends on the call's inputs alone is worked out while the slices run.
struct Join {
    Entry list[kJoinCap];
    double base[SPEC_MAX_BEAMS], inv[SPEC_MAX_BEAMS];   // score(t) = base + x; rank = score * inv
    float basef[SPEC_MAX_BEAMS], invf[SPEC_MAX_BEAMS];
    int state[SPEC_MAX_BEAMS], len[SPEC_MAX_BEAMS];
    float bound[kWarps];
    Entry top[kWarps];
    int count;
};

// (without branches: with them, and the rows' sums one after the other, the join of 64 beams took 63 us for 32)
__device__ __forceinline__ bool above(const Entry& x, const Entry& y) { return (x.key > y.key) | ((x.key == y.key) & (x.tie < y.tie)); }

__device__ __forceinline__ Entry entry_of(const Join& sh, const Params& p, int w, unsigned long long k) {
    const uint32_t token = sh.state[w] == kEnded ? static_cast<uint32_t>(p.eos) : ~static_cast<uint32_t>(k);
    const float x = sh.state[w] == kEnded ? 0.f : key_value(static_cast<unsigned>(k >> 32));
    return Entry{order_key64((sh.base[w] + x) * sh.inv[w]), static_cast<uint32_t>(w) * p.V + token, x};
}

__device__ __forceinline__ void write_pair(const Join& sh, const Params& p, int r, const Entry& e) {
    const int w = e.tie / p.V, token = e.tie - static_cast<uint32_t>(w) * p.V;
    const size_t o = static_cast<size_t>(blockIdx.x) * p.K + r;
    p.score[o] = static_cast<float>(sh.base[w] + e.x);
    p.token[o] = token;
    p.parent[o] = w;
    if (p.ended_out) p.ended_out[o] = sh.state[w] == kEnded || token == p.eos;
    if (p.length_out) p.length_out[o] = sh.len[w];
}

// Many equal ranks: the best one after the other; returns how many there were.
__device__ __noinline__ int join_slowly(Join& sh, const Params& p, const unsigned long long* cand, int per, int n) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Entry last{~0ull, 0, 0.f};
    for (int r = 0; r < p.K; ++r) {
        Entry best{0, 0, 0.f};
        for (int c = threadIdx.x; c < n; c += kThreads) {
            const int w = c / per;
            const unsigned long long k = sh.state[w] == kLive ? cand[c] : 0;
            if (!(sh.state[w] == kLive ? k != 0 : sh.state[w] == kEnded && c == w * per)) continue;
            const Entry e = entry_of(sh, p, w, k);
            if ((r == 0 || above(last, e)) && (!best.key || above(e, best))) best = e;
        }
        for (int o = 16; o > 0; o >>= 1) {
            Entry other;
            other.key = __shfl_xor_sync(0xffffffffu, best.key, o);
            other.tie = __shfl_xor_sync(0xffffffffu, best.tie, o);
            other.x = __shfl_xor_sync(0xffffffffu, best.x, o);
            if (other.key && (!best.key || above(other, best))) best = other;
        }
        if (lane == 0) sh.top[warp] = best;
        __syncthreads();
        best = sh.top[0];
        for (int i = 1; i < kWarps; ++i)
            if (sh.top[i].key && (!best.key || above(sh.top[i], best))) best = sh.top[i];
        __syncthreads();
        if (!best.key) return r;
        if (threadIdx.x == 0) write_pair(sh, p, r, best);
        last = best;
    }
    return p.K;
}

__global__ void __launch_bounds__(kThreads, 2) k_join(const Params p) {
    __shared__ Join sh;
    constexpr int kKeep = 4;          // candidates a thread has in registers; the rest is read twice
    const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.slices, K = p.K;
    const int per = S * K, n = p.W * per;
    const unsigned long long* cand = p.cand + static_cast<size_t>(b) * n;
    if (threadIdx.x == 0) sh.count = 0;
    if (static_cast<int>(threadIdx.x) < p.W) {
        const int w = threadIdx.x, row = b * p.W + w;
        const State st = state_of(p, row);
        const int len = (p.length ? p.length[row] : 0) + (st == kLive ? 1 : 0);
        sh.state[w] = st;
        sh.len[w] = len;
        sh.base[w] = st == kDead ? 0.0 : static_cast<double>(p.scores[row]);
        sh.inv[w] = p.alpha != 0.f ? power(max(len, 1), p.alpha) : 1.0;
    }
    griddep_wait();
    unsigned long long kept[kKeep];   // on their way beside the sums
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int c = threadIdx.x + i * kThreads;
        kept[i] = c < n ? cand[c] : 0;
    }
    __syncthreads();
    // The rows' log-sums: rows warp, warp + 8, .. are this warp's, their slices' sums on their way together; in the end lane i
    // has row i of them.
    constexpr int kRows = SPEC_MAX_BEAMS / kWarps;
    const float2* sums = p.sums + static_cast<size_t>(b) * p.W * S;
    const int own = warp + lane * kWarps;             // this lane's row, if it is one
    float M = -INFINITY, sum = 0.f;
    if (S == 1) {
        if (own < p.W && sh.state[own] == kLive) {
            const float2 ms = sums[own];
            M = ms.x;
            sum = ms.y;
        }
    } else {
        float2 ms[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int w = warp + i * kWarps;
            ms[i] = w < p.W && lane < S && sh.state[w] == kLive ? sums[w * S + lane] : make_float2(-INFINITY, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (warp + i * kWarps >= p.W) break;
            const float top = warp_max(ms[i].x);
            const float all = warp_sum(isfinite(ms[i].x) ? ms[i].y * exp2f((ms[i].x - top) * kLog2e) : 0.f);
            if (lane == i) {
                M = top;
                sum = all;
            }
        }
    }
    float size = 0.f;                 // the largest |base| of the warp's rows
    if (own < p.W) {
        if (sh.state[own] == kLive) {
            if (!isfinite(M)) {       // nothing but -inf, or a logit of +inf
                sh.state[own] = kDead;
                if (M > 0.f) flag_status(p.ws, SPEC_EINVAL);
            } else {
                sh.base[own] -= M + log_parts(sum);
            }
        }
        sh.basef[own] = static_cast<float>(sh.base[own]);
        sh.invf[own] = static_cast<float>(sh.inv[own]);
        if (sh.state[own] != kDead) size = fabsf(sh.basef[own]);
    }
    size = warp_max(size);
    if (lane == 0) sh.bound[warp] = size;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) size = fmaxf(size, sh.bound[i]);
    // c / per by the reciprocal, rounded up: exact, as n * per is below 2^32
    const uint32_t inverse = per > 1 ? static_cast<uint32_t>(0xffffffffu / per + 1) : 0u;
    auto beam_of = [&](int c) { return per > 1 ? static_cast<int>(__umulhi(static_cast<uint32_t>(c), inverse)) : c; };
    auto near_rank = [&](int c, unsigned long long k) {     // in 32 bits; -inf: no pair
        if (c >= n) return -INFINITY;
        const int w = beam_of(c), st = sh.state[w];
        if (!(st == kLive ? k != 0 : st == kEnded && c == w * per)) return -INFINITY;
        // (a finite score less finite logits may pass 32 bits: still a pair)
        return fmaxf((sh.basef[w] + (st == kEnded ? 0.f : key_value(static_cast<unsigned>(k >> 32)))) * sh.invf[w], -3.4028235e38f);
    };
    // a bound as in the slices, lowered by what 32 bits can be off: four roundings of |base| + |x|, |x| <= |base| + |rank| / inv
    float near[kKeep], mine = -INFINITY;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) mine = fmaxf(mine, near[i] = near_rank(threadIdx.x + i * kThreads, kept[i]));
    auto others = [&](auto&& f) {     // the rest, kKeep at a time
        for (int c0 = threadIdx.x + kKeep * kThreads; c0 < n; c0 += kKeep * kThreads) {
            unsigned long long k[kKeep];
#pragma unroll
            for (int i = 0; i < kKeep; ++i) k[i] = c0 + i * kThreads < n ? cand[c0 + i * kThreads] : 0;
#pragma unroll
            for (int i = 0; i < kKeep; ++i) f(c0 + i * kThreads, k[i]);
        }
    };
    others([&](int c, unsigned long long k) { mine = fmaxf(mine, near_rank(c, k)); });
    const unsigned kth = warp_kth(mine == -INFINITY ? 0u : order_key(mine), (K + 3) / 4);
    __syncthreads();                  // sh.bound has been read
    if (lane == 0) sh.bound[warp] = __uint_as_float(kth);
    __syncthreads();
    const unsigned fourth = warp_kth(lane < kWarps ? __float_as_uint(sh.bound[lane]) : 0u, 4);
    float low = fourth ? key_value(fourth) : -INFINITY;
    low -= 2e-6f * (fabsf(low) + size);
    auto offer = [&](int c, unsigned long long k, float r) {
        if (r > -INFINITY && !(r < low)) {
            const int at = atomicAdd(&sh.count, 1);
            if (at < kJoinCap) sh.list[at] = entry_of(sh, p, beam_of(c), k);
        }
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i) offer(threadIdx.x + i * kThreads, kept[i], near[i]);
    others([&](int c, unsigned long long k) { offer(c, k, near_rank(c, k)); });
    __syncthreads();
    const int m = sh.count;
    int written = min(m, K);
    if (m <= kJoinCap) {
        for (int i = threadIdx.x; i < m; i += kThreads) {
            const Entry e = sh.list[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < m; ++j) rank += above(sh.list[j], e);
            if (rank < K) write_pair(sh, p, rank, e);
        }
    } else {
        written = join_slowly(sh, p, cand, per, n);
    }
    for (int r = written + threadIdx.x; r < K; r += kThreads) {
        const size_t o = static_cast<size_t>(b) * K + r;
        p.token[o] = p.parent[o] = -1;
        p.score[o] = -INFINITY;
        if (p.ended_out) p.ended_out[o] = 1;
        if (p.length_out) p.length_out[o] = 0;
    }
}

// Slices of a row: the number that makes the longest SM's work least, in units of a chunk, some 0.4 us: a slice costs its
// chunks and 2.6 more to start and end, a lone one is as long as 6 and 1.4 times its chunks, a candidate in the
// join a two-thousandth.  (768 rows of 131072: 51 us in one slice, 57 in two, 63 in four; 128 rows of 32000: 11.1, 10.6, 11.6;
// 30 rows of 50257: 13.4 in four, 10.4 in twelve.)
int slices_of(int64_t rows, int W, int V, int K) {
    const int64_t sms = device_sm_count();
    const double chunks = V / static_cast<double>(kThreads * kVecs * 8);
    int best = 1;
    double least = 1e300;
    for (int s = 1; s <= kMaxSlices; ++s) {
        const double each = chunks / s, cost = std::max(6.0 + 1.4 * each, static_cast<double>((rows * s + sms - 1) / sms) * (2.6 + each)) + 5e-4 * s * K * W;
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

spec_status check_sizes(int B, int W, int V, int K) {
    if (B < 1 || B > 65535) return fail(SPEC_EINVAL, "B = %d out of 1..65535", B);
    if (W < 1 || W > SPEC_MAX_BEAMS || K < 1 || K > SPEC_MAX_BEAMS)
        return fail(SPEC_EINVAL, "W = %d, K = %d out of 1..%d", W, K, SPEC_MAX_BEAMS);
    if (V < 2 || V > (1 << 24)) return fail(SPEC_EINVAL, "V = %d out of 2..2^24", V);
    return SPEC_OK;
}

// Slices of all rows that a workspace has room for: never fewer for more rows or tokens, so that one that was made for the largest
// call serves every smaller one (slices_of alone takes more of them for fewer rows).  They are at least as many as slices_of wants:
// s slices of rows / SMs = r waves cost r (2.6 s + c) or more for c chunks, one slice the larger of (r + 1) (2.6 + c) and 6 + 1.4 c
// or less, so r s is at most r + 1 + c / 2.6 or 2.4 + 0.54 c.
int64_t slots_of(int64_t rows, int V) {
    const double chunks = V / static_cast<double>(kThreads * kVecs * 8);
    return std::min(rows * kMaxSlices, rows + static_cast<int64_t>(device_sm_count() * (2.4 + 0.54 * chunks)));
}
size_t cand_bytes(int64_t rows, int K, int V) { return round_up(static_cast<size_t>(slots_of(rows, V)) * K * 8, 256); }
size_t bytes_for(int64_t rows, int K, int V) {
    return kWsHeader + cand_bytes(rows, K, V) + round_up(static_cast<size_t>(slots_of(rows, V)) * sizeof(float2), 256);
}

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + bn && y < x + an;
}

}  // namespace beam
}  // namespace spec

using namespace spec;

extern "C" size_t beam_select_workspace_size(int32_t B, int32_t W, int32_t V, int32_t K) {
    clear_error();
    if (beam::check_sizes(B, W, V, K) != SPEC_OK) return 0;
    return beam::bytes_for(static_cast<int64_t>(B) * W, K, V);
}

extern "C" spec_status beam_select(const void* logits, int64_t row_stride, const float* scores, const int32_t* ended,
                                   const int32_t* length, int32_t B, int32_t W, int32_t V, int32_t K, int32_t eos,
                                   float alpha, spec_dtype dt, int32_t* token, int32_t* parent, float* score,
                                   int32_t* ended_out, int32_t* length_out, void* ws, size_t ws_bytes, spec_stream_t s_) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(s_);
    clear_error();
    spec_status st = beam::check_sizes(B, W, V, K);
    if (st != SPEC_OK) return st;
    if (dt != SPEC_BF16 && dt != SPEC_F32) return fail(SPEC_EINVAL, "dtype %d unknown", static_cast<int>(dt));
    if (row_stride < V) return fail(SPEC_EINVAL, "row_stride = %lld is smaller than V = %d", static_cast<long long>(row_stride), V);
    if (eos < -1 || eos >= V) return fail(SPEC_EINVAL, "eos = %d out of -1..V - 1", eos);
    if (ended && eos < 0) return fail(SPEC_EINVAL, "ended beams need the token they go on with: eos = %d", eos);
    if (!(alpha >= 0.f) || !(alpha <= 16.f)) return fail(SPEC_EINVAL, "alpha = %g out of 0..16", alpha);
    if (!logits || !scores || !token || !parent || !score) return fail(SPEC_EINVAL, "logits, scores, token, parent and score must not be NULL");
    if (!aligned16(logits)) return fail(SPEC_EALIGN, "logits must be 16-byte aligned");
    const void* small[] = {scores, ended, length, token, parent, score, ended_out, length_out};
    for (const void* x : small)
        if (!aligned4(x)) return fail(SPEC_EALIGN, "scores, lengths and outputs must be 4-byte aligned");
    const int64_t rows = static_cast<int64_t>(B) * W;
    const int es = dt == SPEC_BF16 ? 2 : 4;
    const size_t in = static_cast<size_t>(rows) * 4, out = static_cast<size_t>(B) * K * 4;
    const void* outs[] = {token, parent, score, ended_out, length_out};
    const void* ins[] = {nullptr, nullptr, scores, ended, length};   // what an output may be written over, where K == W
    for (int i = 0; i < 5; ++i) {
        if (!outs[i]) continue;
        if (beam::overlap(outs[i], out, logits, (static_cast<size_t>(rows - 1) * row_stride + V) * es))
            return fail(SPEC_EINVAL, "an output overlaps the logits");
        for (int j = 0; j < 5; ++j) {
            if (ins[j] && !(i == j && K == W && outs[i] == ins[j]) && beam::overlap(outs[i], out, ins[j], in))
                return fail(SPEC_EINVAL, "an output overlaps an input that is not its own, or of another size");
            if (j > i && outs[j] && beam::overlap(outs[i], out, outs[j], out)) return fail(SPEC_EINVAL, "outputs overlap");
        }
    }
    const int S = static_cast<int>(std::min<int64_t>(beam::slices_of(rows, W, V, K), beam::slots_of(rows, V) / rows));   // at least one
    const size_t need = beam::bytes_for(rows, K, V);
    if (!ws || ws_bytes < need) return fail(SPEC_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
    if (!aligned16(ws)) return fail(SPEC_EALIGN, "workspace must be 16-byte aligned");
    beam::Params p{};
    p.logits = logits; p.stride = row_stride; p.scores = scores; p.ended = ended; p.length = length;
    p.B = B; p.W = W; p.V = V; p.K = K; p.eos = eos; p.slices = S; p.alpha = alpha;
    const int E = 16 / es;
    // whole rounds of the CTA's threads; the last slice takes what is left, one vector more where the row starts inside one
    p.per = static_cast<int>(round_up((V + static_cast<size_t>(S) * E - 1) / (static_cast<size_t>(S) * E), beam::kThreads));
    char* at = static_cast<char*>(ws) + kWsHeader;
    p.cand = reinterpret_cast<unsigned long long*>(at);
    p.sums = reinterpret_cast<float2*>(at + beam::cand_bytes(rows, K, V));
    p.token = token; p.parent = parent; p.score = score; p.ended_out = ended_out; p.length_out = length_out; p.ws = ws;
    auto kern = dt == SPEC_BF16 ? beam::k_slices<__nv_bfloat16> : beam::k_slices<float>;
    SPEC_CUDA_TRY(launch_ex("beam_slices", kern, dim3(static_cast<unsigned>(rows * S)), dim3(beam::kThreads), 0, s, true, p));
    SPEC_CUDA_TRY(launch_ex("beam_join", beam::k_join, dim3(B), dim3(beam::kThreads), 0, s, true, p));
    return SPEC_OK;
}
