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
constexpr int kCap = 1024;            // candidates a slice holds at most
constexpr int kFull = 256;            // from here on they are cut down to K
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
    static __device__ __forceinline__ float top(const uint4 (&v)[kVecs]);
};
template <> __device__ __forceinline__ void Vec<float>::clean(uint4& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) word(v, i) = __float_as_uint(fmaxf(__uint_as_float(word(v, i)), -INFINITY));
}
template <> __device__ __forceinline__ float Vec<float>::at(const uint4& v, int e) { return __uint_as_float(word(v, e)); }
template <> __device__ __forceinline__ float Vec<float>::top(const uint4 (&v)[kVecs]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) m = tc::fmax3(tc::fmax3(m, at(v[i], 0), at(v[i], 1)), at(v[i], 2), at(v[i], 3));
    return m;
}
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
template <> __device__ __forceinline__ float Vec<__nv_bfloat16>::top(const uint4 (&v)[kVecs]) {
    uint32_t m = 0xFF80FF80u;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) m = max_bf16x2(max_bf16x2(m, max_bf16x2(v[i].x, v[i].y)), max_bf16x2(v[i].z, v[i].w));
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
    unsigned long long cand[kCap];
    unsigned long long best[SPEC_MAX_BEAMS];
    int count, kept;
    unsigned bound[kWarps];
    int part[2][kWarps];
    float fpart[kWarps];
};

// The kq-th largest of a warp's values, as order keys; 0 where it has fewer.
__device__ __forceinline__ unsigned warp_kth(unsigned mine, int kq) {
    unsigned top = 0;
    for (int i = 0; i < kq; ++i) {
        top = __reduce_max_sync(0xffffffffu, mine);
        const unsigned who = __ballot_sync(0xffffffffu, mine == top);
        if ((threadIdx.x & 31) == __ffs(who) - 1) mine = 0;
    }
    return top;
}

// Bring cand[0 .. n) down to its K largest, sorted; returns the threshold that later elements must pass.
__device__ float cut(Shared& sh, int n, int K) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const unsigned long long key = sh.cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.cand[j] > key;
        if (rank < K) sh.best[rank] = key;
    }
    __syncthreads();
    const int k = min(n, K);
    if (threadIdx.x < k) sh.cand[threadIdx.x] = sh.best[threadIdx.x];
    if (threadIdx.x == 0) sh.count = k;
    __syncthreads();
    return n >= K ? key_value(static_cast<unsigned>(sh.cand[K - 1] >> 32)) : -INFINITY;
}

__device__ __forceinline__ int block_sum(Shared& sh, int v, int turn) {
    v = __reduce_add_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) sh.part[turn & 1][threadIdx.x >> 5] = v;
    __syncthreads();                  // two buffers in turn: the next call cannot overwrite what is read here
    int sum = 0;
    for (int i = 0; i < kWarps; ++i) sum += sh.part[turn & 1][i];
    return sum;
}

// More elements of one chunk pass the threshold than the list holds (rows of equal logits, logits that rise with
// the token): the K largest of cand[0 .. before) and the chunk by bisection, over the order of the logits, then of the tokens.
template <typename T>
__device__ __noinline__ float cut_chunk(Shared& sh, const uint4 (&raw)[kVecs], int first, int before, int K) {
    constexpr int E = Vec<T>::E;
    const unsigned long long mine = static_cast<int>(threadIdx.x) < before ? sh.cand[threadIdx.x] : 0;   // before < kFull
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
    const unsigned t = lo;
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
    if (static_cast<int>(threadIdx.x) < K) sh.cand[threadIdx.x] = sh.best[threadIdx.x];
    if (threadIdx.x == 0) sh.count = K;
    __syncthreads();
    return key_value(t);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_slices(const Params p) {
    constexpr int E = Vec<T>::E;
    __shared__ Shared sh;
    clear_status_then_trigger(p.ws);
    const int row = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
    if (state_of(p, row) != kLive) return;
    const T* x = static_cast<const T*>(p.logits) + static_cast<int64_t>(row) * p.stride;
    // vectors start at 16-byte boundaries, the first in front of the row where that does not
    const int head = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    const int vecs = (head + p.V + E - 1) / E;
    const int v0 = slice * p.per, v1 = min(vecs, v0 + p.per);
    auto load = [&](int v) {
        const int i = v * E - head;
        uint4 r;
        if (v < v1 && i >= 0 && i + E <= p.V) {
            const uint4* at = reinterpret_cast<const uint4*>(x + i);
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(at));
        } else {                      // the row's ends, element by element
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                constexpr int P = E / 4;   // elements of a word
                w[k] = 0;
#pragma unroll
                for (int h = 0; h < P; ++h) {
                    const int e = i + k * P + h;
                    const float val = v < v1 && e >= 0 && e < p.V ? to_f32<T>(x[e]) : -INFINITY;
                    w[k] |= P == 1 ? __float_as_uint(val) : (__float_as_uint(val) >> 16) << (16 * h);
                }
            }
            r = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return r;
    };
    if (threadIdx.x == 0) sh.count = 0;
    float m = -INFINITY, s = 0.f, thr = -INFINITY;
    int before = 0;
    uint4 next[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) next[v] = load(v0 + v * kThreads + threadIdx.x);
    __syncthreads();
    for (int c = v0; c < v1; c += kVecs * kThreads) {
        uint4 raw[kVecs];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) raw[v] = next[v];
        const int first = (c + static_cast<int>(threadIdx.x)) * E - head;   // of raw[v]: first + v * kThreads * E
        if (c + kVecs * kThreads < v1) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) next[v] = load(c + (kVecs + v) * kThreads + threadIdx.x);
        }
#pragma unroll
        for (int v = 0; v < kVecs; ++v) Vec<T>::clean(raw[v]);
        const float top = Vec<T>::top(raw);
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
        // the first chunk's bound: every warp has kq elements of at least its kq-th largest thread maximum
        const bool begin = c == v0;
        float least = thr;
        if (begin) {
            const unsigned k = warp_kth(order_key(top), (p.K + kWarps - 1) / kWarps);
            if ((threadIdx.x & 31) == 0) sh.bound[threadIdx.x >> 5] = k;
            __syncthreads();
            unsigned low = sh.bound[0];
            for (int i = 1; i < kWarps; ++i) low = min(low, sh.bound[i]);
            least = low ? key_value(low) : -INFINITY;
        }
        auto passes = [&](float v) { return v > least || (begin && v == least && v > -INFINITY); };
        if (passes(top)) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float val = Vec<T>::at(raw[v], e);
                    if (passes(val)) {
                        const int at = atomicAdd(&sh.count, 1);
                        if (at < kCap) sh.cand[at] = make_key(val, first + v * kThreads * E + e);
                    }
                }
        }
        __syncthreads();
        const int n = sh.count;
        __syncthreads();
        if (n > kCap) thr = cut_chunk<T>(sh, raw, first, before, p.K);
        else if (begin || n >= kFull) thr = cut(sh, n, p.K);
        before = sh.count;            // below kFull; a barrier lies between this and the next chunk's first candidate
        __syncthreads();
    }
    cut(sh, before, p.K);
    const size_t out = static_cast<size_t>(row) * p.slices + slice;
    if (static_cast<int>(threadIdx.x) < p.K)
        p.cand[out * p.K + threadIdx.x] = static_cast<int>(threadIdx.x) < sh.count ? sh.cand[threadIdx.x] : 0ull;
    // the slice's maximum and sum
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    uint32_t tie, at;                 // beam * V + token; the candidate's place
};

// log(x), x >= 1, to some 2^-25: logf of a mantissa near 1, where its error is that small, and the exponent's part.
__device__ __forceinline__ double log_parts(float x) {
    int e = static_cast<int>(__float_as_uint(x) >> 23) - 127;
    float f = __uint_as_float((__float_as_uint(x) & 0x7fffffu) | 0x3f800000u);
    if (f > 1.4142135f) { f *= 0.5f; ++e; }
    return e * 0.693147180559945309 + static_cast<double>(logf(f));
}

// Ranks are needed in 64 bits only of those near the K-th: this GPU does two 64-bit operations a clock and SM,
// and a first pass in 32 bits leaves some tens of candidates (all of them in 64 bits: 15 us of 21
// for 8 beams of 32000 tokens).  What depends on the call's inputs alone is worked out while the slices run.
__global__ void __launch_bounds__(kThreads) k_join(const Params p) {
    __shared__ Entry list[kJoinCap];
    __shared__ double s_base[SPEC_MAX_BEAMS], s_inv[SPEC_MAX_BEAMS];   // score(t) = base + x; rank = score * inv
    __shared__ float s_basef[SPEC_MAX_BEAMS], s_invf[SPEC_MAX_BEAMS];
    __shared__ int s_state[SPEC_MAX_BEAMS], s_len[SPEC_MAX_BEAMS];
    __shared__ float s_bound[kWarps];
    __shared__ Entry s_top[kWarps];
    __shared__ int s_count;
    const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.slices, K = p.K;
    if (threadIdx.x == 0) s_count = 0;
    if (threadIdx.x < p.W) {
        const int w = threadIdx.x, row = b * p.W + w;
        const State st = state_of(p, row);
        const int len = (p.length ? p.length[row] : 0) + (st == kLive ? 1 : 0);
        s_state[w] = st;
        s_len[w] = len;
        s_base[w] = st == kDead ? 0.0 : static_cast<double>(p.scores[row]);
        s_inv[w] = p.alpha != 0.f ? pow(static_cast<double>(max(len, 1)), -static_cast<double>(p.alpha)) : 1.0;
    }
    __syncthreads();
    griddep_wait();
    float size = 0.f;                 // the largest |base| of the warp's rows
    for (int w = warp; w < p.W; w += kWarps) {
        if (s_state[w] == kLive) {
            const float2 ms = lane < S ? p.sums[(static_cast<size_t>(b) * p.W + w) * S + lane] : make_float2(-INFINITY, 0.f);
            const float M = warp_max(ms.x);
            const float sum = warp_sum(isfinite(ms.x) ? ms.y * exp2f((ms.x - M) * kLog2e) : 0.f);
            if (lane == 0) {
                if (!isfinite(M)) {   // nothing but -inf, or a logit of +inf
                    s_state[w] = kDead;
                    if (M > 0.f) flag_status(p.ws, SPEC_EINVAL);
                } else {
                    s_base[w] -= M + log_parts(sum);
                }
            }
        }
        if (lane == 0) {
            s_basef[w] = static_cast<float>(s_base[w]);
            s_invf[w] = static_cast<float>(s_inv[w]);
        }
        __syncwarp();
        if (s_state[w] != kDead) size = fmaxf(size, fabsf(s_basef[w]));
    }
    if (lane == 0) s_bound[warp] = size;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) size = fmaxf(size, s_bound[i]);
    const int per = S * K, n = p.W * per;
    const unsigned long long* cand = p.cand + static_cast<size_t>(b) * n;
    auto some_at = [&](int c, int w, float& x, uint32_t& token) {
        if (s_state[w] == kEnded) {
            token = p.eos;
            x = 0.f;
            return c == w * per;
        }
        if (s_state[w] != kLive) return false;
        const unsigned long long k = cand[c];
        token = ~static_cast<uint32_t>(k);
        x = key_value(static_cast<unsigned>(k >> 32));
        return k != 0;
    };
    auto near_rank = [&](int c) {     // -inf: no pair
        const int w = c / per;
        float x;
        uint32_t token;
        return some_at(c, w, x, token) ? (s_basef[w] + x) * s_invf[w] : -INFINITY;
    };
    auto entry_at = [&](int c) {
        const int w = c / per;
        float x;
        uint32_t token;
        if (!some_at(c, w, x, token)) return Entry{0, 0, 0};
        return Entry{order_key64((s_base[w] + x) * s_inv[w]), static_cast<uint32_t>(w) * p.V + token, static_cast<uint32_t>(c)};
    };
    auto above = [](const Entry& x, const Entry& y) { return x.key > y.key || (x.key == y.key && x.tie < y.tie); };
    auto write = [&](int r, const Entry& e) {
        const int w = e.tie / p.V;
        float x;
        uint32_t token;
        some_at(e.at, w, x, token);
        const size_t o = static_cast<size_t>(b) * K + r;
        p.score[o] = static_cast<float>(s_base[w] + x);
        p.token[o] = token;
        p.parent[o] = w;
        if (p.ended_out) p.ended_out[o] = s_state[w] == kEnded || static_cast<int>(token) == p.eos;
        if (p.length_out) p.length_out[o] = s_len[w];
    };
    // a bound as in the slices, lowered by what 32 bits can be off: four roundings of |base| + |x|, |x| <= |base| + |rank| / inv
    float mine = -INFINITY;
    for (int c = threadIdx.x; c < n; c += kThreads) mine = fmaxf(mine, near_rank(c));
    const unsigned kth = warp_kth(mine == -INFINITY ? 0u : order_key(mine), (K + kWarps - 1) / kWarps);
    __syncthreads();                  // s_bound has been read
    if (lane == 0) s_bound[warp] = kth ? key_value(kth) : -INFINITY;
    __syncthreads();
    float low = s_bound[0];
    for (int i = 1; i < kWarps; ++i) low = fminf(low, s_bound[i]);
    low -= 2e-6f * (fabsf(low) + size);
    for (int c = threadIdx.x; c < n; c += kThreads) {
        const float r = near_rank(c);
        if (r > -INFINITY && !(r < low)) {
            const int at = atomicAdd(&s_count, 1);
            if (at < kJoinCap) list[at] = entry_at(c);
        }
    }
    __syncthreads();
    const int m = s_count;
    int written = min(m, K);
    if (m <= kJoinCap) {
        for (int i = threadIdx.x; i < m; i += kThreads) {
            const Entry e = list[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < m; ++j) rank += above(list[j], e);
            if (rank < K) write(rank, e);
        }
    } else {                          // many equal ranks: one after the other
        Entry last{~0ull, 0, 0};
        bool any = true;
        for (written = 0; written < K && any; ++written) {
            Entry best{0, 0, 0};
            for (int c = threadIdx.x; c < n; c += kThreads) {
                const Entry e = entry_at(c);
                if (e.key && (written == 0 || above(last, e)) && (!best.key || above(e, best))) best = e;
            }
            for (int o = 16; o > 0; o >>= 1) {
                Entry other;
                other.key = __shfl_xor_sync(0xffffffffu, best.key, o);
                other.tie = __shfl_xor_sync(0xffffffffu, best.tie, o);
                other.at = __shfl_xor_sync(0xffffffffu, best.at, o);
                if (other.key && (!best.key || above(other, best))) best = other;
            }
            if (lane == 0) s_top[warp] = best;
            __syncthreads();
            best = s_top[0];
            for (int i = 1; i < kWarps; ++i)
                if (s_top[i].key && (!best.key || above(s_top[i], best))) best = s_top[i];
            any = best.key != 0;
            if (!any) break;
            if (threadIdx.x == 0) write(written, best);
            last = best;
            __syncthreads();
        }
    }
    for (int r = written + threadIdx.x; r < K; r += kThreads) {
        const size_t o = static_cast<size_t>(b) * K + r;
        p.token[o] = p.parent[o] = -1;
        p.score[o] = -INFINITY;
        if (p.ended_out) p.ended_out[o] = 1;
        if (p.length_out) p.length_out[o] = 0;
    }
}

// Slices of a row.  Four CTAs fit an SM.  Where there is less than that of work they are as short as 2048
// logits; else there are four rounds of them, so that the last one's gaps cost little, but none
// shorter than 8192, whose start and end cost as much as the rest.
int slices_of(int64_t rows, int V) {
    const int64_t slots = 4 * device_sm_count();
    const int64_t finest = (static_cast<int64_t>(V) + 2047) / 2048, fine = (static_cast<int64_t>(V) + 8191) / 8192;
    const int64_t once = (slots + rows - 1) / rows, rounds = (4 * slots + rows - 1) / rows;
    const int64_t s = std::max(std::min(once, finest), std::min(rounds, fine));
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(s, kMaxSlices)));
}

spec_status check_sizes(int B, int W, int V, int K) {
    if (B < 1 || B > 65535) return fail(SPEC_EINVAL, "B = %d out of 1..65535", B);
    if (W < 1 || W > SPEC_MAX_BEAMS || K < 1 || K > SPEC_MAX_BEAMS)
        return fail(SPEC_EINVAL, "W = %d, K = %d out of 1..%d", W, K, SPEC_MAX_BEAMS);
    if (V < 2 || V > (1 << 24)) return fail(SPEC_EINVAL, "V = %d out of 2..2^24", V);
    return SPEC_OK;
}

// Sizes that any number of slices fits, so that they do not depend on the device.
size_t cand_bytes(int64_t rows, int K, int S) { return round_up(static_cast<size_t>(rows) * S * K * 8, 256); }
size_t bytes_for(int B, int W, int K, int S) {
    const int64_t rows = static_cast<int64_t>(B) * W;
    return kWsHeader + cand_bytes(rows, K, S) + round_up(static_cast<size_t>(rows) * S * sizeof(float2), 256);
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
    return beam::bytes_for(B, W, K, beam::slices_of(static_cast<int64_t>(B) * W, V));
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
    const int S = beam::slices_of(rows, V);
    const size_t need = beam::bytes_for(B, W, K, S);
    if (!ws || ws_bytes < need) return fail(SPEC_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
    if (!aligned16(ws)) return fail(SPEC_EALIGN, "workspace must be 16-byte aligned");
    beam::Params p{};
    p.logits = logits; p.stride = row_stride; p.scores = scores; p.ended = ended; p.length = length;
    p.B = B; p.W = W; p.V = V; p.K = K; p.eos = eos; p.slices = S; p.alpha = alpha;
    const int E = 16 / es;
    p.per = (V / E + 2 + S - 1) / S;   // a row's vectors and one more at each end where it starts inside one
    char* at = static_cast<char*>(ws) + kWsHeader;
    p.cand = reinterpret_cast<unsigned long long*>(at);
    p.sums = reinterpret_cast<float2*>(at + beam::cand_bytes(rows, K, S));
    p.token = token; p.parent = parent; p.score = score; p.ended_out = ended_out; p.length_out = length_out; p.ws = ws;
    auto kern = dt == SPEC_BF16 ? beam::k_slices<__nv_bfloat16> : beam::k_slices<float>;
    SPEC_CUDA_TRY(launch("beam_slices", kern, dim3(static_cast<unsigned>(rows * S)), dim3(beam::kThreads), 0, s, p));
    SPEC_CUDA_TRY(launch_ex("beam_join", beam::k_join, dim3(B), dim3(beam::kThreads), 0, s, true, p));
    return SPEC_OK;
}
