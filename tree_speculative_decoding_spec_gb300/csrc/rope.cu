// Rotary positions on the way from the projections to the cache and the tree.
//
//   kv_append, kv_append_paged   new tokens of a ragged batch: q rotated, k rotated
//                                into the cache, v copied into it
//   tree_rope                    the candidate tree's nodes: q, k_tree, v_tree in the
//                                layout tree_attention reads
//
// A token at position p turns the pair (x, y) number j of each q and k head by
// the angle p * freq[j]: x' = x cos - y sin, y' = x sin + y cos.  The product
// p * freq[j] is taken in 64 bits in units of full turns, its whole turns are
// dropped there, and only the rest (at most half a turn) goes to 32 bits: at
// position 2^22 a 32-bit product would already be off by a quarter of a radian.
// cos and sin are computed once per token, not per head.  The rotation is in
// 32 bits, rounded once to the inputs' type.
//
// Bound by memory: every value is read and written once, in 16-byte accesses.
// A CTA takes one token, or a part of a token's heads when there are few
// tokens.  Its data does not depend on the sequence the token belongs to, so
// every thread issues the loads of its first unit before the CTA looks that up.
// Eight CTAs an SM (32 registers a thread) keep the loads in flight: three units of
// a thread loaded together took 64 registers and 58 us where one at a time took 50.
// What is left beside the loads is issue and shared memory: (cos, sin) laid out so
// that neighbouring units read neighbouring 16 bytes, and heads found by a product
// with a reciprocal, brought 50 to 44 us.  Prompts of 6569 tokens, 64 and 8 heads of
// 128 (269 MB): 44 us, 6.1 TB/s of a copy's 6.8; 32 trees of 64 nodes (84 MB): 16.8 us;
// one token of each of 64 sequences 3.8 us and one tree of 64 nodes 3.3 us, launch
// and look-ups.
#include <algorithm>

#include "common.cuh"

namespace spec {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxD = 1024;

enum Style { kHalf = 0, kPairs = 1, kScalar = 2 };

struct Params {
    const void *q, *k, *v;            // rows of one token: heads x D, dense; token strides below
    int64_t qs, ks, vs;               // elements between tokens
    void *q_out, *k_out, *v_out;      // q_out may be NULL (appends only)
    const double* freq;               // [rot / 2] or NULL
    const int32_t* pos_base;          // [1] or NULL
    const int32_t* prefix_len;        // [B]
    int B, Hq, Hkv, D, rot, interleaved;
    // appends
    const int32_t* seq_start;         // [B + 1]; NULL: tree
    const int32_t* table;             // [B, max_blocks]; NULL: contiguous
    int N, max_blocks, rows, num_blocks;   // rows per (block, head)
    int64_t cap;                      // positions of one sequence
    void* ws;
    // tree
    const int32_t* depth;
    int T;
    uint32_t inv_per, inv_nc;         // 2^32 over the units of a q or k head, of a v head, rounded up (0: one unit)
};

// u / d by its rounded-up reciprocal: exact while u * d < 2^32 (here u < 2^18, d <= 2^8).
__device__ __forceinline__ int quotient(int u, uint32_t inv) { return inv ? static_cast<int>(__umulhi(static_cast<uint32_t>(u), inv)) : u; }

// Where one token goes.
struct Token {
    double pos;
    int64_t q_off, k_off;             // element offset of head 0
    int ok;
};

// Largest b in [0, B) with start[b] <= n, or -1: 32 probes a step, the whole warp.
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ start, int B, int n) {
    const int lane = threadIdx.x & 31;
    int lo = -1, hi = B;              // start[lo] <= n (lo = -1: nothing known), n < start[hi] or hi = B
    while (hi - lo > 1) {
        const int step = (hi - lo - 1 + 31) / 32;
        const int at = lo + 1 + lane * step;
        const bool le = at < hi && start[at] <= n;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        // the leading lanes that say yes: in order for offsets that do not decrease
        const int c = __ffs(~m) ? __ffs(~m) - 1 : 32;
        const int nlo = c > 0 ? lo + 1 + (c - 1) * step : lo;
        const int nhi = c < 32 ? min(hi, lo + 1 + c * step) : hi;
        lo = nlo;
        hi = nhi;
    }
    return lo;
}

// The sequence of new token n and its place in the cache; the whole warp, same answer in every lane.
__device__ __forceinline__ Token place_append(const Params& p, int n) {
    Token t{0.0, 0, 0, 0};
    const int b = find_sequence(p.seq_start, p.B, n);
    if (b < 0) return t;
    const int s0 = p.seq_start[b], s1 = p.seq_start[b + 1];
    if (n < s0 || n >= s1 || s0 < 0 || s1 > p.N) return t;   // a sequence with rows outside 0 .. N gets none
    const int L = p.prefix_len[b];
    if (L < 0 || static_cast<int64_t>(L) + s1 - s0 > p.cap) return t;
    const int at = L + (n - s0);
    int blk = b, row = at;
    if (p.table) {
        blk = p.table[static_cast<size_t>(b) * p.max_blocks + at / p.rows];
        row = at % p.rows;
        if (blk < 0 || blk >= p.num_blocks) return t;
    }
    t.pos = static_cast<double>(at) + (p.pos_base ? static_cast<double>(*p.pos_base) : 0.0);
    t.q_off = static_cast<int64_t>(n) * p.Hq * p.D;
    t.k_off = (static_cast<int64_t>(blk) * p.Hkv * p.rows + row) * p.D;
    t.ok = 1;
    return t;
}

__device__ __forceinline__ Token place_node(const Params& p, int n) {
    const int b = n / p.T, i = n % p.T;
    Token t;
    t.pos = static_cast<double>(p.prefix_len[b]) + p.depth[i] + (p.pos_base ? static_cast<double>(*p.pos_base) : 0.0);
    t.q_off = (static_cast<int64_t>(b) * p.Hq * p.T + i) * p.D;
    t.k_off = (static_cast<int64_t>(b) * p.Hkv * p.T + i) * p.D;
    t.ok = 1;
    return t;
}

// The append's status: one CTA looks at every sequence and every block its tokens go to, and
// stores the word; no other CTA writes it, so nothing has to clear it first.
__device__ void check_append(const Params& p) {
    __shared__ int bad;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int mine = 0;
    if (threadIdx.x == 0 && (p.seq_start[0] < 0 || p.seq_start[p.B] > p.N)) mine = 1;
    constexpr int kWarps = kThreads / 32;
    for (int b0 = warp; b0 < p.B; b0 += kThreads) {        // a lane per sequence, every warp some
        const int b = b0 + lane * kWarps;
        int64_t first = 0, last = -1;                      // the blocks its tokens go to
        if (b < p.B) {
            const int s0 = p.seq_start[b], s1 = p.seq_start[b + 1], L = p.prefix_len[b];
            const int64_t end = static_cast<int64_t>(L) + s1 - s0;
            if (s1 < s0 || (s1 > s0 && (L < 0 || end > p.cap))) {
                mine = 1;
            } else if (p.table && s1 > s0) {
                first = L / p.rows;
                last = (end - 1) / p.rows;
            }
        }
        auto outside = [&](int seq, int64_t j) {
            const int blk = p.table[static_cast<size_t>(seq) * p.max_blocks + j];
            return blk < 0 || blk >= p.num_blocks;
        };
        // one or two blocks by the lane itself, more by the warp
        if (last >= first && last - first < 2 && (outside(b, first) || outside(b, last))) mine = 1;
        for (unsigned many = __ballot_sync(0xffffffffu, last - first >= 2); many; many &= many - 1) {
            const int l = __ffs(many) - 1;
            const int64_t from = __shfl_sync(0xffffffffu, first, l), to = __shfl_sync(0xffffffffu, last, l);
            for (int64_t j = from + lane; j <= to; j += 32)
                if (outside(b0 + l * kWarps, j)) mine = 1;
        }
    }
    if (mine) bad = 1;
    __syncthreads();
    if (threadIdx.x == 0) *static_cast<int4*>(p.ws) = make_int4(bad ? SPEC_EINVAL : SPEC_OK, 0, 0, 0);
}

template <typename T> struct Chunk {
    static constexpr int E = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack(const uint4& c, float (&x)[8]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& c, float (&x)[4]) {
    x[0] = __uint_as_float(c.x); x[1] = __uint_as_float(c.y);
    x[2] = __uint_as_float(c.z); x[3] = __uint_as_float(c.w);
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

template <typename T, int STYLE>
__global__ void __launch_bounds__(kThreads, 8) k_rope(const Params p) {
    constexpr int E = Chunk<T>::E;
    // (cos, sin) of pair j; half style: two pairs of a unit as 16 bytes, neighbouring units side by side
    __shared__ __align__(16) float2 s_cs[kMaxD / 2];
    __shared__ Token s_tok;
    int n = blockIdx.x;
    if (p.seq_start && --n < 0) {     // the append's extra CTA: the first, or the call would end with it
        if (blockIdx.y == 0) check_append(p);
        return;
    }
    const int half = p.rot / 2;
    const int nc = p.D / E;                                        // chunks of a head
    const int np = STYLE == kHalf ? half / E : 0;                  // units that hold both chunks of their pairs
    const int per = STYLE == kHalf ? nc - np : nc;                 // units of a q or k head
    const int uq = p.q ? p.Hq * per : 0, uk = p.Hkv * per, total = uq + uk + p.Hkv * nc;
    const int stride = gridDim.y * kThreads;

    struct Unit {
        const T* src;       // the head's first element
        int head, c, kind;  // kind 0: q, 1: k, 2: v
    };
    auto unit = [&](int u) {
        Unit w;
        if (u < uq) {
            w.kind = 0;
            w.head = quotient(u, p.inv_per);
            w.c = u - w.head * per;
            w.src = static_cast<const T*>(p.q) + n * p.qs + static_cast<int64_t>(w.head) * p.D;
        } else if (u < uq + uk) {
            w.kind = 1;
            w.head = quotient(u - uq, p.inv_per);
            w.c = u - uq - w.head * per;
            w.src = static_cast<const T*>(p.k) + n * p.ks + static_cast<int64_t>(w.head) * p.D;
        } else {
            w.kind = 2;
            w.head = quotient(u - uq - uk, p.inv_nc);
            w.c = u - uq - uk - w.head * nc;
            w.src = static_cast<const T*>(p.v) + n * p.vs + static_cast<int64_t>(w.head) * p.D;
        }
        return w;
    };
    // the chunk index of a unit, and its second chunk's (half style, rotated units only)
    auto first_chunk = [&](const Unit& w) { return STYLE == kHalf && w.kind != 2 && w.c >= np ? w.c + np : w.c; };
    auto paired = [&](const Unit& w) { return STYLE == kHalf && w.kind != 2 && w.c < np; };

    int u = blockIdx.y * kThreads + threadIdx.x;
    Unit w{};
    uint4 a{}, b{};
    if (u < total) {
        w = unit(u);
        a = *reinterpret_cast<const uint4*>(w.src + first_chunk(w) * E);
        if (paired(w)) b = *reinterpret_cast<const uint4*>(w.src + (w.c + np) * E);
    }
    if (threadIdx.x < 32) {
        const Token t = p.seq_start ? place_append(p, n) : place_node(p, n);
        if (threadIdx.x == 0) s_tok = t;
    }
    __syncthreads();
    if (!s_tok.ok) return;
    for (int j = threadIdx.x; j < half; j += kThreads) {
        const double turns = s_tok.pos * (p.freq[j] * 0.15915494309189533577);   // 1 / (2 pi)
        float sn, cs;
        sincospif(2.f * static_cast<float>(turns - rint(turns)), &sn, &cs);
        s_cs[STYLE == kHalf ? 2 * (((j % E) >> 1) * np + j / E) + (j & 1) : j] = make_float2(cs, sn);
    }
    __syncthreads();
    const int64_t hq = p.seq_start ? p.D : static_cast<int64_t>(p.T) * p.D;
    const int64_t hk = p.seq_start ? static_cast<int64_t>(p.rows) * p.D : static_cast<int64_t>(p.T) * p.D;
    while (u < total) {
        T* dst = w.kind == 0 ? static_cast<T*>(p.q_out) + s_tok.q_off + w.head * hq
                             : static_cast<T*>(w.kind == 1 ? p.k_out : p.v_out) + s_tok.k_off + w.head * hk;
        const int c0 = first_chunk(w);
        if (paired(w)) {
            float x[E], y[E], xo[E], yo[E];
            unpack(a, x);
            unpack(b, y);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float4 cs = reinterpret_cast<const float4*>(s_cs)[(e >> 1) * np + w.c];
                xo[e] = x[e] * cs.x - y[e] * cs.y;
                yo[e] = x[e] * cs.y + y[e] * cs.x;
                xo[e + 1] = x[e + 1] * cs.z - y[e + 1] * cs.w;
                yo[e + 1] = x[e + 1] * cs.w + y[e + 1] * cs.z;
            }
            a = pack(xo);
            *reinterpret_cast<uint4*>(dst + (w.c + np) * E) = pack(yo);
        } else if (STYLE == kPairs && w.kind != 2 && c0 * E < p.rot) {
            float x[E];
            unpack(a, x);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 cs = s_cs[(c0 * E + e) / 2];
                const float y0 = x[e] * cs.x - x[e + 1] * cs.y;
                x[e + 1] = x[e] * cs.y + x[e + 1] * cs.x;
                x[e] = y0;
            }
            a = pack(x);
        } else if (STYLE == kScalar && w.kind != 2 && c0 * E < p.rot) {
            // a rotated width whose pairs do not fill whole chunks: element by element
            float x[E];
            unpack(a, x);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int d = c0 * E + e;
                if (d < p.rot) {
                    const bool lower = p.interleaved ? (d & 1) == 0 : d < half;
                    const int j = p.interleaved ? d >> 1 : (lower ? d : d - half);
                    const int other = p.interleaved ? d ^ 1 : (lower ? d + half : d - half);
                    const float2 cs = s_cs[j];
                    const float z = to_f32<T>(w.src[other]);
                    x[e] = lower ? x[e] * cs.x - z * cs.y : z * cs.y + x[e] * cs.x;
                }
            }
            a = pack(x);
        }
        *reinterpret_cast<uint4*>(dst + c0 * E) = a;
        u += stride;
        if (u < total) {
            w = unit(u);
            a = *reinterpret_cast<const uint4*>(w.src + first_chunk(w) * E);
            if (paired(w)) b = *reinterpret_cast<const uint4*>(w.src + (w.c + np) * E);
        }
    }
}

// ---------------------------------------------------------------- host

// Checks shared by the three calls: heads, types, strides, rotation, source pointers.
spec_status check_rows(const void* q, const void* k, const void* v, int64_t qs, int64_t ks, int64_t vs, int Hq, int Hkv,
                       int D, const double* freq, int rot, spec_dtype dt, bool need_q, int tokens) {
    if (dt != SPEC_BF16 && dt != SPEC_F32) return fail(SPEC_EINVAL, "dtype %d unknown", static_cast<int>(dt));
    const int es = dt == SPEC_BF16 ? 2 : 4, E = 16 / es;
    if (Hkv < 1 || Hkv > 1024 || ((q || need_q) && (Hq < 1 || Hq > 1024)))
        return fail(SPEC_EINVAL, "Hq = %d, Hkv = %d out of 1..1024", Hq, Hkv);
    if (D < 1 || D > kMaxD || D % E) return fail(SPEC_EINVAL, "D = %d: 1..%d and a multiple of 16 bytes", D, kMaxD);
    if (tokens > 0 && (!k || !v || (need_q && !q))) return fail(SPEC_EINVAL, "the projections must not be NULL");
    if (rot < 0 || rot > D || rot % 2) return fail(SPEC_EINVAL, "rot = %d: an even number in 0..D", rot);
    if (rot && !freq) return fail(SPEC_EINVAL, "freq is NULL with rot = %d", rot);
    if (freq && (reinterpret_cast<uintptr_t>(freq) & 7u)) return fail(SPEC_EALIGN, "freq must be 8-byte aligned");
    if (ks < static_cast<int64_t>(Hkv) * D || vs < static_cast<int64_t>(Hkv) * D || (q && qs < static_cast<int64_t>(Hq) * D))
        return fail(SPEC_EINVAL, "a token stride is smaller than the token's heads");
    if (ks % E || vs % E || (q && qs % E)) return fail(SPEC_EALIGN, "token strides must be multiples of 16 bytes");
    if (!aligned16(k) || !aligned16(v) || !aligned16(q)) return fail(SPEC_EALIGN, "the projections must be 16-byte aligned");
    return SPEC_OK;
}

bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + static_cast<uintptr_t>(bn) && y < x + static_cast<uintptr_t>(an);
}

template <typename T>
spec_status run(const char* name, Params& p, int tokens, cudaStream_t s) {
    constexpr int E = Chunk<T>::E;
    const int style = p.interleaved ? (p.rot % E ? kScalar : kPairs) : (p.rot % (2 * E) ? kScalar : kHalf);
    const int nc = p.D / E;
    const int per = style == kHalf ? nc - p.rot / 2 / E : nc;
    auto inverse = [](int d) { return d == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + d - 1) / d); };
    p.inv_per = inverse(per);
    p.inv_nc = inverse(nc);
    const int64_t total = static_cast<int64_t>((p.q ? p.Hq : 0) + p.Hkv) * per + static_cast<int64_t>(p.Hkv) * nc;
    // one CTA per token, or as many as give every SM four CTAs while each thread still has a unit
    const int most = static_cast<int>((total + kThreads - 1) / kThreads);
    const int want = (4 * device_sm_count() + tokens - 1) / std::max(tokens, 1);
    const dim3 grid(tokens + (p.seq_start ? 1 : 0), std::max(1, std::min(most, want)));
    auto kern = style == kHalf ? k_rope<T, kHalf> : style == kPairs ? k_rope<T, kPairs> : k_rope<T, kScalar>;
    SPEC_CUDA_TRY(launch(name, kern, grid, dim3(kThreads), 0, s, p));
    return SPEC_OK;
}

spec_status append(Params& p, spec_dtype dt, const void* ws, size_t ws_bytes, cudaStream_t s) {
    spec_status st = check_rows(p.q, p.k, p.v, p.qs, p.ks, p.vs, p.Hq, p.Hkv, p.D, p.freq, p.rot, dt, false, p.N);
    if (st != SPEC_OK) return st;
    const int es = dt == SPEC_BF16 ? 2 : 4;
    if (p.N < 0 || p.N > (1 << 28)) return fail(SPEC_EINVAL, "N = %d out of 0..2^28", p.N);
    if (p.B < 1 || p.B > 65535) return fail(SPEC_EINVAL, "B = %d out of 1..65535", p.B);
    if (!p.seq_start || !p.prefix_len || !p.k_out || !p.v_out)
        return fail(SPEC_EINVAL, "seq_start, prefix_len and the cache must not be NULL");
    if ((p.q != nullptr) != (p.q_out != nullptr)) return fail(SPEC_EINVAL, "q and q_out go together");
    if (!aligned16(p.k_out) || !aligned16(p.v_out) || !aligned16(p.q_out))
        return fail(SPEC_EALIGN, "the cache and q_out must be 16-byte aligned");
    if (!aligned4(p.seq_start) || !aligned4(p.prefix_len) || !aligned4(p.pos_base) || !aligned4(p.table))
        return fail(SPEC_EALIGN, "seq_start, prefix_len, pos_base and the block table must be 4-byte aligned");
    if (!ws || ws_bytes < kWsHeader) return fail(SPEC_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, kWsHeader);
    if (!aligned16(ws)) return fail(SPEC_EALIGN, "workspace must be 16-byte aligned");
    if (p.q && p.N > 0) {
        auto span = [&](int64_t stride, int heads) { return ((p.N - 1) * stride + static_cast<int64_t>(heads) * p.D) * es; };
        const int64_t out = static_cast<int64_t>(p.N) * p.Hq * p.D * es;
        if (overlap(p.q_out, out, p.q, span(p.qs, p.Hq)) || overlap(p.q_out, out, p.k, span(p.ks, p.Hkv)) ||
            overlap(p.q_out, out, p.v, span(p.vs, p.Hkv)))
            return fail(SPEC_EINVAL, "q_out overlaps the projections");
    }
    return dt == SPEC_BF16 ? run<__nv_bfloat16>("kv_append", p, p.N, s) : run<float>("kv_append", p, p.N, s);
}

}  // namespace rope
}  // namespace spec

using namespace spec;

extern "C" size_t kv_append_workspace_size(void) { return kWsHeader; }

extern "C" spec_status kv_append(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                 int64_t v_stride, int32_t N, const int32_t* seq_start, int32_t B, int32_t Hq, int32_t Hkv,
                                 int32_t D, const int32_t* prefix_len, const int32_t* pos_base, const double* freq,
                                 int32_t rot, int32_t interleaved, void* k_cache, void* v_cache, int32_t Lmax,
                                 spec_dtype dt, void* q_out, void* ws, size_t ws_bytes, spec_stream_t s) {
    clear_error();
    if (Lmax < 1 || Lmax > (1 << 22)) return fail(SPEC_EINVAL, "Lmax = %d out of 1..2^22", Lmax);
    rope::Params p{};
    p.q = q; p.k = k; p.v = v;
    p.qs = q_stride; p.ks = k_stride; p.vs = v_stride;
    p.q_out = q_out; p.k_out = k_cache; p.v_out = v_cache;
    p.freq = freq; p.pos_base = pos_base; p.prefix_len = prefix_len;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.D = D; p.rot = rot; p.interleaved = interleaved != 0;
    p.seq_start = seq_start; p.N = N; p.rows = Lmax; p.cap = Lmax; p.ws = ws;
    return rope::append(p, dt, ws, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}

extern "C" spec_status kv_append_paged(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                       int64_t v_stride, int32_t N, const int32_t* seq_start, int32_t B, int32_t Hq,
                                       int32_t Hkv, int32_t D, const int32_t* prefix_len, const int32_t* pos_base,
                                       const double* freq, int32_t rot, int32_t interleaved, void* k_pool, void* v_pool,
                                       int32_t num_blocks, const int32_t* block_table, int32_t max_blocks,
                                       int32_t block_size, spec_dtype dt, void* q_out, void* ws, size_t ws_bytes,
                                       spec_stream_t s) {
    clear_error();
    if (num_blocks < 1 || max_blocks < 1 || block_size < 1)
        return fail(SPEC_EINVAL, "num_blocks = %d, max_blocks = %d, block_size = %d must be positive", num_blocks,
                    max_blocks, block_size);
    if (static_cast<int64_t>(max_blocks) * block_size > (1 << 22))
        return fail(SPEC_EINVAL, "max_blocks * block_size = %lld positions exceed 2^22",
                    static_cast<long long>(max_blocks) * block_size);
    if (!block_table) return fail(SPEC_EINVAL, "block_table must not be NULL");
    rope::Params p{};
    p.q = q; p.k = k; p.v = v;
    p.qs = q_stride; p.ks = k_stride; p.vs = v_stride;
    p.q_out = q_out; p.k_out = k_pool; p.v_out = v_pool;
    p.freq = freq; p.pos_base = pos_base; p.prefix_len = prefix_len;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.D = D; p.rot = rot; p.interleaved = interleaved != 0;
    p.seq_start = seq_start; p.N = N; p.rows = block_size; p.ws = ws;
    p.table = block_table; p.max_blocks = max_blocks; p.num_blocks = num_blocks;
    p.cap = static_cast<int64_t>(max_blocks) * block_size;
    return rope::append(p, dt, ws, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}

extern "C" spec_status tree_rope(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                 int64_t v_stride, const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                 const int32_t* prefix_len, const int32_t* pos_base, const double* freq, int32_t rot,
                                 int32_t interleaved, spec_dtype dt, void* q_out, void* k_tree, void* v_tree,
                                 spec_stream_t s_) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(s_);
    clear_error();
    spec_status st = check_tree(tree);
    if (st != SPEC_OK) return st;
    st = rope::check_rows(q, k, v, q_stride, k_stride, v_stride, Hq, Hkv, D, freq, rot, dt, true, 1);
    if (st != SPEC_OK) return st;
    if (B < 1 || B > 65535) return fail(SPEC_EINVAL, "B = %d out of 1..65535", B);
    if (!prefix_len || !q_out || !k_tree || !v_tree) return fail(SPEC_EINVAL, "prefix_len and the outputs must not be NULL");
    if (!aligned16(q_out) || !aligned16(k_tree) || !aligned16(v_tree)) return fail(SPEC_EALIGN, "the outputs must be 16-byte aligned");
    if (!aligned4(prefix_len) || !aligned4(pos_base)) return fail(SPEC_EALIGN, "prefix_len and pos_base must be 4-byte aligned");
    const int tokens = B * tree->T;
    const int es = dt == SPEC_BF16 ? 2 : 4;
    const struct { const void* x; int64_t stride; int heads; } in[3] = {{q, q_stride, Hq}, {k, k_stride, Hkv}, {v, v_stride, Hkv}};
    const struct { const void* x; int heads; } out[3] = {{q_out, Hq}, {k_tree, Hkv}, {v_tree, Hkv}};
    for (const auto& i : in)
        for (const auto& o : out)
            if (rope::overlap(o.x, static_cast<int64_t>(tokens) * o.heads * D * es, i.x,
                              ((tokens - 1) * i.stride + static_cast<int64_t>(i.heads) * D) * es))
                return fail(SPEC_EINVAL, "an output overlaps the projections");
    rope::Params p{};
    p.q = q; p.k = k; p.v = v;
    p.qs = q_stride; p.ks = k_stride; p.vs = v_stride;
    p.q_out = q_out; p.k_out = k_tree; p.v_out = v_tree;
    p.freq = freq; p.pos_base = pos_base; p.prefix_len = prefix_len;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.D = D; p.rot = rot; p.interleaved = interleaved != 0;
    p.depth = tree->depth; p.T = tree->T;
    return dt == SPEC_BF16 ? rope::run<__nv_bfloat16>("tree_rope", p, tokens, s) : rope::run<float>("tree_rope", p, tokens, s);
}
