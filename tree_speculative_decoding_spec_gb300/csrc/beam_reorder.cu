// Reordering of beams in place: beam w of a sequence takes over what its parent holds.
//
//   beam_reorder                 any state of a beam, one row of bytes
//   kv_reorder, kv_reorder_paged the cached keys and values of positions start[b] .. end[b] - 1
//
// A thread owns one column of 4 to 16 bytes (of a state, or of one position of one head) of all W
// beams: it reads the parents' values into registers and then writes them, so that
// permutations, cycles and parents with several children need neither order nor a second
// buffer.  Beams that keep their own rows are neither read nor written.  Bound by memory: each
// beam that changes is written once, each parent read once (children of one parent read it
// from L1).  W columns have to fit the registers: 16 bytes each up to 16 beams, 8 up to 32,
// 4 up to 64.
#include <algorithm>

#include "common.cuh"

namespace spec {
namespace reorder {

constexpr int kThreads = 256;

struct Params {
    char *x, *y;                      // y NULL: one tensor
    const int32_t* parent;            // [B, W]
    const int32_t *start, *end;       // [B]; NULL: one position (states)
    const int32_t* table;             // [B * W, max_blocks] or NULL
    int B, W, heads, max_blocks, num_blocks;
    int rows;                         // positions of one (block, head)
    int64_t cap;                      // positions of one sequence
    int64_t row_bytes;
    void* ws;
};

__device__ __forceinline__ bool range_of(const Params& p, int b, int& from, int& to) {
    from = 0;
    to = 1;
    if (p.start) {
        from = p.start[b];
        to = p.end[b];
        if (from < 0 || to < from || to > p.cap) {
            to = from;
            return false;
        }
    }
    return true;
}

// The call's status: one CTA looks at every parent, range and table entry and stores the word.
__device__ void check_all(const Params& p) {
    int bad = 0;
    const int rows = p.B * p.W;       // below 2^22
    for (int i = threadIdx.x; i < rows; i += kThreads) {
        const int w = p.parent[i];
        if (w < -1 || w >= p.W) bad = 1;
    }
    if (p.start)
        for (int b = threadIdx.x; b < p.B; b += kThreads) {
            int from, to;
            if (!range_of(p, b, from, to)) bad = 1;
        }
    if (p.table) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        for (int i = warp; i < rows; i += kThreads / 32) {
            int from, to;
            range_of(p, i / p.W, from, to);
            if (to > from)
                for (int j = from / p.rows + lane; j <= (to - 1) / p.rows; j += 32) {
                    const int blk = p.table[static_cast<size_t>(i) * p.max_blocks + j];
                    if (blk < 0 || blk >= p.num_blocks) bad = 1;
                }
        }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *static_cast<int4*>(p.ws) = make_int4(bad ? SPEC_EINVAL : SPEC_OK, 0, 0, 0);
}

// (Without a limit the compiler keeps every beam's addresses beside its values: 172 registers for 8 beams, 88 us for 45.)
template <typename V, int MOST>
__global__ void __launch_bounds__(kThreads, MOST <= 4 ? 6 : MOST <= 8 ? 4 : MOST <= 16 ? 2 : 1) k_reorder(const Params p) {
    griddep_wait();                   // the stream's kernel before this one may still run: its results are behind here
    if (blockIdx.x == 0) {            // one CTA more than there are for the rows
        if (blockIdx.y == 0 && blockIdx.z == 0) check_all(p);
        return;
    }
    __shared__ int s_parent[MOST];
    __shared__ unsigned s_moved[2];
    const int b = blockIdx.y;
    int from, to;
    range_of(p, b, from, to);
    if (threadIdx.x < 64) {
        const int w = threadIdx.x;
        const int q = w < p.W ? p.parent[static_cast<size_t>(b) * p.W + w] : -1;
        const bool moved = q >= 0 && q < p.W && q != w;
        if (w < MOST) s_parent[w] = moved ? q : w;
        const unsigned m = __ballot_sync(0xffffffffu, moved);
        if ((w & 31) == 0) s_moved[w >> 5] = m;
    }
    __syncthreads();
    const unsigned long long moved = s_moved[0] | (static_cast<unsigned long long>(s_moved[1]) << 32);
    if (!moved) return;
    const int h = blockIdx.z < static_cast<unsigned>(p.heads) ? blockIdx.z : blockIdx.z - p.heads;
    char* base = blockIdx.z < static_cast<unsigned>(p.heads) ? p.x : p.y;
    const uint32_t cols = static_cast<uint32_t>(p.row_bytes / static_cast<int64_t>(sizeof(V)));
    // position q of the range, column c of its row; one division, then steps
    const uint32_t first = (blockIdx.x - 1) * kThreads + threadIdx.x, step = (gridDim.x - 1) * kThreads;
    const uint32_t step_q = step / cols, step_c = step - step_q * cols;
    uint32_t q = first / cols, c = first - q * cols;
    const uint32_t count = to - from;
    // Where the beams' rows lie is the same for all of a warp's positions in one page: lane w works it out for beam w
    // (and w + 32) and the others take it from there.  (Each thread for itself: 700 instructions for 8 beams, 41 us where this takes 34.)
    const int lane = threadIdx.x & 31;
    constexpr int kOwn = MOST > 32 ? 2 : 1;
    int64_t own[kOwn];
    auto look_up = [&](int page) {
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            const int w = lane + 32 * k;
            own[k] = -1;
            if (w >= p.W) continue;
            int64_t blk = static_cast<int64_t>(b) * p.W + w;
            if (p.table) {
                blk = p.table[blk * p.max_blocks + page];
                if (blk < 0 || blk >= p.num_blocks) continue;
            }
            own[k] = (blk * p.heads + h) * p.rows * p.row_bytes;
        }
    };
    auto of_beam = [&](int w) -> int64_t {
        int64_t x = __shfl_sync(0xffffffffu, own[0], w & 31);
        if (kOwn > 1) {
            const int64_t y = __shfl_sync(0xffffffffu, own[kOwn - 1], w & 31);
            if (w >= 32) x = y;
        }
        return x;
    };
    if (!p.table) look_up(0);
    for (unsigned todo; (todo = __ballot_sync(0xffffffffu, q < count)) != 0;) {
        const int at = from + static_cast<int>(q);
        const int page = p.table ? at / p.rows : 0;
        const int64_t in = (at - static_cast<int64_t>(page) * p.rows) * p.row_bytes + c * static_cast<int64_t>(sizeof(V));
        while (todo) {                // the pages of the warp's positions, one after the other
            const int now = __shfl_sync(0xffffffffu, page, __ffs(todo) - 1);
            const bool mine = q < count && page == now;
            todo &= ~__ballot_sync(0xffffffffu, mine);
            if (p.table) look_up(now);
            V v[MOST];
            unsigned long long read = 0;
#pragma unroll
            for (int w = 0; w < MOST; ++w)
                if ((moved >> w) & 1) {
                    const int64_t src = of_beam(s_parent[w]);
                    if (src >= 0) {
                        if (mine) v[w] = *reinterpret_cast<const V*>(base + src + in);
                        read |= 1ull << w;
                    }
                }
#pragma unroll
            for (int w = 0; w < MOST; ++w)
                if ((read >> w) & 1) {
                    const int64_t dst = of_beam(w);
                    if (dst >= 0 && mine) __stcs(reinterpret_cast<V*>(base + dst + in), v[w]);   // (not read again here)
                }
        }
        q += step_q;
        c += step_c;
        if (c >= cols) {
            c -= cols;
            ++q;
        }
    }
}

spec_status run(const char* name, const Params& p, int64_t positions, cudaStream_t s) {
    const int64_t rb = p.row_bytes;
    const int width = rb % 16 == 0 && p.W <= 16 ? 16 : rb % 8 == 0 && p.W <= 32 ? 8 : 4;
    void (*kern)(const Params) = width == 16 ? (p.W <= 4 ? k_reorder<uint4, 4> : p.W <= 8 ? k_reorder<uint4, 8> : k_reorder<uint4, 16>)
                                 : width == 8 ? k_reorder<uint2, 32> : k_reorder<uint32_t, 64>;
    // a row of CTAs per sequence, head and tensor: enough for sixteen on every SM, each with work for its threads if
    // every sequence is full
    const int64_t lines = static_cast<int64_t>(p.heads) * (p.y ? 2 : 1);
    const int64_t most = std::max<int64_t>(1, (positions * (rb / width) + kThreads - 1) / kThreads);
    const int64_t want = (16 * device_sm_count() + p.B * lines - 1) / (p.B * lines);
    const unsigned per = static_cast<unsigned>(std::min(most, want));
    SPEC_CUDA_TRY(launch_ex(name, kern, dim3(per + 1, p.B, static_cast<unsigned>(lines)), dim3(kThreads), 0, s, true, p));
    return SPEC_OK;
}

spec_status check_common(const Params& p, size_t ws_bytes) {
    if (p.B < 1 || p.B > 65535) return fail(SPEC_EINVAL, "B = %d out of 1..65535", p.B);
    if (p.W < 1 || p.W > SPEC_MAX_BEAMS) return fail(SPEC_EINVAL, "W = %d out of 1..%d", p.W, SPEC_MAX_BEAMS);
    if (!p.parent) return fail(SPEC_EINVAL, "parent must not be NULL");
    if (!aligned4(p.parent)) return fail(SPEC_EALIGN, "parent must be 4-byte aligned");
    if (!p.ws || ws_bytes < kWsHeader) return fail(SPEC_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, kWsHeader);
    if (!aligned16(p.ws)) return fail(SPEC_EALIGN, "workspace must be 16-byte aligned");
    return SPEC_OK;
}

spec_status kv(const char* name, Params& p, const void* k, const void* v, int Hkv, int D, spec_dtype dt, size_t ws_bytes, cudaStream_t s) {
    spec_status st = check_common(p, ws_bytes);
    if (st != SPEC_OK) return st;
    if (dt != SPEC_BF16 && dt != SPEC_F32) return fail(SPEC_EINVAL, "dtype %d unknown", static_cast<int>(dt));
    const int es = dt == SPEC_BF16 ? 2 : 4;
    if (Hkv < 1 || Hkv > 1024) return fail(SPEC_EINVAL, "Hkv = %d out of 1..1024", Hkv);
    if (D < 1 || D > 1024 || (D * es) % 16) return fail(SPEC_EINVAL, "D = %d: 1..1024 and a multiple of 16 bytes", D);
    if (!k || !v || !p.start || !p.end) return fail(SPEC_EINVAL, "the cache, start and end must not be NULL");
    const uint64_t bytes = static_cast<uint64_t>(p.table ? p.num_blocks : p.B * p.W) * Hkv * p.rows * D * es;
    const uintptr_t ka = reinterpret_cast<uintptr_t>(k), va = reinterpret_cast<uintptr_t>(v);
    if (ka < va + bytes && va < ka + bytes) return fail(SPEC_EINVAL, "keys and values overlap");
    if (!aligned16(k) || !aligned16(v)) return fail(SPEC_EALIGN, "the cache must be 16-byte aligned");
    if (!aligned4(p.start) || !aligned4(p.end) || !aligned4(p.table))
        return fail(SPEC_EALIGN, "start, end and the block table must be 4-byte aligned");
    p.x = static_cast<char*>(const_cast<void*>(k));
    p.y = static_cast<char*>(const_cast<void*>(v));
    p.heads = Hkv;
    p.row_bytes = static_cast<int64_t>(D) * es;
    return run(name, p, p.cap, s);
}

}  // namespace reorder
}  // namespace spec

using namespace spec;

extern "C" size_t beam_reorder_workspace_size(void) { return kWsHeader; }

extern "C" spec_status beam_reorder(void* state, int64_t row_bytes, const int32_t* parent, int32_t B, int32_t W,
                                    void* ws, size_t ws_bytes, spec_stream_t s) {
    clear_error();
    reorder::Params p{};
    p.x = static_cast<char*>(state); p.parent = parent; p.B = B; p.W = W; p.ws = ws;
    spec_status st = reorder::check_common(p, ws_bytes);
    if (st != SPEC_OK) return st;
    if (row_bytes < 4 || row_bytes % 4 || row_bytes > (1ll << 32)) return fail(SPEC_EINVAL, "row_bytes = %lld: a multiple of 4 in 4..2^32", static_cast<long long>(row_bytes));
    if (!state) return fail(SPEC_EINVAL, "state must not be NULL");
    if (!aligned16(state)) return fail(SPEC_EALIGN, "state must be 16-byte aligned");
    p.heads = 1; p.rows = 1; p.cap = 1; p.row_bytes = row_bytes;
    return reorder::run("beam_reorder", p, 1, reinterpret_cast<cudaStream_t>(s));
}

extern "C" spec_status kv_reorder(void* k_cache, void* v_cache, const int32_t* parent, const int32_t* start, const int32_t* end,
                                  int32_t B, int32_t W, int32_t Hkv, int32_t Lmax, int32_t D, spec_dtype dt, void* ws,
                                  size_t ws_bytes, spec_stream_t s) {
    clear_error();
    if (Lmax < 1 || Lmax > (1 << 22)) return fail(SPEC_EINVAL, "Lmax = %d out of 1..2^22", Lmax);
    reorder::Params p{};
    p.parent = parent; p.start = start; p.end = end; p.B = B; p.W = W; p.rows = Lmax; p.cap = Lmax; p.ws = ws;
    return reorder::kv("kv_reorder", p, k_cache, v_cache, Hkv, D, dt, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}

extern "C" spec_status kv_reorder_paged(void* k_pool, void* v_pool, int32_t num_blocks, const int32_t* block_table,
                                        int32_t max_blocks, int32_t block_size, const int32_t* parent, const int32_t* start,
                                        const int32_t* end, int32_t B, int32_t W, int32_t Hkv, int32_t D, spec_dtype dt,
                                        void* ws, size_t ws_bytes, spec_stream_t s) {
    clear_error();
    if (num_blocks < 1 || max_blocks < 1 || block_size < 1)
        return fail(SPEC_EINVAL, "num_blocks = %d, max_blocks = %d, block_size = %d must be positive", num_blocks,
                    max_blocks, block_size);
    if (static_cast<int64_t>(max_blocks) * block_size > (1 << 22))
        return fail(SPEC_EINVAL, "max_blocks * block_size = %lld positions exceed 2^22",
                    static_cast<long long>(max_blocks) * block_size);
    if (!block_table) return fail(SPEC_EINVAL, "block_table must not be NULL");
    reorder::Params p{};
    p.parent = parent; p.start = start; p.end = end; p.B = B; p.W = W; p.ws = ws;
    p.table = block_table; p.max_blocks = max_blocks; p.num_blocks = num_blocks; p.rows = block_size;
    p.cap = static_cast<int64_t>(max_blocks) * block_size;
    return reorder::kv("kv_reorder", p, k_pool, v_pool, Hkv, D, dt, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}
