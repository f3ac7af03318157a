// What the CUDA-core and the tensor-core kernels of kv_weigh share.
#pragma once

#include <cmath>

#include "common.cuh"

namespace spec {
namespace weigh {

struct Params {
    const void* q;                    // [B, Hq, T, D]
    const float* lse;                 // [B, Hq, T]
    const void* k;                    // [B, Hkv, cap, D], or pool [num_blocks, Hkv, rows, D]
    const int32_t* table;             // [B, max_blocks] or NULL
    const int32_t* len;               // [B]: cache length, the rows' keys included
    const int32_t* seen;              // [B] or NULL: tokens of the sequence so far (NULL: len)
    const int32_t* n_rows;            // [B] or NULL: rows that count, the first of T (NULL: T)
    const int32_t *accept_len, *path; // [B], [B, P] or NULL: the rows are the path's nodes
    int P, B, Hq, Hkv, T;
    int rows;                         // positions of one (block, head)
    int cap;                          // positions of one sequence; stride of acc and pos
    int max_blocks, num_blocks;
    float scale, decay;
    float* acc;                       // [B, Hkv, cap]
    int32_t* pos;                     // the same, or NULL
    void* ws;
};

// Of one sequence: keys, rows that count (its last `count` keys are theirs), and whether they make sense.
struct Rows {
    int n, count;
    bool ok;
};
__device__ __forceinline__ Rows rows_of(const Params& p, int b) {
    Rows r;
    r.n = p.len[b];
    r.count = p.path ? p.accept_len[b] + 1 : p.n_rows ? p.n_rows[b] : p.T;
    r.ok = r.n >= 0 && r.n <= p.cap && r.count >= (p.path ? 1 : 0) && r.count <= (p.path ? p.P : p.T) && r.count <= r.n;
    if (r.ok && p.path)
        for (int i = 0; i < r.count; ++i) {   // at most 17, in one line of memory
            const int node = p.path[static_cast<int64_t>(b) * p.P + i];
            if (node < 0 || node >= p.T) r.ok = false;
        }
    return r;
}

__device__ __forceinline__ int node_of(const Params& p, int b, int i) {
    return p.path ? p.path[static_cast<int64_t>(b) * p.P + i] : i;
}

// Row of the keys where position j of a sequence and head lies, -1 in a block outside the pool.
__device__ __forceinline__ int64_t key_row(const Params& p, int b, int h, int j) {
    int64_t blk = b;
    if (p.table) {
        blk = p.table[static_cast<int64_t>(b) * p.max_blocks + j / p.rows];
        if (blk < 0 || blk >= p.num_blocks) return -1;
        j %= p.rows;
    }
    return (blk * p.Hkv + h) * p.rows + j;
}

// Key j's new weight: the rows' own keys start anew.  decay 0 forgets what was there, whatever it was.
__device__ __forceinline__ void store(const Params& p, int b, int h, int j, const Rows& r, float sum) {
    const int64_t at = (static_cast<int64_t>(b) * p.Hkv + h) * p.cap + j;
    const bool fresh = j >= r.n - r.count;
    p.acc[at] = fresh || p.decay == 0.f ? sum : fmaf(p.decay, p.acc[at], sum);
    if (fresh && p.pos) p.pos[at] = (p.seen ? p.seen[b] : r.n) - r.n + j;
}

// bf16, kv_weigh_tc.cu: what it needs behind the workspace's header, and its launches.
size_t weigh_tc_bytes(int g, int T, int path_len);
spec_status weigh_tc_run(const Params& p, int D, void* scratch, cudaStream_t s);

// The call's status: one CTA of N threads looks at every sequence and table entry and stores the word.
template <int N> __device__ void check_all(const Params& p) {
    int bad = 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int b = warp; b < p.B; b += N / 32) {
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
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *static_cast<int4*>(p.ws) = make_int4(bad ? SPEC_EINVAL : SPEC_OK, 0, 0, 0);
}

}  // namespace weigh
}  // namespace spec
