// tree_attention_shared, tree_attention_scored and their paged forms: tree
// attention over a prefix that the whole batch shares, and with capped, biased
// and windowed scores.
//
// For query head h, sequence b, node i (position P = Ls + L_b + depth[i]) and a
// key at position p that the node sees (every shared and cached key, and of the
// tree its ancestors and itself; with a window only p > P - window):
//     x = scale q.k;   x = cap tanh(x / cap);   x = x - slope[h] (P - p)
//     out = sum exp(x) v / sum exp(x),   lse = log sum exp(x)
// The sums run in one pass over the keys with a running maximum, in base 2 and
// in 32 bits; splits of the keys and the shared part are joined by their
// (max, sum, O).  See attention_shared.cuh for how the work is cut.
//
// This file: the CUDA-core items (fp32), the join, the host side.  bf16 items
// are in attention_shared_tc.cu.
#include <algorithm>
#include <cmath>

#include "attention_shared.cuh"
#include "tc.cuh"

namespace spec {
namespace shr {

using tc::ffma2;
using tc::pk2;
using tc::upk2;

// ---------------------------------------------------------------- CUDA-core items

constexpr int FR = 64;   // rows of a block, at most
constexpr int FK = kTile;   // keys of a tile
constexpr int kFmaThreads = 256;

// Thread (rg, kg) = (t / 16, t % 16) holds R rows from R rg, keys kg + 16 j of a tile and output columns
// 4 kg .. of each 64.  fp32 operands have no tensor-core product of their own precision, so the FMA units
// and the shared memory that feeds them bound this kernel: at R = 4, 32 packed FMAs per 8 loads of 16 bytes in
// the score loop; a 64 x 64 tile of head dim 128 takes some 8.5 us, its FMAs alone would 4.2.  The next tile's
// keys and values arrive meanwhile (cp.async, two buffers); rows are 16, 32 or 64 to a block as the call needs
// them, and items of head dim 64 go two to an SM.  8 sequences of 2368 keys and 13 nodes, 8 heads of 128,
// took 265 us before these and 131 with them; 21 of 896 keys and 12 nodes, 4 heads of 64, 65 and 41; two trees
// of 75 nodes behind 3840 keys 84 and 71.  512 threads for head dim 128, two rows each, took 82.
__device__ __forceinline__ void copy_async16(float* dst, const float* src, bool ok) {   // zeros where not ok
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int D, int R>
__global__ void __launch_bounds__(kFmaThreads, D == 64 ? 2 : 1) k_attn_shared_fma(const Params p) {
    using T = float;
    constexpr int FR = kFmaThreads / 16 * R;   // rows of a block
    constexpr int LD = D + 4, LP = FK + 4, DT = D / 16;
    extern __shared__ float4 smem4[];
    float* Qs = reinterpret_cast<float*>(smem4);
    float* KVs = Qs + FR * LD;              // two buffers: keys, then values of a tile
    float* Ps = KVs + 4 * FK * LD;
    const int t = threadIdx.x, rg = t >> 4, kg = t & 15;
    __shared__ int bad;
    if (t == 0) bad = 0;
    griddep_wait();
    griddep_launch();   // the join may start launching: it waits for the partials
    const Plan plan = make_plan(p);
    if (blockIdx.x == 0 && t < 32) publish_plan(p, plan);
    const T* q = static_cast<const T*>(p.q);
    const float scale2 = p.scale * kLog2e, cap2 = p.softcap * kLog2e, incap = p.softcap > 0.f ? p.scale / p.softcap : 0.f;

    Walk walk(p, plan, blockIdx.x);
    for (Item it; walk.next(p, plan, it);) {
        __syncthreads();   // the last item's Q and P are read
        for (int idx = t; idx < FR * (D / 4); idx += kFmaThreads) {
            const int r = idx / (D / 4), c4 = idx % (D / 4);
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (r < it.rows) load4(q + row_of_q(p, it, r) * D + c4 * 4, v);
            *reinterpret_cast<float4*>(&Qs[r * LD + c4 * 4]) = make_float4(v[0], v[1], v[2], v[3]);
        }
        int node[R], pos[R];
        float slope2[R], m_run[R], l_run[R];
        unsigned long long o2[R][DT / 2];     // pairs of columns
#pragma unroll
        for (int ii = 0; ii < R; ++ii) {
            const int r = min(R * rg + ii, it.rows - 1);
            const int b = it.b + (p.gT < p.RB ? r / p.gT : 0);
            const int i = p.gT < p.RB ? r % p.gT : it.rb * p.RB + r;
            node[ii] = i % p.T;
            pos[ii] = plan.Ls + own_len(p, b) + p.depth[node[ii]];
            slope2[ii] = p.slopes ? p.slopes[it.kvh * p.g + i / p.T] * kLog2e : 0.f;
            m_run[ii] = -INFINITY;
            l_run[ii] = 0.f;
#pragma unroll
            for (int e = 0; e < DT / 2; ++e) o2[ii][e] = pk2(0.f, 0.f);
        }
        const int first = it.shared ? plan.sT0 : own_first(p, it.L);
        const int n_pre = it.shared ? plan.nS : own_tiles(p, it.L) - tiles_of(p.T);
        // a tile's keys and values into buffer (tile - t0) % 2; keys past the end become zeros
        auto fetch = [&](int tile) {
            const bool tree = !it.shared && tile >= n_pre;
            const int j0 = (tree ? tile - n_pre : first + tile) * FK;
            const int j_end = tree ? p.T : it.shared ? plan.Ls : it.L;
            float* dst = KVs + ((tile - it.t0) & 1) * (2 * FK * LD);
            for (int x = t; x < FK * (D / 4); x += kFmaThreads) {
                const int jl = x / (D / 4), c4 = x % (D / 4), j = j0 + jl;
                const T *ksrc = static_cast<const T*>(p.kt), *vsrc = static_cast<const T*>(p.vt);
                size_t row = 0;
                bool ok = j < j_end;
                if (tree) {
                    row = (static_cast<size_t>(it.b) * p.Hkv + it.kvh) * p.T + j;
                } else if (p.pg.table) {   // the key's pool block and row
                    ksrc = static_cast<const T*>(p.kc);
                    vsrc = static_cast<const T*>(p.vc);
                    if (ok) {
                        const int blk = it.shared ? p.shared_table[j / p.pg.bs]
                                                  : p.pg.table[static_cast<size_t>(it.b) * p.pg.max_blocks + j / p.pg.bs];
                        ok = blk >= 0 && blk < p.pg.num_blocks;
                        if (!ok) bad = 1;   // the key reads as zeros
                        row = (static_cast<size_t>(ok ? blk : 0) * p.Hkv + it.kvh) * p.pg.bs + j % p.pg.bs;
                    }
                } else if (it.shared) {
                    ksrc = static_cast<const T*>(p.ks);
                    vsrc = static_cast<const T*>(p.vs);
                    row = static_cast<size_t>(it.kvh) * p.Lshared + j;
                } else {
                    ksrc = static_cast<const T*>(p.kc);
                    vsrc = static_cast<const T*>(p.vc);
                    row = (static_cast<size_t>(it.b) * p.Hkv + it.kvh) * p.Lmax + j;
                }
                if (!ok) row = 0;
                copy_async16(dst + jl * LD + c4 * 4, ksrc + row * D + c4 * 4, ok);
                copy_async16(dst + FK * LD + jl * LD + c4 * 4, vsrc + row * D + c4 * 4, ok);
            }
            copy_async_commit();
        };
        fetch(it.t0);
        for (int tile = it.t0; tile < it.t1; ++tile) {
            const bool tree = !it.shared && tile >= n_pre;
            const int j0 = (tree ? tile - n_pre : first + tile) * FK;
            const int j_end = tree ? p.T : it.shared ? plan.Ls : it.L;
            const float *Ks = KVs + ((tile - it.t0) & 1) * (2 * FK * LD), *Vs = Ks + FK * LD;
            __syncthreads();   // the other buffer and P are read
            if (tile + 1 < it.t1) {
                fetch(tile + 1);
                copy_async_wait<1>();
            } else {
                copy_async_wait<0>();
            }
            __syncthreads();

            uint64_t seen[R];   // of a tree tile: the nodes' ancestors and themselves
            if (tree) {
#pragma unroll
                for (int ii = 0; ii < R; ++ii) seen[ii] = p.anc[static_cast<size_t>(node[ii]) * p.words + (j0 >> 6)];
            }
            // two products at a time: even and odd dimensions add up apart
            unsigned long long s2[R][4];
#pragma unroll
            for (int ii = 0; ii < R; ++ii)
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) s2[ii][jj] = pk2(0.f, 0.f);
#pragma unroll (D == 64 ? 2 : 4)
            for (int dd = 0; dd < D; dd += 4) {
                ulonglong2 qa[R], kb[4];
#pragma unroll
                for (int ii = 0; ii < R; ++ii) qa[ii] = *reinterpret_cast<const ulonglong2*>(&Qs[(R * rg + ii) * LD + dd]);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) kb[jj] = *reinterpret_cast<const ulonglong2*>(&Ks[(kg + 16 * jj) * LD + dd]);
#pragma unroll
                for (int ii = 0; ii < R; ++ii)
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj) s2[ii][jj] = ffma2(qa[ii].y, kb[jj].y, ffma2(qa[ii].x, kb[jj].x, s2[ii][jj]));
            }
            float s[R][4];
#pragma unroll
            for (int ii = 0; ii < R; ++ii)
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    float even, odd;
                    upk2(s2[ii][jj], even, odd);
                    s[ii][jj] = even + odd;
                }
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                const int j = j0 + kg + 16 * jj;
                const bool in = j < j_end;
                const int kpos = tree ? (in ? plan.Ls + it.L + p.depth[j] : 0) : it.shared ? j : plan.Ls + j;
#pragma unroll
                for (int ii = 0; ii < R; ++ii) {
                    const int far = pos[ii] - kpos;
                    bool ok = in && (p.window <= 0 || far < p.window);
                    if (tree && ok) ok = (seen[ii] >> (j & 63)) & 1ull;
                    float x = p.softcap > 0.f ? cap2 * tanhf(s[ii][jj] * incap) : s[ii][jj] * scale2;
                    x -= slope2[ii] * static_cast<float>(far);
                    s[ii][jj] = ok ? x : -INFINITY;
                }
            }
#pragma unroll
            for (int ii = 0; ii < R; ++ii) {
                float mt = fmaxf(fmaxf(s[ii][0], s[ii][1]), fmaxf(s[ii][2], s[ii][3]));
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
                const float m_new = fmaxf(m_run[ii], mt);
                const float ref = m_new == -INFINITY ? 0.f : m_new;   // nothing seen so far
                const float alpha = exp2f(m_run[ii] - ref);
                float pr[4], lt = 0.f;
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) { pr[jj] = exp2f(s[ii][jj] - ref); lt += pr[jj]; }
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, off);
                l_run[ii] = l_run[ii] * alpha + lt;
                m_run[ii] = m_new;
#pragma unroll
                for (int e = 0; e < DT / 2; ++e) o2[ii][e] = ffma2(o2[ii][e], pk2(alpha, alpha), pk2(0.f, 0.f));
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) Ps[(R * rg + ii) * LP + kg + 16 * jj] = pr[jj];
            }
            __syncwarp();
#pragma unroll 2
            for (int j = 0; j < FK; j += 4) {
                float4 pj[R];
#pragma unroll
                for (int ii = 0; ii < R; ++ii) pj[ii] = *reinterpret_cast<const float4*>(&Ps[(R * rg + ii) * LP + j]);
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int h = 0; h < DT / 4; ++h) {
                        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&Vs[(j + u) * LD + h * 64 + kg * 4]);
#pragma unroll
                        for (int ii = 0; ii < R; ++ii) {
                            const float w = u == 0 ? pj[ii].x : u == 1 ? pj[ii].y : u == 2 ? pj[ii].z : pj[ii].w;
                            o2[ii][2 * h] = ffma2(pk2(w, w), v.x, o2[ii][2 * h]);
                            o2[ii][2 * h + 1] = ffma2(pk2(w, w), v.y, o2[ii][2 * h + 1]);
                        }
                    }
            }
        }
        const int stride = it.shared ? p.rowsS : p.rowsO;
        float4* part = (it.shared ? p.part_s : p.part_o) + static_cast<size_t>(it.index) * (D / 4 + 1) * stride;
#pragma unroll
        for (int ii = 0; ii < R; ++ii) {
            const int r = R * rg + ii;
            if (r >= it.rows) continue;
            float o[DT];
#pragma unroll
            for (int e = 0; e < DT / 2; ++e) upk2(o2[ii][e], o[2 * e], o[2 * e + 1]);
            if (it.direct) {
                const size_t row = row_of_q(p, it, r);
                const float inv = 1.f / l_run[ii];
#pragma unroll
                for (int h = 0; h < DT / 4; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        static_cast<T*>(p.out)[row * D + h * 64 + kg * 4 + e] = from_f32<T>(o[h * 4 + e] * inv);
                if (p.lse && kg == 0) p.lse[row] = (m_run[ii] + log2f(l_run[ii])) * kLn2;
            } else {
                if (kg == 0) part[r] = make_float4(m_run[ii], l_run[ii], 0.f, 0.f);
#pragma unroll
                for (int h = 0; h < DT / 4; ++h)
                    part[static_cast<size_t>(1 + h * 16 + kg) * stride + r] =
                        make_float4(o[h * 4 + 0], o[h * 4 + 1], o[h * 4 + 2], o[h * 4 + 3]);
            }
        }
    }
    __syncthreads();
    if (t == 0) p.cta_status[blockIdx.x] = bad ? SPEC_EINVAL : SPEC_OK;
}

// ---------------------------------------------------------------- the join

// One CTA of eight warps per (sequence, KV head, 32 rows of its gT), each warp an eighth of the
// columns (four warps with twice the columns each: 1.5 us more in most cases).  Lanes are rows, so
// the partials are read as whole lines; with fewer than 32 rows the lanes left over take other parts
// of the same rows (lane = part * R + row), and shuffles add them up.  The output goes through shared
// memory to leave as whole rows.  Bound by reading the partials once (70B trees over 16K shared keys,
// some 55 MB of them: 15 us), and for few rows by the latency of the look-ups before that (7 us).
constexpr int kJoin = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kJoin) k_attn_shared_join(const Params p, int n_rg, int R) {
    constexpr int C = D / 4 / (kJoin / 32);   // float4 columns per warp
    __shared__ __align__(16) T tile[32][D + 16 / sizeof(T)];   // read 16 bytes at a time
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = divide(blockIdx.x, n_rg), r0 = (blockIdx.x - col * n_rg) * 32;
    const int b = divide(col, p.Hkv), kvh = col - b * p.Hkv;
    const int lr = lane & (R - 1), sub = divide(lane, R), subs = divide(32, R);
    const int i = r0 + lr;                        // row within gT
    const int n = own_tiles(p, own_len(p, b));
    griddep_wait();
    if (blockIdx.x == 0 && warp == 0) {           // the call's status
        int worst = SPEC_OK;
        for (int i = lane; i < p.ctas; i += 32) worst = max(worst, p.cta_status[i]);
        for (int o = 16; o > 0; o >>= 1) worst = max(worst, __shfl_xor_sync(0xffffffffu, worst, o));
        if (lane == 0) *static_cast<int4*>(p.ws) = make_int4(worst, 0, 0, 0);
    }
    const Plan t = *reinterpret_cast<const Plan*>(static_cast<unsigned char*>(p.ws) + kPlanOffset);
    const int rb = divide(r0, p.RB);              // 32 divides RB, or all rows fit one block
    const int sb = p.gT >= p.RB ? b * p.n_rbO + rb : divide(b, p.nbb);
    const int colS = kvh * p.n_rbS + sb, colO = kvh * p.n_rbO + rb, cols = p.Hkv * p.n_rbO;
    const Cuts kO(p, t.q, Place(p, false, n), p.cum[b], colO, p.n_rbO), kS(p, t.q, Place(p, true, t.nS), 0, colS, p.per);
    const int nsS = (t.nS ? kS.count : 0) * p.repS, parts = nsS + kO.count * p.repO;
    if (parts == 1) return;                       // written by its item
    const int rO = i - rb * p.RB, rS = p.gT >= p.RB ? rO : (b - sb * p.nbb) * p.gT + i;
    const bool in = i < p.gT;
    // part k: of the shared items, then of the own ones; item k / rep, copy k % rep (1 or 4)
    auto part = [&](int k, int& rows) -> const float4* {
        const bool shared = k < nsS;
        const int rep = shared ? p.repS : p.repO, cap = shared ? p.rowsS : p.rowsO;
        const int x = shared ? k : k - nsS, item = rep == 1 ? x : x >> 2, copy = rep == 1 ? 0 : x & 3;
        const int slot = shared ? kS.slot(colS, p.Hkv * p.n_rbS, item) : kO.slot(b * cols + colO, p.B * cols, item);
        rows = cap * rep;
        return (shared ? p.part_s : p.part_o) + static_cast<size_t>(slot) * (D / 4 + 1) * rows + copy * cap + (shared ? rS : rO);
    };
    float M = -INFINITY, l = 0.f;
    float4 acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
        for (int k = sub; k < parts; k += 2 * subs) {   // two parts' lines in flight
            const bool two = k + subs < parts;
            int rows0, rows1;
            const float4 *at0 = part(k, rows0), *at1 = part(two ? k + subs : k, rows1);
            const float4 h0 = at0[0];
            float4 h1 = at1[0], v0[C], v1[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                v0[c] = at0[static_cast<size_t>(1 + warp * C + c) * rows0];
                v1[c] = at1[static_cast<size_t>(1 + warp * C + c) * rows1];
            }
            if (!two) h1 = make_float4(-INFINITY, 0.f, 0.f, 0.f);
            // a part in which the row saw nothing (one of NaN scores alone has a NaN sum, and counts)
            const bool none0 = h0.x == -INFINITY && h0.y == 0.f, none1 = h1.x == -INFINITY && h1.y == 0.f;
            const float m = fmaxf(M, fmaxf(h0.x, h1.x)), ref = m == -INFINITY ? 0.f : m;
            const float keep = exp2f(M - ref), w0 = exp2f(h0.x - ref), w1 = exp2f(h1.x - ref);
            M = m;
            l *= keep;
            if (!none0) l += w0 * h0.y;
            if (!none1) l += w1 * h1.y;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                acc[c].x *= keep; acc[c].y *= keep; acc[c].z *= keep; acc[c].w *= keep;
                if (!none0) {
                    acc[c].x += w0 * v0[c].x; acc[c].y += w0 * v0[c].y;
                    acc[c].z += w0 * v0[c].z; acc[c].w += w0 * v0[c].w;
                }
                if (!none1) {
                    acc[c].x += w1 * v1[c].x; acc[c].y += w1 * v1[c].y;
                    acc[c].z += w1 * v1[c].z; acc[c].w += w1 * v1[c].w;
                }
            }
        }
    }
    for (int o = R; o < 32; o <<= 1) {            // the lanes of the same row
        const float M2 = __shfl_xor_sync(0xffffffffu, M, o), m = fmaxf(M, M2), ref = m == -INFINITY ? 0.f : m;
        const float keep = exp2f(M - ref), w = exp2f(M2 - ref);
        M = m;
        const float l2 = __shfl_xor_sync(0xffffffffu, l, o);
        l = l * keep + l2 * w;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float4 a2 = make_float4(__shfl_xor_sync(0xffffffffu, acc[c].x, o), __shfl_xor_sync(0xffffffffu, acc[c].y, o),
                                          __shfl_xor_sync(0xffffffffu, acc[c].z, o), __shfl_xor_sync(0xffffffffu, acc[c].w, o));
            acc[c].x = acc[c].x * keep + a2.x * w; acc[c].y = acc[c].y * keep + a2.y * w;
            acc[c].z = acc[c].z * keep + a2.z * w; acc[c].w = acc[c].w * keep + a2.w * w;
        }
    }
    const float inv = 1.f / l;
    if (sub == 0) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            T* d = &tile[lr][(warp * C + c) * 4];
            d[0] = from_f32<T>(acc[c].x * inv); d[1] = from_f32<T>(acc[c].y * inv);
            d[2] = from_f32<T>(acc[c].z * inv); d[3] = from_f32<T>(acc[c].w * inv);
        }
    }
    const size_t row0 = (static_cast<size_t>(b) * p.Hq + kvh * p.g) * p.T + r0;
    if (in && sub == 0 && warp == 0 && p.lse) p.lse[row0 + lr] = (M + log2f(l)) * kLn2;
    __syncthreads();
    constexpr int E = 16 / sizeof(T);
    const int rows = min(32, p.gT - r0);
    for (int x = threadIdx.x; x < rows * (D / E); x += kJoin) {
        const int r = x / (D / E), c = x % (D / E);
        *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (row0 + r) * D + c * E) = *reinterpret_cast<const uint4*>(&tile[r][c * E]);
    }
}

// ---------------------------------------------------------------- host

HostPlan host_plan(Params& p, bool tc, bool shared, int ctas) {
    HostPlan h{};
    h.tc = tc;
    p.g = p.Hq / p.Hkv;
    p.gT = p.g * p.T;
    // fp32 blocks are as high as their rows need, 64 where sequences are to share keys in them
    p.RB = tc ? kTcRows : (shared && p.Lshared >= p.Lmax) || p.gT > 32 ? FR : p.gT > 16 ? 32 : 16;
    p.nbb = p.gT >= p.RB ? 1 : std::min(p.RB / p.gT, p.B);
    p.n_rbO = (p.gT + p.RB - 1) / p.RB;
    p.n_rbS = p.gT >= p.RB ? p.B * p.n_rbO : (p.B + p.nbb - 1) / p.nbb;
    p.rowsO = std::min(p.gT, p.RB);
    p.rowsS = p.nbb * p.rowsO;
    p.ctas = ctas;
    p.per = p.gT >= p.RB ? p.n_rbO : 1;
    // Costs.  fp32: tiles alone, so that a call with fewer tiles than CTAs is cut into single ones (small scored
    // case 28 us where an item's start counted as a tile, 23 where it counts nothing).  Tensor cores, in thirds
    // of a pair's tile (1700 cycles): a narrow tile, bound by memory or by its softmax, takes two thirds of that,
    // an item's rows some 8000, 5500 or (few rows) 3500 cycles to start and store.  An own column of plain
    // scores ends in a partial tile and the tree's masks, worth another 14 (70B trees over 16K shared keys: the
    // CTAs with own columns ran 450K cycles where the others ran 408K, 254 us without, 225 with); where scores
    // are transformed every tile is as slow as those.  Capped scores take the softmax longer, a pair's two
    // groups in turn on the same units: a narrow tile is four sevenths (32K capped 281 us at two thirds, 269).
    struct Costs {
        int pair, narrow, fix_pair, fix_narrow, fix_few, tail;
    };
    const Costs c = !tc ? Costs{1, 1, 0, 0, 0, 0}
                    : p.softcap > 0.f ? Costs{7, 4, 35, 23, 14, 0}
                    : Costs{3, 2, 15, 10, 6, p.window > 0 || p.slopes ? 0 : 14};
    const int last = p.gT - (p.n_rbO - 1) * p.RB;
    p.wF = c.pair;
    p.fixF = c.fix_pair;
    p.tailF = c.tail;
    auto cost = [&](int rows, int& w, int& fix, int& tail) {
        const bool pair = rows > kTcRows / 2;
        w = pair ? c.pair : c.narrow;
        fix = pair ? c.fix_pair : rows > 32 ? c.fix_narrow : c.fix_few;
        tail = pair ? c.tail : 0;
    };
    int none;
    cost(p.gT >= p.RB ? last : p.rowsS, p.wS, p.fixS, none);
    cost(last, p.wO, p.fixO, p.tailO);
    p.repS = tc && p.rowsS <= 32 ? 4 : 1;
    p.repO = tc && p.rowsO <= 32 ? 4 : 1;
    p.min_piece = tc ? 2 : 1;
    const size_t per_row = sizeof(float) * (p.D + 4);
    const size_t items_s = shared ? static_cast<size_t>(p.Hkv) * p.n_rbS + ctas : 0;   // one slot per column and per cut
    const size_t items_o = static_cast<size_t>(p.B) * p.Hkv * p.n_rbO + ctas;
    h.status_off = kWsHeader;
    h.cum_off = h.status_off + round_up(sizeof(int32_t) * static_cast<size_t>(ctas), 256);
    h.part_s_off = h.cum_off + round_up(sizeof(int32_t) * static_cast<size_t>(p.B), 256);
    h.part_o_off = h.part_s_off + round_up(items_s * p.rowsS * p.repS * per_row, 256);
    h.total = h.part_o_off + round_up(items_o * p.rowsO * p.repO * per_row, 256);
    return h;
}

static spec_status check_shapes(const spec_tree* t, int B, int Hq, int Hkv, int Ls, int Lmax, int D, spec_dtype dt) {
    spec_status st = check_tree(t);
    if (st != SPEC_OK) return st;
    if (dt != SPEC_F32 && dt != SPEC_BF16) return fail(SPEC_EINVAL, "dtype %d unknown", static_cast<int>(dt));
    if (B < 1 || B > 65535) return fail(SPEC_EINVAL, "B = %d out of 1..65535", B);
    if (Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq > 1024) return fail(SPEC_EINVAL, "Hq = %d must be a multiple of Hkv = %d, at most 1024", Hq, Hkv);
    if (D != 64 && D != 128) return fail(SPEC_EUNSUPPORTED, "D = %d: only 64 and 128 are built", D);
    if (Lmax < 1 || Lmax > (1 << 22)) return fail(SPEC_EINVAL, "Lmax = %d out of 1..2^22", Lmax);
    if (Ls < 0 || Ls > (1 << 22)) return fail(SPEC_EINVAL, "the shared capacity %d is out of 1..2^22", Ls);
    const int64_t rows = static_cast<int64_t>(B) * Hq * t->T;
    // the line's length at the largest costs
    const int high = dt == SPEC_BF16 ? kTcRows : FR;
    const int64_t blocks = static_cast<int64_t>(Hkv) * ((static_cast<int64_t>(Hq / Hkv) * t->T + high - 1) / high);
    const int64_t tiles = blocks * B * ((Lmax + 63) / 64 + (t->T + 63) / 64 + (Ls + 63) / 64 + 14);
    if (7 * tiles > INT32_MAX / 2)
        return fail(SPEC_EINVAL, "B * Hkv * (Lmax + the shared capacity) is too large for one call (%lld tiles)",
                    static_cast<long long>(tiles));
    if (rows > (1ll << 30)) return fail(SPEC_EINVAL, "B * Hq * T = %lld query rows exceed 2^30", static_cast<long long>(rows));
    return SPEC_OK;
}

// Parts of the line: resident CTAs.  fp32 items of head dim 64 go two to an SM.
static int parts(spec_dtype dt, int D) { return device_sm_count() * (dt == SPEC_F32 && D == 64 ? 2 : 1); }

static Params shapes(const spec_tree* t, int B, int Hq, int Hkv, int Ls, int Lmax, int D) {
    Params p{};
    p.B = B; p.T = t->T; p.Hq = Hq; p.Hkv = Hkv; p.D = D; p.words = t->words;
    p.Lshared = Ls; p.Lmax = Lmax;
    return p;
}

static size_t workspace(const spec_tree* t, int B, int Hq, int Hkv, int Ls, int Lmax, int D, spec_dtype dt) {
    if (check_shapes(t, B, Hq, Hkv, Ls, Lmax, D, dt) != SPEC_OK) return 0;
    Params p = shapes(t, B, Hq, Hkv, Ls, Lmax, D);
    return host_plan(p, dt == SPEC_BF16, Ls > 0, parts(dt, D)).total;
}

template <int D, int R>
static spec_status run_fma(const Params& p, cudaStream_t s) {
    const size_t rows = kFmaThreads / 16 * R, smem = sizeof(float) * (rows * (D + 4) + 4 * FK * (D + 4) + rows * (FK + 4));
    SPEC_CUDA_TRY(cudaFuncSetAttribute(k_attn_shared_fma<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
    SPEC_CUDA_TRY(launch_ex("attn_shared_fma", k_attn_shared_fma<D, R>, dim3(p.ctas), dim3(kFmaThreads), smem, s, true, p));
    return SPEC_OK;
}
template <int D>
static spec_status run_fma(const Params& p, cudaStream_t s) {
    return p.RB == 64 ? run_fma<D, 4>(p, s) : p.RB == 32 ? run_fma<D, 2>(p, s) : run_fma<D, 1>(p, s);
}

template <typename T>
static spec_status join(const Params& p, cudaStream_t s) {
    const int n_rg = (p.gT + 31) / 32;
    int R = 1;   // rows a CTA joins, a power of two
    while (R < 32 && R < p.gT) R *= 2;
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(p.B) * p.Hkv * n_rg));
    SPEC_CUDA_TRY(launch_ex("attn_shared_join", p.D == 64 ? k_attn_shared_join<T, 64> : k_attn_shared_join<T, 128>, grid,
                            dim3(kJoin), 0, s, true, p, n_rg, R));
    return SPEC_OK;
}

// Every entry point: sizes and pointers in p, with p.shared_len set when there is a shared prefix.
static spec_status run(Params p, const spec_tree* tree, spec_dtype dt, float scale, const spec_score* score, size_t ws_bytes,
                       cudaStream_t s) {
    const bool shared = p.shared_len != nullptr;
    spec_status st = check_shapes(tree, p.B, p.Hq, p.Hkv, p.Lshared, p.Lmax, p.D, dt);
    if (st != SPEC_OK) return st;
    if (!p.pg.table && (static_cast<int64_t>(p.B) * p.Hkv * p.Lmax > INT32_MAX || static_cast<int64_t>(p.Hkv) * p.Lshared > INT32_MAX))
        return fail(SPEC_EINVAL, "a cache of B * Hkv * Lmax (or Hkv * Lshared) >= 2^31 rows");
    if (!p.q || !p.kc || !p.vc || !p.prefix_len || !p.kt || !p.vt || !p.out)
        return fail(SPEC_EINVAL, "q, the cache, prefix_len, tree K/V and out must not be NULL");
    if (scale == 0.f) scale = 1.f / sqrtf(static_cast<float>(p.D));   // the usual 1/sqrt(D)
    if (!(scale > 0.f) || !(scale < 1e30f)) return fail(SPEC_EINVAL, "scale must be positive and finite, or 0");
    p.scale = scale;
    if (score) {
        // a capped score is off by some 2^-22 of the cap: beyond 2^12 that would show beside the weights' rounding to bf16
        if (!(score->softcap == 0.f || (score->softcap >= 1e-6f && score->softcap <= 4096.f)))
            return fail(SPEC_EINVAL, "softcap = %g: 1e-6 to 4096, or 0 for none", score->softcap);
        if (score->window < 0) return fail(SPEC_EINVAL, "window = %d must be positive, or 0", score->window);
        p.softcap = score->softcap;
        p.window = std::min(score->window, 1 << 24);   // beyond every distance, and sums with positions stay within 32 bits
        p.slopes = score->slopes;
    }
    if (!aligned16(p.q) || !aligned16(p.kc) || !aligned16(p.vc) || !aligned16(p.ks) || !aligned16(p.vs) || !aligned16(p.kt) ||
        !aligned16(p.vt) || !aligned16(p.out))
        return fail(SPEC_EALIGN, "tensors must be 16-byte aligned");
    if (!aligned4(p.prefix_len) || !aligned4(p.shared_len) || !aligned4(p.slopes) || !aligned4(p.lse) ||
        !aligned4(p.pg.table) || !aligned4(p.shared_table))
        return fail(SPEC_EALIGN, "lengths, tables, slopes and lse must be 4-byte aligned");
    const int64_t es = dt == SPEC_BF16 ? 2 : 4, out_bytes = static_cast<int64_t>(p.B) * p.Hq * p.T * p.D * es;
    auto on_out = [&](const void* x, int64_t bytes) {   // items write out while others still read their rows
        const uintptr_t a = reinterpret_cast<uintptr_t>(p.out), b = reinterpret_cast<uintptr_t>(x);
        return a < b + static_cast<uintptr_t>(bytes) && b < a + static_cast<uintptr_t>(out_bytes);
    };
    const int64_t tree_bytes = static_cast<int64_t>(p.B) * p.Hkv * p.T * p.D * es;
    if (on_out(p.q, out_bytes) || on_out(p.kt, tree_bytes) || on_out(p.vt, tree_bytes))
        return fail(SPEC_EINVAL, "out overlaps q, k_tree or v_tree");
    p.depth = tree->depth;
    p.anc = tree->anc;
    const HostPlan h = host_plan(p, dt == SPEC_BF16, shared, parts(dt, p.D));
    if (!p.ws || ws_bytes < h.total) return fail(SPEC_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, h.total);
    if (!aligned16(p.ws)) return fail(SPEC_EALIGN, "workspace must be 16-byte aligned");
    unsigned char* base = static_cast<unsigned char*>(p.ws);
    p.cta_status = reinterpret_cast<int32_t*>(base + h.status_off);
    p.cum = reinterpret_cast<int32_t*>(base + h.cum_off);
    p.part_s = reinterpret_cast<float4*>(base + h.part_s_off);
    p.part_o = reinterpret_cast<float4*>(base + h.part_o_off);
    if (h.tc) {
        st = attn_shared_tc_run(p, p.ctas, s);
    } else {
        st = p.D == 64 ? run_fma<64>(p, s) : run_fma<128>(p, s);
    }
    if (st != SPEC_OK) return st;
    return dt == SPEC_BF16 ? join<__nv_bfloat16>(p, s) : join<float>(p, s);
}

static spec_status check_pool(int num_blocks, const int32_t* table, int max_blocks, int bs, int Hkv) {
    if (bs < 16 || bs % 16 != 0) return fail(SPEC_EINVAL, "block_size = %d: a positive multiple of 16", bs);
    if (num_blocks < 1 || max_blocks < 1) return fail(SPEC_EINVAL, "num_blocks = %d, max_blocks = %d must be positive", num_blocks, max_blocks);
    if (static_cast<int64_t>(max_blocks) * bs > (1 << 22))
        return fail(SPEC_EINVAL, "max_blocks * block_size = %lld > 2^22", static_cast<long long>(max_blocks) * bs);
    if (static_cast<int64_t>(num_blocks) * std::max(Hkv, 1) * bs > INT32_MAX)
        return fail(SPEC_EINVAL, "pool of %d blocks too large (num_blocks * Hkv * block_size rows >= 2^31)", num_blocks);
    if (!table) return fail(SPEC_EINVAL, "a block table must not be NULL");
    return SPEC_OK;
}

}  // namespace shr
}  // namespace spec

using namespace spec;

extern "C" size_t tree_attention_shared_workspace_size(const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv,
                                                       int32_t Lshared, int32_t Lmax, int32_t D, spec_dtype dt) {
    clear_error();
    if (Lshared < 1) {
        fail(SPEC_EINVAL, "Lshared = %d must be positive", Lshared);
        return 0;
    }
    return shr::workspace(tree, B, Hq, Hkv, Lshared, Lmax, D, dt);
}

extern "C" size_t tree_attention_scored_workspace_size(const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv,
                                                       int32_t Lmax, int32_t D, spec_dtype dt) {
    clear_error();
    return shr::workspace(tree, B, Hq, Hkv, 0, Lmax, D, dt);
}

extern "C" spec_status tree_attention_shared(const void* q, const void* k_shared, const void* v_shared,
                                             const int32_t* shared_len, int32_t Lshared, const void* k_cache,
                                             const void* v_cache, const int32_t* prefix_len, const void* k_tree,
                                             const void* v_tree, const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv,
                                             int32_t Lmax, int32_t D, float scale, const spec_score* score, spec_dtype dt,
                                             void* out, float* lse, void* ws, size_t ws_bytes, spec_stream_t s) {
    clear_error();
    spec_status st = check_tree(tree);
    if (st != SPEC_OK) return st;
    if (!k_shared || !v_shared || !shared_len) return fail(SPEC_EINVAL, "the shared keys, values and length must not be NULL");
    if (Lshared < 1) return fail(SPEC_EINVAL, "Lshared = %d must be positive", Lshared);
    shr::Params p = shr::shapes(tree, B, Hq, Hkv, Lshared, Lmax, D);
    p.q = q; p.ks = k_shared; p.vs = v_shared; p.kc = k_cache; p.vc = v_cache; p.kt = k_tree; p.vt = v_tree;
    p.shared_len = shared_len; p.prefix_len = prefix_len;
    p.out = out; p.lse = lse; p.ws = ws;
    return shr::run(p, tree, dt, scale, score, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}

extern "C" spec_status tree_attention_shared_paged(const void* q, const void* k_pool, const void* v_pool, int32_t num_blocks,
                                                   const int32_t* shared_table, int32_t shared_blocks,
                                                   const int32_t* shared_len, const int32_t* block_table,
                                                   int32_t max_blocks, int32_t block_size, const int32_t* prefix_len,
                                                   const void* k_tree, const void* v_tree, const spec_tree* tree, int32_t B,
                                                   int32_t Hq, int32_t Hkv, int32_t D, float scale, const spec_score* score,
                                                   spec_dtype dt, void* out, float* lse, void* ws, size_t ws_bytes,
                                                   spec_stream_t s) {
    clear_error();
    spec_status st = check_tree(tree);
    if (st != SPEC_OK) return st;
    st = shr::check_pool(num_blocks, block_table, max_blocks, block_size, Hkv);
    if (st != SPEC_OK) return st;
    st = shr::check_pool(num_blocks, shared_table, shared_blocks, block_size, Hkv);
    if (st != SPEC_OK) return st;
    if (!shared_len) return fail(SPEC_EINVAL, "shared_len must not be NULL");
    shr::Params p = shr::shapes(tree, B, Hq, Hkv, shared_blocks * block_size, max_blocks * block_size, D);
    p.q = q; p.kc = k_pool; p.vc = v_pool; p.kt = k_tree; p.vt = v_tree;
    p.pg.table = block_table; p.pg.max_blocks = max_blocks; p.pg.bs = block_size; p.pg.num_blocks = num_blocks;
    p.shared_table = shared_table;
    p.shared_len = shared_len; p.prefix_len = prefix_len;
    p.out = out; p.lse = lse; p.ws = ws;
    return shr::run(p, tree, dt, scale, score, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}

extern "C" spec_status tree_attention_scored(const void* q, const void* k_cache, const void* v_cache,
                                             const int32_t* prefix_len, const void* k_tree, const void* v_tree,
                                             const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv, int32_t Lmax,
                                             int32_t D, float scale, const spec_score* score, spec_dtype dt, void* out,
                                             float* lse, void* ws, size_t ws_bytes, spec_stream_t s) {
    clear_error();
    spec_status st = check_tree(tree);
    if (st != SPEC_OK) return st;
    shr::Params p = shr::shapes(tree, B, Hq, Hkv, 0, Lmax, D);
    p.q = q; p.kc = k_cache; p.vc = v_cache; p.kt = k_tree; p.vt = v_tree; p.prefix_len = prefix_len;
    p.out = out; p.lse = lse; p.ws = ws;
    return shr::run(p, tree, dt, scale, score, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}

extern "C" spec_status tree_attention_scored_paged(const void* q, const void* k_pool, const void* v_pool, int32_t num_blocks,
                                                   const int32_t* block_table, int32_t max_blocks, int32_t block_size,
                                                   const int32_t* prefix_len, const void* k_tree, const void* v_tree,
                                                   const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                                   float scale, const spec_score* score, spec_dtype dt, void* out,
                                                   float* lse, void* ws, size_t ws_bytes, spec_stream_t s) {
    clear_error();
    spec_status st = check_tree(tree);
    if (st != SPEC_OK) return st;
    st = shr::check_pool(num_blocks, block_table, max_blocks, block_size, Hkv);
    if (st != SPEC_OK) return st;
    shr::Params p = shr::shapes(tree, B, Hq, Hkv, 0, max_blocks * block_size, D);
    p.q = q; p.kc = k_pool; p.vc = v_pool; p.kt = k_tree; p.vt = v_tree; p.prefix_len = prefix_len;
    p.pg.table = block_table; p.pg.max_blocks = max_blocks; p.pg.bs = block_size; p.pg.num_blocks = num_blocks;
    p.out = out; p.lse = lse; p.ws = ws;
    return shr::run(p, tree, dt, scale, score, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}
