// Tensor-core (tcgen05) items of the shared-prefix and scored tree attention:
// bf16, head dim 64 or 128.
//
// One persistent CTA per SM takes items blockIdx.x, blockIdx.x + gridDim.x, ...
// of the cut that attention_shared.cuh describes: 128 query rows against a range
// of 128-key tiles.  Eleven warps, all of which walk the same items:
//   warp 8       TMA: the item's Q block, then its K and V tiles into a ring that
//                runs on across items
//   warps 9, 10  MMA, one thread each: thread g takes the tiles whose running
//                number J (over all items of the CTA) has J % 2 == g -- S_J = Q K_J^T
//                into score buffer g, O_g += P_J V_J with P_J read from TMEM
//   warps 0-3 / 4-7: two softmax groups, group J % 2 for tile J, one thread per
//                query row: S from TMEM, score transform and masks, running maximum
//                and sum in base 2 and 32 bits, P back as bf16 pairs over the first
//                half of the score buffer.  P is rounded to bf16 because the product
//                takes both operands in one type and V is bf16; the sum l is taken
//                before the rounding.  At the end of an item the groups exchange
//                (m, l) and each merges one half of the columns of both O.
// A thread's MMAs run in issue order, so S_{J+2} may overwrite the buffer PV_J
// reads, and S_J complete implies PV_{J-2} complete.  Barriers whose phases both
// MMA threads pass: q_empty (each commits after its last S of the item), o_final
// (after its last PV); o_empty lets the next item's first PV overwrite O once
// every softmax warp has read it.
// V rows that no row sees (past the lengths, past the tree) are zeroed before PV
// reads them: their weight is zero, but zero times a stale infinity is not.
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

constexpr int kRows = 128;       // query rows of a block (MMA M)
constexpr int kKeys = 128;       // keys of a tile
constexpr int kThreads = 352;
constexpr int kHalf = 128 * 128; // bytes of 128 rows x 64 columns

template <int D> struct Cfg {
    static constexpr int kH = D / 64;                      // 64-column halves
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kFull = 2 * kStages;              // landing barriers: each belongs to one MMA thread
    static constexpr int kQ = kH * kHalf;
    static constexpr int kStage = 2 * kH * kHalf;          // K, then V
    static constexpr int kTail = 256 + 2 * kRows * 8;      // barriers, exchange of (m, l)
    static constexpr int kSmem = kQ + kStages * kStage + kTail;
};
constexpr uint32_t kTmemCols = 512;   // S0 [0,128) S1 [128,256) O0 [256, 256 + D) O1 behind it
constexpr uint32_t kO = 2 * kKeys;

struct Maps {
    CUtensorMap q_own, q_shared, kc, vc, ks, vs, kt, vt;
};

// Bounded wait of a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, mbar_wait_or_abort(bar, parity, abort_flag));
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int D, bool kScored>
__global__ void __launch_bounds__(kThreads, 1) k_attn_shared_tc(const __grid_constant__ Maps mp, const Params p, const int page_rows) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((smem_u32(smem) & 1023u) != 0) {   // the swizzle counts address bits: a base elsewhere would scramble tiles
        if (threadIdx.x == 0) flag_status(p.ws, SPEC_EUNSUPPORTED);
        if (blockIdx.x == 0) {             // nothing to join
            for (int b = threadIdx.x; b <= p.B; b += kThreads) p.cum[b] = 0;
            if (threadIdx.x == 0) *reinterpret_cast<Plan*>(static_cast<unsigned char*>(p.ws) + kPlanOffset) = Plan{};
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
    uint64_t* s_full = bars + 5;                  // [group]
    uint64_t* p_full = bars + 7;                  // [group]
    uint64_t* ml_full = bars + 9;                 // [group]
    uint64_t* kv_full = bars + 11;                // [J % kFull]
    uint64_t* kv_empty = kv_full + C::kFull;      // [stage]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kv_empty + C::kStages);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((11 + C::kFull + C::kStages) * 8 + 8 <= 256, "barriers and flags end before the exchange");
    float2* ml = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(bars) + 256);   // [group][row]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 2);
        mbar_init(o_final, 2);
        mbar_init(o_empty, 8);
        mbar_init(drain, 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&ml_full[i], 4);
        }
        for (int i = 0; i < C::kFull; ++i) mbar_init(&kv_full[i], 1);
        for (int i = 0; i < C::kStages; ++i) mbar_init(&kv_empty[i], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(tmem_slot, kTmemCols);
    const Plan plan = make_plan(p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_launch();   // the join may start launching: it waits for the partials
    if (blockIdx.x == 0 && warp == 7) publish_plan(p, plan);

    const int tree_tiles = ceil_div(p.T, kKeys);
    int J = 0;          // running tile number, the same in every role
    int n = 0;          // running item number
    bool ok = true;
    int q_loads = 0;    // (TMA) items whose Q was requested

    if (warp == 8) {
        const uint32_t q_bytes_own = static_cast<uint32_t>(p.rowsO) * 128 * C::kH;
        const uint32_t q_bytes_shared = static_cast<uint32_t>(p.rowsS) * 128 * C::kH;
        const int tree_rows = min(p.T, kKeys);
        for (int id = blockIdx.x; ok && id < plan.items; id += gridDim.x, ++n) {
            const Item it = find_item(p, plan, id);
            const int first = it.shared ? plan.sT0 : own_first(p, it.L);
            const int n_pre = it.shared ? plan.nS : own_tiles(p, it.L) - tree_tiles;
            const int end = it.shared ? plan.Ls : it.L;
            // Q once the last item's scores are done; from the second item on behind its first
            // tile, whose stage frees without this item's Q
            auto load_q = [&]() -> bool {
                if (n > 0 && !warp_wait(q_empty, (n - 1) & 1, abort_flag)) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, it.shared ? q_bytes_shared : q_bytes_own);
                    for (int h = 0; h < C::kH; ++h)
                        tma_load_4d(sQ + h * kHalf, it.shared ? &mp.q_shared : &mp.q_own, q_full, 64 * h, it.rb * kRows, it.kvh, it.b);
                }
                q_loads = n + 1;
                return true;
            };
            if (n == 0) load_q();
            for (int t = it.t0; t < it.t1; ++t, ++J) {
                const int s = J % C::kStages;
                uint8_t* st = sKV + s * C::kStage;
                uint64_t* bar = &kv_full[J % C::kFull];
                const bool tree = !it.shared && t >= n_pre;
                const int k0 = (tree ? t - n_pre : first + t) * kKeys;
                // the lane's pool block, looked up while the stage is still in use
                const bool paged = !tree && p.pg.table;
                const int pieces = paged ? min(kKeys / page_rows, (end - k0 + page_rows - 1) / page_rows) : 0;
                const int piece = lane >> 1;
                int row = 0;
                if (piece < pieces) {
                    const int pos = k0 + piece * page_rows;
                    int blk = it.shared ? p.shared_table[pos / p.pg.bs]
                                        : p.pg.table[static_cast<size_t>(it.b) * p.pg.max_blocks + pos / p.pg.bs];
                    if (blk < 0 || blk >= p.pg.num_blocks) {
                        flag_status(p.ws, SPEC_EINVAL);
                        blk = 0;
                    }
                    row = (blk * p.Hkv + it.kvh) * p.pg.bs + pos % p.pg.bs;
                }
                if (J >= C::kStages && !(ok = warp_wait(&kv_empty[s], ((J / C::kStages) - 1) & 1, abort_flag))) break;
                const int rows = paged ? pieces * page_rows : tree ? tree_rows : kKeys;
                if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(rows) * 128 * C::kH * 2);
                __syncwarp();
                if (paged) {
                    // lane = 2 piece + (K or V)
                    if (piece < pieces) {
                        uint8_t* dst = st + (lane & 1) * (C::kStage / 2) + piece * page_rows * 128;
                        for (int h = 0; h < C::kH; ++h)
                            tma_load_2d(dst + h * kHalf, lane & 1 ? &mp.vc : &mp.kc, bar, 64 * h, row);
                    }
                } else if (lane < 2 * C::kH) {
                    // lane = (K or V) * kH + half
                    const int v = lane / C::kH, h = lane % C::kH;
                    const CUtensorMap* m = tree ? (v ? &mp.vt : &mp.kt) : it.shared ? (v ? &mp.vs : &mp.ks) : (v ? &mp.vc : &mp.kc);
                    const int r0 = tree ? (it.b * p.Hkv + it.kvh) * p.T : it.shared ? it.kvh * p.Lshared : (it.b * p.Hkv + it.kvh) * p.Lmax;
                    tma_load_2d(st + v * (C::kStage / 2) + h * kHalf, m, bar, 64 * h, r0 + k0);
                }
                if (n > 0 && t == it.t0 && !(ok = load_q())) {
                    ++J;
                    break;
                }
            }
        }
    } else if (warp == 9 || warp == 10) {
        const int g = warp - 9;
        const uint32_t idesc_s = idesc_bf16_f32(kRows, kKeys);
        const uint32_t idesc_o = idesc_bf16_f32_bmn(kRows, D);
        const uint64_t qd = sdesc_k128(smem_u32(sQ));
        const uint32_t sb = tmem + g * kKeys;             // this thread's score buffer
        const uint32_t ob = tmem + kO + g * D;            // and its O
        uint32_t p_phase = 0;
        for (int id = blockIdx.x; ok && id < plan.items; id += gridDim.x, ++n) {
            const Item it = find_item(p, plan, id);
            const int first = it.shared ? plan.sT0 : own_first(p, it.L);
            const int n_pre = it.shared ? plan.nS : own_tiles(p, it.L) - tree_tiles;
            const int end = it.shared ? plan.Ls : it.L;
            const int tiles = it.t1 - it.t0;
            if (lane == 0) {
                auto issue_s = [&](int j) -> bool {       // tile j of the item
                    const int jj = J + j;
                    if (!mbar_wait_or_abort(&kv_full[jj % C::kFull], (jj / C::kFull) & 1, abort_flag)) return false;
                    tc_fence_after();
                    const uint64_t kd = sdesc_k128(smem_u32(sKV + (jj % C::kStages) * C::kStage));
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = (k >> 2) * kHalf + (k & 3) * 32;
                        mma_bf16(sb, qd + (off >> 4), kd + (off >> 4), idesc_s, k > 0 ? 1u : 0u);
                    }
                    mma_commit(&s_full[g]);
                    return true;
                };
                int j = (J & 1) == g ? 0 : 1;             // this thread's first tile
                ok = mbar_wait_or_abort(q_full, n & 1, abort_flag);
                if (ok && j < tiles) ok = issue_s(j);
                bool q_done = false, o_clear = n == 0;
                if (ok && j + 2 >= tiles) {               // no further S: the Q block may go
                    mma_commit(q_empty);
                    q_done = true;
                }
                for (bool first_pv = true; ok && j < tiles; j += 2, first_pv = false) {
                    const int jj = J + j, t = it.t0 + j;
                    if (!(ok = mbar_wait_or_abort(&p_full[g], p_phase, abort_flag))) break;
                    p_phase ^= 1u;
                    if (!o_clear) {
                        if (!(ok = mbar_wait_or_abort(o_empty, (n - 1) & 1, abort_flag))) break;
                        o_clear = true;
                    }
                    tc_fence_after();
                    // keys of the tile that any row can see: whole steps of 16
                    const bool tree = !it.shared && t >= n_pre;
                    const int nvalid = tree ? min(kKeys, p.T - (t - n_pre) * kKeys) : min(kKeys, end - (first + t) * kKeys);
                    const int steps = (nvalid + 15) / 16;
                    const uint64_t vd = sdesc_mn128(smem_u32(sKV + (jj % C::kStages) * C::kStage + C::kStage / 2), kHalf, 1024);
                    if (steps == kKeys / 16) {
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)
                            mma_bf16_ts(ob, sb + k * 8, vd + ((k * 2048) >> 4), idesc_o, (first_pv && k == 0) ? 0u : 1u);
                    } else {
                        for (int k = 0; k < steps; ++k)
                            mma_bf16_ts(ob, sb + k * 8, vd + ((k * 2048) >> 4), idesc_o, (first_pv && k == 0) ? 0u : 1u);
                    }
                    mma_commit(&kv_empty[jj % C::kStages]);
                    if (j + 2 < tiles && !(ok = issue_s(j + 2))) break;
                    if (!q_done && j + 4 >= tiles) {
                        mma_commit(q_empty);
                        q_done = true;
                    }
                }
                if (ok) mma_commit(o_final);
            }
            J += tiles;
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
        if (lane == 0) mma_commit(drain);
        __syncwarp();
    } else {
        const int grp = warp >> 2;
        const int r = (warp & 3) * 32 + lane;              // row of the block = TMEM lane
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_col = grp * kKeys, o_col = kO + grp * D;
        const float scale2 = p.scale * kLog2e;
        const bool transformed = kScored && (p.softcap > 0.f || p.slopes);
        const float cap2 = p.softcap * kLog2e, capin = p.softcap > 0.f ? 2.f * kLog2e * p.scale / p.softcap : 0.f;
        const float in_scale = transformed ? 1.f : scale2;   // what the exponent's FFMA still multiplies by
        uint32_t s_phase = 0;
        for (int id = blockIdx.x; ok && id < plan.items; id += gridDim.x, ++n) {
            const Item it = find_item(p, plan, id);
            const int first = it.shared ? plan.sT0 : own_first(p, it.L);
            const int n_pre = it.shared ? plan.nS : own_tiles(p, it.L) - tree_tiles;
            const int end = it.shared ? plan.Ls : it.L;
            const int tiles = it.t1 - it.t0;
            // the row: its place in gT, node, position, slope (rows past the block repeat its last)
            const bool warp_in = (warp & 3) * 32 < it.rows;
            const bool in = r < it.rows;
            const int rr = min(r, it.rows - 1);
            const int ib = p.gT < kRows ? rr / p.gT : 0;
            const int i = p.gT < kRows ? rr - ib * p.gT : it.rb * kRows + rr;
            const int head = i / p.T, node = i - head * p.T;
            int pos = 0;
            float slope2 = 0.f;
            if (kScored) {
                pos = plan.Ls + own_len(p, it.b + ib) + p.depth[node];
                if (p.slopes) slope2 = p.slopes[it.kvh * p.g + head] * kLog2e;
            }
            const uint64_t* anc_row = p.anc + static_cast<size_t>(node) * p.words;
            float m_used = -INFINITY, l = 0.f;
            for (int j = (J & 1) == grp ? 0 : 1; j < tiles; j += 2) {
                const int t = it.t0 + j;
                const bool tree = !it.shared && t >= n_pre;
                const int k0 = (tree ? t - n_pre : first + t) * kKeys;
                const int nvalid = min(kKeys, (tree ? p.T : end) - k0);
                if (!(ok = warp_wait(&s_full[grp], s_phase, abort_flag))) break;
                s_phase ^= 1u;
                tc_fence_after();
                if (warp_in) {
                    float sv[kKeys];
                    {
                        uint32_t s0[32], s1[32], s2[32], s3[32];
                        tmem_ld32(lane_base + s_col, s0);
                        tmem_ld32(lane_base + s_col + 32, s1);
                        tmem_ld32(lane_base + s_col + 64, s2);
                        tmem_ld32(lane_base + s_col + 96, s3);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            sv[e] = __uint_as_float(s0[e]);
                            sv[e + 32] = __uint_as_float(s1[e]);
                            sv[e + 64] = __uint_as_float(s2[e]);
                            sv[e + 96] = __uint_as_float(s3[e]);
                        }
                    }
                    const int kbase = it.shared ? k0 : plan.Ls + k0;   // position of the tile's first key (not the tree's)
                    if (kScored) {
                        if (p.softcap > 0.f) {
                            // cap tanh(x / cap) = cap (1 - 2 / (2^(2 log2e x / cap) + 1))
#pragma unroll
                            for (int e = 0; e < kKeys; ++e) sv[e] = fmaf(-2.f * cap2, rcp(ex2(sv[e] * capin) + 1.f), cap2);
                        } else if (p.slopes) {
#pragma unroll
                            for (int e = 0; e < kKeys; ++e) sv[e] *= scale2;
                        }
                        if (p.slopes) {
                            if (tree) {
                                const int lp = pos - plan.Ls - it.L;   // the node's depth
#pragma unroll
                                for (int e = 0; e < kKeys; ++e)
                                    if (e < nvalid) sv[e] -= slope2 * static_cast<float>(lp - p.depth[k0 + e]);
                            } else {
                                const float b0 = slope2 * static_cast<float>(kbase - pos);
#pragma unroll
                                for (int e = 0; e < kKeys; ++e) sv[e] += fmaf(slope2, static_cast<float>(e), b0);
                            }
                        }
                    }
                    // masks: whole tiles without one take the short way
                    const int lo = kScored && p.window > 0 && !tree ? pos - p.window + 1 - kbase : 0;   // first key seen
                    const bool windowed = kScored && p.window > 0 && (tree ? p.window <= SPEC_MAX_DEPTH : lo > 0);
                    if (tree || nvalid < kKeys || __any_sync(0xffffffffu, windowed)) {
                        uint64_t bits[2];
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const int nv = min(max(nvalid - 64 * w, 0), 64);
                            bits[w] = nv >= 64 ? ~0ull : ((1ull << nv) - 1ull);
                            if (kScored && !tree) {
                                const int nl = min(max(lo - 64 * w, 0), 64);
                                bits[w] &= nl >= 64 ? 0ull : ~0ull << nl;
                            }
                        }
                        if (tree) {   // only the node's ancestors and itself
                            const int w0 = k0 >> 6;
                            bits[0] &= anc_row[w0];
                            bits[1] &= w0 + 1 < p.words ? anc_row[w0 + 1] : 0ull;
                            if (windowed) {
                                const int lp = pos - plan.Ls - it.L;
#pragma unroll
                                for (int w = 0; w < 2; ++w)
                                    for (uint64_t left = bits[w]; left; left &= left - 1) {
                                        const int e = __ffsll(static_cast<long long>(left)) - 1;
                                        if (lp - p.depth[k0 + 64 * w + e] >= p.window) bits[w] &= ~(1ull << e);
                                    }
                            }
                        }
#pragma unroll
                        for (int e = 0; e < kKeys; ++e)
                            if (!((bits[e >> 6] >> (e & 63)) & 1ull)) sv[e] = -INFINITY;
                    }
                    float mx[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        mx[e] = fmax3(fmax3(sv[e], sv[e + 16], sv[e + 32]), fmax3(sv[e + 48], sv[e + 64], sv[e + 80]),
                                      fmax3(sv[e + 96], sv[e + 112], -INFINITY));
                    mx[0] = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmax3(mx[6], mx[7], mx[8]));
                    mx[0] = fmax3(fmax3(mx[0], mx[9], mx[10]), fmax3(mx[11], mx[12], mx[13]), fmaxf(mx[14], mx[15]));
                    const float tmax = mx[0] * in_scale;
                    // the reference maximum moves only when the row's grew by more than 2^8; the TMEM
                    // accesses are the whole warp's, so its rows rescale together (by 1 where nothing grew)
                    float m_new = m_used, alpha = 1.f;
                    bool rescale = false;
                    if (tmax > m_used + 8.f) {
                        if (m_used != -INFINITY) {
                            rescale = true;
                            alpha = ex2(m_used - tmax);
                        }
                        m_new = tmax;
                    }
                    if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(lane_base + o_col + c * 16, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st16(lane_base + o_col + c * 16, o);
                        }
                        l *= alpha;
                    }
                    m_used = m_new;
                    const float nmref = m_used == -INFINITY ? 0.f : -m_used;
                    const unsigned long long sc2 = pk2(in_scale, in_scale), nm2 = pk2(nmref, nmref);
                    float ps[4];
#pragma unroll
                    for (int qc = 0; qc < 4; ++qc) {
                        uint32_t packed[16];
                        unsigned long long acc2 = pk2(0.f, 0.f);
#pragma unroll
                        for (int h2 = 0; h2 < 16; ++h2) {
                            const int e0 = qc * 32 + 2 * h2;
                            float x0, x1;
                            upk2(ffma2(pk2(sv[e0], sv[e0 + 1]), sc2, nm2), x0, x1);
                            const float a0 = ex2(x0), a1 = ex2(x1);
                            acc2 = fadd2(acc2, pk2(a0, a1));
                            const __nv_bfloat162 pr = __floats2bfloat162_rn(a0, a1);   // .x (lower key) low
                            packed[h2] = *reinterpret_cast<const uint32_t*>(&pr);
                        }
                        float acc0, acc1;
                        upk2(acc2, acc0, acc1);
                        ps[qc] = acc0 + acc1;
                        tmem_st16(lane_base + s_col + qc * 16, packed);
                    }
                    l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
                }
                if (nvalid & 15) {
                    // zero V from the last key to the end of its step of 16 (S_J complete: V_J has landed)
                    uint8_t* sv_tile = sKV + ((J + j) % C::kStages) * C::kStage + C::kStage / 2;
                    const int pad = 16 - (nvalid & 15);
                    for (int x = (warp & 3) * 32 + lane; x < pad * 8 * C::kH; x += kRows) {
                        const int row = nvalid + x / (8 * C::kH), c = x % (8 * C::kH);
                        *reinterpret_cast<uint4*>(sv_tile + (c >> 3) * kHalf + row * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[grp]);
            }
            if (!ok) break;
            // the item's end: (m, l) across the groups, then each group joins half the columns
            if (!(ok = warp_wait(o_final, n & 1, abort_flag))) break;
            tc_fence_after();
            ml[grp * kRows + r] = make_float2(m_used, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(&ml_full[grp]);
            if (!(ok = warp_wait(&ml_full[grp ^ 1], n & 1, abort_flag))) break;
            if (warp_in) {
                const float2 other = ml[(grp ^ 1) * kRows + r];
                const float m = fmaxf(m_used, other.x);
                const float ref = m == -INFINITY ? 0.f : m;
                const float mine = ex2(m_used - ref), theirs = ex2(other.x - ref);
                const float a0 = grp == 0 ? mine : theirs, a1 = grp == 0 ? theirs : mine;
                const float lsum = mine * l + theirs * other.y;
                const bool has0 = tiles > 1 || (J & 1) == 0, has1 = tiles > 1 || (J & 1) == 1;   // a group without a tile left O as it was
                const int stride = it.shared ? p.rowsS : p.rowsO;
                float4* part = (it.shared ? p.part_s : p.part_o) + static_cast<size_t>(it.index) * (D / 4 + 1) * stride;
                const float inv = it.direct ? 1.f / lsum : 1.f;
                const size_t row = row_of_q(p, it, rr);
                if (in && grp == 0) {
                    if (!it.direct) part[r] = make_float4(m, lsum, 0.f, 0.f);
                    else if (p.lse) p.lse[row] = (m + log2f(lsum)) * kLn2;
                }
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const int c0 = grp * (D / 2) + c * 32;
                    uint32_t o0[32], o1[32];
                    tmem_ld32(lane_base + kO + c0, o0);
                    tmem_ld32(lane_base + kO + D + c0, o1);
                    tmem_ld_wait();
                    float v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float x0 = has0 ? a0 * __uint_as_float(o0[e]) : 0.f;
                        v[e] = (has1 ? fmaf(a1, __uint_as_float(o1[e]), x0) : x0) * inv;
                    }
                    if (in && !it.direct) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            part[static_cast<size_t>(1 + c0 / 4 + e) * stride + r] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    } else if (in) {
                        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + row * D + c0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t w[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * e + 2 * q], v[8 * e + 2 * q + 1]);
                                w[q] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                            *reinterpret_cast<uint4*>(dst + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_empty);
            J += tiles;
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
        if (warp == 8) {
            for (int j = max(0, J - C::kFull); j < J; ++j) mbar_wait(&kv_full[j % C::kFull], (j / C::kFull) & 1, 100000000ull);
            if (q_loads > 0) mbar_wait(q_full, (q_loads - 1) & 1, 100000000ull);
        }
        if ((warp == 9 || warp == 10) && lane == 0) mbar_wait(drain, 0, 100000000ull);
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- host

template <int D, bool kScored>
static spec_status launch_items(const Maps& m, const Params& p, int page_rows, int blocks, cudaStream_t s) {
    auto kern = k_attn_shared_tc<D, kScored>;
    SPEC_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem));
    SPEC_CUDA_TRY(launch("attn_shared_tc", kern, dim3(blocks), dim3(kThreads), Cfg<D>::kSmem, s, m, p, page_rows));
    return SPEC_OK;
}

spec_status attn_shared_tc_run(const Params& p, int blocks, cudaStream_t s) {
    Maps m;
    memset(&m, 0, sizeof(m));
    const uint64_t B = p.B, Hkv = p.Hkv, T = p.T, D = p.D;
    const uint32_t b1 = static_cast<uint32_t>(std::min(p.gT, kRows));
    SPEC_CUDA_TRY(make_tmap_bf16_4d(&m.q_own, p.q, B, Hkv, p.gT, D, 1, b1));
    SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.kt, p.kt, B * Hkv * T, D, D, static_cast<uint32_t>(std::min(p.T, kKeys))));
    SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.vt, p.vt, B * Hkv * T, D, D, static_cast<uint32_t>(std::min(p.T, kKeys))));
    int page_rows = 0;
    if (p.pg.table) {
        // a box lies inside one block and one tile: the largest power of two that divides both
        page_rows = 16;
        while (page_rows < kKeys && p.pg.bs % (2 * page_rows) == 0) page_rows *= 2;
        const uint64_t rows = static_cast<uint64_t>(p.pg.num_blocks) * Hkv * p.pg.bs;
        SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.kc, p.kc, rows, D, D, page_rows));
        SPEC_CUDA_TRY(make_tmap_bf16_2d(&m.vc, p.vc, rows, D, D, page_rows));
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
        return scored ? launch_items<64, true>(m, p, page_rows, blocks, s) : launch_items<64, false>(m, p, page_rows, blocks, s);
    return scored ? launch_items<128, true>(m, p, page_rows, blocks, s) : launch_items<128, false>(m, p, page_rows, blocks, s);
}

}  // namespace shr
}  // namespace spec
