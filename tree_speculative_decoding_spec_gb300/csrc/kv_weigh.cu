// The attention weight that cached keys receive.
//
//   acc[b, h, j] = decay * acc[b, h, j] + sum over rows r of h's query heads of exp(scale q_r . k_j - lse_r)
//
// for the keys that row r sees: with count rows, row i of a query head sees the keys up to
// n - count + i, n the cache's length with the rows' own keys in it.  The rows are the last
// ones of the sequence: generated tokens, the nodes of an accepted path, a prompt.
// lse comes from the attention that the rows went through, so the probabilities are made again
// from one product and one exponential each, and only keys are read.
//
// Here: the checks, the CUDA-core kernel (fp32) and the entry points.  bf16 goes to the
// tensor cores (kv_weigh_tc.cu).
#include <algorithm>

#include "kv_weigh.cuh"

namespace spec {
namespace weigh {

constexpr int kThreads = 256;
constexpr int kKeys = 64;             // keys of a CTA
constexpr int kGroups = 16;           // 16 groups of four keys by 16 groups of rows
constexpr float kLog2e = 1.4426950408889634f;

// CTAs per 64 keys of one (sequence, KV head), over the rows that see any of them, 16 RPT at a time; where there
// are few such tiles their chunks of rows go to several CTAs in turn, whose sums kv_weigh_parts adds up in order
// (a prompt of 100 rows and 8 heads of 64: 33 us with one, 11 with splits).  A thread has four keys and RPT rows; operands
// lie in shared memory by head dimension, so that four keys come in one read.  CTA 0 of the first head
// writes the status.
//
// Operands are [D][N] with groups of four rows exchanged by the head dimension: a warp reads 128 bytes of each of four rows,
// and its 32 four-element columns meet in no bank; reads of a group of four rows of one element stay whole.  (A row a lane: as many
// lines as lanes for each load; 33 sequences of 512 keys and 42 rows took 51 us where this takes 35.)
template <int N> __device__ __forceinline__ int place(int d, int r) {
    return d * N + ((((r >> 2) ^ ((d >> 2) & (N == 16 ? 3 : 7))) << 2) | (r & 3));
}
template <int D, int N> __device__ __forceinline__ void load_rows(float* s, const float* x, const int64_t* rows) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kEach = (N / 4) * (D / 32) / (kThreads / 32);
    static_assert(kEach * (kThreads / 32) == (N / 4) * (D / 32), "whole rounds of the warps");
    float v[kEach][4] = {};           // all on their way together
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int t = i * (kThreads / 32) + warp;
        const int64_t at = rows[t % (N / 4) * 4 + lane / 8];
        if (at >= 0) load4(x + at * D + (t / (N / 4) * 8 + lane % 8) * 4, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int t = i * (kThreads / 32) + warp;
#pragma unroll
        for (int j = 0; j < 4; ++j) s[place<N>((t / (N / 4) * 8 + lane % 8) * 4 + j, t % (N / 4) * 4 + lane / 8)] = v[i][j];
    }
}

template <int D, int RPT>
__global__ void __launch_bounds__(kThreads) k_weigh_fma(const Params p, int splits, float* parts) {
    constexpr int R = kGroups * RPT;
    extern __shared__ __align__(16) float smem[];
    float* ks = smem;                 // [D][kKeys]
    float* qs = smem + D * kKeys;     // [D][R]
    __shared__ float s_lse[R];
    __shared__ int s_last[R];         // the last key that a row sees; -1: no row
    __shared__ int64_t s_key[kKeys], s_row[R];   // where the keys and rows lie, -1: nowhere
    const int h = blockIdx.y, b = blockIdx.z;
    griddep_wait();                   // the stream's kernel before this one may still run: its results are behind here
    griddep_launch();
    if (blockIdx.x == 0) {
        if (h == 0 && b == 0) check_all<kThreads>(p);
        return;
    }
    const Rows rows = rows_of(p, b);
    const int split = (static_cast<int>(blockIdx.x) - 1) % splits, k0 = (static_cast<int>(blockIdx.x) - 1) / splits * kKeys;
    if (!rows.ok || k0 >= rows.n) return;
    const float* q = static_cast<const float*>(p.q);
    const float* k = static_cast<const float*>(p.k);
    if (threadIdx.x < kKeys) s_key[threadIdx.x] = k0 + static_cast<int>(threadIdx.x) < rows.n ? key_row(p, b, h, k0 + threadIdx.x) : -1;
    __syncthreads();
    load_rows<D, kKeys>(ks, k, s_key);
    const int kg = threadIdx.x % kGroups, rg = threadIdx.x / kGroups;
    const int g = p.Hq / p.Hkv;
    const int i0 = max(0, k0 - (rows.n - rows.count));   // the first row that sees a key of this tile
    const int per = rows.count - i0, total = g * per;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r0 = split * R; r0 < total; r0 += splits * R) {
        __syncthreads();
        if (threadIdx.x < R) {
            const int r = r0 + threadIdx.x;
            s_last[threadIdx.x] = -1;
            s_row[threadIdx.x] = -1;
            if (r < total) {
                const int head = r / per, i = i0 + r - head * per;
                const int64_t at = static_cast<int64_t>(b * p.Hq + h * g + head) * p.T + node_of(p, b, i);
                const float l = p.lse[at];
                s_row[threadIdx.x] = at;
                s_lse[threadIdx.x] = l;
                if (isfinite(l)) s_last[threadIdx.x] = rows.n - rows.count + i;
            }
        }
        __syncthreads();
        load_rows<D, R>(qs, q, s_row);
        __syncthreads();
        // (a warp without rows: 64 sequences' heads of 4000 keys and 8 rows take 68 us so, 103 else)
        if (r0 + (rg & ~1) * RPT >= total) continue;
        float s[4][RPT] = {};
#pragma unroll 8
        for (int d = 0; d < D; ++d) {
            const float4 kk = *reinterpret_cast<const float4*>(&ks[place<kKeys>(d, 4 * kg)]);
            float qq[RPT];
            if constexpr (RPT == 4) {
                const float4 t = *reinterpret_cast<const float4*>(&qs[place<R>(d, 4 * rg)]);
                qq[0] = t.x; qq[1] = t.y; qq[2] = t.z; qq[3] = t.w;
            } else {
                qq[0] = qs[place<R>(d, rg)];
            }
#pragma unroll
            for (int j = 0; j < RPT; ++j) {
                s[0][j] += kk.x * qq[j];
                s[1][j] += kk.y * qq[j];
                s[2][j] += kk.z * qq[j];
                s[3][j] += kk.w * qq[j];
            }
        }
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            const int row = rg * RPT + j, last = s_last[row];
            const float l = s_lse[row];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (k0 + 4 * kg + i <= last) w[i] += exp2f(fmaf(s[i][j], p.scale, -l) * kLog2e);
        }
    }
    // the row groups' sums of each key
    __syncthreads();
    float* sums = smem;               // [kGroups][kKeys]
    for (int i = 0; i < 4; ++i) sums[rg * kKeys + 4 * kg + i] = w[i];
    __syncthreads();
    if (threadIdx.x < kKeys) {
        const int j = k0 + threadIdx.x;
        if (j < rows.n && key_row(p, b, h, j) >= 0) {
            float sum = 0.f;
            for (int i = 0; i < kGroups; ++i) sum += sums[i * kKeys + threadIdx.x];
            if (splits == 1)
                store(p, b, h, j, rows, sum);
            else
                parts[((static_cast<int64_t>(b) * p.Hkv + h) * splits + split) * p.cap + j] = sum;
        }
    }
}

__global__ void __launch_bounds__(kThreads) k_weigh_parts(const Params p, int splits, const float* parts) {
    const int h = blockIdx.y, b = blockIdx.z, j = blockIdx.x * kThreads + threadIdx.x;
    griddep_wait();
    const Rows rows = rows_of(p, b);
    if (!rows.ok || j >= rows.n || key_row(p, b, h, j) < 0) return;
    const float* at = parts + (static_cast<int64_t>(b) * p.Hkv + h) * splits * p.cap + j;
    float sum = 0.f;
    for (int i = 0; i < splits; ++i) sum += at[static_cast<int64_t>(i) * p.cap];
    store(p, b, h, j, rows, sum);
}

// CTAs of a tile: as many as fill the SMs twice, with a chunk of rows each.
int64_t chunks_of(int g, int T, int path_len) {
    const int64_t rows = static_cast<int64_t>(g) * (path_len ? path_len : T);
    return std::min<int64_t>((rows + 4 * kGroups - 1) / (4 * kGroups), 16);
}
int64_t tiles_of(int B, int Hkv, int cap) { return static_cast<int64_t>(B) * Hkv * ((cap + kKeys - 1) / kKeys); }
int splits_of(int B, int Hkv, int g, int T, int path_len, int cap) {
    return static_cast<int>(std::max<int64_t>(1, std::min(chunks_of(g, T, path_len), 2 * device_sm_count() / tiles_of(B, Hkv, cap))));
}
// Their sums: room for every tile's splits, of which there are 2 SMs in all at most.  It never shrinks as a size grows (splits
// do as B or the cache grows), so that a workspace made for the largest call serves every smaller one.
size_t parts_bytes(int B, int Hkv, int g, int T, int path_len, int cap) {
    const int64_t chunks = chunks_of(g, T, path_len);
    return chunks > 1 ? std::min<int64_t>(tiles_of(B, Hkv, cap) * chunks, 2 * device_sm_count()) * kKeys * sizeof(float) : 0;
}

template <int D>
spec_status run_fma(const Params& p, float* parts, cudaStream_t s) {
    const int most = p.Hq / p.Hkv * (p.path ? p.P : p.T);
    // one row a thread or four (8 sequences of 1000 keys and 8 heads of 8: 8 rows 19 and 22 us, 16 rows 28 and 25, 32 rows 50 and 28)
    const bool wide = most > kGroups / 2;
    const int splits = splits_of(p.B, p.Hkv, p.Hq / p.Hkv, p.T, p.path ? p.P : 0, p.cap);
    auto kern = wide ? k_weigh_fma<D, 4> : k_weigh_fma<D, 1>;
    const size_t smem = sizeof(float) * D * (kKeys + kGroups * (wide ? 4 : 1));
    if (smem > 40960) SPEC_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
    SPEC_CUDA_TRY(launch_ex("kv_weigh_fma", kern, dim3((p.cap + kKeys - 1) / kKeys * splits + 1, p.Hkv, p.B), dim3(kThreads), smem, s, true, p, splits, parts));
    if (splits > 1)
        SPEC_CUDA_TRY(launch_ex("kv_weigh_parts", k_weigh_parts, dim3((p.cap + kThreads - 1) / kThreads, p.Hkv, p.B), dim3(kThreads), 0, s, true, p, splits, parts));
    return SPEC_OK;
}

bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + static_cast<uintptr_t>(bn) && y < x + static_cast<uintptr_t>(an);
}

spec_status check_sizes(int B, int Hq, int Hkv, int T, int path_len, int64_t cap, int D, spec_dtype dt) {
    if (dt != SPEC_BF16 && dt != SPEC_F32) return fail(SPEC_EINVAL, "dtype %d unknown", static_cast<int>(dt));
    if (D != 64 && D != 128) return fail(SPEC_EUNSUPPORTED, "D = %d: only 64 and 128", D);
    if (B < 1 || B > 65535) return fail(SPEC_EINVAL, "B = %d out of 1..65535", B);
    if (Hkv < 1 || Hq < 1 || Hq > 1024 || Hq % Hkv) return fail(SPEC_EINVAL, "Hq = %d (1..1024) must be a multiple of Hkv = %d", Hq, Hkv);
    if (T < 1 || T > (1 << 22)) return fail(SPEC_EINVAL, "T = %d out of 1..2^22", T);
    if (path_len < 0 || path_len > SPEC_MAX_DEPTH + 1) return fail(SPEC_EINVAL, "path_len = %d out of 0..%d", path_len, SPEC_MAX_DEPTH + 1);
    if (cap < 1 || cap > (1 << 22)) return fail(SPEC_EINVAL, "%lld positions out of 1..2^22", static_cast<long long>(cap));
    return SPEC_OK;
}

size_t bytes_for(int B, int Hkv, int g, int T, int path_len, int cap, spec_dtype dt) {
    if (dt == SPEC_BF16) return kWsHeader + weigh_tc_bytes(g, T, path_len);
    return kWsHeader + parts_bytes(B, Hkv, g, T, path_len, cap);
}

spec_status run(Params& p, int D, spec_dtype dt, size_t ws_bytes, cudaStream_t s) {
    spec_status st = check_sizes(p.B, p.Hq, p.Hkv, p.T, p.path ? p.P : 0, p.cap, D, dt);
    if (st != SPEC_OK) return st;
    if ((p.accept_len != nullptr) != (p.path != nullptr)) return fail(SPEC_EINVAL, "accept_len and accept_path go together");
    if (p.path && p.n_rows) return fail(SPEC_EINVAL, "n_rows with an accepted path");
    if (p.path && p.P < 1) return fail(SPEC_EINVAL, "path_len = %d with an accepted path", p.P);
    if (!(p.scale >= 0.f) || std::isinf(p.scale)) return fail(SPEC_EINVAL, "scale = %g: positive, or 0 for 1/sqrt(D)", p.scale);
    if (!(p.decay >= 0.f) || !(p.decay <= 1.f)) return fail(SPEC_EINVAL, "decay = %g out of 0..1", p.decay);
    if (!p.q || !p.lse || !p.k || !p.len || !p.acc) return fail(SPEC_EINVAL, "q, lse, the keys, prefix_len and acc must not be NULL");
    if (!aligned16(p.q) || !aligned16(p.k)) return fail(SPEC_EALIGN, "q and the keys must be 16-byte aligned");
    const void* small[] = {p.lse, p.len, p.seen, p.n_rows, p.accept_len, p.path, p.table, p.acc, p.pos};
    for (const void* x : small)
        if (!aligned4(x)) return fail(SPEC_EALIGN, "lse, lengths, paths, tables, acc and pos must be 4-byte aligned");
    const int es = dt == SPEC_BF16 ? 2 : 4;
    const int64_t out = static_cast<int64_t>(p.B) * p.Hkv * p.cap * 4;
    const struct { const void* x; int64_t n; } in[] = {
        {p.q, static_cast<int64_t>(p.B) * p.Hq * p.T * D * es}, {p.lse, static_cast<int64_t>(p.B) * p.Hq * p.T * 4},
        {p.k, static_cast<int64_t>(p.table ? p.num_blocks : p.B) * p.Hkv * p.rows * D * es}, {p.len, p.B * 4ll}, {p.seen, p.B * 4ll},
        {p.n_rows, p.B * 4ll}, {p.accept_len, p.B * 4ll}, {p.path, 4ll * p.B * p.P}, {p.table, 4ll * p.B * p.max_blocks}};
    for (const auto& i : in)
        if (overlap(p.acc, out, i.x, i.n) || overlap(p.pos, out, i.x, i.n)) return fail(SPEC_EINVAL, "acc or pos overlaps an input");
    if (overlap(p.acc, out, p.pos, out)) return fail(SPEC_EINVAL, "acc overlaps pos");
    const size_t need = bytes_for(p.B, p.Hkv, p.Hq / p.Hkv, p.T, p.path ? p.P : 0, p.cap, dt);
    if (!p.ws || ws_bytes < need) return fail(SPEC_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
    if (!aligned16(p.ws)) return fail(SPEC_EALIGN, "workspace must be 16-byte aligned");
    if (p.scale == 0.f) p.scale = 1.f / sqrtf(static_cast<float>(D));
    if (dt == SPEC_BF16) return weigh_tc_run(p, D, static_cast<char*>(p.ws) + kWsHeader, s);
    float* parts = reinterpret_cast<float*>(static_cast<char*>(p.ws) + kWsHeader);
    return D == 64 ? run_fma<64>(p, parts, s) : run_fma<128>(p, parts, s);
}

}  // namespace weigh
}  // namespace spec

using namespace spec;

extern "C" size_t kv_weigh_workspace_size(int32_t B, int32_t Hq, int32_t Hkv, int32_t T, int32_t path_len, int32_t Lmax,
                                          int32_t D, spec_dtype dt) {
    clear_error();
    if (weigh::check_sizes(B, Hq, Hkv, T, path_len, Lmax, D, dt) != SPEC_OK) return 0;
    return weigh::bytes_for(B, Hkv, Hq / Hkv, T, path_len, Lmax, dt);
}

extern "C" spec_status kv_weigh(const void* q, const float* lse, const void* k_cache, const int32_t* prefix_len,
                                const int32_t* seen, const int32_t* n_rows, const int32_t* accept_len,
                                const int32_t* accept_path, int32_t path_len, int32_t B, int32_t Hq, int32_t Hkv, int32_t T,
                                int32_t Lmax, int32_t D, float scale, float decay, spec_dtype dt, float* acc, int32_t* pos,
                                void* ws, size_t ws_bytes, spec_stream_t s) {
    clear_error();
    weigh::Params p{};
    p.q = q; p.lse = lse; p.k = k_cache; p.len = prefix_len; p.seen = seen; p.n_rows = n_rows;
    p.accept_len = accept_len; p.path = accept_path; p.P = path_len;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.T = T; p.rows = Lmax; p.cap = Lmax;
    p.scale = scale; p.decay = decay; p.acc = acc; p.pos = pos; p.ws = ws;
    return weigh::run(p, D, dt, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}

extern "C" spec_status kv_weigh_paged(const void* q, const float* lse, const void* k_pool, int32_t num_blocks,
                                      const int32_t* block_table, int32_t max_blocks, int32_t block_size,
                                      const int32_t* prefix_len, const int32_t* seen, const int32_t* n_rows,
                                      const int32_t* accept_len, const int32_t* accept_path, int32_t path_len, int32_t B,
                                      int32_t Hq, int32_t Hkv, int32_t T, int32_t D, float scale, float decay, spec_dtype dt,
                                      float* acc, int32_t* pos, void* ws, size_t ws_bytes, spec_stream_t s) {
    clear_error();
    if (num_blocks < 1 || max_blocks < 1 || block_size < 16 || block_size % 16)
        return fail(SPEC_EINVAL, "num_blocks = %d, max_blocks = %d must be positive, block_size = %d a multiple of 16", num_blocks,
                    max_blocks, block_size);
    if (static_cast<int64_t>(max_blocks) * block_size > (1 << 22))
        return fail(SPEC_EINVAL, "max_blocks * block_size = %lld positions exceed 2^22",
                    static_cast<long long>(max_blocks) * block_size);
    if (!block_table) return fail(SPEC_EINVAL, "block_table must not be NULL");
    weigh::Params p{};
    p.q = q; p.lse = lse; p.k = k_pool; p.len = prefix_len; p.seen = seen; p.n_rows = n_rows;
    p.accept_len = accept_len; p.path = accept_path; p.P = path_len;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.T = T; p.rows = block_size; p.cap = max_blocks * block_size;
    p.table = block_table; p.max_blocks = max_blocks; p.num_blocks = num_blocks;
    p.scale = scale; p.decay = decay; p.acc = acc; p.pos = pos; p.ws = ws;
    return weigh::run(p, D, dt, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}
