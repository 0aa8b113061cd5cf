// pc_embedding.cu -- lookup of feature rows with a scale, and its gradient by
// sorted tokens.
//
//   out[b, t, :] = scale table[b, idx[b, t], :]
//   grad_table[b, v, :] = scale sum of grad_out[b, t, :] over idx[b, t] = v
//
// Forward: a group of threads a token, three tokens in flight.  Bound: memory, the writes
// of the output.
//
// Backward: the tokens are sorted by their row with a stable radix sort of 32-bit
// keys (b V + idx; absent tokens last): per digit of at most 9 bits the blocks'
// histograms, their sums over the blocks before, and a scatter in which a warp
// ranks 32 keys at a time by the lanes that hold the same digit.  Then groups
// of threads walk over chunks of 64 sorted tokens (fewer in small calls), write the rows
// that begin and end there, and leave the sums of rows that reach over a chunk's border,
// which are joined afterwards: a row's chunks in their order, of a row of more than 32
// chunks in 32s summed by a kernel of their own, and these in 32s again as long as there
// can be more than 256 of them.  So a frequent row is many groups' work, and its chain of
// additions grows with the logarithm of its tokens.  Everything in float32 and in a fixed
// order.
// Bound: memory, the gradient's rows read once in the order of the table's, and in small
// calls the launches.  Measured, 500,000 tokens of 256 float32, a table of 100,000 rows:
// forward 118 us (5.2 TB/s), backward 33 of sorting, 110 of sums (4.7 TB/s), 24 of joins,
// each launch by itself (they overlap, and the zeros are written under the sort); 16 x
// 16,384 tokens of 128 bfloat16: forward 17 us.
#include "pc_device.cuh"
#include "pc_internal.h"
#include "pc_launch.cuh"
#include "pc_vec.cuh"
#include "pointcloud.h"

#include <cstdio>

namespace pcn {
namespace {

constexpr int EMB_THREADS = 256;
constexpr int RUN2 = 32;  // chunks of a second sum, these of a third, and so on
// The levels of sums, that of the chunks' heads the first: with at most 2^31 / 16 chunks
// the fifth has at most 128.
constexpr int LEVELS = 5, TOP = 256;

// --- forward ------------------------------------------------------------------

// G threads a token, U tokens a thread at a time.
constexpr int FORWARD_TOKENS = 3;
template <class T, int V>
__global__ void __launch_bounds__(EMB_THREADS)
emb_forward_kernel(const T *__restrict__ table, int64_t rows, int C,
                   const int64_t *__restrict__ idx, int64_t per_cloud, FastDiv clouds,
                   int64_t tokens, float scale, T *__restrict__ out, int G, int *status) {
    constexpr int U = FORWARD_TOKENS;
    using R = RawV<T, V>;
    const int per = EMB_THREADS / G, g = threadIdx.x / G, l = threadIdx.x - g * G;
    const int64_t t0 = int64_t(blockIdx.x) * (per * U) + g;
    if (g >= per) return;
    const T *from[U];  // nullptr: no row
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t t = t0 + u * per;
        from[u] = nullptr;
        if (t >= tokens) continue;
        const int64_t r = idx[t];
        int64_t cloud = 0;
        if (per_cloud < tokens)
            cloud = tokens < (int64_t(1) << 31) ? clouds.div(uint32_t(t)) : t / per_cloud;
        if (r >= 0 && r < rows)
            from[u] = table + (cloud * rows + r) * C;
        else if (r != -1)
            raise_status(status, PC_ERR_INVALID_ARGUMENT);
    }
    for (int c = l * V; c < C; c += G * V) {
        R raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            raw[u] = from[u] ? *reinterpret_cast<const R *>(from[u] + c) : R{};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + u * per;
            if (t >= tokens) break;
            if (scale != 1.0f && from[u]) {  // (a row that is not scaled is copied)
                float v[V];
                widen<T, V>(raw[u], v);
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] *= scale;
                Vec<T, V>::store(reinterpret_cast<T *>(&raw[u]), v);
            }
            // (written past the caches: they keep the table)
            __stcs(reinterpret_cast<R *>(out + t * C + c), raw[u]);
        }
    }
}

// --- the sort -------------------------------------------------------------------

constexpr int ITEMS = 4, TILE = EMB_THREADS * ITEMS;
constexpr int DIGITS = 512;  // of a pass, at most

struct SortArgs {
    const int64_t *idx;            // first pass: keys are formed from these
    const uint2 *in;               // later passes: key, token
    uint2 *out;
    uint32_t *count;               // [digits][blocks], then the sums over the blocks before
    uint32_t *total;               // [digits]
    int64_t rows;                  // V
    uint32_t per_cloud;            // T
    uint32_t n, absent;            // tokens; the key of those without a row
    int blocks, shift, bits;
    int *status;
    // Blocks from `blocks` on write zeros to this kernel's share of the table's gradient,
    // under the sort, which leaves memory idle: words [zero0, zero1) of 16 bytes, or of 2
    // where the table is not aligned (`narrow`).
    void *zero;
    size_t zero0, zero1;
    bool narrow;
};

// True in a block that writes zeros, and has.
__device__ __forceinline__ bool write_zeros(const SortArgs &a) {
    if (blockIdx.x < a.blocks) return false;
    const size_t step = size_t(gridDim.x - a.blocks) * EMB_THREADS;
    size_t i = a.zero0 + size_t(blockIdx.x - a.blocks) * EMB_THREADS + threadIdx.x;
    if (a.narrow)
        for (; i < a.zero1; i += step) static_cast<uint16_t *>(a.zero)[i] = 0;
    else
        for (; i < a.zero1; i += step) static_cast<uint4 *>(a.zero)[i] = make_uint4(0, 0, 0, 0);
    return true;
}

__device__ __forceinline__ uint32_t sort_key(const SortArgs &a, uint32_t i, bool report) {
    const int64_t r = a.idx[i];
    if (r >= 0 && r < a.rows) return i / a.per_cloud * uint32_t(a.rows) + uint32_t(r);
    if (report && r != -1) raise_status(a.status, PC_ERR_INVALID_ARGUMENT);
    return a.absent;
}

__global__ void __launch_bounds__(EMB_THREADS) sort_count_kernel(SortArgs a) {
    let_next_start();
    after_previous();
    if (write_zeros(a)) return;
    __shared__ uint32_t hist[DIGITS];
    hist[threadIdx.x] = hist[threadIdx.x + EMB_THREADS] = 0;
    __syncthreads();
    const uint32_t mask = (1u << a.bits) - 1, i0 = blockIdx.x * uint32_t(TILE) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
        const uint32_t i = i0 + u * EMB_THREADS;
        if (i < a.n) {
            const uint32_t key = a.idx ? sort_key(a, i, true) : a.in[i].x;
            atomicAdd(&hist[(key >> a.shift) & mask], 1u);
        }
    }
    __syncthreads();
    for (uint32_t d = threadIdx.x; d <= mask; d += EMB_THREADS)
        a.count[size_t(d) * a.blocks + blockIdx.x] = hist[d];
}

// A warp a digit: the sums over the blocks before, in place, and the total.
__global__ void __launch_bounds__(EMB_THREADS) sort_scan_kernel(SortArgs a) {
    let_next_start();
    after_previous();
    const int d = blockIdx.x * (EMB_THREADS / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (d >= 1 << a.bits) return;
    uint32_t *row = a.count + size_t(d) * a.blocks, sum = 0;
    for (int i = 0; i < a.blocks; i += 32) {
        const uint32_t v = i + lane < a.blocks ? row[i + lane] : 0;
        uint32_t s = v;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t t = __shfl_up_sync(~0u, s, o);
            if (lane >= o) s += t;
        }
        if (i + lane < a.blocks) row[i + lane] = sum + s - v;
        sum += __shfl_sync(~0u, s, 31);
    }
    if (lane == 0) a.total[d] = sum;
}

__global__ void __launch_bounds__(EMB_THREADS) sort_scatter_kernel(SortArgs a) {
    let_next_start();
    after_previous();
    if (write_zeros(a)) return;
    constexpr int WARPS = EMB_THREADS / 32;
    __shared__ uint32_t hist[WARPS][DIGITS], sums[WARPS];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, t = threadIdx.x;
    const uint32_t mask = (1u << a.bits) - 1;
    // the warp's 32 ITEMS consecutive tokens
    uint2 it[ITEMS];
    uint32_t rank[ITEMS];
    const uint32_t i0 = blockIdx.x * uint32_t(TILE) + warp * (32 * ITEMS) + lane;
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
        const uint32_t i = i0 + 32 * u;
        it[u] = make_uint2(0, i);
        if (i < a.n) {
            if (a.idx)
                it[u].x = sort_key(a, i, false);
            else
                it[u] = a.in[i];
        }
    }
    for (int d = lane; d < DIGITS; d += 32) hist[warp][d] = 0;
    // where the digits 2 t and 2 t + 1 start
    uint32_t tot[2], before[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t d = 2 * t + k;
        tot[k] = d <= mask ? a.total[d] : 0;
        before[k] = d <= mask ? a.count[size_t(d) * a.blocks + blockIdx.x] : 0;
    }
    uint32_t s = tot[0] + tot[1];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t v = __shfl_up_sync(~0u, s, o);
        if (lane >= o) s += v;
    }
    if (lane == 31) sums[warp] = s;
    __syncwarp();
    // ranks among the warp's tokens
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
        // (tokens past the end rank among themselves)
        const bool in = i0 + 32 * u < a.n;
        const uint32_t d = (it[u].x >> a.shift) & mask;
        const uint32_t peers = __match_any_sync(~0u, in ? d : 0xffffffffu);
        const uint32_t had = in ? hist[warp][d] : 0;
        rank[u] = had + __popc(peers & lanemask_lt());
        __syncwarp();
        if (in && lane == __ffs(peers) - 1) hist[warp][d] = had + __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) s += sums[w];
    s -= tot[0] + tot[1];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t run = s + before[k];
        s += tot[k];
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const uint32_t v = hist[w][2 * t + k];
            hist[w][2 * t + k] = run;
            run += v;
        }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < ITEMS; ++u)
        if (i0 + 32 * u < a.n)
            a.out[hist[warp][(it[u].x >> a.shift) & mask] + rank[u]] = it[u];
}

// --- the rows' sums ---------------------------------------------------------------

struct SumArgs {
    const void *dy;
    const uint2 *sorted;  // row, token
    float *tail;          // [chunks][C], as part[0]: see emb_chunk_kernel
    float *part[LEVELS];  // heads; sums of RUN2 of these whose chunks are one row's; ...
    int levels;
    void *dtable;
    uint32_t n, rows;     // tokens, rows of all tables
    int C, run;           // tokens of a chunk
    float scale;
};

template <class T, int V>
__device__ __forceinline__ void put_row(const SumArgs &a, uint32_t row, int c, float (&sum)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] *= a.scale;
    Vec<T, V>::store(static_cast<T *>(a.dtable) + size_t(row) * a.C + c, sum);
}

// A chunk of `run` sorted tokens, by G threads: a row whose tokens all lie in the chunk
// is written; of one that goes on from the chunk before, the sum goes to the chunk's head,
// of one that goes on in the next alone, to its tail.
template <class T, int V>
__global__ void __launch_bounds__(EMB_THREADS) emb_chunk_kernel(SumArgs a, int G) {
    let_next_start();
    after_previous();
    constexpr int U = 8;
    using R = RawV<T, V>;
    const int per = EMB_THREADS / G, g = threadIdx.x / G, l = threadIdx.x - g * G;
    const uint32_t k = blockIdx.x * per + g;
    if (g >= per || uint64_t(k) * a.run >= a.n) return;
    const uint32_t i0 = k * a.run, i1 = min(a.n, i0 + a.run);
    const uint32_t first = a.sorted[i0].x, none = 0xffffffffu;
    if (first >= a.rows) return;
    const bool from = i0 > 0 && a.sorted[i0 - 1].x == first;
    const uint32_t after = i1 < a.n ? a.sorted[i1].x : none;
    for (int c = l * V; c < a.C; c += G * V) {
        const T *dy = static_cast<const T *>(a.dy) + c;
        float sum[V];
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] = 0.0f;
        uint32_t cur = first;
        bool open = from;
        // the row `cur` ends, or the chunk does
        auto close = [&]() {
            if (open)
                Vec<float, V>::store(a.part[0] + size_t(k) * a.C + c, sum);
            else
                put_row<T, V>(a, cur, c, sum);
            open = false;
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] = 0.0f;
        };
        uint2 next[U];  // a batch ahead
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = i0 + u < i1 ? a.sorted[i0 + u] : make_uint2(none, 0);
        for (uint32_t i = i0; i < i1; i += U) {
            uint2 it[U];
            R raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                it[u] = next[u];
                if (it[u].x < a.rows)
                    raw[u] = __ldcs(reinterpret_cast<const R *>(dy + size_t(it[u].y) * a.C));
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                next[u] = i + U + u < i1 ? a.sorted[i + U + u] : make_uint2(none, 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (it[u].x == none) continue;  // past the chunk's end
                if (it[u].x != cur && cur < a.rows) close();
                cur = it[u].x;
                if (cur < a.rows) {
                    float v[V];
                    widen<T, V>(raw[u], v);
#pragma unroll
                    for (int e = 0; e < V; ++e) sum[e] += v[e];
                }
            }
        }
        if (cur < a.rows) {
            if (!open && after == cur)
                Vec<float, V>::store(a.tail + size_t(k) * a.C + c, sum);
            else
                close();
        }
    }
}

template <int V>
__device__ __forceinline__ void add_parts(const float *part, uint32_t i0, uint32_t i1, int c, int C,
                                          float (&sum)[V]) {
#pragma unroll 8
    for (uint32_t i = i0; i < i1; ++i) {
        float v[V];
        Vec<float, V>::load(part + size_t(i) * C + c, v);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += v[e];
    }
}

// Adds a level's parts [b, e) in their order.  The row fills those below `last`, so where
// the next level has sums of such, they stand for them.
template <int V, int L>
__device__ __forceinline__ void add_level(const SumArgs &a, uint32_t b, uint32_t e, uint32_t last,
                                          int c, float (&sum)[V]) {
    if constexpr (L + 1 < LEVELS) {
        const uint32_t j0 = (b + RUN2 - 1) / RUN2, j1 = last / RUN2;
        if (L + 1 < a.levels && j0 < j1) {
            add_parts<V>(a.part[L], b, j0 * RUN2, c, a.C, sum);
            add_level<V, L + 1>(a, j0, j1, j1, c, sum);
            add_parts<V>(a.part[L], j1 * RUN2, e, c, a.C, sum);
            return;
        }
    }
    add_parts<V>(a.part[L], b, e, c, a.C, sum);
}

// RUN2 parts of a level, of `span` tokens together, that one row fills and came into.
template <int V>
__global__ void __launch_bounds__(EMB_THREADS)
emb_second_kernel(SumArgs a, int G, const float *part, float *to, uint32_t span) {
    let_next_start();
    after_previous();
    const int per = EMB_THREADS / G, g = threadIdx.x / G, l = threadIdx.x - g * G;
    const uint32_t j = blockIdx.x * per + g;
    if (g >= per || (uint64_t(j) + 1) * span > a.n) return;
    const uint32_t row = a.sorted[j * span].x;
    if (row >= a.rows || a.sorted[j * span + span - 1].x != row) return;
    if (j == 0 || a.sorted[j * span - 1].x != row) return;
    for (int c = l * V; c < a.C; c += G * V) {
        float sum[V];
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] = 0.0f;
        add_parts<V>(part, j * RUN2, (j + 1) * RUN2, c, a.C, sum);
        Vec<float, V>::store(to + size_t(j) * a.C + c, sum);
    }
}

// The rows that go on beyond the chunk k that they begin in: its tail and the heads of the
// chunks after it.
template <class T, int V>
__global__ void __launch_bounds__(EMB_THREADS) emb_join_kernel(SumArgs a, int G) {
    let_next_start();
    after_previous();
    const int per = EMB_THREADS / G, g = threadIdx.x / G, l = threadIdx.x - g * G;
    const uint32_t k = blockIdx.x * per + g;
    if (g >= per || (uint64_t(k) + 1) * a.run >= a.n) return;
    const uint32_t i0 = k * a.run, i1 = i0 + a.run, row = a.sorted[i1].x;
    if (row >= a.rows || a.sorted[i1 - 1].x != row) return;
    if (k > 0 && a.sorted[i0].x == row && a.sorted[i0 - 1].x == row) return;  // began before
    // the last chunk that starts with the row
    uint32_t lo = k + 1, hi = (a.n - 1) / a.run;
    if (lo < hi && a.sorted[(lo + 1) * a.run].x != row) hi = lo;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        if (a.sorted[mid * a.run].x == row)
            lo = mid;
        else
            hi = mid - 1;
    }
    // heads [k + 1, lo], whose chunks the row fills, but perhaps the last
    for (int c = l * V; c < a.C; c += G * V) {
        float sum[V];
        Vec<float, V>::load(a.tail + size_t(k) * a.C + c, sum);
        add_level<V, 0>(a, k + 1, lo + 1, lo, c, sum);
        put_row<T, V>(a, row, c, sum);
    }
}

// --- launches ---------------------------------------------------------------------

// Threads of a row of `nv` vectors: a warp takes rows of more in several goes.
int emb_group(int nv) { return nv < 32 ? nv : nv <= 64 ? (nv + 1) / 2 : 32; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class T, int V>
cudaError_t emb_forward(const DeviceInfo &dev, const void *table, int64_t V_, int C,
                        const int64_t *idx, int64_t T_, int64_t tokens, float scale, void *out,
                        cudaStream_t st) {
    const int G = emb_group(C / V), per = EMB_THREADS / G;
    const int64_t blocks = ceil_div(tokens, per * FORWARD_TOKENS);
    if (blocks > 2147483647) return cudaErrorInvalidConfiguration;
    emb_forward_kernel<T, V><<<unsigned(blocks), EMB_THREADS, 0, st>>>(
        static_cast<const T *>(table), V_, C, idx, T_,
        FastDiv(T_ < (int64_t(1) << 31) ? uint32_t(T_) : 1), tokens, scale, static_cast<T *>(out), G,
        dev.status_word);
    return cudaGetLastError();
}

template <class T, int V>
cudaError_t emb_sums(const SumArgs &a, cudaStream_t st) {
    const int G = emb_group(a.C / V), per = EMB_THREADS / G;
    auto blocks = [&](int64_t n) { return unsigned(ceil_div(n, per)); };
    const int64_t chunks = ceil_div(a.n, a.run);
    cudaError_t e =
        launch(true, emb_chunk_kernel<T, V>, blocks(chunks), EMB_THREADS, 0, st, a, G);
    const int nv = a.C / V, G2 = nv < EMB_THREADS ? nv : EMB_THREADS, per2 = EMB_THREADS / G2;
    int64_t sums = chunks, span = a.run;
    for (int l = 1; e == cudaSuccess && l < a.levels; ++l) {
        sums /= RUN2, span *= RUN2;
        e = launch(true, emb_second_kernel<V>, unsigned(ceil_div(sums, per2)), EMB_THREADS, 0, st, a,
                   G2, a.part[l - 1], a.part[l], uint32_t(span));
    }
    if (e == cudaSuccess && chunks > 1)
        e = launch(true, emb_join_kernel<T, V>, unsigned(ceil_div(chunks - 1, per2)), EMB_THREADS,
                   0, st, a, G2);
    return e;
}

// The widest vectors that rows of C elements at these addresses can have.
template <class T>
int emb_vector(int64_t C, const void *p, const void *q) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q);
    int V = 16 / int(sizeof(T));
    while (V > 1 && (C % V || bits % (V * sizeof(T)))) V /= 2;
    return V;
}

template <class T>
cudaError_t emb_forward_any(const DeviceInfo &dev, const void *table, int64_t V, int C,
                            const int64_t *idx, int64_t T_, int64_t tokens, float scale, void *out,
                            cudaStream_t st) {
    switch (emb_vector<T>(C, table, out)) {
        case 8:
            return emb_forward<T, sizeof(T) == 2 ? 8 : 4>(dev, table, V, C, idx, T_, tokens, scale,
                                                          out, st);
        case 4: return emb_forward<T, 4>(dev, table, V, C, idx, T_, tokens, scale, out, st);
        case 2: return emb_forward<T, 2>(dev, table, V, C, idx, T_, tokens, scale, out, st);
        default: return emb_forward<T, 1>(dev, table, V, C, idx, T_, tokens, scale, out, st);
    }
}

template <class T>
cudaError_t emb_sums_any(const SumArgs &a, cudaStream_t st) {
    switch (emb_vector<T>(a.C, a.dy, a.dtable)) {
        case 8: return emb_sums<T, sizeof(T) == 2 ? 8 : 4>(a, st);
        case 4: return emb_sums<T, 4>(a, st);
        case 2: return emb_sums<T, 2>(a, st);
        default: return emb_sums<T, 1>(a, st);
    }
}

cudaError_t emb_backward(const DeviceInfo &dev, const void *dy, int dtype, int64_t B, int64_t V,
                         int C, const int64_t *idx, int64_t T, float scale, void *dtable,
                         cudaStream_t st) {
    const size_t es = dtype == PC_F32 ? 4 : 2, bytes = size_t(B) * V * C * es;
    if (B * T == 0) return cudaMemsetAsync(dtable, 0, bytes, st);
    SumArgs a{};
    a.dy = dy, a.dtable = dtable, a.n = uint32_t(B * T), a.rows = uint32_t(B * V), a.C = C;
    a.scale = scale;
    // 64 tokens a chunk, or 32 or 16 where that leaves the SMs short of warps
    const int64_t warps = ceil_div(int64_t(C) * es * a.n, 512), enough = int64_t(dev.sm_count) * 8;
    a.run = warps / 64 >= enough ? 64 : warps / 32 >= enough ? 32 : 16;
    // keys 0 .. rows, the last for absent tokens
    int bits = 0;
    while ((int64_t(1) << bits) <= int64_t(a.rows)) ++bits;
    const int passes = (bits + 8) / 9, each = (bits + passes - 1) / passes;
    const int blocks = int((int64_t(a.n) + TILE - 1) / TILE);
    auto round = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t list = round(size_t(a.n) * sizeof(uint2));
    const size_t count = round((size_t(blocks) + 1) * (size_t(1) << each) * 4);
    const size_t chunks = size_t(ceil_div(a.n, a.run));
    size_t sums[LEVELS] = {chunks}, parts = round(chunks * C * 4);  // (heads)
    for (a.levels = 1; a.levels < LEVELS; ++a.levels) {
        const size_t below = sums[a.levels - 1];
        if (below <= (a.levels == 1 ? RUN2 : TOP)) break;
        sums[a.levels] = below / RUN2;
        parts += round(sums[a.levels] * C * 4);
    }
    char *mem = nullptr;
    cudaError_t e = scratch_alloc(dev, reinterpret_cast<void **>(&mem),
                      2 * list + count + round(chunks * C * 4) + parts, st);
    if (e != cudaSuccess) return e;
    uint2 *lists[2] = {reinterpret_cast<uint2 *>(mem), reinterpret_cast<uint2 *>(mem + list)};
    SortArgs s{};
    s.idx = idx, s.rows = V, s.per_cloud = uint32_t(T), s.n = a.n, s.absent = a.rows;
    s.count = reinterpret_cast<uint32_t *>(mem + 2 * list);
    s.total = s.count + (size_t(blocks) << each);
    s.blocks = blocks, s.bits = each, s.status = dev.status_word;
    // rows without tokens are 0 (the others are written again): a share of the zeros in
    // each of the counts and scatters
    s.zero = dtable, s.narrow = reinterpret_cast<uintptr_t>(dtable) % 16 || bytes % 16;
    const size_t words = bytes / (s.narrow ? 2 : 16), shares = 2 * size_t(passes);
    auto with_zeros = [&](size_t share) {
        s.zero0 = words * share / shares, s.zero1 = words * (share + 1) / shares;
        const int64_t want = ceil_div(int64_t(s.zero1 - s.zero0), EMB_THREADS * 8);
        const int64_t most = int64_t(dev.sm_count) * 4;
        return unsigned(blocks + (want < most ? want : most));
    };
    for (int p = 0; p < passes; ++p) {
        s.shift = p * each;
        s.out = lists[p % 2];
        unsigned grid = with_zeros(2 * p);
        if (e == cudaSuccess) e = launch(p > 0, sort_count_kernel, grid, EMB_THREADS, 0, st, s);
        if (e == cudaSuccess)
            e = launch(true, sort_scan_kernel, ((1 << each) + 7) / 8, EMB_THREADS, 0, st, s);
        grid = with_zeros(2 * p + 1);
        if (e == cudaSuccess) e = launch(true, sort_scatter_kernel, grid, EMB_THREADS, 0, st, s);
        s.idx = nullptr, s.in = s.out;
    }
    a.sorted = s.out;
    a.tail = reinterpret_cast<float *>(mem + 2 * list + count);
    a.part[0] = a.tail + round(chunks * C * 4) / sizeof(float);
    for (int l = 1; l < a.levels; ++l)
        a.part[l] = a.part[l - 1] + round(sums[l - 1] * C * 4) / sizeof(float);
    if (e == cudaSuccess)
        e = dtype == PC_F32 ? emb_sums_any<float>(a, st) : emb_sums_any<bf16>(a, st);
    const cudaError_t f = scratch_free(mem, st);
    return e == cudaSuccess ? f : e;
}

int emb_check(const char *what, int dtype, int64_t B, int64_t V, int64_t C, int64_t T,
              double scale, int64_t most) {
    char m[200];
    const char *why = nullptr;
    int code = PC_ERR_INVALID_ARGUMENT;
    if (B < 0 || V < 0 || C < 0 || T < 0)
        why = "negative size";
    else if (dtype != PC_F32 && dtype != PC_BF16)
        why = "dtype must be PC_F32 or PC_BF16";
    else if (!(scale >= -3.4e38 && scale <= 3.4e38))
        why = "scale must be finite";
    else if (C > 65536 || (B > 0 && (V > most / B || T > most / B)))
        why = "C above 65536, or B V or B T beyond the supported range",
        code = PC_ERR_UNSUPPORTED;
    if (why == nullptr) return PC_OK;
    std::snprintf(m, sizeof(m), "%s: %s", what, why);
    return api_fail(code, m);
}

int emb_cuda(const char *what, cudaError_t e) {
    if (e == cudaSuccess) return PC_OK;
    char m[200];
    std::snprintf(m, sizeof(m), "%s: %s", what, cudaGetErrorString(e));
    return api_fail(PC_ERR_CUDA, m);
}

}  // namespace
}  // namespace pcn

extern "C" int pc_embedding(const void *table, int dtype, int64_t B, int64_t V, int64_t C,
                            const int64_t *idx, int64_t T, double scale, void *out,
                            void *stream) {
    using namespace pcn;
    int rc = emb_check("embedding", dtype, B, V, C, T, scale, int64_t(1) << 40);
    if (rc != PC_OK) return rc;
    if (B == 0 || C == 0 || T == 0) return PC_OK;
    const DeviceInfo *dev = nullptr;
    if ((rc = api_current_device(&dev)) != PC_OK) return rc;
    const size_t es = dtype == PC_F32 ? 4 : 2;
    if (V > 0 && (rc = api_check_ptr(table, dev->device, es, "table")) != PC_OK) return rc;
    if ((rc = api_check_ptr(idx, dev->device, 8, "idx")) != PC_OK) return rc;
    if ((rc = api_check_ptr(out, dev->device, es, "out")) != PC_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return emb_cuda("embedding",
                    dtype == PC_F32
                        ? emb_forward_any<float>(*dev, table, V, int(C), idx, T, B * T,
                                                 float(scale), out, st)
                        : emb_forward_any<bf16>(*dev, table, V, int(C), idx, T, B * T,
                                                float(scale), out, st));
}

extern "C" int pc_embedding_backward(const void *grad_out, int dtype, int64_t B, int64_t V,
                                     int64_t C, const int64_t *idx, int64_t T, double scale,
                                     void *grad_table, void *stream) {
    using namespace pcn;
    int rc = emb_check("embedding_backward", dtype, B, V, C, T, scale,
                       (int64_t(1) << 31) - (int64_t(1) << 20));
    if (rc != PC_OK) return rc;
    if (B == 0 || V == 0 || C == 0) return PC_OK;
    const DeviceInfo *dev = nullptr;
    if ((rc = api_current_device(&dev)) != PC_OK) return rc;
    const size_t es = dtype == PC_F32 ? 4 : 2;
    if (T > 0) {
        if ((rc = api_check_ptr(grad_out, dev->device, es, "grad_out")) != PC_OK) return rc;
        if ((rc = api_check_ptr(idx, dev->device, 8, "idx")) != PC_OK) return rc;
    }
    if ((rc = api_check_ptr(grad_table, dev->device, es, "grad_table")) != PC_OK) return rc;
    return emb_cuda("embedding_backward",
                    emb_backward(*dev, grad_out, dtype, B, V, int(C), idx, T, float(scale),
                                 grad_table, static_cast<cudaStream_t>(stream)));
}
