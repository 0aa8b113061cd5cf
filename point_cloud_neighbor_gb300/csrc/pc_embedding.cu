// pc_embedding.cu -- lookup of feature rows with a scale, and its gradient by
// sorted tokens.
//
//   out[b, t, :] = scale table[b, idx[b, t], :]
//   grad_table[b, v, :] = scale sum of grad_out[b, t, :] over idx[b, t] = v
//
// Forward: a thread a vector of up to 16 bytes, four in flight.  Bound: memory,
// the writes of the output.
//
// Backward: the tokens are sorted by their row with a stable radix sort of 32-bit
// keys (b V + idx; absent tokens last): per digit of at most 8 bits the blocks'
// histograms, their sums over the blocks before, and a scatter in which a warp
// ranks 32 keys at a time by the lanes that hold the same digit.  Then every
// row of the table finds its run of tokens by bisection and adds it up, in the
// order of the tokens, and is written once, zeros among them.  Runs of more
// than 64 tokens are added in chunks of 64 consecutive sorted tokens, and these in
// chunks of 64 again, by kernels of their own before, so that one frequent row
// is not one thread group's work.  Everything in float32 and in a fixed order.
// Bound: memory, the gradient's rows read once in the order of the table's.
#include "pc_device.cuh"
#include "pc_internal.h"
#include "pc_vec.cuh"
#include "pointcloud.h"

#include <cstdio>

namespace pcn {
namespace {

constexpr int EMB_THREADS = 256;
constexpr int RUN = 64;  // tokens of a chunk, chunks of a second chunk

// --- forward ------------------------------------------------------------------

template <class T, int V>
__global__ void __launch_bounds__(EMB_THREADS)
emb_forward_kernel(const T *__restrict__ table, int64_t rows, int C, const int64_t *__restrict__ idx,
                   int64_t T_, int64_t tokens, float scale, T *__restrict__ out, int *status) {
    constexpr int U = 4;
    const int nv = C / V;
    const int64_t total = tokens * nv, step = int64_t(gridDim.x) * EMB_THREADS;
    for (int64_t i0 = int64_t(blockIdx.x) * EMB_THREADS + threadIdx.x; i0 < total;
         i0 += U * step) {
        float v[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * step;
#pragma unroll
            for (int e = 0; e < V; ++e) v[u][e] = 0.0f;
            if (i < total) {
                const int64_t t = i / nv;
                const int c = int(i - t * nv) * V;
                const int64_t r = idx[t];
                if (r >= 0 && r < rows)
                    Vec<T, V>::load(table + (t / T_ * rows + r) * C + c, v[u]);
                else if (r != -1)
                    raise_status(status, PC_ERR_INVALID_ARGUMENT);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * step;
            if (i < total) {
#pragma unroll
                for (int e = 0; e < V; ++e) v[u][e] *= scale;
                Vec<T, V>::store(out + i * V, v[u]);
            }
        }
    }
}

// --- the sort -------------------------------------------------------------------

constexpr int ITEMS = 8, TILE = EMB_THREADS * ITEMS;

struct SortArgs {
    const int64_t *idx;            // first pass: keys are formed from these
    const uint32_t *keys, *vals;   // later passes
    uint32_t *out_keys, *out_vals;
    uint32_t *count;               // [digits][blocks], then the sums over the blocks before
    uint32_t *total;               // [digits]
    int64_t rows, per_cloud;       // V, T
    uint32_t n, absent;            // tokens; the key of those without a row
    int blocks, shift, bits;
    int *status;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs &a, uint32_t i, bool report) {
    if (a.idx == nullptr) return a.keys[i];
    const int64_t r = a.idx[i];
    if (r >= 0 && r < a.rows) return uint32_t(i / a.per_cloud * a.rows + r);
    if (report && r != -1) raise_status(a.status, PC_ERR_INVALID_ARGUMENT);
    return a.absent;
}

__global__ void __launch_bounds__(EMB_THREADS) sort_count_kernel(SortArgs a) {
    __shared__ uint32_t hist[256];
    hist[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t mask = (1u << a.bits) - 1, i0 = blockIdx.x * uint32_t(TILE) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
        const uint32_t i = i0 + u * EMB_THREADS;
        if (i < a.n) atomicAdd(&hist[(sort_key(a, i, true) >> a.shift) & mask], 1u);
    }
    __syncthreads();
    if (threadIdx.x <= mask) a.count[size_t(threadIdx.x) * a.blocks + blockIdx.x] = hist[threadIdx.x];
}

// A warp a digit: the sums over the blocks before, in place, and the total.
__global__ void __launch_bounds__(EMB_THREADS) sort_scan_kernel(SortArgs a) {
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
    constexpr int WARPS = EMB_THREADS / 32;
    __shared__ uint32_t hist[WARPS][256], base[256], sums[WARPS];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, t = threadIdx.x;
    const uint32_t mask = (1u << a.bits) - 1;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) hist[w][t] = 0;
    // where the digits start
    const uint32_t tot = t <= mask ? a.total[t] : 0;
    uint32_t s = tot;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t v = __shfl_up_sync(~0u, s, o);
        if (lane >= o) s += v;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    for (int w = 0; w < warp; ++w) s += sums[w];
    base[t] = s - tot + (t <= mask ? a.count[size_t(t) * a.blocks + blockIdx.x] : 0);
    // ranks within the warp's 32 ITEMS consecutive tokens
    uint32_t key[ITEMS], val[ITEMS], rank[ITEMS];
    const uint32_t i0 = blockIdx.x * uint32_t(TILE) + warp * (32 * ITEMS) + lane;
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
        const uint32_t i = i0 + 32 * u;
        key[u] = val[u] = 0;
        if (i < a.n) {
            key[u] = sort_key(a, i, false);
            val[u] = a.idx ? i : a.vals[i];
        }
    }
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
        // (tokens past the end rank among themselves)
        const bool in = i0 + 32 * u < a.n;
        const uint32_t d = (key[u] >> a.shift) & mask;
        const uint32_t peers = __match_any_sync(~0u, in ? d : 0xffffffffu);
        const uint32_t before = in ? hist[warp][d] : 0;
        rank[u] = before + __popc(peers & lanemask_lt());
        __syncwarp();
        if (in && lane == __ffs(peers) - 1) hist[warp][d] = before + __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    uint32_t run = base[t];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const uint32_t v = hist[w][t];
        hist[w][t] = run;
        run += v;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < ITEMS; ++u)
        if (i0 + 32 * u < a.n) {
            const uint32_t at = hist[warp][(key[u] >> a.shift) & mask] + rank[u];
            a.out_keys[at] = key[u];
            a.out_vals[at] = val[u];
        }
}

// --- the rows' sums ---------------------------------------------------------------

struct SumArgs {
    const void *dy;
    const uint32_t *keys, *vals;
    float *part1, *part2;  // sums of chunks of RUN tokens, of RUN such chunks
    void *dtable;
    uint32_t n;
    int64_t rows;          // of all tables
    int C;
    float scale;
};

// sum += rows [i0, i1) of sorted tokens
template <class T, int V>
__device__ __forceinline__ void add_tokens(const SumArgs &a, uint32_t i0, uint32_t i1, int c,
                                           float (&sum)[V]) {
    constexpr int U = 4;
    const T *dy = static_cast<const T *>(a.dy) + c;
    uint32_t i = i0;
    for (; i + U <= i1; i += U) {
        float v[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) Vec<T, V>::load(dy + size_t(a.vals[i + u]) * a.C, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += v[u][e];
    }
    for (; i < i1; ++i) {
        float v[V];
        Vec<T, V>::load(dy + size_t(a.vals[i]) * a.C, v);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += v[e];
    }
}
template <int V>
__device__ __forceinline__ void add_parts(const float *part, uint32_t i0, uint32_t i1, int c, int C,
                                          float (&sum)[V]) {
#pragma unroll 4
    for (uint32_t i = i0; i < i1; ++i) {
        float v[V];
        Vec<float, V>::load(part + size_t(i) * C + c, v);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += v[e];
    }
}

// Chunks of one row alone: of tokens (LEVEL 1), of chunks (LEVEL 2).  A thread
// a vector of a chunk.
template <class T, int V, int LEVEL>
__global__ void __launch_bounds__(EMB_THREADS) emb_chunk_kernel(SumArgs a) {
    const int nv = a.C / V;
    const int64_t i = int64_t(blockIdx.x) * EMB_THREADS + threadIdx.x;
    const uint32_t span = LEVEL == 1 ? RUN : RUN * RUN;
    const int64_t k = i / nv;
    const int c = int(i - k * nv) * V;
    if ((k + 1) * span > a.n) return;
    const uint32_t i0 = uint32_t(k) * span, first = a.keys[i0];
    if (first >= a.rows || a.keys[i0 + span - 1] != first) return;
    float sum[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = 0.0f;
    if (LEVEL == 1)
        add_tokens<T, V>(a, i0, i0 + RUN, c, sum);
    else
        add_parts<V>(a.part1, uint32_t(k) * RUN, uint32_t(k + 1) * RUN, c, a.C, sum);
    Vec<float, V>::store((LEVEL == 1 ? a.part1 : a.part2) + size_t(k) * a.C + c, sum);
}

// the first sorted token whose row is not below `row`
__device__ __forceinline__ uint32_t lower_bound(const uint32_t *keys, uint32_t n, uint32_t row) {
    uint32_t lo = 0, hi = n;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (keys[mid] < row)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// G threads a row of the table.
template <class T, int V>
__global__ void __launch_bounds__(EMB_THREADS) emb_rows_kernel(SumArgs a, int G) {
    const int per = EMB_THREADS / G, g = threadIdx.x / G, l = threadIdx.x % G;
    __shared__ uint32_t bounds[EMB_THREADS + 1];
    const int64_t r0 = int64_t(blockIdx.x) * per;
    for (int i = threadIdx.x; i <= per; i += EMB_THREADS)
        bounds[i] = lower_bound(a.keys, a.n, uint32_t(min(r0 + int64_t(i), a.rows)));
    __syncthreads();
    const int64_t row = r0 + g;
    if (g >= per || row >= a.rows) return;
    const uint32_t s = bounds[g], e = bounds[g + 1];
    for (int c = l * V; c < a.C; c += G * V) {
        float sum[V];
#pragma unroll
        for (int k = 0; k < V; ++k) sum[k] = 0.0f;
        // whole chunks of the row: [c0, c1), and of those whole second chunks [d0, d1)
        const uint32_t c0 = (s + RUN - 1) / RUN, c1 = e / RUN;
        if (c0 >= c1) {
            add_tokens<T, V>(a, s, e, c, sum);
        } else {
            const uint32_t d0 = (c0 + RUN - 1) / RUN, d1 = c1 / RUN;
            add_tokens<T, V>(a, s, c0 * RUN, c, sum);
            if (d0 >= d1) {
                add_parts<V>(a.part1, c0, c1, c, a.C, sum);
            } else {
                add_parts<V>(a.part1, c0, d0 * RUN, c, a.C, sum);
                add_parts<V>(a.part2, d0, d1, c, a.C, sum);
                add_parts<V>(a.part1, d1 * RUN, c1, c, a.C, sum);
            }
            add_tokens<T, V>(a, c1 * RUN, e, c, sum);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) sum[k] *= a.scale;
        Vec<T, V>::store(static_cast<T *>(a.dtable) + row * a.C + c, sum);
    }
}

// --- launches ---------------------------------------------------------------------

template <class T, int V>
cudaError_t emb_forward(const DeviceInfo &dev, const void *table, int64_t V_, int C,
                        const int64_t *idx, int64_t T_, int64_t tokens, float scale, void *out,
                        cudaStream_t st) {
    const int64_t want = (tokens * (C / V) + 4 * EMB_THREADS - 1) / (4 * EMB_THREADS);
    const int64_t most = int64_t(dev.sm_count) * 8 * 16;
    emb_forward_kernel<T, V><<<unsigned(want < most ? want : most), EMB_THREADS, 0, st>>>(
        static_cast<const T *>(table), V_, C, idx, T_, tokens, scale, static_cast<T *>(out),
        dev.status_word);
    return cudaGetLastError();
}

template <class T, int V>
cudaError_t emb_sums(const SumArgs &a, cudaStream_t st) {
    const int nv = a.C / V;
    auto blocks = [&](int64_t chunks) {
        return unsigned((chunks * nv + EMB_THREADS - 1) / EMB_THREADS);
    };
    if (a.n >= RUN) emb_chunk_kernel<T, V, 1><<<blocks(a.n / RUN), EMB_THREADS, 0, st>>>(a);
    if (a.n >= RUN * RUN)
        emb_chunk_kernel<T, V, 2><<<blocks(a.n / (RUN * RUN)), EMB_THREADS, 0, st>>>(a);
    const int G = nv < EMB_THREADS ? nv : EMB_THREADS, per = EMB_THREADS / G;
    emb_rows_kernel<T, V><<<unsigned((a.rows + per - 1) / per), EMB_THREADS, 0, st>>>(a, G);
    return cudaGetLastError();
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
    SumArgs a{};
    a.dy = dy, a.dtable = dtable, a.n = uint32_t(B * T), a.rows = B * V, a.C = C, a.scale = scale;
    // keys 0 .. rows, the last for absent tokens
    int bits = 0;
    while ((int64_t(1) << bits) <= a.rows) ++bits;
    const int passes = (bits + 7) / 8, each = (bits + passes - 1) / passes;
    const int blocks = int((int64_t(a.n) + TILE - 1) / TILE);
    auto round = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t list = round(size_t(a.n) * 4), count = round((size_t(blocks) + 1) * 256 * 4);
    const size_t part1 = round(size_t(a.n / RUN) * C * 4);
    const size_t part2 = round(size_t(a.n / (RUN * RUN)) * C * 4);
    char *mem = nullptr;
    cudaError_t e = scratch_alloc(dev, reinterpret_cast<void **>(&mem),
                                  4 * list + count + part1 + part2, st);
    if (e != cudaSuccess) return e;
    uint32_t *lists[2][2];  // [which][keys, tokens]
    for (int i = 0; i < 4; ++i) lists[i / 2][i % 2] = reinterpret_cast<uint32_t *>(mem + i * list);
    SortArgs s{};
    s.idx = idx, s.rows = V, s.per_cloud = T, s.n = a.n, s.absent = uint32_t(a.rows);
    s.count = reinterpret_cast<uint32_t *>(mem + 4 * list);
    s.total = s.count + size_t(256) * blocks;
    s.blocks = blocks, s.bits = each, s.status = dev.status_word;
    if (a.n > 0)
        for (int p = 0; p < passes; ++p) {
            s.shift = p * each;
            s.out_keys = lists[p % 2][0], s.out_vals = lists[p % 2][1];
            sort_count_kernel<<<blocks, EMB_THREADS, 0, st>>>(s);
            sort_scan_kernel<<<((1 << each) + 7) / 8, EMB_THREADS, 0, st>>>(s);
            sort_scatter_kernel<<<blocks, EMB_THREADS, 0, st>>>(s);
            s.idx = nullptr, s.keys = s.out_keys, s.vals = s.out_vals;
        }
    a.keys = lists[(passes + 1) % 2][0], a.vals = lists[(passes + 1) % 2][1];
    a.part1 = reinterpret_cast<float *>(mem + 4 * list + count);
    a.part2 = reinterpret_cast<float *>(mem + 4 * list + count + part1);
    e = cudaGetLastError();
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
