// pc_layer_norm.cu -- layer norm over the last axis, forward and backward.
//
//   mean = sum x / C, var = sum (x - mean)^2 / C, rstd = 1 / sqrt(var + eps)
//   y  = (x - mean) rstd w + b
//   xhat = (x - mean) rstd, g = dy w
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),
//   dw = sum_rows dy xhat,  db = sum_rows dy.
//
// Bound: memory.  A row is read once by TPR threads (8 for C <= 128, a warp up
// to C of about 1000, a block of 256 beyond) and written once; the variance is
// summed from the centred values in registers, so no cancellation of sums of
// squares.  All sums are float32.
//
// Rows of an odd C start at any multiple of the element size, yet the rows
// together are one packed array.  A thread group takes every G-th row, G a
// multiple of the V elements of a 16-byte vector, so its rows all start at
// the same offset within a vector: it reads the aligned vectors that cover
// the row, the first and last of them in part.  So every C has 16-byte loads,
// and a thread's columns are the same in all its rows: weight, bias and the
// columns' gradient sums stay in registers.
//
// The weight gradients need a sum over all rows.  Each backward block walks
// its share of the rows with the columns' sums in registers, adds its groups'
// in a fixed order and writes one row of partial sums; a second kernel adds
// the blocks' rows in a fixed order.  No atomics: the result does not change
// from run to run.
//
// What counts is the bytes in flight.  A thread's rows come through a ring of
// slots in shared memory, up to 4 rows deep, by asynchronous copies; a slot is
// written and read by one thread alone, so there is nothing to wait for but the
// thread's own copies.  Blocks are small (128 threads) and fill the registers.
// Measured, 100,000 x 512 float32: forward 73 us (5.6 TB/s), backward 108 us
// (5.7 TB/s); C = 515: 76 and 121 us (with the next row in registers 85 and
// 147 us, with one element a load 158 and 368 us); 65,536 x 1024 bfloat16: 50
// us (5.4 TB/s) and 84 us (4.8 TB/s; registers 60 and 102 us); 100,000 x 515
// bfloat16: 76 and 96 us (registers 78 and 136 us), bound by instructions.
#include "pc_internal.h"
#include "pc_vec.cuh"
#include "pointcloud.h"

#include <cstdio>

namespace pcn {
namespace {

// Threads of a block: small blocks fill the registers of a SM better.
__host__ __device__ constexpr int ln_threads(int tpr) { return tpr > 128 ? tpr : 128; }
constexpr int LN_MAX_C = 8192;

struct LnArgs {
    const void *x, *dy, *w, *b;
    void *y;  // forward: y; backward: dx
    float *mean, *rstd;
    float *part;  // backward: [gridDim.x][2][C]
    int64_t rows;
    int C;
    float eps;
};

// Sum over the TPR threads that share a row, the same value in each.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *red) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if (TPR > 32) {
        __syncthreads();  // red may still be read from the last sum
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) v += red[i];
    }
    return v;
}

// 1 / sqrt(v) from the hardware's approximation and a step of Newton's method;
// infinity for 0 (a constant row with eps 0) as it is.
__device__ __forceinline__ float inv_sqrt(float v) {
    const float r = rsqrtf(v), d = fmaf(-v * r, r, 1.0f);
    return v > 0.0f && v < INFINITY ? fmaf(0.5f * r, d, r) : r;
}

// V elements on their way through a slot of shared memory that one thread
// alone writes and reads.  At the ends of a row a vector has elements of the
// neighbouring rows too (`edge`); one that would leave the array, of which
// `left` elements remain, is read in part, zeros beyond.
template <class T, int V>
struct Slot {
    static constexpr int BYTES = V * int(sizeof(T));
    static __device__ __forceinline__ void copy(unsigned char *slot, const T *p, bool edge,
                                                int64_t left) {
        if (V == 1) {
            *reinterpret_cast<T *>(slot) = *p;
        } else {
            const int n = edge && left < V ? int(left) * int(sizeof(T)) : 16;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             uint32_t(__cvta_generic_to_shared(slot))),
                         "l"(p), "r"(n)
                         : "memory");
        }
    }
    // as float32
    static __device__ __forceinline__ void get(const unsigned char *slot, float *f) {
        Vec<T, V>::load(reinterpret_cast<const T *>(slot), f);
    }
    // 0 where the column col + e is not one of the row
    static __device__ __forceinline__ void zero(int col, int C, float *f) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (col + e < 0 || col + e >= C) f[e] = 0.0f;
    }
    static __device__ __forceinline__ void store(T *p, bool edge, int col, int C,
                                                 const float *f) {
        if (!edge) {
            Vec<T, V>::store(p, f);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (col + e >= 0 && col + e < C) Vec<T, 1>::store(p + e, f + e);
        }
    }
};

// A thread's vectors, the same in all its rows: vector i has the columns
// first + i TPR V and on; bit i of `live`: some are the row's, of `edge`: not all.
template <int V, int N, int TPR>
struct Columns {
    int first, C;
    unsigned live = 0, edge = 0;
    __device__ __forceinline__ Columns(int t, int shift, int C_) : first(t * V - shift), C(C_) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (col(i) < C) live |= 1u << i;
            if (col(i) < 0 || col(i) + V > C) edge |= 1u << i;
        }
    }
    __device__ __forceinline__ int col(int i) const { return first + i * TPR * V; }
    __device__ __forceinline__ bool is_live(int i) const { return live >> i & 1; }
    __device__ __forceinline__ bool is_edge(int i) const { return edge >> i & 1; }
};

// Rows a thread has on their way, and its ring of slots for ARRAYS inputs:
// slot (stage, array, i) of a thread is BYTES from its neighbours', so a warp's
// accesses are contiguous.
template <class T, int V, int N, int TPR, int ARRAYS>
struct Ring {
    static constexpr int THREADS = ln_threads(TPR);
    static constexpr int ROW = ARRAYS * N * THREADS * Slot<T, V>::BYTES;
    static constexpr int DEEP = 65536 / ROW;
    static constexpr int STAGES = DEEP > 4 ? 4 : DEEP < 2 ? 2 : DEEP;
    static constexpr int BYTES = STAGES * ROW;
    static __device__ __forceinline__ unsigned char *slot(unsigned char *ring, int stage,
                                                          int array, int i) {
        return ring +
               (size_t((stage * ARRAYS + array) * N + i) * THREADS + threadIdx.x) *
                   Slot<T, V>::BYTES;
    }
    static __device__ __forceinline__ void close() {
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // the oldest of STAGES rows is there
    static __device__ __forceinline__ void wait() {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    }
};

template <class WT, int V>
__device__ __forceinline__ void load_param(const void *p, int col, int C, float fill, float *v) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        v[e] = fill;
        if (p != nullptr && col + e >= 0 && col + e < C)
            Vec<WT, 1>::load(static_cast<const WT *>(p) + col + e, v + e);
    }
}

// A thread takes the vectors t, t + TPR, ... (N of V elements) that cover its
// row; vector i has the columns V (t + i TPR) - shift and on.  A slot is filled
// again once the row's first sum has used what was in it.
template <class T, class WT, int V, int N, int TPR>
__global__ void __launch_bounds__(ln_threads(TPR)) ln_forward_kernel(const LnArgs a) {
    constexpr int THREADS = ln_threads(TPR), RPB = THREADS / TPR;
    __shared__ float red[THREADS / 32];
    const int t = threadIdx.x % TPR;
    const int64_t step = int64_t(gridDim.x) * RPB, total = a.rows * a.C;
    int64_t row = int64_t(blockIdx.x) * RPB + threadIdx.x / TPR;
    const Columns<V, N, TPR> c(t, V > 1 ? int(row * a.C % V) : 0, a.C);
    int64_t at = row * a.C + c.first;  // the thread's first vector
    const int64_t stride = step * a.C;
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.y);
    using R = Ring<T, V, N, TPR, 1>;
    extern __shared__ __align__(16) unsigned char ring[];
    auto fetch = [&](int ahead, int stage) {
        if (row + ahead * step < a.rows) {
            const int64_t f = at + ahead * stride;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (c.is_live(i))
                    Slot<T, V>::copy(R::slot(ring, stage, 0, i), x + f + i * TPR * V,
                                     c.is_edge(i), total - (f + i * TPR * V));
        }
        R::close();
    };
#pragma unroll
    for (int i = 0; i < R::STAGES; ++i) fetch(i, i);
    float w[N][V], b[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        load_param<WT, V>(a.w, c.col(i), a.C, 1.0f, w[i]);
        load_param<WT, V>(a.b, c.col(i), a.C, 0.0f, b[i]);
    }
    // the groups of a warp go round together: they share its shuffles
    const int64_t rounds = (a.rows + step - 1) / step;
    const float inv_c = 1.0f / float(a.C);
    int stage = 0;
    for (int64_t k = 0; k < rounds; ++k, row += step, at += stride) {
        const bool in = row < a.rows;
        float v[N][V];
        float s = 0.0f;
        R::wait();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            Slot<T, V>::get(R::slot(ring, stage, 0, i), v[i]);
            if (c.is_edge(i)) Slot<T, V>::zero(c.col(i), a.C, v[i]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) s += v[i][e];
        const float mean = row_sum<TPR>(s, red) * inv_c;
        fetch(R::STAGES, stage);
        stage = stage + 1 == R::STAGES ? 0 : stage + 1;
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] -= mean;
            if (c.is_edge(i)) Slot<T, V>::zero(c.col(i), a.C, v[i]);
#pragma unroll
            for (int e = 0; e < V; ++e) q = fmaf(v[i][e], v[i][e], q);
        }
        const float rstd = inv_sqrt(fmaf(row_sum<TPR>(q, red), inv_c, a.eps));
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] = fmaf(v[i][e] * rstd, w[i][e], b[i][e]);
            if (in && c.is_live(i))
                Slot<T, V>::store(y + at + i * TPR * V, c.is_edge(i), c.col(i), a.C, v[i]);
        }
        if (in && t == 0 && a.mean != nullptr) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
    }
}

template <class T, class WT, int V, int N, int TPR>
__global__ void __launch_bounds__(ln_threads(TPR)) ln_backward_kernel(const LnArgs a) {
    constexpr int THREADS = ln_threads(TPR), RPB = THREADS / TPR;
    __shared__ float red[THREADS / 32];
    using R = Ring<T, V, N, TPR, 2>;
    extern __shared__ __align__(16) unsigned char ring[];
    const int t = threadIdx.x % TPR;
    const int64_t step = int64_t(gridDim.x) * RPB, total = a.rows * a.C;
    int64_t row = int64_t(blockIdx.x) * RPB + threadIdx.x / TPR;
    const Columns<V, N, TPR> c(t, V > 1 ? int(row * a.C % V) : 0, a.C);
    int64_t at = row * a.C + c.first;  // the thread's first vector
    const int64_t stride = step * a.C;
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
    T *dx = static_cast<T *>(a.y);
    float mean_n = 0.0f, rstd_n = 0.0f;
    auto fetch = [&](int ahead, int stage) {
        if (row + ahead * step < a.rows) {
            const int64_t f = at + ahead * stride;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (c.is_live(i)) {
                    const int64_t g = f + i * TPR * V;
                    Slot<T, V>::copy(R::slot(ring, stage, 0, i), x + g, c.is_edge(i), total - g);
                    Slot<T, V>::copy(R::slot(ring, stage, 1, i), dy + g, c.is_edge(i), total - g);
                }
        }
        R::close();
    };
    auto stats = [&](int64_t r) {
        if (r < a.rows) mean_n = a.mean[r], rstd_n = a.rstd[r];
    };
#pragma unroll
    for (int i = 0; i < R::STAGES; ++i) fetch(i, i);
    stats(row);
    float dw[N][V], db[N][V], w[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        load_param<WT, V>(a.w, c.col(i), a.C, 1.0f, w[i]);
#pragma unroll
        for (int e = 0; e < V; ++e) dw[i][e] = db[i][e] = 0.0f;
    }
    const float inv_c = 1.0f / float(a.C);
    const int64_t rounds = (a.rows + step - 1) / step;
    int stage = 0;
    for (int64_t k = 0; k < rounds; ++k, row += step, at += stride) {
        const bool in = row < a.rows;
        R::wait();
        float xv[N][V], gv[N][V];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            Slot<T, V>::get(R::slot(ring, stage, 0, i), xv[i]);
            Slot<T, V>::get(R::slot(ring, stage, 1, i), gv[i]);
            if (c.is_edge(i)) {
                Slot<T, V>::zero(c.col(i), a.C, xv[i]);
                Slot<T, V>::zero(c.col(i), a.C, gv[i]);
            }
        }
        if (!in) {  // past the rows: nothing was read, no part in the columns' sums
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) xv[i][e] = gv[i][e] = 0.0f;
        }
        const float mean = mean_n, rstd = rstd_n;
        stats(row + step);
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {  // (dy is 0 outside the row)
                const float xh = (xv[i][e] - mean) * rstd;
                dw[i][e] = fmaf(gv[i][e], xh, dw[i][e]);
                db[i][e] += gv[i][e];
                const float g = gv[i][e] * w[i][e];
                s0 += g;
                s1 = fmaf(g, xh, s1);
                xv[i][e] = xh;
                gv[i][e] = g;
            }
        const float c0 = row_sum<TPR>(s0, red) * inv_c;
        fetch(R::STAGES, stage);
        stage = stage + 1 == R::STAGES ? 0 : stage + 1;
        const float c1 = row_sum<TPR>(s1, red) * inv_c;
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < V; ++e) xv[i][e] = rstd * (gv[i][e] - fmaf(xv[i][e], c1, c0));
            if (in && c.is_live(i))
                Slot<T, V>::store(dx + at + i * TPR * V, c.is_edge(i), c.col(i), a.C, xv[i]);
        }
    }
    if (a.part == nullptr) return;
    float *part = a.part + size_t(blockIdx.x) * 2 * a.C;
    if (RPB > 1) {
        // the groups' sums side by side in the ring, then a thread a column
        __syncthreads();  // (the ring's last groups of copies are empty)
        constexpr int ROW = V * N * TPR, S = V == 1 ? 1 : 4;
        float *sums = reinterpret_cast<float *>(ring);  // [RPB][2][ROW]
        float *mine = sums + (threadIdx.x / TPR) * 2 * ROW + t * V;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < V; e += S) {
                Vec<float, S>::store(mine + i * TPR * V + e, dw[i] + e);
                Vec<float, S>::store(mine + ROW + i * TPR * V + e, db[i] + e);
            }
        __syncthreads();
        for (int n = threadIdx.x; n < 2 * a.C; n += THREADS) {
            const float *p = sums + (n < a.C ? n : ROW + n - a.C);
            const int64_t first = int64_t(blockIdx.x) * RPB;
            float s = 0.0f;
#pragma unroll
            for (int g = 0; g < RPB; ++g)
                s += p[g * 2 * ROW + (V > 1 ? int((first + g) * a.C % V) : 0)];
            part[n] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int n = c.col(i) + e;
                if (n >= 0 && n < a.C) {
                    part[n] = dw[i][e];
                    part[a.C + n] = db[i][e];
                }
            }
    }
}

// The blocks' partial sums added in a fixed order: a block takes 32 columns,
// its 32 warps every 32nd row of partial sums, then one sum over the warps.
template <class WT>
__global__ void __launch_bounds__(1024)
ln_param_kernel(const float *part, int nparts, int C, WT *dw, WT *db) {
    __shared__ float acc[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < 2 * C)
        for (int p = threadIdx.y; p < nparts; p += 32) s += part[size_t(p) * 2 * C + c];
    acc[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < 2 * C) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += acc[i][threadIdx.x];
        WT *out = c < C ? dw : db;
        if (out != nullptr) Vec<WT, 1>::store(out + (c < C ? c : c - C), &s);
    }
}

struct LnLaunch {
    const DeviceInfo *dev;
    cudaStream_t stream;
    bool backward, params;
    // backward with params: the partial sums, one row of 2 C for each block
    void *part;
    int blocks;
};

template <class T, class WT, int V, int N, int TPR>
cudaError_t ln_launch(LnArgs a, LnLaunch &l) {
    constexpr int THREADS = ln_threads(TPR), RPB = THREADS / TPR;
    const int64_t want = (a.rows + RPB - 1) / RPB;
    constexpr int FORWARD = Ring<T, V, N, TPR, 1>::BYTES;
    constexpr int SUMS = RPB > 1 ? RPB * 2 * 4 * V * N * TPR : 0;  // of the block's groups
    constexpr int RING2 = Ring<T, V, N, TPR, 2>::BYTES, BACKWARD = RING2 > SUMS ? RING2 : SUMS;
    // As many blocks as are resident together, at most 8 a SM (which bounds the
    // partial sums); a multiple of 8 where a group takes several rows, so that the
    // rows of a group are a multiple of V apart.
    static std::atomic<uint64_t> allowed[2] = {{0}, {0}};
    cudaError_t e =
        l.backward ? allow_smem(ln_backward_kernel<T, WT, V, N, TPR>, BACKWARD, l.dev->device,
                                allowed[1])
                   : allow_smem(ln_forward_kernel<T, WT, V, N, TPR>, FORWARD, l.dev->device,
                                allowed[0]);
    if (e != cudaSuccess) return e;
    static std::atomic<int> resident[2][64] = {};  // of each device
    std::atomic<int> &kept = resident[l.backward][l.dev->device & 63];
    int per_sm = kept.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        e = l.backward ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                             &per_sm, ln_backward_kernel<T, WT, V, N, TPR>, THREADS, BACKWARD)
                       : cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                             &per_sm, ln_forward_kernel<T, WT, V, N, TPR>, THREADS, FORWARD);
        if (e != cudaSuccess) return e;
        per_sm = per_sm < 1 ? 1 : per_sm > 8 ? 8 : per_sm;
        kept.store(per_sm, std::memory_order_relaxed);
    }
    const int64_t most = (int64_t(l.dev->sm_count) * per_sm + 7) / 8 * 8;
    const unsigned blocks = unsigned(want < most ? want : most);
    if (l.params) {
        e = scratch_alloc(*l.dev, &l.part, size_t(blocks) * 2 * a.C * sizeof(float), l.stream);
        if (e != cudaSuccess) return e;
        a.part = static_cast<float *>(l.part);
        l.blocks = int(blocks);
    }
    if (l.backward)
        ln_backward_kernel<T, WT, V, N, TPR><<<blocks, THREADS, BACKWARD, l.stream>>>(a);
    else
        ln_forward_kernel<T, WT, V, N, TPR><<<blocks, THREADS, FORWARD, l.stream>>>(a);
    return cudaGetLastError();
}

// Vectors a thread holds: the smallest number that covers any row's `vecs`.
template <class T, class WT, int V, int TPR>
cudaError_t ln_pick_n(const LnArgs &a, LnLaunch &l, int vecs) {
    const int n = (vecs + TPR - 1) / TPR;
    constexpr int M = 32 / V;  // at most 32 elements a thread
    if (n <= 1)
        return ln_launch<T, WT, V, 1, TPR>(a, l);
    if (n <= 2)
        return ln_launch<T, WT, V, 2 <= M ? 2 : M, TPR>(a, l);
    if (n <= 3)
        return ln_launch<T, WT, V, 3 <= M ? 3 : M, TPR>(a, l);
    if (n <= 4)
        return ln_launch<T, WT, V, 4 <= M ? 4 : M, TPR>(a, l);
    if (n <= 5)
        return ln_launch<T, WT, V, 5 <= M ? 5 : M, TPR>(a, l);
    if (n <= 6)
        return ln_launch<T, WT, V, 6 <= M ? 6 : M, TPR>(a, l);
    return ln_launch<T, WT, V, M, TPR>(a, l);
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <class T, class WT>
cudaError_t ln_pick_v(const LnArgs &a, LnLaunch &l) {
    constexpr int W = 16 / sizeof(T);
    // a row that starts at any offset may touch one vector more
    const int vecs = a.C % W == 0 ? a.C / W : (a.C + 2 * W - 2) / W;
    if (aligned(a.x, 16) && aligned(a.y, 16) && aligned(a.dy, 16) && vecs <= 256 * (32 / W)) {
        if (vecs <= 8 * (16 / W))
            return ln_pick_n<T, WT, W, 8>(a, l, vecs);
        if (vecs <= 32 * (32 / W)) return ln_pick_n<T, WT, W, 32>(a, l, vecs);
        return ln_pick_n<T, WT, W, 256>(a, l, vecs);
    }
    return a.C <= 32 * 32 ? ln_launch<T, WT, 1, 32, 32>(a, l)
                          : ln_launch<T, WT, 1, 32, 256>(a, l);
}

cudaError_t ln_dispatch(const LnArgs &a, int dtype, int param_dtype, LnLaunch &l) {
    if (dtype == PC_F32) return ln_pick_v<float, float>(a, l);
    if (param_dtype == PC_F32) return ln_pick_v<bf16, float>(a, l);
    return ln_pick_v<bf16, bf16>(a, l);
}

int ln_check(const char *what, int dtype, int param_dtype, int64_t rows, int64_t C) {
    char m[160];
    if (rows < 0 || C < 0) {
        std::snprintf(m, sizeof(m), "%s: negative size", what);
        return api_fail(PC_ERR_INVALID_ARGUMENT, m);
    }
    if ((dtype != PC_F32 && dtype != PC_BF16) ||
        (param_dtype != PC_F32 && param_dtype != dtype)) {
        std::snprintf(m, sizeof(m),
                      "%s: dtype must be PC_F32 or PC_BF16 and param_dtype PC_F32 or dtype "
                      "(got %d, %d)", what, dtype, param_dtype);
        return api_fail(PC_ERR_INVALID_ARGUMENT, m);
    }
    if (C > LN_MAX_C || rows > (int64_t(1) << 31) - 1) {
        std::snprintf(m, sizeof(m), "%s: C=%lld above %d or rows=%lld beyond 32 bits", what,
                      (long long)C, LN_MAX_C, (long long)rows);
        return api_fail(PC_ERR_UNSUPPORTED, m);
    }
    return PC_OK;
}

int ln_cuda(const char *what, cudaError_t e) {
    if (e == cudaSuccess) return PC_OK;
    char m[200];
    std::snprintf(m, sizeof(m), "%s: %s", what, cudaGetErrorString(e));
    return api_fail(PC_ERR_CUDA, m);
}

}  // namespace
}  // namespace pcn

extern "C" int pc_layer_norm(const void *x, int dtype, int64_t rows, int64_t C,
                             const void *weight, const void *bias, int param_dtype,
                             double eps, void *out, float *out_mean, float *out_rstd,
                             void *stream) {
    using namespace pcn;
    int rc = ln_check("layer_norm", dtype, param_dtype, rows, C);
    if (rc != PC_OK) return rc;
    if (!(eps >= 0.0 && eps <= 1e30))
        return api_fail(PC_ERR_INVALID_ARGUMENT, "layer_norm: eps must be finite and >= 0");
    if ((out_mean == nullptr) != (out_rstd == nullptr))
        return api_fail(PC_ERR_INVALID_ARGUMENT,
                        "layer_norm: out_mean and out_rstd go together");
    if (rows == 0 || C == 0) return PC_OK;
    const DeviceInfo *dev = nullptr;
    if ((rc = api_current_device(&dev)) != PC_OK) return rc;
    const int d = dev->device;
    const size_t es = dtype == PC_F32 ? 4 : 2, ps = param_dtype == PC_F32 ? 4 : 2;
    if ((rc = api_check_ptr(x, d, es, "x")) != PC_OK) return rc;
    if ((rc = api_check_ptr(out, d, es, "out")) != PC_OK) return rc;
    if (weight && (rc = api_check_ptr(weight, d, ps, "weight")) != PC_OK) return rc;
    if (bias && (rc = api_check_ptr(bias, d, ps, "bias")) != PC_OK) return rc;
    if (out_mean) {
        if ((rc = api_check_ptr(out_mean, d, 4, "out_mean")) != PC_OK) return rc;
        if ((rc = api_check_ptr(out_rstd, d, 4, "out_rstd")) != PC_OK) return rc;
    }
    LnArgs a{};
    a.x = x, a.w = weight, a.b = bias, a.y = out, a.mean = out_mean, a.rstd = out_rstd;
    a.rows = rows, a.C = int(C), a.eps = float(eps);
    LnLaunch l{dev, static_cast<cudaStream_t>(stream), false, false, nullptr, 0};
    return ln_cuda("layer_norm", ln_dispatch(a, dtype, param_dtype, l));
}

extern "C" int pc_layer_norm_backward(const void *grad_out, const void *x, int dtype,
                                      int64_t rows, int64_t C, const float *mean,
                                      const float *rstd, const void *weight,
                                      int param_dtype, void *grad_x, void *grad_weight,
                                      void *grad_bias, void *stream) {
    using namespace pcn;
    int rc = ln_check("layer_norm_backward", dtype, param_dtype, rows, C);
    if (rc != PC_OK) return rc;
    if (C == 0) return PC_OK;
    if (rows == 0 && grad_weight == nullptr && grad_bias == nullptr) return PC_OK;
    const DeviceInfo *dev = nullptr;
    if ((rc = api_current_device(&dev)) != PC_OK) return rc;
    const int d = dev->device;
    const size_t es = dtype == PC_F32 ? 4 : 2, ps = param_dtype == PC_F32 ? 4 : 2;
    if (rows > 0) {
        if ((rc = api_check_ptr(grad_out, d, es, "grad_out")) != PC_OK) return rc;
        if ((rc = api_check_ptr(x, d, es, "x")) != PC_OK) return rc;
        if ((rc = api_check_ptr(mean, d, 4, "mean")) != PC_OK) return rc;
        if ((rc = api_check_ptr(rstd, d, 4, "rstd")) != PC_OK) return rc;
        if ((rc = api_check_ptr(grad_x, d, es, "grad_x")) != PC_OK) return rc;
    }
    if (weight && (rc = api_check_ptr(weight, d, ps, "weight")) != PC_OK) return rc;
    if (grad_weight && (rc = api_check_ptr(grad_weight, d, ps, "grad_weight")) != PC_OK)
        return rc;
    if (grad_bias && (rc = api_check_ptr(grad_bias, d, ps, "grad_bias")) != PC_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool params = grad_weight != nullptr || grad_bias != nullptr;
    LnArgs a{};
    a.x = x, a.dy = grad_out, a.w = weight, a.y = grad_x;
    a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
    a.rows = rows, a.C = int(C);
    LnLaunch l{dev, st, true, params && rows > 0, nullptr, 0};
    cudaError_t e = rows > 0 ? ln_dispatch(a, dtype, param_dtype, l) : cudaSuccess;
    if (e == cudaSuccess && params) {
        const unsigned g = unsigned((2 * C + 31) / 32);
        const float *part = static_cast<const float *>(l.part);
        if (param_dtype == PC_F32)
            ln_param_kernel<float><<<g, dim3(32, 32), 0, st>>>(
                part, l.blocks, int(C), static_cast<float *>(grad_weight),
                static_cast<float *>(grad_bias));
        else
            ln_param_kernel<bf16><<<g, dim3(32, 32), 0, st>>>(
                part, l.blocks, int(C), static_cast<bf16 *>(grad_weight),
                static_cast<bf16 *>(grad_bias));
        e = cudaGetLastError();
    }
    if (l.part != nullptr) {
        const cudaError_t f = scratch_free(l.part, st);
        if (e == cudaSuccess) e = f;
    }
    return ln_cuda("layer_norm_backward", e);
}
