// pc_group_norm_cl.cu -- group norm of clouds that fit the shared memory of a
// thread block cluster: everything read once, in one launch.
//
// The blocks of a cluster (1 to 16) share the valid rows of a cloud.  Each copies
// its rows, one contiguous piece of memory, into shared memory (bulk copies in
// up to eight pieces, so that the sums of the first run under the copies of the
// others; fewer than 16 bytes at either end, where the rows do not start or end on a
// 16-byte boundary, by plain loads), sums them as the kernels of
// pc_group_norm.cu do, reads the other blocks' group sums from their shared memory
// after a cluster barrier, joins all of them in the order of the blocks, and writes its
// rows' results from shared memory.  Backward the same with x and grad_out; the
// channels' sums for the parameters' gradients go to global memory and are added
// by a second kernel.
//
// Bound: latency of the copy, the barrier and the store, then instructions.  Measured, 16
// ragged clouds of up to 1024 x 384 bfloat16: forward 17 us (6 blocks a cloud), backward 21
// us (9; 22 and 28 us by the kernels for any size); 64 x 384 8 us.
#include "pc_device.cuh"
#include "pc_group_norm.cuh"
#include "pc_launch.cuh"
#include "pointcloud.h"

namespace pcn {
namespace {

constexpr int CT = 512;      // threads
constexpr int PIECES = 8;    // at most

struct ClArgs {
    GnArgs a;
    int K, room;             // blocks of a cluster; bytes of a slab in shared memory
    bool withhold;
    uint64_t timeout_ns;
    int *status;
};

// A block's rows of one array on their way to shared memory.
struct Slab {
    const unsigned char *g0, *a0, *a1;  // the rows; their 16-byte aligned inside [a0, a1)
    unsigned char *at;                  // where the first row lands
    uint64_t *bars;
    int row, n, pieces;                 // bytes of a row, rows
    // `batch`: rows that all threads take in one go; a piece has at least as many
    __device__ __forceinline__ Slab(const void *p, int64_t first, int rows, int row_bytes,
                                    unsigned char *room, uint64_t *bars_, int batch)
        : bars(bars_), row(row_bytes), n(rows), pieces(max(1, min(PIECES, rows / batch))) {
        g0 = static_cast<const unsigned char *>(p) + first * row_bytes;
        const uintptr_t u = reinterpret_cast<uintptr_t>(g0), e = u + uintptr_t(n) * row;
        at = room + (u & 15);
        uintptr_t s = (u + 15) & ~uintptr_t(15), t = e & ~uintptr_t(15);
        if (s > e) s = e;
        if (t < s) t = s;
        a0 = reinterpret_cast<const unsigned char *>(s);
        a1 = reinterpret_cast<const unsigned char *>(t);
    }
    // the end of piece j, a multiple of 16 bytes behind a0
    __device__ __forceinline__ const unsigned char *bound(int j) const {
        return j >= pieces - 1 ? a1 : a0 + unsigned(a1 - a0) / 16 * (j + 1) / unsigned(pieces) * 16;
    }
    // One thread: all copies (or none, a testing hook).
    __device__ __forceinline__ void issue(bool withhold) const {
        const unsigned char *s = a0;
        for (int j = 0; j < pieces; ++j) {
            const unsigned char *e = bound(j);
            const unsigned bytes = unsigned(e - s);
            if (!withhold) {
                mbar_arrive_expect_tx(&bars[j], bytes);
                if (bytes) bulk_g2s(at + (s - g0), s, bytes, &bars[j]);
            }
            s = e;
        }
    }
    // All threads: the bytes outside the aligned inside, elements of E bytes.
    template <int E>
    __device__ __forceinline__ void edges(int t) const {
        const int head = int(a0 - g0) / E, end = n * row / E, tail = int(a1 - g0) / E;
        const int i = t < head ? t : t >= 16 && tail + (t - 16) < end ? tail + (t - 16) : -1;
        if (t >= 32 || i < 0) return;
        if (E == 2)
            reinterpret_cast<uint16_t *>(at)[i] = reinterpret_cast<const uint16_t *>(g0)[i];
        else
            reinterpret_cast<uint32_t *>(at)[i] = reinterpret_cast<const uint32_t *>(g0)[i];
    }
    // the rows that are there after piece j
    __device__ __forceinline__ int rows(int j) const {
        return j >= pieces - 1 ? n : n == 0 ? 0 : int(bound(j) - g0) / row;
    }
};

__device__ __forceinline__ float ld_cluster(const float *p, unsigned rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_shared_rank(p, rank))
                 : "memory");
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A thread's vector of channels and its rows r, r + R, ...
template <int V>
struct ClPlace {
    int tpr, R, r, c;
    bool on;
    __device__ __forceinline__ explicit ClPlace(int C) {
        tpr = C / V, R = CT / tpr;
        r = int(threadIdx.x) / tpr;
        c = (int(threadIdx.x) - r * tpr) * V;
        on = r < R;
    }
};

// Shared memory behind the slabs: barriers, the threads' exchange, the groups' values.
struct ClShared {
    uint64_t *bars;
    float *count, *red, *g1, *g2, *g3, *g4;
    __device__ __forceinline__ ClShared(unsigned char *p, int G, int exchange) {
        bars = reinterpret_cast<uint64_t *>(p);
        count = reinterpret_cast<float *>(p + 2 * PIECES * 8);
        red = count + CT;
        g1 = red + exchange, g2 = g1 + G, g3 = g2 + G, g4 = g3 + G;
    }
};
// floats of the exchange: two a channel for half of the rows of threads, 16-byte aligned
__host__ __device__ inline int cl_exchange(int C, int V) {
    const int R = CT / (C / V), h = R / 2;
    return ((h > 1 ? h : 1) * C * 2 + 3) / 4 * 4;
}

// A copy did not come in time: the block's results are unspecified.  Copies that
// are still under way end before the block does.
__device__ __noinline__ void give_up(const ClArgs &k, uint64_t *bars, int nx, int ndy) {
    raise_status(k.status, PC_ERR_DEVICE_TIMEOUT);
    bool ok = !k.withhold;
    for (int j = 0; j < nx; ++j) ok = ok && mbar_wait_bounded(&bars[j], 0, k.timeout_ns);
    for (int j = 0; j < ndy; ++j)
        ok = ok && mbar_wait_bounded(&bars[PIECES + j], 0, k.timeout_ns);
}

template <class T, int V>
__global__ void __launch_bounds__(CT, 1) gn_cluster_forward_kernel(ClArgs k) {
    extern __shared__ __align__(16) unsigned char smem[];
    const GnArgs &a = k.a;
    constexpr int U = 4;
    const ClShared sh(smem + k.room, a.G, cl_exchange(a.C, V));
    const unsigned rank = k.K > 1 ? cluster_ctarank() : 0;
    const int64_t b = blockIdx.x / unsigned(k.K);
    const int64_t len = gn_len(a, b);
    const GnSplit split(len, k.K);
    const int64_t r0 = split.row(int(rank));
    const int n = split.rows(int(rank));
    const int64_t cloud = b * a.L * a.C;
    const ClPlace<V> p(a.C);
    const Slab x(static_cast<const T *>(a.x) + cloud, r0, n, a.C * int(sizeof(T)), smem, sh.bars,
                 4 * p.R);
    if (threadIdx.x == 0) {
        for (int j = 0; j < PIECES; ++j) mbar_init(&sh.bars[j], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        x.issue(k.withhold && blockIdx.x == 0);
    }
    x.edges<sizeof(T)>(threadIdx.x);
    float wv[V], bv[V];
    int gv[V];
    gn_groups(p.on ? p.c : 0, a.cg, gv);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int c = (p.on ? p.c : 0) + e;
        wv[e] = gn_param<T>(a.w, a.wf32, c, 1.0f);
        bv[e] = gn_param<T>(a.b, a.wf32, c, 0.0f);
    }
    __syncthreads();
    bool ok = true;
    const T *xs = reinterpret_cast<const T *>(x.at) + p.c;
    // the thread's own rows: their mean, then the squares around it.  Means are sums of
    // differences from one of the values, here and below: around a large mean the sums of
    // the values themselves would round by a unit of that at every step.
    float m[V], s[V], base[V];
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = s[e] = base[e] = 0.0f;
    int r = p.r;
    for (int j = 0; j < x.pieces; ++j) {
        ok = ok && mbar_wait_bounded(&sh.bars[j], 0, k.timeout_ns);
        const int end = p.on ? x.rows(j) : 0;
#pragma unroll 4
        for (; r < end; r += p.R) {
            float v[V];
            Vec<T, V>::load(xs + r * a.C, v);
            if (r == p.r)
#pragma unroll
                for (int e = 0; e < V; ++e) base[e] = v[e];
#pragma unroll
            for (int e = 0; e < V; ++e) m[e] += v[e] - base[e];
        }
    }
    float cnt = p.on && n > p.r ? float((n - p.r + p.R - 1) / p.R) : 0.0f;
    if (cnt > 0.0f) {
        const float inv = 1.0f / cnt;
#pragma unroll
        for (int e = 0; e < V; ++e) m[e] = fmaf(m[e], inv, base[e]);
#pragma unroll 4
        for (int i = p.r; i < n; i += p.R) {
            float v[V];
            Vec<T, V>::load(xs + i * a.C, v);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = v[e] - m[e];
                s[e] = fmaf(d, d, s[e]);
            }
        }
    }
    if (!ok) give_up(k, sh.bars, x.pieces, 0);
    // the rows of threads: the upper half gives its moments to the lower, value e of
    // all its threads side by side
    for (int live = p.R; live > 1;) {
        const int h = (live + 1) / 2, step = (live - h) * p.tpr;
        if (p.on && p.r >= h && p.r < live) {
            float *o = sh.red + int(threadIdx.x) - h * p.tpr;
#pragma unroll
            for (int e = 0; e < V; ++e) o[2 * e * step] = m[e], o[(2 * e + 1) * step] = s[e];
            sh.count[p.r - h] = cnt;
        }
        __syncthreads();
        if (p.on && p.r + h < live && sh.count[p.r] > 0.0f) {
            const float *o = sh.red + threadIdx.x;
            const float nb = sh.count[p.r], t = cnt + nb, f = __fdividef(nb, t);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = o[2 * e * step] - m[e];
                s[e] += fmaf(d * d, cnt * f, o[(2 * e + 1) * step]);
                m[e] = fmaf(d, f, m[e]);
            }
            cnt = t;
        }
        __syncthreads();
        live = h;
    }
    if (p.on && p.r == 0) {
        Vec<float, V>::store(sh.red + p.c, m);
        Vec<float, V>::store(sh.red + a.C + p.c, s);
    }
    __syncthreads();
    // the channels of a group, a warp each: all have n values
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int g = warp; g < a.G; g += CT / 32) {
        float sum = 0.0f, sq = 0.0f;
        const float first = sh.red[g * a.cg];
        for (int c = lane; c < a.cg; c += 32) sum += sh.red[g * a.cg + c] - first;
        const float mean = first + warp_sum(sum) / float(a.cg);
        for (int c = lane; c < a.cg; c += 32) {
            const float d = sh.red[g * a.cg + c] - mean;
            sq += fmaf(d * d, float(n), sh.red[a.C + g * a.cg + c]);
        }
        sq = warp_sum(sq);
        if (lane == 0) sh.g1[g] = mean, sh.g2[g] = sq;
    }
    if (k.K > 1)
        cluster_sync_all();
    else
        __syncthreads();
    for (int g = threadIdx.x; g < a.G; g += CT) {
        float mean = 0.0f, sq = 0.0f;
        if (k.K == 1) {
            mean = sh.g1[g], sq = sh.g2[g];
        } else {
            float mi[16], si[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < k.K) mi[i] = ld_cluster(sh.g1 + g, i), si[i] = ld_cluster(sh.g2 + g, i);
            const float rows = 1.0f / fmaxf(float(len), 1.0f);
            // (the first block has rows if any has)
#pragma unroll
            for (int i = 1; i < 16; ++i)
                if (i < k.K && split.rows(i) > 0)
                    mean = fmaf(float(split.rows(i)) * rows, mi[i] - mi[0], mean);
            mean += mi[0];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < k.K) {
                    const float d = mi[i] - mean;
                    const float w = float(split.rows(i));
                    sq += fmaf(d * d, w * float(a.cg), si[i]);
                }
        }
        const float rstd =
            len > 0 ? 1.0f / sqrtf(sq / (float(len) * float(a.cg)) + a.eps) : 0.0f;
        sh.g3[g] = mean, sh.g4[g] = rstd;
        if (rank == 0 && a.mean != nullptr)
            a.mean[b * a.G + g] = mean, a.rstd[b * a.G + g] = rstd;
    }
    __syncthreads();
    if (k.K > 1) cluster_arrive();  // this block has read what it needs
    if (p.on) {
        float mean[V];
#pragma unroll
        for (int e = 0; e < V; ++e) mean[e] = sh.g3[gv[e]], wv[e] *= sh.g4[gv[e]];
        T *y = static_cast<T *>(a.y) + cloud + p.c;
        for (int i = p.r; i < n; i += U * p.R) {
            float v[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * p.R < n) Vec<T, V>::load(xs + (i + u * p.R) * a.C, v[u]);
            act_switch(a.act, [&](auto act) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        v[u][e] = act_value<act.value, sizeof(T) == 2>(
                            fmaf(v[u][e] - mean[e], wv[e], bv[e]));
            });
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * p.R < n) Vec<T, V>::store(y + (r0 + i + u * p.R) * a.C, v[u]);
        }
        // the block's share of the rows past the length
        float zero[V];
#pragma unroll
        for (int e = 0; e < V; ++e) zero[e] = 0.0f;
        const GnSplit past(a.L - len, k.K);
        const int64_t z1 = len + past.row(int(rank) + 1);
        for (int64_t i = len + past.row(int(rank)) + p.r; i < z1; i += p.R)
            Vec<T, V>::store(y + i * a.C, zero);
    }
    if (k.K > 1) {
        __syncwarp();
        cluster_wait();  // the others have read from this block's memory
    }
}

template <class T, int V>
__global__ void __launch_bounds__(CT, 1) gn_cluster_backward_kernel(ClArgs k) {
    extern __shared__ __align__(16) unsigned char smem[];
    let_next_start();
    const GnArgs &a = k.a;
    constexpr int U = V >= 4 ? 2 : 4;
    const ClShared sh(smem + 2 * k.room, a.G, cl_exchange(a.C, V));
    const unsigned rank = k.K > 1 ? cluster_ctarank() : 0;
    const int64_t b = blockIdx.x / unsigned(k.K);
    const int64_t len = gn_len(a, b);
    const GnSplit split(len, k.K);
    const int64_t r0 = split.row(int(rank));
    const int n = split.rows(int(rank));
    const int64_t cloud = b * a.L * a.C;
    const int row = a.C * int(sizeof(T));
    const ClPlace<V> p(a.C);
    const Slab x(static_cast<const T *>(a.x) + cloud, r0, n, row, smem, sh.bars, U * p.R);
    const Slab dy(static_cast<const T *>(a.dy) + cloud, r0, n, row, smem + k.room,
                  sh.bars + PIECES, U * p.R);
    if (threadIdx.x == 0) {
        for (int j = 0; j < 2 * PIECES; ++j) mbar_init(&sh.bars[j], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        x.issue(k.withhold && blockIdx.x == 0);
        dy.issue(k.withhold && blockIdx.x == 0);
    }
    x.edges<sizeof(T)>(threadIdx.x);
    dy.edges<sizeof(T)>(threadIdx.x);
    const GnChannels<T, V> ch(a, b, p.on ? p.c : 0);
    __syncthreads();
    bool ok = true;
    const T *xs = reinterpret_cast<const T *>(x.at) + p.c;
    const T *ds = reinterpret_cast<const T *>(dy.at) + p.c;
    float t1[V], t2[V];
#pragma unroll
    for (int e = 0; e < V; ++e) t1[e] = t2[e] = 0.0f;
    int r = p.r;
    for (int j = 0; j < x.pieces; ++j) {
        ok = ok && mbar_wait_bounded(&sh.bars[j], 0, k.timeout_ns) &&
             mbar_wait_bounded(&sh.bars[PIECES + j], 0, k.timeout_ns);
        const int end = p.on ? min(x.rows(j), dy.rows(j)) : 0;
        for (; r < end; r += U * p.R) {
            // (the rows of a batch past the piece's end are its first ones again, and not added)
            float v[U][V], g[U][V];
            const int q = min(U, (end - r + p.R - 1) / p.R);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = r + (u < q ? u : 0) * p.R;
                Vec<T, V>::load(xs + i * a.C, v[u]);
                Vec<T, V>::load(ds + i * a.C, g[u]);
            }
            ch.form(a.act, v, g);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u < q)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        t1[e] += g[u][e];
                        t2[e] = fmaf(g[u][e], v[u][e], t2[e]);
                    }
            if (q < U) {
                r += q * p.R;
                break;
            }
        }
    }
    if (!ok) give_up(k, sh.bars, x.pieces, x.pieces);
    for (int live = p.R; live > 1;) {
        const int h = (live + 1) / 2, step = (live - h) * p.tpr;
        if (p.on && p.r >= h && p.r < live) {
            float *o = sh.red + int(threadIdx.x) - h * p.tpr;
#pragma unroll
            for (int e = 0; e < V; ++e) o[2 * e * step] = t1[e], o[(2 * e + 1) * step] = t2[e];
        }
        __syncthreads();
        if (p.on && p.r + h < live) {
            const float *o = sh.red + threadIdx.x;
#pragma unroll
            for (int e = 0; e < V; ++e) t1[e] += o[2 * e * step], t2[e] += o[(2 * e + 1) * step];
        }
        __syncthreads();
        live = h;
    }
    if (p.on && p.r == 0) {
        float *part = a.cpart ? a.cpart + (b * k.K + rank) * 2 * a.C + p.c : nullptr;
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (part) part[e] = t1[e], part[a.C + e] = t2[e];
        // (weighted for the groups' sums)
#pragma unroll
        for (int e = 0; e < V; ++e) t1[e] *= ch.w[e], t2[e] *= ch.w[e];
        Vec<float, V>::store(sh.red + p.c, t1);
        Vec<float, V>::store(sh.red + a.C + p.c, t2);
    }
    if (a.y == nullptr) return;  // (the same in all blocks)
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int g = warp; g < a.G; g += CT / 32) {
        float u1 = 0.0f, u2 = 0.0f;
        for (int c = g * a.cg + lane; c < (g + 1) * a.cg; c += 32)
            u1 += sh.red[c], u2 += sh.red[a.C + c];
        u1 = warp_sum(u1), u2 = warp_sum(u2);
        if (lane == 0) sh.g1[g] = u1, sh.g2[g] = u2;
    }
    if (k.K > 1)
        cluster_sync_all();
    else
        __syncthreads();
    const float inv = len > 0 ? 1.0f / (float(len) * float(a.cg)) : 0.0f;
    for (int g = threadIdx.x; g < a.G; g += CT) {
        float u1 = 0.0f, u2 = 0.0f;
        if (k.K == 1) {
            u1 = sh.g1[g], u2 = sh.g2[g];
        } else {
            float q1[16], q2[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < k.K) q1[i] = ld_cluster(sh.g1 + g, i), q2[i] = ld_cluster(sh.g2 + g, i);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < k.K) u1 += q1[i], u2 += q2[i];
        }
        sh.g3[g] = u1 * inv, sh.g4[g] = u2 * inv;
    }
    __syncthreads();
    if (k.K > 1) cluster_arrive();
    if (p.on) {
        float h1[V], h2[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            h1[e] = sh.g3[ch.group[e]], h2[e] = sh.g4[ch.group[e]];
        T *dx = static_cast<T *>(a.y) + cloud + p.c;
        for (int i = p.r; i < n; i += U * p.R) {
            float v[U][V], g[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * p.R < n) {
                    Vec<T, V>::load(xs + (i + u * p.R) * a.C, v[u]);
                    Vec<T, V>::load(ds + (i + u * p.R) * a.C, g[u]);
                }
            ch.form(a.act, v, g);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * p.R < n) {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        v[u][e] = ch.rstd[e] *
                                  (fmaf(g[u][e], ch.w[e], -h1[e]) - v[u][e] * h2[e]);
                    Vec<T, V>::store(dx + (r0 + i + u * p.R) * a.C, v[u]);
                }
        }
        float zero[V];
#pragma unroll
        for (int e = 0; e < V; ++e) zero[e] = 0.0f;
        const GnSplit past(a.L - len, k.K);
        const int64_t z1 = len + past.row(int(rank) + 1);
        for (int64_t i = len + past.row(int(rank)) + p.r; i < z1; i += p.R)
            Vec<T, V>::store(dx + i * a.C, zero);
    }
    if (k.K > 1) {
        __syncwarp();
        cluster_wait();
    }
}

// A span of rows of the channels' sums, 32 columns a block, 32 warps every 32nd row: to a
// row of `next`, or where it is NULL (one span) to dw and db.
template <class T>
__global__ void __launch_bounds__(1024)
gn_param_kernel(const float *part, int64_t nparts, int C, bool f32, void *db, void *dw,
                float *next) {
    let_next_start();
    after_previous();
    __shared__ float acc[32][33];
    const unsigned columns = (2 * C + 31) / 32, span = blockIdx.x / columns;
    const int c = int(blockIdx.x - span * columns) * 32 + threadIdx.x;
    const int64_t p0 = int64_t(span) * GN_SPAN, p1 = min(nparts, p0 + GN_SPAN);
    float s = 0.0f;
    if (c < 2 * C)
#pragma unroll 4
        for (int64_t p = p0 + threadIdx.y; p < p1; p += 32) s += part[p * 2 * C + c];
    acc[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < 2 * C) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += acc[i][threadIdx.x];
        if (next != nullptr) {
            next[int64_t(span) * 2 * C + c] = s;
            return;
        }
        void *out = c < C ? db : dw;
        const int at = c < C ? c : c - C;
        if (out == nullptr) return;
        if (f32)
            static_cast<float *>(out)[at] = s;
        else
            Vec<T, 1>::store(static_cast<T *>(out) + at, &s);
    }
}

template <class T, int V>
cudaError_t run(const DeviceInfo &dev, GnArgs a, bool backward, const GnCluster &p,
                cudaStream_t st) {
    static std::atomic<uint64_t> done[2] = {{0}, {0}};
    const void *fn = backward ? reinterpret_cast<const void *>(gn_cluster_backward_kernel<T, V>)
                              : reinterpret_cast<const void *>(gn_cluster_forward_kernel<T, V>);
    cudaError_t e;
    const uint64_t bit = uint64_t(1) << (dev.device & 63);
    if (!(done[backward].load(std::memory_order_relaxed) & bit)) {
        if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      int(dev.smem_per_block_optin))) != cudaSuccess ||
            (e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) !=
                cudaSuccess)
            return e;
        done[backward].fetch_or(bit, std::memory_order_relaxed);
    }
    void *scratch = nullptr;
    const bool params = backward && (a.dw || a.db);
    const int64_t rows = a.B * p.blocks;
    if (params) {
        const size_t floats = size_t(rows) * 2 * a.C + gn_param_room(rows, a.C);
        if ((e = scratch_alloc(dev, &scratch, floats * sizeof(float), st)) != cudaSuccess) return e;
        a.cpart = static_cast<float *>(scratch);
    }
    ClArgs k{a, p.blocks, p.bytes, (debug_stall() & PC_STALL_GROUP_NORM) != 0, wait_timeout_ns(),
             dev.status_word};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.B * p.blocks));
    cfg.blockDim = dim3(CT);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(p.blocks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.blocks > 1 ? 1 : 0;
    void *args[] = {&k};
    e = cudaLaunchKernelExC(&cfg, fn, args);
    if (e == cudaSuccess && params)
        e = gn_param_sums(a, sizeof(T) == 2 ? PC_BF16 : PC_F32, a.cpart, rows,
                          a.cpart + size_t(rows) * 2 * a.C, st);
    if (scratch) {
        const cudaError_t f = scratch_free(scratch, st);
        if (e == cudaSuccess) e = f;
    }
    return e;
}

// How many clusters of K blocks that fill their SMs run at once (0: none, as may be
// beyond the portable size of 8); asked once for each device and size.
int active_clusters(const DeviceInfo &dev, int K) {
    if (K == 1) return dev.sm_count;
    static std::atomic<int> known[64][17] = {};  // one more than the number
    std::atomic<int> &at = known[dev.device & 63][K];
    int v = at.load(std::memory_order_relaxed);
    if (v > 0) return v - 1;
    const void *fn = reinterpret_cast<const void *>(gn_cluster_backward_kernel<bf16, 8>);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(K);
    cfg.blockDim = dim3(CT);
    cfg.dynamicSmemBytes = dev.smem_per_block_optin;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = K;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(dev.smem_per_block_optin)) != cudaSuccess ||
        cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    at.store(n + 1, std::memory_order_relaxed);
    return n;
}

}  // namespace

size_t gn_param_room(int64_t n, int C) {
    size_t floats = 0;
    while (n > GN_SPAN) {
        n = (n + GN_SPAN - 1) / GN_SPAN;
        floats += size_t(n) * 2 * C;
    }
    return floats;
}

cudaError_t gn_param_sums(const GnArgs &a, int dtype, const float *rows, int64_t n, float *room,
                          cudaStream_t st) {
    const unsigned columns = unsigned((2 * a.C + 31) / 32);
    auto kernel = dtype == PC_F32 ? gn_param_kernel<float> : gn_param_kernel<bf16>;
    while (n > GN_SPAN) {
        const int64_t spans = (n + GN_SPAN - 1) / GN_SPAN;
        const cudaError_t e = launch(true, kernel, unsigned(spans) * columns, dim3(32, 32), 0, st,
                                     rows, n, a.C, a.wf32, a.db, a.dw, room);
        if (e != cudaSuccess) return e;
        rows = room, n = spans;
        room += size_t(spans) * 2 * a.C;
    }
    return launch(true, kernel, columns, dim3(32, 32), 0, st, rows, n, a.C, a.wf32, a.db, a.dw,
                  nullptr);
}

GnCluster gn_cluster_plan(const DeviceInfo &dev, const GnArgs &a, int dtype, int V,
                          bool backward) {
    GnCluster p;
    if (a.C / V > CT || a.L < 1) return p;
    const int64_t row = int64_t(a.C) * (dtype == PC_F32 ? 4 : 2), slabs = backward ? 2 : 1;
    const int64_t behind = 2 * PIECES * 8 + (cl_exchange(a.C, V) + CT + 4 * int64_t(a.G)) * 4;
    auto room = [&](int K) { return ((a.L + K - 1) / K * row + 30) / 16 * 16; };
    // Estimates in us.  A wave of clusters takes a block's values and a part that does not
    // depend on them; the kernels for any size spread the values over all SMs, read them
    // twice and are three launches.  Measured, forward / backward with all gradients:
    // 16 x 1024 x 384 bf16 ragged (6 blocks a cloud in one wave / 9 in two) 16.9 / 23 against
    // 21.9 / 28.2 (4 blocks 20.9, 8 18.5 / 24.6, 12 21.9 / 33, 16 28.8 / 37); 4 x 4093 x 195 bf16 (16 blocks, element by
    // element) 25.9 / 40.4 against 22.8 / 30.9; 1 x 64 x 384 forward 8 against 11.
    const int VB = V * (dtype == PC_F32 ? 4 : 2);
    const double each = (VB >= 16 ? 0.13 : VB >= 8 ? 0.2 : VB >= 4 ? 0.3 : 0.45) / 1000 *
                        (backward ? 1.3 : 1.0);
    double least = (backward ? 16.0 : 12.0) +
                   1.5 * each * double(a.B) * double(a.L) * a.C / dev.sm_count;
    for (int K = 1; K <= 16; ++K) {
        if ((a.L + K - 1) / K > (int64_t(1) << 28) / row) continue;
        const int64_t smem = slabs * room(K) + behind;
        if (smem > int64_t(dev.smem_per_block_optin) || a.B * K > 2147483647) continue;
        const int at_once = active_clusters(dev, K);
        if (at_once == 0) continue;
        // (a last wave that is not full costs less: fewer blocks, often of short clouds)
        const double waves = a.B <= at_once
                                 ? 1.0
                                 : double(a.B / at_once) + (a.B % at_once ? 0.6 : 0.0);
        const double cost = waves * (4.0 + 0.35 * K + each * double((a.L + K - 1) / K) * a.C);
        if (cost < 0.97 * least) {
            least = cost;
            p.blocks = K, p.bytes = int(room(K)), p.smem = size_t(smem);
        }
    }
    return p;
}

cudaError_t gn_cluster_run(const DeviceInfo &dev, GnArgs a, int dtype, int V, bool backward,
                           const GnCluster &p, cudaStream_t st) {
    if (dtype == PC_F32) {
        if (V == 4) return run<float, 4>(dev, a, backward, p, st);
        if (V == 2) return run<float, 2>(dev, a, backward, p, st);
        return run<float, 1>(dev, a, backward, p, st);
    }
    if (V == 8) return run<bf16, 8>(dev, a, backward, p, st);
    if (V == 4) return run<bf16, 4>(dev, a, backward, p, st);
    if (V == 2) return run<bf16, 2>(dev, a, backward, p, st);
    return run<bf16, 1>(dev, a, backward, p, st);
}

}  // namespace pcn
