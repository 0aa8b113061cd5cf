// pc_group_norm.cu -- group norm of channels-last features over each cloud's
// valid points, with an activation, forward and backward.
//
//   n = lengths[b] * C / G,  mean = sum x / n,  var = sum (x - mean)^2 / n,
//   xhat = (x - mean) rstd,  z = xhat w + b,  y = act(z)
//   d = dy act'(z),  g = d w,
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),
//   dw = sum d xhat,  db = sum d   (over clouds and points).
//
// A row of C channels holds all groups and a group reaches over all rows, so
// every pass walks rows: a thread keeps V neighbouring channels (16 bytes
// where C allows) and takes every R-th row of its block's share, a block 256
// threads.  The channels' values (w, b, mean, rstd) stay in registers.
//
// Forward: (1) each block the mean and the sum of squares around it of each
// group over its rows, (2) these joined per group, (3) y.  Sums of squares
// are around means at every step: U rows at a time in registers (their mean,
// then the squares), joined pairwise by
//   n = nA + nB, d = mB - mA, m = mA + d nB / n, S = SA + SB + d^2 nA nB / n,
// so nothing cancels, whatever the mean or an outlier is.
// Backward: (1) each block the sums of d and d xhat of each channel, (2)
// these joined per cloud and channel, (3) dx from the groups' sums, and in
// blocks of their own dw and db.
// No atomics; every join has a fixed order.  Passes run as many blocks as are resident
// together, and (3) walks backwards through its rows.  Clouds that fit a thread block
// cluster take pc_group_norm_cl.cu instead where that is estimated to be shorter.
//
// Bound: memory for large clouds, latency and launches for small ones.  Measured, 100,000 x
// 512 float32: (1) 41 us, (3) 61 us, backward (1) 78 us, (3) 95 us (5.0, 6.7, 5.3 and 6.5
// TB/s); 4 x 4093 x 195 bfloat16 (one element a load): 9, 11, 11 and 16 us.
#include "pc_group_norm.cuh"
#include "pc_launch.cuh"
#include "pointcloud.h"

#include <atomic>
#include <cstdio>

namespace pcn {
namespace {

// V elements written past the caches' other contents.
template <class T, int V>
__device__ __forceinline__ void stream(T *p, const float *v) {
    if constexpr (V * sizeof(T) == 16) {
        float4 t;
        Vec<T, V>::store(reinterpret_cast<T *>(&t), v);
        __stcs(reinterpret_cast<float4 *>(p), t);
    } else {
        Vec<T, V>::store(p, v);
    }
}

// The place of a block: its cloud, chunk of channels, share of the rows; and
// a thread's vector of channels and first row.
template <int V>
struct GnPlace {
    int64_t b;
    int blk, chunk, c0, width, tpr, R, c, r;
    bool on;
    __device__ __forceinline__ GnPlace(const GnArgs &a, int nblk) {
        unsigned i = blockIdx.x;
        blk = int(i % unsigned(nblk)), i /= unsigned(nblk);
        chunk = int(i % unsigned(a.nchunk));
        b = i / unsigned(a.nchunk);
        if (a.per == 0) {
            c0 = chunk * a.width;
            width = min(a.width, a.C - c0);
        } else {
            const int g = chunk / a.per, k = chunk - g * a.per;
            c0 = g * a.cg + k * a.width;
            width = min(a.width, a.cg - k * a.width);
        }
        tpr = width / V;
        R = GN_THREADS / tpr;
        r = int(threadIdx.x) / tpr;
        c = c0 + (int(threadIdx.x) - r * tpr) * V;
        on = r < R;
    }
};

// Forward 1: the pieces' moments over a block's rows.
template <class T, int V>
__global__ void __launch_bounds__(GN_THREADS) gn_stats_kernel(GnArgs a) {
    let_next_start();
    after_previous();
    constexpr int U = 8;  // rows in registers
    __shared__ float sm[GN_THREADS * V], ss[GN_THREADS * V], sn[GN_THREADS];
    const GnPlace<V> p(a, a.nblk);
    const int64_t len = gn_len(a, p.b);
    const GnSplit split(len, a.nblk);
    const int64_t r0 = split.row(p.blk), r1 = split.row(p.blk + 1);
    const T *x = static_cast<const T *>(a.x) + p.b * a.L * a.C + p.c;
    float n = 0.0f, m[V], s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = s[e] = 0.0f;
    if (p.on)
        for (int64_t r = r0 + p.r; r < r1; r += int64_t(U) * p.R) {
            RawV<T, V> raw[U];
            float k = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = r + int64_t(u) * p.R < r1;
                if (in)
                    raw[u] = *reinterpret_cast<const RawV<T, V> *>(x + (r + int64_t(u) * p.R) * a.C);
                k += in ? 1.0f : 0.0f;
            }
            const float inv = 1.0f / k, t = n + k, f = k / t, h = n * f;
            float sum[V], sq[V];
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] = sq[e] = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u < int(k)) {
                    float v[V];
                    widen<T, V>(raw[u], v);
#pragma unroll
                    for (int e = 0; e < V; ++e) sum[e] += v[e];
                }
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] *= inv;  // the mean
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u < int(k)) {
                    float v[V];
                    widen<T, V>(raw[u], v);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float d = v[e] - sum[e];
                        sq[e] = fmaf(d, d, sq[e]);
                    }
                }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = sum[e] - m[e];
                s[e] += fmaf(d * d, h, sq[e]);
                m[e] = fmaf(d, f, m[e]);
            }
            n = t;
        }
    // the block's rows, halves joined to halves
    const int at = int(threadIdx.x) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) sm[at + e] = m[e], ss[at + e] = s[e];
    sn[threadIdx.x] = p.on ? n : 0.0f;
    __syncthreads();
    for (int k = p.R; k > 1;) {
        const int h = (k + 1) / 2;
        if (p.on && p.r + h < k) {
            const int o = int(threadIdx.x) + h * p.tpr;
            const float nb = sn[o], t = n + nb;
            if (nb > 0.0f) {
                const float f = nb / t;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = sm[o * V + e] - m[e];
                    s[e] += fmaf(d * d, n * f, ss[o * V + e]);
                    m[e] = fmaf(d, f, m[e]);
                    sm[at + e] = m[e], ss[at + e] = s[e];
                }
                n = t;
                sn[threadIdx.x] = n;
            }
        }
        __syncthreads();
        k = h;
    }
    // the channels of a group, or of the group's part that the block has, by a warp
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const float rows = float(r1 - r0);
    const int each = a.per ? p.width : a.cg;
    float2 *out = a.gpart + (p.b * a.nblk + p.blk) * (a.per ? a.nchunk : a.G) +
                  (a.per ? p.chunk : p.c0 / a.cg);
    for (int g = warp; g < p.width / each; g += GN_THREADS / 32) {
        Moments t;
        for (int c = lane; c < each; c += 32)
            t.join(rows, sm[g * each + c], ss[g * each + c]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float nb = __shfl_down_sync(~0u, t.n, o), mb = __shfl_down_sync(~0u, t.m, o),
                        sb = __shfl_down_sync(~0u, t.s, o);
            t.join(nb, mb, sb);
        }
        if (lane == 0) out[g] = make_float2(t.m, t.s);
    }
}

// Forward 2: a group's moments over all blocks; a block per cloud and group.
__global__ void __launch_bounds__(128) gn_join_kernel(GnArgs a) {
    let_next_start();
    after_previous();
    const int64_t bg = blockIdx.x, b = bg / a.G;
    const int g = int(bg % a.G), per = a.per ? a.per : 1, all = a.G * per;
    const int64_t len = gn_len(a, b);
    const GnSplit split(len, a.nblk);
    Moments t;
    for (int i = threadIdx.x; i < a.nblk * per; i += 128) {
        const int blk = i / per, k = i % per;
        const float2 v = a.gpart[(b * a.nblk + blk) * all + g * per + k];
        const int each = a.per ? min(a.width, a.cg - k * a.width) : a.cg;
        t.join(float(split.rows(blk)) * float(each), v.x, v.y);
    }
    __shared__ float red[3][4];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float nb = __shfl_down_sync(~0u, t.n, o), mb = __shfl_down_sync(~0u, t.m, o),
                    sb = __shfl_down_sync(~0u, t.s, o);
        t.join(nb, mb, sb);
    }
    if (lane == 0) red[0][warp] = t.n, red[1][warp] = t.m, red[2][warp] = t.s;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < 4; ++i) t.join(red[0][i], red[1][i], red[2][i]);
        a.mean[bg] = t.m;
        a.rstd[bg] = len > 0 ? 1.0f / sqrtf(t.s / t.n + a.eps) : 0.0f;
    }
}

// Forward 3
template <class T, int V>
__global__ void __launch_bounds__(GN_THREADS) gn_apply_kernel(GnArgs a, int nblk) {
    let_next_start();
    after_previous();
    constexpr int U = V >= 4 ? 4 : 8;
    const GnPlace<V> p(a, nblk);
    if (!p.on) return;
    const int64_t len = gn_len(a, p.b);
    const GnSplit split(a.L, nblk);
    const int64_t r0 = split.row(p.blk), r1 = split.row(p.blk + 1);
    const int64_t at = p.b * a.L * a.C + p.c;
    const T *x = static_cast<const T *>(a.x) + at;
    T *y = static_cast<T *>(a.y) + at;
    float mean[V], f[V], o[V];
    int group[V];
    gn_groups(p.c, a.cg, group);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int64_t g = p.b * a.G + group[e];
        mean[e] = a.mean[g];
        f[e] = a.rstd[g] * gn_param<T>(a.w, a.wf32, p.c + e, 1.0f);
        o[e] = gn_param<T>(a.b, a.wf32, p.c + e, 0.0f);
    }
    // from the end, where the second level cache still has what the first pass read
    const int64_t step = int64_t(U) * p.R, first = r0 + p.r;
    for (int64_t r = first < r1 ? first + (r1 - 1 - first) / step * step : -1; r >= first;
         r -= step) {
        float v[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r + int64_t(u) * p.R < r1 && r + int64_t(u) * p.R < len)
                Vec<T, V>::load(x + (r + int64_t(u) * p.R) * a.C, v[u]);
        act_switch(a.act, [&](auto act) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    v[u][e] = act_value<act.value, sizeof(T) == 2>(
                        fmaf(v[u][e] - mean[e], f[e], o[e]));
        });
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = r + int64_t(u) * p.R;
            if (i >= len)
#pragma unroll
                for (int e = 0; e < V; ++e) v[u][e] = 0.0f;
            if (i < r1) stream<T, V>(y + i * a.C, v[u]);
        }
    }
}

// Backward 1: the channels' sums of d and d xhat over a block's rows.
template <class T, int V>
__global__ void __launch_bounds__(GN_THREADS) gn_sums_kernel(GnArgs a) {
    let_next_start();
    after_previous();
    constexpr int U = 2;  // rows in flight
    __shared__ float s1[GN_THREADS * V], s2[GN_THREADS * V];
    const GnPlace<V> p(a, a.nblk);
    const int64_t len = gn_len(a, p.b);
    const GnSplit split(len, a.nblk);
    const int64_t r0 = split.row(p.blk), r1 = split.row(p.blk + 1);
    const int64_t at = p.b * a.L * a.C + p.c;
    const T *x = static_cast<const T *>(a.x) + at, *dy = static_cast<const T *>(a.dy) + at;
    float t1[V], t2[V];
#pragma unroll
    for (int e = 0; e < V; ++e) t1[e] = t2[e] = 0.0f;
    if (p.on) {
        const GnChannels<T, V> ch(a, p.b, p.c);
        for (int64_t r = r0 + p.r; r < r1; r += int64_t(U) * p.R) {
            RawV<T, V> rx[U], rg[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + int64_t(u) * p.R < r1) {
                    const int64_t i = (r + int64_t(u) * p.R) * a.C;
                    rx[u] = *reinterpret_cast<const RawV<T, V> *>(x + i);
                    rg[u] = *reinterpret_cast<const RawV<T, V> *>(dy + i);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + int64_t(u) * p.R < r1) {
                    float v[1][V], g[1][V];
                    widen<T, V>(rx[u], v[0]);
                    widen<T, V>(rg[u], g[0]);
                    ch.template form<1>(a.act, v, g);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        t1[e] += g[0][e];
                        t2[e] = fmaf(g[0][e], v[0][e], t2[e]);
                    }
                }
        }
    }
    const int o = int(threadIdx.x) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) s1[o + e] = t1[e], s2[o + e] = t2[e];
    __syncthreads();
    for (int k = p.R; k > 1;) {
        const int h = (k + 1) / 2;
        if (p.on && p.r + h < k) {
            const int q = o + h * p.tpr * V;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                t1[e] += s1[q + e], t2[e] += s2[q + e];
                s1[o + e] = t1[e], s2[o + e] = t2[e];
            }
        }
        __syncthreads();
        k = h;
    }
    float *out = a.cpart + (p.b * a.nblk + p.blk) * 2 * a.C + p.c0;
    for (int c = threadIdx.x; c < p.width; c += GN_THREADS) out[c] = s1[c], out[a.C + c] = s2[c];
}

// Backward 2: the blocks' sums added up, per cloud and channel; 32 columns a
// block, 32 warps every 32nd of the blocks' sums.
__global__ void __launch_bounds__(1024) gn_channel_kernel(GnArgs a) {
    let_next_start();
    after_previous();
    __shared__ float acc[32][33];
    const int cols = (2 * a.C + 31) / 32;
    const int64_t b = blockIdx.x / cols;
    const int c = int(blockIdx.x % cols) * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < 2 * a.C)
        for (int i = threadIdx.y; i < a.nblk; i += 32)
            s += a.cpart[(b * a.nblk + i) * 2 * a.C + c];
    acc[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < 2 * a.C) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += acc[i][threadIdx.x];
        a.chan[b * 2 * a.C + c] = s;
    }
}

// Up to as many clouds a thread adds dw and db one cloud after the other, in blocks of
// the last kernel; for more in kernels of their own (gn_param_sums): 8192 clouds of
// 32 x 128 bfloat16 took 836 us with all of them in one thread's chain, 571 us so.
constexpr int PARAM_CLOUDS = 64;

// Backward 3: dx.  The last `nparam` blocks add the channels' sums over the clouds,
// of which there are few (PARAM_CLOUDS) then: dw and db.
template <class T, int V>
__global__ void __launch_bounds__(GN_THREADS) gn_dx_kernel(GnArgs a, int nblk, int nparam) {
    let_next_start();
    after_previous();
    constexpr int U = V >= 4 ? 2 : 4;
    if (blockIdx.x >= gridDim.x - nparam) {
        const int c = int(blockIdx.x - (gridDim.x - nparam)) * GN_THREADS + threadIdx.x;
        if (c >= 2 * a.C) return;
        float s = 0.0f;
        for (int64_t b = 0; b < a.B; ++b) s += a.chan[b * 2 * a.C + c];
        void *out = c < a.C ? a.db : a.dw;
        const int at = c < a.C ? c : c - a.C;
        if (out == nullptr) return;
        if (a.wf32)
            static_cast<float *>(out)[at] = s;
        else
            Vec<T, 1>::store(static_cast<T *>(out) + at, &s);
        return;
    }
    // the groups' means of g and g xhat: a warp for a group, or several for few groups
    __shared__ float m1[GN_THREADS * V], m2[GN_THREADS * V], q1[8], q2[8];
    const GnPlace<V> p(a, nblk);
    const int64_t len = gn_len(a, p.b);
    const float inv = len > 0 ? 1.0f / (float(len) * float(a.cg)) : 0.0f;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g0 = p.c0 / a.cg, g1 = (p.c0 + p.width - 1) / a.cg;
    const float *chan = a.chan + p.b * 2 * a.C;
    const int ng = g1 - g0 + 1, wpg = ng < 8 ? 8 / ng : 1;
    for (int g = g0 + warp / wpg; g <= g1; g += 8 / wpg) {
        float u1 = 0.0f, u2 = 0.0f;
        const int end = (g + 1) * a.cg;
#pragma unroll 4
        for (int c = g * a.cg + warp % wpg * 32 + lane; c < end; c += 32 * wpg) {
            const float w = gn_param<T>(a.w, a.wf32, c, 1.0f);
            u1 = fmaf(w, chan[c], u1);
            u2 = fmaf(w, chan[a.C + c], u2);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            u1 += __shfl_xor_sync(~0u, u1, o);
            u2 += __shfl_xor_sync(~0u, u2, o);
        }
        if (wpg == 1 && lane == 0) m1[g - g0] = u1 * inv, m2[g - g0] = u2 * inv;
        if (wpg > 1 && lane == 0) q1[warp] = u1, q2[warp] = u2;  // (one round of the loop)
    }
    if (wpg > 1) {
        __syncthreads();
        if (threadIdx.x < ng) {
            float u1 = 0.0f, u2 = 0.0f;
            for (int i = 0; i < wpg; ++i)
                u1 += q1[threadIdx.x * wpg + i], u2 += q2[threadIdx.x * wpg + i];
            m1[threadIdx.x] = u1 * inv, m2[threadIdx.x] = u2 * inv;
        }
    }
    __syncthreads();
    if (!p.on) return;
    const GnSplit split(a.L, nblk);
    const int64_t r0 = split.row(p.blk), r1 = split.row(p.blk + 1);
    const int64_t at = p.b * a.L * a.C + p.c;
    const T *x = static_cast<const T *>(a.x) + at, *dy = static_cast<const T *>(a.dy) + at;
    T *dx = static_cast<T *>(a.y) + at;
    const GnChannels<T, V> ch(a, p.b, p.c);
    float h1[V], h2[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        h1[e] = m1[ch.group[e] - g0];
        h2[e] = m2[ch.group[e] - g0];
    }
    const int64_t step = int64_t(U) * p.R, first = r0 + p.r;
    for (int64_t r = first < r1 ? first + (r1 - 1 - first) / step * step : -1; r >= first;
         r -= step) {
        float v[U][V], g[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = r + int64_t(u) * p.R;
            if (i < r1 && i < len) {
                Vec<T, V>::load(x + i * a.C, v[u]);
                Vec<T, V>::load(dy + i * a.C, g[u]);
            }
        }
        ch.form(a.act, v, g);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = r + int64_t(u) * p.R;
            float t[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                t[e] = i < len ? ch.rstd[e] *
                                     (fmaf(g[u][e], ch.w[e], -h1[e]) - v[u][e] * h2[e])
                               : 0.0f;
            if (i < r1) stream<T, V>(dx + i * a.C, t);
        }
    }
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

// Channels of a chunk for vectors of V, or 0 where V does not fit: at most 256
// vectors, whole groups or, of groups wider than that, `per` parts of one.
int gn_width(int C, int cg, int V, int *per) {
    const int most = GN_THREADS * V;
    *per = 0;
    if (C % V) return 0;
    if (C <= most) return C;
    const int unit = cg / gcd(cg, V) * V;
    if (unit <= most) return most / unit * unit;
    if (cg % V || cg <= most) return 0;
    *per = (cg + most - 1) / most;
    return ((cg + *per - 1) / *per + V - 1) / V * V;
}

struct GnPlan {
    const DeviceInfo *dev;
    cudaStream_t stream;
    bool backward;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Blocks that share a cloud's rows: as many as are resident together, so that each has
// a long share, and none without a batch of rows.
template <class K>
cudaError_t gn_blocks(K kernel, std::atomic<int> (&resident)[64], const DeviceInfo &dev,
                      int64_t sets, int64_t L, int batch, int *out) {
    std::atomic<int> &kept = resident[dev.device & 63];
    int per_sm = kept.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        const cudaError_t e =
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, GN_THREADS, 0);
        if (e != cudaSuccess) return e;
        per_sm = per_sm < 1 ? 1 : per_sm > 8 ? 8 : per_sm;
        kept.store(per_sm, std::memory_order_relaxed);
    }
    int64_t n = int64_t(dev.sm_count) * per_sm / sets;
    const int64_t want = ceil_div(L, batch);
    if (n > want) n = want;
    *out = int(n < 1 ? 1 : n);
    return cudaSuccess;
}

template <class T, int V>
cudaError_t gn_run(GnArgs a, const GnPlan &p) {
    const int R = GN_THREADS / (a.width / V);
    const int64_t sets = a.B * a.nchunk;
    const int batch = R * (p.backward ? 2 : V >= 4 ? 4 : 8);
    static std::atomic<int> resident[4][64] = {};
    int second = 1;  // blocks a cloud of the second pass
    cudaError_t e;
    if (!p.backward) {
        e = gn_blocks(gn_stats_kernel<T, V>, resident[0], *p.dev, sets, a.L, batch, &a.nblk);
        if (e == cudaSuccess)
            e = gn_blocks(gn_apply_kernel<T, V>, resident[1], *p.dev, sets, a.L, batch, &second);
    } else {
        e = gn_blocks(gn_sums_kernel<T, V>, resident[2], *p.dev, sets, a.L, batch, &a.nblk);
        if (e == cudaSuccess)
            e = gn_blocks(gn_dx_kernel<T, V>, resident[3], *p.dev, sets, a.L, batch, &second);
    }
    if (e != cudaSuccess) return e;
    // (B C is at most 2^30, so no grid is beyond 31 bits)
    cudaStream_t st = p.stream;
    const unsigned grid = unsigned(sets * a.nblk), grid2 = unsigned(sets * second);
    void *scratch = nullptr;
    if (!p.backward) {
        const size_t parts = size_t(a.B) * a.nblk * (a.per ? a.nchunk : a.G) * sizeof(float2);
        const size_t stats = a.mean == nullptr ? size_t(a.B) * a.G * sizeof(float) : 0;
        if ((e = scratch_alloc(*p.dev, &scratch, parts + 2 * stats, st)) != cudaSuccess) return e;
        a.gpart = static_cast<float2 *>(scratch);
        if (a.mean == nullptr) {
            a.mean = reinterpret_cast<float *>(static_cast<char *>(scratch) + parts);
            a.rstd = a.mean + a.B * a.G;
        }
        e = launch(false, gn_stats_kernel<T, V>, grid, GN_THREADS, 0, st, a);
        if (e == cudaSuccess)
            e = launch(true, gn_join_kernel, unsigned(a.B * a.G), 128, 0, st, a);
        if (e == cudaSuccess)
            e = launch(true, gn_apply_kernel<T, V>, grid2, GN_THREADS, 0, st, a, second);
    } else {
        const bool params = a.dw || a.db, apart = params && a.B > PARAM_CLOUDS;
        const size_t parts = size_t(a.B) * a.nblk * 2 * a.C, chan = size_t(a.B) * 2 * a.C;
        const size_t room = apart ? gn_param_room(a.B, a.C) : 0;
        if ((e = scratch_alloc(*p.dev, &scratch, (parts + chan + room) * sizeof(float), st)) !=
            cudaSuccess)
            return e;
        a.cpart = static_cast<float *>(scratch);
        a.chan = a.cpart + parts;
        e = launch(false, gn_sums_kernel<T, V>, grid, GN_THREADS, 0, st, a);
        if (e == cudaSuccess)
            e = launch(true, gn_channel_kernel, unsigned(a.B * ((2 * a.C + 31) / 32)), dim3(32, 32),
                       0, st, a);
        if (e == cudaSuccess && apart)
            e = gn_param_sums(a, sizeof(T) == 2 ? PC_BF16 : PC_F32, a.chan, a.B, a.chan + chan, st);
        const int nparam = params && !apart ? int(ceil_div(2 * a.C, GN_THREADS)) : 0;
        const unsigned dxgrid = a.y ? grid2 : 0;
        if (e == cudaSuccess && dxgrid + nparam > 0)
            e = launch(true, gn_dx_kernel<T, V>, dxgrid + nparam, GN_THREADS, 0, st, a, second,
                       nparam);
    }
    const cudaError_t f = scratch_free(scratch, st);
    return e == cudaSuccess ? f : e;
}

template <class T>
cudaError_t gn_dispatch(GnArgs a, const GnPlan &p) {
    uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                     reinterpret_cast<uintptr_t>(a.dy);
    const int dtype = sizeof(T) == 2 ? PC_BF16 : PC_F32;
    for (int V = 16 / int(sizeof(T)); V >= 1; V /= 2) {
        if (bits % (V * sizeof(T)) || a.C % V) continue;
        const GnCluster cl = gn_cluster_plan(*p.dev, a, dtype, V, p.backward);
        if (cl.blocks > 0)
            return gn_cluster_run(*p.dev, a, dtype, V, p.backward, cl, p.stream);
        a.width = gn_width(a.C, a.cg, V, &a.per);
        if (a.width == 0) continue;
        a.nchunk = a.per ? a.G * a.per : (a.C + a.width - 1) / a.width;
        switch (V) {
            case 8: return gn_run<T, sizeof(T) == 2 ? 8 : 4>(a, p);
            case 4: return gn_run<T, 4>(a, p);
            case 2: return gn_run<T, 2>(a, p);
            default: return gn_run<T, 1>(a, p);
        }
    }
    return cudaErrorInvalidValue;
}

int gn_check(const char *what, int dtype, int param_dtype, int64_t B, int64_t L, int64_t C,
             int64_t groups, int activation) {
    char m[200];
    if (B < 0 || L < 0 || C < 0) {
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
    if (groups < 1 || C % groups) {
        std::snprintf(m, sizeof(m), "%s: groups=%lld must divide the %lld channels", what,
                      (long long)groups, (long long)C);
        return api_fail(PC_ERR_INVALID_ARGUMENT, m);
    }
    if (activation < PC_ACT_NONE || activation > PC_ACT_SIGMOID) {
        std::snprintf(m, sizeof(m), "%s: unknown activation %d", what, activation);
        return api_fail(PC_ERR_INVALID_ARGUMENT, m);
    }
    // (so that every grid and every count of a cloud's values stays in range)
    if (C > GN_MAX_C || L > 2147483647 || (C > 0 && B > (int64_t(1) << 30) / C)) {
        std::snprintf(m, sizeof(m), "%s: C=%lld above %d, L beyond 32 bits or B C beyond 2^30",
                      what, (long long)C, GN_MAX_C);
        return api_fail(PC_ERR_UNSUPPORTED, m);
    }
    return PC_OK;
}

int gn_cuda(const char *what, cudaError_t e) {
    if (e == cudaSuccess) return PC_OK;
    char m[200];
    std::snprintf(m, sizeof(m), "%s: %s", what, cudaGetErrorString(e));
    return api_fail(PC_ERR_CUDA, m);
}

}  // namespace
}  // namespace pcn

extern "C" int pc_group_norm(const void *x, int dtype, int64_t B, int64_t L, int64_t C,
                             int64_t groups, const void *weight, const void *bias,
                             int param_dtype, double eps, int activation,
                             const int64_t *lengths, void *out, float *out_mean,
                             float *out_rstd, void *stream) {
    using namespace pcn;
    int rc = gn_check("group_norm", dtype, param_dtype, B, L, C, groups, activation);
    if (rc != PC_OK) return rc;
    if (!(eps >= 0.0 && eps <= 1e30))
        return api_fail(PC_ERR_INVALID_ARGUMENT, "group_norm: eps must be finite and >= 0");
    if ((out_mean == nullptr) != (out_rstd == nullptr))
        return api_fail(PC_ERR_INVALID_ARGUMENT,
                        "group_norm: out_mean and out_rstd go together");
    if (B == 0 || C == 0 || (L == 0 && out_mean == nullptr)) return PC_OK;
    const DeviceInfo *dev = nullptr;
    if ((rc = api_current_device(&dev)) != PC_OK) return rc;
    const int d = dev->device;
    const size_t es = dtype == PC_F32 ? 4 : 2, ps = param_dtype == PC_F32 ? 4 : 2;
    if (L > 0) {
        if ((rc = api_check_ptr(x, d, es, "x")) != PC_OK) return rc;
        if ((rc = api_check_ptr(out, d, es, "out")) != PC_OK) return rc;
    }
    if (weight && (rc = api_check_ptr(weight, d, ps, "weight")) != PC_OK) return rc;
    if (bias && (rc = api_check_ptr(bias, d, ps, "bias")) != PC_OK) return rc;
    if (lengths && (rc = api_check_ptr(lengths, d, 8, "lengths")) != PC_OK) return rc;
    if (out_mean) {
        if ((rc = api_check_ptr(out_mean, d, 4, "out_mean")) != PC_OK) return rc;
        if ((rc = api_check_ptr(out_rstd, d, 4, "out_rstd")) != PC_OK) return rc;
    }
    GnArgs a{};
    a.x = x, a.w = weight, a.b = bias, a.y = out, a.mean = out_mean, a.rstd = out_rstd;
    a.lengths = lengths, a.B = B, a.L = L, a.C = int(C), a.G = int(groups);
    a.cg = int(C / groups), a.eps = float(eps), a.act = activation;
    a.wf32 = param_dtype == PC_F32;
    GnPlan p{dev, static_cast<cudaStream_t>(stream), false};
    return gn_cuda("group_norm", dtype == PC_F32 ? gn_dispatch<float>(a, p)
                                                 : gn_dispatch<bf16>(a, p));
}

extern "C" int pc_group_norm_backward(const void *grad_out, const void *x, int dtype, int64_t B,
                                      int64_t L, int64_t C, int64_t groups, const float *mean,
                                      const float *rstd, const void *weight, const void *bias,
                                      int param_dtype, int activation, const int64_t *lengths,
                                      void *grad_x, void *grad_weight, void *grad_bias,
                                      void *stream) {
    using namespace pcn;
    int rc = gn_check("group_norm_backward", dtype, param_dtype, B, L, C, groups, activation);
    if (rc != PC_OK) return rc;
    if (C == 0 || (!grad_x && !grad_weight && !grad_bias)) return PC_OK;
    const DeviceInfo *dev = nullptr;
    if ((rc = api_current_device(&dev)) != PC_OK) return rc;
    const int d = dev->device;
    const size_t es = dtype == PC_F32 ? 4 : 2, ps = param_dtype == PC_F32 ? 4 : 2;
    const bool empty = B == 0 || L == 0;
    if (!empty) {
        if ((rc = api_check_ptr(grad_out, d, es, "grad_out")) != PC_OK) return rc;
        if ((rc = api_check_ptr(x, d, es, "x")) != PC_OK) return rc;
        if ((rc = api_check_ptr(mean, d, 4, "mean")) != PC_OK) return rc;
        if ((rc = api_check_ptr(rstd, d, 4, "rstd")) != PC_OK) return rc;
        if (grad_x && (rc = api_check_ptr(grad_x, d, es, "grad_x")) != PC_OK) return rc;
    }
    if (weight && (rc = api_check_ptr(weight, d, ps, "weight")) != PC_OK) return rc;
    if (bias && (rc = api_check_ptr(bias, d, ps, "bias")) != PC_OK) return rc;
    if (lengths && B > 0 && (rc = api_check_ptr(lengths, d, 8, "lengths")) != PC_OK) return rc;
    if (grad_weight && (rc = api_check_ptr(grad_weight, d, ps, "grad_weight")) != PC_OK)
        return rc;
    if (grad_bias && (rc = api_check_ptr(grad_bias, d, ps, "grad_bias")) != PC_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (empty) {  // no rows: the parameters' gradients are 0
        cudaError_t e = cudaSuccess;
        if (grad_weight) e = cudaMemsetAsync(grad_weight, 0, size_t(C) * ps, st);
        if (grad_bias && e == cudaSuccess) e = cudaMemsetAsync(grad_bias, 0, size_t(C) * ps, st);
        return gn_cuda("group_norm_backward", e);
    }
    GnArgs a{};
    a.x = x, a.dy = grad_out, a.w = weight, a.b = bias, a.y = grad_x;
    a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
    a.dw = grad_weight, a.db = grad_bias;
    a.lengths = lengths, a.B = B, a.L = L, a.C = int(C), a.G = int(groups);
    a.cg = int(C / groups), a.act = activation;
    a.wf32 = param_dtype == PC_F32;
    GnPlan p{dev, st, true};
    return gn_cuda("group_norm_backward", dtype == PC_F32 ? gn_dispatch<float>(a, p)
                                                          : gn_dispatch<bf16>(a, p));
}
