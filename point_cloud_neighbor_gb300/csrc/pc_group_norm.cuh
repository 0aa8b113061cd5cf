// pc_group_norm.cuh -- pieces the group norm kernels share.
#pragma once

#include "pc_act.cuh"
#include "pc_internal.h"
#include "pc_vec.cuh"

namespace pcn {

constexpr int GN_THREADS = 256;
constexpr int GN_MAX_C = 16384;

struct GnArgs {
    const void *x, *dy, *w, *b;
    void *y;                 // forward: y; backward: dx
    const int64_t *lengths;
    float *mean, *rstd;      // [B, G]
    float2 *gpart;           // forward: [B][nblk][G, or chunks] mean and sum of squares
    float *cpart;            // backward: [B][nblk][2][C]
    float *chan;             // backward: [B][2][C]
    void *dw, *db;
    int64_t B, L;
    int C, G, cg;            // channels, groups, channels of a group
    int width, nchunk;       // channels of a chunk (a block's), chunks
    int per;                 // chunks of a group wider than a block, else 0
    int nblk;                // blocks that share a cloud's rows
    float eps;
    int act;
    bool wf32;               // weight and bias are float32
};

__device__ __forceinline__ int64_t gn_len(const GnArgs &a, int64_t b) {
    if (a.lengths == nullptr) return a.L;
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : n > a.L ? a.L : n;
}

// How `parts` blocks share n rows (below 2^31): the first each of them, and so on.
struct GnSplit {
    int64_t n, each;
    __device__ __forceinline__ GnSplit(int64_t n_, int parts)
        : n(n_), each((uint32_t(n_) + uint32_t(parts) - 1) / uint32_t(parts)) {}
    __device__ __forceinline__ int64_t row(int part) const { return min(n, each * part); }
    __device__ __forceinline__ int rows(int part) const { return int(row(part + 1) - row(part)); }
};

// The groups of V neighbouring channels from c on.
template <int V>
__device__ __forceinline__ void gn_groups(int c, int cg, int (&g)[V]) {
    int at = c / cg, left = (at + 1) * cg - c;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (left == 0) ++at, left = cg;
        g[e] = at;
        --left;
    }
}

template <class T>
__device__ __forceinline__ float gn_param(const void *p, bool f32, int c, float none) {
    if (p == nullptr) return none;
    if (f32) return static_cast<const float *>(p)[c];
    float v;
    Vec<T, 1>::load(static_cast<const T *>(p) + c, &v);
    return v;
}

// A count, a mean and a sum of squares around it.
struct Moments {
    float n = 0.0f, m = 0.0f, s = 0.0f;
    __device__ __forceinline__ void join(float nb, float mb, float sb) {
        const float t = n + nb;
        if (nb == 0.0f) return;
        const float f = nb / t, d = mb - m;
        s = s + fmaf(d * d, n * f, sb);
        m = fmaf(d, f, m);
        n = t;
    }
};

// The values of a thread's channels in the backward passes.
template <class T, int V>
struct GnChannels {
    float mean[V], rstd[V], w[V], b[V];
    int group[V];
    __device__ __forceinline__ GnChannels(const GnArgs &a, int64_t cloud, int c) {
        gn_groups(c, a.cg, group);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int64_t g = cloud * a.G + group[e];
            mean[e] = a.mean[g], rstd[e] = a.rstd[g];
            w[e] = gn_param<T>(a.w, a.wf32, c + e, 1.0f);
            b[e] = gn_param<T>(a.b, a.wf32, c + e, 0.0f);
        }
    }
    // x and dy of U vectors become xhat and d
    template <int U>
    __device__ __forceinline__ void form(int act, float (&x)[U][V], float (&dy)[U][V]) const {
        act_switch(act, [&](auto a) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float slope;
                    x[u][e] = (x[u][e] - mean[e]) * rstd[e];
                    act_both<a.value, sizeof(T) == 2>(fmaf(x[u][e], w[e], b[e]), slope);
                    dy[u][e] *= slope;
                }
        });
    }
};

// dw and db (a's) from n rows of the channels' sums of d and d xhat, [n][2][C]: rows in
// spans of GN_SPAN, whose sums are the next rows, as long as there are several.  So a
// channel's chain of additions grows by 64 for a factor of GN_SPAN in n.  `room`:
// gn_param_room(n, C) floats.  Launched behind the kernel that writes the rows.
constexpr int GN_SPAN = 1024;
size_t gn_param_room(int64_t n, int C);
cudaError_t gn_param_sums(const GnArgs &a, int dtype, const float *rows, int64_t n, float *room,
                          cudaStream_t st);

// Clouds that fit the shared memory of a cluster (pc_group_norm_cl.cu): whether these
// do, and the launch.
struct GnCluster {
    int blocks = 0;       // of a cloud; 0: does not fit
    int bytes = 0;        // of a slab's room in shared memory
    size_t smem = 0;
};
GnCluster gn_cluster_plan(const DeviceInfo &dev, const GnArgs &a, int dtype, int V, bool backward);
cudaError_t gn_cluster_run(const DeviceInfo &dev, GnArgs a, int dtype, int V, bool backward,
                           const GnCluster &p, cudaStream_t st);

}  // namespace pcn
