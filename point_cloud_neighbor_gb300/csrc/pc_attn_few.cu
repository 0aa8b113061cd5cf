// pc_attn_few.cu -- the attention passes for few queries per key head (at most
// 8 forward, 4 backward, counted over the heads that share the key head): one
// new token, a class token or a few object queries against a long cloud.
//
// Bound: memory, every key and value once.  A block takes a part of the keys
// for all the queries of a key head.  A key belongs to LPK lanes, 16 bytes of
// its channels each; the lanes form the score by shuffles, and every group of
// LPK lanes has its own running maximum, sum and accumulator, joined at the
// end: in the warp, the block, and over the blocks by the join kernels.  The
// queries stay in registers; all arithmetic is float32.  Forward, the keys of
// several steps are on their way at once.
//
// Measured, one query over 100,000 keys, 8 heads of 64: bfloat16 43 us (205 MB:
// 4.8 TB/s) and 8 us for the join, float32 83 us in all (4.9 TB/s); the
// tensor-core kernels take 74 and 278 us, as every block has one row in use.
// Backward 107 us (bfloat16, with the output's low part) and 162 us.
//
// Backward, one pass gives all gradients: a key's own gradients are complete
// in its lanes (all queries of its head are there), the queries' are summed
// over the keys like the forward accumulators.
#include "pc_attn.cuh"
#include "pointcloud.h"

namespace pcn {
namespace {

constexpr int FEW_THREADS = 256, FEW_WARPS = FEW_THREADS / 32;

template <class T>
struct alignas(16) FewChunk {
    T e[16 / sizeof(T)];
    __device__ __forceinline__ void load(const T *p) {
        *this = *reinterpret_cast<const FewChunk *>(p);
    }
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

struct FewBlock {  // what a block works on
    int b, hk, split, nq, nk, j0, j1;
};

__device__ __forceinline__ FewBlock few_block(const AttnArgs &a, int step) {
    FewBlock w;
    int64_t idx = blockIdx.x;
    w.split = int(idx % a.nsplit);
    idx /= a.nsplit;
    w.hk = int(idx % a.Hkv), w.b = int(idx / a.Hkv);
    w.nq = attn_len(a.qlen, w.b, a.Lq), w.nk = attn_len(a.rlen, w.b, a.Lk);
    // backward, the keys past the length get their zeros too
    const int64_t steps = (int64_t(a.Lk) + step - 1) / step;
    w.j0 = int(steps * w.split / a.nsplit * step);
    w.j1 = int(min(int64_t(a.Lk), steps * (w.split + 1) / a.nsplit * step));
    return w;
}

template <int LPK>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LPK / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <class T, int LPK, int R>
__global__ void __launch_bounds__(FEW_THREADS, R == 1 ? 3 : R == 2 ? 2 : 1)
few_forward_kernel(const AttnArgs a) {
    constexpr int V = 16 / sizeof(T), KPW = 32 / LPK, STEP = FEW_WARPS * KPW;
    constexpr int U = R <= 2 ? 4 : 2;  // steps on their way at once
    __shared__ float sm[FEW_WARPS][R][LPK * V + 2];
    const FewBlock w = few_block(a, STEP);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int gl = lane % LPK, c0 = gl * V;
    const bool chan = c0 < a.D, bias = a.slopes != nullptr;
    const int G = a.H / a.Hkv, rows = G * a.Lq;
    const float c2 = a.scale * ATTN_LOG2E;
    float q[R][V], px[R][3], ws[R], m[R], l[R], acc[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int g = r / a.Lq, i = r - g * a.Lq, h = w.hk * G + g;
        const bool in = r < rows && i < w.nq;
#pragma unroll
        for (int e = 0; e < V; ++e) q[r][e] = acc[r][e] = 0.0f;
        m[r] = -INFINITY, l[r] = 0.0f, ws[r] = 0.0f;
        px[r][0] = px[r][1] = px[r][2] = 0.0f;
        if (in && chan) {
            Vec<T, V>::load(static_cast<const T *>(a.q) + w.b * a.qs[0] + i * a.qs[1] +
                                h * a.qs[2] + c0,
                            q[r]);
#pragma unroll
            for (int e = 0; e < V; ++e) q[r][e] *= c2;
        }
        if (in && bias) {
            const float *p = a.qxyz + (int64_t(w.b) * a.Lq + i) * 3;
            px[r][0] = p[0], px[r][1] = p[1], px[r][2] = p[2];
            ws[r] = a.slopes[h] * ATTN_LOG2E;
        }
    }
    const T *kb = static_cast<const T *>(a.k) + w.b * a.ks[0] + w.hk * a.ks[2] + c0;
    const T *vb = static_cast<const T *>(a.v) + w.b * a.vs[0] + w.hk * a.vs[2] + c0;
    const float *yb = a.rxyz + int64_t(w.b) * a.Lk * 3;
    const int j1 = min(w.j1, w.nk);
    // the thread's key in step 0, and the strides of a step
    const int mine = warp * KPW + lane / LPK;
    const int64_t ks = a.ks[1] * STEP, vs = a.vs[1] * STEP;
    const T *kp = kb + (w.j0 + mine) * a.ks[1], *vp = vb + (w.j0 + mine) * a.vs[1];
    const float *yp = yb + int64_t(w.j0 + mine) * 3;
    for (int j = w.j0 + mine; j - mine < j1; j += U * STEP) {
        FewChunk<T> kc[U], vc[U];
        float y[U][3];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            in[u] = j + u * STEP < j1;
#pragma unroll
            for (int e = 0; e < V; ++e) kc[u].e[e] = vc[u].e[e] = T(0.0f);
            if (in[u] && chan) {
                kc[u].load(kp + u * ks);
                vc[u].load(vp + u * vs);
            }
            if (bias)
#pragma unroll
                for (int e = 0; e < 3; ++e) y[u][e] = in[u] ? yp[u * 3 * STEP + e] : 0.0f;
        }
        kp += U * ks, vp += U * vs, yp += U * 3 * STEP;
        float z[R][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float kx[V];
            Vec<T, V>::load(kc[u].e, kx);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float s = 0.0f;
#pragma unroll
                for (int e = 0; e < V; ++e) s = fmaf(q[r][e], kx[e], s);
                z[r][u] = group_sum<LPK>(s);
                if (bias) {
                    const float dx = px[r][0] - y[u][0], dy = px[r][1] - y[u][1],
                                dz = px[r][2] - y[u][2];
                    z[r][u] = fmaf(fmaf(dz, dz, fmaf(dy, dy, dx * dx)), -ws[r], z[r][u]);
                }
                if (!in[u]) z[r][u] = -INFINITY;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float mn = m[r];
#pragma unroll
            for (int u = 0; u < U; ++u) mn = fmaxf(mn, z[r][u]);
            const float base = mn == -INFINITY ? 0.0f : mn;
            const float f = ex2(m[r] - base);
            m[r] = mn;
            l[r] *= f;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[r][e] *= f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                z[r][u] = ex2(z[r][u] - base);
                l[r] += z[r][u];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float vx[V];
            Vec<T, V>::load(vc[u].e, vx);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int e = 0; e < V; ++e) acc[r][e] = fmaf(z[r][u], vx[e], acc[r][e]);
        }
    }
    // the groups of the warp, then the warps of the block
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int o = LPK; o < 32; o <<= 1) {
            const float mo = __shfl_xor_sync(0xffffffffu, m[r], o);
            const float mn = fmaxf(m[r], mo), base = mn == -INFINITY ? 0.0f : mn;
            const float f = exp2f(m[r] - base), fo = exp2f(mo - base);
            m[r] = mn;
            l[r] = l[r] * f + __shfl_xor_sync(0xffffffffu, l[r], o) * fo;
#pragma unroll
            for (int e = 0; e < V; ++e)
                acc[r][e] = acc[r][e] * f + __shfl_xor_sync(0xffffffffu, acc[r][e], o) * fo;
        }
        if (lane < LPK)
#pragma unroll
            for (int e = 0; e < V; ++e) sm[warp][r][c0 + e] = acc[r][e];
        if (lane == 0) sm[warp][r][LPK * V] = m[r], sm[warp][r][LPK * V + 1] = l[r];
    }
    __syncthreads();
    const int64_t hrows = int64_t(a.B) * a.H * a.Lq;
    for (int t = threadIdx.x; t < rows * a.D; t += FEW_THREADS) {
        const int r = t / a.D, c = t - r * a.D;
        const int g = r / a.Lq, i = r - g * a.Lq, h = w.hk * G + g;
        float mn = -INFINITY;
#pragma unroll
        for (int k = 0; k < FEW_WARPS; ++k) mn = fmaxf(mn, sm[k][r][LPK * V]);
        const float base = mn == -INFINITY ? 0.0f : mn;
        float s = 0.0f, v = 0.0f;
#pragma unroll
        for (int k = 0; k < FEW_WARPS; ++k) {
            const float f = exp2f(sm[k][r][LPK * V] - base);
            s = fmaf(sm[k][r][LPK * V + 1], f, s);
            v = fmaf(sm[k][r][c], f, v);
        }
        const int64_t orow = (int64_t(w.b) * a.Lq + i) * a.H + h;
        const int64_t hrow = (int64_t(w.b) * a.H + h) * a.Lq + i;
        const bool any = i < w.nq && w.nk > 0;
        if (a.nsplit > 1) {
            a.part[(int64_t(w.split) * hrows + orow) * a.D + c] = v;
            if (c == 0) {
                a.part_ml[int64_t(w.split) * 2 * hrows + hrow] = mn;
                a.part_ml[(int64_t(w.split) * 2 + 1) * hrows + hrow] = s;
            }
        } else {
            v = any ? v / s : 0.0f;
            Vec<T, 1>::store(static_cast<T *>(a.out) + orow * a.D + c, &v);
            if (a.low != nullptr) {
                v = rest<T>(v);
                Vec<T, 1>::store(static_cast<T *>(a.low) + orow * a.D + c, &v);
            }
            if (c == 0 && a.lse != nullptr)
                a.lse[hrow] = any ? (mn + log2f(s)) * ATTN_LN2 : -INFINITY;
        }
    }
}

template <class T, int LPK, int R>
__global__ void __launch_bounds__(FEW_THREADS, R == 1 ? 3 : R == 2 ? 2 : 1)
few_backward_kernel(const AttnArgs a) {
    constexpr int V = 16 / sizeof(T), KPW = 32 / LPK, STEP = FEW_WARPS * KPW;
    constexpr int U = 2;
    __shared__ float sm[FEW_WARPS][R][LPK * V + 4];
    const FewBlock w = few_block(a, STEP);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int gl = lane % LPK, c0 = gl * V;
    const bool chan = c0 < a.D, bias = a.slopes != nullptr;
    const int G = a.H / a.Hkv, rows = G * a.Lq;
    const float c2 = a.scale * ATTN_LOG2E;
    // q times scale: the scores need it, and so do the keys' gradients
    float q[R][V], go[R][V], px[R][3], ws[R], lse2[R], del[R], dq[R][V];
    LongSum wa[R], we[R], wd[R], wp[R];
    unsigned live = 0;  // a bit a row: the others take no part, whatever the keys hold
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int g = r / a.Lq, i = r - g * a.Lq, h = w.hk * G + g;
        const bool in = r < rows && i < w.nq;
#pragma unroll
        for (int e = 0; e < V; ++e) q[r][e] = go[r][e] = dq[r][e] = 0.0f;
        ws[r] = px[r][0] = px[r][1] = px[r][2] = del[r] = 0.0f;
        lse2[r] = INFINITY;
        if (in && chan) {
            Vec<T, V>::load(static_cast<const T *>(a.q) + w.b * a.qs[0] + i * a.qs[1] +
                                h * a.qs[2] + c0,
                            q[r]);
            Vec<T, V>::load(static_cast<const T *>(a.go) +
                                ((int64_t(w.b) * a.Lq + i) * a.H + h) * a.D + c0,
                            go[r]);
        }
        if (in) {
            const int64_t at = (int64_t(w.b) * a.H + h) * a.Lq + i;
            live |= 1u << r;
            lse2[r] = a.lse2[at], del[r] = a.delta[at];
            if (bias) {
                const float *p = a.qxyz + (int64_t(w.b) * a.Lq + i) * 3;
                px[r][0] = p[0], px[r][1] = p[1], px[r][2] = p[2];
                ws[r] = a.slopes[h] * ATTN_LOG2E;
            }
        }
    }
    const T *kb = static_cast<const T *>(a.k) + w.b * a.ks[0] + w.hk * a.ks[2] + c0;
    const T *vb = static_cast<const T *>(a.v) + w.b * a.vs[0] + w.hk * a.vs[2] + c0;
    const float *yb = a.rxyz + int64_t(w.b) * a.Lk * 3;
    const float one = attn_ds_factor(w.nk);
    for (int j = w.j0; j < w.j1; j += U * STEP) {
        FewChunk<T> kc[U], vc[U];
        float y[U][3];
        int at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            at[u] = j + u * STEP + warp * KPW + lane / LPK;
            const bool in = at[u] < w.j1 && at[u] < w.nk;
#pragma unroll
            for (int e = 0; e < V; ++e) kc[u].e[e] = vc[u].e[e] = T(0.0f);
            if (in && chan) {
                kc[u].load(kb + at[u] * a.ks[1]);
                vc[u].load(vb + at[u] * a.vs[1]);
            }
            if (bias)
#pragma unroll
                for (int e = 0; e < 3; ++e) y[u][e] = in ? yb[int64_t(at[u]) * 3 + e] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = at[u] < w.j1 && at[u] < w.nk;
            float kx[V], vx[V], dk[V], dv[V];
            Vec<T, V>::load(kc[u].e, kx);
            Vec<T, V>::load(vc[u].e, vx);
#pragma unroll
            for (int e = 0; e < V; ++e) dk[e] = dv[e] = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float s = 0.0f, dp = 0.0f;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    s = fmaf(q[r][e], kx[e], s);
                    dp = fmaf(go[r][e], vx[e], dp);
                }
                s = group_sum<LPK>(s);
                dp = group_sum<LPK>(dp);
                float z = s * c2, d2 = 0.0f;
                if (bias) {
                    const float dx = px[r][0] - y[u][0], dy = px[r][1] - y[u][1],
                                dz = px[r][2] - y[u][2];
                    d2 = fmaf(dz, dz, fmaf(dy, dy, dx * dx));
                    z = fmaf(d2, -ws[r], z);
                }
                const bool on = in && (live >> r & 1);
                const float p = on ? ex2(z - lse2[r]) : 0.0f;
                const float ds = on ? p * (dp - del[r]) : 0.0f;
                wa[r].add(ds * d2);
                we[r].add(p * d2);
                wd[r].add(ds);
                wp[r].add(p);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    dq[r][e] = fmaf(ds, kx[e], dq[r][e]);
                    dk[e] = fmaf(ds, q[r][e], dk[e]);
                    dv[e] = fmaf(p, go[r][e], dv[e]);
                }
            }
            if (a.dk != nullptr && at[u] < w.j1 && chan) {
                const int64_t o = ((int64_t(w.b) * a.Lk + at[u]) * a.Hkv + w.hk) * a.D + c0;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    dk[e] = in ? dk[e] * (one * a.scale) : 0.0f;
                    dv[e] = in ? dv[e] : 0.0f;
                }
                Vec<T, V>::store(static_cast<T *>(a.dk) + o, dk);
                Vec<T, V>::store(static_cast<T *>(a.dv) + o, dv);
            }
        }
    }
    if (a.dq == nullptr) return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float ta = wa[r].value(), te = we[r].value(), td = wd[r].value(), tp = wp[r].value();
#pragma unroll
        for (int o = LPK; o < 32; o <<= 1) {
            ta += __shfl_xor_sync(0xffffffffu, ta, o);
            te += __shfl_xor_sync(0xffffffffu, te, o);
            td += __shfl_xor_sync(0xffffffffu, td, o);
            tp += __shfl_xor_sync(0xffffffffu, tp, o);
#pragma unroll
            for (int e = 0; e < V; ++e) dq[r][e] += __shfl_xor_sync(0xffffffffu, dq[r][e], o);
        }
        if (lane < LPK)
#pragma unroll
            for (int e = 0; e < V; ++e) sm[warp][r][c0 + e] = dq[r][e];
        if (lane == 0) {
            sm[warp][r][LPK * V] = ta;
            sm[warp][r][LPK * V + 1] = te;
            sm[warp][r][LPK * V + 2] = td;
            sm[warp][r][LPK * V + 3] = tp;
        }
    }
    __syncthreads();
    const int64_t hrows = int64_t(a.B) * a.H * a.Lq;
    const int per = a.D + (a.rowsum != nullptr ? 4 : 0);
    for (int t = threadIdx.x; t < rows * per; t += FEW_THREADS) {
        const int r = t / per, c = t - r * per;
        const int g = r / a.Lq, i = r - g * a.Lq, h = w.hk * G + g;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < FEW_WARPS; ++k) v += sm[k][r][c < a.D ? c : LPK * V + c - a.D];
        v = i < w.nq ? one * v : 0.0f;  // (past the length weights of 0, but keys that may be NaN)
        const int64_t orow = (int64_t(w.b) * a.Lq + i) * a.H + h;
        const int64_t hrow = (int64_t(w.b) * a.H + h) * a.Lq + i;
        if (c >= a.D) {
            a.rowsum[(int64_t(w.split) * 4 + c - a.D) * hrows + hrow] = v;
        } else if (a.nsplit > 1) {
            a.part[(int64_t(w.split) * hrows + orow) * a.D + c] = v;
        } else {
            v *= a.scale;
            Vec<T, 1>::store(static_cast<T *>(a.dq) + orow * a.D + c, &v);
        }
    }
}

template <class T, int LPK>
cudaError_t few_rows(const AttnArgs &a, bool backward, unsigned blocks, cudaStream_t st) {
    const int rows = a.H / a.Hkv * a.Lq;
    if (backward) {
        if (rows <= 1)
            few_backward_kernel<T, LPK, 1><<<blocks, FEW_THREADS, 0, st>>>(a);
        else if (rows <= 2)
            few_backward_kernel<T, LPK, 2><<<blocks, FEW_THREADS, 0, st>>>(a);
        else
            few_backward_kernel<T, LPK, 4><<<blocks, FEW_THREADS, 0, st>>>(a);
    } else if (rows <= 1) {
        few_forward_kernel<T, LPK, 1><<<blocks, FEW_THREADS, 0, st>>>(a);
    } else if (rows <= 2) {
        few_forward_kernel<T, LPK, 2><<<blocks, FEW_THREADS, 0, st>>>(a);
    } else if (rows <= 4) {
        few_forward_kernel<T, LPK, 4><<<blocks, FEW_THREADS, 0, st>>>(a);
    } else {
        few_forward_kernel<T, LPK, 8><<<blocks, FEW_THREADS, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

bool attn_few_fits(const AttnArgs &a, size_t elem, bool backward) {
    const int64_t v = 16 / int64_t(elem);
    const int64_t rows = int64_t(a.H / a.Hkv) * a.Lq;
    if (rows > (backward ? 4 : 8) || a.Lq < 1 || a.Lk < 1 || a.D % v != 0) return false;
    auto ok = [&](const void *p, const int64_t *s) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 &&
               (s == nullptr || (s[0] % v == 0 && s[1] % v == 0 && s[2] % v == 0));
    };
    return ok(a.q, a.qs) && ok(a.k, a.ks) && ok(a.v, a.vs) &&
           (!backward || (ok(a.go, nullptr) && ok(a.dk, nullptr) && ok(a.dv, nullptr)));
}

int attn_few_parts(const DeviceInfo &dev, const AttnArgs &a, size_t elem, bool backward) {
    // A block for every 4 steps of its warps at least, and about 8 blocks a SM.
    const int64_t lanes = int64_t(a.D) * elem / 16;
    const int64_t lpk = elem == 2 ? (lanes <= 4 ? 4 : lanes <= 8 ? 8 : 16)
                                  : (lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32);
    const int64_t each = FEW_WARPS * (32 / lpk) * (backward ? 4 : 8);
    const int64_t base = int64_t(a.B) * a.Hkv, most = (a.Lk + each - 1) / each;
    int64_t n = (int64_t(dev.sm_count) * 8 + base - 1) / base;
    if (n > most) n = most;
    if (n > 256) n = 256;
    return n < 1 ? 1 : int(n);
}

cudaError_t launch_attn_few(const AttnArgs &a, size_t elem, bool backward, cudaStream_t st) {
    const int64_t blocks = int64_t(a.B) * a.Hkv * a.nsplit;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const unsigned g = unsigned(blocks);
    const int lanes = int(a.D * elem / 16);
    if (elem == 2) {
        if (lanes <= 4) return few_rows<bf16, 4>(a, backward, g, st);
        if (lanes <= 8) return few_rows<bf16, 8>(a, backward, g, st);
        return few_rows<bf16, 16>(a, backward, g, st);
    }
    if (lanes <= 8) return few_rows<float, 8>(a, backward, g, st);
    if (lanes <= 16) return few_rows<float, 16>(a, backward, g, st);
    return few_rows<float, 32>(a, backward, g, st);
}

}  // namespace pcn
