// pc_attn.cu -- attention over point tokens with a bias by squared distance
// and lengths masks: the C ABI, the choice of kernels, the joins of split
// passes, and kernels in float32 instructions for what the others do not take.
// Formulas and the three passes are in pc_attn.cuh.
#include "pc_attn.cuh"
#include "pointcloud.h"

#include <algorithm>
#include <cmath>
#include <cstdio>

namespace pcn {
namespace {

// ---------------------------------------------------------------------------
// float32 arithmetic on tiles of 64 rows by 64 streamed rows, 256 threads as
// 16 x 16: a thread forms 4 x 4 scores (rows ty + 16 i, columns tx + 16 j)
// and 4 rows by DP / 16 channels of the accumulators.  Any channels, strides
// and alignment.  Bound by shared-memory reads (8 of 16 bytes for 64
// multiply-adds); 1024 queries and keys, 8 heads of 64 with the bias: forward 105
// us, backward 378 us, against 27 and 56 us on the tensor cores.
// ---------------------------------------------------------------------------
constexpr int SB = 64;           // rows of a tile, both sides
constexpr int ST = 256;          // threads
constexpr int SP = SB + 4;       // row pitch of a score tile

constexpr size_t simt_smem(int mode, int DP) {
    const size_t tile = size_t(SB) * (DP + 4), sc = size_t(SB) * SP;
    return 4 * ((mode == ATTN_FWD ? 3 : 4) * tile + (mode == ATTN_DKV ? 2 : 1) * sc + 6 * SB);
}

// 64 rows of D channels into smem as float32, zeros past row `n` and past D.
template <class T, int DP>
__device__ __forceinline__ void load_rows(float *dst, const T *src, int64_t stride, int r0,
                                          int n, int D, bool vec) {
    constexpr int LD = DP + 4;
    if (vec) {
        for (int i = threadIdx.x; i < SB * DP / 4; i += ST) {
            const int r = i / (DP / 4), c = (i % (DP / 4)) * 4;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (r0 + r < n && c < D) Vec<T, 4>::load(src + int64_t(r0 + r) * stride + c, v);
            Vec<float, 4>::store(dst + r * LD + c, v);
        }
    } else {
        for (int i = threadIdx.x; i < SB * DP; i += ST) {
            const int r = i / DP, c = i % DP;
            float v = 0.0f;
            if (r0 + r < n && c < D) Vec<T, 1>::load(src + int64_t(r0 + r) * stride + c, &v);
            dst[r * LD + c] = v;
        }
    }
}

// s[i][j] = X[ty + 16 i] . Y[tx + 16 j]
template <int DP>
__device__ __forceinline__ void tile_scores(const float *X, const float *Y, int ty, int tx,
                                            float (&s)[4][4]) {
    constexpr int LD = DP + 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        float x[4][4], y[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) Vec<float, 4>::load(X + (ty + 16 * i) * LD + d, x[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) Vec<float, 4>::load(Y + (tx + 16 * j) * LD + d, y[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][j] = fmaf(x[i][e], y[j][e], s[i][j]);
    }
}

// acc[i][64 g + ...] += sum_c P[ty + 16 i][c] Y[c][4 tx + 64 g ...]
template <int DP>
__device__ __forceinline__ void tile_accumulate(const float *P, const float *Y, int ty, int tx,
                                                float (&acc)[4][DP / 16]) {
    constexpr int LD = DP + 4;
#pragma unroll 2
    for (int c = 0; c < SB; c += 4) {
        float p[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) Vec<float, 4>::load(P + (ty + 16 * i) * SP + c, p[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int g = 0; g < DP / 64; ++g) {
                float y[4];
                Vec<float, 4>::load(Y + (c + e) * LD + 64 * g + 4 * tx, y);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int f = 0; f < 4; ++f)
                        acc[i][4 * g + f] = fmaf(p[i][e], y[f], acc[i][4 * g + f]);
            }
    }
}

template <class T, int MODE, int DP>
__global__ void __launch_bounds__(ST) attn_simt_kernel(const AttnArgs a, const bool vec) {
    extern __shared__ float sm[];
    constexpr int TILE = SB * (DP + 4);
    constexpr bool BWD = MODE != ATTN_FWD;
    float *X1 = sm, *X2 = X1 + (BWD ? TILE : 0);
    float *Y1 = X2 + TILE, *Y2 = Y1 + TILE;
    float *P = Y2 + TILE, *S = P + (MODE == ATTN_DKV ? SB * SP : 0);
    float *yp = S + SB * SP;       // x, y, z of the streamed rows, [3][64]
    float *ylse = yp + 3 * SB, *ydel = ylse + SB;

    const int LX = MODE == ATTN_DKV ? a.Lk : a.Lq;
    const int NH = MODE == ATTN_DKV ? a.Hkv : a.H;
    const int G = a.H / a.Hkv;
    const int ntile = (LX + SB - 1) / SB;
    int64_t idx = blockIdx.x;
    const int split = int(idx % a.nsplit);
    idx /= a.nsplit;
    const int tile = int(idx % ntile);
    idx /= ntile;
    const int head = int(idx % NH), b = int(idx / NH);
    const int nq = attn_len(a.qlen, b, a.Lq), nk = attn_len(a.rlen, b, a.Lk);
    const int nx = MODE == ATTN_DKV ? nk : nq, ny = MODE == ATTN_DKV ? nq : nk;
    const int r0 = tile * SB;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const bool bias = a.slopes != nullptr;
    const float c2 = a.scale * ATTN_LOG2E;

    auto qrow = [&](int h) { return static_cast<const T *>(a.q) + b * a.qs[0] + h * a.qs[2]; };
    auto krow = [&](int h) { return static_cast<const T *>(a.k) + b * a.ks[0] + h * a.ks[2]; };
    auto vrow = [&](int h) { return static_cast<const T *>(a.v) + b * a.vs[0] + h * a.vs[2]; };
    auto grow = [&](int h) {
        return static_cast<const T *>(a.go) + (int64_t(b) * a.Lq * a.H + h) * a.D;
    };
    const int64_t gs = int64_t(a.H) * a.D;

    const int hk = MODE == ATTN_DKV ? head : head / G;
    if (MODE == ATTN_DKV) {
        load_rows<T, DP>(X1, krow(hk), a.ks[1], r0, nx, a.D, vec);
        load_rows<T, DP>(X2, vrow(hk), a.vs[1], r0, nx, a.D, vec);
    } else {
        load_rows<T, DP>(X1, qrow(head), a.qs[1], r0, nx, a.D, vec);
        if (BWD) load_rows<T, DP>(X2, grow(head), gs, r0, nx, a.D, vec);
    }
    float px[4][3];  // positions of the thread's rows
    float lse2[4], del[4];
    const float *xpos = MODE == ATTN_DKV ? a.rxyz : a.qxyz;
    const float *ypos = MODE == ATTN_DKV ? a.qxyz : a.rxyz;
    const int LY = MODE == ATTN_DKV ? a.Lq : a.Lk;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + ty + 16 * i;
#pragma unroll
        for (int e = 0; e < 3; ++e)
            px[i][e] = bias && r < nx ? xpos[(int64_t(b) * LX + r) * 3 + e] : 0.0f;
        if (MODE == ATTN_DQ) {
            const int64_t at = (int64_t(b) * a.H + head) * a.Lq + r;
            lse2[i] = r < nx ? a.lse2[at] : INFINITY;  // P = 0
            del[i] = r < nx ? a.delta[at] : 0.0f;
        }
    }
    float acc[4][DP / 16], acc2[4][DP / 16];
    float mx[4], sum[4];
    LongSum wa[4], we[4], wd[4], wp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int e = 0; e < DP / 16; ++e) acc[i][e] = acc2[i][e] = 0.0f;
        mx[i] = -INFINITY;
        sum[i] = 0.0f;
    }

    const int nyt = (ny + SB - 1) / SB;
    const int64_t items = nx > r0 ? int64_t(nyt) * (MODE == ATTN_DKV ? G : 1) : 0;
    const int64_t it0 = items * split / a.nsplit, it1 = items * (split + 1) / a.nsplit;
    for (int64_t it = it0; it < it1; ++it) {
        const int h = MODE == ATTN_DKV ? hk * G + int(it / nyt) : head;
        const int y0 = int(MODE == ATTN_DKV ? it % nyt : it) * SB;
        __syncthreads();
        if (MODE == ATTN_DKV) {
            load_rows<T, DP>(Y1, qrow(h), a.qs[1], y0, ny, a.D, vec);
            load_rows<T, DP>(Y2, grow(h), gs, y0, ny, a.D, vec);
            if (threadIdx.x < SB) {
                const int r = y0 + threadIdx.x;
                const int64_t at = (int64_t(b) * a.H + h) * a.Lq + r;
                ylse[threadIdx.x] = r < ny ? a.lse2[at] : INFINITY;
                ydel[threadIdx.x] = r < ny ? a.delta[at] : 0.0f;
            }
        } else {
            load_rows<T, DP>(Y1, krow(hk), a.ks[1], y0, ny, a.D, vec);
            load_rows<T, DP>(Y2, vrow(hk), a.vs[1], y0, ny, a.D, vec);
        }
        if (bias)
            for (int i = threadIdx.x; i < 3 * SB; i += ST) {
                const int r = i / 3, e = i % 3;
                yp[e * SB + r] = y0 + r < ny ? ypos[(int64_t(b) * LY + y0 + r) * 3 + e] : 0.0f;
            }
        __syncthreads();
        const float ws = bias ? a.slopes[h] * ATTN_LOG2E : 0.0f;
        float s[4][4], dp[4][4], d2[4][4];
        tile_scores<DP>(X1, Y1, ty, tx, s);
        if (BWD) tile_scores<DP>(X2, Y2, ty, tx, dp);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = tx + 16 * j;
            const float yx = yp[c], yy = yp[SB + c], yz = yp[2 * SB + c];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float z = s[i][j] * c2;
                if (bias) {
                    const float dx = px[i][0] - yx, dy = px[i][1] - yy, dz = px[i][2] - yz;
                    d2[i][j] = fmaf(dz, dz, fmaf(dy, dy, dx * dx));
                    z = fmaf(d2[i][j], -ws, z);
                }
                if (MODE != ATTN_DKV && y0 + c >= ny) z = -INFINITY;
                s[i][j] = z;
            }
        }
        if (MODE == ATTN_FWD) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float m = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                m = fmaxf(m, mx[i]);
                const float base = m == -INFINITY ? 0.0f : m;
                const float keep = exp2f(mx[i] - base);
                mx[i] = m;
                float t = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = exp2f(s[i][j] - base);
                    t += s[i][j];
                    P[(ty + 16 * i) * SP + tx + 16 * j] = s[i][j];
                }
                sum[i] = fmaf(sum[i], keep, t);
#pragma unroll
                for (int e = 0; e < DP / 16; ++e) acc[i][e] *= keep;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float ta = 0.0f, te = 0.0f, td = 0.0f, tp = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = tx + 16 * j;
                    const float p = exp2f(s[i][j] - (MODE == ATTN_DKV ? ylse[c] : lse2[i]));
                    const float ds = p * (dp[i][j] - (MODE == ATTN_DKV ? ydel[c] : del[i]));
                    if (MODE == ATTN_DQ && bias) {
                        ta = fmaf(ds, d2[i][j], ta);
                        te = fmaf(p, d2[i][j], te);
                        td += ds;
                        tp += p;
                    }
                    if (MODE == ATTN_DKV) P[(ty + 16 * i) * SP + c] = p;
                    S[(ty + 16 * i) * SP + c] = ds;
                }
                if (MODE == ATTN_DQ && bias)
                    wa[i].add(ta), we[i].add(te), wd[i].add(td), wp[i].add(tp);
            }
        }
        __syncthreads();
        if (MODE == ATTN_FWD) {
            tile_accumulate<DP>(P, Y2, ty, tx, acc);
        } else {
            tile_accumulate<DP>(S, Y1, ty, tx, acc);
            if (MODE == ATTN_DKV) tile_accumulate<DP>(P, Y2, ty, tx, acc2);
        }
    }

    const int64_t rows = int64_t(a.B) * LX * NH;
    const float one = MODE == ATTN_FWD ? 1.0f : attn_ds_factor(nk);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + ty + 16 * i;
        const int64_t hrow = (int64_t(b) * a.H + head) * a.Lq + r;  // FWD, DQ
        if (MODE == ATTN_FWD) {
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
        }
        if (MODE == ATTN_DQ && bias) {
            float ta = one * wa[i].value(), te = we[i].value(), td = one * wd[i].value(),
                  tp = wp[i].value();
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) {
                ta += __shfl_xor_sync(0xffffffffu, ta, o);
                te += __shfl_xor_sync(0xffffffffu, te, o);
                td += __shfl_xor_sync(0xffffffffu, td, o);
                tp += __shfl_xor_sync(0xffffffffu, tp, o);
            }
            if (tx == 0 && r < LX && a.rowsum != nullptr) {
                const int64_t n = int64_t(a.B) * a.H * a.Lq;
                float *w = a.rowsum + int64_t(split) * 4 * n + hrow;
                w[0] = ta, w[n] = te, w[2 * n] = td, w[3 * n] = tp;
            }
        }
        if (r >= LX) continue;
        const int64_t orow = (int64_t(b) * LX + r) * NH + head;
        if (a.nsplit > 1) {
            float *p1 = a.part + (int64_t(split) * rows + orow) * a.D;
            float *p2 = p1 + int64_t(a.nsplit) * rows * a.D;
#pragma unroll
            for (int e = 0; e < DP / 16; ++e) {
                const int c = 64 * (e / 4) + 4 * tx + e % 4;
                if (c < a.D) {
                    p1[c] = r < nx ? one * acc[i][e] : 0.0f;
                    if (MODE == ATTN_DKV) p2[c] = r < nx ? acc2[i][e] : 0.0f;
                }
            }
            if (MODE == ATTN_FWD && tx == 0) {
                const int64_t n = int64_t(a.B) * a.H * a.Lq;
                a.part_ml[int64_t(split) * 2 * n + hrow] = mx[i];
                a.part_ml[(int64_t(split) * 2 + 1) * n + hrow] = sum[i];
            }
            continue;
        }
        const bool any = r < nx && (MODE != ATTN_FWD || ny > 0);
        const float f = MODE == ATTN_FWD ? 1.0f / sum[i] : one * a.scale;
        T *o1 = static_cast<T *>(MODE == ATTN_FWD  ? a.out
                                 : MODE == ATTN_DQ ? a.dq
                                                   : a.dk) + orow * a.D;
        T *o2 = static_cast<T *>(a.dv) + orow * a.D;
#pragma unroll
        for (int e = 0; e < DP / 16; ++e) {
            const int c = 64 * (e / 4) + 4 * tx + e % 4;
            if (c < a.D) {
                const float w = any ? acc[i][e] * f : 0.0f;
                Vec<T, 1>::store(o1 + c, &w);
                if (MODE == ATTN_FWD && a.low != nullptr) {
                    const float l = rest<T>(w);
                    Vec<T, 1>::store(static_cast<T *>(a.low) + orow * a.D + c, &l);
                }
                if (MODE == ATTN_DKV) {
                    const float u = r < nx ? acc2[i][e] : 0.0f;
                    Vec<T, 1>::store(o2 + c, &u);
                }
            }
        }
        if (MODE == ATTN_FWD && tx == 0 && a.lse != nullptr)
            a.lse[hrow] = any ? (mx[i] + log2f(sum[i])) * ATTN_LN2 : -INFINITY;
    }
}

// delta_i = (out_i + low_i) . dout_i, and lse in base-2 units with +inf for rows
// without keys (their weights 2^(z - lse2) are then 0): LPR lanes per (token, head),
// V channels at a time.  (16 x 1024 tokens, 8 heads of 64 in bfloat16: a warp per
// row and one channel a load 32 us, 8 lanes per row 5 us.)
template <class T, int V, int LPR>
__global__ void __launch_bounds__(256)
attn_delta_kernel(const T *out, const T *low, const T *go, const float *lse, int64_t rows,
                  int Lq, int H, int D, float *delta, float *lse2) {
    const int64_t row = (int64_t(blockIdx.x) * 256 + threadIdx.x) / LPR;  // (b Lq + i) H + h
    const int lane = threadIdx.x % LPR;
    float s = 0.0f;
    if (row < rows)
        for (int c = lane * V; c < D; c += LPR * V) {
            float o[V], g[V];
            Vec<T, V>::load(out + row * D + c, o);
            Vec<T, V>::load(go + row * D + c, g);
            if (low != nullptr) {
                float l[V];
                Vec<T, V>::load(low + row * D + c, l);
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] += l[e];  // (16 bits: exact)
            }
#pragma unroll
            for (int e = 0; e < V; ++e) s = fmaf(o[e], g[e], s);
        }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (row < rows && lane == 0) {
        const int64_t tok = row / H, b = tok / Lq;
        const int64_t at = (b * H + row % H) * Lq + (tok - b * Lq);
        delta[at] = s;
        lse2[at] = lse[at] == -INFINITY ? INFINITY : lse[at] * ATTN_LOG2E;
    }
}

template <class T>
void launch_delta(const AttnArgs &a, const T *out, const T *low, int64_t rows, float *delta,
                  float *lse2, cudaStream_t st) {
    const T *go = static_cast<const T *>(a.go);
    constexpr int W = 16 / sizeof(T);
    auto aligned = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    const bool wide = a.D % W == 0 && aligned(out) && aligned(low) && aligned(go);
    const unsigned g8 = unsigned((rows * 8 + 255) / 256), g32 = unsigned((rows * 32 + 255) / 256);
    if (wide)
        attn_delta_kernel<T, W, 8><<<g8, 256, 0, st>>>(out, low, go, a.lse, rows, a.Lq, a.H,
                                                       a.D, delta, lse2);
    else
        attn_delta_kernel<T, 1, 32><<<g32, 256, 0, st>>>(out, low, go, a.lse, rows, a.Lq, a.H,
                                                         a.D, delta, lse2);
}

// Joins the parts of a split forward pass: a thread per V channels of a row.
template <class T, int V>
__global__ void __launch_bounds__(256) attn_join_forward_kernel(const AttnArgs a) {
    const int64_t rows = int64_t(a.B) * a.Lq * a.H;
    const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int groups = a.D / V;
    const int64_t row = id / groups;
    if (row >= rows) return;
    const int c = int(id - row * groups) * V;
    const int64_t tok = row / a.H, b = tok / a.Lq;
    const int i = int(tok - b * a.Lq);
    const int64_t hrow = (b * a.H + (row - tok * a.H)) * a.Lq + i;
    const float *ml = a.part_ml + hrow;
    float m = -INFINITY;
#pragma unroll 4
    for (int s = 0; s < a.nsplit; ++s) m = fmaxf(m, ml[int64_t(s) * 2 * rows]);
    const float base = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, v[V] = {};
#pragma unroll 4
    for (int s = 0; s < a.nsplit; ++s) {
        const float w = exp2f(ml[int64_t(s) * 2 * rows] - base);
        float p[V];
        Vec<float, V>::load(a.part + (int64_t(s) * rows + row) * a.D + c, p);
        l = fmaf(w, ml[(int64_t(s) * 2 + 1) * rows], l);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = fmaf(w, p[e], v[e]);
    }
    const bool any = attn_row_has_keys(a, int(b), i);
    const float f = 1.0f / l;
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = any ? v[e] * f : 0.0f;
    Vec<T, V>::store(static_cast<T *>(a.out) + row * a.D + c, v);
    if (a.low != nullptr) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = rest<T>(v[e]);
        Vec<T, V>::store(static_cast<T *>(a.low) + row * a.D + c, v);
    }
    if (c == 0 && a.lse != nullptr)
        a.lse[hrow] = any ? (m + log2f(l)) * ATTN_LN2 : -INFINITY;
}

// out = factor * sum of the parts, V elements a thread; a second array of the
// same size follows with blockIdx.y = 1.
template <class T, int V>
__global__ void __launch_bounds__(256)
attn_join_sum_kernel(const float *part, int nsplit, int64_t n, float factor, T *out, T *out2) {
    const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * V;
    if (i >= n) return;
    if (blockIdx.y == 1) part += int64_t(nsplit) * n, out = out2, factor = 1.0f;
    float v[V] = {};
#pragma unroll 4
    for (int s = 0; s < nsplit; ++s) {
        float p[V];
        Vec<float, V>::load(part + int64_t(s) * n + i, p);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] += p[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] *= factor;
    Vec<T, V>::store(out + i, v);
}

// Few rows and many parts: a block per row of the output (forward, or dq), the
// parts over its threads.  The row's sums for the slopes' gradient are joined
// too and left as those of part 0.
template <class T, bool FWD>
__global__ void __launch_bounds__(1024) attn_join_rows_kernel(const AttnArgs a) {
    __shared__ float wt[256], red[32], part[1024];
    const int64_t rows = int64_t(a.B) * a.Lq * a.H, row = blockIdx.x;
    const int64_t tok = row / a.H, b = tok / a.Lq;
    const int i = int(tok - b * a.Lq), t = threadIdx.x;
    const int64_t hrow = (b * a.H + (row - tok * a.H)) * a.Lq + i;
    // the sum or the maximum over the block, in a fixed order
    auto over = [&](float v, bool most) {
        for (int o = 16; o > 0; o >>= 1) {
            const float u = __shfl_xor_sync(0xffffffffu, v, o);
            v = most ? fmaxf(v, u) : v + u;
        }
        __syncthreads();
        if (t % 32 == 0) red[t / 32] = v;
        __syncthreads();
        v = red[0];
        for (int k = 1; k < 32; ++k) v = most ? fmaxf(v, red[k]) : v + red[k];
        return v;
    };
    const bool mine = t < a.nsplit;  // at most 256 parts
    float f = FWD ? 0.0f : a.scale;
    if (FWD) {
        const float *ml = a.part_ml + int64_t(t) * 2 * rows + hrow;
        const float mt = mine ? ml[0] : -INFINITY;
        const float m = over(mt, true), base = m == -INFINITY ? 0.0f : m;
        const float w = mine ? exp2f(mt - base) : 0.0f;
        if (t < 256) wt[t] = w;
        const float l = over(mine ? w * ml[rows] : 0.0f, false);
        const bool any = attn_row_has_keys(a, int(b), i);
        if (any) f = 1.0f / l;
        if (t == 0 && a.lse != nullptr)
            a.lse[hrow] = any ? (m + log2f(l)) * ATTN_LN2 : -INFINITY;
    } else if (a.rowsum != nullptr) {
        for (int e = 0; e < 4; ++e) {
            const float *w = a.rowsum + (int64_t(t) * 4 + e) * rows + hrow;
            const float v = over(mine ? *w : 0.0f, false);
            if (t == 0) a.rowsum[e * rows + hrow] = v;
        }
    }
    __syncthreads();
    // C channels at a time, 1024 / C threads for each
    const int C = a.D > 64 ? 128 : a.D > 32 ? 64 : 32, K = 1024 / C, k = t / C, c = t % C;
    float v = 0.0f;
    if (c < a.D)
#pragma unroll 8
        for (int s = k; s < a.nsplit; s += K) {
            const float p = a.part[(int64_t(s) * rows + row) * a.D + c];
            v = FWD ? fmaf(p, wt[s], v) : v + p;
        }
    part[t] = v;
    __syncthreads();
    if (k == 0 && c < a.D) {
        for (int u = 1; u < K; ++u) v += part[u * C + c];
        v = f == 0.0f ? 0.0f : v * f;
        Vec<T, 1>::store(static_cast<T *>(FWD ? a.out : a.dq) + row * a.D + c, &v);
        if (FWD && a.low != nullptr) {
            v = rest<T>(v);
            Vec<T, 1>::store(static_cast<T *>(a.low) + row * a.D + c, &v);
        }
    }
}

template <class T, int V>
void launch_join(const AttnArgs &a, int mode, int64_t rows, cudaStream_t st) {
    const int64_t n = rows * a.D;
    const unsigned g = unsigned((n / V + 255) / 256);
    if (mode == ATTN_FWD)
        attn_join_forward_kernel<T, V><<<g, 256, 0, st>>>(a);
    else
        attn_join_sum_kernel<T, V><<<dim3(g, mode == ATTN_DKV ? 2 : 1), 256, 0, st>>>(
            a.part, a.nsplit, n, a.scale, static_cast<T *>(mode == ATTN_DKV ? a.dk : a.dq),
            static_cast<T *>(a.dv));
}

// dslope_h = -sum over rows of (dS d2 - (dS) (P d2)), each row's sums joined
// over the parts first: a block per head, float64 over the rows (the GPU has few
// such units: 4 x 1021 rows of 6 heads take 13 us, with float64 in a row too 59), a
// fixed order.  A row's exact dS sum to 0; what they sum to here is the error of
// delta, and the second term takes its effect out.  The row's P are divided by what
// they sum to: lse, from which they come, is rounded to float32 (3e-7 of a weight at
// lse = 8), and where the forward pass formed the bias through the products and this
// one from differences it is off by up to 2^-20 slope R^2.
// With `tiles` the sums are already one number for each tile of a head's rows.
__global__ void __launch_bounds__(1024)
attn_slope_kernel(const AttnArgs a, int tiles, float *dslopes) {
    __shared__ double red[32];
    const int h = blockIdx.x;
    const int64_t n = int64_t(a.B) * a.H * a.Lq;
    double t = 0.0;
    if (tiles > 0) {
        for (int64_t r = threadIdx.x; r < int64_t(a.B) * tiles; r += 1024)
            t += double(a.rowsum[(r / tiles * a.H + h) * tiles + r % tiles]);
    } else {
        for (int64_t r = threadIdx.x; r < int64_t(a.B) * a.Lq; r += 1024) {
            const int64_t b = r / a.Lq, at = (b * a.H + h) * a.Lq + (r - b * a.Lq);
            LongSum w[4];
#pragma unroll 2  // (further, and the loads' registers spill)
            for (int s = 0; s < a.nsplit; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e].add(a.rowsum[(int64_t(s) * 4 + e) * n + at]);
            t += double(attn_slope_row(w[0].value(), w[1].value(), w[2].value(), w[3].value()));
        }
    }
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
        t = 0.0;
        for (int i = 0; i < 32; ++i) t += red[i];
        dslopes[h] = float(-t);
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
template <class T, int MODE, int DP>
cudaError_t simt_launch(const AttnArgs &a, bool vec, int64_t blocks, cudaStream_t st) {
    constexpr size_t smem = simt_smem(MODE, DP);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        allow_smem(attn_simt_kernel<T, MODE, DP>, int(smem), a.device, done);
    if (e != cudaSuccess) return e;
    attn_simt_kernel<T, MODE, DP><<<unsigned(blocks), ST, smem, st>>>(a, vec);
    return cudaGetLastError();
}

template <class T, int MODE>
cudaError_t simt_pick(const AttnArgs &a, bool vec, int64_t blocks, cudaStream_t st) {
    return a.D <= 64 ? simt_launch<T, MODE, 64>(a, vec, blocks, st)
                     : simt_launch<T, MODE, 128>(a, vec, blocks, st);
}

bool strides_fit(const AttnArgs &a, int v, size_t bytes) {
    auto ok = [&](const void *p, const int64_t *s) {
        return reinterpret_cast<uintptr_t>(p) % bytes == 0 && s[0] % v == 0 && s[1] % v == 0 &&
               s[2] % v == 0;
    };
    return a.D % v == 0 && ok(a.q, a.qs) && ok(a.k, a.ks) && ok(a.v, a.vs) &&
           reinterpret_cast<uintptr_t>(a.go) % bytes == 0;
}

struct Scratch {
    const DeviceInfo *dev;
    cudaStream_t st;
    void *p = nullptr;
    ~Scratch() {
        if (p != nullptr) scratch_free(p, st);
    }
    cudaError_t take(size_t bytes) { return scratch_alloc(*dev, &p, bytes, st); }
};

// Parts of the streamed side.  A block takes about `start` us before its
// first tile and `tile` us a tile; blocks run in waves of `slots`; parts have
// to be joined, which takes another launch and moves every partial sum twice.
// The number with the smallest estimate, at most 1 GiB of partial sums beyond
// what the longest part asks for.
// (Measured, one query over 100,000 keys, 8 heads of 64: 1 part 1029 us, 8
// parts 144, 19 parts 72, 38 parts 90; 256 queries and keys, 8 clouds of 8
// heads: 1 part 13 us, 2 parts 25.)
int pick_split(int64_t slots, int64_t base, int64_t items, int64_t part_floats, float start,
               float tile, int64_t most_items) {
    // no more than `most_items` a part, as far as 8 GiB and 256 parts allow
    int64_t first = (items + most_items - 1) / most_items;
    first = std::min(first, (int64_t(1) << 31) / std::max(part_floats, int64_t(1)));
    first = std::max(std::min(first, int64_t(256)), int64_t(1));
    int best = int(first);
    float least = INFINITY;
    for (int64_t n = first; n <= items && n <= 256; ++n) {
        if (n > first && n * part_floats > (int64_t(1) << 28)) break;
        const int64_t waves = (base * n + slots - 1) / slots, each = (items + n - 1) / n;
        float t = float(waves) * (start + tile * float(each));
        if (n > 1) t += 4.0f + float(n * part_floats) * (8.0f / 4e6f);
        if (t < least) least = t, best = int(n);
        if (n > first && base * (n - 1) > 4 * slots) break;  // more waves do not help
    }
    return best;
}

// Which kernels run a pass: few queries, tensor cores (bfloat16), tensor cores
// in three parts (float32), or float32 instructions (what is left: bfloat16
// rows that are not 16-byte aligned, sides without rows, and float32 with more
// clouds than three planes each are numbered in 32 bits).
enum AttnPath { PATH_FEW, PATH_TC, PATH_PARTS, PATH_SIMT };

template <class T>
AttnPath pick_path(const AttnArgs &a, bool backward) {
    if (attn_few_fits(a, sizeof(T), backward)) return PATH_FEW;
    if (sizeof(T) == 4) return attn_tc32_fits(a) ? PATH_PARTS : PATH_SIMT;
    return attn_tc_fits(a, backward ? ATTN_DQ : ATTN_FWD) ? PATH_TC : PATH_SIMT;
}

// A pass: its number of parts, blocks and scratch.
struct Pass {
    AttnArgs a;
    int mode;
    bool slopes;             // DQ: row sums for the slopes' gradient
    int64_t rows, ntile, base, blocks;
    size_t part, ml, floats;  // scratch: partial sums, forward statistics, all
};

template <class T>
Pass plan_pass(const DeviceInfo &dev, const AttnArgs &a, int mode, AttnPath path, bool slopes) {
    Pass p{a, mode, slopes};
    const bool dkv = mode == ATTN_DKV, wide = a.D > 64;
    const int64_t LX = dkv ? a.Lk : a.Lq, LY = dkv ? a.Lq : a.Lk, NH = dkv ? a.Hkv : a.H;
    const int64_t xr = path == PATH_TC      ? attn_tc_rows(mode)
                       : path == PATH_PARTS ? attn_tc32_rows(a, mode)
                                            : SB;
    const int64_t nyt = (LY + ATTN_TC_TILE - 1) / ATTN_TC_TILE;
    static_assert(SB == ATTN_TC_TILE, "all kernels stream tiles of 64 rows");
    p.ntile = (LX + xr - 1) / xr;
    p.base = p.ntile * NH * a.B;
    p.rows = int64_t(a.B) * LX * NH;
    // Two blocks fit a SM, one of the tensor-core kernels.  Us a tile takes
    // (measured with all its rows in use).
    const int64_t slots = int64_t(dev.sm_count) * (path == PATH_SIMT ? 2 : 1);
    const float tile = path == PATH_TC      ? (wide ? 1.4f : 1.1f)
                       : path == PATH_PARTS ? (mode == ATTN_FWD ? 1.7f : dkv ? 3.2f : 2.4f) *
                                                  (wide ? 2.0f : 1.0f)
                                            : (wide ? 12.0f : 6.0f);
    p.a.nsplit = path == PATH_FEW
                     ? attn_few_parts(dev, a, sizeof(T), mode == ATTN_DQ)
                     : pick_split(slots, p.base, dkv ? nyt * (a.H / a.Hkv) : nyt,
                                  p.rows * a.D * (dkv ? 2 : 1), 5.0f, tile,
                                  path == PATH_TC ? ATTN_TC_CHAIN : INT64_MAX / 2);
    p.blocks = p.base * p.a.nsplit;
    const size_t n = size_t(p.a.nsplit), hrows = size_t(a.B) * a.H * a.Lq;
    p.part = n > 1 ? n * size_t(p.rows) * a.D * (dkv ? 2 : 1) : 0;
    p.ml = n > 1 && mode == ATTN_FWD ? n * 2 * hrows : 0;
    p.floats = (p.part + p.ml + (slopes ? n * 4 * hrows + size_t(p.base) : 0) + 3) / 4 * 4;
    return p;
}

void place_pass(Pass &p, float *space) {
    p.a.part = space;
    p.a.part_ml = space + p.part;
    p.a.rowsum = p.slopes ? p.a.part_ml + p.ml : nullptr;
}

// What follows the kernel of a pass: its parts joined, the slopes' gradient.
template <class T>
void finish_pass(Pass &p, AttnPath path, float *dslopes, cudaStream_t st) {
    AttnArgs &a = p.a;
    const bool one_part = a.nsplit == 1;
    auto aligned = [](const void *q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
    if (!one_part) {
        // (8 rows of 64 in 152 parts: 27 us a thread per 4 channels, 8 us a block per row)
        if (p.mode != ATTN_DKV && a.nsplit >= 8 && p.rows <= 4096) {
            if (p.mode == ATTN_FWD)
                attn_join_rows_kernel<T, true><<<unsigned(p.rows), 1024, 0, st>>>(a);
            else
                attn_join_rows_kernel<T, false><<<unsigned(p.rows), 1024, 0, st>>>(a);
            a.nsplit = 1;  // for the slopes' sums
        } else if (a.D % 4 == 0 && aligned(a.out) && aligned(a.low) && aligned(a.dq) &&
                   aligned(a.dk) && aligned(a.dv)) {
            launch_join<T, 4>(a, p.mode, p.rows, st);
        } else {
            launch_join<T, 1>(a, p.mode, p.rows, st);
        }
    }
    if (p.slopes)
        attn_slope_kernel<<<a.H, 1024, 0, st>>>(
            a, (path == PATH_TC || path == PATH_PARTS) && one_part ? int(p.ntile) : 0, dslopes);
}

template <class T>
cudaError_t run_forward(const DeviceInfo &dev, const AttnArgs &a, cudaStream_t st) {
    const AttnPath path = pick_path<T>(a, false);
    Pass p = plan_pass<T>(dev, a, ATTN_FWD, path, false);
    if (p.blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    Scratch ws{&dev, st};
    const size_t bytes =
        p.floats * sizeof(float) + (path == PATH_PARTS ? attn_split_bytes(a, false) : 0);
    cudaError_t e = bytes > 0 ? ws.take(bytes) : cudaSuccess;
    if (e != cudaSuccess) return e;
    float *space = static_cast<float *>(ws.p);
    place_pass(p, space);
    if (path == PATH_FEW) {
        e = launch_attn_few(p.a, sizeof(T), false, st);
    } else if (path == PATH_TC) {
        e = launch_attn_tc_forward(p.a, unsigned(p.blocks), st);
    } else if (path == PATH_PARTS) {
        AttnSplit s;
        e = launch_attn_split(a, false, space + p.floats, &s, st);
        if (e == cudaSuccess) e = launch_attn_tc32_forward(p.a, s, unsigned(p.blocks), st);
    } else {
        e = simt_pick<T, ATTN_FWD>(p.a, strides_fit(a, 4, 4 * sizeof(T)), p.blocks, st);
    }
    if (e != cudaSuccess) return e;
    finish_pass<T>(p, path, nullptr, st);
    return cudaGetLastError();
}

template <class T>
cudaError_t run_backward(const DeviceInfo &dev, AttnArgs a, const void *out, const void *low,
                         float *dslopes, cudaStream_t st) {
    const int64_t rows = int64_t(a.B) * a.Lq * a.H;
    const int64_t keys = a.dk == nullptr ? 0 : int64_t(a.B) * a.Lk * a.Hkv;
    const bool slopes = dslopes != nullptr && a.slopes != nullptr;
    if (rows == 0) {  // no queries: the keys' gradients are 0
        const size_t n = size_t(keys) * a.D * sizeof(T);
        cudaError_t e = slopes ? cudaMemsetAsync(dslopes, 0, size_t(a.H) * 4, st) : cudaSuccess;
        if (e == cudaSuccess && n > 0) e = cudaMemsetAsync(a.dk, 0, n, st);
        if (e == cudaSuccess && n > 0) e = cudaMemsetAsync(a.dv, 0, n, st);
        return e;
    }
    if (a.dq == nullptr && keys == 0) return cudaSuccess;
    const AttnPath path = pick_path<T>(a, true);
    Pass dq = plan_pass<T>(dev, a, ATTN_DQ, path, slopes);
    Pass dkv = plan_pass<T>(dev, a, ATTN_DKV, path == PATH_FEW ? PATH_SIMT : path, false);
    // no such pass (few queries: one kernel forms all)
    if (path == PATH_FEW || keys == 0) dkv.blocks = 0, dkv.part = dkv.floats = 0;
    if (a.dq == nullptr) {
        if (path != PATH_FEW) dq.blocks = 0;
        dq.part = dq.floats = 0;
    }
    if (dq.blocks + dkv.blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const size_t sides = (size_t(rows) * 2 + 3) / 4 * 4;  // delta, lse2
    // a bfloat16 output without its low part: both again (a multiple of 16 bytes each)
    const bool again = sizeof(T) == 2 && low == nullptr;
    const size_t outs = again ? (size_t(rows) * a.D + 7) / 8 * 8 : 0;
    const size_t tail = 2 * outs * sizeof(T);
    Scratch ws{&dev, st};
    cudaError_t e = ws.take((sides + dq.floats + dkv.floats) * sizeof(float) + tail +
                            (path == PATH_PARTS ? attn_split_bytes(a, true) : 0));
    if (e != cudaSuccess) return e;
    if (again) {
        AttnArgs f = a;
        f.out = static_cast<char *>(ws.p) + (sides + dq.floats + dkv.floats) * sizeof(float);
        f.low = static_cast<T *>(f.out) + outs;
        f.lse = nullptr;
        f.dq = f.dk = f.dv = nullptr;
        if ((e = run_forward<T>(dev, f, st)) != cudaSuccess) return e;
        out = f.out, low = f.low;
    }
    float *delta = static_cast<float *>(ws.p), *space = delta + sides;
    dq.a.delta = dkv.a.delta = delta;
    dq.a.lse2 = dkv.a.lse2 = delta + rows;
    place_pass(dq, space);
    place_pass(dkv, space + dq.floats);
    launch_delta<T>(a, static_cast<const T *>(out), static_cast<const T *>(low), rows, delta,
                    delta + rows, st);
    const unsigned nq = unsigned(dq.blocks), nk = unsigned(dkv.blocks);
    if (path == PATH_FEW) {
        e = launch_attn_few(dq.a, sizeof(T), true, st);
    } else if (path == PATH_TC) {
        e = launch_attn_tc_backward(dkv.a, nk, dq.a, nq, st);
    } else if (path == PATH_PARTS) {
        AttnSplit s;
        e = launch_attn_split(a, true, space + dq.floats + dkv.floats, &s, st);
        if (e == cudaSuccess) e = launch_attn_tc32_backward(dkv.a, nk, dq.a, nq, s, st);
    } else {
        const bool vec = strides_fit(a, 4, 4 * sizeof(T));
        e = nq > 0 ? simt_pick<T, ATTN_DQ>(dq.a, vec, nq, st) : cudaSuccess;
        if (e == cudaSuccess && nk > 0) e = simt_pick<T, ATTN_DKV>(dkv.a, vec, nk, st);
    }
    if (e != cudaSuccess) return e;
    if (nk > 0) finish_pass<T>(dkv, path, nullptr, st);
    if (a.dq != nullptr) finish_pass<T>(dq, path, dslopes, st);
    return cudaGetLastError();
}

// The checks both directions share; fills `a`.  *done: nothing to run.
int attn_check(const char *what, AttnArgs &a, const DeviceInfo **dev, const void *q,
               const void *k, const void *v, int dtype, int64_t B, int64_t Lq, int64_t Lk,
               int64_t H, int64_t Hkv, int64_t D, const int64_t *qs, const int64_t *ks,
               const int64_t *vs, double scale, const float *qxyz, const float *rxyz,
               const float *slopes, const int64_t *qlen, const int64_t *rlen) {
    char m[220];
    auto bad = [&](int code, const char *why) {
        std::snprintf(m, sizeof(m), "%s: %s", what, why);
        return api_fail(code, m);
    };
    if (B < 0 || Lq < 0 || Lk < 0 || H < 0 || Hkv < 0)
        return bad(PC_ERR_INVALID_ARGUMENT, "negative size");
    if (D < 1) return bad(PC_ERR_INVALID_ARGUMENT, "D must be at least 1");
    if (dtype != PC_F32 && dtype != PC_BF16)
        return bad(PC_ERR_INVALID_ARGUMENT, "dtype must be PC_F32 or PC_BF16");
    if (H > 0 && (Hkv < 1 || H % Hkv != 0))
        return bad(PC_ERR_INVALID_ARGUMENT, "Hkv must divide H");
    // (the kernels divide the slopes by it in float32)
    if (!(scale >= 1e-30 && scale <= 1e30))
        return bad(PC_ERR_INVALID_ARGUMENT, "scale must be between 1e-30 and 1e30");
    // (an empty side has no positions to point at)
    if (slopes != nullptr ? (qxyz == nullptr && B > 0 && Lq > 0) || (rxyz == nullptr && B > 0 && Lk > 0)
                          : qxyz != nullptr || rxyz != nullptr)
        return bad(PC_ERR_INVALID_ARGUMENT, "slopes, query_xyz and ref_xyz go together");
    if (D > 128) return bad(PC_ERR_UNSUPPORTED, "D above 128");
    const int64_t lim = int64_t(1) << 30;
    if (Lq > lim || Lk > lim || B > lim || H > 65536 ||
        (B > 0 && H > 0 && (Lq > Lk ? Lq : Lk) > (int64_t(1) << 36) / (B * H)))
        return bad(PC_ERR_UNSUPPORTED, "sizes beyond what the kernels index");
    a.B = int(B), a.Lq = int(Lq), a.Lk = int(Lk), a.H = int(H), a.Hkv = int(Hkv);
    a.D = int(D), a.scale = float(scale), a.nsplit = 1;
    auto strides = [&](int64_t *to, const int64_t *s, int64_t L, int64_t heads) {
        to[0] = s ? s[0] : L * heads * D;
        to[1] = s ? s[1] : heads * D;
        to[2] = s ? s[2] : D;
    };
    strides(a.qs, qs, Lq, H);
    strides(a.ks, ks, Lk, Hkv);
    strides(a.vs, vs, Lk, Hkv);
    a.q = q, a.k = k, a.v = v, a.slopes = slopes, a.qxyz = qxyz, a.rxyz = rxyz;
    a.qlen = qlen, a.rlen = rlen;
    if (B == 0 || H == 0 || (Lq == 0 && Lk == 0)) return PC_OK;
    int rc = api_current_device(dev);
    if (rc != PC_OK) return rc;
    const int d = (*dev)->device;
    const size_t es = dtype == PC_F32 ? 4 : 2;
    a.device = d;
    a.status = (*dev)->status_word;
    a.timeout_ns = wait_timeout_ns();
    if (Lq > 0 && (rc = api_check_ptr(q, d, es, "q")) != PC_OK) return rc;
    if (Lk > 0) {
        if ((rc = api_check_ptr(k, d, es, "k")) != PC_OK) return rc;
        if ((rc = api_check_ptr(v, d, es, "v")) != PC_OK) return rc;
    }
    if (slopes) {
        if ((rc = api_check_ptr(slopes, d, 4, "slopes")) != PC_OK) return rc;
        if (Lq > 0 && (rc = api_check_ptr(qxyz, d, 4, "query_xyz")) != PC_OK) return rc;
        if (Lk > 0 && (rc = api_check_ptr(rxyz, d, 4, "ref_xyz")) != PC_OK) return rc;
    }
    if (qlen && (rc = api_check_ptr(qlen, d, 8, "query_lengths")) != PC_OK) return rc;
    if (rlen && (rc = api_check_ptr(rlen, d, 8, "ref_lengths")) != PC_OK) return rc;
    return PC_OK;
}

int attn_cuda(const char *what, cudaError_t e) {
    if (e == cudaSuccess) return PC_OK;
    char m[200];
    std::snprintf(m, sizeof(m), "%s: %s", what, cudaGetErrorString(e));
    return api_fail(PC_ERR_CUDA, m);
}

}  // namespace
}  // namespace pcn

extern "C" int pc_attention(const void *q, const void *k, const void *v, int dtype, int64_t B,
                            int64_t Lq, int64_t Lk, int64_t H, int64_t Hkv, int64_t D,
                            const int64_t *q_strides, const int64_t *k_strides,
                            const int64_t *v_strides, double scale, const float *query_xyz,
                            const float *ref_xyz, const float *slopes,
                            const int64_t *query_lengths, const int64_t *ref_lengths,
                            void *out, float *out_lse, void *stream) {
    return pc_attention_ex(q, k, v, dtype, B, Lq, Lk, H, Hkv, D, q_strides, k_strides, v_strides,
                           scale, query_xyz, ref_xyz, slopes, query_lengths, ref_lengths, out,
                           nullptr, out_lse, stream);
}

extern "C" int pc_attention_ex(const void *q, const void *k, const void *v, int dtype, int64_t B,
                               int64_t Lq, int64_t Lk, int64_t H, int64_t Hkv, int64_t D,
                               const int64_t *q_strides, const int64_t *k_strides,
                               const int64_t *v_strides, double scale, const float *query_xyz,
                               const float *ref_xyz, const float *slopes,
                               const int64_t *query_lengths, const int64_t *ref_lengths,
                               void *out, void *out_low, float *out_lse, void *stream) {
    using namespace pcn;
    AttnArgs a{};
    const DeviceInfo *dev = nullptr;
    int rc = attn_check("attention", a, &dev, q, k, v, dtype, B, Lq, Lk, H, Hkv, D, q_strides,
                        k_strides, v_strides, scale, query_xyz, ref_xyz, slopes, query_lengths,
                        ref_lengths);
    if (rc != PC_OK) return rc;
    if (out_low != nullptr && dtype != PC_BF16)
        return api_fail(PC_ERR_INVALID_ARGUMENT, "attention: out_low is of a bfloat16 output");
    if (dev == nullptr || Lq == 0) return PC_OK;
    const int d = dev->device;
    if ((rc = api_check_ptr(out, d, dtype == PC_F32 ? 4 : 2, "out")) != PC_OK) return rc;
    if (out_low && (rc = api_check_ptr(out_low, d, 2, "out_low")) != PC_OK) return rc;
    if (out_lse && (rc = api_check_ptr(out_lse, d, 4, "out_lse")) != PC_OK) return rc;
    a.out = out, a.low = out_low, a.lse = out_lse;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == PC_F32 ? run_forward<float>(*dev, a, st)
                                          : run_forward<bf16>(*dev, a, st);
    return attn_cuda("attention", e);
}

extern "C" int pc_attention_backward(
    const void *grad_out, const void *q, const void *k, const void *v, const void *out,
    const float *lse, int dtype, int64_t B, int64_t Lq, int64_t Lk, int64_t H, int64_t Hkv,
    int64_t D, const int64_t *q_strides, const int64_t *k_strides, const int64_t *v_strides,
    double scale, const float *query_xyz, const float *ref_xyz, const float *slopes,
    const int64_t *query_lengths, const int64_t *ref_lengths, void *grad_q, void *grad_k,
    void *grad_v, float *grad_slopes, void *stream) {
    return pc_attention_backward_ex(grad_out, q, k, v, out, nullptr, lse, dtype, B, Lq, Lk, H,
                                    Hkv, D, q_strides, k_strides, v_strides, scale, query_xyz,
                                    ref_xyz, slopes, query_lengths, ref_lengths, grad_q, grad_k,
                                    grad_v, grad_slopes, stream);
}

extern "C" int pc_attention_backward_ex(
    const void *grad_out, const void *q, const void *k, const void *v, const void *out,
    const void *out_low, const float *lse, int dtype, int64_t B, int64_t Lq, int64_t Lk,
    int64_t H, int64_t Hkv, int64_t D, const int64_t *q_strides, const int64_t *k_strides,
    const int64_t *v_strides, double scale, const float *query_xyz, const float *ref_xyz,
    const float *slopes, const int64_t *query_lengths, const int64_t *ref_lengths, void *grad_q,
    void *grad_k, void *grad_v, float *grad_slopes, void *stream) {
    using namespace pcn;
    const bool empty_q = B == 0 || Lq == 0 || H == 0, empty_k = B == 0 || Lk == 0 || H == 0;
    if ((!empty_k && (grad_k == nullptr) != (grad_v == nullptr)) ||
        (!empty_q && grad_q == nullptr && grad_slopes != nullptr))
        return api_fail(PC_ERR_INVALID_ARGUMENT,
                        "attention_backward: grad_k and grad_v go together, grad_slopes needs "
                        "grad_q");
    AttnArgs a{};
    const DeviceInfo *dev = nullptr;
    int rc = attn_check("attention_backward", a, &dev, q, k, v, dtype, B, Lq, Lk, H, Hkv, D,
                        q_strides, k_strides, v_strides, scale, query_xyz, ref_xyz, slopes,
                        query_lengths, ref_lengths);
    if (rc != PC_OK) return rc;
    if (grad_slopes != nullptr && slopes == nullptr)
        return api_fail(PC_ERR_INVALID_ARGUMENT, "attention_backward: grad_slopes without slopes");
    if (out_low != nullptr && dtype != PC_BF16)
        return api_fail(PC_ERR_INVALID_ARGUMENT,
                        "attention_backward: out_low is of a bfloat16 output");
    if (dev == nullptr) {  // an empty problem: only the slopes' gradient can have elements
        if (grad_slopes == nullptr || H == 0) return PC_OK;
        if ((rc = api_current_device(&dev)) != PC_OK) return rc;
        if ((rc = api_check_ptr(grad_slopes, dev->device, 4, "grad_slopes")) != PC_OK) return rc;
        return attn_cuda("attention_backward",
                         cudaMemsetAsync(grad_slopes, 0, size_t(H) * 4,
                                         static_cast<cudaStream_t>(stream)));
    }
    const int d = dev->device;
    const size_t es = dtype == PC_F32 ? 4 : 2;
    if (Lq > 0) {
        if ((rc = api_check_ptr(grad_out, d, es, "grad_out")) != PC_OK) return rc;
        if ((rc = api_check_ptr(out, d, es, "out")) != PC_OK) return rc;
        if (out_low && (rc = api_check_ptr(out_low, d, 2, "out_low")) != PC_OK) return rc;
        if ((rc = api_check_ptr(lse, d, 4, "lse")) != PC_OK) return rc;
        if (grad_q && (rc = api_check_ptr(grad_q, d, es, "grad_q")) != PC_OK) return rc;
    }
    if (Lk > 0 && grad_k) {
        if ((rc = api_check_ptr(grad_k, d, es, "grad_k")) != PC_OK) return rc;
        if ((rc = api_check_ptr(grad_v, d, es, "grad_v")) != PC_OK) return rc;
    }
    if (grad_slopes && (rc = api_check_ptr(grad_slopes, d, 4, "grad_slopes")) != PC_OK)
        return rc;
    a.go = grad_out, a.lse = const_cast<float *>(lse);
    a.dq = grad_q, a.dk = grad_k, a.dv = grad_v;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == PC_F32
                              ? run_backward<float>(*dev, a, out, nullptr, grad_slopes, st)
                              : run_backward<bf16>(*dev, a, out, out_low, grad_slopes, st);
    return attn_cuda("attention_backward", e);
}
