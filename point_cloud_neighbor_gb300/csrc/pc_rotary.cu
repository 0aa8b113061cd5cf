// pc_rotary.cu -- rotary positions with several axes, for queries and keys in
// one launch.
//
//   pair p = a F + f of a head's channels turns by t = position[a] freq[a, f]:
//     (u, v) -> (u cos t - v sin t, v cos t + u sin t),
//   p < R = A F; channels past the 2 R turned ones are copied.  A pair is
//   channels (2p, 2p + 1) (interleaved) or (p, R + p) (half-split).  The
//   gradient is the same turn by -t.
//
// Bound: memory (every element read and written once; 6 flops a pair).  The
// sines and cosines depend on the token and the pair only: a block computes
// those of its tokens once, in shared memory.  A thread takes V channels (16
// bytes) of one token: it keeps their sines and cosines in registers and goes
// over the heads, several loads at a time, the first of them issued before
// the block's sines are ready.
//
// Measured: 32 x 512 tokens, 6 + 6 heads of 64 in float32 18 us (5.7 TB/s);
// 16,384 tokens, 16 + 4 heads of 128 in bfloat16, interleaved 37 us (4.5 TB/s),
// half-split with 63 pairs 52 us: its partners start 7 elements into a vector
// and are read as two vectors each.
//
// The product position * freq is formed exactly (its rounding error by FMA)
// and the error enters the sine and cosine to first order, so the angle
// loses nothing to the float32 product at large coordinates.
#include "pc_internal.h"
#include "pc_vec.cuh"
#include "pointcloud.h"

#include <cmath>
#include <cstdio>

namespace pcn {
namespace {

constexpr int ROT_THREADS = 128;
constexpr int ROT_MAX_PAIRS = 4096;   // (cos, sin) of one token in 32 KB
constexpr int ROT_MAX_D = 16384;

struct RotTensor {
    const void *x = nullptr;
    void *y = nullptr;        // [B, L, heads, D] packed
    int64_t sb = 0, sl = 0, sh = 0;  // strides of x in elements
    int heads = 0;
};

struct RotArgs {
    RotTensor q, k;
    const float *pos, *freq;
    int64_t tokens;  // B L
    int L, D, A, F, T;
    int heads_each;  // heads of a group
    float sign;
    FastDiv per_token, per_group, pairs, by_l;  // per_group: units of a head
};

template <class T, int V>
struct alignas(V * sizeof(T)) RotChunk {  // V channels as they are in memory
    T e[V];
    __device__ __forceinline__ void load(const T *p) {
        *this = *reinterpret_cast<const RotChunk *>(p);
    }
};

// (cos, sin) of the block's tokens: cs[token][R]
__device__ __forceinline__ void rot_table(const RotArgs &a, float2 *cs, int64_t t0, int nt,
                                          int R) {
    for (int i = threadIdx.x; i < nt * R; i += ROT_THREADS) {
        const int tk = a.pairs.div(i), p = i - tk * R;
        const int ax = p / a.F;
        const float pos = a.pos[(t0 + tk) * a.A + ax], f = a.freq[p];
        const float ang = pos * f;
        const float err = fmaf(pos, f, -ang);
        float s, c;
        sincosf(ang, &s, &c);
        cs[i] = make_float2(fmaf(-s, err, c), a.sign * fmaf(c, err, s));
    }
}

// V channels from V u on of every head of a thread's group.  In a half-split
// row the partners of V channels are V channels R away, which start S = R mod V
// elements into a vector: they come from the two vectors that hold them.
// Channels below R have them at c0 + R = lo + S on, those below 2 R at
// c0 - R = hi + (V - S) on; one unit of a row may hold both kinds.
template <class T, int V, bool INTER, int S>
__global__ void __launch_bounds__(ROT_THREADS) rotary_kernel(const RotArgs a) {
    extern __shared__ float2 cs[];
    constexpr int HB = INTER ? 4 : 2;         // heads on their way at once
    constexpr int NW = INTER ? V / 2 : V;
    using Chunk = RotChunk<T, V>;
    const int R = a.A * a.F;
    const int64_t t0 = int64_t(blockIdx.x) * a.T;
    const int nt = int(min(int64_t(a.T), a.tokens - t0));
    const int heads = a.q.heads + a.k.heads;
    const int n = nt * int(a.per_token.d);
    bool ready = false;
    for (int i0 = 0; i0 < n; i0 += ROT_THREADS) {
        const int i = min(i0 + int(threadIdx.x), n - 1);
        const bool in = i0 + int(threadIdx.x) < n;
        const int tk = a.per_token.div(i);
        const int r = i - tk * int(a.per_token.d);
        const int group = a.per_group.div(r);
        const int u = r - group * int(a.per_group.d);
        const int64_t tok = t0 + tk, b = a.by_l.div(uint32_t(tok)), l = tok - b * a.L;
        const int c0 = u * V;
        const int64_t qo = b * a.q.sb + l * a.q.sl, ko = b * a.k.sb + l * a.k.sl;
        const int h0 = group * a.heads_each, h1 = in ? min(heads, h0 + a.heads_each) : h0;
        const bool low = c0 < R, high = !INTER && c0 + V > R && c0 < 2 * R;
        const int lo = c0 + R - S, hi = c0 - R + S - (S > 0 ? V : 0);
        const int at = low ? lo : hi;  // of the unit's first kind
        Chunk own[HB], pa[HB], pb[HB], qa[HB], qb[HB];
        auto source = [&](int h) {
            return h < a.q.heads ? static_cast<const T *>(a.q.x) + qo + h * a.q.sh
                                 : static_cast<const T *>(a.k.x) + ko + (h - a.q.heads) * a.k.sh;
        };
        auto fetch = [&](int h) {
#pragma unroll
            for (int j = 0; j < HB; ++j)
                if (h + j < h1) {
                    const T *x = source(h + j);
                    own[j].load(x + c0);
                    if (!INTER && c0 < 2 * R) {
                        if (at >= 0) pa[j].load(x + at);
                        if (S > 0 && at + V < a.D) pb[j].load(x + at + V);
                        if (S > 0 && low && high) {
                            if (hi >= 0) qa[j].load(x + hi);
                            qb[j].load(x + hi + V);
                        }
                    }
                }
        };
        fetch(h0);
        if (!ready) {  // (every thread comes here in its first round)
            rot_table(a, cs, t0, nt, R);
            __syncthreads();
            ready = true;
        }
        // cosines and signed sines of the unit
        float2 w[NW];
#pragma unroll
        for (int e = 0; e < NW; ++e) {
            const int c = u * NW + e;
            const bool first = c < R, turned = c < (INTER ? R : 2 * R);
            w[e] = turned ? cs[tk * R + (first ? c : c - R)] : make_float2(1.0f, 0.0f);
            if (!INTER && first) w[e].y = -w[e].y;
        }
        for (int h = h0; h < h1; h += HB) {
            T *y[HB];
            float v[HB][V];
#pragma unroll
            for (int j = 0; j < HB; ++j) {
                const int hh = h + j;
                y[j] = hh < a.q.heads
                           ? static_cast<T *>(a.q.y) + (tok * a.q.heads + hh) * a.D + c0
                           : static_cast<T *>(a.k.y) +
                                 (tok * a.k.heads + hh - a.q.heads) * a.D + c0;
                Vec<T, V>::load(own[j].e, v[j]);
                if (INTER) {
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) {
                        const float p0 = v[j][2 * e], p1 = v[j][2 * e + 1];
                        if (u * NW + e < R) {
                            v[j][2 * e] = fmaf(p0, w[e].x, -(p1 * w[e].y));
                            v[j][2 * e + 1] = fmaf(p1, w[e].x, p0 * w[e].y);
                        }
                    }
                } else if (c0 < 2 * R) {
                    float p[2 * V], o[V];
                    Vec<T, V>::load(pa[j].e, p);
                    if (S > 0) Vec<T, V>::load(pb[j].e, p + V);
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        o[e] = S == 0 ? p[e] : low ? p[e + S] : p[e + (V - S) % V];
                    if (S > 0 && low && high) {
                        Vec<T, V>::load(qa[j].e, p);
                        Vec<T, V>::load(qb[j].e, p + V);
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            if (c0 + e >= R) o[e] = p[e + (V - S) % V];
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (c0 + e < 2 * R) v[j][e] = fmaf(v[j][e], w[e].x, o[e] * w[e].y);
                }
            }
            if (h + HB < h1) fetch(h + HB);
#pragma unroll
            for (int j = 0; j < HB; ++j)
                if (h + j < h1) Vec<T, V>::store(y[j], v[j]);
        }
    }
}

// Any alignment: one pair, or one copied channel, at a time.
template <class T, bool INTER>
__global__ void __launch_bounds__(ROT_THREADS) rotary_scalar_kernel(const RotArgs a) {
    extern __shared__ float2 cs[];
    const int R = a.A * a.F;
    const int64_t t0 = int64_t(blockIdx.x) * a.T;
    const int nt = int(min(int64_t(a.T), a.tokens - t0));
    rot_table(a, cs, t0, nt, R);
    __syncthreads();
    const int n = nt * int(a.per_token.d);
    for (int i = threadIdx.x; i < n; i += ROT_THREADS) {
        const int tk = a.per_token.div(i);
        const int r = i - tk * int(a.per_token.d);
        int h = a.per_group.div(r);
        const int u = r - h * int(a.per_group.d);
        const int64_t tok = t0 + tk, b = a.by_l.div(uint32_t(tok));
        const RotTensor &t = h < a.q.heads ? a.q : a.k;
        if (h >= a.q.heads) h -= a.q.heads;
        const T *x = static_cast<const T *>(t.x) + b * t.sb + (tok - b * a.L) * t.sl +
                     int64_t(h) * t.sh;
        T *y = static_cast<T *>(t.y) + (tok * t.heads + h) * a.D;
        if (u < R) {
            const int c0 = INTER ? 2 * u : u, c1 = INTER ? 2 * u + 1 : R + u;
            const float2 w = cs[tk * R + u];
            float p0, p1;
            Vec<T, 1>::load(x + c0, &p0);
            Vec<T, 1>::load(x + c1, &p1);
            const float q0 = fmaf(p0, w.x, -(p1 * w.y)), q1 = fmaf(p1, w.x, p0 * w.y);
            Vec<T, 1>::store(y + c0, &q0);
            Vec<T, 1>::store(y + c1, &q1);
        } else {
            y[R + u] = x[R + u];
        }
    }
}

bool rot_fits(const RotTensor &t, int D, int v, size_t es) {
    if (t.heads == 0) return true;
    return D % v == 0 && t.sb % v == 0 && t.sl % v == 0 && t.sh % v == 0 &&
           reinterpret_cast<uintptr_t>(t.x) % (v * es) == 0 &&
           reinterpret_cast<uintptr_t>(t.y) % (v * es) == 0;
}

template <class T, int V, bool INTER, int S>
cudaError_t rot_launch(const DeviceInfo &dev, RotArgs a, cudaStream_t st) {
    const int R = a.A * a.F, units = V > 1 ? a.D / V : a.D - R;
    const int heads = a.q.heads + a.k.heads;
    // Heads of a group: all of them, unless the tokens are too few to give every
    // SM 1024 threads.
    int64_t groups = heads;
    if (V > 1) {
        const int64_t one = a.tokens * units, want = int64_t(dev.sm_count) * 1024;
        groups = (want + one - 1) / one;
        if (groups > heads) groups = heads;
    }
    a.heads_each = int((heads + groups - 1) / groups);
    const int64_t per = int64_t(units) * ((heads + a.heads_each - 1) / a.heads_each);
    // Tokens of a block: one unit a thread (so that the sines are shared out
    // among all threads), but first enough blocks for the GPU, and the block's
    // sines within 32 KB.
    int64_t T_ = (V > 1 ? ROT_THREADS : 4 * ROT_THREADS) / per;
    const int64_t spread = (a.tokens + dev.sm_count - 1) / dev.sm_count;
    if (T_ > spread) T_ = spread;
    if (R > 0 && T_ > ROT_MAX_PAIRS / R) T_ = ROT_MAX_PAIRS / R;
    if (T_ < 1) T_ = 1;
    a.T = int(T_);
    a.per_group = FastDiv(uint32_t(units));
    a.per_token = FastDiv(uint32_t(per));
    a.pairs = FastDiv(uint32_t(R > 0 ? R : 1));
    a.by_l = FastDiv(uint32_t(a.L));
    const unsigned blocks = unsigned((a.tokens + a.T - 1) / a.T);
    const size_t smem = size_t(a.T) * R * sizeof(float2);
    if constexpr (V > 1)
        rotary_kernel<T, V, INTER, S><<<blocks, ROT_THREADS, smem, st>>>(a);
    else
        rotary_scalar_kernel<T, INTER><<<blocks, ROT_THREADS, smem, st>>>(a);
    return cudaGetLastError();
}

template <class T>
cudaError_t rot_dispatch(const DeviceInfo &dev, const RotArgs &a, bool inter,
                         cudaStream_t st) {
    constexpr int W = 16 / sizeof(T);
    const bool wide = rot_fits(a.q, a.D, W, sizeof(T)) && rot_fits(a.k, a.D, W, sizeof(T));
    if (inter)
        return wide ? rot_launch<T, W, true, 0>(dev, a, st)
                    : rot_launch<T, 1, true, 0>(dev, a, st);
    if (!wide) return rot_launch<T, 1, false, 0>(dev, a, st);
    switch (a.A * a.F % W) {
        case 0: return rot_launch<T, W, false, 0>(dev, a, st);
        case 1: return rot_launch<T, W, false, 1>(dev, a, st);
        case 2: return rot_launch<T, W, false, 2>(dev, a, st);
        case 3: return rot_launch<T, W, false, 3>(dev, a, st);
        case 4: return rot_launch<T, W, false, 4 % W>(dev, a, st);
        case 5: return rot_launch<T, W, false, 5 % W>(dev, a, st);
        case 6: return rot_launch<T, W, false, 6 % W>(dev, a, st);
        default: return rot_launch<T, W, false, 7 % W>(dev, a, st);
    }
}

}  // namespace
}  // namespace pcn

extern "C" int pc_rotary(const void *q, const void *k, int dtype, int64_t B, int64_t L,
                         int64_t H, int64_t Hkv, int64_t D, const int64_t *q_strides,
                         const int64_t *k_strides, const float *positions,
                         const float *freqs, int64_t A, int64_t F, int flags, void *out_q,
                         void *out_k, void *stream) {
    using namespace pcn;
    char m[200];
    if (B < 0 || L < 0 || H < 0 || Hkv < 0 || D < 0 || F < 0)
        return api_fail(PC_ERR_INVALID_ARGUMENT, "rotary: negative size");
    if (dtype != PC_F32 && dtype != PC_BF16)
        return api_fail(PC_ERR_INVALID_ARGUMENT, "rotary: dtype must be PC_F32 or PC_BF16");
    if (flags & ~(PC_ROTARY_HALF_SPLIT | PC_ROTARY_INVERSE))
        return api_fail(PC_ERR_INVALID_ARGUMENT, "rotary: unknown flags");
    if (A < 1 || A > 4) {
        std::snprintf(m, sizeof(m), "rotary: 1 <= A <= 4 axes (got %lld)", (long long)A);
        return api_fail(PC_ERR_INVALID_ARGUMENT, m);
    }
    if (F > D || 2 * A * F > D) {
        std::snprintf(m, sizeof(m), "rotary: 2 A F = %lld turned channels of D = %lld",
                      (long long)(2 * A * F), (long long)D);
        return api_fail(PC_ERR_INVALID_ARGUMENT, m);
    }
    if (D > ROT_MAX_D || A * F > ROT_MAX_PAIRS || H > 65536 || Hkv > 65536 ||
        D * (H + Hkv) > (int64_t(1) << 26) || L >= (int64_t(1) << 31) ||
        (L > 0 && B >= (int64_t(1) << 31) / L))
        return api_fail(PC_ERR_UNSUPPORTED, "rotary: sizes beyond what the kernel runs");
    if (B == 0 || L == 0 || D == 0 || H + Hkv == 0) return PC_OK;
    const DeviceInfo *dev = nullptr;
    int rc = api_current_device(&dev);
    if (rc != PC_OK) return rc;
    const int d = dev->device;
    const size_t es = dtype == PC_F32 ? 4 : 2;
    RotArgs a{};
    auto take = [&](RotTensor &t, const void *x, void *y, int64_t heads,
                    const int64_t *s, const char *xn, const char *yn) {
        if (heads == 0) return int(PC_OK);
        int r;
        if ((r = api_check_ptr(x, d, es, xn)) != PC_OK) return r;
        if ((r = api_check_ptr(y, d, es, yn)) != PC_OK) return r;
        t.x = x, t.y = y, t.heads = int(heads);
        t.sb = s ? s[0] : L * heads * D;
        t.sl = s ? s[1] : heads * D;
        t.sh = s ? s[2] : D;
        return int(PC_OK);
    };
    if ((rc = take(a.q, q, out_q, H, q_strides, "q", "out_q")) != PC_OK) return rc;
    if ((rc = take(a.k, k, out_k, Hkv, k_strides, "k", "out_k")) != PC_OK) return rc;
    if (F > 0) {
        if ((rc = api_check_ptr(positions, d, 4, "positions")) != PC_OK) return rc;
        if ((rc = api_check_ptr(freqs, d, 4, "freqs")) != PC_OK) return rc;
    }
    a.pos = positions, a.freq = freqs;
    a.tokens = B * L, a.L = int(L), a.D = int(D), a.A = int(A), a.F = int(F);
    a.sign = (flags & PC_ROTARY_INVERSE) ? -1.0f : 1.0f;
    const bool inter = !(flags & PC_ROTARY_HALF_SPLIT);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == PC_F32 ? rot_dispatch<float>(*dev, a, inter, st)
                                          : rot_dispatch<bf16>(*dev, a, inter, st);
    if (e != cudaSuccess) {
        std::snprintf(m, sizeof(m), "rotary: %s", cudaGetErrorString(e));
        return api_fail(PC_ERR_CUDA, m);
    }
    return PC_OK;
}
