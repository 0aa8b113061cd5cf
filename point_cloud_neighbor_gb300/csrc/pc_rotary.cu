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
// those of its tokens once, in shared memory, for all query and key heads.
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

constexpr int ROT_THREADS = 256;
constexpr int ROT_MAX_PAIRS = 4096;   // (cos, sin) of one token in 32 KB
constexpr int ROT_MAX_TOKENS = 64;    // per block

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
    float sign;
    FastDiv per_token, per_head, pairs, by_l;
};

// A unit of work of a head.  Vectorised: V channels starting at V u
// (interleaved), or the V pairs starting at V u (half-split, u < R / V) and
// then the V copied channels each.  Scalar (V = 1): one pair, then the copied
// channels one by one.
template <class T, int V, bool INTER>
__global__ void __launch_bounds__(ROT_THREADS) rotary_kernel(const RotArgs a) {
    extern __shared__ float2 cs[];  // [tokens of the block][R]
    const int R = a.A * a.F;
    const int64_t t0 = int64_t(blockIdx.x) * a.T;
    const int nt = int(min(int64_t(a.T), a.tokens - t0));
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
    __syncthreads();
    const int units = a.per_head.d;  // per head
    const int n = nt * int(a.per_token.d);
    for (int i = threadIdx.x; i < n; i += ROT_THREADS) {
        const int tk = a.per_token.div(i);
        int r = i - tk * int(a.per_token.d);
        int h = a.per_head.div(r);
        const int u = r - h * units;
        const int64_t tok = t0 + tk;
        const RotTensor &t = h < a.q.heads ? a.q : a.k;
        if (h >= a.q.heads) h -= a.q.heads;
        const int64_t b = a.by_l.div(uint32_t(tok));
        const T *x = static_cast<const T *>(t.x) + b * t.sb + (tok - b * a.L) * t.sl +
                     int64_t(h) * t.sh;
        T *y = static_cast<T *>(t.y) + (tok * t.heads + h) * a.D;
        const float2 *w = cs + tk * R;
        if (INTER && V > 1) {
            float v[V];
            Vec<T, V>::load(x + u * V, v);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                const int p = u * (V / 2) + e;
                if (p < R) {
                    const float2 c = w[p];
                    const float p0 = v[2 * e], p1 = v[2 * e + 1];
                    v[2 * e] = fmaf(p0, c.x, -(p1 * c.y));
                    v[2 * e + 1] = fmaf(p1, c.x, p0 * c.y);
                }
            }
            Vec<T, V>::store(y + u * V, v);
        } else {
            const int turned = V > 1 ? R / V : R;
            if (u < turned) {
                const int c0 = INTER ? 2 * u : u * V, c1 = INTER ? 2 * u + 1 : R + u * V;
                float p0[V], p1[V];
                Vec<T, V>::load(x + c0, p0);
                Vec<T, V>::load(x + c1, p1);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 c = w[u * V + e];
                    const float q0 = p0[e], q1 = p1[e];
                    p0[e] = fmaf(q0, c.x, -(q1 * c.y));
                    p1[e] = fmaf(q1, c.x, q0 * c.y);
                }
                Vec<T, V>::store(y + c0, p0);
                Vec<T, V>::store(y + c1, p1);
            } else {
                const int c = 2 * R + (u - turned) * V;
                float v[V];
                Vec<T, V>::load(x + c, v);
                Vec<T, V>::store(y + c, v);
            }
        }
    }
}

bool rot_fits(const RotTensor &t, int D, int v, size_t es) {
    if (t.heads == 0) return true;
    return D % v == 0 && t.sb % v == 0 && t.sl % v == 0 && t.sh % v == 0 &&
           reinterpret_cast<uintptr_t>(t.x) % (v * es) == 0 &&
           reinterpret_cast<uintptr_t>(t.y) % (v * es) == 0;
}

template <class T, int V, bool INTER>
cudaError_t rot_launch(const DeviceInfo &dev, RotArgs a, cudaStream_t st) {
    const int R = a.A * a.F;
    const int units = INTER && V > 1 ? a.D / V
                      : V > 1        ? R / V + (a.D - 2 * R) / V
                                     : R + (a.D - 2 * R);
    const int64_t per = int64_t(units) * (a.q.heads + a.k.heads);
    // tokens of a block: about four units a thread, but first enough blocks
    // for the GPU, and the block's sines within 32 KB
    int64_t T_ = (4 * ROT_THREADS + per - 1) / per;
    const int64_t spread = (a.tokens + dev.sm_count * 4 - 1) / (dev.sm_count * 4);
    if (T_ > spread) T_ = spread;
    if (T_ > ROT_MAX_TOKENS) T_ = ROT_MAX_TOKENS;
    if (R > 0 && T_ > ROT_MAX_PAIRS / R) T_ = ROT_MAX_PAIRS / R;
    if (T_ < 1) T_ = 1;
    a.T = int(T_);
    a.per_head = FastDiv(uint32_t(units));
    a.per_token = FastDiv(uint32_t(per));
    a.pairs = FastDiv(uint32_t(R > 0 ? R : 1));
    a.by_l = FastDiv(uint32_t(a.L));
    const int64_t blocks = (a.tokens + a.T - 1) / a.T;
    rotary_kernel<T, V, INTER>
        <<<unsigned(blocks), ROT_THREADS, size_t(a.T) * R * sizeof(float2), st>>>(a);
    return cudaGetLastError();
}

template <class T>
cudaError_t rot_dispatch(const DeviceInfo &dev, const RotArgs &a, bool inter,
                         cudaStream_t st) {
    constexpr int W = 16 / sizeof(T);
    const bool wide = rot_fits(a.q, a.D, W, sizeof(T)) && rot_fits(a.k, a.D, W, sizeof(T));
    const int R = a.A * a.F;
    if (inter)
        return wide ? rot_launch<T, W, true>(dev, a, st) : rot_launch<T, 1, true>(dev, a, st);
    return wide && R % W == 0 ? rot_launch<T, W, false>(dev, a, st)
                              : rot_launch<T, 1, false>(dev, a, st);
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
    if (D > 65536 || A * F > ROT_MAX_PAIRS || H > 65536 || Hkv > 65536 ||
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
