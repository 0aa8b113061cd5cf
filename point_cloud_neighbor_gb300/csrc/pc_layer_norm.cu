// pc_layer_norm.cu -- layer norm over the last axis, forward and backward.
//
//   mean = sum x / C, var = sum (x - mean)^2 / C, rstd = 1 / sqrt(var + eps)
//   y  = (x - mean) rstd w + b
//   xhat = (x - mean) rstd, g = dy w
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),
//   dw = sum_rows dy xhat,  db = sum_rows dy.
//
// Bound: memory.  A row is read once into registers (by one warp, or by a
// block of 256 threads for C > 1024) and written once; the variance is summed
// from the centred values in registers, so no cancellation of sums of
// squares.  All sums are float32.
//
// The weight gradients need a sum over all rows.  Each backward block walks
// its share of the rows with the columns' sums in registers, joins its warps
// in a fixed order and writes one row of partial sums; a second kernel adds
// the blocks' rows in a fixed order.  No atomics: the result does not change
// from run to run.
#include "pc_internal.h"
#include "pc_vec.cuh"
#include "pointcloud.h"

#include <cstdio>

namespace pcn {
namespace {

constexpr int LN_THREADS = 256;
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
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
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

template <class WT, int V>
__device__ __forceinline__ void load_param(const void *p, int at, float fill, float *v) {
    if (p == nullptr) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = fill;
    } else {
        Vec<WT, V>::load(static_cast<const WT *>(p) + at, v);
    }
}

// A thread holds the vectors t, t + TPR, ... (N of V elements) of its row.
template <class T, class WT, int V, int N, int TPR>
__global__ void __launch_bounds__(LN_THREADS) ln_forward_kernel(const LnArgs a) {
    __shared__ float red[LN_THREADS / 32];
    constexpr int RPB = LN_THREADS / TPR;
    const int64_t row = int64_t(blockIdx.x) * RPB + threadIdx.x / TPR;
    if (row >= a.rows) return;  // a whole warp, or (TPR = 256) never
    const int t = threadIdx.x % TPR;
    const T *x = static_cast<const T *>(a.x) + row * a.C;
    float v[N][V];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = (t + i * TPR) * V;
        if (at < a.C) {
            Vec<T, V>::load(x + at, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) s += v[i][e];
    const float mean = row_sum<TPR>(s, red) / float(a.C);
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if ((t + i * TPR) * V < a.C)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[i][e] -= mean;
                q = fmaf(v[i][e], v[i][e], q);
            }
    const float rstd = 1.0f / sqrtf(row_sum<TPR>(q, red) / float(a.C) + a.eps);
    T *y = static_cast<T *>(a.y) + row * a.C;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = (t + i * TPR) * V;
        if (at < a.C) {
            float w[V], b[V];
            load_param<WT, V>(a.w, at, 1.0f, w);
            load_param<WT, V>(a.b, at, 0.0f, b);
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] = fmaf(v[i][e] * rstd, w[e], b[e]);
            Vec<T, V>::store(y + at, v[i]);
        }
    }
    if (t == 0 && a.mean != nullptr) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
}

template <class T, class WT, int V, int N, int TPR>
__global__ void __launch_bounds__(LN_THREADS) ln_backward_kernel(const LnArgs a) {
    __shared__ float red[LN_THREADS / 32];
    extern __shared__ float col[];  // [2][C], TPR = 32 only
    constexpr int RPB = LN_THREADS / TPR;
    const int t = threadIdx.x % TPR;
    float dw[N][V], db[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) dw[i][e] = db[i][e] = 0.0f;
    const float inv_c = 1.0f / float(a.C);
    for (int64_t row = int64_t(blockIdx.x) * RPB + threadIdx.x / TPR; row < a.rows;
         row += int64_t(gridDim.x) * RPB) {
        const T *x = static_cast<const T *>(a.x) + row * a.C;
        const T *dy = static_cast<const T *>(a.dy) + row * a.C;
        float xv[N][V], gv[N][V];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (t + i * TPR) * V;
            if (at < a.C) {
                Vec<T, V>::load(x + at, xv[i]);
                Vec<T, V>::load(dy + at, gv[i]);
            }
        }
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (t + i * TPR) * V;
            if (at < a.C) {
                float w[V];
                load_param<WT, V>(a.w, at, 1.0f, w);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = (xv[i][e] - mean) * rstd;
                    dw[i][e] = fmaf(gv[i][e], xh, dw[i][e]);
                    db[i][e] += gv[i][e];
                    const float g = gv[i][e] * w[e];
                    s0 += g;
                    s1 = fmaf(g, xh, s1);
                    xv[i][e] = xh;
                    gv[i][e] = g;
                }
            }
        }
        const float c0 = row_sum<TPR>(s0, red) * inv_c;
        const float c1 = row_sum<TPR>(s1, red) * inv_c;
        T *dx = static_cast<T *>(a.y) + row * a.C;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (t + i * TPR) * V;
            if (at < a.C) {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    xv[i][e] = rstd * (gv[i][e] - fmaf(xv[i][e], c1, c0));
                Vec<T, V>::store(dx + at, xv[i]);
            }
        }
    }
    if (a.part == nullptr) return;
    float *part = a.part + size_t(blockIdx.x) * 2 * a.C;
    if (TPR == 32) {
        // join the block's warps, one after the other
        for (int w = 0; w < RPB; ++w) {
            if (int(threadIdx.x / 32) == w)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int at = (t + i * TPR) * V;
                    if (at < a.C)
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            float *c = col + at + e;
                            c[0] = w == 0 ? dw[i][e] : c[0] + dw[i][e];
                            c[a.C] = w == 0 ? db[i][e] : c[a.C] + db[i][e];
                        }
                }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * a.C; c += LN_THREADS) part[c] = col[c];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (t + i * TPR) * V;
            if (at < a.C)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    part[at + e] = dw[i][e];
                    part[a.C + at + e] = db[i][e];
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
    bool backward;
    int blocks;
    cudaStream_t stream;
};

template <class T, class WT, int V, int N, int TPR>
void ln_launch(const LnArgs &a, const LnLaunch &l) {
    if (l.backward)
        ln_backward_kernel<T, WT, V, N, TPR>
            <<<l.blocks, LN_THREADS, TPR == 32 ? size_t(a.C) * 8 : 0, l.stream>>>(a);
    else
        ln_forward_kernel<T, WT, V, N, TPR><<<l.blocks, LN_THREADS, 0, l.stream>>>(a);
}

// Elements a thread holds: 8, 16 or 32, the smallest that covers the row.
template <class T, class WT, int V, int TPR>
void ln_pick_n(const LnArgs &a, const LnLaunch &l) {
    if (a.C <= TPR * 8)
        ln_launch<T, WT, V, 8 / V, TPR>(a, l);
    else if (a.C <= TPR * 16)
        ln_launch<T, WT, V, 16 / V, TPR>(a, l);
    else
        ln_launch<T, WT, V, 32 / V, TPR>(a, l);
}

template <class T, class WT, int V>
void ln_pick_tpr(const LnArgs &a, const LnLaunch &l) {
    if (a.C <= 1024)
        ln_pick_n<T, WT, V, 32>(a, l);
    else
        ln_pick_n<T, WT, V, 256>(a, l);
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Widest vector every row, parameter and gradient is aligned to.
template <class T, class WT>
void ln_pick_v(const LnArgs &a, const LnLaunch &l) {
    constexpr int W = 16 / sizeof(T);
    auto fits = [&](int v) {
        return a.C % v == 0 && aligned(a.x, v * sizeof(T)) && aligned(a.y, v * sizeof(T)) &&
               aligned(a.dy, v * sizeof(T)) && aligned(a.w, min(v * sizeof(WT), size_t(16))) &&
               aligned(a.b, min(v * sizeof(WT), size_t(16)));
    };
    if (fits(W))
        ln_pick_tpr<T, WT, W>(a, l);
    else if (sizeof(T) == 2 && fits(2))
        ln_pick_tpr<T, WT, sizeof(T) == 2 ? 2 : 1>(a, l);
    else
        ln_pick_tpr<T, WT, 1>(a, l);
}

void ln_dispatch(const LnArgs &a, int dtype, int param_dtype, const LnLaunch &l) {
    if (dtype == PC_F32)
        ln_pick_v<float, float>(a, l);
    else if (param_dtype == PC_F32)
        ln_pick_v<bf16, float>(a, l);
    else
        ln_pick_v<bf16, bf16>(a, l);
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
    const int rpb = C <= 1024 ? LN_THREADS / 32 : 1;
    const LnLaunch l{false, int((rows + rpb - 1) / rpb), static_cast<cudaStream_t>(stream)};
    ln_dispatch(a, dtype, param_dtype, l);
    return ln_cuda("layer_norm", cudaGetLastError());
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
    const int rpb = C <= 1024 ? LN_THREADS / 32 : 1;
    const int64_t want = (rows + rpb - 1) / rpb;
    const int most = dev->sm_count * 4;
    const int blocks = int(want < most ? want : most);
    LnArgs a{};
    a.x = x, a.dy = grad_out, a.w = weight, a.y = grad_x;
    a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
    a.rows = rows, a.C = int(C);
    cudaError_t e = cudaSuccess;
    void *part = nullptr;
    if (params && blocks > 0) {
        e = scratch_alloc(*dev, &part, size_t(blocks) * 2 * C * sizeof(float), st);
        if (e != cudaSuccess) return ln_cuda("layer_norm_backward: scratch", e);
        a.part = static_cast<float *>(part);
    }
    if (blocks > 0) ln_dispatch(a, dtype, param_dtype, LnLaunch{true, blocks, st});
    if (params) {
        const unsigned g = unsigned((2 * C + 31) / 32);
        if (param_dtype == PC_F32)
            ln_param_kernel<float><<<g, dim3(32, 32), 0, st>>>(
                a.part, blocks, int(C), static_cast<float *>(grad_weight),
                static_cast<float *>(grad_bias));
        else
            ln_param_kernel<bf16><<<g, dim3(32, 32), 0, st>>>(
                a.part, blocks, int(C), static_cast<bf16 *>(grad_weight),
                static_cast<bf16 *>(grad_bias));
    }
    e = cudaGetLastError();
    if (part != nullptr) {
        const cudaError_t f = scratch_free(part, st);
        if (e == cudaSuccess) e = f;
    }
    return ln_cuda("layer_norm_backward", e);
}
