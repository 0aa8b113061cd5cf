// pc_gated.cu -- gated projection act(x Wg^T + bg) * (x Wu^T + bu), forward and
// backward.
#include "pc_act.cuh"
#include "pc_internal.h"
#include "pc_vec.cuh"
#include "pointcloud.h"

#include <cstdio>

namespace pcn {
namespace {

constexpr int TM = 64, TK = 16;

struct GatedArgs {
    const void *x, *wg, *wu, *bg, *bu, *dy;
    void *y, *dx, *dwg, *dwu, *dbg, *dbu;
    float *da, *du;  // [rows, F]
    int64_t rows;
    int C, F, act;
};

template <class T>
__device__ __forceinline__ float at(const void *p, int64_t i) {
    float v;
    Vec<T, 1>::load(static_cast<const T *>(p) + i, &v);
    return v;
}

// acc[i][j] += sum over k < K of A(m0 + 4 ty + i, k) B(n0 + 4 tx + j, k), in chains
// of 256 so that the error of a long sum stays that of a short one
template <class FA, class FB>
__device__ __forceinline__ void product(float (&acc)[4][4], int64_t M, int N, int64_t K,
                                        int64_t m0, int n0, FA A, FB B, float *sa, float *sb) {
    const int t = threadIdx.x, tx = t % 16, ty = t / 16;
    float sum[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += TK) {
        for (int i = t; i < TM * TK; i += 256) {
            const int m = i / TK, k = i % TK;
            sa[k * TM + m] = m0 + m < M && k0 + k < K ? A(m0 + m, k0 + k) : 0.0f;
            sb[k * TM + m] = n0 + m < N && k0 + k < K ? B(n0 + m, k0 + k) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < TK; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j)
                    sum[i][j] = fmaf(sa[k * TM + 4 * ty + i], sb[k * TM + 4 * tx + j], sum[i][j]);
        __syncthreads();
        if (k0 % 256 == 256 - TK || k0 + TK >= K)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] += sum[i][j], sum[i][j] = 0.0f;
    }
}

// y, or with dy the gradients of a and u.
template <class T, bool BWD>
__global__ void __launch_bounds__(256) gated_kernel(GatedArgs a) {
    __shared__ float sa[TM * TK], sb[TM * TK];
    const int64_t m0 = int64_t(blockIdx.x) * TM;
    const int n0 = blockIdx.y * TM;
    float g[4][4] = {}, u[4][4] = {};
    auto X = [&](int64_t m, int64_t k) { return at<T>(a.x, m * a.C + k); };
    product(g, a.rows, a.F, a.C, m0, n0, X,
            [&](int64_t n, int64_t k) { return at<T>(a.wg, n * a.C + k); }, sa, sb);
    product(u, a.rows, a.F, a.C, m0, n0, X,
            [&](int64_t n, int64_t k) { return at<T>(a.wu, n * a.C + k); }, sa, sb);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + threadIdx.x / 16 * 4 + i;
            const int n = n0 + threadIdx.x % 16 * 4 + j;
            if (m >= a.rows || n >= a.F) continue;
            const float zg = g[i][j] + (a.bg ? at<T>(a.bg, n) : 0.0f);
            const float zu = u[i][j] + (a.bu ? at<T>(a.bu, n) : 0.0f);
            if (!BWD) {
                const float v = act_value<sizeof(T) == 2>(a.act, zg) * zu;
                Vec<T, 1>::store(static_cast<T *>(a.y) + m * a.F + n, &v);
            } else {
                float slope;
                const float f = act_both<sizeof(T) == 2>(a.act, zg, slope);
                const float dy = at<T>(a.dy, m * a.F + n);
                a.da[m * a.F + n] = dy * zu * slope;
                a.du[m * a.F + n] = dy * f;
            }
        }
}

template <class T>
__global__ void __launch_bounds__(256) gated_dx_kernel(GatedArgs a) {
    __shared__ float sa[TM * TK], sb[TM * TK];
    const int64_t m0 = int64_t(blockIdx.x) * TM;
    const int n0 = blockIdx.y * TM;
    float d[4][4] = {};
    product(d, a.rows, a.C, a.F, m0, n0, [&](int64_t m, int64_t k) { return a.da[m * a.F + k]; },
            [&](int64_t n, int64_t k) { return at<T>(a.wg, k * a.C + n); }, sa, sb);
    product(d, a.rows, a.C, a.F, m0, n0, [&](int64_t m, int64_t k) { return a.du[m * a.F + k]; },
            [&](int64_t n, int64_t k) { return at<T>(a.wu, k * a.C + n); }, sa, sb);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + threadIdx.x / 16 * 4 + i;
            const int n = n0 + threadIdx.x % 16 * 4 + j;
            if (m < a.rows && n < a.C)
                Vec<T, 1>::store(static_cast<T *>(a.dx) + m * a.C + n, &d[i][j]);
        }
}

template <class T>
__global__ void __launch_bounds__(256) gated_dw_kernel(GatedArgs a) {
    __shared__ float sa[TM * TK], sb[TM * TK];
    const int64_t m0 = int64_t(blockIdx.x) * TM;
    const int n0 = blockIdx.y * TM;
    const float *g = blockIdx.z ? a.du : a.da;
    float d[4][4] = {};
    product(d, a.F, a.C, a.rows, m0, n0, [&](int64_t m, int64_t k) { return g[k * a.F + m]; },
            [&](int64_t n, int64_t k) { return at<T>(a.x, k * a.C + n); }, sa, sb);
    T *out = static_cast<T *>(blockIdx.z ? a.dwu : a.dwg);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + threadIdx.x / 16 * 4 + i;
            const int n = n0 + threadIdx.x % 16 * 4 + j;
            if (m < a.F && n < a.C) Vec<T, 1>::store(out + m * a.C + n, &d[i][j]);
        }
}

template <class T>
__global__ void __launch_bounds__(256) gated_db_kernel(GatedArgs a) {
    __shared__ float acc[256];
    const int n = blockIdx.x;
    const float *g = blockIdx.y ? a.du : a.da;
    float s = 0.0f;
    for (int64_t m = threadIdx.x; m < a.rows; m += 256) s += g[m * a.F + n];
    acc[threadIdx.x] = s;
    __syncthreads();
    for (int h = 128; h > 0; h /= 2) {
        if (threadIdx.x < h) acc[threadIdx.x] += acc[threadIdx.x + h];
        __syncthreads();
    }
    if (threadIdx.x == 0) Vec<T, 1>::store(static_cast<T *>(blockIdx.y ? a.dbu : a.dbg) + n, acc);
}

unsigned tiles(int64_t n) { return unsigned((n + TM - 1) / TM); }

template <class T>
cudaError_t gated_forward(const GatedArgs &a, cudaStream_t st) {
    gated_kernel<T, false><<<dim3(tiles(a.rows), tiles(a.F)), 256, 0, st>>>(a);
    return cudaGetLastError();
}

template <class T>
cudaError_t gated_backward(const DeviceInfo &dev, GatedArgs a, cudaStream_t st) {
    void *p = nullptr;
    cudaError_t e = scratch_alloc(dev, &p, size_t(a.rows) * a.F * 8, st);
    if (e != cudaSuccess) return e;
    a.da = static_cast<float *>(p), a.du = a.da + a.rows * a.F;
    gated_kernel<T, true><<<dim3(tiles(a.rows), tiles(a.F)), 256, 0, st>>>(a);
    if (a.dx) gated_dx_kernel<T><<<dim3(tiles(a.rows), tiles(a.C)), 256, 0, st>>>(a);
    if (a.dwg) gated_dw_kernel<T><<<dim3(tiles(a.F), tiles(a.C), 2), 256, 0, st>>>(a);
    if (a.dbg) gated_db_kernel<T><<<dim3(a.F, 2), 256, 0, st>>>(a);
    e = cudaGetLastError();
    const cudaError_t f = scratch_free(p, st);
    return e == cudaSuccess ? f : e;
}

int gated_fail(const char *what, const char *why, int code) {
    char m[200];
    std::snprintf(m, sizeof(m), "%s: %s", what, why);
    return api_fail(code, m);
}

int gated_check(const char *what, int dtype, int64_t rows, int64_t C, int64_t F, const void *bg,
                const void *bu, int activation) {
    if (rows < 0 || C < 0 || F < 0)
        return gated_fail(what, "negative size", PC_ERR_INVALID_ARGUMENT);
    if (dtype != PC_F32 && dtype != PC_BF16)
        return gated_fail(what, "dtype must be PC_F32 or PC_BF16", PC_ERR_INVALID_ARGUMENT);
    if ((bg == nullptr) != (bu == nullptr))
        return gated_fail(what, "b_gate and b_up go together", PC_ERR_INVALID_ARGUMENT);
    if (activation < PC_ACT_NONE || activation > PC_ACT_SIGMOID)
        return gated_fail(what, "unknown activation", PC_ERR_INVALID_ARGUMENT);
    if (C < 1 && F > 0 && rows > 0)
        return gated_fail(what, "C must be at least 1", PC_ERR_INVALID_ARGUMENT);
    if (rows > 2147483647 - 65536 || C > 65536 || F > 65536)
        return gated_fail(what, "rows beyond 32 bits, or C or F above 65536",
                          PC_ERR_UNSUPPORTED);
    return PC_OK;
}

int gated_cuda(const char *what, cudaError_t e) {
    if (e == cudaSuccess) return PC_OK;
    return gated_fail(what, cudaGetErrorString(e), PC_ERR_CUDA);
}

}  // namespace
}  // namespace pcn

extern "C" int pc_gated_linear(const void *x, int dtype, int64_t rows, int64_t C, int64_t F,
                               const void *w_gate, const void *w_up, const void *b_gate,
                               const void *b_up, int activation, void *out, void *stream) {
    using namespace pcn;
    int rc = gated_check("gated_linear", dtype, rows, C, F, b_gate, b_up, activation);
    if (rc != PC_OK) return rc;
    if (rows == 0 || F == 0) return PC_OK;
    const DeviceInfo *dev = nullptr;
    if ((rc = api_current_device(&dev)) != PC_OK) return rc;
    const int d = dev->device;
    const size_t es = dtype == PC_F32 ? 4 : 2;
    if ((rc = api_check_ptr(x, d, es, "x")) != PC_OK) return rc;
    if ((rc = api_check_ptr(w_gate, d, es, "w_gate")) != PC_OK) return rc;
    if ((rc = api_check_ptr(w_up, d, es, "w_up")) != PC_OK) return rc;
    if (b_gate && (rc = api_check_ptr(b_gate, d, es, "b_gate")) != PC_OK) return rc;
    if (b_up && (rc = api_check_ptr(b_up, d, es, "b_up")) != PC_OK) return rc;
    if ((rc = api_check_ptr(out, d, es, "out")) != PC_OK) return rc;
    GatedArgs a{};
    a.x = x, a.wg = w_gate, a.wu = w_up, a.bg = b_gate, a.bu = b_up, a.y = out;
    a.rows = rows, a.C = int(C), a.F = int(F), a.act = activation;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return gated_cuda("gated_linear",
                      dtype == PC_F32 ? gated_forward<float>(a, st) : gated_forward<bf16>(a, st));
}

extern "C" int pc_gated_linear_backward(const void *grad_out, const void *x, int dtype,
                                        int64_t rows, int64_t C, int64_t F, const void *w_gate,
                                        const void *w_up, const void *b_gate, const void *b_up,
                                        int activation, void *grad_x, void *grad_w_gate,
                                        void *grad_w_up, void *grad_b_gate, void *grad_b_up,
                                        void *stream) {
    using namespace pcn;
    const char *what = "gated_linear_backward";
    int rc = gated_check(what, dtype, rows, C, F, b_gate, b_up, activation);
    if (rc != PC_OK) return rc;
    if ((grad_w_gate == nullptr) != (grad_w_up == nullptr) ||
        (grad_b_gate == nullptr) != (grad_b_up == nullptr))
        return gated_fail(what, "the weights' gradients go together, and the biases'",
                          PC_ERR_INVALID_ARGUMENT);
    if (!grad_x && !grad_w_gate && !grad_b_gate) return PC_OK;
    const DeviceInfo *dev = nullptr;
    if ((rc = api_current_device(&dev)) != PC_OK) return rc;
    const int d = dev->device;
    const size_t es = dtype == PC_F32 ? 4 : 2;
    const bool empty = rows == 0 || F == 0;
    if (!empty) {
        if ((rc = api_check_ptr(grad_out, d, es, "grad_out")) != PC_OK) return rc;
        if ((rc = api_check_ptr(x, d, es, "x")) != PC_OK) return rc;
        if ((rc = api_check_ptr(w_gate, d, es, "w_gate")) != PC_OK) return rc;
        if ((rc = api_check_ptr(w_up, d, es, "w_up")) != PC_OK) return rc;
        if (b_gate && (rc = api_check_ptr(b_gate, d, es, "b_gate")) != PC_OK) return rc;
        if (b_up && (rc = api_check_ptr(b_up, d, es, "b_up")) != PC_OK) return rc;
    }
    void *outs[5] = {rows * C > 0 ? grad_x : nullptr, F * C > 0 ? grad_w_gate : nullptr,
                     F * C > 0 ? grad_w_up : nullptr, F > 0 ? grad_b_gate : nullptr,
                     F > 0 ? grad_b_up : nullptr};
    const char *names[5] = {"grad_x", "grad_w_gate", "grad_w_up", "grad_b_gate", "grad_b_up"};
    for (int i = 0; i < 5; ++i)
        if (outs[i] && (rc = api_check_ptr(outs[i], d, es, names[i])) != PC_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (empty) {
        const int64_t n[5] = {rows * C, F * C, F * C, F, F};
        for (int i = 0; i < 5; ++i)
            if (outs[i]) {
                const cudaError_t e = cudaMemsetAsync(outs[i], 0, size_t(n[i]) * es, st);
                if (e != cudaSuccess) return gated_cuda(what, e);
            }
        return PC_OK;
    }
    GatedArgs a{};
    a.x = x, a.wg = w_gate, a.wu = w_up, a.bg = b_gate, a.bu = b_up, a.dy = grad_out;
    a.dx = outs[0], a.dwg = outs[1], a.dwu = outs[2], a.dbg = outs[3], a.dbu = outs[4];
    a.rows = rows, a.C = int(C), a.F = int(F), a.act = activation;
    return gated_cuda(what, dtype == PC_F32 ? gated_backward<float>(*dev, a, st)
                                            : gated_backward<bf16>(*dev, a, st));
}
