// pc_gated.cu -- gated projection act(x Wg^T + bg) * (x Wu^T + bu), forward and
// backward.
#include "pc_gated.cuh"
#include "pointcloud.h"

#include <cstdio>

namespace pcn {
namespace {

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
    // (chains of C products, tile numbers and grids of 32 bits)
    if (rows > (int64_t(1) << 30) || C > 16384 || F > 65536)
        return gated_fail(what, "rows beyond 2^30, C above 16384 or F above 65536",
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
                               const void *b_up, int activation, void *out, void *workspace,
                               size_t workspace_bytes, void *stream) {
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
    a.workspace = workspace, a.workspace_bytes = workspace_bytes;
    if (workspace && (rc = api_check_ptr(workspace, d, 256, "workspace")) != PC_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return gated_cuda("gated_linear", gated_tc_forward(*dev, a, dtype, st));
}

extern "C" int pc_gated_linear_backward(const void *grad_out, const void *x, int dtype,
                                        int64_t rows, int64_t C, int64_t F, const void *w_gate,
                                        const void *w_up, const void *b_gate, const void *b_up,
                                        int activation, void *grad_x, void *grad_w_gate,
                                        void *grad_w_up, void *grad_b_gate, void *grad_b_up,
                                        void *workspace, size_t workspace_bytes, void *stream) {
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
    a.workspace = workspace, a.workspace_bytes = workspace_bytes;
    if (workspace && (rc = api_check_ptr(workspace, d, 256, "workspace")) != PC_OK) return rc;
    return gated_cuda(what, gated_tc_backward(*dev, a, dtype, st));
}

extern "C" size_t pc_gated_linear_workspace_bytes(int dtype, int64_t rows, int64_t C, int64_t F,
                                                  int gradients) {
    using namespace pcn;
    const DeviceInfo *dev = nullptr;
    if (gated_check("gated_linear_workspace_bytes", dtype, rows, C, F, nullptr, nullptr,
                    PC_ACT_NONE) != PC_OK ||
        rows == 0 || F == 0 || api_current_device(&dev) != PC_OK)
        return 0;
    GatedArgs a{};
    a.rows = rows, a.C = int(C), a.F = int(F);
    if (gradients & PC_GATED_UNALIGNED)  // (no multiple of 16, and not looked at)
        a.x = a.wg = a.wu = reinterpret_cast<const char *>(uintptr_t(2));
    void *some = &a;  // (only which gradients there are counts)
    if (gradients & PC_GATED_GRAD_X) a.dx = some;
    if (gradients & PC_GATED_GRAD_WEIGHT) a.dwg = a.dwu = some;
    if (gradients & PC_GATED_GRAD_BIAS) a.dbg = a.dbu = some;
    return gated_tc_scratch(
        *dev, a, dtype,
        (gradients & (PC_GATED_GRAD_X | PC_GATED_GRAD_WEIGHT | PC_GATED_GRAD_BIAS)) != 0);
}
