// pc_gated.cuh -- arguments of the gated projection and its kernels' launches.
#pragma once

#include "pc_internal.h"
#include "pc_vec.cuh"

namespace pcn {

struct GatedArgs {
    const void *x, *wg, *wu, *bg, *bu, *dy;
    void *y, *dx, *dwg, *dwu, *dbg, *dbu;
    int64_t rows;
    int C, F, act;
    void *workspace;
    size_t workspace_bytes;
};

// On the tensor cores (pc_gated_tc.cu), any sizes and alignment; the scratch these take.
size_t gated_tc_scratch(const DeviceInfo &dev, const GatedArgs &a, int dtype, bool backward);
cudaError_t gated_tc_forward(const DeviceInfo &dev, const GatedArgs &a, int dtype,
                             cudaStream_t st);
cudaError_t gated_tc_backward(const DeviceInfo &dev, const GatedArgs &a, int dtype,
                              cudaStream_t st);

}  // namespace pcn
