// pc_attn.cuh -- what the attention kernels share: their arguments, the
// three passes and the launchers.
//
//   z_ij = scale q_i.k_j - slope_h |x_i - y_j|^2,  j < ref_length,
//   P = softmax_j(z), out = P v, lse_i = log sum_j exp(z_ij);
//   delta_i = out_i . dout_i = sum_j P_ij dP_ij, dP = dout v^T, dS = P (dP - delta),
//   dq = scale dS k, dk = scale dS^T q, dv = P^T dout,
//   dslope_h = -sum_ij dS_ij |x_i - y_j|^2.
// A cloud with one key has P = 1 and dS = 0 exactly: delta and dP, which are summed
// in different orders, would leave their rounding.  Sums of its dS are taken as 0.
//
// Every pass keeps a tile of rows (its `stationary` side) and walks over the
// other side in tiles (`streamed`):
//   FWD  rows q        streams k, v      acc = P v
//   DQ   rows q, dout  streams k, v      acc = dS k
//   DKV  rows k, v     streams q, dout   acc = P^T dout and dS^T q, over all
//                                        query heads that share the key head.
// The backward pass forms the scores twice instead of adding into dq with
// atomics, so the order of every sum is fixed.
//
// delta takes the output before its rounding.  Where P has few large weights
// dP is near delta and dS = P (dP - delta) small: half a unit of a bfloat16 output
// is then as large as dS itself (dq off by 0.0034 of its norm at 16 keys with slopes
// of 8, by 0.6 at 2, where a result rounded once has 0.0017).  So a forward pass
// can write what the rounding left as a second bfloat16 array, `low`, for 2 bytes
// an element, and delta adds it.  A backward call without it runs the forward pass
// again for both arrays (4096 tokens, 16 + 4 heads of 128: 752 us instead of 585).
#pragma once

#include "pc_internal.h"
#include "pc_vec.cuh"

#include <stdint.h>

namespace pcn {

enum AttnMode { ATTN_FWD = 0, ATTN_DQ = 1, ATTN_DKV = 2 };

constexpr float ATTN_LOG2E = 1.4426950408889634f;
constexpr float ATTN_LN2 = 0.6931471805599453f;

struct AttnArgs {
    const void *q, *k, *v, *go;             // go: dout, packed [B, Lq, H, D]
    int64_t qs[3], ks[3], vs[3];            // strides (batch, length, head), elements
    const float *qxyz, *rxyz, *slopes;      // all three or none
    const int64_t *qlen, *rlen;             // or NULL
    int B, Lq, Lk, H, Hkv, D;
    float scale;
    void *out;                              // FWD
    void *low;                              // FWD: what rounding out to bfloat16 left, or NULL
    float *lse;                             // FWD: written if not NULL
    const float *delta, *lse2;              // backward: [B, H, Lq], see attn_delta_kernel
    void *dq, *dk, *dv;  // dq, or dk and dv, may be NULL: not asked for
    // the streamed side in nsplit parts: their accumulators, joined afterwards
    int nsplit;
    float *part;     // [nsplit][rows of the output][D] (DKV: dk, then dv)
    float *part_ml;  // FWD: [nsplit][2][B H Lq] (maximum in base-2 units, sum)
    // DQ with slopes: per row sums of dS d2, P d2, dS and P, [nsplit][4][B H Lq], each
    // a LongSum of a few columns' sums; or
    // (tensor cores, one part) one number a block, [B H][tiles]
    float *rowsum;
    int device;
    int *status;
    uint64_t timeout_ns;
};

__device__ __forceinline__ int attn_len(const int64_t *len, int b, int L) {
    if (len == nullptr) return L;
    const int64_t n = len[b];
    return n < 0 ? 0 : n > L ? L : int(n);
}

// A float32 sum of any length: what an addition rounds away is taken from the next
// number (Kahan's sum: off by 2 units of the sum of magnitudes, whatever the
// length).  For the slopes' gradient, whose terms are as many as pairs: plain chains
// over 65,536 equal terms were off by 1.6e-4 of their sum.
struct LongSum {
    float s = 0.0f, over = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float y = v - over, t = s + y;
        over = (t - s) - y;
        s = t;
    }
    __device__ __forceinline__ float value() const { return s; }
};

// What a row adds to -dslope: its sums of dS d2, P d2, dS and P, the P made to add up
// to 1.
__device__ __forceinline__ float attn_slope_row(float a, float e, float d, float p) {
    return p == 0.0f ? 0.0f : fmaf(-d, e / p, a) / p;
}

// Whether a query row has anything to attend to, which the lengths alone decide:
// its sum of weights may be NaN (a NaN in a valid row or key, a score that
// overflowed), and that is what the row then shows.
__device__ __forceinline__ bool attn_row_has_keys(const AttnArgs &a, int b, int i) {
    return i < attn_len(a.qlen, b, a.Lq) && attn_len(a.rlen, b, a.Lk) > 0;
}

// The factor of sums of dS: see above.
__device__ __forceinline__ float attn_ds_factor(int nk) { return nk > 1 ? 1.0f : 0.0f; }

// Rows a block keeps in the tensor-core kernels, and rows of a streamed tile.
constexpr int attn_tc_rows(int mode) { return mode == ATTN_FWD ? 256 : 128; }
constexpr int ATTN_TC_TILE = 64;
// Tiles whose sums run in one chain of the bfloat16 kernels' accumulators.  The tensor
// cores cut off what an addition leaves below the accumulator's last place: sums of
// one sign lose 4.4e-7 of themselves a tile (measured: 1.8e-3 over 4096 tiles, as
// much as a bfloat16's rounding, and always towards 0).  Parts of 256 tiles (16,384
// rows), joined in float32, keep that below 1.2e-4.
constexpr int ATTN_TC_CHAIN = 256;

// Whether the tensor-core kernels (pc_attn_tc.cu; bfloat16) take these sizes,
// strides and alignments: channels a multiple of 8 and 16-byte aligned rows.
bool attn_tc_fits(const AttnArgs &a, int mode);
cudaError_t launch_attn_tc_forward(const AttnArgs &a, unsigned blocks, cudaStream_t st);
// Both backward passes: `first` blocks of DKV and `second` of DQ in one launch.
cudaError_t launch_attn_tc_backward(const AttnArgs &dkv, unsigned first, const AttnArgs &dq,
                                    unsigned second, cudaStream_t st);

// Few queries per key head (pc_attn_few.cu); backward, one launch writes dk and
// dv and the parts of dq.  nsplit comes from attn_few_parts.
bool attn_few_fits(const AttnArgs &a, size_t elem, bool backward);
int attn_few_parts(const DeviceInfo &dev, const AttnArgs &a, size_t elem, bool backward);
cudaError_t launch_attn_few(const AttnArgs &a, size_t elem, bool backward, cudaStream_t st);

// float32 on the tensor cores (pc_attn_tc32.cu): the arrays as three
// bfloat16 parts [3][B, L, heads, Dp] each, written into `space` once a call.
struct AttnSplit {
    const bf16 *q, *k, *v, *go;
    int Dp;
};
bool attn_tc32_fits(const AttnArgs &a);
int attn_tc32_rows(const AttnArgs &a, int mode);  // rows a block keeps
size_t attn_split_bytes(const AttnArgs &a, bool backward);
cudaError_t launch_attn_split(const AttnArgs &a, bool backward, void *space, AttnSplit *s,
                              cudaStream_t st);
cudaError_t launch_attn_tc32_forward(const AttnArgs &a, const AttnSplit &s, unsigned blocks,
                                     cudaStream_t st);
cudaError_t launch_attn_tc32_backward(const AttnArgs &dkv, unsigned first, const AttnArgs &dq,
                                      unsigned second, const AttnSplit &s, cudaStream_t st);

}  // namespace pcn
