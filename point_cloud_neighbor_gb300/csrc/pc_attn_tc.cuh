// pc_attn_tc.cuh -- pieces the two tensor-core attention kernels share.
#pragma once

#include "pc_attn.cuh"
#include "pc_tcgen05.cuh"
#include "pc_tiles.cuh"

namespace pcn {
namespace {

constexpr int XR = 128;  // rows of a product
constexpr int YR = ATTN_TC_TILE;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float2 pair(const uint32_t *r, int i) {
    return make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
}
// v = hi + lo to 2^-16 of v, both bfloat16
__device__ __forceinline__ void split_bf16(float2 v, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(v.x, v.y);
    const float2 h = unpack_bf16(hi);
    lo = pack_bf16(v.x - h.x, v.y - h.y);
}

// Squared distances of one point to four columns, in pairs.
__device__ __forceinline__ void dist4(const float *cd, int c, float2 nx, float2 ny, float2 nz,
                                      float2 &d0, float2 &d1) {
    const float4 x = *reinterpret_cast<const float4 *>(cd + c);
    const float4 y = *reinterpret_cast<const float4 *>(cd + YR + c);
    const float4 z = *reinterpret_cast<const float4 *>(cd + 2 * YR + c);
    float2 a = __fadd2_rn(make_float2(x.x, x.y), nx), b = __fadd2_rn(make_float2(x.z, x.w), nx);
    d0 = __fmul2_rn(a, a), d1 = __fmul2_rn(b, b);
    a = __fadd2_rn(make_float2(y.x, y.y), ny), b = __fadd2_rn(make_float2(y.z, y.w), ny);
    d0 = __ffma2_rn(a, a, d0), d1 = __ffma2_rn(b, b, d1);
    a = __fadd2_rn(make_float2(z.x, z.y), nz), b = __fadd2_rn(make_float2(z.z, z.w), nz);
    d0 = __ffma2_rn(a, a, d0), d1 = __ffma2_rn(b, b, d1);
}

// The slopes' sums of a block's 128 rows, a thread each in four warps: with one
// part the rows' values are complete and added up here, one number a block
// (`red`: 4 floats); else the rows' sums go to their part.
__device__ __forceinline__ void put_slope_sums(const AttnArgs &a, const float (&t)[4], int split,
                                               int64_t hrow, bool in, int quad, int lane,
                                               float *red, unsigned bid) {
    if (a.nsplit > 1) {
        const int64_t n = int64_t(a.B) * a.H * a.Lq;
        if (in) {
            float *o = a.rowsum + int64_t(split) * 4 * n + hrow;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e * n] = t[e];
        }
        return;
    }
    float v = attn_slope_row(t[0], t[1], t[2], t[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) red[quad] = v;
    named_barrier_sync(2, 128);
    if (quad == 0 && lane == 0) a.rowsum[bid] = (red[0] + red[1]) + (red[2] + red[3]);
}

// The head and first row of a block's tiles, one after the other: `heads`
// query heads of `end` rows each (DKV), else one head.
struct TileWalk {
    int h, y, end;
    bool wrap;
    __device__ __forceinline__ TileWalk(bool wrap_, int h0, int tiles, int64_t first, int skip)
        : h(h0), y(0), end(tiles * YR), wrap(wrap_) {
        if (tiles > 0) {
            if (wrap) h += int(first / tiles);
            y = int(wrap ? first % tiles : first) * YR;
            next(skip);
        }
    }
    __device__ __forceinline__ void next(int tiles = 1) {
        y += tiles * YR;
        if (wrap)
            while (y >= end) y -= end, ++h;
    }
};

// [B, L, heads, D] as boxes of 64 rows by 64 channels.
bool make_map(CUtensorMap *map, const void *p, const int64_t *s, int64_t B, int64_t L,
              int64_t heads, int64_t D) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(L), cuuint64_t(heads), cuuint64_t(B)};
    // the stride of an axis of one element is never used: any valid one
    const cuuint64_t strides[3] = {cuuint64_t(L > 1 ? s[1] : D) * 2,
                                   cuuint64_t(heads > 1 ? s[2] : D) * 2,
                                   cuuint64_t(B > 1 ? s[0] : D) * 2};
    const cuuint32_t box[4] = {64, YR, 1, 1}, ones[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box,
              ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace pcn
