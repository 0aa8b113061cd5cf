// pc_attn_tc.cu -- the attention passes of pc_attn.cuh on the tensor cores,
// for bfloat16.
//
// A block keeps 128 rows and walks over the other side in tiles of 64:
//   scores   S = X1 Y1^T (and dP = X2 Y2^T), both operands in shared memory,
//            the result in tensor memory, one lane per row;
//   weights  a thread owns a row: it reads its scores, adds the bias, and
//            writes P (and dS) back as bfloat16 over the scores;
//   sums     acc += P Y2 (and dS Y1), the weights read from tensor memory,
//            the same shared-memory tile now contracted along its rows.
// One warp copies tiles (tensor maps, 128-byte swizzle; zeros past the
// arrays' ends) and the columns' positions, one warp issues the products,
// the others compute weights.  The score buffers alternate, so the products
// of one tile run under the weights of another.
//
// Both operands of a product have one type, and bfloat16 alone would cost P
// and dS 2^-9 on average: each is written as the sum of two bfloat16 (2^-17)
// and multiplied twice.  The sums of P, the statistics and all accumulators
// are float32, and the slopes' gradient uses the unrounded weights.
//
// What lies past a cloud's length is masked in the weights; rows of a
// streamed tile past the length (they would meet weights that are 0, and 0
// times NaN is NaN) are overwritten with zeros in shared memory.
//
// Every wait is bounded: when one runs out the block raises the status word,
// lets its copies and products finish, frees its tensor memory and returns;
// its outputs are then unspecified.
#include "pc_attn.cuh"
#include "pc_tcgen05.cuh"
#include "pc_tiles.cuh"
#include "pointcloud.h"

namespace pcn {
namespace {

constexpr int XR = ATTN_TC_ROWS, YR = ATTN_TC_TILE;

struct AttnMaps {
    CUtensorMap q, k, v, go;
};

template <int MODE, int DP>
struct Cfg {
    static constexpr bool BWD = MODE != ATTN_FWD;
    // Warps of the weights: W sets that take tiles in turn, CH groups of four
    // in a set that share a tile's columns.  NB score buffers.
    static constexpr int W = BWD ? 2 : 1, CH = 2;
    static constexpr int NB = 2;
    // The weights as a sum of two bfloat16 (see the top of the file).
    static constexpr bool TWO_P = MODE != ATTN_DQ, TWO_S = BWD;
    static constexpr int STAGES = BWD ? (DP == 64 ? 6 : 3) : (DP == 64 ? 4 : 2);
    static constexpr int BLOCKS = BWD ? 1 : 2;  // per SM
    static constexpr int CWARPS = 4 * W * CH;
    static constexpr int THREADS = 32 * (CWARPS + 2);
    // tensor memory columns: score buffers first, then the accumulators
    static constexpr int BUF = BWD ? 2 * YR : YR;
    static constexpr int ACC = NB * BUF;
    static constexpr int NACC = MODE == ATTN_DKV ? 2 : 1;
    static constexpr int COLS = ACC + NACC * DP <= 256 ? 256 : 512;
    static constexpr int XBYTES = XR * DP * 2, YBYTES = YR * DP * 2;
    static constexpr int XS = BWD ? 2 : 1;
    static constexpr int COLDATA = 5 * YR * 4;  // x, y, z, lse, delta of the streamed rows
    static constexpr size_t TILES = size_t(XS) * XBYTES + size_t(STAGES) * 2 * YBYTES;
    // per row and group: the slope's sums (DQ), or two maxima and a sum (FWD)
    static constexpr int ROWDATA = W * CH * 3 * XR * 4;
    static constexpr size_t SMEM = 1024 + TILES + size_t(STAGES) * COLDATA + ROWDATA + 256;
};

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

// 32 consecutive channels of a row: bfloat16, or float32 for a part.
__device__ __forceinline__ void store_row32(bf16 *p, const float (&v)[32], int c0, int D) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (c0 + 8 * i < D) Vec<bf16, 8>::store(p + 8 * i, v + 8 * i);
}
__device__ __forceinline__ void store_row32(float *p, const float (&v)[32], int c0, int D) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c0 + 4 * i < D) Vec<float, 4>::store(p + 4 * i, v + 4 * i);
}

template <int MODE, int DP, bool BIAS>
__global__ void __launch_bounds__(Cfg<MODE, DP>::THREADS, Cfg<MODE, DP>::BLOCKS)
attn_tc_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnMaps maps,
               const bool withhold) {
    using C = Cfg<MODE, DP>;
    constexpr bool BWD = C::BWD;
    constexpr int STAGES = C::STAGES, NB = C::NB, W = C::W, CH = C::CH;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char *X1 = base, *X2 = X1 + (BWD ? C::XBYTES : 0);
    unsigned char *Y = X1 + C::XS * C::XBYTES;  // stage s: Y1, Y2
    float *coldata = reinterpret_cast<float *>(Y + size_t(STAGES) * 2 * C::YBYTES);
    float *rsum = coldata + STAGES * (C::COLDATA / 4);  // [W CH][3][XR]
    uint64_t *full = reinterpret_cast<uint64_t *>(rsum + C::ROWDATA / 4);
    uint64_t *empty = full + STAGES, *sfull = empty + STAGES, *pfull = sfull + NB;
    uint64_t *xfull = pfull + NB, *accfull = xfull + 1, *pvdone = accfull + 1;
    uint64_t *mxbar = pvdone + 1;  // [4]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mxbar + 4);
    volatile int *stop = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int LX = MODE == ATTN_DKV ? a.Lk : a.Lq, LY = MODE == ATTN_DKV ? a.Lq : a.Lk;
    const int NH = MODE == ATTN_DKV ? a.Hkv : a.H;
    const int G = a.H / a.Hkv;
    const int ntile = (LX + XR - 1) / XR;
    int64_t idx = blockIdx.x;
    const int split = int(idx % a.nsplit);
    idx /= a.nsplit;
    const int tile = int(idx % ntile);
    idx /= ntile;
    const int head = int(idx % NH), b = int(idx / NH);
    const int nq = attn_len(a.qlen, b, a.Lq), nk = attn_len(a.rlen, b, a.Lk);
    const int nx = MODE == ATTN_DKV ? nk : nq, ny = MODE == ATTN_DKV ? nq : nk;
    const int r0 = tile * XR;
    const int hk = MODE == ATTN_DKV ? head : head / G;
    const int nyt = (ny + YR - 1) / YR;
    const int64_t items = nx > r0 ? int64_t(nyt) * (MODE == ATTN_DKV ? G : 1) : 0;
    const int64_t it0 = items * split / a.nsplit;
    const int n = int(items * (split + 1) / a.nsplit - it0);  // tiles of this block

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1 + 4 * CH);
        }
        for (int s = 0; s < NB; ++s) {
            mbar_init(&sfull[s], 1);
            mbar_init(&pfull[s], 4 * CH);
        }
        mbar_init(xfull, 1);
        mbar_init(accfull, 1);
        mbar_init(pvdone, 1);
        for (int s = 0; s < 4; ++s) mbar_init(&mxbar[s], CH);
        *stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == C::CWARPS + 1) tmem_alloc(tmem_slot, C::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // A bounded wait of a whole warp; false: stop.
    auto wait = [&](uint64_t *bar, unsigned parity) {
        const WaitResult w = mbar_wait_or_stop(bar, parity, stop, a.timeout_ns);
        if (w == WAIT_TIMEOUT) {
            *stop = 1;
            raise_status(a.status, PC_ERR_DEVICE_TIMEOUT);
        }
        return __all_sync(0xffffffffu, w == WAIT_OK) != 0;
    };
    auto item_head = [&](int k) {
        return MODE == ATTN_DKV ? hk * G + int((it0 + k) / nyt) : head;
    };
    auto item_row = [&](int k) {
        return int(MODE == ATTN_DKV ? (it0 + k) % nyt : it0 + k) * YR;
    };

    if (warp == C::CWARPS) {
        // ---- copies ---------------------------------------------------------------
        if (n > 0 && lane == 0) {
            mbar_arrive_expect_tx(xfull, C::XS * C::XBYTES);
            const CUtensorMap *m1 = MODE == ATTN_DKV ? &maps.k : &maps.q;
            const CUtensorMap *m2 = MODE == ATTN_DKV ? &maps.v : &maps.go;
            for (int p = 0; p < DP / 64; ++p)
                for (int h = 0; h < 2; ++h) {
                    const int at = p * XR * 128 + h * YR * 128;
                    tma_load_4d(X1 + at, m1, 64 * p, r0 + YR * h, head, b, xfull);
                    if (BWD) tma_load_4d(X2 + at, m2, 64 * p, r0 + YR * h, head, b, xfull);
                }
        }
        int issued = 0;
        for (int k = 0; k < n; ++k) {
            const int s = k % STAGES;
            if (k >= STAGES && !wait(&empty[s], unsigned((k / STAGES - 1) & 1))) break;
            if (withhold && blockIdx.x == 0) break;
            const int h = item_head(k), y0 = item_row(k);
            if (BIAS || MODE == ATTN_DKV) {
                float *cd = coldata + s * (C::COLDATA / 4);
                for (int c = lane; c < YR; c += 32) {
                    // past the array's end: any row, its weight is masked
                    const int64_t r = min(y0 + c, LY - 1);
                    if (BIAS) {
                        const float *p =
                            (MODE == ATTN_DKV ? a.qxyz : a.rxyz) + (int64_t(b) * LY + r) * 3;
                        cp_async_4(cd + c, p);
                        cp_async_4(cd + YR + c, p + 1);
                        cp_async_4(cd + 2 * YR + c, p + 2);
                    }
                    if (MODE == ATTN_DKV) {
                        const int64_t at = (int64_t(b) * a.H + h) * a.Lq + r;
                        cp_async_4(cd + 3 * YR + c, a.lse2 + at);
                        cp_async_4(cd + 4 * YR + c, a.delta + at);
                    }
                }
                cp_async_mbar_arrive(&full[s]);
                __syncwarp();
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[s], 2 * C::YBYTES);
                const CUtensorMap *m1 = MODE == ATTN_DKV ? &maps.q : &maps.k;
                const CUtensorMap *m2 = MODE == ATTN_DKV ? &maps.go : &maps.v;
                const int hy = MODE == ATTN_DKV ? h : hk;
                unsigned char *y1 = Y + size_t(s) * 2 * C::YBYTES, *y2 = y1 + C::YBYTES;
                for (int p = 0; p < DP / 64; ++p) {
                    tma_load_4d(y1 + p * YR * 128, m1, 64 * p, y0, hy, b, &full[s]);
                    tma_load_4d(y2 + p * YR * 128, m2, 64 * p, y0, hy, b, &full[s]);
                }
            }
            issued = k + 1;
        }
        // nothing is in flight when the block ends
        if (n > 0) mbar_wait_bounded(xfull, 0, a.timeout_ns);
        for (int k = max(0, issued - STAGES); k < issued; ++k)
            mbar_wait_bounded(&full[k % STAGES], unsigned((k / STAGES) & 1), a.timeout_ns);
    } else if (warp == C::CWARPS + 1) {
        // ---- products ---------------------------------------------------------------
        bool ok = n > 0 && wait(xfull, 0);
        const uint64_t x1 = smem_desc(smem_u32(X1), 16), x2 = smem_desc(smem_u32(X2), 16);
        auto scores = [&](int k) {
            const int s = k % STAGES, buf = k % NB;
            if (!wait(&full[s], unsigned((k / STAGES) & 1))) return false;
            unsigned char *y1 = Y + size_t(s) * 2 * C::YBYTES, *y2 = y1 + C::YBYTES;
            const int valid = ny - item_row(k);
            if (valid < YR && ny < LY) {
                const uint4 zero = make_uint4(0, 0, 0, 0);
                for (int p = 0; p < DP / 64; ++p)
                    for (int i = valid * 8 + lane; i < YR * 8; i += 32) {
                        if (BWD) reinterpret_cast<uint4 *>(y1 + p * YR * 128)[i] = zero;
                        if (MODE != ATTN_DQ) reinterpret_cast<uint4 *>(y2 + p * YR * 128)[i] = zero;
                    }
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (lane == 0) {
                constexpr uint32_t id = mma_idesc(YR, false);
                const uint32_t d = tmem + buf * C::BUF;
                const uint64_t d1 = smem_desc(smem_u32(y1), 16), d2 = smem_desc(smem_u32(y2), 16);
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    const uint64_t xo = (i / 4) * (XR * 128 / 16) + (i % 4) * 2;
                    const uint64_t yo = (i / 4) * (YR * 128 / 16) + (i % 4) * 2;
                    mma_ss(d, x1 + xo, d1 + yo, id, i > 0);
                }
                if (BWD)
#pragma unroll
                    for (int i = 0; i < DP / 16; ++i) {
                        const uint64_t xo = (i / 4) * (XR * 128 / 16) + (i % 4) * 2;
                        const uint64_t yo = (i / 4) * (YR * 128 / 16) + (i % 4) * 2;
                        mma_ss(d + YR, x2 + xo, d2 + yo, id, i > 0);
                    }
                mma_commit(&sfull[buf]);
            }
            __syncwarp();
            return true;
        };
        for (int k = 0; ok && k < NB - 1 && k < n; ++k) ok = scores(k);
        for (int k = 0; ok && k < n; ++k) {
            // the buffer of tile k - 1: its sums were issued before, and
            // products run in the order of their issue
            if (k + NB - 1 < n && !(ok = scores(k + NB - 1))) break;
            const int s = k % STAGES, buf = k % NB;
            if (!(ok = wait(&pfull[buf], unsigned((k / NB) & 1)))) break;
            tc_fence_after();
            if (lane == 0) {
                constexpr uint32_t id = mma_idesc(DP, true);
                unsigned char *y1 = Y + size_t(s) * 2 * C::YBYTES, *y2 = y1 + C::YBYTES;
                const uint64_t d1 = smem_desc(smem_u32(y1), YR * 128),
                               d2 = smem_desc(smem_u32(y2), YR * 128);
                const uint32_t p = tmem + buf * C::BUF, acc = tmem + C::ACC;
#pragma unroll
                for (int i = 0; i < YR / 16; ++i) {
                    // step i: 16 weights in 8 columns, their low parts in the next 8
                    const uint32_t at = p + 16 * i, as = at + YR;
                    const uint64_t yo = i * (16 * 128 / 16);
                    const bool more = k > 0 || i > 0;
                    if (MODE == ATTN_FWD) {
                        mma_ts(acc, at, d2 + yo, id, more);
                        if (C::TWO_P) mma_ts(acc, at + 8, d2 + yo, id, true);
                    } else {
                        mma_ts(acc, as, d1 + yo, id, more);
                        if (C::TWO_S) mma_ts(acc, as + 8, d1 + yo, id, true);
                    }
                    if (MODE == ATTN_DKV) {
                        mma_ts(acc + DP, at, d2 + yo, id, more);
                        if (C::TWO_P) mma_ts(acc + DP, at + 8, d2 + yo, id, true);
                    }
                }
                mma_commit(&empty[s]);
                if (MODE == ATTN_FWD) mma_commit(pvdone);
            }
            __syncwarp();
        }
        if (lane == 0) mma_commit(accfull);
        __syncwarp();
        mbar_wait_bounded(accfull, 0, a.timeout_ns);  // before the tensor memory is freed
    } else {
        // ---- weights ------------------------------------------------------------------
        const int quad = warp % 4, grp = warp / 4, half = grp % CH, wg = grp / CH;
        const int row = r0 + quad * 32 + lane;
        const bool live = r0 + quad * 32 < nx;  // of the warp: else nothing is read of its rows
        const uint32_t lanes = uint32_t(quad * 32) << 16;
        const float c2 = a.scale * ATTN_LOG2E;
        const float2 c22 = make_float2(c2, c2);
        float2 nx2 = make_float2(0.0f, 0.0f), ny2 = nx2, nz2 = nx2, nb2 = nx2;
        if (BIAS) {
            if (row < nx) {
                const float *p =
                    (MODE == ATTN_DKV ? a.rxyz : a.qxyz) + (int64_t(b) * LX + row) * 3;
                nx2 = make_float2(-p[0], -p[0]);
                ny2 = make_float2(-p[1], -p[1]);
                nz2 = make_float2(-p[2], -p[2]);
            }
            // the bias in units of the raw scores
            const float w = -a.slopes[head] / a.scale;
            if (MODE != ATTN_DKV) nb2 = make_float2(w, w);
        }
        float nlse = -INFINITY, ndel = 0.0f;  // DQ: -lse in base 2, -delta
        if (MODE == ATTN_DQ && row < nx) {
            const int64_t at = (int64_t(b) * a.H + head) * a.Lq + row;
            nlse = -a.lse2[at];
            ndel = -a.delta[at];
        }
        float mc = -INFINITY;                        // FWD: the row's maximum, base 2
        float2 l2 = make_float2(0.0f, 0.0f);         // FWD: the row's sum
        float2 wa = l2, we = l2, wd = l2;            // DQ: the slope's sums
        const bool sums = MODE == ATTN_DQ && BIAS && a.rowsum != nullptr;
        int hcur = -1;
        bool ok = true;
        for (int k = wg; k < n; k += W) {
            const int s = k % STAGES, buf = k % NB;
            if (!(ok = wait(&sfull[buf], unsigned((k / NB) & 1)))) break;
            if (!(ok = wait(&full[s], unsigned((k / STAGES) & 1)))) break;
            tc_fence_after();
            const float *cd = coldata + s * (C::COLDATA / 4) + 32 * half;
            const uint32_t sb = tmem + lanes + buf * C::BUF + 32 * half;
            const int valid = ny - item_row(k) - 32 * half;  // columns of this half, if < 32
            if (MODE == ATTN_DKV && BIAS && item_head(k) != hcur) {
                hcur = item_head(k);
                const float w = -a.slopes[hcur] / a.scale;
                nb2 = make_float2(w, w);
            }
            if (MODE == ATTN_FWD && live) {
                uint32_t r[32];
                tmem_ld32(sb, r);
                tmem_wait_ld();
                if (BIAS)
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        float2 d0, d1;
                        dist4(cd, c, nx2, ny2, nz2, d0, d1);
                        const float2 u = __ffma2_rn(d0, nb2, pair(r, c));
                        const float2 v = __ffma2_rn(d1, nb2, pair(r, c + 2));
                        r[c] = __float_as_uint(u.x), r[c + 1] = __float_as_uint(u.y);
                        r[c + 2] = __float_as_uint(v.x), r[c + 3] = __float_as_uint(v.y);
                    }
                if (valid < 32)
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (c >= valid) r[c] = __float_as_uint(-INFINITY);
                float m = -INFINITY;
#pragma unroll
                for (int c = 0; c < 32; c += 2)
                    m = fmax3(m, __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
                // the row's maximum over both halves; the slots alternate, so
                // one exchange a tile is enough
                float *mx = rsum + (k & 1) * CH * XR + quad * 32 + lane;
                mx[half * XR] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(&mxbar[quad]);
                if (!(ok = wait(&mxbar[quad], unsigned(k & 1)))) break;
                m = fmaxf(m, mx[(half ^ 1) * XR]) * c2;
                // The base of the exponents follows the maximum only when it
                // grew by more than 2^8 (the weights stay below 256, far from
                // float32's and bfloat16's ends): the accumulator is seldom
                // rescaled.
                const bool need = m > mc + 8.0f;
                if (__any_sync(0xffffffffu, need)) {
                    const float mn = need ? m : mc;
                    const float f = mn == -INFINITY ? 1.0f : ex2(mc - mn);
                    mc = mn;
                    l2.x *= f;
                    l2.y *= f;
                    if (k > 0) {
                        if (!(ok = wait(pvdone, unsigned((k - 1) & 1)))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < DP / CH; c += 8) {
                            const uint32_t at = tmem + lanes + C::ACC + half * (DP / CH) + c;
                            uint32_t o[8];
                            tmem_ld8(at, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st8(at, o);
                        }
                    }
                }
                const float mb = mc == -INFINITY ? 0.0f : -mc;
                const float2 mb2 = make_float2(mb, mb);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[8], lo[8];
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        float2 t = __ffma2_rn(pair(r, 16 * h + c), c22, mb2);
                        t.x = ex2(t.x);
                        t.y = ex2(t.y);
                        l2 = __fadd2_rn(l2, t);
                        split_bf16(t, p[c / 2], lo[c / 2]);
                    }
                    tmem_st8(sb + 16 * h, p);
                    if (C::TWO_P) tmem_st8(sb + 16 * h + 8, lo);
                }
            } else if (live) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t r[16], g[16], p[8], plo[8], q[8], qlo[8];
                    tmem_ld16(sb + 16 * h, r);
                    tmem_ld16(sb + YR + 16 * h, g);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        float2 d[2];
                        if (BIAS) dist4(cd, 16 * h + c, nx2, ny2, nz2, d[0], d[1]);
                        float4 cl, cdl;
                        if (MODE == ATTN_DKV) {
                            cl = *reinterpret_cast<const float4 *>(cd + 3 * YR + 16 * h + c);
                            cdl = *reinterpret_cast<const float4 *>(cd + 4 * YR + 16 * h + c);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int i = c + 2 * e, col = 16 * h + i;
                            float2 u = pair(r, i);
                            if (BIAS) u = __ffma2_rn(d[e], nb2, u);
                            float2 nl = make_float2(nlse, nlse), nd = make_float2(ndel, ndel);
                            if (MODE == ATTN_DKV) {
                                nl = e == 0 ? make_float2(-cl.x, -cl.y) : make_float2(-cl.z, -cl.w);
                                nd = e == 0 ? make_float2(-cdl.x, -cdl.y)
                                            : make_float2(-cdl.z, -cdl.w);
                            }
                            u = __ffma2_rn(u, c22, nl);
                            u.x = ex2(u.x);
                            u.y = ex2(u.y);
                            float2 ds = __fmul2_rn(u, __fadd2_rn(pair(g, i), nd));
                            if (valid < 32) {
                                if (col >= valid) u.x = ds.x = 0.0f;
                                if (col + 1 >= valid) u.y = ds.y = 0.0f;
                            }
                            if (sums) {
                                if (valid < 32) {  // 0 times a masked NaN
                                    if (col >= valid) d[e].x = 0.0f;
                                    if (col + 1 >= valid) d[e].y = 0.0f;
                                }
                                wd = __fadd2_rn(wd, ds);
                                wa = __ffma2_rn(ds, d[e], wa);
                                we = __ffma2_rn(u, d[e], we);
                            }
                            if (MODE == ATTN_DKV) split_bf16(u, p[i / 2], plo[i / 2]);
                            split_bf16(ds, q[i / 2], qlo[i / 2]);
                        }
                    }
                    if (MODE == ATTN_DKV) {
                        tmem_st8(sb + 16 * h, p);
                        if (C::TWO_P) tmem_st8(sb + 16 * h + 8, plo);
                    }
                    tmem_st8(sb + YR + 16 * h, q);
                    if (C::TWO_S) tmem_st8(sb + YR + 16 * h + 8, qlo);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&pfull[buf]);
                mbar_arrive(&empty[s]);
            }
        }
        const int64_t hrow = (int64_t(b) * a.H + head) * a.Lq + row;  // FWD, DQ
        const int64_t hrows = int64_t(a.B) * a.H * a.Lq;
        if (MODE == ATTN_DQ && BIAS) {
            if (sums) {
                float *t = rsum + grp * 3 * XR + quad * 32 + lane;
                t[0] = wa.x + wa.y;
                t[XR] = we.x + we.y;
                t[2 * XR] = wd.x + wd.y;
            }
            named_barrier_sync(1, C::CWARPS * 32);
            if (sums && grp == 0 && row < LX) {
                float *o = a.rowsum + split * 3 * hrows + hrow;
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    float t = 0.0f;
#pragma unroll
                    for (int i = 0; i < W * CH; ++i)
                        t += rsum[(i * 3 + e) * XR + quad * 32 + lane];
                    o[e * hrows] = row < nx ? t : 0.0f;
                }
            }
        }
        float l = l2.x + l2.y;
        if (MODE == ATTN_FWD) {  // the row's sum over both halves
            float *t = rsum + 2 * CH * XR + quad * 32 + lane;
            t[half * XR] = l;
            named_barrier_sync(1, C::CWARPS * 32);
            l = t[0] + t[XR];
        }
        const bool any = MODE == ATTN_FWD ? row < nx && l > 0.0f : row < nx;
        if (MODE == ATTN_FWD && row < LX && half == 0) {
            if (a.nsplit > 1) {
                a.part_ml[int64_t(split) * 2 * hrows + hrow] = mc;
                a.part_ml[(int64_t(split) * 2 + 1) * hrows + hrow] = l;
            } else if (a.lse != nullptr) {
                a.lse[hrow] = any ? (mc + log2f(l)) * ATTN_LN2 : -INFINITY;
            }
        }
        if (ok && n > 0) ok = wait(accfull, 0);
        tc_fence_after();
        const int64_t orow = (int64_t(b) * LX + row) * NH + head;
        const int64_t rows = int64_t(a.B) * LX * NH;
        // the groups share the accumulators' columns
        for (int ch = grp; ch < C::NACC * DP / 32; ch += W * CH) {
            const int acc = ch / (DP / 32), c0 = (ch % (DP / 32)) * 32;
            uint32_t r[32];
            float v[32];
            __syncwarp();
            if (n > 0 && ok) {
                tmem_ld32(tmem + lanes + C::ACC + ch * 32, r);
                tmem_wait_ld();
            }
            const float f = a.nsplit > 1 ? 1.0f
                            : MODE == ATTN_FWD ? 1.0f / l
                            : acc == 0         ? a.scale
                                               : 1.0f;
#pragma unroll
            for (int e = 0; e < 32; ++e)
                v[e] = n > 0 && ok && any ? __uint_as_float(r[e]) * f : 0.0f;
            if (row >= LX) {
                // past the array's end: nothing to store
            } else if (a.nsplit > 1) {
                store_row32(a.part + ((int64_t(acc) * a.nsplit + split) * rows + orow) * a.D + c0,
                            v, c0, a.D);
            } else {
                void *o = MODE == ATTN_FWD ? a.out : MODE == ATTN_DQ ? a.dq : acc ? a.dv : a.dk;
                store_row32(static_cast<bf16 *>(o) + orow * a.D + c0, v, c0, a.D);
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == C::CWARPS + 1) tmem_free(tmem, C::COLS);
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

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

template <int MODE, int DP, bool BIAS>
cudaError_t tc_launch(const AttnArgs &a, const AttnMaps &m, int64_t blocks, cudaStream_t st) {
    using C = Cfg<MODE, DP>;
    const cudaError_t e =
        cudaFuncSetAttribute(attn_tc_kernel<MODE, DP, BIAS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::SMEM));
    if (e != cudaSuccess) return e;
    attn_tc_kernel<MODE, DP, BIAS><<<unsigned(blocks), C::THREADS, C::SMEM, st>>>(
        a, m, (debug_stall() & PC_STALL_ATTENTION) != 0);
    return cudaGetLastError();
}

template <int MODE>
cudaError_t tc_pick(const AttnArgs &a, const AttnMaps &m, int64_t blocks, cudaStream_t st) {
    if (a.D <= 64)
        return a.slopes ? tc_launch<MODE, 64, true>(a, m, blocks, st)
                        : tc_launch<MODE, 64, false>(a, m, blocks, st);
    return a.slopes ? tc_launch<MODE, 128, true>(a, m, blocks, st)
                    : tc_launch<MODE, 128, false>(a, m, blocks, st);
}

}  // namespace

bool attn_tc_fits(const AttnArgs &a, int mode) {
    if (a.D % 8 != 0 || a.Lq < 1 || a.Lk < 1) return false;
    auto aligned = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    auto fits = [&](const void *p, const int64_t *s, int64_t L, int64_t heads) {
        auto ok = [](int64_t stride, int64_t extent) {
            return extent <= 1 || (stride > 0 && stride % 8 == 0 && stride < (int64_t(1) << 38));
        };
        return aligned(p) && ok(s[0], a.B) && ok(s[1], L) && ok(s[2], heads);
    };
    if (!fits(a.q, a.qs, a.Lq, a.H) || !fits(a.k, a.ks, a.Lk, a.Hkv) ||
        !fits(a.v, a.vs, a.Lk, a.Hkv))
        return false;
    if (mode == ATTN_FWD) return aligned(a.out);
    return aligned(a.go) && aligned(a.dq) && aligned(a.dk) && aligned(a.dv);
}

cudaError_t launch_attn_tc(const AttnArgs &a, int mode, int64_t blocks, cudaStream_t st) {
    AttnMaps m{};
    const int64_t gs[3] = {int64_t(a.Lq) * a.H * a.D, int64_t(a.H) * a.D, a.D};
    if (!make_map(&m.q, a.q, a.qs, a.B, a.Lq, a.H, a.D) ||
        !make_map(&m.k, a.k, a.ks, a.B, a.Lk, a.Hkv, a.D) ||
        !make_map(&m.v, a.v, a.vs, a.B, a.Lk, a.Hkv, a.D) ||
        (mode != ATTN_FWD && !make_map(&m.go, a.go, gs, a.B, a.Lq, a.H, a.D)))
        return cudaErrorInvalidValue;
    return mode == ATTN_FWD  ? tc_pick<ATTN_FWD>(a, m, blocks, st)
           : mode == ATTN_DQ ? tc_pick<ATTN_DQ>(a, m, blocks, st)
                             : tc_pick<ATTN_DKV>(a, m, blocks, st);
}

}  // namespace pcn
