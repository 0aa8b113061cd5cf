// pc_attn_tc.cu -- the attention passes of pc_attn.cuh on the tensor cores,
// for bfloat16.
//
// A block keeps rows (FWD 2 x 128, DQ and DKV 128) and walks over the other
// side in tiles of 64:
//   scores   S = X1 Y1^T (and dP = X2 Y2^T), both operands in shared memory,
//            the result in tensor memory, one lane per row;
//   weights  a thread owns half a row: it reads its scores and writes P (and
//            dS) back as bfloat16 over them;
//   sums     acc += P Y2 (and dS Y1), the weights read from tensor memory,
//            the same shared-memory tile now contracted along its rows.
// One warp copies tiles (tensor maps, 128-byte swizzle; zeros past the
// arrays' ends), two prepare the positions, one issues the products, 16
// compute weights in two units of 8: FWD one unit per 128 rows, DQ and DKV
// units that take tiles in turn.  Each unit has score buffers of its own, so
// products run under weights.
//
// The bias -b |x - y|^2 (b = slope / scale, in units of the raw scores) is
// 2 b x.y - b |y|^2 - b |x|^2: a product over 27 more channels, in which every
// number is a sum of three bfloat16 (all pairs of parts above 2^-24), added by
// two more steps of the same products.  The coordinates are taken relative to
// the block's first row; the parts are exact to float32, but the three terms
// cancel where x is near y, which costs up to 2^-20 b R^2.  So a tile takes
// this way only where slope R^2 <= 256 (R: the farthest of the block's rows
// and the tile's from the center); elsewhere, and where the slopes' gradient
// needs the distances themselves, the threads form the distance from the
// coordinates' differences.  Per score the threads' work falls from about 10
// instructions to 5.
//
// Both operands of a product have one type, and P in bfloat16 alone would cost
// up to 2^-8 of a term (the output's and dv's error against float64 0.0024
// instead of 0.0017, which is the rounding of the result): P is written as the
// sum of two bfloat16 (2^-17) and multiplied twice.  So is dS: in one bfloat16,
// at any number of rows, dq and dk would be off by 0.0024 too (it would save 9 to
// 15% of the backward pass).  The sums of P, the statistics and all accumulators
// are float32, and the slopes' gradient uses the unrounded weights.
//
// What lies past a cloud's length is masked in the weights; rows of a
// streamed tile past the length (they would meet weights that are 0, and 0
// times NaN is NaN) are overwritten with zeros in shared memory.
//
// Measured, 4864 queries and keys, 16 heads: 64 channels, forward 137 us (707
// TFLOP/s of 4 D a score; with the bias 165 us), both backward passes with delta 370
// us (655 TFLOP/s of 10 D; 441 us, with the slopes' gradient 571 us); 128 channels 169
// us (1147; 207 us) and 640 us (757; 719 and 822 us).  The weights' threads issue on
// 60% of the cycles, the tensor cores' math is active on about 40%.  The products
// are small (128 x 64 x 16), so what issues them matters: from a branch on a lane
// index each took 80 to 150 cycles, from an elected lane 30 to 70, from one thread
// that runs the whole loop they are limited by the tensor cores' queue.
//
// Every wait on a barrier is bounded: when one runs out the block raises the status
// word, lets its copies and products finish, frees its tensor memory and returns;
// its outputs are then unspecified.  The allocation of tensor memory has no bound
// of its own: it waits while another block on the SM holds some.  No two blocks of
// these kernels fit one SM, so that can only be another library's kernel, and for
// as long as that runs.
#include "pc_attn_tc.cuh"
#include "pointcloud.h"

#include <type_traits>

namespace pcn {
namespace {

constexpr float AUG_MOST = 256.0f;  // of slope R^2: see above

struct AttnMaps {
    CUtensorMap q, k, v, go;
};

template <int MODE, int DP>
struct Cfg {
    static constexpr bool BWD = MODE != ATTN_FWD, FWD_ = !BWD;
    static constexpr int T = BWD ? 1 : 2;       // row tiles of the block
    static constexpr int CWARPS = 16;           // two units of two halves of four warps
    static constexpr int THREADS = 32 * (CWARPS + 4);
    static constexpr int STAGES = DP == 64 ? 6 : 3;
    // Tensor memory columns: score buffers (FWD two a unit; else of S and dP, one
    // a unit, and for up to 64 channels a third, so that the scores of a unit's
    // next tile are there before its weights are used up), then the accumulators.
    static constexpr int NBUF = FWD_ ? 4 : DP == 64 ? 3 : 2, BUF = BWD ? 2 * YR : YR;
    static constexpr int ACC = NBUF * BUF;
    static constexpr int NACC = MODE == ATTN_DQ ? 1 : 2;  // FWD: one a unit
    // The rows kept, where tensor memory has room for them: a product that reads
    // both operands from shared memory is bound by that (48 cycles instead of 32
    // for 128 x 64 x 16).
    static constexpr int XCOL = ACC + NACC * DP;
    static constexpr bool X_TMEM = XCOL + DP <= 512;
    static constexpr int COLS = 512;
    static_assert(XCOL <= COLS, "tensor memory");
    static constexpr int XBYTES = XR * DP * 2, YBYTES = YR * DP * 2;
    static constexpr int XT = BWD ? 2 : T;      // tiles kept
    static constexpr int XAUG = XR * 64, YAUG = YR * 64;  // 32 channels
    static constexpr int STAGE = 2 * YBYTES + YAUG;
    // per stage: x, y, z, -lse, -delta of the streamed rows; flag, bias factor
    static constexpr int COLF = 5 * YR + 4;
    static constexpr int ROWF = 2 * 8 * XR + 4;  // per unit: exchanged row values
    static constexpr size_t XSMEM = X_TMEM ? 0 : size_t(XT) * XBYTES;
    static constexpr size_t SMEM = 1024 + XSMEM + size_t(T) * XAUG +
                                   size_t(STAGES) * (STAGE + COLF * 4) + ROWF * 4 + 512;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(SMEM > 114 * 1024, "one block a SM: none waits for tensor memory");
};

// A number as three bfloat16, the low one of what the others leave.
struct Parts {
    float h, m, l;
    __device__ __forceinline__ explicit Parts(float v) {
        h = __bfloat162float(__float2bfloat16_rn(v));
        m = __bfloat162float(__float2bfloat16_rn(v - h));
        l = (v - h) - m;  // rounded when packed
    }
};

// The 27 channels of a row, in 64-byte rows with the 64-byte swizzle:
// d = position - center; `query`: the side that carries b, else the keys'.
__device__ __forceinline__ void write_aug(unsigned char *tile, int row, bool query, float dx,
                                          float dy, float dz, float b) {
    const float n = fmaf(dz, dz, fmaf(dy, dy, dx * dx));
    const float f = query ? 2.0f * b : 1.0f;
    const Parts p[4] = {Parts(f * dx), Parts(f * dy), Parts(f * dz), Parts(query ? b : -n)};
    float v[32];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        // pairs of parts: hh, hm, mh, hl, lh, mm
        v[6 * e] = p[e].h;
        v[6 * e + 1] = query ? p[e].h : p[e].m;
        v[6 * e + 2] = query ? p[e].m : p[e].h;
        v[6 * e + 3] = query ? p[e].h : p[e].l;
        v[6 * e + 4] = query ? p[e].l : p[e].h;
        v[6 * e + 5] = p[e].m;
    }
    const Parts t(-b * n);
    v[24] = query ? t.h : 1.0f;
    v[25] = query ? t.m : 1.0f;
    v[26] = query ? t.l : 1.0f;
#pragma unroll
    for (int e = 27; e < 32; ++e) v[e] = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        Vec<bf16, 8>::store(reinterpret_cast<bf16 *>(tile + row * 64 + ((c ^ ((row >> 1) & 3)) * 16)),
                            v + 8 * c);
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

// One pass of block `bid`.
template <int MODE, int DP, bool BIAS>
__device__ __forceinline__ void attn_tc_pass(const AttnArgs &a, const AttnMaps &maps,
                                             const bool withhold, const unsigned bid) {
    using C = Cfg<MODE, DP>;
    constexpr bool BWD = C::BWD, FWD = !BWD, DKV = MODE == ATTN_DKV;
    constexpr bool COLS = BIAS || DKV;  // the weights read data of the streamed rows
    constexpr int STAGES = C::STAGES, T = C::T;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char *X = base;  // FWD: q of both tiles; else X1, X2 (if not in tensor memory)
    unsigned char *Y = X + C::XSMEM;               // stage s: Y1, Y2, channels of the bias
    unsigned char *xaug = Y + size_t(STAGES) * C::STAGE;
    float *coldata = reinterpret_cast<float *>(xaug + T * C::XAUG);
    float *rowdata = coldata + STAGES * C::COLF;   // [unit][8][XR]
    uint64_t *full = reinterpret_cast<uint64_t *>(rowdata + C::ROWF);
    uint64_t *empty = full + STAGES, *sfull = empty + STAGES, *pfull = sfull + C::NBUF;
    uint64_t *xfull = pfull + C::NBUF, *accfull = xfull + 1;
    uint64_t *fixed = accfull + 1, *mxbar = fixed + STAGES;  // mxbar: [unit][quad]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mxbar + 8);
    int *xr2 = reinterpret_cast<int *>(tmem_slot + 1);  // R^2 of the block's rows, as bits
    volatile int *stop = reinterpret_cast<volatile int *>(xr2 + 1);

    // (values broadcast by a shuffle are known to be the same in all lanes: the
    // branches on them, and what the products' operands are formed from, then
    // stay in uniform registers)
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int LX = DKV ? a.Lk : a.Lq, LY = DKV ? a.Lq : a.Lk;
    const int NH = DKV ? a.Hkv : a.H;
    const int G = a.H / a.Hkv;
    const int ntile = (LX + T * XR - 1) / (T * XR);
    int64_t idx = bid;
    const int split = int(idx % a.nsplit);
    idx /= a.nsplit;
    const int tile = int(idx % ntile);
    idx /= ntile;
    const int head = int(idx % NH), b = int(idx / NH);
    const int nq = attn_len(a.qlen, b, a.Lq), nk = attn_len(a.rlen, b, a.Lk);
    const int nx = uniform(DKV ? nk : nq), ny = uniform(DKV ? nq : nk);
    const int r0 = tile * T * XR;
    const int hk = DKV ? head : head / G;
    const int nyt = (ny + YR - 1) / YR;
    const int64_t items = nx > r0 ? int64_t(nyt) * (DKV ? G : 1) : 0;
    const int64_t it0 = items * split / a.nsplit;
    const int n = uniform(int(items * (split + 1) / a.nsplit - it0));  // tiles of this block
    const float *xpos = DKV ? a.rxyz : a.qxyz, *ypos = DKV ? a.qxyz : a.rxyz;
    const bool ragged = ny < LY && ny % YR != 0;  // the last tile has rows past the length
    // the slopes' gradient needs the distances themselves
    const bool sums = MODE == ATTN_DQ && BIAS && a.rowsum != nullptr;

    // the row of a thread that computes weights
    const int quad = warp % 4, half = (warp / 4) % 2, unit = (warp / 8) % 2;
    const int xt = FWD ? unit : 0;
    const int row = r0 + xt * XR + quad * 32 + lane;
    float px = 0.0f, py = 0.0f, pz = 0.0f, cx = 0.0f, cy = 0.0f, cz = 0.0f;
    if (BIAS && n > 0) {
        const float *c = xpos + (int64_t(b) * LX + r0) * 3;
        cx = c[0], cy = c[1], cz = c[2];
        if (warp < C::CWARPS && row < nx) {
            const float *p = xpos + (int64_t(b) * LX + row) * 3;
            px = p[0], py = p[1], pz = p[2];
        }
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], COLS ? 2 : 1);
            mbar_init(&fixed[s], 1);
            mbar_init(&empty[s], 1 + (COLS ? (FWD ? 16 : 8) : 0));
        }
        for (int s = 0; s < C::NBUF; ++s) {
            mbar_init(&sfull[s], 1);
            mbar_init(&pfull[s], 8);
        }
        mbar_init(xfull, 1);
        mbar_init(accfull, 1);
        for (int s = 0; s < 8; ++s) mbar_init(&mxbar[s], 2);
        *xr2 = 0;
        *stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == C::CWARPS + 1) tmem_alloc(tmem_slot, C::COLS);
    tc_fence_before();
    __syncthreads();
    if (C::X_TMEM && n > 0 && warp < C::CWARPS) {
        // FWD: each unit its tile's q, half the channels each; else unit 0 X1 and
        // unit 1 X2.  Two channels a column, zeros past the rows and channels.
        tc_fence_after();
        const bf16 *src;
        if (FWD || (MODE == ATTN_DQ && unit == 0))
            src = static_cast<const bf16 *>(a.q) + b * a.qs[0] + head * a.qs[2] +
                  int64_t(row) * a.qs[1];
        else if (MODE == ATTN_DQ)
            src = static_cast<const bf16 *>(a.go) +
                  ((int64_t(b) * a.Lq + row) * a.H + head) * a.D;
        else if (unit == 0)
            src = static_cast<const bf16 *>(a.k) + b * a.ks[0] + head * a.ks[2] +
                  int64_t(row) * a.ks[1];
        else
            src = static_cast<const bf16 *>(a.v) + b * a.vs[0] + head * a.vs[2] +
                  int64_t(row) * a.vs[1];
        const uint32_t at = uint32_t(uniform(int(*tmem_slot))) + (uint32_t(quad * 32) << 16) +
                            C::XCOL + unit * (DP / 2) + half * (DP / 4);
#pragma unroll
        for (int c = 0; c < DP / 2; c += 16) {
            uint32_t r[8];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int ch = half * (DP / 2) + c + 8 * e;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (row < nx && ch < a.D) v = *reinterpret_cast<const uint4 *>(src + ch);
                r[4 * e] = v.x, r[4 * e + 1] = v.y, r[4 * e + 2] = v.z, r[4 * e + 3] = v.w;
            }
            tmem_st8(at + c / 2, r);
        }
        tmem_wait_st();
        tc_fence_before();
    }
    if (C::X_TMEM && !BIAS) __syncthreads();
    if (BIAS && n > 0) {
        if (warp < C::CWARPS && half == 0 && (FWD || unit == 0)) {
            const bool in = row < nx;
            const float dx = in ? px - cx : 0.0f, dy = in ? py - cy : 0.0f,
                        dz = in ? pz - cz : 0.0f;
            write_aug(xaug + xt * C::XAUG, quad * 32 + lane, !DKV, dx, dy, dz,
                      DKV ? 0.0f : a.slopes[head] / a.scale);
            // (a NaN or an infinity counts as the largest: no tile takes the products)
            const float r2 = fmaf(dz, dz, fmaf(dy, dy, dx * dx));
            atomicMax(xr2, __float_as_int(r2 <= 1e30f ? r2 : 1e30f));
            fence_proxy_async_smem();
        }
        __syncthreads();
    }
    tc_fence_after();
    const uint32_t tmem = uniform(int(*tmem_slot));

    // A bounded wait of a whole warp; false: stop.
    auto wait = [&](uint64_t *bar, unsigned parity) {
        const WaitResult w = mbar_wait_or_stop(bar, parity, stop, a.timeout_ns);
        if (w == WAIT_TIMEOUT) {
            *stop = 1;
            raise_status(a.status, PC_ERR_DEVICE_TIMEOUT);
        }
        return __all_sync(0xffffffffu, w == WAIT_OK) != 0;
    };
    auto walk = [&](int skip) {
        return TileWalk(DKV, DKV ? hk * G : head, n > 0 ? nyt : 0, it0, skip);
    };

    if (warp == C::CWARPS) {
        // ---- copies ---------------------------------------------------------------
        if (!C::X_TMEM && n > 0 && elect_one()) {
            mbar_arrive_expect_tx(xfull, C::XT * C::XBYTES);
            for (int p = 0; p < DP / 64; ++p)
                for (int h = 0; h < 2; ++h) {
                    unsigned char *at = X + p * XR * 128 + h * YR * 128;
                    const int r = r0 + YR * h;
                    tma_load_4d(at, DKV ? &maps.k : &maps.q, 64 * p, r, head, b, xfull);
                    if (FWD)
                        tma_load_4d(at + C::XBYTES, &maps.q, 64 * p, r + XR, head, b, xfull);
                    else
                        tma_load_4d(at + C::XBYTES, DKV ? &maps.v : &maps.go, 64 * p, r, head, b,
                                    xfull);
                }
        }
        // Rows of a tile past the length are overwritten with zeros once the tile
        // is there: LAG tiles later, so that copies stay ahead.  A tile's stage is
        // free only after the scores of the next tiles (NBUF - 1 of them, FWD one),
        // which wait for their zeros, were issued: those zeros come before the
        // wait for the stage that the next copy goes to.
        constexpr int LAG = STAGES - 1 - (FWD ? 1 : C::NBUF - 1) < 2
                                ? STAGES - 1 - (FWD ? 1 : C::NBUF - 1)
                                : 2;
        static_assert(LAG >= 0, "more stages than score buffers");
        TileWalk late = walk(0);
        auto fix = [&](int k) {
            const int valid = ny - late.y, s = k % STAGES;
            late.next();
            if (!ragged || valid >= YR) return true;
            if (!wait(&full[s], unsigned((k / STAGES) & 1))) return false;
            unsigned char *y1 = Y + size_t(s) * C::STAGE, *y2 = y1 + C::YBYTES;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            for (int p = 0; p < DP / 64; ++p)
                for (int i = valid * 8 + lane; i < YR * 8; i += 32) {
                    if (BWD) reinterpret_cast<uint4 *>(y1 + p * YR * 128)[i] = zero;
                    if (MODE != ATTN_DQ) reinterpret_cast<uint4 *>(y2 + p * YR * 128)[i] = zero;
                }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&fixed[s]);
            return true;
        };
        int issued = 0;
        bool ok = true;
        TileWalk at = walk(0);
        for (int k = 0; ok && k < n; ++k, at.next()) {
            const int s = k % STAGES;
            if (k >= STAGES && !wait(&empty[s], unsigned((k / STAGES - 1) & 1))) break;
            if (withhold && bid == 0) break;
            if (elect_one()) {
                const int y0 = at.y, hy = DKV ? at.h : hk;
                mbar_arrive_expect_tx(&full[s], 2 * C::YBYTES);
                unsigned char *y1 = Y + size_t(s) * C::STAGE, *y2 = y1 + C::YBYTES;
                for (int p = 0; p < DP / 64; ++p) {
                    tma_load_4d(y1 + p * YR * 128, DKV ? &maps.q : &maps.k, 64 * p, y0, hy, b,
                                &full[s]);
                    tma_load_4d(y2 + p * YR * 128, DKV ? &maps.go : &maps.v, 64 * p, y0, hy, b,
                                &full[s]);
                }
            }
            issued = k + 1;
            if (k >= LAG) ok = fix(k - LAG);
        }
        if (issued == n)
            for (int k = max(0, n - LAG); ok && k < n; ++k) ok = fix(k);
        // nothing is in flight when the block ends
        if (!C::X_TMEM && n > 0) mbar_wait_bounded(xfull, 0, a.timeout_ns);
        for (int k = max(0, issued - STAGES); k < issued; ++k)
            mbar_wait_bounded(&full[k % STAGES], unsigned((k / STAGES) & 1), a.timeout_ns);
    } else if (COLS && warp >= C::CWARPS + 2) {
        // ---- positions: two warps, every other tile each ------------------------------
        const int first = warp - (C::CWARPS + 2);
        TileWalk at = walk(first);
        float nxt[2][5], slope_nxt = 0.0f;  // of the warp's next tile: loaded a tile ahead
        auto fetch = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t r = at.y + lane + 32 * i;
                const bool in = r < ny;
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    nxt[i][e] = BIAS && in ? ypos[(int64_t(b) * LY + r) * 3 + e] : 0.0f;
                if (DKV) {
                    const int64_t o = (int64_t(b) * a.H + at.h) * a.Lq + r;
                    nxt[i][3] = in ? -a.lse2[o] : -INFINITY;
                    nxt[i][4] = in ? -a.delta[o] : 0.0f;
                }
            }
            if (BIAS) slope_nxt = a.slopes[at.h];
        };
        const float xmost = BIAS ? __int_as_float(*xr2) : 0.0f;
        if (first < n) fetch();
        int s = 0;
        unsigned phase = 1;  // of the stage's last release: none in the first round
        for (int k = 0; k < n; ++k, ++s) {
            if (s == STAGES) s = 0, phase ^= 1;
            // (no release is passed over: a parity tells only the last from the
            // one before)
            if (k >= STAGES && !wait(&empty[s], phase)) break;
            if ((k & 1) != first) continue;
            float cur[2][5];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 5; ++e) cur[i][e] = nxt[i][e];
            const float slope = slope_nxt;
            const int valid = ny - at.y;
            at.next(2);
            if (k + 2 < n) fetch();
            float *cd = coldata + s * C::COLF;
            bool direct = true;
            if (BIAS) {
                float r2 = xmost;
                float d[2][3];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool in = lane + 32 * i < valid;
                    d[i][0] = in ? cur[i][0] - cx : 0.0f;
                    d[i][1] = in ? cur[i][1] - cy : 0.0f;
                    d[i][2] = in ? cur[i][2] - cz : 0.0f;
                    const float t = fmaf(d[i][2], d[i][2], fmaf(d[i][1], d[i][1], d[i][0] * d[i][0]));
                    r2 = fmaxf(r2, t <= 1e30f ? t : 1e30f);
                }
                direct = __any_sync(0xffffffffu, !(fabsf(slope) * r2 <= AUG_MOST)) || sums;
                if (!direct) {
                    unsigned char *ya = Y + size_t(s) * C::STAGE + 2 * C::YBYTES;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        write_aug(ya, lane + 32 * i, DKV, d[i][0], d[i][1], d[i][2],
                                  DKV ? slope / a.scale : 0.0f);
                    fence_proxy_async_smem();
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (BIAS && direct)
#pragma unroll
                    for (int e = 0; e < 3; ++e) cd[e * YR + lane + 32 * i] = cur[i][e];
                if (DKV) {
                    cd[3 * YR + lane + 32 * i] = cur[i][3];
                    cd[4 * YR + lane + 32 * i] = cur[i][4];
                }
            }
            if (lane == 0) {
                cd[5 * YR] = direct ? 1.0f : 0.0f;
                cd[5 * YR + 1] = -slope / a.scale;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
        }
    } else if (warp == C::CWARPS + 1) {
        // ---- products ---------------------------------------------------------------
        // One thread runs the loop.  The other warps of its scheduler are busy, so
        // every instruction counts: running stage numbers, operands by addition.
        if (elect_one()) {
            const uint32_t x1 = smem_operand(smem_u32(X)), x2 = x1 + C::XBYTES / 16;
            const uint32_t xa = smem_operand(smem_u32(xaug));
            const uint32_t yk = smem_operand(smem_u32(Y));
            const uint32_t yr = smem_operand(smem_u32(Y), YR * 128);
            const float *flag = coldata + 5 * YR;
            struct Stage {
                int s = 0;
                unsigned phase = 0;
                __device__ __forceinline__ void next() {
                    if (++s == STAGES) s = 0, phase ^= 1;
                }
            } in, out;  // tiles whose scores, whose sums are issued
            TileWalk at = walk(0);
            unsigned fixes = 0;  // a bit per stage: the parity of its next fix
            auto await = [&](uint64_t *bar, unsigned parity) {
                const WaitResult w = mbar_wait_or_stop(bar, parity, stop, a.timeout_ns);
                if (w == WAIT_TIMEOUT) {
                    *stop = 1;
                    raise_status(a.status, PC_ERR_DEVICE_TIMEOUT);
                }
                return w == WAIT_OK;
            };
            auto tile_ready = [&]() {
                if (!await(&full[in.s], in.phase)) return false;
                const int valid = ny - at.y;
                at.next();
                if (ragged && valid < YR) {
                    const unsigned parity = (fixes >> in.s) & 1;
                    fixes ^= 1u << in.s;
                    return await(&fixed[in.s], parity);
                }
                return true;
            };
            // the scores of the tile `in` for a unit, into its buffer
            auto scores = [&](int u, int buf) {
                constexpr uint32_t id = mma_idesc(YR, false);
                const uint32_t d = tmem + buf * C::BUF;
                const uint32_t x = FWD ? x1 + u * (C::XBYTES / 16) : x1;
                const uint32_t y = yk + in.s * (C::STAGE / 16);
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    const uint32_t yo = y + (i / 4) * (YR * 128 / 16) + (i % 4) * 2;
                    if (C::X_TMEM)
                        mma_ts<SMEM_128B>(d, tmem + C::XCOL + u * (DP / 2) + 8 * i, yo, id, i > 0);
                    else
                        mma_ss<SMEM_128B>(d, x + (i / 4) * (XR * 128 / 16) + (i % 4) * 2, yo, id,
                                          i > 0);
                }
                if (BIAS && flag[in.s * C::COLF] == 0.0f) {
                    const uint32_t xb = FWD ? xa + u * (C::XAUG / 16) : xa;
                    const uint32_t yb = y + 2 * C::YBYTES / 16;
                    mma_ss<SMEM_64B>(d, xb, yb, id, true);
                    mma_ss<SMEM_64B>(d, xb + 2, yb + 2, id, true);
                }
                if (BWD)
#pragma unroll
                    for (int i = 0; i < DP / 16; ++i) {
                        const uint32_t yo = y + C::YBYTES / 16 + (i / 4) * (YR * 128 / 16) +
                                            (i % 4) * 2;
                        if (C::X_TMEM)
                            mma_ts<SMEM_128B>(d + YR, tmem + C::XCOL + DP / 2 + 8 * i, yo, id,
                                              i > 0);
                        else
                            mma_ss<SMEM_128B>(d + YR, x2 + (i / 4) * (XR * 128 / 16) + (i % 4) * 2,
                                              yo, id, i > 0);
                    }
                mma_commit(&sfull[buf]);
            };
            // the sums of the tile `out` from a unit's weights
            auto accumulate = [&](int u, int buf, bool first) {
                constexpr uint32_t id = mma_idesc(DP, true);
                const uint32_t d1 = yr + out.s * (C::STAGE / 16), d2 = d1 + C::YBYTES / 16;
                const uint32_t p = tmem + buf * C::BUF, acc = tmem + C::ACC + (FWD ? u * DP : 0);
#pragma unroll
                for (int i = 0; i < YR / 16; ++i) {
                    // step i: 16 weights in 8 columns, their low parts in the next 8
                    const uint32_t at = p + 16 * i, as = at + YR;
                    constexpr uint32_t step = 16 * 128 / 16;
                    const bool more = !first || i > 0;
                    if (FWD) {
                        mma_ts<SMEM_128B>(acc, at, d2 + i * step, id, more);
                        mma_ts<SMEM_128B>(acc, at + 8, d2 + i * step, id, true);
                    } else {
                        mma_ts<SMEM_128B>(acc, as, d1 + i * step, id, more);
                        mma_ts<SMEM_128B>(acc, as + 8, d1 + i * step, id, true);
                    }
                    if (DKV) {
                        mma_ts<SMEM_128B>(acc + DP, at, d2 + i * step, id, more);
                        mma_ts<SMEM_128B>(acc + DP, at + 8, d2 + i * step, id, true);
                    }
                }
            };
            bool ok = n > 0 && (C::X_TMEM || await(xfull, 0));
            // Products run in the order of their issue, so a score buffer may be
            // filled again as soon as the sums that read it were issued.
            if (FWD) {
                const bool two = r0 + XR < nx;
                if (ok && (ok = tile_ready())) {
                    scores(0, 0);
                    if (two) scores(1, 2);
                    in.next();
                }
                for (int k = 0; ok && k < n; ++k) {
                    const int cur = k & 1, nxt = cur ^ 1;
                    const unsigned parity = unsigned(k >> 1) & 1;
                    const bool more = k + 1 < n;
                    if (more && !(ok = tile_ready())) break;
                    // (past the last tile the commit alone tells that the sums
                    // before it are complete: a unit may wait for that to rescale)
                    if (more)
                        scores(0, nxt);
                    else
                        mma_commit(&sfull[nxt]);
                    if (!(ok = await(&pfull[cur], parity))) break;
                    tc_fence_after();
                    accumulate(0, cur, k == 0);
                    if (two) {
                        if (more)
                            scores(1, 2 + nxt);
                        else
                            mma_commit(&sfull[2 + nxt]);
                        if (!(ok = await(&pfull[2 + cur], parity))) break;
                        tc_fence_after();
                        accumulate(1, 2 + cur, k == 0);
                    }
                    mma_commit(&empty[out.s]);
                    out.next();
                    in.next();
                }
            } else {
                constexpr int AHEAD = C::NBUF;
                for (int k = 0; ok && k < AHEAD && k < n; ++k)
                    if ((ok = tile_ready())) {
                        scores(0, k);
                        in.next();
                    }
                int buf = 0;
                unsigned parity = 0;
                for (int k = 0; ok && k < n; ++k) {
                    if (!(ok = await(&pfull[buf], parity))) break;
                    tc_fence_after();
                    accumulate(0, buf, k == 0);
                    mma_commit(&empty[out.s]);
                    out.next();
                    if (k + AHEAD < n && (ok = tile_ready())) {
                        scores(0, buf);
                        in.next();
                    }
                    if (++buf == AHEAD) buf = 0, parity ^= 1;
                }
            }
            mma_commit(accfull);
            mbar_wait_bounded(accfull, 0, a.timeout_ns);  // before the tensor memory is freed
        }
        __syncwarp();
    } else if (warp < C::CWARPS) {
        // ---- weights ------------------------------------------------------------------
        const bool live = r0 + xt * XR + quad * 32 < nx;  // else nothing is read of its rows
        const bool unit_live = r0 + xt * XR < nx;         // else it has no products
        const uint32_t lanes = uint32_t(quad * 32) << 16;
        const float c2 = a.scale * ATTN_LOG2E;
        const float2 c22 = make_float2(c2, c2);
        const float2 nx2 = make_float2(-px, -px), ny2 = make_float2(-py, -py),
                     nz2 = make_float2(-pz, -pz);
        float nlse = -INFINITY, ndel = 0.0f;  // DQ: -lse in base 2, -delta
        if (MODE == ATTN_DQ && row < nx) {
            const int64_t at = (int64_t(b) * a.H + head) * a.Lq + row;
            nlse = -a.lse2[at];
            ndel = -a.delta[at];
        }
        float mc = -INFINITY;                        // FWD: the row's maximum, base 2
        float2 l2 = make_float2(0.0f, 0.0f);         // FWD: the row's sum
        LongSum wa, we, wd, wp;                      // DQ: the slope's sums
        float *rd = rowdata + unit * 8 * XR + quad * 32 + lane;
        bool ok = true;
        int s = FWD ? 0 : unit, sbuf = unit;  // stage; BWD: score buffer
        unsigned phase = 0, sphase = 0;
        TileWalk at = walk(FWD ? 0 : unit);
        for (int k = FWD ? 0 : unit; k < n; k += FWD ? 1 : 2, s += FWD ? 1 : 2) {
            if (s >= STAGES) s -= STAGES, phase ^= 1;
            if (BWD && sbuf >= C::NBUF) sbuf -= C::NBUF, sphase ^= 1;
            const int buf = FWD ? 2 * unit + (k & 1) : sbuf;
            if (unit_live && !(ok = wait(&sfull[buf], FWD ? unsigned((k >> 1) & 1) : sphase)))
                break;
            sbuf += 2;
            if (COLS && !(ok = wait(&full[s], phase))) break;
            tc_fence_after();
            const float *cd = coldata + s * C::COLF + 32 * half;
            const uint32_t sb = tmem + lanes + buf * C::BUF + 32 * half;
            const int valid = ny - at.y - 32 * half;  // columns of this half, if < 32
            at.next(FWD ? 1 : 2);
            const bool direct = BIAS && coldata[s * C::COLF + 5 * YR] != 0.0f;
            const float nb = BIAS ? coldata[s * C::COLF + 5 * YR + 1] : 0.0f;
            const float2 nb2 = make_float2(nb, nb);
            if (FWD && live) {
                uint32_t r[32];
                tmem_ld32(sb, r);
                tmem_wait_ld();
                if (direct)
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
                float *mx = rd + (k & 1) * 2 * XR;
                mx[half * XR] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(&mxbar[unit * 4 + quad]);
                if (!(ok = wait(&mxbar[unit * 4 + quad], unsigned(k & 1)))) break;
                m = fmaxf(m, mx[(half ^ 1) * XR]) * c2;
                // The base of the exponents follows the maximum only when it
                // grew by more than 2^16 (the weights stay below 65536, far from
                // float32's and bfloat16's ends): the accumulator is seldom
                // rescaled.
                const bool need = m > mc + 16.0f;
                if (__any_sync(0xffffffffu, need)) {
                    const float mn = need ? m : mc;
                    const float f = mn == -INFINITY ? 1.0f : ex2(mc - mn);
                    mc = mn;
                    l2.x *= f;
                    l2.y *= f;
                    if (k > 0) {
                        // the sums of the tile before come ahead of the next
                        // tile's scores
                        if (!(ok = wait(&sfull[buf ^ 1], unsigned(((k + 1) >> 1) & 1)))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < DP / 2; c += 8) {
                            const uint32_t at =
                                tmem + lanes + C::ACC + unit * DP + half * (DP / 2) + c;
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
                    tmem_st8(sb + 16 * h + 8, lo);
                }
            } else if (BWD && live) {
                auto weights = [&](auto tail_, auto direct_) {
                    constexpr bool TAIL = decltype(tail_)::value, DIRECT = decltype(direct_)::value;
                    float2 ta = make_float2(0.0f, 0.0f), te = ta, td = ta, tp = ta;  // of the tile
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t r[16], g[16], p[8], plo[8], q[8], qlo[8];
                        tmem_ld16(sb + 16 * h, r);
                        tmem_ld16(sb + YR + 16 * h, g);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            float2 d[2];
                            if (DIRECT) dist4(cd, 16 * h + c, nx2, ny2, nz2, d[0], d[1]);
                            float4 cl, cdl;
                            if (DKV) {
                                cl = *reinterpret_cast<const float4 *>(cd + 3 * YR + 16 * h + c);
                                cdl = *reinterpret_cast<const float4 *>(cd + 4 * YR + 16 * h + c);
                            }
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int i = c + 2 * e, col = 16 * h + i;
                                float2 u = pair(r, i);
                                if (DIRECT) u = __ffma2_rn(d[e], nb2, u);
                                float2 nl = make_float2(nlse, nlse), nd = make_float2(ndel, ndel);
                                if (DKV) {
                                    nl = e == 0 ? make_float2(cl.x, cl.y) : make_float2(cl.z, cl.w);
                                    nd = e == 0 ? make_float2(cdl.x, cdl.y)
                                                : make_float2(cdl.z, cdl.w);
                                }
                                u = __ffma2_rn(u, c22, nl);
                                u.x = ex2(u.x);
                                u.y = ex2(u.y);
                                float2 ds = __fmul2_rn(u, __fadd2_rn(pair(g, i), nd));
                                if (TAIL) {
                                    if (col >= valid) u.x = ds.x = 0.0f;
                                    if (col + 1 >= valid) u.y = ds.y = 0.0f;
                                }
                                if (MODE == ATTN_DQ && DIRECT && sums) {
                                    td = __fadd2_rn(td, ds);
                                    tp = __fadd2_rn(tp, u);
                                    ta = __ffma2_rn(ds, d[e], ta);
                                    te = __ffma2_rn(u, d[e], te);
                                }
                                if (DKV) split_bf16(u, p[i / 2], plo[i / 2]);
                                split_bf16(ds, q[i / 2], qlo[i / 2]);
                            }
                        }
                        if (DKV) {
                            tmem_st8(sb + 16 * h, p);
                            tmem_st8(sb + 16 * h + 8, plo);
                        }
                        tmem_st8(sb + YR + 16 * h, q);
                        tmem_st8(sb + YR + 16 * h + 8, qlo);
                    }
                    if (MODE == ATTN_DQ && DIRECT && sums) {
                        wd.add(td.x + td.y);
                        wa.add(ta.x + ta.y);
                        we.add(te.x + te.y);
                        wp.add(tp.x + tp.y);
                    }
                };
                constexpr std::true_type yes{};
                constexpr std::false_type no{};
                constexpr std::integral_constant<bool, BIAS> differences{};
                if (valid < 32) {
                    if (BIAS && direct)
                        weights(yes, differences);
                    else
                        weights(yes, no);
                } else {
                    if (BIAS && direct)
                        weights(no, differences);
                    else
                        weights(no, no);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (unit_live) mbar_arrive(&pfull[buf]);
                if (COLS) mbar_arrive(&empty[s]);
            }
        }
        const int64_t hrow = (int64_t(b) * a.H + head) * a.Lq + row;  // FWD, DQ
        const int64_t hrows = int64_t(a.B) * a.H * a.Lq;
        const float one = FWD ? 1.0f : attn_ds_factor(nk);
        if (MODE == ATTN_DQ && BIAS) {
            // the sums of a row's four groups, in the exchange buffer as [unit][half][4]
            if (sums) {
                rd[(half * 4) * XR] = wa.value();
                rd[(half * 4 + 1) * XR] = we.value();
                rd[(half * 4 + 2) * XR] = wd.value();
                rd[(half * 4 + 3) * XR] = wp.value();
            }
            named_barrier_sync(1, C::CWARPS * 32);
            if (sums && unit == 0 && half == 0) {
                float t[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    t[e] = (rd[e * XR] + rd[(4 + e) * XR]) + (rd[(8 + e) * XR] + rd[(12 + e) * XR]);
                    t[e] = row < nx ? one * t[e] : 0.0f;
                }
                put_slope_sums(a, t, split, hrow, row < LX, quad, lane, rowdata + 16 * XR, bid);
            }
        }
        float l = l2.x + l2.y;
        if (FWD) {  // the row's sum over both halves
            rd[(4 + half) * XR] = l;
            named_barrier_sync(1, C::CWARPS * 32);
            l = rd[4 * XR] + rd[5 * XR];
        }
        const bool any = row < nx && (!FWD || ny > 0);
        if (FWD && row < LX && half == 0) {
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
        // the groups of a row share its accumulators' columns
        const bool have = n > 0 && ok && unit_live;
        constexpr int CHUNKS = (FWD ? 1 : C::NACC) * DP / 32;
        for (int ch = FWD ? half : 2 * unit + half; ch < CHUNKS; ch += FWD ? 2 : 4) {
            const int acc = ch / (DP / 32), c0 = (ch % (DP / 32)) * 32;
            uint32_t r[32];
            float v[32];
            __syncwarp();
            if (have) {
                tmem_ld32(tmem + lanes + C::ACC + (FWD ? unit * DP : 0) + ch * 32, r);
                tmem_wait_ld();
            }
            const float f = FWD ? (a.nsplit > 1 ? 1.0f : 1.0f / l)
                            : acc != 0 ? 1.0f : a.nsplit > 1 ? one : one * a.scale;
#pragma unroll
            for (int e = 0; e < 32; ++e)
                v[e] = have && any ? __uint_as_float(r[e]) * f : 0.0f;
            if (row >= LX) {
                // past the array's end: nothing to store
            } else if (a.nsplit > 1) {
                store_row32(a.part + ((int64_t(acc) * a.nsplit + split) * rows + orow) * a.D + c0,
                            v, c0, a.D);
            } else {
                void *o = FWD ? a.out : MODE == ATTN_DQ ? a.dq : acc ? a.dv : a.dk;
                store_row32(static_cast<bf16 *>(o) + orow * a.D + c0, v, c0, a.D);
                if (FWD && a.low != nullptr) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = rest<bf16>(v[e]);
                    store_row32(static_cast<bf16 *>(a.low) + orow * a.D + c0, v, c0, a.D);
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == C::CWARPS + 1) tmem_free(tmem, C::COLS);
}

template <int DP, bool BIAS>
__global__ void __launch_bounds__(Cfg<ATTN_FWD, DP>::THREADS, 1)
attn_tc_forward_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnMaps maps,
                       const bool withhold) {
    attn_tc_pass<ATTN_FWD, DP, BIAS>(a, maps, withhold, blockIdx.x);
}

// Both backward passes in one launch, the keys' first: their blocks are fewer
// and longer, and the queries' fill what they leave of the GPU.
template <int DP, bool BIAS>
__global__ void __launch_bounds__(Cfg<ATTN_DQ, DP>::THREADS, 1)
attn_tc_backward_kernel(const __grid_constant__ AttnArgs dkv, const __grid_constant__ AttnArgs dq,
                        const __grid_constant__ AttnMaps maps, const unsigned first,
                        const bool withhold) {
    if (blockIdx.x < first)
        attn_tc_pass<ATTN_DKV, DP, BIAS>(dkv, maps, withhold, blockIdx.x);
    else
        attn_tc_pass<ATTN_DQ, DP, BIAS>(dq, maps, withhold, blockIdx.x - first);
}

bool tc_maps(const AttnArgs &a, bool backward, AttnMaps &m) {
    const int64_t gs[3] = {int64_t(a.Lq) * a.H * a.D, int64_t(a.H) * a.D, a.D};
    return make_map(&m.q, a.q, a.qs, a.B, a.Lq, a.H, a.D) &&
           make_map(&m.k, a.k, a.ks, a.B, a.Lk, a.Hkv, a.D) &&
           make_map(&m.v, a.v, a.vs, a.B, a.Lk, a.Hkv, a.D) &&
           (!backward || make_map(&m.go, a.go, gs, a.B, a.Lq, a.H, a.D));
}

bool withheld() { return (debug_stall() & PC_STALL_ATTENTION) != 0; }

template <int DP, bool BIAS>
cudaError_t tc_forward(const AttnArgs &a, unsigned blocks, cudaStream_t st) {
    using C = Cfg<ATTN_FWD, DP>;
    AttnMaps m{};
    if (!tc_maps(a, false, m)) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        allow_smem(attn_tc_forward_kernel<DP, BIAS>, int(C::SMEM), a.device, done);
    if (e != cudaSuccess) return e;
    attn_tc_forward_kernel<DP, BIAS><<<blocks, C::THREADS, C::SMEM, st>>>(a, m, withheld());
    return cudaGetLastError();
}

template <int DP, bool BIAS>
cudaError_t tc_backward(const AttnArgs &dkv, unsigned first, const AttnArgs &dq, unsigned second,
                        cudaStream_t st) {
    using C = Cfg<ATTN_DQ, DP>;
    constexpr size_t other = Cfg<ATTN_DKV, DP>::SMEM;
    constexpr int smem = int(C::SMEM > other ? C::SMEM : other);
    static_assert(C::THREADS == Cfg<ATTN_DKV, DP>::THREADS, "one launch");
    AttnMaps m{};
    if (!tc_maps(dq, true, m)) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(attn_tc_backward_kernel<DP, BIAS>, smem, dq.device, done);
    if (e != cudaSuccess) return e;
    attn_tc_backward_kernel<DP, BIAS>
        <<<first + second, C::THREADS, smem, st>>>(dkv, dq, m, first, withheld());
    return cudaGetLastError();
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
    if (mode == ATTN_FWD) return aligned(a.out) && aligned(a.low);
    return aligned(a.go) && aligned(a.dq) && aligned(a.dk) && aligned(a.dv);
}

cudaError_t launch_attn_tc_forward(const AttnArgs &a, unsigned blocks, cudaStream_t st) {
    if (a.D <= 64)
        return a.slopes ? tc_forward<64, true>(a, blocks, st) : tc_forward<64, false>(a, blocks, st);
    return a.slopes ? tc_forward<128, true>(a, blocks, st) : tc_forward<128, false>(a, blocks, st);
}

cudaError_t launch_attn_tc_backward(const AttnArgs &dkv, unsigned first, const AttnArgs &dq,
                                    unsigned second, cudaStream_t st) {
    if (dq.D <= 64)
        return dq.slopes ? tc_backward<64, true>(dkv, first, dq, second, st)
                         : tc_backward<64, false>(dkv, first, dq, second, st);
    return dq.slopes ? tc_backward<128, true>(dkv, first, dq, second, st)
                     : tc_backward<128, false>(dkv, first, dq, second, st);
}

}  // namespace pcn
