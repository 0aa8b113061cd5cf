// pc_attn_tc32.cu -- the attention passes of pc_attn.cuh on the tensor cores,
// for float32.
//
// A float32 is the sum of three bfloat16 (8 bits each), and a product of two
// such sums is six products of bfloat16 to about 2^-24: low x high, high x low,
// middle x middle, middle x high, high x middle, high x high.  A first kernel
// writes the three parts of q, k, v (and dout) as three arrays, rows padded to
// 8 channels; the passes then read tiles of them by tensor maps, whatever the
// strides and the number of channels were.  P and dS are split by the threads
// that compute them.
//
// The tensor cores add into their float32 accumulators with truncation (a
// quarter to three quarters of a unit a step are lost, measured), which over a
// long chain is a bias.  So a chain is one tile long, the small products come
// first in it, and the tiles are added up in registers, rounded to nearest.
//
// A block keeps 128 rows and walks over the other side in tiles of 64; eight
// warps compute weights, a thread half a row; two score buffers, so that the
// products of one tile run under the weights of another.  The parts of more
// than 64 channels leave room for less in the backward passes: 64 rows (of
// products of 128: half the rate), one stage and one score buffer.  The bias
// is formed from coordinates' differences.
//
// Bound: the products, six times those of bfloat16.  Measured, 4 x 1021 tokens,
// 6 heads of 48 padded to 64: forward 60 us, both backward passes 162 us (258
// and 930 us in float32 instructions); 2 x 2048, 8 heads of 96: 227 us forward.
// Short clouds are the other way round: 32 x 64 tokens, 8 heads of 64, forward 21 us
// and 15 in float32 instructions; 4 x 128 of 64 15 and 13, of 128 22 and 17.
//
// Lengths, waits and their end, and the allocation of tensor memory, as in
// pc_attn_tc.cu.
#include "pc_attn_tc.cuh"
#include "pointcloud.h"

namespace pcn {
namespace {

struct SplitMaps {
    CUtensorMap q, k, v, go;  // [3 B, L, heads, Dp] bfloat16
};

template <int MODE, int DP>
struct Cfg32 {
    static constexpr bool BWD = MODE != ATTN_FWD, WIDE = DP == 128;
    static constexpr int CWARPS = 8, THREADS = 32 * (CWARPS + 4);
    static constexpr int ROWS = BWD && WIDE ? 64 : XR;  // rows kept
    static constexpr int NB = BWD && WIDE ? 1 : 2;      // score buffers
    static constexpr int STAGES = WIDE ? (BWD ? 1 : 2) : MODE == ATTN_DKV ? 2 : 4;
    // Tensor memory: score buffers (S, dP and room for the parts of P and dS),
    // the tile's sums, and where there is room the rows kept.
    static constexpr int BUF = MODE == ATTN_FWD ? 96 : MODE == ATTN_DQ ? 128 : 192;
    static constexpr int NACC = MODE == ATTN_DKV ? 2 : 1;
    static constexpr int ACC = NB * BUF, XCOL = ACC + NACC * DP;
    static constexpr int XCOLS = 3 * DP / 2;            // three parts of one array
    static constexpr bool X_TMEM = MODE == ATTN_FWD || (MODE == ATTN_DQ && !WIDE);
    static_assert(XCOL + (X_TMEM ? (BWD ? 2 : 1) * XCOLS : 0) <= 512, "tensor memory");
    static constexpr int XP = ROWS * DP * 2, YP = YR * DP * 2;  // bytes of a part
    static constexpr size_t XSMEM = X_TMEM ? 0 : 6 * XP;
    static constexpr int STAGE = 6 * YP;
    static constexpr int COLF = 5 * YR + 4;
    static constexpr int ROWF = 6 * XR + 4;
    static constexpr size_t SMEM =
        1024 + XSMEM + size_t(STAGES) * (STAGE + COLF * 4) + ROWF * 4 + 512;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(SMEM > 114 * 1024, "one block a SM: none waits for tensor memory");
};

// The six products, the smallest first: part of the one, part of the other.
__device__ constexpr int PAIR_A[6] = {2, 0, 1, 1, 0, 0};
__device__ constexpr int PAIR_B[6] = {0, 2, 1, 0, 1, 0};

// Two numbers as three pairs of bfloat16.
__device__ __forceinline__ void split3(float2 v, uint32_t &h, uint32_t &m, uint32_t &l) {
    h = pack_bf16(v.x, v.y);
    float2 t = unpack_bf16(h);
    v = make_float2(v.x - t.x, v.y - t.y);
    m = pack_bf16(v.x, v.y);
    t = unpack_bf16(m);
    l = pack_bf16(v.x - t.x, v.y - t.y);
}

// 32 channels of a row, any D and alignment.
__device__ __forceinline__ void store_row(float *p, const float (&v)[32], int c0, int D) {
    if (D % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c0 + 4 * i < D) Vec<float, 4>::store(p + 4 * i, v + 4 * i);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (c0 + i < D) p[i] = v[i];
    }
}

// One pass of block `bid`.
template <int MODE, int DP, bool BIAS>
__device__ __forceinline__ void attn_tc32_pass(const AttnArgs &a, const SplitMaps &maps,
                                               const AttnSplit &split_ptr, const bool withhold,
                                               const unsigned bid) {
    using C = Cfg32<MODE, DP>;
    constexpr bool BWD = C::BWD, FWD = !BWD, DKV = MODE == ATTN_DKV;
    constexpr int STAGES = C::STAGES;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *X = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char *Y = X + C::XSMEM;  // stage s: three parts of Y1, of Y2
    float *coldata = reinterpret_cast<float *>(Y + size_t(STAGES) * C::STAGE);
    float *rowdata = coldata + STAGES * C::COLF;  // [6][XR]
    uint64_t *full = reinterpret_cast<uint64_t *>(rowdata + C::ROWF);
    uint64_t *empty = full + STAGES, *fixed = empty + STAGES, *sfull = fixed + STAGES;
    uint64_t *pfull = sfull + 2, *tfull = pfull + 2, *xfull = tfull + 1;
    uint64_t *accdone = xfull + 1, *mxbar = accdone + 1;  // mxbar: [quad]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mxbar + 4);
    volatile int *stop = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int LX = DKV ? a.Lk : a.Lq, LY = DKV ? a.Lq : a.Lk;
    const int NH = DKV ? a.Hkv : a.H;
    const int G = a.H / a.Hkv;
    const int ntile = (LX + C::ROWS - 1) / C::ROWS;
    int64_t idx = bid;
    const int split = int(idx % a.nsplit);
    idx /= a.nsplit;
    const int tile = int(idx % ntile);
    idx /= ntile;
    const int head = int(idx % NH), b = int(idx / NH);
    const int nq = attn_len(a.qlen, b, a.Lq), nk = attn_len(a.rlen, b, a.Lk);
    const int nx = uniform(DKV ? nk : nq), ny = uniform(DKV ? nq : nk);
    const int r0 = tile * C::ROWS;
    const int hk = DKV ? head : head / G;
    const int nyt = (ny + YR - 1) / YR;
    const int64_t items = nx > r0 ? int64_t(nyt) * (DKV ? G : 1) : 0;
    const int64_t it0 = items * split / a.nsplit;
    const int n = uniform(int(items * (split + 1) / a.nsplit - it0));
    const float *xpos = DKV ? a.rxyz : a.qxyz, *ypos = DKV ? a.qxyz : a.rxyz;
    const bool ragged = ny < LY && ny % YR != 0;
    const int quad = warp % 4, half = (warp / 4) % 2;
    // (lanes of products past the rows kept have no row)
    const int row = quad * 32 < C::ROWS ? r0 + quad * 32 + lane : 0x7fffffff;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 2);
            mbar_init(&empty[s], 1 + C::CWARPS);
            mbar_init(&fixed[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sfull[s], 1);
            mbar_init(&pfull[s], C::CWARPS);
        }
        mbar_init(tfull, 1);
        mbar_init(xfull, 1);
        mbar_init(accdone, 1);
        for (int s = 0; s < 4; ++s) mbar_init(&mxbar[s], 2);
        *stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == C::CWARPS + 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(int(*tmem_slot));
    const uint32_t lanes = uint32_t(quad * 32) << 16;
    if (C::X_TMEM && n > 0 && warp < C::CWARPS) {
        // the parts of q (and dout), half the channels each
#pragma unroll
        for (int t = 0; t < (BWD ? 2 : 1); ++t)
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                const bf16 *src = (t == 0 ? split_ptr.q : split_ptr.go) +
                                  ((int64_t(p * a.B + b) * a.Lq + row) * a.H + head) *
                                      split_ptr.Dp;
#pragma unroll
                for (int c = 0; c < DP / 32; ++c) {
                    uint32_t r[8];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int ch = half * (DP / 2) + 16 * c + 8 * e;
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (row < nx && ch < split_ptr.Dp)
                            v = *reinterpret_cast<const uint4 *>(src + ch);
                        r[4 * e] = v.x, r[4 * e + 1] = v.y, r[4 * e + 2] = v.z, r[4 * e + 3] = v.w;
                    }
                    tmem_st8(tmem + lanes + C::XCOL + t * C::XCOLS + p * (DP / 2) + half * (DP / 4) +
                                 8 * c,
                             r);
                }
            }
        tmem_wait_st();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

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
            mbar_arrive_expect_tx(xfull, 6 * C::XP);
            for (int p = 0; p < 3; ++p)
                for (int c = 0; c < DP / 64; ++c)
                    for (int h = 0; h < C::ROWS / YR; ++h) {
                        unsigned char *at =
                            X + p * C::XP + c * C::ROWS * 128 + h * YR * 128;
                        tma_load_4d(at, DKV ? &maps.k : &maps.q, 64 * c, r0 + YR * h, head,
                                    p * a.B + b, xfull);
                        tma_load_4d(at + 3 * C::XP, DKV ? &maps.v : &maps.go, 64 * c, r0 + YR * h,
                                    head, p * a.B + b, xfull);
                    }
        }
        TileWalk late = walk(0);
        auto fix = [&](int k) {
            const int valid = ny - late.y, s = k % STAGES;
            late.next();
            if (!ragged || valid >= YR) return true;
            if (!wait(&full[s], unsigned((k / STAGES) & 1))) return false;
            uint4 *y = reinterpret_cast<uint4 *>(Y + size_t(s) * C::STAGE);
            for (int p = 0; p < 6; ++p)
                if (BWD ? DKV || p < 3 : p >= 3)
                    for (int c = 0; c < DP / 64; ++c)
                        for (int i = valid * 8 + lane; i < YR * 8; i += 32)
                            y[p * (C::YP / 16) + c * YR * 8 + i] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&fixed[s]);
            return true;
        };
        int issued = 0;
        bool ok = true;
        TileWalk at = walk(0);
        // (as in pc_attn_tc.cu; one score buffer does not look a tile ahead)
        constexpr int LAG = C::NB == 1 ? STAGES - 1 : STAGES > 3 ? 2 : STAGES - 2;
        for (int k = 0; ok && k < n; ++k, at.next()) {
            const int s = k % STAGES;
            if (k >= STAGES && !wait(&empty[s], unsigned((k / STAGES - 1) & 1))) break;
            if (withhold && bid == 0) break;
            if (elect_one()) {
                const int hy = DKV ? at.h : hk;
                mbar_arrive_expect_tx(&full[s], 6 * C::YP);
                unsigned char *y = Y + size_t(s) * C::STAGE;
                for (int p = 0; p < 3; ++p)
                    for (int c = 0; c < DP / 64; ++c) {
                        tma_load_4d(y + p * C::YP + c * YR * 128, DKV ? &maps.q : &maps.k, 64 * c,
                                    at.y, hy, p * a.B + b, &full[s]);
                        tma_load_4d(y + (3 + p) * C::YP + c * YR * 128, DKV ? &maps.go : &maps.v,
                                    64 * c, at.y, hy, p * a.B + b, &full[s]);
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
    } else if (warp >= C::CWARPS + 2) {
        // ---- positions: two warps, every other tile each ------------------------------
        const int first = warp - (C::CWARPS + 2);
        TileWalk at = walk(first);
        float nxt[2][5], slope_nxt = 0.0f;
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
            at.next(2);
            if (k + 2 < n) fetch();
            float *cd = coldata + s * C::COLF;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 5; ++e)
                    if (e < 3 ? BIAS : DKV) cd[e * YR + lane + 32 * i] = cur[i][e];
            if (lane == 0) cd[5 * YR] = -slope / a.scale;
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
        }
    } else if (warp == C::CWARPS + 1) {
        // ---- products, issued by one thread -------------------------------------------
        if (elect_one()) {
            const uint32_t x0 = smem_operand(smem_u32(X)), yk = smem_operand(smem_u32(Y));
            const uint32_t yr = smem_operand(smem_u32(Y), YR * 128);
            int in = 0, out = 0;  // stages of the tiles whose scores, whose sums come next
            unsigned phase = 0, fixes = 0;
            TileWalk at = walk(0);
            auto await = [&](uint64_t *bar, unsigned parity) {
                const WaitResult w = mbar_wait_or_stop(bar, parity, stop, a.timeout_ns);
                if (w == WAIT_TIMEOUT) {
                    *stop = 1;
                    raise_status(a.status, PC_ERR_DEVICE_TIMEOUT);
                }
                return w == WAIT_OK;
            };
            auto scores = [&](int buf) {
                if (!await(&full[in], phase)) return false;
                const int valid = ny - at.y;
                at.next();
                if (ragged && valid < YR) {
                    const unsigned parity = (fixes >> in) & 1;
                    fixes ^= 1u << in;
                    if (!await(&fixed[in], parity)) return false;
                }
                constexpr uint32_t id = mma_idesc(YR, false);
                const uint32_t d = tmem + buf * C::BUF, y = yk + in * (C::STAGE / 16);
#pragma unroll
                for (int t = 0; t < (BWD ? 2 : 1); ++t)
#pragma unroll
                    for (int p = 0; p < 6; ++p)
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i) {
                            const uint32_t yo = y + (3 * t + PAIR_B[p]) * (C::YP / 16) +
                                                (i / 4) * (YR * 128 / 16) + 2 * (i % 4);
                            if (C::X_TMEM)
                                mma_ts<SMEM_128B>(d + t * YR,
                                                  tmem + C::XCOL + C::XCOLS * t +
                                                      (DP / 2) * PAIR_A[p] + 8 * i,
                                                  yo, id, p > 0 || i > 0);
                            else
                                mma_ss<SMEM_128B>(d + t * YR,
                                                  x0 + (3 * t + PAIR_A[p]) * (C::XP / 16) +
                                                      (i / 4) * (C::ROWS * 128 / 16) + 2 * (i % 4),
                                                  yo, id, p > 0 || i > 0);
                        }
                mma_commit(&sfull[buf]);
                if (++in == STAGES) in = 0, phase ^= 1;
                return true;
            };
            // where the parts of the weights of step i lie in a buffer
            auto part = [](bool ds, int p, int i) -> uint32_t {
                if (MODE == ATTN_FWD) return p < 2 ? 16 * i + 8 * p : 64 + 8 * i;
                if (MODE == ATTN_DQ) return p < 2 ? 64 + 16 * i + 8 * p : 16 * i;
                return p < 2 ? (ds ? 64 : 0) + 16 * i + 8 * p : (ds ? 160 : 128) + 8 * i;
            };
            auto accumulate = [&](int buf) {
                constexpr uint32_t id = mma_idesc(DP, true);
                const uint32_t d = tmem + buf * C::BUF, y = yr + out * (C::STAGE / 16);
#pragma unroll
                for (int t = 0; t < C::NACC; ++t) {
                    const bool ds = BWD && t == 0;  // dS Y1; else P Y2
#pragma unroll
                    for (int p = 0; p < 6; ++p)
#pragma unroll
                        for (int i = 0; i < YR / 16; ++i)
                            mma_ts<SMEM_128B>(tmem + C::ACC + t * DP, d + part(ds, PAIR_A[p], i),
                                              y + ((ds ? 0 : 3) + PAIR_B[p]) * (C::YP / 16) +
                                                  i * (16 * 128 / 16),
                                              id, p > 0 || i > 0);
                }
                mma_commit(tfull);
                mma_commit(&empty[out]);
                if (++out == STAGES) out = 0;
            };
            bool ok = n > 0 && (C::X_TMEM || await(xfull, 0)) && scores(0);
            for (int k = 0; ok && k < n; ++k) {
                // Products run in the order of their issue: a buffer is free again
                // once the sums that read it were issued.
                const int buf = C::NB == 2 ? k & 1 : 0;
                if (C::NB == 2 && k + 1 < n && !(ok = scores(buf ^ 1))) break;
                if (!(ok = await(&pfull[buf], unsigned(C::NB == 2 ? k >> 1 : k) & 1))) break;
                tc_fence_after();
                accumulate(buf);
                if (C::NB == 1 && k + 1 < n) ok = scores(0);
            }
            mma_commit(accdone);
            mbar_wait_bounded(accdone, 0, a.timeout_ns);  // before the tensor memory is freed
        }
        __syncwarp();
    } else {
        // ---- weights ------------------------------------------------------------------
        const bool live = quad * 32 < C::ROWS && r0 + quad * 32 < nx;
        const float c2 = a.scale * ATTN_LOG2E;
        const float2 c22 = make_float2(c2, c2);
        float px = 0.0f, py = 0.0f, pz = 0.0f;
        if (BIAS && row < nx) {
            const float *p = xpos + (int64_t(b) * LX + row) * 3;
            px = p[0], py = p[1], pz = p[2];
        }
        const float2 nx2 = make_float2(-px, -px), ny2 = make_float2(-py, -py),
                     nz2 = make_float2(-pz, -pz);
        float nlse = -INFINITY, ndel = 0.0f;
        if (MODE == ATTN_DQ && row < nx) {
            const int64_t at = (int64_t(b) * a.H + head) * a.Lq + row;
            nlse = -a.lse2[at];
            ndel = -a.delta[at];
        }
        float mc = -INFINITY;
        float2 l2 = make_float2(0.0f, 0.0f);
        LongSum wa, we, wd, wp;  // DQ: the slope's sums
        const bool sums = MODE == ATTN_DQ && BIAS && a.rowsum != nullptr;
        float *rd = rowdata + quad * 32 + lane;
        float acc[C::NACC][DP / 2];
#pragma unroll
        for (int t = 0; t < C::NACC; ++t)
#pragma unroll
            for (int e = 0; e < DP / 2; ++e) acc[t][e] = 0.0f;
        // the sums of tile k into the registers
        auto drain = [&](int k) {
            if (!wait(tfull, unsigned(k & 1))) return false;
            tc_fence_after();
            if (live)
#pragma unroll
                for (int t = 0; t < C::NACC; ++t)
#pragma unroll
                    for (int c = 0; c < DP / 64; ++c) {
                        uint32_t r[32];
                        tmem_ld32(tmem + lanes + C::ACC + t * DP + half * (DP / 2) + 32 * c, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) acc[t][32 * c + e] += __uint_as_float(r[e]);
                    }
            return true;
        };
        bool ok = true;
        int s = 0;
        unsigned phase = 0;
        TileWalk at = walk(0);
        for (int k = 0; k < n; ++k) {
            const int buf = C::NB == 2 ? k & 1 : 0;
            if (!(ok = wait(&sfull[buf], unsigned(C::NB == 2 ? k >> 1 : k) & 1))) break;
            if (!(ok = wait(&full[s], phase))) break;
            tc_fence_after();
            const float *cd = coldata + s * C::COLF + 32 * half;
            const uint32_t sb = tmem + lanes + buf * C::BUF;
            const int valid = ny - at.y - 32 * half;
            at.next();
            const float nb = BIAS ? coldata[s * C::COLF + 5 * YR] : 0.0f;
            const float2 nb2 = make_float2(nb, nb);
            float f = 1.0f;  // FWD: what the base's change does to the sums so far
            if (FWD && live) {
                uint32_t r[32];
                tmem_ld32(sb + 32 * half, r);
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
                float *mx = rd + (k & 1) * 2 * XR;
                mx[half * XR] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(&mxbar[quad]);
                if (!(ok = wait(&mxbar[quad], unsigned(k & 1)))) break;
                m = fmaxf(m, mx[(half ^ 1) * XR]) * c2;
                if (m > mc + 16.0f) {  // as in pc_attn_tc.cu
                    f = ex2(mc - m);
                    mc = m;
                    l2.x *= f;
                    l2.y *= f;
                }
                const float mb = mc == -INFINITY ? 0.0f : -mc;
                const float2 mb2 = make_float2(mb, mb);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[3][8];
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        float2 t = __ffma2_rn(pair(r, 16 * h + c), c22, mb2);
                        t.x = ex2(t.x);
                        t.y = ex2(t.y);
                        l2 = __fadd2_rn(l2, t);
                        split3(t, p[0][c / 2], p[1][c / 2], p[2][c / 2]);
                    }
                    const int i = 2 * half + h;
                    tmem_st8(sb + 16 * i, p[0]);
                    tmem_st8(sb + 16 * i + 8, p[1]);
                    tmem_st8(sb + 64 + 8 * i, p[2]);
                }
            } else if (BWD && live) {
                float2 ta = make_float2(0.0f, 0.0f), te = ta, td = ta, tp = ta;  // of the tile
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = 2 * half + h;
                    uint32_t r[16], g[16], p[3][8], q[3][8];
                    tmem_ld16(sb + 16 * i, r);
                    tmem_ld16(sb + YR + 16 * i, g);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        float2 d[2];
                        if (BIAS) dist4(cd, 16 * h + c, nx2, ny2, nz2, d[0], d[1]);
                        float4 cl, cdl;
                        if (DKV) {
                            cl = *reinterpret_cast<const float4 *>(cd + 3 * YR + 16 * h + c);
                            cdl = *reinterpret_cast<const float4 *>(cd + 4 * YR + 16 * h + c);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = c + 2 * e, col = 16 * h + j;
                            float2 u = pair(r, j);
                            if (BIAS) u = __ffma2_rn(d[e], nb2, u);
                            float2 nl = make_float2(nlse, nlse), nd = make_float2(ndel, ndel);
                            if (DKV) {
                                nl = e == 0 ? make_float2(cl.x, cl.y) : make_float2(cl.z, cl.w);
                                nd = e == 0 ? make_float2(cdl.x, cdl.y) : make_float2(cdl.z, cdl.w);
                            }
                            u = __ffma2_rn(u, c22, nl);
                            u.x = ex2(u.x);
                            u.y = ex2(u.y);
                            float2 ds = __fmul2_rn(u, __fadd2_rn(pair(g, j), nd));
                            if (col >= valid) u.x = ds.x = 0.0f;
                            if (col + 1 >= valid) u.y = ds.y = 0.0f;
                            if (sums) {
                                td = __fadd2_rn(td, ds);
                                tp = __fadd2_rn(tp, u);
                                ta = __ffma2_rn(ds, d[e], ta);
                                te = __ffma2_rn(u, d[e], te);
                            }
                            if (DKV) split3(u, p[0][j / 2], p[1][j / 2], p[2][j / 2]);
                            split3(ds, q[0][j / 2], q[1][j / 2], q[2][j / 2]);
                        }
                    }
                    if (DKV) {
                        tmem_st8(sb + 16 * i, p[0]);
                        tmem_st8(sb + 16 * i + 8, p[1]);
                        tmem_st8(sb + 128 + 8 * i, p[2]);
                    }
                    tmem_st8(sb + 64 + 16 * i, q[0]);
                    tmem_st8(sb + 64 + 16 * i + 8, q[1]);
                    tmem_st8(sb + (DKV ? 160 + 8 * i : 16 * i), q[2]);
                }
                if (sums) {
                    wd.add(td.x + td.y);
                    wa.add(ta.x + ta.y);
                    we.add(te.x + te.y);
                    wp.add(tp.x + tp.y);
                }
            }
            // the sums of the tile before leave tensor memory before this
            // tile's come
            if (k > 0 && !(ok = drain(k - 1))) break;
            if (FWD && f != 1.0f)
#pragma unroll
                for (int e = 0; e < DP / 2; ++e) acc[0][e] *= f;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&pfull[buf]);
                mbar_arrive(&empty[s]);
            }
            if (++s == STAGES) s = 0, phase ^= 1;
        }
        if (ok && n > 0) ok = drain(n - 1);
        const int64_t hrow = (int64_t(b) * a.H + head) * a.Lq + row;  // FWD, DQ
        const int64_t hrows = int64_t(a.B) * a.H * a.Lq;
        const float one = FWD ? 1.0f : attn_ds_factor(nk);
        float l = l2.x + l2.y;
        if (MODE == ATTN_DQ) {
            if (half == 1) {
                rd[0] = wa.value();
                rd[XR] = we.value();
                rd[2 * XR] = wd.value();
                rd[3 * XR] = wp.value();
            }
            named_barrier_sync(1, C::CWARPS * 32);
            if (sums && half == 0) {
                float t[4] = {wa.value() + rd[0], we.value() + rd[XR], wd.value() + rd[2 * XR],
                              wp.value() + rd[3 * XR]};
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = row < nx ? one * t[e] : 0.0f;
                put_slope_sums(a, t, split, hrow, row < LX, quad, lane, rowdata + 6 * XR, bid);
            }
        }
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
        if (row < LX) {
            const int64_t orow = (int64_t(b) * LX + row) * NH + head;
            const int64_t rows = int64_t(a.B) * LX * NH;
#pragma unroll
            for (int t = 0; t < C::NACC; ++t) {
                const float g = FWD ? (a.nsplit > 1 ? 1.0f : 1.0f / l)
                                : t != 0 ? 1.0f : a.nsplit > 1 ? one : one * a.scale;
#pragma unroll
                for (int c = 0; c < DP / 64; ++c) {
                    const int c0 = half * (DP / 2) + 32 * c;
                    float v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = any ? acc[t][32 * c + e] * g : 0.0f;
                    if (a.nsplit > 1) {
                        store_row(
                            a.part + ((int64_t(t) * a.nsplit + split) * rows + orow) * a.D + c0, v,
                            c0, a.D);
                    } else {
                        void *o = FWD ? a.out : MODE == ATTN_DQ ? a.dq : t ? a.dv : a.dk;
                        store_row(static_cast<float *>(o) + orow * a.D + c0, v, c0, a.D);
                    }
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == C::CWARPS + 1) tmem_free(tmem, 512);
}

template <int DP, bool BIAS>
__global__ void __launch_bounds__(Cfg32<ATTN_FWD, DP>::THREADS, 1)
attn_tc32_forward_kernel(const __grid_constant__ AttnArgs a,
                         const __grid_constant__ SplitMaps maps, const AttnSplit s,
                         const bool withhold) {
    attn_tc32_pass<ATTN_FWD, DP, BIAS>(a, maps, s, withhold, blockIdx.x);
}

// Both backward passes in one launch, the keys' (the longer blocks) first.
template <int DP, bool BIAS>
__global__ void __launch_bounds__(Cfg32<ATTN_DQ, DP>::THREADS, 1)
attn_tc32_backward_kernel(const __grid_constant__ AttnArgs dkv,
                          const __grid_constant__ AttnArgs dq,
                          const __grid_constant__ SplitMaps maps, const AttnSplit s,
                          const unsigned first, const bool withhold) {
    if (blockIdx.x < first)
        attn_tc32_pass<ATTN_DKV, DP, BIAS>(dkv, maps, s, withhold, blockIdx.x);
    else
        attn_tc32_pass<ATTN_DQ, DP, BIAS>(dq, maps, s, withhold, blockIdx.x - first);
}

// The three parts of an array [B, L, heads, D] of any strides, rows padded
// with zeros to Dp channels: out[3][B, L, heads, Dp].
struct SplitArgs {
    const float *x[4];
    int64_t sb[4], sl[4], sh[4];
    bf16 *out[4];
    int L[4], heads[4];
    int64_t rows[4];  // B L heads
    int D, Dp;
};

__global__ void __launch_bounds__(256) attn_split_kernel(const SplitArgs a) {
    const int which = blockIdx.y, groups = a.Dp / 8;
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t row = i / groups;
    if (row >= a.rows[which]) return;
    const int c0 = int(i - row * groups) * 8, heads = a.heads[which];
    const int64_t tok = row / heads, h = row - tok * heads, b = tok / a.L[which];
    const float *x = a.x[which] + b * a.sb[which] + (tok - b * a.L[which]) * a.sl[which] +
                     h * a.sh[which];
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c0 + e < a.D ? x[c0 + e] : 0.0f;
    uint32_t p[3][4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        split3(make_float2(v[2 * e], v[2 * e + 1]), p[0][e], p[1][e], p[2][e]);
#pragma unroll
    for (int t = 0; t < 3; ++t)
        *reinterpret_cast<uint4 *>(a.out[which] + (t * a.rows[which] + row) * a.Dp + c0) =
            make_uint4(p[t][0], p[t][1], p[t][2], p[t][3]);
}

bool tc32_maps(const AttnArgs &a, const AttnSplit &s, bool backward, SplitMaps &m) {
    const int64_t D = s.Dp, planes = 3 * int64_t(a.B);
    const int64_t qs[3] = {int64_t(a.Lq) * a.H * D, int64_t(a.H) * D, D};
    const int64_t ks[3] = {int64_t(a.Lk) * a.Hkv * D, int64_t(a.Hkv) * D, D};
    return make_map(&m.q, s.q, qs, planes, a.Lq, a.H, D) &&
           make_map(&m.k, s.k, ks, planes, a.Lk, a.Hkv, D) &&
           make_map(&m.v, s.v, ks, planes, a.Lk, a.Hkv, D) &&
           (!backward || make_map(&m.go, s.go, qs, planes, a.Lq, a.H, D));
}

bool withheld() { return (debug_stall() & PC_STALL_ATTENTION) != 0; }

template <int DP, bool BIAS>
cudaError_t tc32_forward(const AttnArgs &a, const AttnSplit &s, unsigned blocks,
                         cudaStream_t st) {
    using C = Cfg32<ATTN_FWD, DP>;
    SplitMaps m{};
    if (!tc32_maps(a, s, false, m)) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        allow_smem(attn_tc32_forward_kernel<DP, BIAS>, int(C::SMEM), a.device, done);
    if (e != cudaSuccess) return e;
    attn_tc32_forward_kernel<DP, BIAS><<<blocks, C::THREADS, C::SMEM, st>>>(a, m, s, withheld());
    return cudaGetLastError();
}

template <int DP, bool BIAS>
cudaError_t tc32_backward(const AttnArgs &dkv, unsigned first, const AttnArgs &dq,
                          unsigned second, const AttnSplit &s, cudaStream_t st) {
    using C = Cfg32<ATTN_DQ, DP>;
    constexpr size_t other = Cfg32<ATTN_DKV, DP>::SMEM;
    constexpr int smem = int(C::SMEM > other ? C::SMEM : other);
    static_assert(C::THREADS == Cfg32<ATTN_DKV, DP>::THREADS, "one launch");
    SplitMaps m{};
    if (!tc32_maps(dq, s, true, m)) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(attn_tc32_backward_kernel<DP, BIAS>, smem, dq.device, done);
    if (e != cudaSuccess) return e;
    attn_tc32_backward_kernel<DP, BIAS>
        <<<first + second, C::THREADS, smem, st>>>(dkv, dq, m, s, first, withheld());
    return cudaGetLastError();
}

}  // namespace

// (the planes of the parts, 3 B of them, are numbered in 32 bits)
bool attn_tc32_fits(const AttnArgs &a) {
    return a.Lq >= 1 && a.Lk >= 1 && a.B <= 0x7fffffff / 3;
}

int attn_tc32_rows(const AttnArgs &a, int mode) {
    return mode != ATTN_FWD && a.D > 64 ? 64 : XR;
}

size_t attn_split_bytes(const AttnArgs &a, bool backward) {
    const size_t Dp = size_t(a.D + 7) / 8 * 8;
    const size_t nq = size_t(a.B) * a.Lq * a.H, nk = size_t(a.B) * a.Lk * a.Hkv;
    return 3 * sizeof(bf16) * Dp * (nq * (backward ? 2 : 1) + 2 * nk);
}

cudaError_t launch_attn_split(const AttnArgs &a, bool backward, void *space, AttnSplit *s,
                              cudaStream_t st) {
    SplitArgs x{};
    x.D = a.D, x.Dp = (a.D + 7) / 8 * 8;
    const int64_t gs[3] = {int64_t(a.Lq) * a.H * a.D, int64_t(a.H) * a.D, a.D};
    const void *src[4] = {a.q, a.k, a.v, a.go};
    const int64_t *str[4] = {a.qs, a.ks, a.vs, gs};
    bf16 *at = static_cast<bf16 *>(space);
    int64_t most = 0;
    for (int i = 0; i < (backward ? 4 : 3); ++i) {
        const bool q = i == 0 || i == 3;
        x.x[i] = static_cast<const float *>(src[i]);
        x.sb[i] = str[i][0], x.sl[i] = str[i][1], x.sh[i] = str[i][2];
        x.L[i] = q ? a.Lq : a.Lk, x.heads[i] = q ? a.H : a.Hkv;
        x.rows[i] = int64_t(a.B) * x.L[i] * x.heads[i];
        x.out[i] = at;
        at += 3 * x.rows[i] * x.Dp;
        if (x.rows[i] > most) most = x.rows[i];
    }
    s->q = x.out[0], s->k = x.out[1], s->v = x.out[2], s->go = x.out[3], s->Dp = x.Dp;
    const int64_t blocks = (most * (x.Dp / 8) + 255) / 256;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    attn_split_kernel<<<dim3(unsigned(blocks), backward ? 4 : 3), 256, 0, st>>>(x);
    return cudaGetLastError();
}

cudaError_t launch_attn_tc32_forward(const AttnArgs &a, const AttnSplit &s, unsigned blocks,
                                     cudaStream_t st) {
    if (a.D <= 64)
        return a.slopes ? tc32_forward<64, true>(a, s, blocks, st)
                        : tc32_forward<64, false>(a, s, blocks, st);
    return a.slopes ? tc32_forward<128, true>(a, s, blocks, st)
                    : tc32_forward<128, false>(a, s, blocks, st);
}

cudaError_t launch_attn_tc32_backward(const AttnArgs &dkv, unsigned first, const AttnArgs &dq,
                                      unsigned second, const AttnSplit &s, cudaStream_t st) {
    if (dq.D <= 64)
        return dq.slopes ? tc32_backward<64, true>(dkv, first, dq, second, s, st)
                         : tc32_backward<64, false>(dkv, first, dq, second, s, st);
    return dq.slopes ? tc32_backward<128, true>(dkv, first, dq, second, s, st)
                     : tc32_backward<128, false>(dkv, first, dq, second, s, st);
}

}  // namespace pcn
