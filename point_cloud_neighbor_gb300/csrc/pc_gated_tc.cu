// pc_gated_tc.cu -- the gated projection on the tensor cores.
//
//   FWD   a = x Wg^T, u = x Wu^T, y = act(a) u
//   GRAD  a and u again, da = dy u act'(a), du = dy act(a)
//   DX    dx = da Wg + du Wu
//   DW    dWg = da^T x, dWu = du^T x
//
// All four are one kernel: persistent blocks walk over output tiles of BN columns and 128
// rows, or 256 that two blocks of a cluster share (FWD, GRAD: BN / 2 hidden units, whose
// rows of Wg and Wu lie side by side in the B tile, so that a thread finds a and u of
// the same unit in its own row of the accumulator).  One warp copies operand tiles, 64
// deep, by tensor maps into a ring of stages; one thread issues the products; 8 or 16
// warps take the accumulators, of which there are two, so that the products of one
// tile run under the other's arithmetic and stores.  What is contracted along its rows
// (DX: the weights; DW: both sides) is read as it lies, by MN-major operands.  Zeros past
// the arrays' ends make every size fit.
//
// Two blocks: each has half the rows of A and half of B's, the first issues the products
// of both.  A block alone reads 12 KB of operands for 128 x 256 x 16 products (128
// cycles) while 12 KB are copied in, 190 bytes a cycle of the 128 that shared memory
// gives: it ran at 1.38 times the products' cycles.  Two need 126.
//
// y, dy, da and du, which are as large as the result, go through a warp's room in shared
// memory: by tensor maps (dy a tile ahead), or where rows are not 16-byte aligned, and
// for y and dy in float32, row by row with neighbouring lanes at neighbouring columns.
//
// float32 runs as three bfloat16 parts of each operand and six products,
// low x high, high x low, middle x middle, middle x high, high x middle, high x
// high (to 2^-24).  A stage is one part of both operands, free as soon as the last
// product that takes it is issued.  The tensor cores cut their sums off instead of
// rounding them, so a chain is 64 long, the small products first, and the chains
// are added up in registers.  A bfloat16 chain over rows or hidden units takes at most
// 16,384 of them, joined in float32.
//
// da and du are operands of two products each.  bfloat16 calls take two bfloat16 parts
// of them, what the first leaves and then the first itself (to 2^-17): one part is a rounding
// of its own, which left dx and dW off by 1.41 times what rounding the results does.  So
// the products of DX and DW are twice as many; a stage has both parts, and what they are
// multiplied with once.  float32 calls take three parts.
//
// The biases' gradients are summed from the unrounded da and du: 32 rows by
// shuffles in GRAD, the parts in a kernel of their own.
//
// DX and DW split their contraction among blocks where there are few tiles; the
// parts are added in a fixed order by a kernel of its own.
//
// Bound: the products, and where C is small the epilogue; GRAD of wide layers also the
// 8 bytes a unit that it writes.  Measured, each launch alone, bfloat16: 32,768 x 1024 x 4096
// 268, 387, 556 and 561 us (2,050, 1,420, 1,980 and 1,960 TFLOP/s of 4 rows C F each, DX
// and DW 8); 16,384 x 384 x 1024 19, 45, 44 and 37 us; 100,000 x 512 x 2048 with gelu and
// biases 241 us forward (250 to 298 in a run of such calls, with the clock that the power
// limit leaves); 32 x 384 x 1024 4 us.  float32, 4084 x 387 x 1021 with gelu and biases: 43,
// 58, 33 and 34 us, and 5 to split the operands.  da and du in one part took 350, 300 and 301
// us instead of 387, 556 and 561; their two parts by tensor maps of 16 units instead of 32-byte
// stores 449 instead of 400 (in a pass).
//
// Waits are bounded and end as in pc_attn_tc.cu; the blocks take more than half a
// SM's shared memory, so none waits for another's tensor memory.
#include "pc_act.cuh"
#include "pc_gated.cuh"
#include "pc_launch.cuh"
#include "pc_tcgen05.cuh"
#include "pc_tiles.cuh"
#include "pointcloud.h"

#include <cfloat>
#include <type_traits>

namespace pcn {
namespace {

enum { G_FWD = 0, G_GRAD = 1, G_DX = 2, G_DW = 3 };
constexpr int BM = 128, BK = 64, CHAIN = 16384;
constexpr int PANEL = 64 * 128;  // bytes of a 64 x 64 panel of an MN-major operand

struct GemmMaps {
    CUtensorMap a0, a1, b0, b1;
    CUtensorMap dy, o0, o1;  // boxes of 32 rows: GRAD dy, float32 da, du; FWD y in o0
};

// Columns of a row of parts, so that all are 16-byte aligned.
__host__ __device__ inline int pad4(int n) { return (n + 3) / 4 * 4; }

struct GemmArgs {
    int64_t M;           // rows of the output
    int N;               // its columns
    int kb0, kb;         // stages of the first part of the contraction (DX: da), of all
    int mt, nt, nsplit;  // tiles; parts of the contraction, none of them empty,
    int per;             // of as many stages each (the last: at most)
    void *out, *out2;    // y; dx; dWg and dWu
    float *part;         // [nsplit][rows of all outputs][pad4(N)] where nsplit > 1
    const void *bg, *bu, *dy;
    bf16 *d;             // [da, du][parts of each: grad_parts][M][ld]
    float *bpart;        // GRAD: [4 mt][da, du][N], sums over 32 rows, or NULL
    int ld, act;
    bool vec, dvec;      // rows of the output, of dy, in 16-byte vectors
    bool withhold;
    uint64_t timeout_ns;
    int *status;
};

// Parts of da and du in calls whose operands have P.
__host__ __device__ constexpr int grad_parts(int P) { return P == 1 ? 2 : P; }

template <int MODE, int P, int BN, int CG>
struct GCfg {
    static constexpr bool PAIR = MODE == G_FWD || MODE == G_GRAD;
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN / CG * 128;
    static constexpr int M = BM * CG;  // rows of a tile
    // parts of A in a stage, beside one of B: both of da or du in bfloat16
    static constexpr int AP = !PAIR && P == 1 ? grad_parts(P) : 1;
    static constexpr int STAGE = AP * A_BYTES + B_BYTES;
    // Warps that take the accumulators: four for the 128 rows, times parts of the columns.
    // 16 where a tile's arithmetic outlasts its products otherwise (4084 x 387 x 1021
    // float32: with 8 the gradients of gelu took half as long again).
    static constexpr int EWARPS = PAIR && (BN == 256 || (P > 1 && BN == 128)) ? 16 : 8;
    static constexpr int THREADS = 32 * (4 + EWARPS);
    static constexpr int COLS = 2 * BN;               // tensor memory
    static constexpr int NL = BN / (EWARPS / 4);      // columns of a thread
    static constexpr int CH = PAIR ? NL / 2 : 32;     // PAIR: hidden units, else of a chunk
    static_assert(!PAIR || CH == 32 || CH == 16, "chunks");
    // PAIR: a warp's tiles of 32 rows by CH units of the arrays that are as large as the
    // result, on their way from or to global memory (bfloat16: TILE bytes each): dy; y; in
    // float32 da and du.  As tensor maps have them, or (float32, unaligned rows) as place()
    // does.
    static constexpr bool STAGED = PAIR && BN >= 128;
    static constexpr int TILE = 64 * CH;
    // (plain results: where rows are not 16-byte aligned)
    static constexpr int ROOM =
        !PAIR ? 1024 * (P > 1 ? 4 : 2) : !STAGED ? 0 : (P > 1 ? 2 : 1) * TILE;
    static constexpr int FIT = (227 * 1024 - 1024 - 512 - EWARPS * ROOM) / STAGE,
                         STAGES = FIT > 8 ? 8 : FIT;
    static_assert(STAGES >= 2 * P, "shared memory");
    static constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE + EWARPS * ROOM + 512;
    static_assert(SMEM > 114 * 1024 && SMEM <= 227 * 1024, "one block a SM");
};

// The six products of three parts, the smallest first.
__device__ constexpr int PART_A[6] = {2, 0, 1, 1, 0, 0};
__device__ constexpr int PART_B[6] = {0, 2, 1, 0, 1, 0};

template <int CH>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[CH]) {
    uint32_t r[CH];
    if constexpr (CH == 32)
        tmem_ld32(addr, r);
    else
        tmem_ld16(addr, r);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i] = __uint_as_float(r[i]);
}

// `left` columns of a row.
template <class T, int CH>
__device__ __forceinline__ void put(T *p, const float (&v)[CH], int left, bool vec) {
    constexpr int V = 16 / sizeof(T);
    if (vec) {
#pragma unroll
        for (int i = 0; i < CH / V; ++i)
            if (V * i < left) Vec<T, V>::store(p + V * i, v + V * i);
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (i < left) Vec<T, 1>::store(p + i, v + i);
    }
}
template <class T, int CH>
__device__ __forceinline__ void take(const T *p, float (&v)[CH], int left, bool vec) {
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i] = 0.0f;
    if (vec) {
#pragma unroll
        for (int i = 0; i < CH / V; ++i)
            if (V * i < left) Vec<T, V>::load(p + V * i, v + V * i);
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (i < left) Vec<T, 1>::load(p + i, v + i);
    }
}

// 16 bytes of a lane's row of CH bfloat16 of a tile, as a tensor map has it with a swizzle
// over rows of 64 or 32 bytes.
template <int CH>
__device__ __forceinline__ unsigned char *row_part(unsigned char *tile, int lane, int c) {
    return tile + lane * (2 * CH) +
           ((CH == 32 ? c ^ ((lane >> 1) & 3) : c ^ ((lane >> 2) & 1)) * 16);
}
// N of them from column o on.
template <int CH, int N>
__device__ __forceinline__ void put_row(unsigned char *tile, int lane, int o, const float *v) {
#pragma unroll
    for (int c = 0; c < N / 8; ++c)
        Vec<bf16, 8>::store(reinterpret_cast<bf16 *>(row_part<CH>(tile, lane, o / 8 + c)),
                            v + 8 * c);
}

// What rounding v to bfloat16 leaves for a second part: nothing where that is infinite.
__device__ __forceinline__ float left_over(float v) {
    const float f = __bfloat162float(__float2bfloat16_rn(v));
    return fabsf(f) <= FLT_MAX ? v - f : 0.0f;
}

// P parts of eight numbers, `plane` elements apart.
template <int P>
__device__ __forceinline__ void put_parts(bf16 *p, int64_t plane, const float *v) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[i];
#pragma unroll
    for (int k = 0; k < P; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = pack_bf16(t[2 * i], t[2 * i + 1]);
            if (P == 2) {
                t[2 * i] = left_over(t[2 * i]), t[2 * i + 1] = left_over(t[2 * i + 1]);
            } else {
                const float2 f = unpack_bf16(w[i]);
                t[2 * i] -= f.x, t[2 * i + 1] -= f.y;
            }
        }
        *reinterpret_cast<uint4 *>(p + k * plane) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Two parts of 16 numbers, `plane` elements apart: 32 bytes each, a whole sector of memory
// in one store, so that a lane writes its row without a detour through shared memory.
__device__ __forceinline__ void put_both(bf16 *p, int64_t plane, const float (&v)[16]) {
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = v[i];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = pack_bf16(t[2 * i], t[2 * i + 1]);
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + k * plane),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                     "r"(w[7])
                     : "memory");
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] = left_over(t[i]);
    }
}

// The sums of CH columns over the warp's rows: that of column c in the lanes with
// lane % CH = c.  Halves of the columns change places at every step.
template <int CH>
__device__ __forceinline__ float column_sums(const float (&x)[CH], int lane) {
    float v[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        v[i] = x[i];
        if (CH < 32) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
    }
#pragma unroll
    for (int o = CH / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const bool high = lane & o;
            const float keep = high ? v[i + o] : v[i], give = high ? v[i] : v[i + o];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    return v[0];
}

template <int MODE, int P, int BN, int CG>
__global__ void __launch_bounds__(GCfg<MODE, P, BN, CG>::THREADS, 1)
gated_gemm_kernel(const __grid_constant__ GemmMaps maps, const GemmArgs a) {
    using C = GCfg<MODE, P, BN, CG>;
    using T = std::conditional_t<P == 1, bf16, float>;
    constexpr int STAGES = C::STAGES, CH = C::CH;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char *rooms = base + size_t(STAGES) * C::STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(rooms + C::EWARPS * C::ROOM);
    uint64_t *empty = full + STAGES, *accfull = empty + STAGES, *accempty = accfull + 2;
    uint64_t *done = accempty + 2, *dybar = done + 1;  // dybar: of each warp
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(dybar + C::EWARPS);
    volatile int *stop = reinterpret_cast<volatile int *>(tmem_slot + 1);

    let_next_start();
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int tiles = a.mt * a.nt, items = tiles * a.nsplit;
    // the blocks of a tile: one, or a cluster of two with 128 rows each
    const int rank = CG > 1 ? int(cluster_ctarank()) : 0;
    const int first = int(blockIdx.x) / CG, step = int(gridDim.x) / CG;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
        for (int s = 0; s < 2; ++s)
            mbar_init(&accfull[s], 1), mbar_init(&accempty[s], CG * C::EWARPS);
        mbar_init(done, 1);
        for (int s = 0; s < C::EWARPS; ++s) mbar_init(&dybar[s], 1);
        *stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc<CG>(tmem_slot, C::COLS);
    tc_fence_before();
    __syncthreads();
    if (CG > 1) cluster_sync_all();  // both blocks' barriers exist
    tc_fence_after();
    after_previous();
    const uint32_t tmem = uniform(int(*tmem_slot));

    // A bounded wait; false: stop.
    auto await = [&](uint64_t *bar, unsigned parity) {
        const WaitResult w = mbar_wait_or_stop(bar, parity, stop, a.timeout_ns);
        if (w == WAIT_TIMEOUT) {
            *stop = 1;
            raise_status(a.status, PC_ERR_DEVICE_TIMEOUT);
        }
        return w == WAIT_OK;
    };
    // an item: a tile and a part of its contraction
    struct Item {
        int m, n, k0, k1, split;
        __device__ __forceinline__ Item(const GemmArgs &a, int i, int tiles) {
            split = unsigned(i) / unsigned(tiles);
            const unsigned t = i - split * tiles;
            m = t / unsigned(a.nt), n = t - m * a.nt;
            k0 = split * a.per;
            k1 = min(a.kb, k0 + a.per);
        }
    };

    if (warp == 0) {
        // ---- copies ---------------------------------------------------------------
        if (elect_one()) {
            int s = 0;
            unsigned phase = 1;  // (of the ring's first round: passes at once)
            int64_t issued = 0;
            bool ok = !(a.withhold && first == 0);
            for (int i = first; ok && i < items; i += step) {
                const Item it(a, i, tiles);
                const int dw_mt = a.mt / 2;  // DW: tiles of dWg, then of dWu
                const int m0 = (MODE == G_DW && it.m >= dw_mt ? it.m - dw_mt : it.m) * C::M +
                               rank * BM;
                for (int k = it.k0; ok && k < it.k1; ++k)
#pragma unroll
                    for (int p = P - 1; p >= 0; --p) {
                        if (!(ok = await(&empty[s], phase))) break;
                        unsigned char *A = base + size_t(s) * C::STAGE;
                        unsigned char *B = A + C::AP * C::A_BYTES;
                        // (both blocks' bytes are counted in the first)
                        uint64_t *bar = &full[s];
                        if (rank == 0) mbar_arrive_expect_tx(bar, CG * C::STAGE);
                        const uint32_t pair_bar = CG > 1 ? map_shared_rank(bar, 0) : 0;
                        auto load_part = [&](unsigned char *to, const CUtensorMap *map, int c,
                                             int r, int part) {
                            if (CG > 1)
                                tma_load_3d_pair(to, map, c, r, part, pair_bar);
                            else
                                tma_load_3d(to, map, c, r, part, bar);
                        };
                        auto load = [&](unsigned char *to, const CUtensorMap *map, int c, int r) {
                            load_part(to, map, c, r, p);
                        };
                        auto load_a = [&](int at, const CUtensorMap *map, int c, int r) {
#pragma unroll
                            for (int ap = 0; ap < C::AP; ++ap)
                                load_part(A + ap * C::A_BYTES + at, map, c, r, p + ap);
                        };
                        if (C::PAIR) {
                            load(A, &maps.a0, k * BK, m0);
                            if (CG > 1) {  // the first block Wg, the second Wu
                                load(B, rank ? &maps.b1 : &maps.b0, k * BK, it.n * (BN / 2));
                            } else {
                                load(B, &maps.b0, k * BK, it.n * (BN / 2));
                                load(B + C::B_BYTES / 2, &maps.b1, k * BK, it.n * (BN / 2));
                            }
                        } else {
                            const int n0 = it.n * BN + rank * (BN / CG);
                            if (MODE == G_DX) {
                                const bool up = k >= a.kb0;
                                const int f = (up ? k - a.kb0 : k) * BK;
                                load_a(0, up ? &maps.a1 : &maps.a0, f, m0);
#pragma unroll
                                for (int j = 0; j < BN / CG / 64; ++j)
                                    load(B + j * PANEL, up ? &maps.b1 : &maps.b0, n0 + 64 * j, f);
                            } else {
#pragma unroll
                                for (int j = 0; j < BM / 64; ++j)
                                    load_a(j * PANEL, it.m >= dw_mt ? &maps.a1 : &maps.a0,
                                           m0 + 64 * j, k * BK);
#pragma unroll
                                for (int j = 0; j < BN / CG / 64; ++j)
                                    load(B + j * PANEL, &maps.b0, n0 + 64 * j, k * BK);
                            }
                        }
                        ++issued;
                        if (++s == STAGES) s = 0, phase ^= 1;
                    }
            }
            // nothing is in flight when the blocks end
            for (int64_t k = rank ? issued : issued > STAGES ? issued - STAGES : 0; k < issued; ++k)
                mbar_wait_bounded(&full[k % STAGES], unsigned((k / STAGES) & 1), a.timeout_ns);
        }
    } else if (warp == 1) {
        // ---- products, of both blocks by the first ------------------------------------
        if (elect_one() && rank == 0) {
            constexpr bool AR = MODE == G_DW, BR = !C::PAIR;  // contracted along their rows
            constexpr uint32_t id = mma_idesc(BN, BR, AR, C::M);
            constexpr uint32_t da = AR ? 16 * 128 / 16 : 2, db = BR ? 16 * 128 / 16 : 2;
            const uint32_t a0 = smem_operand(smem_u32(base), AR ? PANEL : 16);
            const uint32_t b0 = smem_operand(smem_u32(base) + C::AP * C::A_BYTES, BR ? PANEL : 16);
            int s = 0, buf = 0;
            unsigned phase = 0, aphase = 1;
            bool ok = true;
            auto commit = [](uint64_t *bar) {
                if (CG > 1)
                    mma_commit_pair(bar);
                else
                    mma_commit(bar);
            };
            for (int i = first; ok && i < items; i += step) {
                const Item it(a, i, tiles);
                for (int k = it.k0; k < it.k1; ++k) {
                    // (float32: an accumulator for every 64 of the depth)
                    const bool fresh = P > 1 || k == it.k0;
                    if (fresh && !(ok = await(&accempty[buf], aphase))) break;
                    int at[P];  // the stages of the parts, which come in falling order
#pragma unroll
                    for (int p = P - 1; p >= 0; --p) {
                        ok = ok && await(&full[s], phase);
                        at[p] = s;
                        if (++s == STAGES) s = 0, phase ^= 1;
                    }
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + buf * BN;
                    // a stage is free after the last product that takes its part
#pragma unroll
                    for (int q = 0; q < (P == 1 ? C::AP : 6); ++q) {
                        const int pa = P == 1 ? 0 : PART_A[q], pb = P == 1 ? 0 : PART_B[q];
                        const int ap = P == 1 ? C::AP - 1 - q : 0;
                        const uint32_t as = a0 + at[pa] * (C::STAGE / 16) + ap * (C::A_BYTES / 16),
                                       bs = b0 + at[pb] * (C::STAGE / 16);
#pragma unroll
                        for (int j = 0; j < BK / 16; ++j)
                            if (CG > 1)
                                mma_ss_pair<SMEM_128B>(d, as + j * da, bs + j * db, id,
                                                       !fresh || q > 0 || j > 0);
                            else
                                mma_ss<SMEM_128B>(d, as + j * da, bs + j * db, id,
                                                  !fresh || q > 0 || j > 0);
                        if (P == 1 ? q == C::AP - 1 : q == 5) commit(&empty[at[0]]);
                        if (P > 1 && q == 4) commit(&empty[at[P > 1 ? 1 : 0]]);
                        if (P > 1 && q == 1) commit(&empty[at[P > 1 ? 2 : 0]]);
                    }
                    if (P > 1 || k + 1 == it.k1) {
                        commit(&accfull[buf]);
                        buf ^= 1;
                        if (buf == 0) aphase ^= 1;
                    }
                }
            }
            commit(done);
            mbar_wait_bounded(done, 0, a.timeout_ns);
        }
    } else if (warp >= 4) {
        // ---- accumulators -------------------------------------------------------------
        const int quad = warp % 4, part = (warp - 4) / 4;  // its rows, its columns
        const uint32_t lanes = uint32_t(quad * 32) << 16;
        int buf = 0;
        unsigned phase = 0;
        bool ok = true;
        auto wait = [&]() { return __all_sync(0xffffffffu, await(&accfull[buf], phase)) != 0; };
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG > 1)
                    mbar_arrive_cluster(map_shared_rank(&accempty[buf], 0));
                else
                    mbar_arrive(&accempty[buf]);
            }
            buf ^= 1;
            if (buf == 0) phase ^= 1;
        };
        unsigned char *room = rooms + (warp - 4) * C::ROOM, *dyroom = room;  // the warp's
        const bool leader = elect_one();
        // Where column c of row r of an unaligned array is, so that neither the lanes of a
        // row nor those of a column meet in a bank.
        auto place = [](int r, int c) {
            if (P == 1) return r * 32 + ((((c >> 1) ^ (r >> 1)) << 1) | (c & 1));
            return CH == 32 ? r * 32 + (c ^ r) : r * 16 + (c ^ ((r >> 1) & 15));
        };
        constexpr int W = P > 1 ? 1 : 2;
        static_assert(!C::STAGED || P > 1 || CH == 32, "bfloat16 goes in rows of 32");
        // the rows that go with one instruction, a lane's row and column among them
        constexpr int RS = C::STAGED ? 32 / CH : 1;
        const int lr = lane / CH, lc = lane % CH;
        auto rows_in = [&](T *to, const T *from, int64_t r0, int c0) {
            T v[32 / RS];  // (all loads before the first store)
            from += (r0 + lr) * a.N + c0 + lc;
            const int rows = c0 + lc < a.N ? int(min(a.M - r0, int64_t(32))) : 0;
#pragma unroll
            for (int r = 0; r < 32; r += RS, from += RS * a.N)
                v[r / RS] = r + lr < rows ? *from : T(0.0f);
#pragma unroll
            for (int r = 0; r < 32; r += RS) to[place(r + lr, lc)] = v[r / RS];
        };
        auto rows_out = [&](T *to, const T *from, int64_t r0, int c0) {
            T v[32 / RS];
#pragma unroll
            for (int r = 0; r < 32; r += RS) v[r / RS] = from[place(r + lr, lc)];
            to += (r0 + lr) * a.N + c0 + lc;
            const int rows = c0 + lc < a.N ? int(min(a.M - r0, int64_t(32))) : 0;
#pragma unroll
            for (int r = 0; r < 32; r += RS, to += RS * a.N)
                if (r + lr < rows) *to = v[r / RS];
        };
        // the warp's tile of an item
        auto tile_row = [&](const Item &it) { return it.m * C::M + rank * BM + quad * 32; };
        auto tile_column = [&](const Item &it) { return it.n * (BN / 2) + part * CH; };
        // dy is copied a tile ahead
        constexpr bool AHEAD = MODE == G_GRAD && C::STAGED && P == 1;
        uint64_t *mydy = &dybar[warp - 4];
        unsigned dyphase = 0;
        bool dyahead = false;  // under way
        auto dy_ahead = [&](int i) {
            dyahead = i < items;
            if (!dyahead) return;
            const Item it(a, i, tiles);
            mbar_arrive_expect_tx(mydy, C::TILE);
            tma_load_3d(dyroom, &maps.dy, tile_column(it), tile_row(it), 0, mydy);
        };
        if (AHEAD && a.dvec && leader) dy_ahead(first);
        for (int i = first; i < items; i += step) {
            const Item it(a, i, tiles);
            float sum[P == 1 ? 1 : C::NL];
            if (P > 1) {
                if (MODE == G_GRAD && C::STAGED) {  // (under the products)
                    if (leader) bulk_wait_read_all();
                    __syncwarp();
                    rows_in(reinterpret_cast<T *>(dyroom), static_cast<const T *>(a.dy),
                            tile_row(it), tile_column(it));
                }
#pragma unroll
                for (int c = 0; c < (P == 1 ? 1 : C::NL); ++c) sum[c] = 0.0f;
                for (int k = it.k0; k < it.k1; ++k) {
                    if (!(ok = wait())) break;
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < C::NL / CH; ++j) {
                        float v[CH];
                        tmem_load<CH>(tmem + lanes + buf * BN +
                                          (C::PAIR ? j * (BN / 2) + part * CH
                                                   : part * C::NL + j * CH),
                                      v);
#pragma unroll
                        for (int c = 0; c < CH; ++c) sum[(P == 1 ? 0 : j * CH + c)] += v[c];
                    }
                    release();
                }
                if (!ok) break;
            }
            if constexpr (C::PAIR) {
                // units at a time
                constexpr int SUB = C::EWARPS == 16 || (MODE == G_GRAD && C::STAGED) ? 16 : CH;
                const int64_t row0 = tile_row(it), row = row0 + lane;
                const int c0 = tile_column(it), left = row < a.M ? a.N - c0 : 0;
                const bool live = row0 < a.M && c0 < a.N;  // the warp has something to write
                const T *dysrc = static_cast<const T *>(a.dy);
                constexpr int DP = grad_parts(P);
                uint4 dyraw[AHEAD ? 4 : 1];  // the thread's 32 units of dy
                if constexpr (AHEAD) {
                    if (a.dvec) {
                        if (!(ok = __all_sync(0xffffffffu, await(mydy, dyphase)))) break;
                        dyphase ^= 1;
                        dyahead = false;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            dyraw[c] = *reinterpret_cast<const uint4 *>(row_part<CH>(dyroom, lane, c));
                        // (every lane's loads are done before the next copy is issued: they
                        // can wait behind stores for longer than the copy takes)
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (leader) dy_ahead(i + step);
                    } else {
                        rows_in(reinterpret_cast<T *>(dyroom), dysrc, row0, c0);
                        __syncwarp();
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            (&dyraw[c / 4].x)[c % 4] = *reinterpret_cast<const uint32_t *>(
                                reinterpret_cast<const T *>(dyroom) + place(lane, 2 * c));
                        __syncwarp();
                    }
                }
                if (P == 1) {
                    if (!(ok = wait())) break;
                    tc_fence_after();
                }
                if (C::STAGED) {
                    if (P == 1 && MODE == G_FWD && leader) bulk_wait_read_all();  // the room is free
                    __syncwarp();
                }
#pragma unroll
                for (int h = 0; h < CH / SUB; ++h) {
                    const int o = h * SUB;  // of the warp's units
                    float dy[MODE == G_GRAD ? SUB : 1], g[SUB], u[SUB];
                    if constexpr (MODE == G_GRAD) {
                        const T *mine = reinterpret_cast<const T *>(dyroom);
                        if constexpr (!C::STAGED) {
                            take<T, SUB>(dysrc + row * a.N + c0, dy, left, a.dvec);
                        } else if constexpr (AHEAD) {
#pragma unroll
                            for (int c = 0; c < SUB / 8; ++c)
                                Vec<bf16, 8>::load(
                                    reinterpret_cast<const bf16 *>(&dyraw[o / 8 + c]), dy + 8 * c);
                        } else {
#pragma unroll
                            for (int c = 0; c < SUB; ++c) dy[c] = float(mine[place(lane, o + c)]);
                        }
                    }
                    if (P == 1) {
                        tmem_load<SUB>(tmem + lanes + buf * BN + part * CH + o, g);
                        tmem_load<SUB>(tmem + lanes + buf * BN + BN / 2 + part * CH + o, u);
                        if (o + SUB == CH) release();
                    } else {
#pragma unroll
                        for (int c = 0; c < SUB; ++c)
                            g[c] = sum[P == 1 ? 0 : o + c], u[c] = sum[P == 1 ? 0 : CH + o + c];
                    }
                    if (a.bg != nullptr) {
                        float bg = 0.0f, bu = 0.0f;  // of unit lane
                        if (lane < SUB && c0 + o + lane < a.N) {
                            Vec<T, 1>::load(static_cast<const T *>(a.bg) + c0 + o + lane, &bg);
                            Vec<T, 1>::load(static_cast<const T *>(a.bu) + c0 + o + lane, &bu);
                        }
#pragma unroll
                        for (int c = 0; c < SUB; ++c) {
                            g[c] += __shfl_sync(0xffffffffu, bg, c);
                            u[c] += __shfl_sync(0xffffffffu, bu, c);
                        }
                    }
                    if constexpr (MODE == G_FWD) {
                        act_switch(a.act, [&](auto act) {
#pragma unroll
                            for (int c = 0; c < SUB; ++c)
                                g[c] = act_value<act.value, P == 1>(g[c]) * u[c];
                        });
                        if (!C::STAGED)
                            put<T, SUB>(static_cast<T *>(a.out) + row * a.N + c0, g, left, a.vec);
                        else if (P == 1 && a.vec)
                            put_row<CH, SUB>(room, lane, o, g);
                        else
#pragma unroll
                            for (int c = 0; c < SUB; c += W)
                                Vec<T, W>::store(reinterpret_cast<T *>(room) + place(lane, o + c),
                                                 g + c);
                    } else {
                        act_switch(a.act, [&](auto act) {
#pragma unroll
                            for (int c = 0; c < SUB; ++c) {
                                float slope;
                                const float f = act_both<act.value, P == 1>(g[c], slope);
                                g[c] = dy[c] * u[c] * slope;
                                u[c] = dy[c] * f;
                            }
                        });
                        if (a.bpart != nullptr) {  // (before they are rounded)
                            // (rows past the end have the biases' values, times 0)
                            if (row >= a.M)
#pragma unroll
                                for (int c = 0; c < SUB; ++c) g[c] = u[c] = 0.0f;
                            const float sg = column_sums<SUB>(g, lane);
                            const float su = column_sums<SUB>(u, lane);
                            float *to = a.bpart +
                                        ((int64_t(it.m) * CG + rank) * 4 + quad) * 2 * a.N + c0 +
                                        o + lane;
                            if (lane < SUB && c0 + o + lane < a.N) to[0] = sg, to[a.N] = su;
                        }
                        if constexpr (!C::STAGED) {
                            const int64_t plane = a.M * a.ld;
                            bf16 *to = a.d + row * a.ld + c0;
#pragma unroll
                            for (int c = 0; c < SUB; c += 8)
                                if (c < left) {  // (the rows' padding takes zeros)
                                    put_parts<DP>(to + c, plane, g + c);
                                    put_parts<DP>(to + DP * plane + c, plane, u + c);
                                }
                        } else if constexpr (P == 1) {
                            if (row < a.M && c0 + o < a.N) {
                                const int64_t plane = a.M * a.ld;
                                bf16 *to = a.d + row * a.ld + c0 + o;
                                put_both(to, plane, g);
                                put_both(to + DP * plane, plane, u);
                            }
                            __syncwarp();  // (the loads from tensor memory take whole warps)
                        } else {
                            // three parts, one after the other through the room
                            __syncwarp();
#pragma unroll
                            for (int k = 0; k < P; ++k) {
                                if (k > 0) {
                                    if (leader) bulk_wait_read_all();
                                    __syncwarp();
                                }
                                put_row<CH, SUB>(room, lane, 0, g);
                                put_row<CH, SUB>(room + C::TILE, lane, 0, u);
                                fence_proxy_async_smem();
                                __syncwarp();
                                if (leader && live) {
                                    tma_store_3d(&maps.o0, room, c0, int(row0), k);
                                    tma_store_3d(&maps.o1, room + C::TILE, c0, int(row0), k);
                                    bulk_commit();
                                }
#pragma unroll
                                for (int c = 0; c < SUB; ++c)
                                    g[c] = rest<bf16>(g[c]), u[c] = rest<bf16>(u[c]);
                            }
                        }
                    }
                }
                if constexpr (C::STAGED && MODE == G_FWD) {
                    if (P == 1 && a.vec) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (leader && live) {
                            tma_store_3d(&maps.o0, room, c0, int(row0), 0);
                            bulk_commit();
                        }
                    } else {
                        __syncwarp();
                        rows_out(static_cast<T *>(a.out), reinterpret_cast<const T *>(room), row0,
                                 c0);
                        __syncwarp();
                    }
                }
            } else {
                constexpr int n = C::NL / CH;
                const int dw_mt = a.mt / 2;
                const bool up = MODE == G_DW && it.m >= dw_mt;
                const int64_t row =
                    int64_t(up ? it.m - dw_mt : it.m) * C::M + rank * BM + quad * 32 + lane;
                if (P == 1) {
                    if (!(ok = wait())) break;
                    tc_fence_after();
                }
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    float v[CH];
                    if (P == 1) {
                        tmem_load<CH>(tmem + lanes + buf * BN + part * C::NL + j * CH, v);
                        if (j == n - 1) release();
                    } else {
#pragma unroll
                        for (int c = 0; c < CH; ++c) v[c] = sum[P == 1 ? 0 : j * CH + c];
                    }
                    const int c0 = it.n * BN + part * C::NL + j * CH;
                    const int left = row < a.M ? a.N - c0 : 0;
                    T *out = static_cast<T *>(up ? a.out2 : a.out);
                    if (a.nsplit > 1) {
                        const int64_t all = MODE == G_DW ? 2 * a.M : a.M;
                        put<float, CH>(
                            a.part + (it.split * all + (up ? a.M : 0) + row) * pad4(a.N) + c0, v,
                            row < a.M ? pad4(a.N) - c0 : 0, true);
                    } else if (a.vec) {
                        put<T, CH>(out + row * a.N + c0, v, left, true);
                    } else {
#pragma unroll
                        for (int c = 0; c < CH; c += W)
                            Vec<T, W>::store(reinterpret_cast<T *>(room) + place(lane, c), v + c);
                        __syncwarp();
                        rows_out(out, reinterpret_cast<const T *>(room), row - lane, c0);
                        __syncwarp();
                    }
                }
            }
        }
        // nothing is in flight when the block ends
        if (leader) bulk_wait_read_all();
        if (AHEAD && dyahead && !ok) mbar_wait_bounded(mydy, dyphase, a.timeout_ns);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (CG > 1) cluster_sync_all();  // neither block's memory is in use any more
    if (warp == 2) {
        tc_fence_after();
        tmem_free<CG>(tmem, C::COLS);
    }
}

// --- operands that the tensor maps cannot read as they are -------------------------

struct PackJob {
    const void *src;
    bf16 *dst;       // [P][rows][ld]
    int64_t rows;
    int C, ld, blocks;
    bool vec;
};
struct PackJobs {
    PackJob job[3];
};
constexpr int PACK_ROWS = 8;

// Rows of T as P bfloat16 parts, padded to eight columns.
template <class T, int P>
__global__ void __launch_bounds__(256) gated_pack_kernel(PackJobs jobs) {
    let_next_start();
    // (copied by constant indices: an index computed here would put them in local memory)
    int b = blockIdx.x;
    PackJob j = jobs.job[0];
    if (b >= j.blocks) {
        b -= j.blocks;
        j = jobs.job[1];
        if (b >= j.blocks) {
            b -= j.blocks;
            j = jobs.job[2];
        }
    }
    const int64_t r0 = int64_t(b) * PACK_ROWS;
    const int rows = int(min(int64_t(PACK_ROWS), j.rows - r0));
    const int groups = j.ld / 8;
    for (int i = threadIdx.x; i < rows * groups; i += 256) {
        const int64_t r = r0 + i / groups;
        const int c = i % groups * 8;
        float v[8];
        take<T, 8>(static_cast<const T *>(j.src) + r * j.C + c, v, j.C - c, j.vec);
        put_parts<P>(j.dst + r * j.ld + c, j.rows * j.ld, v);
    }
}

// --- sums of parts -------------------------------------------------------------------

// The sum over the parts, in their order, of rows of N columns: the first `half` rows to
// out, the others to out2.  A thread four columns.
template <class T>
__global__ void __launch_bounds__(256)
gated_join_kernel(const float *part, int nparts, int64_t rows, int64_t half, int N, FastDiv groups,
                  bool vec, T *out, T *out2) {
    let_next_start();
    after_previous();
    const int ld = pad4(N);
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x, all = rows * (ld / 4);
    if (i >= all) return;
    const int64_t row = all < (int64_t(1) << 31) ? groups.div(uint32_t(i)) : i / (ld / 4);
    const int c = int(i - row * (ld / 4)) * 4;
    const float *p = part + row * ld + c;
    float s[4];
    Vec<float, 4>::load(p, s);
#pragma unroll 4
    for (int k = 1; k < nparts; ++k) {
        float v[4];
        Vec<float, 4>::load(p + k * rows * ld, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += v[e];
    }
    T *to = (row < half ? out + row * N : out2 + (row - half) * N) + c;
    if (vec) {
        Vec<T, 4>::store(to, s);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < N) Vec<T, 1>::store(to + e, s + e);
    }
}

// The biases' gradients: 32 columns a block, 32 warps every 32nd part, in a fixed order.
template <class T>
__global__ void __launch_bounds__(1024)
gated_bias_kernel(const float *part, int nparts, int F, T *dbg, T *dbu) {
    let_next_start();
    after_previous();
    __shared__ float acc[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < 2 * F)
#pragma unroll 4
        for (int p = threadIdx.y; p < nparts; p += 32) s += part[int64_t(p) * 2 * F + c];
    acc[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < 2 * F) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += acc[i][threadIdx.x];
        Vec<T, 1>::store(c < F ? dbg + c : dbu + (c - F), &s);
    }
}

// --- host ------------------------------------------------------------------------------

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int pad8(int64_t n) { return int((n + 7) / 8 * 8); }
bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Rows of bfloat16, P parts, that a tensor map can read.
struct Operand {
    const bf16 *p = nullptr;
    int64_t rows = 0;
    int cols = 0, ld = 0, parts = 1;
};

// Boxes of `columns` (64, 32 or 16) columns by `box` rows of one part.
bool make_map3(CUtensorMap *map, const Operand &o, int box, int columns = 64) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {cuuint64_t(o.cols), cuuint64_t(o.rows), cuuint64_t(o.parts)};
    const cuuint64_t strides[2] = {cuuint64_t(o.ld) * 2, cuuint64_t(o.rows) * o.ld * 2};
    const cuuint32_t b[3] = {cuuint32_t(columns), cuuint32_t(box), 1}, ones[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf16 *>(o.p), dims, strides, b,
              ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              columns == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
              : columns == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                              : CU_TENSOR_MAP_SWIZZLE_32B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The same of a result or its gradient in bfloat16, 32 x 32.
bool make_tile_map(CUtensorMap *map, const void *p, int64_t rows, int cols, int ld) {
    Operand o;
    o.p = static_cast<const bf16 *>(p), o.rows = rows, o.cols = cols, o.ld = ld;
    return make_map3(map, o, 32, 32);
}

// Scratch handed out in pieces: sizes first, then addresses.
struct Scratch {
    size_t bytes = 0;
    char *base = nullptr;
    size_t take(size_t n) {
        const size_t at = bytes;
        bytes += (n + 1023) / 1024 * 1024;
        return at;
    }
};

// The kinds of a tile: its columns, and the blocks that share it.
struct GemmKind {
    int BN, CG;
    // SM cycles, measured: 64 of the depth (32,768 x 8192 x 1024 bf16, all SMs; the products
    // alone take 512, 256, 256 and 192); a tile's epilogue, which runs under the next tile's
    // products: forward (silu), gradients, plain results; a launch's start and end.
    double stage, forward, grad, plain, fixed;
};
constexpr GemmKind KINDS[] = {{256, 2, 620, 4400, 7000, 2600, 6300},
                              {128, 2, 350, 2650, 3500, 1500, 6300},
                              {128, 1, 385, 3000, 4100, 1500, 4200},
                              {64, 1, 277, 2400, 4100, 1000, 4200}};

// The kind of tile and the parts of the contraction, by the smallest estimate.  bfloat16 DX
// and DW: two products for one.  float32: six, epilogues three times as long (and no tiles
// of 256 columns, whose sums a thread could not hold).  Parts cost their writes and reads and
// a launch.  (With da and du in two parts the choices for the three passes of 2048 x 1024 x
// 1024, 8192 x 256 x 4096, 32,768 x 1024 x 4096 and 65,536 x 128 x 256 are within 10% of the
// best kind, which is what two runs of one kind differ by.)
struct GemmPlan {
    int BN = 0, CG = 1, nsplit = 1, per = 1;
    int rows() const { return BM * CG; }
};
GemmPlan plan_gemm(int sms, int mode, int P, int64_t M, int64_t N, int64_t kb) {
    GemmPlan best;
    double least = 1e300;
    const bool pair = mode == G_FWD || mode == G_GRAD;
    for (const GemmKind &kind : KINDS) {
        if (P > 1 && kind.BN == 256) continue;
        const double stage = kind.stage * (P > 1 ? 6.3 : pair ? 1.0 : grad_parts(P));
        const double epilogue = (mode == G_FWD    ? kind.forward
                                 : mode == G_GRAD ? kind.grad
                                                  : kind.plain) *
                                (P == 1 ? 1.0 : 3.0);
        const int64_t tall = BM * kind.CG, units = sms / kind.CG;
        const int64_t mtiles = mode == G_DW ? 2 * ceil_div(M / 2, tall) : ceil_div(M, tall);
        const int64_t tiles = mtiles * ceil_div(N, pair ? kind.BN / 2 : kind.BN);
        // (a part has a row of a chain's length at most in bfloat16)
        const int64_t fewest = !pair && P == 1 ? ceil_div(kb * BK, CHAIN) : 1;
        const int64_t most = pair ? 1 : kb < 64 ? kb : 64;
        for (int64_t ns = fewest; ns <= (most > fewest ? most : fewest); ++ns) {
            if (ns > fewest && tiles * (ns - 1) > 8 * units) break;  // (waves enough)
            const double k = double(ceil_div(kb, ns)) * stage;
            double cost = double(ceil_div(tiles * ns, units)) * (k > epilogue ? k : epilogue) +
                          epilogue + kind.fixed;
            if (ns > 1) cost += 6000 + 8.0 * double(ns) * double(M) * double(N) / 3000;
            if (cost < least)
                least = cost, best.BN = kind.BN, best.CG = kind.CG, best.nsplit = int(ns);
        }
    }
    best.per = int(ceil_div(kb, best.nsplit));
    best.nsplit = int(ceil_div(kb, best.per));
    return best;
}

template <int MODE, int P, int BN, int CG>
cudaError_t run_gemm(const DeviceInfo &dev, const GemmMaps &maps, const GemmArgs &g, bool behind,
                     cudaStream_t st) {
    using C = GCfg<MODE, P, BN, CG>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        allow_smem(gated_gemm_kernel<MODE, P, BN, CG>, int(C::SMEM), dev.device, done);
    if (e != cudaSuccess) return e;
    const int64_t items = int64_t(g.mt) * g.nt * g.nsplit, units = dev.sm_count / CG;
    if (items > (int64_t(1) << 30)) return cudaErrorInvalidConfiguration;
    const unsigned blocks = unsigned(items < units ? items : units) * CG;
    return launch_clusters(behind, gated_gemm_kernel<MODE, P, BN, CG>, blocks, C::THREADS, C::SMEM,
                           st, CG, maps, g);
}
template <int MODE, int P>
cudaError_t run_gemm(const DeviceInfo &dev, const GemmMaps &maps, const GemmArgs &g,
                     const GemmPlan &p, bool behind, cudaStream_t st) {
    if (p.CG == 2) {
        if constexpr (P == 1)
            if (p.BN == 256) return run_gemm<MODE, P, 256, 2>(dev, maps, g, behind, st);
        return run_gemm<MODE, P, 128, 2>(dev, maps, g, behind, st);
    }
    return p.BN == 128 ? run_gemm<MODE, P, 128, 1>(dev, maps, g, behind, st)
                       : run_gemm<MODE, P, 64, 1>(dev, maps, g, behind, st);
}

template <class T>
cudaError_t join(const float *part, int nparts, int64_t rows, int64_t half, int N, void *out,
                 void *out2, cudaStream_t st) {
    T *o = static_cast<T *>(out), *o2 = static_cast<T *>(out2);
    const bool vec = N % 4 == 0 && aligned16(out) && (out2 == nullptr || aligned16(out2));
    const int groups = pad4(N) / 4;
    return launch(true, gated_join_kernel<T>, unsigned(ceil_div(rows * groups, 256)), 256, 0, st,
                  part, nparts, rows, half, N, FastDiv(groups), vec, o, o2);
}

// x and the weights as operands, split or copied where they have to be.
struct Inputs {
    Operand x, wg, wu;
    size_t at[3];
    bool packed[3];
    bool any() const { return packed[0] || packed[1] || packed[2]; }
};
template <class T, int P>
void plan_inputs(const GatedArgs &a, Inputs &in, Scratch &s) {
    Operand *o[3] = {&in.x, &in.wg, &in.wu};
    const void *src[3] = {a.x, a.wg, a.wu};
    for (int i = 0; i < 3; ++i) {
        o[i]->rows = i ? a.F : a.rows, o[i]->cols = a.C, o[i]->parts = P;
        in.packed[i] = P > 1 || a.C % 8 || !aligned16(src[i]);
        o[i]->ld = in.packed[i] ? pad8(a.C) : a.C;
        if (in.packed[i])
            in.at[i] = s.take(size_t(P) * o[i]->rows * o[i]->ld * sizeof(bf16));
        else
            o[i]->p = static_cast<const bf16 *>(src[i]);
    }
}
template <class T, int P>
cudaError_t pack_inputs(const GatedArgs &a, Inputs &in, const Scratch &s, cudaStream_t st) {
    Operand *o[3] = {&in.x, &in.wg, &in.wu};
    const void *src[3] = {a.x, a.wg, a.wu};
    PackJobs jobs{};
    int n = 0;
    int64_t blocks = 0;
    for (int i = 0; i < 3; ++i) {
        if (!in.packed[i]) continue;
        bf16 *dst = reinterpret_cast<bf16 *>(s.base + in.at[i]);
        o[i]->p = dst;
        PackJob &j = jobs.job[n++];
        j.src = src[i], j.dst = dst, j.rows = o[i]->rows, j.C = a.C, j.ld = o[i]->ld;
        j.blocks = int(ceil_div(j.rows, PACK_ROWS));
        j.vec = a.C % (16 / sizeof(T)) == 0 && aligned16(src[i]);
        blocks += j.blocks;
    }
    if (n == 0) return cudaSuccess;
    gated_pack_kernel<T, P><<<unsigned(blocks), 256, 0, st>>>(jobs);
    return cudaGetLastError();
}

GemmArgs gemm_args(const DeviceInfo &dev, const GatedArgs &a) {
    GemmArgs g{};
    g.bg = a.bg, g.bu = a.bu, g.dy = a.dy, g.act = a.act;
    g.timeout_ns = wait_timeout_ns(), g.status = dev.status_word;
    g.withhold = (debug_stall() & PC_STALL_GATED) != 0;
    g.nsplit = 1;
    return g;
}

// What a backward call keeps in scratch.
struct BackwardPlan {
    Scratch s;
    Inputs in;
    int ld = 0, kf = 0, kr = 0;
    GemmPlan pg, px, pw;
    size_t d_at = 0, part_x = 0, part_w = 0, part_b = 0;
};
template <class T, int P>
BackwardPlan plan_backward(const DeviceInfo &dev, const GatedArgs &a) {
    BackwardPlan b;
    plan_inputs<T, P>(a, b.in, b.s);
    b.ld = P == 1 ? (a.F + 15) / 16 * 16 : pad8(a.F);  // (16 units go in one store: put_both)
    b.d_at = b.s.take(size_t(2) * grad_parts(P) * a.rows * b.ld * sizeof(bf16));
    b.pg = plan_gemm(dev.sm_count, G_GRAD, P, a.rows, a.F, ceil_div(a.C, BK));
    b.kf = int(ceil_div(a.F, BK)), b.kr = int(ceil_div(a.rows, BK));
    if (a.dx) {
        b.px = plan_gemm(dev.sm_count, G_DX, P, a.rows, a.C, 2 * b.kf);
        if (b.px.nsplit > 1)
            b.part_x = b.s.take(size_t(b.px.nsplit) * a.rows * pad4(a.C) * sizeof(float));
    }
    if (a.dwg) {
        b.pw = plan_gemm(dev.sm_count, G_DW, P, 2 * int64_t(a.F), a.C, b.kr);
        if (b.pw.nsplit > 1)
            b.part_w = b.s.take(size_t(b.pw.nsplit) * 2 * a.F * pad4(a.C) * sizeof(float));
    }
    if (a.dbg)
        b.part_b = b.s.take(size_t(ceil_div(a.rows, b.pg.rows())) * b.pg.CG * 4 * 2 * a.F *
                            sizeof(float));
    return b;
}

// The caller's workspace where it is large enough, else the library's pool.
struct Memory {
    cudaStream_t st;
    void *own = nullptr;
    cudaError_t take(const DeviceInfo &dev, Scratch &s, const GatedArgs &a) {
        if (s.bytes == 0) return cudaSuccess;
        if (a.workspace != nullptr && a.workspace_bytes >= s.bytes) {
            s.base = static_cast<char *>(a.workspace);
            return cudaSuccess;
        }
        const cudaError_t e = scratch_alloc(dev, &own, s.bytes, st);
        s.base = static_cast<char *>(own);
        return e;
    }
    cudaError_t give(cudaError_t e) {
        if (own == nullptr) return e;
        const cudaError_t f = scratch_free(own, st);
        return e == cudaSuccess ? f : e;
    }
};

template <class T, int P>
cudaError_t forward(const DeviceInfo &dev, const GatedArgs &a, cudaStream_t st) {
    Scratch s;
    Inputs in;
    plan_inputs<T, P>(a, in, s);
    Memory memory{st};
    cudaError_t e = memory.take(dev, s, a);
    if (e != cudaSuccess) return e;
    e = pack_inputs<T, P>(a, in, s, st);
    if (e == cudaSuccess) {
        GemmArgs g = gemm_args(dev, a);
        g.M = a.rows, g.N = a.F, g.kb = int(ceil_div(a.C, BK)), g.kb0 = g.kb;
        const GemmPlan p = plan_gemm(dev.sm_count, G_FWD, P, g.M, g.N, g.kb);
        g.mt = int(ceil_div(a.rows, p.rows())), g.per = p.per;
        g.nt = int(ceil_div(a.F, p.BN / 2));
        g.out = a.y, g.vec = a.F % (16 / sizeof(T)) == 0 && aligned16(a.y);
        GemmMaps m{};
        const bool ok = make_map3(&m.a0, in.x, BM) && make_map3(&m.b0, in.wg, p.BN / 2) &&
                        make_map3(&m.b1, in.wu, p.BN / 2) &&
                        (P > 1 || !g.vec || make_tile_map(&m.o0, a.y, a.rows, a.F, a.F));
        e = ok ? run_gemm<G_FWD, P>(dev, m, g, p, in.any(), st) : cudaErrorInvalidValue;
    }
    return memory.give(e);
}

template <class T, int P>
cudaError_t backward(const DeviceInfo &dev, const GatedArgs &a, cudaStream_t st) {
    BackwardPlan b = plan_backward<T, P>(dev, a);
    Scratch &s = b.s;
    Inputs &in = b.in;
    const int ld = b.ld, kf = b.kf, kr = b.kr;
    const GemmPlan p = b.pg, px = b.px, pw = b.pw;
    const size_t part_x = b.part_x, part_w = b.part_w, part_b = b.part_b;
    Memory memory{st};
    cudaError_t e = memory.take(dev, s, a);
    if (e != cudaSuccess) return e;
    e = pack_inputs<T, P>(a, in, s, st);
    Operand d[2];
    for (int i = 0; i < 2; ++i) {
        d[i].rows = a.rows, d[i].cols = a.F, d[i].ld = ld, d[i].parts = grad_parts(P);
        d[i].p = reinterpret_cast<const bf16 *>(s.base + b.d_at) +
                 int64_t(i) * d[i].parts * a.rows * ld;
    }
    auto partials = [&](size_t at) { return reinterpret_cast<float *>(s.base + at); };
    if (e == cudaSuccess) {
        GemmArgs g = gemm_args(dev, a);
        g.M = a.rows, g.N = a.F, g.kb = int(ceil_div(a.C, BK)), g.kb0 = g.kb;
        g.mt = int(ceil_div(a.rows, p.rows())), g.per = p.per;
        g.nt = int(ceil_div(a.F, p.BN / 2));
        g.d = const_cast<bf16 *>(d[0].p), g.ld = ld;
        g.dvec = a.F % (16 / sizeof(T)) == 0 && aligned16(a.dy);
        if (a.dbg) g.bpart = partials(part_b);
        GemmMaps m{};
        const bool ok = make_map3(&m.a0, in.x, BM) &&
                        make_map3(&m.b0, in.wg, p.BN / 2) &&
                        make_map3(&m.b1, in.wu, p.BN / 2) &&
                        (P == 1 || (make_map3(&m.o0, d[0], 32, 16) &&
                                    make_map3(&m.o1, d[1], 32, 16))) &&
                        (P > 1 || !g.dvec || make_tile_map(&m.dy, a.dy, a.rows, a.F, a.F));
        e = ok ? run_gemm<G_GRAD, P>(dev, m, g, p, in.any(), st) : cudaErrorInvalidValue;
    }
    if (e == cudaSuccess && a.dx) {
        GemmArgs g = gemm_args(dev, a);
        g.M = a.rows, g.N = a.C, g.kb0 = kf, g.kb = 2 * kf;
        g.mt = int(ceil_div(a.rows, px.rows()));
        g.nt = int(ceil_div(a.C, px.BN)), g.nsplit = px.nsplit, g.per = px.per;
        g.out = a.dx, g.vec = a.C % (16 / sizeof(T)) == 0 && aligned16(a.dx);
        g.part = partials(part_x);
        GemmMaps m{};
        const bool ok = make_map3(&m.a0, d[0], BM) &&
                        make_map3(&m.a1, d[1], BM) &&
                        make_map3(&m.b0, in.wg, 64) && make_map3(&m.b1, in.wu, 64);
        e = ok ? run_gemm<G_DX, P>(dev, m, g, px, true, st) : cudaErrorInvalidValue;
        if (e == cudaSuccess && g.nsplit > 1)
            e = join<T>(g.part, g.nsplit, a.rows, a.rows, a.C, a.dx, nullptr, st);
    }
    if (e == cudaSuccess && a.dwg) {
        GemmArgs g = gemm_args(dev, a);
        g.M = a.F, g.N = a.C, g.kb = kr, g.kb0 = kr;
        g.mt = 2 * int(ceil_div(a.F, pw.rows()));
        g.nt = int(ceil_div(a.C, pw.BN)), g.nsplit = pw.nsplit, g.per = pw.per;
        g.out = a.dwg, g.out2 = a.dwu;
        g.vec = a.C % (16 / sizeof(T)) == 0 && aligned16(a.dwg) && aligned16(a.dwu);
        g.part = partials(part_w);
        GemmMaps m{};
        const bool ok = make_map3(&m.a0, d[0], 64) && make_map3(&m.a1, d[1], 64) &&
                        make_map3(&m.b0, in.x, 64);
        e = ok ? run_gemm<G_DW, P>(dev, m, g, pw, true, st) : cudaErrorInvalidValue;
        if (e == cudaSuccess && g.nsplit > 1)
            e = join<T>(g.part, g.nsplit, 2 * int64_t(a.F), a.F, a.C, a.dwg, a.dwu, st);
    }
    if (e == cudaSuccess && a.dbg) {
        e = launch(true, gated_bias_kernel<T>, unsigned(ceil_div(2 * a.F, 32)), dim3(32, 32), 0, st,
                   partials(part_b), int(4 * p.CG * ceil_div(a.rows, p.rows())), a.F,
                   static_cast<T *>(a.dbg), static_cast<T *>(a.dbu));
    }
    return memory.give(e);
}

}  // namespace

size_t gated_tc_scratch(const DeviceInfo &dev, const GatedArgs &a, int dtype, bool backward) {
    if (backward)
        return (dtype == PC_F32 ? plan_backward<float, 3>(dev, a) : plan_backward<bf16, 1>(dev, a))
            .s.bytes;
    Scratch s;
    Inputs in;
    if (dtype == PC_F32)
        plan_inputs<float, 3>(a, in, s);
    else
        plan_inputs<bf16, 1>(a, in, s);
    return s.bytes;
}
cudaError_t gated_tc_forward(const DeviceInfo &dev, const GatedArgs &a, int dtype,
                             cudaStream_t st) {
    return dtype == PC_F32 ? forward<float, 3>(dev, a, st) : forward<bf16, 1>(dev, a, st);
}
cudaError_t gated_tc_backward(const DeviceInfo &dev, const GatedArgs &a, int dtype,
                              cudaStream_t st) {
    return dtype == PC_F32 ? backward<float, 3>(dev, a, st) : backward<bf16, 1>(dev, a, st);
}

}  // namespace pcn
