// sq_fp8.cu -- products of e4m3 codes with one power-of-two scale for each block of 128, dense or
// grouped by expert, on tcgen05 (kind::mxf8f6f4 with block scales, fp32 sums in tensor memory).
//
//   forward   y[m, n]  = sum_k x[m, k] W[n, k]
//   gated     h[m, n]  = act(g) u,  g and u such sums of two weights
//   backward  dx[m, k] = sum_n dy[m, n] W[n, k], gated: sum over both weights
//
// Tensor-memory lanes hold tokens, columns output channels (few rows: see below).  A = the rows' codes
// (K-major); B = the weight's codes, K-major forward and N-major backward (they are read as they lie,
// never transposed).  Gated: B is a tile of the gate's rows and the same rows of the up projection, so
// that both sums of an output lie in one lane and the activation is applied as they leave tensor
// memory; backward the summed axis simply runs through both weights.
//
// Scales.  The tensor cores take one e8m0 byte for each row of A and of B and 32 values; a block of
// 128 is four of them with the same byte.  A word holds the bytes of a group of four neighbouring
// blocks, the instruction names the one to use, so that a row's scales for 512 values are one 32-bit
// word in tensor memory.  Sets of four feeder warps, one for each 32 lanes, write the words there, up
// to four groups ahead of the products.  (Copied by the issuing thread from shared memory instead,
// tcgen05.cp, each group held the tensor pipe up by some 600 cycles.)
//
// Few rows (FUSE, see fp8_rounds_rows): the feeders round the rows themselves, straight into the operand's
// shared-memory layout, and the call is one kernel.  There the operands change places: lanes hold up to 128
// channels (gated: the gate's in lanes 0 .. 63, the up projection's from 64 on), columns 16 or 32 rows.  With
// the rows as lanes, the tensor cores multiplied 128 of them for the 8 that were there: 8 x 16384 x 6144,
// gated, took 36 us, and 42 once the power cap had lowered the clocks, instead of 33.5 for as long as it runs.
//
// CTA (CG = 1, tiles of 128 tokens x up to 224 columns, backward 256) or CTA pair (CG = 2, 256 x up to
// 256), one CTA per SM, persistent: 8 epilogue warps (few rows: 4), TMA producers, feeders (few rows: two
// sets), and an issuer that also allocates tensor memory.  Outputs leave by TMA where a warp's 32 rows
// are all the tile's.  Gated forwards are at the limit of 128 registers a thread, by which the
// pair's spills 24 bytes (its epilogue holds 32 columns of both sums).
//
// Accuracy: see kSumGroups.
//
// Few tiles (CG = 1): a cluster of CTAs shares a tile, each with some of the groups, and joins the
// partial sums over distributed shared memory, in the order of the CTAs' ranks.
//
// What bounds it, in a stream of calls (us a call with the rounding; many at a stretch in brackets, where the
// power cap lowers the clocks):
//   4480 x 16384 x 6144   forward 334 (387), gradient 365 (431), gated 692 (801): tensor pipe 89 to 92 % active
//                         (forward alone 295 us, 3.06 PFLOP/s), then the power cap
//   8300 rows of 61 experts, gated 2 x 1408 x 2048   88 (105): 59 % of DRAM, tiles of a few rows more than 128
//   8 x 16384 x 6144, gated   33.5: the weights' bytes at 6.0 TB/s
//   32 rows of 27 experts, 2816 x 2048   30.4 (156 MB: 5.1 TB/s): the last tiles
//   1 x 6144 x 6144       10.0: start, 38 MB from DRAM, the join of two CTAs' sums
//   777 x 4240 x 2832     21.0: one round of tiles behind the rounding
#include <cuda.h>

#include <type_traits>

#include "sq_fp8.cuh"
#include "sq_kernels.h"
#include "sq_ptx.cuh"
#include "sq_w8a8.cuh"

namespace sq {

enum Fp8Mode { kFp8Fwd = 0, kFp8Gated = 1, kFp8Bwd = 2 };

constexpr int kFChunk = 128;                      // summed values (bytes) of a shared-memory row
// Tensor memory: two accumulators from columns 0 and 224 on (0 and 192 where a tile has 256 columns:
// they share 64), then four buffers of 16 columns with a group's scales, 8 for B and 4 for A.  Fewer
// buffers would not do: from the end of a group's products to the next scales in its buffer of both
// CTAs it takes some 2500 cycles, more than a group's products (4480 x 16384 x 6144: 405 us with two,
// 337 with four).
constexpr int kFBufs = 4;
constexpr int kFPatchBytes = 32 * 64;             // a warp's 32 rows x 64 bytes on their way out
constexpr int kFuseRows = 16;
constexpr int kFMaxSplit = 8;
constexpr int kFPartBytes = 24 * 1024;            // FUSE: places for the other CTAs' sums
constexpr int kFUpRow = 64;                       // FUSE, gated: lane of the up projection's first channel
// Accuracy: each tensor-core step of 32 products cuts the fp32 sum that it adds to towards zero, and the loss grows
// faster than the length.  Relative to the result's size it is 1e-7 for 2048 values, 5e-7 for 6144, 2e-6 for 16384, 5e-6 for
// 32768 (3e-5 for 2^17, 4e-4 for 2^20).  So a CTA's accumulator takes at most so many groups of an fp32 result's sum at a
// time, and the parts, a launch each, are added to y.  (In tensor memory there is no room for a third accumulator
// beside wide tiles.)  Gradient of 4480 x 131072 x 6144: 2.98 ms, in one part 2.91; 300 x 131072 x 4096: 0.48, 0.38.
constexpr int kSumGroups = 64;
constexpr int kPrefetchBytes = 64 * 1024;         // of weight into L2 before the kernel in front has ended, each CTA

template <int CG, int MODE, bool FUSE>
struct Fp8Cfg {
    static constexpr int kEpi = FUSE ? 4 : 8;     // epilogue warps
    static constexpr int kProducers = CG == 2 || FUSE ? 2 : 3;
    static constexpr int kSets = FUSE ? 2 : 1;    // of four feeder warps
    static constexpr int kThreads = 32 * (kEpi + kProducers + 4 * kSets + 1);
    static constexpr uint32_t kTmemCols = 512, kScaleCol = 448;
    static constexpr int kMaxStages = CG == 2 ? 12 : 24;
    // shared memory: the ring, then
    //   patches of the stores; FUSE: a split tile's sums from the other CTAs, and the up projection's of
    //   four warps.  (CG = 1: the MMA reads 128 rows of A, up to 16 KB behind the last stage.)
    static constexpr int kPatches = CG == 2 && MODE != kFp8Bwd ? 2 : 1;       // of an epilogue warp
    static constexpr int kPatchBytes = FUSE ? kFPartBytes + 4096 : 8 * kPatches * kFPatchBytes;
    static constexpr int kPlanOff = kPatchBytes;
    static constexpr int kFeedOff = kPlanOff + (2 * kMaxExperts + 4) * 4;     // [sets][2][32] words (FUSE)
    static constexpr int kBarOff = kFeedOff + kSets * 2 * 32 * 4;
    // full, empty, sf_full, sf_empty, acc_full[2], acc_empty[2], drain, peers, parts
    static constexpr int kNumBars = 2 * kMaxStages + 2 * kFBufs + 7;
    static constexpr int kRestBytes = kBarOff + 8 * kNumBars + 16;
    static constexpr int kRing = (FUSE ? 184 : kPatches == 2 ? 180 : 192) * 1024;
    static constexpr int kSmemBytes = kRing + kRestBytes + 1024;
    // e4m3 x e4m3, e8m0 scales; the weight N-major backward; 128 CG rows (columns / 8 << 17 comes at run time)
    static constexpr uint32_t kIdesc = (1u << 23) | (MODE == kFp8Bwd ? 1u << (FUSE ? 15 : 16) : 0u) | ((uint32_t)(8 * CG) << 24);
    static constexpr uint32_t kWStep16 = MODE == kFp8Bwd ? (32u * 128u) >> 4 : 2u;   // the weight's descriptor step per MMA
};

struct Fp8Args {
    const int32_t *offsets;
    const uint32_t *words;    // row scales, [halves * groups, M]
    const uint16_t *x, *g, *u;   // FUSE: the rows themselves
    const uint8_t *ws[2];     // weight scales, [E, nbs, kbs]
    void *y;
    uint16_t *g_out, *u_out;
    uint32_t *status;
    uint8_t *zero[3];         // FUSE: outputs whose rows outside every expert become 0
    int64_t zero_row_bytes[3];
    int64_t M, width;         // rows, and columns of y
    int64_t L;                // length of the summed axis (of one weight)
    int E, act, out_bf16, finite_check, keep_status;
    int nbs, kbs;             // blocks of a weight along N and K
    int blocks;               // blocks of the summed axis (of one weight)
    int halves;               // weights that the sum runs through
    int tile;                 // output channels of a tile
    int a_rows;               // rows that a stage (FUSE: a group) reserves
    int boxed_rows;           // up to so many rows come in boxes of 32
    int per;                  // chunks of a stage: 1, 2 or 4
    int stages;
    int prefetch;             // FUSE: chunks of a tile fetched into L2 before the kernel in front has ended
    int split;                // CTAs of a cluster that share a tile (CG = 1)
    int slot1;                // column of the second accumulator
    int lo, hi;               // groups of the sum that this launch takes
};

template <int CG>
__device__ __forceinline__ bool fp8_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag, uint32_t *status)
{
    return CG == 2 ? mbar_wait_cluster(bar, parity, abort_flag, status) : mbar_wait(bar, parity, abort_flag, status);
}

// warp-uniform bounded wait: lane 0 polls, the verdict is broadcast
template <int CG>
__device__ __forceinline__ bool fp8_warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag,
                                              uint32_t *status, int lane)
{
    int ok = 1;
    if (lane == 0)
        ok = fp8_wait<CG>(bar, parity, abort_flag, status) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

__device__ __forceinline__ bool one_lane()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// A warp's place for 32 rows x 64 bytes on their way out, or two in turn.
struct Fp8Patch {
    uint8_t *mem;
    int lane, turn;
};

__device__ __forceinline__ uint32_t sum_bits(uint32_t a, uint32_t b)
{
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}

// One warp's 32 rows x 64 bytes to y through its patch: by TMA (map, box of 64 bytes x 32 rows at x, y),
// or where not all of them exist (map NULL) row by row, so that a row's 64 bytes leave in one run.
// dst: row 0's first byte; the first `rows` rows and `bytes` bytes (a multiple of 16) of each exist.  ADDS (map
// NULL): fp32 values, added to what is there.
template <int PATCHES, bool ADDS>
__device__ __forceinline__ void store_rows64(const uint32_t (&v)[16], Fp8Patch &out, const CUtensorMap *map, int x,
                                             int y, uint8_t *dst, int64_t row_bytes, int rows, int bytes)
{
    const int lane = out.lane;
    uint8_t *patch = out.mem + (PATCHES == 2 ? out.turn * kFPatchBytes : 0);
    out.turn ^= 1;
    if (lane == 0) {                              // what was in it has left
        if (PATCHES == 2)
            bulk_wait_group_read1();
        else
            bulk_wait_group_read0();
    }
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 4; ++p)                   // (the order that the 64-byte swizzle of the map has)
        *reinterpret_cast<uint4 *>(patch + lane * 64 + ((p ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
    if (map) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && rows > 0)
            tma_store_2d(map, smem_u32(patch), x, y);
    } else {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (lane >> 2), p = lane & 3;
            uint4 w = *reinterpret_cast<const uint4 *>(patch + row * 64 + ((p ^ ((row >> 1) & 3)) << 4));
            if (row < rows && 16 * p < bytes) {
                uint4 *to = reinterpret_cast<uint4 *>(dst + row * row_bytes + 16 * p);
                if constexpr (ADDS) {
                    const uint4 o = *to;
                    w = make_uint4(sum_bits(w.x, o.x), sum_bits(w.y, o.y), sum_bits(w.z, o.z), sum_bits(w.w, o.w));
                }
                *to = w;
            }
        }
        __syncwarp();
    }
    if (lane == 0)
        bulk_commit_group();                      // (empty without a map: the patches are counted in groups)
}

// 32 neighbouring columns of y from fp32 values, as bf16 or fp32, through the patch; the first `cols` of them
// and `rows` rows exist.
template <int PATCHES, bool ADDS>
__device__ __forceinline__ void store_cols(const float (&o)[32], Fp8Patch &out, const CUtensorMap *map, void *y,
                                           int64_t row, int64_t col, int64_t width, int rows, int cols, bool bf16)
{
    uint8_t *dst = reinterpret_cast<uint8_t *>(y) + (bf16 ? 2 : 4) * (row * width + col);
    uint32_t v[16];
    if (bf16) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = f32x2_to_bf16x2_bits(o[2 * i], o[2 * i + 1]);
        store_rows64<PATCHES, false>(v, out, map, (int)col, (int)row, dst, 2 * width, rows, 2 * cols);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = __float_as_uint(o[16 * h + i]);
            store_rows64<PATCHES, ADDS>(v, out, map, (int)col + 16 * h, (int)row, dst + 64 * h, 4 * width, rows,
                                        4 * (cols - 16 * h));
        }
    }
}

// What a group of four blocks is: number g2 of the tile's, of weight `half`.
struct Fp8Walk {
    int groups, blocks;       // of one weight
    int lo, hi;               // the CTA's groups of a tile

    __device__ __forceinline__ void at(int g2, int &half, int &grp, int &live) const
    {
        half = g2 >= groups ? 1 : 0;
        grp = g2 - half * groups;
        live = min(kFp8Group, blocks - kFp8Group * grp);
    }
};

// ADDS: fp32 results, added to what y holds
template <int CG, int MODE, bool FUSE, bool ADDS>
__global__ void __launch_bounds__(Fp8Cfg<CG, MODE, FUSE>::kThreads, 1)
    sq_fp8_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmX32,
                  const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmW2,
                  const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmG,
                  const __grid_constant__ CUtensorMap tmU, const Fp8Args args)
{
    using Cfg = Fp8Cfg<CG, MODE, FUSE>;
    constexpr bool BWD = MODE == kFp8Bwd, GATED = MODE == kFp8Gated;
    static_assert(!FUSE || CG == 1, "few rows take tiles of one CTA");
    static_assert(!ADDS || !GATED, "the activation needs the whole sums");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *rest = smem + Cfg::kRing;
    int32_t *plan_mem = reinterpret_cast<int32_t *>(rest + Cfg::kPlanOff);
    uint64_t *bars = reinterpret_cast<uint64_t *>(rest + Cfg::kBarOff);
    const uint32_t bar_full = smem_u32(bars);                          // leader: both CTAs' stage ready
    const uint32_t bar_empty = bar_full + 8 * Cfg::kMaxStages;         // each CTA: its stage may be refilled
    const uint32_t bar_sf_full = bar_empty + 8 * Cfg::kMaxStages;      // leader: a group's scales (FUSE: and rows) ready
    const uint32_t bar_sf_empty = bar_sf_full + 8 * kFBufs;            // each CTA: the group's products are done
    const uint32_t bar_acc_full = bar_sf_empty + 8 * kFBufs;           // each CTA: accumulator ready
    const uint32_t bar_acc_empty = bar_acc_full + 16;                  // leader: accumulator read
    const uint32_t bar_drain = bar_acc_empty + 16;                     // leader: every MMA finished
    const uint32_t bar_peers = bar_drain + 8;                          // split: the other CTAs' rings may be written
    const uint32_t bar_parts = bar_peers + 8;                          // split: bytes of their sums
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + Cfg::kNumBars);
    volatile uint32_t *abort_flag = tmem_holder + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int split = CG == 1 ? args.split : 1;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;            // in the pair
    const int part = split > 1 ? (int)cluster_ctarank() : 0;           // of the tile's groups
    const bool leader = rank == 0;
    // Roles: epilogue, producers, feeders, issuer.  A warp reaches the 32 lanes of tensor memory that its
    // number modulo 4 gives: the epilogue and a set of feeders need all four.
    constexpr int kIssuer = Cfg::kEpi + Cfg::kProducers + 4 * Cfg::kSets;
    constexpr int kProducer = Cfg::kEpi, kFeeder = kProducer + Cfg::kProducers;
    const bool producer = warp >= kProducer && warp < kProducer + Cfg::kProducers;
    const bool feeder = warp >= kFeeder && warp < kFeeder + 4 * Cfg::kSets;

    if (threadIdx.x == 0) {
        for (int st = 0; st < Cfg::kMaxStages; ++st) {
            mbar_init(bar_full + 8 * st, 1);
            mbar_init(bar_empty + 8 * st, 1);
        }
        for (int i = 0; i < kFBufs; ++i) {
            mbar_init(bar_sf_full + 8 * i, 4 * CG);
            mbar_init(bar_sf_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_acc_full + 8 * i, 1);
            mbar_init(bar_acc_empty + 8 * i, CG * Cfg::kEpi);
        }
        mbar_init(bar_drain, 1);
        mbar_init(bar_peers, max(split - 1, 1));
        mbar_init(bar_parts, 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == kIssuer) {
        if (CG == 2) {
            tmem_alloc2(smem_u32(tmem_holder), Cfg::kTmemCols);
            tmem_relinquish2();
        } else {
            tmem_alloc(smem_u32(tmem_holder), Cfg::kTmemCols);
            tmem_relinquish();
        }
    }
    if (warp == kProducer && lane == 0) {
        if (!FUSE)
            prefetch_tmap(&tmX);
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmW2);
    }
    // The kernel in front: without FUSE it is this call's rounding, which lets this one start after its
    // own wait, so that the offsets and the weight are there; with FUSE it can be any.
    if (FUSE && args.E > 0)
        grid_dep_wait();
    grid_dep_launch();                            // the next call may be set up
    I8Plan plan;
    plan.E = args.E > 0 ? args.E : 1;
    plan.start = plan_mem;
    plan.prefix = plan_mem + kMaxExperts + 1;
    plan.wts = (int)((args.width + args.tile - 1) / args.tile);
    plan.tok_tile = 128 * CG;
    if (args.E > 0) {
        plan.build(args.offsets, args.M, threadIdx.x, Cfg::kThreads);
    } else if (threadIdx.x == 0) {
        plan.start[0] = plan.prefix[0] = 0;
        plan.start[1] = (int32_t)args.M;
        plan.prefix[1] = (int32_t)((args.M + plan.tok_tile - 1) / plan.tok_tile);
    }
    tc_fence_before();
    if (CG == 2 || split > 1)
        cluster_sync();                           // barriers of every CTA initialised, TMEM allocated
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;

    const int tiles = plan.tiles();
    const int unit = (int)blockIdx.x / (CG * split);
    const int units = (int)gridDim.x / (CG * split);
    const int per = args.per;
    const int T = args.tile;
    const int b_rows = GATED ? (CG == 2 ? T : 2 * T) : T / CG;         // rows (backward: columns) of B in this CTA
    const int cols = GATED ? 2 * T : T;                                // columns of the accumulator
    const int a_bytes = args.a_rows * kFChunk;                         // of a chunk
    const int boxes = BWD ? (b_rows + 127) / 128 : 1;                  // of 128 columns (backward)
    const int b_bytes = (BWD ? 128 * boxes : b_rows) * kFChunk;
    const int chunk_bytes = FUSE ? (GATED ? (kFUpRow + T) * kFChunk : b_bytes) : a_bytes + b_bytes;
    const int stage_bytes = per * chunk_bytes;
    const int stages = args.stages;
    const uint32_t slot1 = (uint32_t)args.slot1;
    const int shared_cols = max(cols - (int)slot1, 0);                 // that the accumulators share
    const int ring0 = FUSE ? kFBufs * kFp8Group * a_bytes : 0;         // FUSE: the rows of four groups, then the stages
    Fp8Walk walk;
    walk.blocks = args.blocks;
    walk.groups = (args.blocks + kFp8Group - 1) / kFp8Group;
    const int first = GATED ? 0 : args.lo, many = GATED ? walk.groups * args.halves : args.hi - args.lo;
    walk.lo = first + many * part / split;
    walk.hi = first + many * (part + 1) / split;

    if (producer) {
        // ------------------------------------------------------------ producers (every CTA)
        // Producer p takes every P-th stage of the unit's work (a copy takes a thread some 100 cycles to
        // issue, a stage's waiting and counting more).
        constexpr int P = Cfg::kProducers;
        const int p = warp - kProducer;
        const bool issue = one_lane();
        const uint32_t s0 = smem_u32(smem) + ring0;
        // chunks of weight `half` from block `block` on, of tile t
        auto weight_box = [&](const I8Tile &t, int half, int x, auto &&copy) {
            const int n0 = t.wt * T;
            if (BWD) {
                for (int b = 0; b < boxes; ++b)
                    copy(half ? &tmW2 : &tmW, b * 128 * kFChunk, n0 + (int)rank * b_rows + 128 * b, x);
            } else if (GATED && CG == 1) {
                copy(&tmW, 0, x, n0);
                copy(&tmW2, (FUSE ? kFUpRow : T) * kFChunk, x, n0);
            } else if (GATED) {
                copy(rank ? &tmW2 : &tmW, 0, x, n0);
            } else {
                copy(&tmW, 0, x, n0 + (int)rank * b_rows);
            }
        };
        auto load_w = [&](uint32_t dst, uint32_t fb, const I8Tile &t, uint32_t bytes, int half, int block, int chunks) {
            if (leader)
                mbar_arrive_expect_tx(fb, chunks * bytes);
            for (int u = 0; u < chunks; ++u)
                weight_box(t, half, (block + u) * kFChunk, [&](const CUtensorMap *m, int at, int x, int y) {
                    tma_load_3d<CG>(dst + u * chunk_bytes + at, m, x, y, t.e, fb);
                });
        };
        // Rows of CTA r of the pair: of one expert at most t.rows.  Up to 96 come in boxes of 32, since an
        // expert's few rows would otherwise bring as many of the next ones' (and what is not brought is
        // multiplied all the same: the lanes behind the tile's rows are not looked at).
        auto live_of = [&](const I8Tile &t, int r) { return min(max(t.rows - 128 * r, 0), 128); };
        auto rows_brought = [&](int live) { return live > args.boxed_rows ? args.a_rows : (live + 31) / 32 * 32; };
        auto load_x = [&](uint32_t dst, uint32_t fb, int row, int live, int block, int chunks) {
            const bool whole = live > args.boxed_rows;
            for (int u = 0; u < chunks; ++u)
                for (int b = 0; b < live; b += whole ? 128 : 32) {
                    const CUtensorMap *m = whole ? &tmX : &tmX32;
                    if (CG == 2)
                        tma_load_2d_pair(dst + u * chunk_bytes + b * kFChunk, m, (block + u) * kFChunk, row + b, fb);
                    else
                        tma_load_2d(dst + u * chunk_bytes + b * kFChunk, m, (block + u) * kFChunk, row + b, fb);
                }
        };
        // a stage's bytes, of one chunk: both CTAs'
        auto bytes_of = [&](const I8Tile &t) {
            int rows = 0;
            for (int r = 0; !FUSE && r < CG; ++r)
                rows += rows_brought(live_of(t, r));
            return (uint32_t)(rows * kFChunk + CG * b_bytes);
        };
        const uint32_t w_off = FUSE ? 0 : a_bytes;
        int e = 0, early = 0;                     // stages of the first tile whose weight is on its way
        if (unit < tiles && !(FUSE && args.E > 0)) {
            const I8Tile t = plan.find(unit, e);
            const int most = FUSE ? args.prefetch / per : stages;
            int n = 0;
            for (int g2 = walk.lo; g2 < walk.hi && n < most; ++g2) {
                int half, grp, live;
                walk.at(g2, half, grp, live);
                for (int u = 0; u < live && n < most; u += per, ++n) {
                    const int block = kFp8Group * grp + u, chunks = min(per, live - u);
                    if (!issue || n % P != p)
                        continue;
                    if (FUSE)                     // (into L2: the kernel in front may have written the weight)
                        for (int v = 0; v < chunks; ++v)
                            weight_box(t, half, (block + v) * kFChunk,
                                       [&](const CUtensorMap *m, int, int x, int y) { tma_prefetch_3d(m, x, y, t.e); });
                    else
                        load_w(s0 + w_off + n * stage_bytes, bar_full + 8 * n, t, bytes_of(t), half, block, chunks);
                }
            }
            early = FUSE ? 0 : n;
        }
        if (!(FUSE && args.E > 0))
            grid_dep_wait();                      // codes and scales of the rows
        e = 0;
        int stage = 0, turn = p;                  // turn: stages of the others before this warp's next one
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = unit; ok && tile < tiles; tile += units) {
            const I8Tile t = plan.find(tile, e);
            const uint32_t bytes = bytes_of(t);
            const int live_rows = live_of(t, (int)rank);
            for (int g2 = walk.lo; ok && g2 < walk.hi; ++g2) {
                int half, grp, live;
                walk.at(g2, half, grp, live);
                const int row = t.row0 + half * (int)args.M + (int)rank * 128;
                for (int u = 0; u < live; u += per) {
                    if (--turn < 0) {
                        turn = P - 1;
                        const int block = kFp8Group * grp + u, chunks = min(per, live - u);
                        const uint32_t dst = s0 + stage * stage_bytes, fb = bar_full + 8 * stage;
                        const bool fresh = early <= 0;
                        if (fresh && !mbar_wait(bar_empty + 8 * stage, phase ^ 1u, abort_flag, args.status)) {
                            ok = false;
                            break;
                        }
                        if (issue) {
                            if (fresh)
                                load_w(dst + w_off, fb, t, bytes, half, block, chunks);
                            if (!FUSE)
                                load_x(dst, fb, row, live_rows, block, chunks);
                        }
                    }
                    --early;
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        // let every load that was issued land (and be consumed) before the CTA exits
        for (int st = 0; st < stages; ++st) {
            (void)mbar_wait(bar_empty + 8 * stage, phase ^ 1u, abort_flag, args.status);
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        __syncwarp();
    } else if (feeder) {
        // ------------------------------------------------------------ feeders (every CTA)
        // Warp q of a set writes lanes 32 q .. + 31 of tensor memory, which hold the same words in each
        // quarter: line l of column j is row 32 j + l.  Set s takes every S-th group.
        constexpr int S = Cfg::kSets;
        const int set = (warp - kFeeder) >> 2, q = warp & 3;
        const int wq = (warp - kFeeder) & 3;                           // (which of the set's four)
        const uint32_t full_leader = CG == 2 ? mapa_shared(bar_sf_full, 0) : bar_sf_full;
        const uint32_t sf_lanes = tmem_base + ((uint32_t)(32 * q) << 16) + Cfg::kScaleCol;
        const int64_t expert_blocks = (int64_t)args.nbs * args.kbs;
        uint32_t *const feeds = reinterpret_cast<uint32_t *>(rest + Cfg::kFeedOff) + 64 * set;
        if (!(FUSE && args.E > 0))
            grid_dep_wait();
        struct Item {
            I8Tile t;
            int tile, g2, number, e;
        };
        // this set's first or next group
        auto advance = [&](Item &it, int by) {
            it.number += by;
            it.g2 += by;
            while (it.g2 >= walk.hi) {
                it.tile += units;
                if (it.tile >= tiles)
                    return false;
                it.t = plan.find(it.tile, it.e);
                it.g2 -= walk.hi - walk.lo;
            }
            return true;
        };
        constexpr int R = FUSE ? 2 : 1;                    // rows of a warp fetched in advance
        struct Raw {
            uint32_t rw[FUSE ? 1 : 4], v;
            uint4 x[FUSE ? R : 1][2];
        };
        const bool pair_grad = FUSE && BWD && args.g != nullptr;       // the rows: gradients of a gated pair
        // a lane's 16 values of row r of the item's rows, 0 behind their end
        auto load16 = [&](const uint16_t *src, const Item &it, int64_t col, int r, uint4 (&a)[2]) {
            const bool live = r < it.t.rows && col < args.L;
            const uint4 *ptr = reinterpret_cast<const uint4 *>(src + ((int64_t)it.t.row0 + r) * args.L + col);
            a[0] = live ? __ldg(ptr) : make_uint4(0u, 0u, 0u, 0u);
            a[1] = live ? __ldg(ptr + 1) : make_uint4(0u, 0u, 0u, 0u);
        };
        auto fetch = [&](const Item &it, Raw &r) {
            int half, grp, live;
            walk.at(it.g2, half, grp, live);
            if constexpr (FUSE) {
                if (!pair_grad)
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        load16(args.x, it, (int64_t)grp * (kFp8Block * kFp8Group) + 16 * lane, wq + 4 * i, r.x[i]);
            } else {
                const int mine = min(max(it.t.rows - (int)rank * 128, 0), 128);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    r.rw[j] = 32 * j + lane < mine ? __ldg(args.words + (int64_t)it.g2 * args.M + it.t.row0 +
                                                           (int)rank * 128 + 32 * j + lane)
                                                   : 0u;
            }
            // bytes of the (at most three) blocks that the tile's channels lie in, four along the sum:
            // lanes 4 b + i; gated: the up projection's at 16 + 4 b + i
            const int ch = it.t.wt * T / kFp8Block + ((lane >> 2) & 3), kb = kFp8Group * grp + (lane & 3);
            const bool second = GATED ? lane >= 16 : half != 0;
            const int nb = BWD ? kb : ch, kk = BWD ? ch : kb;
            r.v = nb < args.nbs && kk < args.kbs
                      ? (uint32_t)__ldg((second ? args.ws[1] : args.ws[0]) + it.t.e * expert_blocks +
                                        (int64_t)nb * args.kbs + kk)
                      : 0u;
        };
        bool bad = false;
        // writes group `cur` to tensor memory (FUSE: and its rows to shared memory); false: gave up
        auto put = [&](const Item &cur, const Raw &raw) {
            const int buf = cur.number & (kFBufs - 1);
            // (few rows: a warp that gave up goes on, since the others of its set may wait for it)
            if (!fp8_warp_wait<CG>(bar_sf_empty + 8 * buf, ((uint32_t)(cur.number / kFBufs) & 1u) ^ 1u, abort_flag,
                                   args.status, lane) &&
                !FUSE)
                return false;
            uint32_t rw[4] = {0u, 0u, 0u, 0u}, ww[FUSE ? 4 : 8];     // words of the rows and of the weight
            if constexpr (FUSE) {
                // rows wq, wq + 4, ... of the tile, rounded into the operand's layout: rows of 128 bytes,
                // 16-byte piece i of row r at i ^ (r % 8); a lane has one piece
                int half, grp, live;
                walk.at(cur.g2, half, grp, live);
                const int64_t col = (int64_t)grp * (kFp8Block * kFp8Group) + 16 * lane;
                uint8_t *dst = smem + buf * (kFp8Group * a_bytes) + (lane >> 3) * a_bytes;
                const int n = cur.t.rows;
                // (two in turn: the barrier of the next group lies between a read and the next write)
                uint32_t *feed = feeds + 32 * ((cur.number / S) & 1);
                auto round_row = [&](int r, const auto &v) {
                    uint32_t byte;
                    const uint4 c = quantise16(v, byte, bad);
                    *reinterpret_cast<uint4 *>(dst + r * kFChunk + (((lane & 7) ^ (r & 7)) << 4)) = c;
                    const uint32_t word = scale_word(byte, lane);
                    if (lane == 0)
                        feed[r] = word;
                };
                if (pair_grad) {
                    for (int r = wq; r < n; r += 4) {
                        uint4 a[3][2];
                        load16(args.x, cur, col, r, a[0]);
                        load16(args.g, cur, col, r, a[1]);
                        load16(args.u, cur, col, r, a[2]);
                        uint64_t dg[8], du[8];
                        if (args.act == 0)
                            pair_gradients<0>(a[0], a[1], a[2], dg, du);
                        else
                            pair_gradients<1>(a[0], a[1], a[2], dg, du);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            dg[i] = half ? du[i] : dg[i];
                        round_row(r, dg);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        if (wq + 4 * i < n) {
                            round_row(wq + 4 * i, raw.x[i]);
                        }
                    for (int r = wq + 4 * R; r < n; r += 4) {
                        uint4 a[2];
                        load16(args.x, cur, col, r, a);
                        round_row(r, a);
                    }
                }
                fence_proxy_async_smem();
                named_barrier_sync(2 + set, 128);          // the set's words and rows are there
                rw[0] = lane < n ? feed[lane] : 0u;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    rw[j] = raw.rw[j];
            }
            uint32_t v = raw.v << (8 * (lane & 3));
            v |= __shfl_xor_sync(0xffffffffu, v, 1);
            v |= __shfl_xor_sync(0xffffffffu, v, 2);
            const int n0 = cur.t.wt * T;
#pragma unroll
            for (int j = 0; j < (FUSE ? 4 : 8); ++j) {
                const int r = 32 * j + lane, up = FUSE ? kFUpRow : T;
                const bool second = GATED && r >= up;
                const int ch = n0 + (second ? r - up : r);
                ww[j] = __shfl_sync(0xffffffffu, v, 4 * ((ch / kFp8Block - n0 / kFp8Block) & 3) + (second ? 16 : 0));
            }
            tc_fence_after();
            if constexpr (FUSE) {
                tmem_st_4cols(sf_lanes + 16 * buf, rw);
                tmem_st_4cols(sf_lanes + 16 * buf + 8, ww);
            } else {
                tmem_st_8cols(sf_lanes + 16 * buf, ww);
                tmem_st_4cols(sf_lanes + 16 * buf + 8, rw);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2)
                    mbar_arrive_cluster(full_leader + 8 * buf);
                else
                    mbar_arrive(full_leader + 8 * buf);
            }
            return true;
        };
        // kAhead groups in turn: the next ones' values are on their way while one is written (a load takes
        // 2 us and more while the weights stream).  Few rows: none, since two sets take turns anyway and more
        // code takes longer to fetch in a call that runs it once.
        constexpr int kAhead = FUSE ? 1 : 3;
        Item items[kAhead];
        Raw raws[kAhead];
        Item next;                                // the last one fetched
        next.tile = unit;
        next.e = 0;
        next.g2 = walk.lo;
        next.number = 0;
        bool more = unit < tiles && walk.lo < walk.hi;
        if (more) {
            next.t = plan.find(unit, next.e);
            more = advance(next, set);
        }
        if constexpr (kAhead == 1) {
#pragma unroll 1
            while (more) {
                fetch(next, raws[0]);
                if (!put(next, raws[0]))
                    break;
                more = advance(next, S);
            }
        } else {
            int held = 0;                         // fetched, not yet written
#pragma unroll
            for (int d = 0; d < kAhead - 1; ++d)
                if (more) {
                    items[d] = next;
                    fetch(next, raws[d]);
                    ++held;
                    more = advance(next, S);
                }
            bool ok = true;
            while (ok && held > 0) {
#pragma unroll
                for (int d = 0; d < kAhead; ++d) {
                    if (!ok || held == 0)
                        break;
                    if (more) {
                        items[(d + kAhead - 1) % kAhead] = next;
                        fetch(next, raws[(d + kAhead - 1) % kAhead]);
                        ++held;
                        more = advance(next, S);
                    }
                    ok = put(items[d], raws[d]);
                    --held;
                }
            }
        }
        if (FUSE && args.finite_check && bad)
            atomicOr(args.status, kStatusNonfinite);
        __syncwarp();
    } else if (warp == kIssuer) {
        // ------------------------------------------------------------ MMA issuer (leader)
        if (leader) {
            // (few rows: the kernel in front may be any, and longer than a wait for the feeders may take)
            if (FUSE && args.E == 0)
                grid_dep_wait();
            const bool issue = one_lane();
            const uint32_t s0 = smem_u32(smem) + ring0;
            // the rows' and the weight's descriptors (backward: from 128 columns of the weight to the next 128 it
            // is 16 KB)
            const uint64_t dR = sdesc_sw128(FUSE ? smem_u32(smem) : s0);
            const uint32_t dR0 = (uint32_t)dR, dW0 = ((uint32_t)sdesc_sw128(s0 + (FUSE ? 0 : a_bytes)) & 0xFFFFu) |
                                                     (BWD ? (128u * kFChunk >> 4) << 16 : 1u << 16);
            const uint32_t desc_hi = (uint32_t)(dR >> 32);
            const uint32_t stage16 = stage_bytes >> 4, chunk16 = chunk_bytes >> 4, a16 = a_bytes >> 4;
            const uint32_t idesc0 = Cfg::kIdesc | (uint32_t)((FUSE ? args.a_rows : cols) >> 3) << 17;
            auto commit = [&](uint32_t bar) {
                if (CG == 2)
                    tc_commit2_both(bar);
                else
                    tc_commit(bar);
            };
            // One thread issues, the warp runs the loops on uniform values.  What lies between two stages'
            // products is time in which the tensor pipe runs dry (it takes few products in advance), so a
            // whole group is unrolled, for each number of chunks that a stage can have.
            auto run = [&](auto chunks) {
                constexpr int PER = decltype(chunks)::value;
                int stage = 0;
                uint32_t phase = 0, off = 0;               // off: the stage's, in 16 bytes
                uint32_t buf = 0, buf_phase = 0;
                int count = 0;
                for (int tile = unit; tile < tiles; tile += units, ++count) {
                    const uint32_t acc = tmem_base + ((count & 1) ? slot1 : 0u);
                    // the tile before last (same accumulator) has left tensor memory; where the accumulators
                    // overlap, the last one's shared columns have (and all of the one before)
                    const int last = count - (shared_cols > 0 ? 1 : 2);
                    if (last >= 0 && !fp8_wait<CG>(bar_acc_empty + 8 * (last & 1), (uint32_t)((last >> 1) & 1),
                                                   abort_flag, args.status))
                        return;
                    uint32_t sum = 0;
                    int left = walk.blocks - kFp8Group * (walk.lo >= walk.groups ? walk.lo - walk.groups : walk.lo);
                    for (int g2 = walk.lo; g2 < walk.hi; ++g2) {
                        if (!fp8_wait<CG>(bar_sf_full + 8 * buf, buf_phase, abort_flag, args.status))
                            return;
                        const uint32_t sf = tmem_base + Cfg::kScaleCol + 16 * buf;
#pragma unroll
                        for (int u0 = 0; u0 < kFp8Group; u0 += PER) {
                            if (u0 > 0 && u0 >= left)
                                break;
                            if (!fp8_wait<CG>(bar_full + 8 * stage, phase, abort_flag, args.status))
                                return;
                            tc_fence_after();
                            if (issue) {
#pragma unroll
                                for (int u = 0; u < PER; ++u) {
                                    if (u > 0 && u0 + u >= left)
                                        break;
                                    const uint32_t idesc = idesc0 | (uint32_t)(u0 + u) << 4 | (uint32_t)(u0 + u) << 29;
                                    const uint32_t r = FUSE ? dR0 + (buf * kFp8Group + u0 + u) * a16
                                                            : dR0 + off + u * chunk16;
                                    const uint32_t w = dW0 + off + u * chunk16;
#pragma unroll
                                    for (int k = 0; k < kFChunk / 32; ++k) {
                                        const uint32_t rk = r + 2 * k, wk = w + Cfg::kWStep16 * k;
                                        mma_fp8<CG>(acc, FUSE ? wk : rk, FUSE ? rk : wk, desc_hi, idesc, sf + 8, sf,
                                                    u0 + u + k > 0 ? 1u : sum);
                                    }
                                }
                                commit(bar_empty + 8 * stage);
                            }
                            off += stage16;
                            if (++stage == stages) {
                                stage = 0;
                                off = 0;
                                phase ^= 1u;
                            }
                        }
                        if (issue)
                            commit(bar_sf_empty + 8 * buf);
                        sum = 1u;
                        if (++buf == (uint32_t)kFBufs) {
                            buf = 0;
                            buf_phase ^= 1u;
                        }
                        left -= kFp8Group;
                        if (left <= 0)
                            left = walk.blocks;            // the second weight's
                    }
                    if (issue)
                        commit(bar_acc_full + 8 * (count & 1));
                }
            };
            if (per == 1)
                run(std::integral_constant<int, 1>());
            else if (per == 2)
                run(std::integral_constant<int, 2>());
            else
                run(std::integral_constant<int, 4>());
            // all issued MMAs must finish before tensor memory is released
            if (issue) {
                if (CG == 2)
                    tc_commit2_local(bar_drain);
                else
                    tc_commit(bar_drain);
            }
            (void)mbar_wait(bar_drain, 0, abort_flag, args.status);
        }
        __syncwarp();
    } else if constexpr (FUSE) {
        // ------------------------------------------------------------ epilogue, few rows (every CTA)
        // A lane of warp q holds channel 32 q + lane of the tile (gated: the up projection's from kFUpRow on), a
        // column a row, 16 columns at a time.
        const int q = warp, slots = args.a_rows;
        const bool second = GATED && 32 * q >= kFUpRow;
        const int ch = 32 * q + lane - (second ? kFUpRow : 0);
        const bool ybf = args.out_bf16 != 0;
        float *const exchange = reinterpret_cast<float *>(rest + kFPartBytes) + (q & 1) * 512 + lane;
        int count = 0, e = 0;
        if (args.E == 0)
            grid_dep_wait();
        if (blockIdx.x == 0 && q == 0)
            fp8_begin_call(args.offsets, args.E, args.M, args.keep_status, args.status, lane);
        if (args.E > 0)                                                // rows of no expert: 0
            for (int k = 0; k < 3; ++k) {
                if (!args.zero[k])
                    continue;
                const int64_t n16 = args.zero_row_bytes[k] / 16, lo = plan.start[0], hi = plan.start[args.E];
                for (int64_t m = 0; m < args.M; ++m)
                    if (m < lo || m >= hi)
                        for (int64_t c = (int64_t)(4 * blockIdx.x + q) * 32 + lane; c < n16; c += 128 * (int64_t)gridDim.x)
                            *reinterpret_cast<uint4 *>(args.zero[k] + m * args.zero_row_bytes[k] + 16 * c) =
                                make_uint4(0u, 0u, 0u, 0u);
            }
        // 16 rows' values of the lane's channel, `rows` of them real, to a matrix of the width of y
        auto put = [&](const float (&v)[16], void *to, bool bf16, int64_t row, int64_t col, int rows) {
            const int64_t at = row * args.width + col;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                if (bf16) {
                    uint16_t *dst = reinterpret_cast<uint16_t *>(to) + at + i * args.width;
                    const uint32_t w = f32x2_to_bf16x2_bits(v[i], v[i + 1]);
                    if (i < rows)
                        dst[0] = (uint16_t)w;
                    if (i + 1 < rows)
                        dst[args.width] = (uint16_t)(w >> 16);
                } else {
                    float *dst = reinterpret_cast<float *>(to) + at + i * args.width;
                    if (i < rows)
                        dst[0] = ADDS ? dst[0] + v[i] : v[i];
                    if (i + 1 < rows)
                        dst[args.width] = ADDS ? dst[args.width] + v[i + 1] : v[i + 1];
                }
            }
        };
        // sums of rows b .. b + 15 of tile t: out (gated: the gate's warp gets the up projection's from its fellow)
        auto finish = [&](const I8Tile &t, int b, float (&v)[16], bool real) {
            const int64_t col = (int64_t)t.wt * T + ch, row = (int64_t)t.row0 + b;
            int rows = real && ch < T && col < args.width ? t.rows - b : 0;
            if (!SQ_DCHECK(rows <= 0 || row + min(rows, 16) <= args.M, args.status))
                rows = 0;
            if constexpr (GATED) {
                if (args.g_out)
                    put(v, second ? args.u_out : args.g_out, true, row, col, rows);
                if (second) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        exchange[32 * i] = v[i];
                }
                named_barrier_sync(4 + (q & 1), 64);
                if (!second) {
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const uint64_t g = f2_pack(v[i], v[i + 1]), u = f2_pack(exchange[32 * i], exchange[32 * i + 32]);
                        f2_unpack(f2_mul(args.act == 0 ? act_value<0>(g) : act_value<1>(g), u), v[i], v[i + 1]);
                    }
                }
                named_barrier_sync(4 + (q & 1), 64);                   // (what was read may be written again)
                if (!second)
                    put(v, args.y, ybf, row, col, rows);
            } else {
                put(v, args.y, ybf, row, col, rows);
            }
        };
        auto load = [&](uint32_t taddr, float (&v)[16]) {
            uint32_t a[16];
            __syncwarp();
            tmem_ld_16cols(taddr, a);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = __uint_as_float(a[i]);
        };
        // The first turn is a dry one, while the products run.  It reads what tensor memory happens to hold and
        // writes nothing, so that the code is there when it is needed (a split tile's sums came together 4 us
        // after its products without, 1.5 us with it).
        bool dry = true;
        if (split == 1) {
#pragma unroll 1
            for (int tile = unit; tile < tiles;) {
                const I8Tile t = plan.find(tile, e);
                const int slot = count & 1;
                // (one that gave up goes on without effect, as its fellow may wait for it)
                const bool real = !dry && fp8_warp_wait<CG>(bar_acc_full + 8 * slot, (uint32_t)((count >> 1) & 1), abort_flag,
                                                            args.status, lane);
                tc_fence_after();
                const uint32_t acc = tmem_base + ((uint32_t)(32 * q) << 16) + (slot ? slot1 : 0u);
#pragma unroll 1
                for (int b = 0; b < slots && (b == 0 || (!dry && b < t.rows)); b += 16) {
                    float v[16];
                    load(acc + b, v);
                    finish(t, b, v, real);
                }
                tc_fence_before();
                __syncwarp();
                if (!dry) {
                    if (lane == 0)
                        mbar_arrive(bar_acc_empty + 8 * slot);
                    tile += units;
                    ++count;
                }
                dry = false;
            }
        }
        // One tile a cluster.  Each warp's channels are finished by one CTA (gated: the gate's and the up
        // projection's by the same), to which the others send theirs.
        const int owner = (GATED ? q & 1 : q) % split, place0 = GATED ? q >> 1 : q / split;
        const uint32_t acc = tmem_base + ((uint32_t)(32 * q) << 16);
#pragma unroll 1
        for (int turn = 0; split > 1 && unit < tiles && turn < 2; ++turn) {
            dry = turn == 0;
            bool real = !dry && fp8_warp_wait<CG>(bar_acc_full, 0, abort_flag, args.status, lane);
            tc_fence_after();
            const I8Tile t = plan.find(unit, e);
            const int quads = (t.rows + 3) / 4;                        // rows are sent in fours
            if (q == 0 && lane == 0 && !dry) {
                int mine = 0;                                          // warps whose channels this CTA finishes
                for (int w = 0; w < 4; ++w)
                    mine += (GATED ? w & 1 : w) % split == part ? 1 : 0;
                mbar_arrive_expect_tx(bar_parts, mine * (split - 1) * quads * 512);
            }
            // [place0][from][quad][lane] float4
            auto place = [&](int from, int quad) {
                return (uint32_t)(((place0 * split + from) * quads + quad) * 32 + lane) * 16u;
            };
            if (owner != part || dry) {
                const uint32_t dst = mapa_shared(smem_u32(rest), owner), bar = mapa_shared(bar_parts, owner);
#pragma unroll 1
                for (int b = 0; b < slots && b < t.rows; b += 16) {
                    float v[16];
                    load(acc + b, v);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (real && b / 4 + j < quads)
                            st_async_v4(dst + place(part, b / 4 + j), v + 4 * j, bar);
                }
            }
            if (owner == part || dry) {
                real = real && fp8_warp_wait<2>(bar_parts, 0, abort_flag, args.status, lane);
#pragma unroll 1
                for (int b = 0; b < slots && b < t.rows; b += 16) {
                    float v[16];
                    load(acc + b, v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (b / 4 + j >= quads)
                            break;
                        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        for (int from = 0; from < split; ++from) {     // the parts in order
                            const float4 w = from == part ? make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3])
                                                          : *reinterpret_cast<const float4 *>(rest + place(from, b / 4 + j));
                            sum.x += w.x;
                            sum.y += w.y;
                            sum.z += w.z;
                            sum.w += w.w;
                        }
                        v[4 * j] = sum.x;
                        v[4 * j + 1] = sum.y;
                        v[4 * j + 2] = sum.z;
                        v[4 * j + 3] = sum.w;
                    }
                    finish(t, b, v, real);
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue (every CTA)
        // Warp w: lanes 32 (w % 4) .. + 31, the first (w < 4) or second half of the tile's channels, C at a
        // time.
        const int wq = warp & 3, wh = warp >> 2;
        const uint32_t acc_empty_leader = CG == 2 ? mapa_shared(bar_acc_empty, 0) : bar_acc_empty;
        Fp8Patch out = {rest + warp * (Cfg::kPatches * kFPatchBytes), lane, 0};
        const bool ybf = args.out_bf16 != 0;
        constexpr int C = 32;
        const int chunks = (T + C - 1) / C;
        const int own = (chunks + 1 - wh) / 2;
        auto chunk_of = [&](int i) { return wh * ((chunks + 1) / 2) + i; };
        // a chunk's columns from fp32 sums (gated: q the up projection's)
        auto finish = [&](const I8Tile &t, int c, int rows, int64_t row, const float (&r)[C], const float (&q)[GATED ? C : 1]) {
            const int64_t col = (int64_t)t.wt * T + c;
            const int live = (int)min((int64_t)min(T - c, C), args.width - col);
            if (live <= 0 || !SQ_DCHECK(rows <= 0 || (row + rows <= args.M && col + live <= args.width), args.status))
                return;
            // all 32 rows and C columns are the tile's, or lie behind the matrix's end
            const bool whole = !ADDS && (rows == 32 || args.E == 0) && (live == C || col + live == args.width);
            auto put_out = [&](const float (&o)[C], const CUtensorMap &m, void *to, bool bf16) {
                store_cols<Cfg::kPatches, ADDS>(o, out, whole ? &m : nullptr, to, row, col, args.width, rows, live, bf16);
            };
            if constexpr (GATED) {
                if (args.g_out) {
                    put_out(r, tmG, args.g_out, true);
                    put_out(q, tmU, args.u_out, true);
                }
                float o[C];
                if (args.act == 0) {
#pragma unroll
                    for (int j = 0; j < C; j += 2)
                        f2_unpack(f2_mul(act_value<0>(f2_pack(r[j], r[j + 1])), f2_pack(q[j], q[j + 1])), o[j], o[j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < C; j += 2)
                        f2_unpack(f2_mul(act_value<1>(f2_pack(r[j], r[j + 1])), f2_pack(q[j], q[j + 1])), o[j], o[j + 1]);
                }
                put_out(o, tmY, args.y, ybf);
            } else {
                put_out(r, tmY, args.y, ybf);
            }
        };
        auto load_chunk = [&](uint32_t acc, int c, float (&r)[C], float (&q)[GATED ? C : 1]) {
            uint32_t a[C];
            __syncwarp();
            tmem_ld_32cols(acc + c, a);
            if constexpr (GATED) {
                uint32_t b[C];
                tmem_ld_32cols(acc + T + c, b);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < C; ++j)
                    q[j] = __uint_as_float(b[j]);
            } else {
                tmem_wait_ld();
            }
#pragma unroll
            for (int j = 0; j < C; ++j)
                r[j] = __uint_as_float(a[j]);
        };
        int count = 0, e = 0;
        grid_dep_wait();
        if (split == 1) {
#pragma unroll 1
            for (int tile = unit; tile < tiles; tile += units, ++count) {
                const I8Tile t = plan.find(tile, e);
                const int slot = count & 1;
                if (!fp8_warp_wait<CG>(bar_acc_full + 8 * slot, (uint32_t)((count >> 1) & 1), abort_flag, args.status,
                                       lane))
                    break;
                tc_fence_after();
                const uint32_t acc = tmem_base + ((uint32_t)(32 * wq) << 16) + (slot ? slot1 : 0u);
                const int first_row = (int)rank * 128 + 32 * wq;
                const int rows = min(t.rows - first_row, 32);          // (may be negative)
                auto release = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (CG == 2)
                            mbar_arrive_cluster(acc_empty_leader + 8 * slot);
                        else
                            mbar_arrive(acc_empty_leader + 8 * slot);
                    }
                };
                // overlapping accumulators: the chunks that they share first (the last of the one at column
                // 0, the first of the other), then the next tile may start
                const int held = rows <= 0 ? 0 : shared_cols > 0 ? min(shared_cols / C, own) : own;
                if (held == 0)
                    release();
                if (rows > 0)
                    for (int i = 0; i < own; ++i) {
                        const int c = C * chunk_of(slot ? i : own - 1 - i);
                        float r[C], q[GATED ? C : 1];
                        load_chunk(acc, c, r, q);
                        if (i == held - 1)
                            release();
                        finish(t, c, rows, (int64_t)t.row0 + first_row, r, q);
                    }
            }
        }
        // One tile a cluster.  Each chunk of its columns is finished by one CTA, owner(c), to which the others
        // send theirs, into the ring, once a CTA whose products are done has told the others that it is free.
        if (split > 1 && unit < tiles && fp8_warp_wait<CG>(bar_acc_full, 0, abort_flag, args.status, lane)) {
            constexpr int kParts = GATED ? 2 : 1;
            tc_fence_after();
            const I8Tile t = plan.find(unit, e);
            const uint32_t acc = tmem_base + ((uint32_t)(32 * wq) << 16);
            const int rows = min(t.rows - 32 * wq, 32);
            auto owner = [&](int c) { return c % split; };
            int mine = 0;                                              // chunks that this CTA finishes
            for (int c = 0; c < chunks; ++c)
                mine += owner(c) == part ? 1 : 0;
            if (wq == 0 && wh == 0) {
                if (lane < split && lane != part)
                    mbar_arrive_cluster(mapa_shared(bar_peers, lane));
                if (lane == 0)
                    mbar_arrive_expect_tx(bar_parts, mine * (split - 1) * t.rows * (4 * C) * kParts);
            }
            // place of a chunk's part from CTA `from`: [c / split][from][gate, up][quarter][C / 4][lane] float4
            auto place = [&](int c, int from, int which) {
                return (uint32_t)((((c / split * split + from) * kParts + which) * 4 + wq) * (C / 4) * 32 + lane) * 16u;
            };
            const uint32_t s0 = smem_u32(smem);
            bool ok = fp8_warp_wait<2>(bar_peers, 0, abort_flag, args.status, lane);
            if (ok && rows > 0)
                for (int i = 0; i < own; ++i) {
                    const int c = chunk_of(i), to = owner(c);
                    if (to == part)
                        continue;
                    float r[C], q[GATED ? C : 1];
                    load_chunk(acc, C * c, r, q);
                    const uint32_t dst = mapa_shared(s0, to), bar = mapa_shared(bar_parts, to);
                    if (lane < rows)
#pragma unroll
                        for (int j = 0; j < C / 4; ++j) {
                            st_async_v4(dst + place(c, part, 0) + j * 512, r + 4 * j, bar);
                            if constexpr (GATED)
                                st_async_v4(dst + place(c, part, 1) + j * 512, q + 4 * j, bar);
                        }
                }
            __syncwarp();
            ok = ok && fp8_warp_wait<2>(bar_parts, 0, abort_flag, args.status, lane);
            if (ok && rows > 0)
                for (int i = 0; i < own; ++i) {
                    const int c = chunk_of(i);
                    if (owner(c) != part)
                        continue;
                    float r[C], q[GATED ? C : 1];
                    load_chunk(acc, C * c, r, q);
                    auto join = [&](float *v, int which, int j) {      // four columns: the parts in order
                        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        for (int from = 0; from < split; ++from) {
                            const float4 w = from == part || lane >= rows ? make_float4(v[0], v[1], v[2], v[3])
                                                          : *reinterpret_cast<const float4 *>(
                                                                smem + place(c, from, which) + j * 512);
                            sum.x += w.x;
                            sum.y += w.y;
                            sum.z += w.z;
                            sum.w += w.w;
                        }
                        v[0] = sum.x;
                        v[1] = sum.y;
                        v[2] = sum.z;
                        v[3] = sum.w;
                    };
#pragma unroll
                    for (int j = 0; j < C / 4; ++j) {
                        join(r + 4 * j, 0, j);
                        if constexpr (GATED)
                            join(q + 4 * j, 1, j);
                    }
                    finish(t, C * c, rows, (int64_t)t.row0 + 32 * wq, r, q);
                }
        }
        if (lane == 0)
            bulk_wait_group_all();
        __syncwarp();
    }

    tc_fence_before();
    if (CG == 2 || split > 1)
        cluster_meet();                               // no CTA leaves while another may still signal it
    else
        __syncthreads();
    tc_fence_after();
    if (warp == kIssuer) {
        if (CG == 2)
            tmem_dealloc2(tmem_base, Cfg::kTmemCols);
        else
            tmem_dealloc(tmem_base, Cfg::kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
namespace {

typedef CUresult (*PFN_encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                               const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

PFN_encode encode_fn()
{
    static PFN_encode fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn = reinterpret_cast<PFN_encode>(p);
    }
    return fn;
}

// byte matrices [outer, rows, inner] in a row, boxes of box_rows x 128; what lies outside one of them
// reads as 0 (a box that ends behind an expert's last row does not see the next expert's)
bool byte_map(CUtensorMap *m, const void *base, int64_t inner, int64_t rows, int64_t outer, int box_rows)
{
    const PFN_encode fn = encode_fn();
    if (!fn)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)outer};
    const cuuint64_t strides[2] = {(cuuint64_t)inner, (cuuint64_t)(inner * rows)};
    const cuuint32_t box[3] = {kFChunk, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, outer > 0 ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A tile and its split: how a call's tiles are cut (see pick).
struct Fp8Shape {
    int cg, tile, split;
};

// what runs on the device at once: clusters of `split` one-CTA tiles, and CTA pairs
struct Fp8Room {
    unsigned long long ctx = 0;
    int clusters[kFMaxSplit + 1] = {};
    int pairs = 0;
    uint32_t *status = nullptr;                   // the library's word
};
constexpr int kMaxDev = 64;

void cluster_attr(cudaLaunchAttribute &at, int size)
{
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)size;
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
}

// an output [rows, width], boxes of 32 rows x 64 bytes
bool out_map(CUtensorMap *m, const void *base, int64_t width, int64_t rows, bool bf16)
{
    const PFN_encode fn = encode_fn();
    if (!fn)
        return false;
    const int size = bf16 ? 2 : 4;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(width * size)};
    const cuuint32_t box[2] = {(cuuint32_t)(64 / size), 32};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(base),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG, int MODE, bool FUSE, bool ADDS>
cudaError_t allow_smem(int dev, unsigned long long ctx)
{
    static unsigned long long seen[kMaxDev];
    if (ctx != 0 && seen[dev] == ctx)
        return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(sq_fp8_kernel<CG, MODE, FUSE, ADDS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Fp8Cfg<CG, MODE, FUSE>::kSmemBytes);
    if (e == cudaSuccess)
        seen[dev] = ctx;
    return e;
}

// (not every SM finds its partners inside its GPC)
template <int CG, int MODE>
int resident_clusters(int size, int sms)
{
    using Cfg = Fp8Cfg<CG, MODE, false>;
    cudaLaunchConfig_t o = {};
    cudaLaunchAttribute at[1];
    cluster_attr(at[0], size);
    o.gridDim = dim3((unsigned)(sms / size * size));
    o.blockDim = dim3(Cfg::kThreads);
    o.dynamicSmemBytes = Cfg::kSmemBytes;
    o.attrs = at;
    o.numAttrs = 1;
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, sq_fp8_kernel<CG, MODE, false, false>, &o);
    (void)cudaGetLastError();
    return e == cudaSuccess && n > 0 && n < sms / size ? n : sms / size;
}

cudaError_t room_of(int dev, unsigned long long ctx, int sms, const Fp8Room **out)
{
    static Fp8Room rooms[kMaxDev];
    Fp8Room &r = rooms[dev];
    if (ctx == 0 || r.ctx != ctx) {
        cudaError_t e = allow_smem<2, kFp8Fwd, false, false>(dev, ctx);
        if (e == cudaSuccess)
            e = allow_smem<1, kFp8Fwd, false, false>(dev, ctx);
        if (e == cudaSuccess)
            e = library_status_word(&r.status);
        if (e != cudaSuccess)
            return e;
        r.pairs = resident_clusters<2, kFp8Fwd>(2, sms);
        r.clusters[1] = sms;
        for (int n = 2; n <= kFMaxSplit; ++n)
            r.clusters[n] = resident_clusters<1, kFp8Fwd>(n, sms);
        r.ctx = ctx;
    }
    *out = &r;
    return cudaSuccess;
}

template <int CG, int MODE, bool FUSE>
cudaError_t launch_fp8(const Fp8GemmLaunch &g, const Fp8QuantArgs &q, const Fp8Shape &sh, int dev, const Fp8Room &room,
                       cudaStream_t stream)
{
    static_assert(kSumGroups >= kFMaxSplit, "every CTA of a cluster has a group");
    using Cfg = Fp8Cfg<CG, MODE, FUSE>;
    constexpr bool BWD = MODE == kFp8Bwd, GATED = MODE == kFp8Gated;
    if (cudaError_t e = allow_smem<CG, MODE, FUSE, false>(dev, room.ctx); e != cudaSuccess)
        return e;
    const int tile = sh.tile;
    const int64_t Em = g.E > 0 ? g.E : 1;
    const int64_t summed = BWD ? g.N : g.K;
    const int halves = BWD && g.gated ? 2 : 1;
    const int b_rows = BWD ? (tile / CG + 127) / 128 * 128 : GATED ? (CG == 2 ? tile : 2 * tile) : tile / CG;
    Fp8Args a;
    a.offsets = g.offsets;
    a.words = g.words;
    a.x = q.x;
    a.g = q.g;
    a.u = q.u;
    a.ws[0] = g.wscales[0];
    a.ws[1] = g.gated ? g.wscales[1] : g.wscales[0];
    a.y = g.y;
    a.g_out = g.g_out;
    a.u_out = g.u_out;
    a.status = g.status;
    for (int i = 0; i < 3; ++i) {
        a.zero[i] = q.zero[i];
        a.zero_row_bytes[i] = q.zero_row_bytes[i];
    }
    a.M = g.M;
    a.width = BWD ? g.K : g.N;
    a.L = summed;
    a.E = g.E;
    a.act = g.act;
    a.out_bf16 = g.out_bf16;
    a.finite_check = q.finite_check;
    a.keep_status = q.keep_status;
    a.nbs = (int)((g.N + kFp8Block - 1) / kFp8Block);
    a.kbs = (int)((g.K + kFp8Block - 1) / kFp8Block);
    a.blocks = (int)((summed + kFp8Block - 1) / kFp8Block);
    a.halves = halves;
    a.tile = tile;
    a.a_rows = FUSE ? (int)((g.M + 15) / 16 * 16) : CG == 2 || g.M >= 128 ? 128 : (int)((g.M + 31) / 32 * 32);
    const int cols = GATED ? 2 * tile : tile;
    a.slot1 = cols > 224 ? 192 : 224;
    a.boxed_rows = g.E > 0 ? (a.a_rows - 1) / 32 * 32 : 0;
    a.split = sh.split;
    CUtensorMap tmX, tmX32, tmW, tmW2, tmY, tmG, tmU;
    const int w_rows = BWD ? 128 : GATED ? tile : tile / CG;
    bool ok = byte_map(&tmW, g.wcodes[0], g.K, g.N, Em, w_rows);
    tmX = tmX32 = tmW2 = tmY = tmG = tmU = tmW;
    if (!FUSE)
        ok = ok && byte_map(&tmX, g.codes, summed, halves * g.M, 0, a.a_rows);
    if (!FUSE && a.boxed_rows > 0)
        ok = ok && byte_map(&tmX32, g.codes, summed, halves * g.M, 0, 32);
    if (g.gated)
        ok = ok && byte_map(&tmW2, g.wcodes[1], g.K, g.N, Em, w_rows);
    if (!FUSE)
        ok = ok && out_map(&tmY, g.y, a.width, g.M, g.out_bf16 != 0);
    if (!FUSE && g.g_out)
        ok = ok && out_map(&tmG, g.g_out, a.width, g.M, true) && out_map(&tmU, g.u_out, a.width, g.M, true);
    if (!ok)
        return cudaErrorInvalidValue;
    // the stages: as many chunks as leave four of them
    const int ring = Cfg::kRing - (FUSE ? kFBufs * kFp8Group * a.a_rows * kFChunk : 0);
    const int chunk = (FUSE ? (GATED ? kFUpRow + tile : b_rows) : a.a_rows + b_rows) * kFChunk;
    a.prefetch = kPrefetchBytes / chunk;
    a.per = 1;                // a pair: two where that leaves three stages (4480 x 16384 x 6144: 295 us, with one 328)
    if (CG == 2 && 6 * chunk <= ring)
        a.per = 2;
    if (CG == 1)
        while (a.per < 4 && 2 * a.per * chunk * 4 <= ring)
            a.per *= 2;
    a.stages = ring / (a.per * chunk);
    if (a.stages > Cfg::kMaxStages)
        a.stages = Cfg::kMaxStages;
    if (a.stages < 2)
        return cudaErrorInvalidValue;
    // dependent launch: set-up and the first weight tiles overlap the rounding in front
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cluster_attr(at[1], CG * sh.split);
    const int64_t some = g.E > 0 ? (g.E < g.M ? g.E : g.M) : 0;                  // experts: the most row tiles
    const int64_t work = (a.width + tile - 1) / tile * (g.E > 0 ? some + g.M / (128 * CG) : (g.M + 128 * CG - 1) / (128 * CG));
    const int64_t most = CG == 2 ? room.pairs : room.clusters[sh.split];
    const int units = (int)(work < most ? work : most);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * CG * sh.split));
    cfg.blockDim = dim3(Cfg::kThreads);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = CG * sh.split > 1 ? 2 : 1;
    // Long sums of fp32 results: a launch for each part, which adds to the ones before (the gated forward needs both
    // sums whole; a bf16 result's own rounding is larger than what is lost).  Each waits for the one in front before it
    // touches y.
    const int groups = (int)fp8_groups(summed) * halves;
    const int most_groups = kSumGroups * sh.split;
    const int parts = GATED || g.out_bf16 ? 1 : (groups + most_groups - 1) / most_groups;
    for (int i = 0; i < parts; ++i) {
        a.lo = (int)((int64_t)groups * i / parts);
        a.hi = (int)((int64_t)groups * (i + 1) / parts);
        cudaError_t e = cudaSuccess;
        if (i == 0) {
            e = cudaLaunchKernelEx(&cfg, sq_fp8_kernel<CG, MODE, FUSE, false>, tmX, tmX32, tmW, tmW2, tmY, tmG, tmU, a);
        } else if constexpr (!GATED) {
            a.keep_status = 1;
            a.zero[0] = a.zero[1] = a.zero[2] = nullptr;
            e = allow_smem<CG, MODE, FUSE, true>(dev, room.ctx);
            if (e == cudaSuccess)
                e = cudaLaunchKernelEx(&cfg, sq_fp8_kernel<CG, MODE, FUSE, true>, tmX, tmX32, tmW, tmW2, tmY, tmG, tmU, a);
        }
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

// How a call's tiles are cut: the candidate with the least time by a simple count of cycles.  A chunk
// of 128 summed values takes the longer of its products (2 cycles a column; one CTA: 140 more) and its
// copies (about 66 bytes a cycle and SM); between overlapping accumulators the products pause; a tile's
// groups may be shared by a cluster where all tiles run at once, which costs some 8000 cycles (of clusters
// larger than two, some room is left: the last one waited for SMs that other kernels still held, 262 x 1616 x
// 14080 in 45 clusters of three of 45 that fit took 31.6 us, with 39 of them 24.1).  A pair's start takes 700
// more.  One-CTA tiles are wider than 128 columns too: of 22 dense calls that take such, 0.91 of the time with 128
// (gradient of 301 x 11664 x 11040 58 us, 76; gated 278 x 8624 x 2176 20.5, 24.4; at worst gated 192 x 6272 x 304
// 9.6, 9.4).  Backward a CTA's columns start at 32-byte sectors (4480 x 16384 x 6144, pairs of 192, 224 and 256
// columns: 423, 450, 361 us).
// Few rows: products of 128 channels whatever the tile has, 190 cycles and 2 a row of the operand; a group at
// least as long as its rounding; 30 for each CTA, which all read the rows; 1200 and 200 a CTA for a shared
// tile.  Measured, us a call of one token, 6144 x 6144, tiles of 48, 64, 80 channels 12.1, 11.2, 11.8, two CTAs
// on tiles of 96, 112, 128 channels 10.5, 10.2, 10.0; over 100 calls with sizes at random the choice was 2 %
// from the fastest candidate on average and 23 % at worst (few of many experts, which the host cannot know).
//
// Experts: the host does not see the offsets.  It counts a row tile for each expert that can have rows,
// or half of one and the whole ones that all rows make; no more than one and the whole ones each.
// Measured, us a call, one CTA 128 and 224 columns wide (backward 256), pair 224 (256): 8192 rows of 61
// experts, gated, 2 x 1408 x 2048: 95, 86, 95; 8192 of 64, backward, 2816 x 2048: 97, 89, 104; 8192 of 8,
// 4096 x 2048: 90, 77, 74; 1500 of 64, 2816 x 2048: 70, 71, 90.  So pairs from 512 rows an expert on, and
// tiles of 128 columns at most up to 32 (bound by the weights' bytes).
Fp8Shape pick(const Fp8GemmLaunch &g, bool fuse, const Fp8Room &room)
{
    const int64_t width = g.bwd ? g.K : g.N, summed = g.bwd ? g.N : g.K;
    const int weights = g.gated && !g.bwd ? 2 : 1;             // columns of B for an output channel
    const int64_t groups = fp8_groups(summed) * (g.gated && g.bwd ? 2 : 1);
    const int64_t experts = g.E > 0 ? (g.E < g.M ? g.E : g.M) : 1, mean = g.M / experts;
    Fp8Shape best = {1, 128 / weights, 1};
    int64_t best_cost = INT64_MAX;
    auto offer = [&](int cg, int cols, int split) {
        const int tile = cols / weights;
        const int64_t whole = g.M / (128 * cg), col_tiles = (width + tile - 1) / tile;
        int64_t rows = (g.M + 128 * cg - 1) / (128 * cg), most_rows = rows;
        if (g.E > 0) {
            rows = experts / 2 + whole > experts ? experts / 2 + whole : experts;
            most_rows = experts + whole;
        }
        const int64_t units = cg == 2 ? room.pairs : room.clusters[split];
        if (split > 1 && most_rows * col_tiles > (split > 2 ? units * 15 / 16 : units))
            return;
        const int64_t tiles = rows * col_tiles;
        // (in eighths; many rounds of tiles that are only an estimate: half of one for the last)
        const int64_t rounds8 = g.E > 0 && tiles > 2 * units ? tiles * 8 / units + 4 : (tiles + units - 1) / units * 8;
        const int64_t a = fuse ? 0 : cg == 2 || mean >= 96 ? 128 : (mean + 31) / 32 * 32;
        const int64_t b = g.bwd ? (cols / cg + 127) / 128 * 128 : cols / cg;
        const int64_t mma = cg == 2 ? 2 * cols : fuse ? 190 + (g.M + 15) / 16 * 32 : 140 + 2 * cols, copy = (a + b) * kFChunk / (fuse ? 72 : 66);
        const int64_t group = kFp8Group * (mma > copy ? mma : copy), rounding = fuse ? 250 + (weights < 2 && g.gated ? 1000 : 450) * ((mean + 3) / 4) : 0;
        const int64_t ctas = (tiles < units ? tiles : units) * split;
        const int64_t cost = rounds8 * ((groups + split - 1) / split * (group > rounding ? group : rounding) + (cols > 224 ? 2500 : 500)) / 8 +
                             (fuse ? 30 * ctas + (split == 1 ? 0 : 1200 + 200 * split) :
                                     10 * cols + (split == 1 ? 0 : 8000) + (cg == 2 ? 700 : 0));
        if (cost < best_cost) {
            best_cost = cost;
            best = {cg, tile, split};
        }
    };
    if (!fuse && (g.E == 0 || mean >= 512))
        for (int cols = 256; cols >= 64; cols -= g.bwd ? 64 : 32)
            offer(2, cols, 1);
    // (what shared memory holds of the others' sums)
    const int most = fuse ? (weights == 2 ? (g.M > 16 ? 3 : 6) : g.M > 16 ? 6 : kFMaxSplit) : weights == 2 ? 6 : kFMaxSplit;
    const int widest = mean > 32 ? (g.bwd ? 256 : 224) : 128;
    for (int cols = widest; cols >= (g.bwd ? 128 : 32); cols -= g.bwd ? 128 : 16)
        for (int split = 1; split <= most && split <= groups && (split == 1 || cols <= 128); ++split)
            offer(1, cols, split);
    return best;
}

template <int CG, bool FUSE>
cudaError_t launch_mode(const Fp8GemmLaunch &g, const Fp8QuantArgs &q, const Fp8Shape &sh, int dev,
                        const Fp8Room &room, cudaStream_t stream)
{
    if (g.bwd)
        return launch_fp8<CG, kFp8Bwd, FUSE>(g, q, sh, dev, room, stream);
    return g.gated ? launch_fp8<CG, kFp8Gated, FUSE>(g, q, sh, dev, room, stream)
                   : launch_fp8<CG, kFp8Fwd, FUSE>(g, q, sh, dev, room, stream);
}

}  // namespace

// Every CTA rounds the rows for itself: that saves a launch (some 3 us, and 2.5 of the host's time), and costs
// more with each row, most for a gated pair's gradients.  Measured, us a call, one kernel and two: 7 x 4128 x 1536 6.2, 8.5;
// 16 x 6784 x 880 5.7, 8.7; gradients of 15 x 6784 x 1584 8.5, 13.6, 24 x 8192 x 9216 26.8, 23.4 and
// 31 x 7680 x 11136 49.8, 21.9; gated gradients of 6 x 1248 x 1248 6.4, 10.5, 7 x 9216 x 4224 24.6, 23.7 and
// 17 x 3712 x 4560 21.1, 18.0.  Of experts a tile has only some of the rows; and small weights are shared by
// fewer CTAs: of 45 calls with N K <= 2^24 and 17 to 32 rows (gated gradients 9 to 16) one kernel took 0.91 of the
// time of two (24 x 1280 x 6032 9.4, 13.5; at worst 32 x 7200 x 1392 10.6, 8.7), called one by one 0.86.
bool fp8_rounds_rows(int E, int64_t M, int64_t N, int64_t K, bool gated_bwd)
{
    const bool twice = E > 1 || (K > 0 && N <= (int64_t(1) << 24) / K);
    return M <= kFuseRows * (twice ? 2 : 1) / (gated_bwd ? 2 : 1);
}

static cudaError_t current_room(int sms, int *dev, const Fp8Room **room)
{
    if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDev)
        return cudaErrorInvalidDevice;
    return room_of(*dev, current_context_id(), sms, room);
}

cudaError_t fp8_status_word(int sms, uint32_t **p)
{
    int dev = 0;
    const Fp8Room *room = nullptr;
    const cudaError_t e = current_room(sms, &dev, &room);
    if (e == cudaSuccess)
        *p = room->status;
    return e;
}

cudaError_t launch_fp8_gemm(const Fp8GemmLaunch &g, const Fp8QuantArgs &q, int sms, cudaStream_t stream)
{
    int dev = 0;
    const Fp8Room *room = nullptr;
    if (cudaError_t e = current_room(sms, &dev, &room); e != cudaSuccess)
        return e;
    const bool fuse = fp8_rounds_rows(g.E, g.M, g.N, g.K, g.bwd && g.gated);
    const Fp8Shape sh = pick(g, fuse, *room);
    if (sh.cg == 2)
        return launch_mode<2, false>(g, q, sh, dev, *room, stream);
    return fuse ? launch_mode<1, true>(g, q, sh, dev, *room, stream) : launch_mode<1, false>(g, q, sh, dev, *room, stream);
}

}  // namespace sq
