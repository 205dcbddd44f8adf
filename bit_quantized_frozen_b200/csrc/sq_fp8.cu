// sq_fp8.cu -- products of e4m3 codes with one power-of-two scale for each block of 128, dense or
// grouped by expert, on tcgen05 (kind::mxf8f6f4 with block scales, fp32 sums in tensor memory).
//
//   forward   y[m, n]  = sum_k x[m, k] W[n, k]
//   gated     h[m, n]  = act(g) u,  g and u such sums of two weights
//   backward  dx[m, k] = sum_n dy[m, n] W[n, k], gated: sum over both weights
//
// Tensor-memory lanes hold tokens, columns output channels.  A = the rows' codes (K-major); B =
// the weight's codes, K-major forward and N-major backward (they are read as they lie, never
// transposed).  Gated: B is a tile of the gate's rows and the same rows of the up projection, so
// that both sums of an output lie in one lane and the activation is applied as they leave tensor
// memory; backward the summed axis simply runs through both weights.
//
// Scales.  The tensor cores take one e8m0 byte for each row of A and of B and 32 values; a block of
// 128 is four of them with the same byte.  A word holds the bytes of four neighbouring blocks, the
// instruction names the one to use, so that a row's scales for 512 values are one 32-bit word in
// tensor memory.  The scale warps lay the words of a tile out in shared memory (rows r, r + 32,
// r + 64, r + 96 of 128 in one 16-byte line), the issuing thread copies them into tensor memory in
// front of the products that need them.
//
// CTA (CG = 1, tiles of 128 tokens x up to 128 columns) or CTA pair (CG = 2, 256 x 256) per SM,
// persistent: 8 epilogue warps, TMA producers, scale warps and an issuer that also allocates tensor
// memory.  Two accumulators, 256 columns wide at columns 0 and 224: they share 32 columns, which the
// epilogue reads first, so that the scales find room behind them (480 .. 511) and the next tile's
// products still start almost at once.
#include <cuda.h>

#include "sq_fp8.cuh"
#include "sq_kernels.h"
#include "sq_ptx.cuh"
#include "sq_w8a8.cuh"

namespace sq {

enum Fp8Mode { kFp8Fwd = 0, kFp8Gated = 1, kFp8Bwd = 2 };

constexpr int kFChunk = 128;                      // summed values (bytes) of a shared-memory row
constexpr uint32_t kFSlot1 = 224;                 // second accumulator
constexpr uint32_t kFScaleCol = 480;              // two buffers of 16 columns: 8 for B, 4 for A
constexpr uint32_t kFTmemCols = 512;
constexpr int kFEpiWarps = 8;
constexpr int kFPatchBytes = 32 * 64;             // a warp's 32 rows x 64 bytes on their way out
constexpr int kFSfSlots = 4;                      // shared-memory copies of the scale words
constexpr int kFSfBytes = 512 + 1024;             // of A's 128 rows and of B's 256

template <int CG, int MODE>
struct Fp8Cfg {
    static constexpr int kProducers = CG == 2 ? 1 : 2;
    static constexpr int kScaleWarps = CG == 2 ? 2 : 4;
    static constexpr int kThreads = 32 * (kFEpiWarps + kProducers + kScaleWarps + 1);
    static constexpr int kRing = 192 * 1024;
    static constexpr int kMaxStages = CG == 2 ? 6 : 24;
    static constexpr int kPatchOff = kRing;       // (CG = 1: the MMA reads 128 rows of A, up to 16 KB behind the last stage)
    static constexpr int kSfOff = kPatchOff + kFEpiWarps * kFPatchBytes;
    static constexpr int kPlanOff = kSfOff + kFSfSlots * kFSfBytes;
    static constexpr int kBarOff = kPlanOff + (2 * kMaxExperts + 4) * 4;
    // full, empty, sf_full, sf_empty, acc_full[2], acc_empty, drain
    static constexpr int kNumBars = 2 * kMaxStages + 2 * kFSfSlots + 4;
    static constexpr int kSmemBytes = kBarOff + 8 * kNumBars + 16 + 1024;
    // e4m3 x e4m3, e8m0 scales; B N-major backward; 128 CG rows (columns / 8 << 17 comes at run time)
    static constexpr uint32_t kIdesc = (1u << 23) | (MODE == kFp8Bwd ? 1u << 16 : 0u) | ((uint32_t)(8 * CG) << 24);
    static constexpr uint32_t kBStep16 = MODE == kFp8Bwd ? (32u * 128u) >> 4 : 2u;   // B descriptor step per MMA
};

struct Fp8Args {
    const int32_t *offsets;
    const uint32_t *words;    // row scales, [halves * groups, M]
    const uint8_t *ws[2];     // weight scales, [E, nbs, kbs]
    void *y;
    uint16_t *g_out, *u_out;
    uint32_t *status;
    int64_t M, width;         // rows, and columns of y
    int E, act, out_bf16;
    int N;                    // weight rows of an expert (coordinates of TMA boxes)
    int nbs, kbs;             // blocks of a weight along N and K
    int blocks;               // blocks of the summed axis (of one weight)
    int halves;               // weights that the sum runs through
    int tile;                 // output channels of a tile
    int a_rows;               // rows of A that a stage reserves (CG = 1)
    int per;                  // chunks of a stage: 1, 2 or 4
    int stages;
};

template <int CG>
__device__ __forceinline__ bool fp8_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag, uint32_t *status)
{
    return CG == 2 ? mbar_wait_cluster(bar, parity, abort_flag, status) : mbar_wait(bar, parity, abort_flag, status);
}

// bounded wait with acquire at cluster scope
__device__ __forceinline__ bool fp8_wait_acquire(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag,
                                                 uint32_t *status)
{
    return mbar_wait_cluster(bar, parity, abort_flag, status) && mbar_try_wait_acquire_cluster(bar, parity);
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

// One warp's 32 rows x 64 bytes to y: through the patch, so that a row's 64 bytes leave in one run.
// dst: row 0's first byte; the first `rows` rows and `bytes` bytes (a multiple of 16) of each exist.
__device__ __forceinline__ void store_rows64(const uint32_t (&v)[16], uint8_t *patch, int lane, uint8_t *dst,
                                             int64_t row_bytes, int rows, int bytes)
{
#pragma unroll
    for (int p = 0; p < 4; ++p)
        *reinterpret_cast<uint4 *>(patch + lane * 64 + ((p ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 2), p = lane & 3;
        const uint4 w = *reinterpret_cast<const uint4 *>(patch + row * 64 + ((p ^ ((row >> 1) & 3)) << 4));
        if (row < rows && 16 * p < bytes)
            *reinterpret_cast<uint4 *>(dst + row * row_bytes + 16 * p) = w;
    }
    __syncwarp();
}

// 32 columns of y from fp32 values, as bf16 or fp32; `cols` of them exist
__device__ __forceinline__ void store_cols32(const float (&o)[32], uint8_t *patch, int lane, void *y, int64_t row,
                                             int64_t col, int64_t width, int rows, int cols, bool bf16)
{
    uint32_t v[16];
    if (bf16) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = f32x2_to_bf16x2_bits(o[2 * i], o[2 * i + 1]);
        store_rows64(v, patch, lane, reinterpret_cast<uint8_t *>(y) + 2 * (row * width + col), 2 * width, rows, 2 * cols);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = __float_as_uint(o[16 * h + i]);
            store_rows64(v, patch, lane, reinterpret_cast<uint8_t *>(y) + 4 * (row * width + col + 16 * h), 4 * width,
                         rows, 4 * (cols - 16 * h));
        }
    }
}

template <int CG, int MODE>
__global__ void __cluster_dims__(CG, 1, 1) __launch_bounds__(Fp8Cfg<CG, MODE>::kThreads, 1)
    sq_fp8_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                  const __grid_constant__ CUtensorMap tmW2, const Fp8Args args)
{
    using Cfg = Fp8Cfg<CG, MODE>;
    constexpr bool BWD = MODE == kFp8Bwd, GATED = MODE == kFp8Gated;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int32_t *plan_mem = reinterpret_cast<int32_t *>(smem + Cfg::kPlanOff);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kBarOff);
    const uint32_t bar_full = smem_u32(bars);                          // leader: both CTAs' stage ready
    const uint32_t bar_empty = bar_full + 8 * Cfg::kMaxStages;         // each CTA: its stage may be refilled
    const uint32_t bar_sf_full = bar_empty + 8 * Cfg::kMaxStages;      // leader: both CTAs' scale words ready
    const uint32_t bar_sf_empty = bar_sf_full + 8 * kFSfSlots;         // each CTA: they have been copied
    const uint32_t bar_acc_full = bar_sf_empty + 8 * kFSfSlots;        // each CTA: accumulator ready
    const uint32_t bar_acc_empty = bar_acc_full + 16;                  // leader: the shared columns have been read
    const uint32_t bar_drain = bar_acc_empty + 8;                      // leader: every MMA finished
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + Cfg::kNumBars);
    volatile uint32_t *abort_flag = tmem_holder + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    constexpr int kProducer = kFEpiWarps, kScale = kProducer + Cfg::kProducers, kIssuer = kScale + Cfg::kScaleWarps;

    if (threadIdx.x == 0) {
        for (int st = 0; st < Cfg::kMaxStages; ++st) {
            mbar_init(bar_full + 8 * st, 1);
            mbar_init(bar_empty + 8 * st, 1);
        }
        for (int i = 0; i < kFSfSlots; ++i) {
            mbar_init(bar_sf_full + 8 * i, CG);
            mbar_init(bar_sf_empty + 8 * i, 1);
        }
        mbar_init(bar_acc_full, 1);
        mbar_init(bar_acc_full + 8, 1);
        mbar_init(bar_acc_empty, CG * kFEpiWarps);
        mbar_init(bar_drain, 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == kIssuer) {
        if (CG == 2) {
            tmem_alloc2(smem_u32(tmem_holder), kFTmemCols);
            tmem_relinquish2();
        } else {
            tmem_alloc(smem_u32(tmem_holder), kFTmemCols);
            tmem_relinquish();
        }
    }
    if (warp == kProducer && lane == 0) {
        prefetch_tmap(&tmX);
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmW2);
    }
    grid_dep_launch();                            // the next call's rounding may be set up
    // the offsets are an input of the call: they are there before the kernel in front starts
    I8Plan plan;
    plan.E = args.E > 0 ? args.E : 1;
    plan.start = plan_mem;
    plan.prefix = plan_mem + kMaxExperts + 1;
    plan.wts = (int)((args.width + args.tile - 1) / args.tile);
    plan.tok_tile = 128 * CG;
    plan.build(args.E > 0 ? args.offsets : nullptr, args.M, threadIdx.x, Cfg::kThreads);
    tc_fence_before();
    if (CG == 2)
        cluster_sync();                           // barriers of both CTAs initialised, TMEM allocated
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;

    const int tiles = plan.tiles();
    const int unit = (int)blockIdx.x / CG;
    const int units = (int)gridDim.x / CG;
    const int per = args.per;
    const int T = args.tile;
    const int b_rows = GATED ? (CG == 2 ? T : 2 * T) : T / CG;         // rows of B (columns) that this CTA loads
    const int cols = GATED ? 2 * T : T;                                // columns of the accumulator
    const int a_bytes = (CG == 2 ? 128 : args.a_rows) * kFChunk;
    const int chunk_bytes = a_bytes + (BWD ? 128 : b_rows) * kFChunk;
    const int stage_bytes = per * chunk_bytes;
    const int stages = args.stages;
    const int half_steps = (args.blocks + per - 1) / per;
    const int steps = half_steps * args.halves;
    const int groups = (args.blocks + kFp8Group - 1) / kFp8Group;      // scale words of one weight's summed axis

    if (warp >= kProducer && warp < kScale) {
        // ------------------------------------------------------------ producers (every CTA)
        // Producer p fills stages p, p + P, ... with every P-th step of the unit's work.
        constexpr int P = Cfg::kProducers;
        const int p = warp - kProducer;
        const bool issue = one_lane();
        const uint32_t s0 = smem_u32(smem);
        auto boxes_of = [&](const I8Tile &t) { return CG == 2 ? 4 : (t.rows + 31) / 32; };   // of 32 rows
        auto load_w = [&](int stage, const I8Tile &t, int step) {
            const uint32_t fb = bar_full + 8 * stage;
            const int half = step >= half_steps ? 1 : 0;
            const int x0 = (step - half * half_steps) * per * kFChunk;
            if (leader)
                mbar_arrive_expect_tx(fb, CG * per * (boxes_of(t) * 32 + (BWD ? 128 : b_rows)) * kFChunk);
            const int n0 = t.wt * T;
            for (int u = 0; u < per; ++u) {
                const uint32_t sB = s0 + stage * stage_bytes + u * chunk_bytes + a_bytes;
                const int x = x0 + u * kFChunk;
                if (BWD) {
                    tma_load_3d<CG>(sB, half ? &tmW2 : &tmW, n0 + (int)rank * 128, x, t.e, fb);
                } else if (GATED && CG == 1) {
                    tma_load_3d<CG>(sB, &tmW, x, n0, t.e, fb);
                    tma_load_3d<CG>(sB + T * kFChunk, &tmW2, x, n0, t.e, fb);
                } else if (GATED) {
                    tma_load_3d<CG>(sB, rank ? &tmW2 : &tmW, x, n0, t.e, fb);
                } else {
                    tma_load_3d<CG>(sB, &tmW, x, n0 + (int)rank * b_rows, t.e, fb);
                }
            }
        };
        auto load_x = [&](int stage, const I8Tile &t, int step) {
            const uint32_t fb = bar_full + 8 * stage;
            const int half = step >= half_steps ? 1 : 0;
            const int x0 = (step - half * half_steps) * per * kFChunk;
            const int row = t.row0 + half * (int)args.M + (int)rank * 128;
            const int boxes = boxes_of(t);
            for (int u = 0; u < per; ++u) {
                const uint32_t sA = s0 + stage * stage_bytes + u * chunk_bytes;
                if (CG == 2)
                    tma_load_2d_pair(sA, &tmX, x0 + u * kFChunk, row, fb);
                else
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(sA + b * 32 * kFChunk, &tmX, x0 + u * kFChunk, row + 32 * b, fb);
            }
        };
        int e = 0, early = 0;                     // steps of the first tile whose weight is on its way
        if (unit < tiles) {
            const I8Tile t = plan.find(unit, e);
            early = min(steps, stages);
            if (issue)
                for (int i = p; i < early; i += P)
                    load_w(i, t, i);
        }
        grid_dep_wait();                          // codes and scales of the rows
        e = 0;
        int stage = p;
        uint32_t phase = 0;
        bool ok = true;
        int skip = p;                             // steps of the others before this producer's next one
        for (int tile = unit; ok && tile < tiles; tile += units) {
            const I8Tile t = plan.find(tile, e);
            int c = skip;
            for (; c < steps; c += P) {
                const bool fresh = early <= p;
                if (fresh && !mbar_wait(bar_empty + 8 * stage, phase ^ 1u, abort_flag, args.status)) {
                    ok = false;
                    break;
                }
                early -= P;
                if (issue) {
                    if (fresh)
                        load_w(stage, t, c);
                    load_x(stage, t, c);
                }
                stage += P;
                if (stage >= stages) {
                    stage = p;
                    phase ^= 1u;
                }
            }
            skip = c - steps;
        }
        // let every load that was issued land (and be consumed) before the CTA exits
        for (int st = p; st < stages; st += P) {
            (void)mbar_wait(bar_empty + 8 * stage, phase ^ 1u, abort_flag, args.status);
            stage += P;
            if (stage >= stages) {
                stage = p;
                phase ^= 1u;
            }
        }
        __syncwarp();
    } else if (warp >= kScale && warp < kIssuer) {
        // ------------------------------------------------------------ scale warps (every CTA)
        // Warp s takes every S-th group of four blocks.  Its words: this CTA's rows of A, all of B's.
        constexpr int S = Cfg::kScaleWarps;
        const int s = warp - kScale;
        const uint32_t full_leader = CG == 2 ? mapa_shared(bar_sf_full, 0) : bar_sf_full;
        const int64_t expert_blocks = (int64_t)args.nbs * args.kbs;
        grid_dep_wait();
        int e = 0, next = s, count = 0;           // groups so far
        bool ok = true;
        for (int tile = unit; ok && tile < tiles; tile += units) {
            const I8Tile t = plan.find(tile, e);
            const int mine = min(max(t.rows - (int)rank * 128, 0), 128);
            const int n0 = t.wt * T, nb0 = n0 / kFp8Block;
            for (int g2 = 0; g2 < groups * args.halves; ++g2, ++count) {
                if (count != next)
                    continue;
                next += S;
                const int half = g2 >= groups ? 1 : 0, grp = g2 - half * groups;
                const int slot = count % kFSfSlots;
                uint32_t aw[4], bw[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 32 * j + lane;
                    aw[j] = r < mine ? __ldg(args.words + (int64_t)g2 * args.M + t.row0 + (int)rank * 128 + r) : 0u;
                }
                // bytes of the (at most three) blocks that the tile's channels lie in, four along the
                // sum: lanes 4 b + i; gated: the up projection's at 16 + 4 b + i
                uint32_t v = 0;
                {
                    const int b = (lane >> 2) & 3, ch = nb0 + b, kb = kFp8Group * grp + (lane & 3);
                    const bool second = GATED ? lane >= 16 : half != 0;
                    const int nb = BWD ? kb : ch, kk = BWD ? ch : kb;
                    if (nb < args.nbs && kk < args.kbs)
                        v = __ldg((second ? args.ws[1] : args.ws[0]) + t.e * expert_blocks + (int64_t)nb * args.kbs + kk);
                    v <<= 8 * (lane & 3);
                    v |= __shfl_xor_sync(0xffffffffu, v, 1);
                    v |= __shfl_xor_sync(0xffffffffu, v, 2);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = 32 * j + lane;
                    const bool second = GATED && r >= T;
                    const int ch = n0 + (second ? r - T : r);
                    bw[j] = __shfl_sync(0xffffffffu, v, 4 * ((ch / kFp8Block - nb0) & 3) + (second ? 16 : 0));
                }
                if (!fp8_warp_wait<CG>(bar_sf_empty + 8 * slot, ((uint32_t)(count / kFSfSlots) & 1u) ^ 1u, abort_flag,
                                       args.status, lane)) {
                    ok = false;
                    break;
                }
                uint4 *line = reinterpret_cast<uint4 *>(smem + Cfg::kSfOff + slot * kFSfBytes) + lane;
                line[0] = make_uint4(aw[0], aw[1], aw[2], aw[3]);
                line[32] = make_uint4(bw[0], bw[1], bw[2], bw[3]);
                if (CG == 2)
                    line[64] = make_uint4(bw[4], bw[5], bw[6], bw[7]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2)
                        mbar_arrive_release_cluster(full_leader + 8 * slot);
                    else
                        mbar_arrive(full_leader + 8 * slot);
                }
            }
        }
        __syncwarp();
    } else if (warp == kIssuer) {
        // ------------------------------------------------------------ MMA issuer (leader)
        if (leader) {
            const bool issue = one_lane();
            const uint32_t s0 = smem_u32(smem);
            const uint64_t dA0 = sdesc_sw128(s0), dB0 = sdesc_sw128(s0 + a_bytes);
            const uint64_t dS0 = sdesc_sf(s0 + Cfg::kSfOff);
            const uint32_t stage16 = stage_bytes >> 4, chunk16 = chunk_bytes >> 4;
            const uint32_t idesc0 = Cfg::kIdesc | (uint32_t)(cols >> 3) << 17;
            int stage = 0;
            uint32_t phase = 0;
            uint64_t dA = dA0, dB = dB0;
            int count = 0, group = 0;
            bool ok = true;
            for (int tile = unit; ok && tile < tiles; tile += units, ++count) {
                const uint32_t acc = tmem_base + ((count & 1) ? kFSlot1 : 0u);
                // the columns that the previous tile's accumulator shares with this one have been read
                // (and all of the one before it)
                if (count >= 1 && !fp8_wait<CG>(bar_acc_empty, (uint32_t)((count - 1) & 1), abort_flag, args.status))
                    break;
                tc_fence_after();
                for (int c = 0; c < steps && ok; ++c) {
                    const int kb0 = (c >= half_steps ? c - half_steps : c) * per;
                    if (!fp8_wait<CG>(bar_full + 8 * stage, phase, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    for (int u = 0; u < per && kb0 + u < args.blocks; ++u) {
                        const int kb = kb0 + u;
                        if ((kb & 3) == 0) {               // the next four blocks' scales
                            const int slot = group % kFSfSlots;
                            const uint32_t parity = (uint32_t)(group / kFSfSlots) & 1u;
                            if (!(CG == 2 ? fp8_wait_acquire(bar_sf_full + 8 * slot, parity, abort_flag, args.status)
                                          : mbar_wait(bar_sf_full + 8 * slot, parity, abort_flag, args.status))) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            if (issue) {
                                const uint32_t sf = tmem_base + kFScaleCol + 16 * (group & 1);
                                const uint64_t d = dS0 + (uint32_t)(slot * kFSfBytes >> 4);
                                if (CG == 2) {
                                    tmem_cp2_32x128b_x4(sf + 8, d);
                                    tmem_cp2_32x128b_x4(sf, d + 32);
                                    tmem_cp2_32x128b_x4(sf + 4, d + 64);
                                    tc_commit2_both(bar_sf_empty + 8 * slot);
                                } else {
                                    tmem_cp_32x128b_x4(sf + 8, d);
                                    tmem_cp_32x128b_x4(sf, d + 32);
                                    tc_commit(bar_sf_empty + 8 * slot);
                                }
                            }
                            ++group;
                        }
                        if (issue) {
                            const uint32_t sf = tmem_base + kFScaleCol + 16 * ((group - 1) & 1);
                            const uint32_t idesc = idesc0 | (uint32_t)(kb & 3) << 4 | (uint32_t)(kb & 3) << 29;
#pragma unroll
                            for (int k = 0; k < kFChunk / 32; ++k)
                                mma_fp8<CG>(acc, dA + u * chunk16 + 2 * k, dB + u * chunk16 + Cfg::kBStep16 * k, idesc,
                                            sf + 8, sf, (c > 0 || u > 0 || k > 0) ? 1u : 0u);
                        }
                    }
                    if (!ok)
                        break;
                    if (issue) {
                        if (CG == 2)
                            tc_commit2_both(bar_empty + 8 * stage);
                        else
                            tc_commit(bar_empty + 8 * stage);
                    }
                    dA += stage16;
                    dB += stage16;
                    if (++stage == stages) {
                        stage = 0;
                        dA = dA0;
                        dB = dB0;
                        phase ^= 1u;
                    }
                }
                if (ok && issue) {
                    if (CG == 2)
                        tc_commit2_both(bar_acc_full + 8 * (count & 1));
                    else
                        tc_commit(bar_acc_full + 8 * (count & 1));
                }
            }
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
    } else {
        // ------------------------------------------------------------ epilogue (every CTA)
        // Warp w: lanes 32 (w % 4) .. + 31, the first (w < 4) or second half of the tile's channels, 32
        // at a time, from the end that the other accumulator shares.
        const int wq = warp & 3, wh = warp >> 2;
        const uint32_t acc_empty_leader = CG == 2 ? mapa_shared(bar_acc_empty, 0) : bar_acc_empty;
        uint8_t *patch = smem + Cfg::kPatchOff + warp * kFPatchBytes;
        const bool ybf = args.out_bf16 != 0;
        const int chunks = (T + 31) / 32, c_first = wh ? (chunks + 1) / 2 : 0;
        const int own = wh ? chunks - c_first : (chunks + 1) / 2;
        int count = 0, e = 0;
        grid_dep_wait();
        for (int tile = unit; tile < tiles; tile += units, ++count) {
            const I8Tile t = plan.find(tile, e);
            const int slot = count & 1;
            if (!fp8_warp_wait<CG>(bar_acc_full + 8 * slot, (uint32_t)((count >> 1) & 1), abort_flag, args.status, lane))
                break;
            tc_fence_after();
            const uint32_t acc = tmem_base + ((uint32_t)(32 * wq) << 16) + (slot ? kFSlot1 : 0u);
            const int first_row = (int)rank * 128 + 32 * wq;
            const int rows = min(t.rows - first_row, 32);              // (may be negative)
            const int64_t row = (int64_t)t.row0 + first_row;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2)
                        mbar_arrive_cluster(acc_empty_leader);
                    else
                        mbar_arrive(acc_empty_leader);
                }
            };
            if (own == 0)
                release();
            for (int i = 0; i < own; ++i) {
                const int c = 32 * (c_first + (slot ? i : own - 1 - i));
                const int64_t col = (int64_t)t.wt * T + c;
                const int64_t left = args.width - col;
                const int live = (int)min((int64_t)min(T - c, 32), left);
                float o[32];
                uint32_t r[32];
                __syncwarp();
                if constexpr (GATED) {
                    uint32_t q[32];
                    tmem_ld_32cols(acc + c, r);
                    tmem_ld_32cols(acc + T + c, q);
                    tmem_wait_ld();
                    if (i == 0)
                        release();
                    if (rows <= 0 || live <= 0)
                        continue;
                    if (args.act == 0) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[j] = act_value<0>(__uint_as_float(r[j])) * __uint_as_float(q[j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[j] = act_value<1>(__uint_as_float(r[j])) * __uint_as_float(q[j]);
                    }
                    if (args.g_out) {
                        float f[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            f[j] = __uint_as_float(r[j]);
                        store_cols32(f, patch, lane, args.g_out, row, col, args.width, rows, live, true);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            f[j] = __uint_as_float(q[j]);
                        store_cols32(f, patch, lane, args.u_out, row, col, args.width, rows, live, true);
                    }
                } else {
                    tmem_ld_32cols(acc + c, r);
                    tmem_wait_ld();
                    if (i == 0)
                        release();
                    if (rows <= 0 || live <= 0)
                        continue;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        o[j] = __uint_as_float(r[j]);
                }
                if (SQ_DCHECK(row + rows <= args.M && col + live <= args.width, args.status))
                    store_cols32(o, patch, lane, args.y, row, col, args.width, rows, live, ybf);
            }
        }
        __syncwarp();
    }

    tc_fence_before();
    if (CG == 2)
        cluster_meet();                               // no CTA leaves while its peer may still signal it
    else
        __syncthreads();
    tc_fence_after();
    if (warp == kIssuer) {
        if (CG == 2)
            tmem_dealloc2(tmem_base, kFTmemCols);
        else
            tmem_dealloc(tmem_base, kFTmemCols);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
namespace {

typedef CUresult (*PFN_encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                               const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// byte matrices [outer, rows, inner] in a row, boxes of box_rows x 128; what lies outside one of them
// reads as 0 (a box that ends behind an expert's last row does not see the next expert's)
bool byte_map(CUtensorMap *m, const void *base, int64_t inner, int64_t rows, int64_t outer, int box_rows)
{
    static PFN_encode fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return false;
        fn = reinterpret_cast<PFN_encode>(p);
    }
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)outer};
    const cuuint64_t strides[2] = {(cuuint64_t)inner, (cuuint64_t)(inner * rows)};
    const cuuint32_t box[3] = {kFChunk, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, outer > 0 ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG, int MODE>
cudaError_t launch_fp8(const Fp8GemmLaunch &g, int tile, int sms, cudaStream_t stream)
{
    using Cfg = Fp8Cfg<CG, MODE>;
    constexpr bool BWD = MODE == kFp8Bwd, GATED = MODE == kFp8Gated;
    constexpr int kMaxDev = 64;
    static unsigned long long ctx_seen[kMaxDev];
    static int resident_units[kMaxDev];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev)
        return cudaErrorInvalidDevice;
    const unsigned long long ctx = current_context_id();
    if (ctx == 0 || ctx_seen[dev] != ctx) {
        cudaError_t e = cudaFuncSetAttribute(sq_fp8_kernel<CG, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Cfg::kSmemBytes);
        if (e != cudaSuccess)
            return e;
        int units = sms / CG;
        if (CG == 2) {                            // not every SM can pair up inside its GPC
            cudaLaunchConfig_t q = {};
            q.gridDim = dim3(2 * units);
            q.blockDim = dim3(Cfg::kThreads);
            q.dynamicSmemBytes = Cfg::kSmemBytes;
            int resident = 0;
            e = cudaOccupancyMaxActiveClusters(&resident, sq_fp8_kernel<CG, MODE>, &q);
            (void)cudaGetLastError();
            if (e == cudaSuccess && resident > 0 && resident < units)
                units = resident;
        }
        resident_units[dev] = units;
        ctx_seen[dev] = ctx;
    }
    const int64_t Em = g.E > 0 ? g.E : 1;
    const int64_t summed = BWD ? g.N : g.K;
    const int halves = BWD && g.gated ? 2 : 1;
    const int b_rows = BWD ? 128 : GATED ? (CG == 2 ? tile : 2 * tile) : tile / CG;
    CUtensorMap tmX, tmW, tmW2;
    const int w_rows = BWD ? 128 : GATED ? tile : tile / CG;
    bool ok = byte_map(&tmX, g.codes, summed, halves * g.M, 0, CG == 2 ? 128 : 32) &&
              byte_map(&tmW, g.wcodes[0], g.K, g.N, Em, w_rows);
    tmW2 = tmW;
    if (g.gated)
        ok = ok && byte_map(&tmW2, g.wcodes[1], g.K, g.N, Em, w_rows);
    if (!ok)
        return cudaErrorInvalidValue;
    Fp8Args a;
    a.offsets = g.offsets;
    a.words = g.words;
    a.ws[0] = g.wscales[0];
    a.ws[1] = g.gated ? g.wscales[1] : g.wscales[0];
    a.y = g.y;
    a.g_out = g.g_out;
    a.u_out = g.u_out;
    a.status = g.status;
    a.M = g.M;
    a.width = BWD ? g.K : g.N;
    a.E = g.E;
    a.act = g.act;
    a.out_bf16 = g.out_bf16;
    a.N = (int)g.N;
    a.nbs = (int)((g.N + kFp8Block - 1) / kFp8Block);
    a.kbs = (int)((g.K + kFp8Block - 1) / kFp8Block);
    a.blocks = (int)((summed + kFp8Block - 1) / kFp8Block);
    a.halves = halves;
    a.tile = tile;
    a.a_rows = CG == 2 || g.M >= 128 ? 128 : (int)((g.M + 31) / 32 * 32);
    a.per = 1;
    const int chunk = (a.a_rows + b_rows) * kFChunk;
    if (CG == 1)
        while (a.per < 4 && 2 * a.per * chunk * 4 <= Cfg::kRing)
            a.per *= 2;
    a.stages = Cfg::kRing / (a.per * chunk);
    if (a.stages > Cfg::kMaxStages)
        a.stages = Cfg::kMaxStages;
    a.stages = a.stages / Cfg::kProducers * Cfg::kProducers;
    // dependent launch: set-up and the first weight tiles overlap the rounding in front
    int64_t work = (a.width + tile - 1) / tile * ((g.M + 128 * CG - 1) / (128 * CG) + (g.E > 0 ? g.E : 0));
    const int units = (int)(work < resident_units[dev] ? work : resident_units[dev]);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * CG));
    cfg.blockDim = dim3(Cfg::kThreads);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sq_fp8_kernel<CG, MODE>, tmX, tmW, tmW2, a);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmLaunch &g, int sms, cudaStream_t stream)
{
    const int64_t rows = g.E > 1 ? (g.M + g.E - 1) / g.E : g.M;        // (experts: the mean)
    const int64_t width = g.bwd ? g.K : g.N;
    if (rows > 128) {
        if (g.bwd)
            return launch_fp8<2, kFp8Bwd>(g, 256, sms, stream);
        return g.gated ? launch_fp8<2, kFp8Gated>(g, 128, sms, stream) : launch_fp8<2, kFp8Fwd>(g, 256, sms, stream);
    }
    if (g.bwd)
        return launch_fp8<1, kFp8Bwd>(g, 128, sms, stream);
    // one CTA: an equal share of the channels for every SM
    const int most = g.gated ? 64 : 128;
    int64_t tile = (width + sms - 1) / sms;
    tile = (tile + 15) / 16 * 16;
    if (tile > most || g.E > 0)
        tile = most;
    return g.gated ? launch_fp8<1, kFp8Gated>(g, (int)tile, sms, stream)
                   : launch_fp8<1, kFp8Fwd>(g, (int)tile, sms, stream);
}

}  // namespace sq
