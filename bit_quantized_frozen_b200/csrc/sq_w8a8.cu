// sq_w8a8.cu -- products of 8-bit integers with one scale per token and one per
// channel, dense or grouped by expert, on tcgen05 (kind::i8, 32-bit integer sums
// in tensor memory, exact).
//
//   forward   y[m, n]  = s_x[m] s_w[n] sum_k q_x[m, k] Q[n, k] + low[m] . lora_up[n]
//   backward  dx[m, :] = H256( s_g[m] sum_n q_g[m, n] Q[n, :] ) + low[m] . lora_down[k]
//
// The tensor-memory lanes hold the side whose factors a thread can keep in
// registers, the columns the other side:
//   forward   lanes = output channels (A = Q, K-major), columns = NT tokens
//             (B = q_x, K-major).  A warp then writes 32 neighbouring outputs of
//             one token, the channel's scale and its 16 low-rank values stay in
//             registers, and few tokens make a narrow tile (NT = 16) that reads
//             each weight byte once.
//   backward  lanes = tokens (A = q_g, K-major), columns = 256 input features
//             (B = Q, N-major: the sum runs over Q's rows, which are never
//             transposed).  A thread holds a whole 256-block of its token, so the
//             rotation is done on the accumulator.
//
// The low-rank product (rank 16) is part of the epilogue.  Forward it is 8 packed fp32 FMAs a
// value, with the lane's factors in registers and the tokens' in shared memory; mma.sync on bf16
// terms would hold up the integer MMAs (4480 tokens, N = 16384, K = 6144: 315 us a call against
// 360; 6001 rows of 8 experts, 6144 x 4096: 166 against 200, short runs both).  Backward the FMA
// units are busy with the rotation and mma.sync on three bf16 terms is faster (8192 rows of 64
// experts, 2816 x 2048: 136 us against 150; 509 tokens: 24 against 29).  Two terms, 16 bits, would
// take 150.1 us of such a call in a long run instead of 151.1.
//
// Measured on B200, 4480 x 16384 x 6144, in a short run: forward 267 us (3.38 POP/s, the integer
// tensor pipe 90 % active at 1.6 GHz), backward 295 to 315 us (82 %).  With the quantisation a call
// takes 308 and 378 us in a short run, 365 and 450 us after a second of calls, when the power cap
// has taken the clocks further down.  24 tokens on the same weight: 26 us a call (the weight's
// 101 MB at 49 % of the DRAM rate in the product, the rest is the start and the end of one tile).
//
// CTA (CG = 1) or CTA pair (CG = 2, 256 x 256 tiles) per SM, persistent: 4 or 8 epilogue
// warps, one to four TMA producers, an MMA issuer that also allocates tensor memory.  Two
// accumulators in tensor memory: the next tile's MMAs run while one drains.
// Weight tiles of the first stages are fetched before the kernel waits for the
// quantisation kernel in front of it.
//
// Forward, a tile's MMAs and loads cover only the boxes of tokens that it has (the instruction's
// column count is set per tile), so that an expert with few rows costs few.  Backward the tokens
// are the lanes: a tile is loaded, multiplied and rotated for 256 tokens, however many it has.
//
// Few tokens (CG = 1) are bound by the weight's bytes: each CTA takes an equal share of
// all channels, to four of them, as tiles of up to 128, so that every SM reads the same
// amount.  (Splitting the summed axis over idle SMs instead, with the partial sums joined
// through L2, cost 4 us at 16 tokens and 15 us and more with 256-column tiles.)
#include <cuda.h>

#include "sq_device.cuh"
#include "sq_kernels.h"
#include "sq_ptx.cuh"
#include "sq_w8a8.cuh"
#include "sq_w8a8_stage.h"

namespace sq {

constexpr int kChunk = kI8Chunk;

template <int NT, int CG, bool BWD>
struct I8Cfg {
    static constexpr int kLaneTile = 128 * CG;                       // A rows of the tile
    static constexpr int kColsPerCta = NT / CG;                      // B rows (or columns) each CTA loads
    static constexpr int kBox = NT >= 64 ? 32 : 16;                  // token rows per TMA box (forward)
    static constexpr int kABytes = 128 * kChunk;
    static constexpr int kBBytes = kColsPerCta * kChunk;
    static constexpr int kStageBytes = kABytes + kBBytes;
    // epilogue warps: one per 32 lanes and, in wide tiles, per half of the columns
    static constexpr int kColHalves = NT >= 64 ? 2 : 1;
    static constexpr int kEpiThreads = 128 * kColHalves;
    // producer warps, each with its own stages
    static constexpr int kProducers = CG == 2 ? 1 : i8_producers(NT);
    static constexpr int kThreads = kEpiThreads + 32 * kProducers + 32;   // + MMA issuer
    // bytes from one column's low-rank values to the next in shared memory (bf16 backward, fp32
    // forward): the four columns that a warp reads at once lie in different banks
    static constexpr int kLowPitch = BWD ? 48 : 80;
    static constexpr int kPatchBytes = BWD ? 0 : 2 * 8 * 36 * 4;     // a warp's two store patches
    // stages: fixed for a CTA pair; with CG = 1 as many as fit with the A rows that the CTA's
    // tiles have (the MMAs read 128 rows all the same: behind the tile's own lie other bytes of
    // the CTA's shared memory, and their lanes of the accumulator are not looked at)
    static constexpr int kRing = CG == 1 ? i8_ring_bytes(NT) : (BWD ? 192 : 160) * 1024;
    static constexpr int kStages = CG == 1 ? kI8MaxStages : kRing / kStageBytes;
    static constexpr int kPatchOff = kRing;
    static constexpr int kLowOff = kPatchOff + (kEpiThreads / 32) * kPatchBytes;
    static constexpr int kScaleOff = kLowOff + NT * kLowPitch;       // column scales [NT] fp32 (forward)
    static constexpr int kPlanOff = kScaleOff + NT * 4;              // start and prefix of every expert
    static constexpr int kBarOff = kPlanOff + (2 * kMaxExperts + 4) * 4;
    static constexpr int kNumBars = 2 * kStages + 5;                 // full, empty, acc_full[2], acc_empty[2], drain
    static constexpr int kSmemBytes = kBarOff + 8 * kNumBars + 32 + 1024;
    static constexpr uint32_t kTmemCols = 2 * NT < 32 ? 32 : 2 * NT;
    // instruction descriptor, without columns / 8 << 17 and rows / 16 << 24
    static constexpr uint32_t kIdesc = (2u << 4) | (1u << 7) | (1u << 10) | (BWD ? 1u << 16 : 0u);
    static constexpr uint32_t kBStep16 = BWD ? (32u * 128u) >> 4 : 2u;   // B descriptor step per MMA (32 values)
};

struct I8Args {
    const int32_t *offsets;
    const float *scales;      // per token
    const float *low;         // per token [M, 16] or NULL
    const float *wscales;     // per channel (forward)
    const uint16_t *factor;   // lane-side (forward: lora_up) or column-side (backward: lora_down) factor
    void *y;
    uint32_t *status;
    int64_t M, N, K;          // N, K of one expert
    int E;
    int out_bf16;
    int tok;                  // tokens of a tile (forward; at most NT)
    int box;                  // weight rows of a tmA box
};

// what a unit does next: tile t, its lanes (channels from n0 on; backward: tokens)
struct I8Work {
    I8Tile t;
    int n0, lanes;
};

// CG = 2: every units-th tile; CG = 1: the CTA's share of the channels
template <int CG, bool BWD>
struct I8Units {
    const I8Plan &plan;
    I8ChannelWalk share;
    int tile, tiles, units, e;
    int64_t N;

    __device__ __forceinline__ I8Units(const I8Plan &p, const I8ChannelWalk &c, int tiles_, int unit, int units_,
                                       int64_t N_)
        : plan(p), share(c), tile(unit), tiles(tiles_), units(units_), e(0), N(N_)
    {
    }
    __device__ __forceinline__ bool next(I8Work &w)
    {
        if (CG == 1) {
            if (!share.next())
                return false;
            w.t = plan.find(share.tile, e);
            w.n0 = share.n0;
            w.lanes = share.channels;
        } else {
            if (tile >= tiles)
                return false;
            w.t = plan.find(tile, e);
            w.n0 = BWD ? 0 : w.t.wt * 256;
            w.lanes = BWD ? w.t.rows : (int)min((int64_t)256, N - w.n0);
            tile += units;
        }
        return true;
    }
};

// one lane of the warp
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// the same in every lane (as it is already), told to the compiler
__device__ __forceinline__ int uniform(int v)
{
    return __shfl_sync(0xffffffffu, v, 0);
}

template <int CG>
__device__ __forceinline__ bool acc_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag,
                                         uint32_t *status)
{
    return CG == 2 ? mbar_wait_cluster(bar, parity, abort_flag, status) : mbar_wait(bar, parity, abort_flag, status);
}

template <int NT, int CG, bool BWD>
__global__ void __cluster_dims__(CG, 1, 1) __launch_bounds__(I8Cfg<NT, CG, BWD>::kThreads, 1)
    sq_i8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmBox, const __grid_constant__ CUtensorMap tmA64,
                 const __grid_constant__ CUtensorMap tmA16, const I8Args args)
{
    using Cfg = I8Cfg<NT, CG, BWD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *col_scale = reinterpret_cast<float *>(smem + Cfg::kScaleOff);
    int32_t *plan_mem = reinterpret_cast<int32_t *>(smem + Cfg::kPlanOff);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kBarOff);
    const uint32_t bar_full = smem_u32(bars);
    const uint32_t bar_empty = bar_full + 8 * Cfg::kStages;
    const uint32_t bar_acc_full = bar_empty + 8 * Cfg::kStages;
    const uint32_t bar_acc_empty = bar_acc_full + 16;
    const uint32_t bar_drain = bar_acc_empty + 16;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + Cfg::kNumBars);
    volatile uint32_t *abort_flag = tmem_holder + 1;
    volatile uint32_t *verdict = tmem_holder + 2;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int st = 0; st < Cfg::kStages; ++st) {
            mbar_init(bar_full + 8 * st, 1);
            mbar_init(bar_empty + 8 * st, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_acc_full + 8 * i, 1);
            mbar_init(bar_acc_empty + 8 * i, CG * Cfg::kEpiThreads / 32);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    constexpr int kProducer = Cfg::kEpiThreads / 32, kIssuer = kProducer + Cfg::kProducers;      // warps
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
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        if (!BWD)
            prefetch_tmap(&tmBox);
        if (CG == 1) {
            prefetch_tmap(&tmA64);
            prefetch_tmap(&tmA16);
        }
    }
    grid_dep_launch();                            // the next call's quantisation may be set up
    // the offsets are an input of the call: they are there before the kernel in front starts
    I8Plan plan;
    plan.E = args.E > 0 ? args.E : 1;
    plan.start = plan_mem;
    plan.prefix = plan_mem + kMaxExperts + 1;
    plan.wts = CG == 1 ? 1 : BWD ? (int)(args.K / NT) : (int)((args.N + Cfg::kLaneTile - 1) / Cfg::kLaneTile);
    plan.tok_tile = BWD ? Cfg::kLaneTile : args.tok;
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
    const I8ChannelWalk share(CG == 1 ? tiles : 0, args.N, unit, units);
    using Units = I8Units<CG, BWD>;
    auto all_work = [&]() { return Units(plan, share, tiles, unit, units, args.N); };
    // stages of equal chunks; CG = 1: as the CTA's share needs them
    I8Stages lay = {Cfg::kABytes, Cfg::kStageBytes, 1, Cfg::kStageBytes, Cfg::kStages};
    if (CG == 1)
        lay = i8_stages(i8_stage_rows(share.largest(), args.box), Cfg::kBBytes, Cfg::kRing, Cfg::kProducers);
    const int a_bytes = lay.a_bytes, chunk_bytes = lay.chunk_bytes, per = lay.per, stage_bytes = lay.stage_bytes;
    const int stages = lay.stages;
    // CG = 1: tiles of at most 64 channels take the 64-row MMA, which reads half as much of A and puts
    // 16 rows into each quarter of the lanes
    const bool m64 = CG == 1 && a_bytes <= 64 * kChunk;
    const int steps = (int)(((BWD ? args.N : args.K) / kChunk + per - 1) / per);      // stages of a tile
    // columns of the accumulator a tile uses (forward: its tokens, in whole boxes of both CTAs)
    auto columns = [&](const I8Tile &t) {
        return BWD ? NT : (t.rows + CG * Cfg::kBox - 1) / (CG * Cfg::kBox) * (CG * Cfg::kBox);
    };

    if (warp >= kProducer && warp < kIssuer) {
        // ------------------------------------------------------------ producers (every CTA)
        // Producer p fills stages p, p + P, ... with every P-th step of the unit's work.  The whole
        // warp runs the loop on uniform values and one lane issues, which keeps the address
        // arithmetic off the path between two copies.
        constexpr int P = Cfg::kProducers;
        const int p = warp - kProducer;
        const bool issue = elect_one();
        const uint32_t s0 = smem_u32(smem);
        auto load = [&](const void *tm, uint32_t dst, int x, int y, uint32_t bar) {
            if (CG == 2)
                tma_load_2d_pair(dst, tm, x, y, bar);
            else
                tma_load_2d(dst, tm, x, y, bar);
        };
        // what is the same for every step of a tile
        struct Aim {
            int wrow, rows;           // weight: first row, rows (forward; in whole 8-row groups)
            int xrow, mine;           // row operand: first row, rows
            uint32_t bytes;           // of a stage (both CTAs)
        };
        auto aim_at = [&](const I8Work &w) {
            Aim m;
            const int cols = columns(w.t);
            m.rows = CG == 1 ? i8_weight_rows(w.lanes, args.box) : 128;
            const int copied = CG == 1 ? i8_copied_rows(m.rows, args.box) : 128;
            m.wrow = w.t.e * (int)args.N + (BWD ? 0 : w.n0 + (int)rank * 128);
            m.mine = BWD ? 128 : cols / CG;
            m.xrow = w.t.row0 + (int)rank * m.mine;
            m.bytes = per * (CG * copied + cols) * kChunk;
            m.wrow = uniform(m.wrow);
            m.rows = uniform(m.rows);
            m.xrow = uniform(m.xrow);
            m.mine = uniform(m.mine);
            m.bytes = (uint32_t)uniform((int)m.bytes);
            return m;
        };
        auto load_w = [&](int stage, const Aim &m, int wt, int step) {
            const uint32_t fb = bar_full + 8 * stage;
            if (leader)
                mbar_arrive_expect_tx(fb, m.bytes);
            for (int u = 0; u < per; ++u) {
                const uint32_t sA = s0 + stage * stage_bytes + u * chunk_bytes;
                const int x = (step * per + u) * kChunk;
                if (BWD) {
                    load(&tmB, sA + a_bytes, wt * NT + (int)rank * Cfg::kColsPerCta, m.wrow + x, fb);
                } else if (CG == 2) {
                    load(&tmA, sA, x, m.wrow, fb);
                } else {
                    i8_weight_copies(m.rows, args.box, [&](int kind, int at) {
                        load(kind == 0 ? &tmA : kind == 1 ? &tmA64 : &tmA16, sA + at * kChunk, x, m.wrow + at, fb);
                    });
                }
            }
        };
        auto load_x = [&](int stage, const Aim &m, int step) {
            const uint32_t fb = bar_full + 8 * stage;
            for (int u = 0; u < per; ++u) {
                const uint32_t sX = s0 + stage * stage_bytes + u * chunk_bytes + (BWD ? 0 : a_bytes);
                const int x = (step * per + u) * kChunk;
                if (BWD || m.mine == Cfg::kColsPerCta) {
                    load(BWD ? &tmA : &tmB, sX, x, m.xrow, fb);
                } else {
                    for (int r = 0; r < m.mine; r += Cfg::kBox)
                        load(&tmBox, sX + r * kChunk, x, m.xrow + r, fb);
                }
            }
        };
        I8Work w;
        int early = 0;                            // steps of the first tile whose weight operand is on its way
        if (Units first = all_work(); first.next(w)) {
            early = min(steps, stages);
            const Aim m = aim_at(w);
            const int wt = uniform(w.t.wt);
            if (issue)
                for (int i = p; i < early; i += P)
                    load_w(i, m, wt, i);
        }
        grid_dep_wait();                          // codes, scales and low-rank input of the rows
        int stage = p;
        uint32_t phase = 0;
        bool ok = true;
        int skip = p;                             // steps of the others before this producer's next one
        for (Units work = all_work(); ok && work.next(w);) {
            const Aim m = aim_at(w);
            const int wt = uniform(w.t.wt);
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
                        load_w(stage, m, wt, c);
                    load_x(stage, m, c);
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
    } else if (warp == kIssuer) {
        // ------------------------------------------------------------ MMA issuer (leader)
        if (leader) {
            const bool issue = elect_one();
            const uint32_t s0 = smem_u32(smem);
            const uint64_t dA0 = sdesc_sw128(s0), dB0 = sdesc_sw128(s0 + a_bytes);
            const uint32_t stage16 = stage_bytes >> 4, chunk16 = chunk_bytes >> 4;
            int stage = 0;
            uint32_t phase = 0;
            uint64_t dA = dA0, dB = dB0;
            int count = 0;
            bool ok = true;
            I8Work w;
            for (Units work = all_work(); ok && work.next(w); ++count) {
                const uint32_t idesc = Cfg::kIdesc | (uint32_t)uniform(columns(w.t) >> 3) << 17 |
                                       (uint32_t)(m64 ? 4 : Cfg::kLaneTile >> 4) << 24;
                const uint32_t acc = tmem_base + ((count & 1) ? (uint32_t)NT : 0u);
                // the tile before last (same accumulator) has left tensor memory
                if (count >= 2 && !acc_wait<CG>(bar_acc_empty + 8 * (count & 1), (uint32_t)(((count >> 1) - 1) & 1),
                                                abort_flag, args.status))
                    break;
                tc_fence_after();
                for (int c = 0; c < steps; ++c) {
                    if (!acc_wait<CG>(bar_full + 8 * stage, phase, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (issue) {
                        for (int u = 0; u < per; ++u)
#pragma unroll
                            for (int k = 0; k < kChunk / 32; ++k)
                                mma_i8<CG>(acc, dA + u * chunk16 + 2 * k, dB + u * chunk16 + Cfg::kBStep16 * k, idesc,
                                           (c > 0 || u > 0 || k > 0) ? 1u : 0u);
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
        // Thread 0 alone waits (bounded); the epilogue's threads meet at named barrier 1, so that
        // they always take the same way out.
        const int et = threadIdx.x;
        constexpr int ET = Cfg::kEpiThreads;
        const int wq = warp & 3;                           // lanes 32 wq .. + 31 of tensor memory
        const int wh = warp >> 2;                          // which warp of those lanes
        const int g = lane >> 2, q = lane & 3;             // place in a fragment
        const uint32_t acc_empty_leader = CG == 2 ? mapa_shared(bar_acc_empty, 0) : bar_acc_empty;
        uint8_t *col_low = smem + Cfg::kLowOff;
        uint8_t *patch = smem + Cfg::kPatchOff + warp * Cfg::kPatchBytes;
        const bool ybf = args.out_bf16 != 0;
        const bool with_low = args.low != nullptr;
        const int64_t width = BWD ? args.K : args.N;      // columns of y
        grid_dep_wait();
        int count = 0;
        I8Work w;
        for (Units work = all_work(); work.next(w); ++count) {
            const I8Tile &t = w.t;
            const int slot = count & 1;
            named_barrier_sync(1, ET);                     // the previous tile's column factors are used up
            if (with_low) {
                // the columns' low-rank values: lora_down's rows (backward), the tokens' t (forward)
                const char *src = BWD ? reinterpret_cast<const char *>(
                                            args.factor + ((int64_t)t.e * args.K + (int64_t)t.wt * NT) * kI8Rank)
                                      : reinterpret_cast<const char *>(args.low + (int64_t)t.row0 * kI8Rank);
                constexpr int kPieces = BWD ? 2 : 4;       // of 16 bytes a column
                const int pieces = kPieces * (BWD ? NT : t.rows);
                // (with many tiles a CTA the copies run under the loads below; with one, plain loads
                // end 1 us earlier)
                for (int i = et; i < pieces; i += ET) {
                    uint8_t *dst = col_low + i / kPieces * Cfg::kLowPitch + i % kPieces * 16;
                    if (CG == 2 && !BWD)
                        cp_async16(smem_u32(dst), src + 16 * i, true);
                    else
                        *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(src + 16 * i);
                }
            }
            static_assert(BWD || NT <= ET, "a token's scale for each thread");
            const float token_scale = !BWD && et < t.rows ? args.scales[t.row0 + et] : 0.0f;
            // the lanes' scales and low-rank values (lane r of a fragment half: 16 h + g + 8 i)
            const int span = m64 ? 16 : 32;                // rows of the tile in a quarter of the lanes
            const int lane0 = (int)rank * 128 + span * wq; // first row of the warp in the tile
            const int64_t base = (BWD ? t.row0 : w.n0) + lane0;
            // (rows behind the tile's last one repeat that one; their sums are not stored)
            const float lscale = BWD ? args.scales[t.row0 + min(lane0 + lane, w.lanes - 1)] : 0.0f;
            float fscale[2][2];                            // forward: per fragment row
            uint64_t lane_low[2][2][BWD ? 1 : 8];          // forward: lora_up's rows
            uint32_t ufrag[2][BWD ? kLowParts : 1][4];     // backward: A operand of the low-rank product
            int64_t lrow[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    lrow[h][i] = min(lane0 + 16 * h + g + 8 * i, w.lanes - 1);
                    lrow[h][i] += BWD ? (int64_t)t.row0 : (int64_t)t.e * args.N + w.n0;
                    if (!BWD)
                        fscale[h][i] = __ldg(args.wscales + lrow[h][i]);
                }
            if constexpr (BWD) {
                float2 v[2][2][2];                         // ranks 2 q + 8 k, 2 q + 8 k + 1
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            v[h][i][k] = with_low ? *reinterpret_cast<const float2 *>(args.low + lrow[h][i] * kI8Rank +
                                                                                      2 * q + 8 * k)
                                                  : make_float2(0.0f, 0.0f);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t x[kLowParts], y[kLowParts];
                            split3(v[h][i][k].x, x);
                            split3(v[h][i][k].y, y);
#pragma unroll
                            for (int p = 0; p < kLowParts; ++p)
                                ufrag[h][p][i + 2 * k] = x[p] | y[p] << 16;
                        }
            } else {
                uint4 v[2][2][2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            v[h][i][k] = with_low ? __ldg(reinterpret_cast<const uint4 *>(args.factor + lrow[h][i] * kI8Rank) + k)
                                                  : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        pairs16(v[h][i][0], v[h][i][1], lane_low[h][i]);
            }
            if (!BWD && et < NT)
                col_scale[et] = token_scale;
            if (et == 0)
                *verdict = acc_wait<CG>(bar_acc_full + 8 * slot, (uint32_t)((count >> 1) & 1), abort_flag, args.status)
                               ? 1u
                               : 0u;
            if (CG == 2 && !BWD)
                cp_async_wait_all();
            named_barrier_sync(1, ET);
            if (*verdict == 0u)
                break;
            tc_fence_after();
            const uint32_t acc = tmem_base + ((uint32_t)(32 * wq) << 16) + (slot ? (uint32_t)NT : 0u);
            if constexpr (BWD) {
                // strides 1 .. 16 inside each 32 columns, back into tensor memory
                for (int c = 4 * wh; c < 4 * wh + 4; ++c) {
                    uint32_t r[32];
                    __syncwarp();
                    tmem_ld_32cols(acc + 32 * c, r);
                    tmem_wait_ld();
                    uint64_t v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float a = __fmul_rn(__int2float_rn((int32_t)r[2 * i]), lscale);
                        const float b = __fmul_rn(__int2float_rn((int32_t)r[2 * i + 1]), lscale);
                        v[i] = f2_pack(__fadd_rn(a, b), __fsub_rn(a, b));
                    }
#pragma unroll
                    for (int h = 1; h <= 8; h <<= 1)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if ((i & h) == 0) {
                                const uint64_t a = v[i], b = v[i + h];
                                v[i] = f2_add(a, b);
                                v[i + h] = f2_sub(a, b);
                            }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float a, b;
                        f2_unpack(v[i], a, b);
                        r[2 * i] = __float_as_uint(a);
                        r[2 * i + 1] = __float_as_uint(b);
                    }
                    tmem_st_32cols(acc + 32 * c, r);
                }
                tmem_wait_st();
                tc_fence_before();
                named_barrier_sync(1, ET);             // both halves of the columns are written
                tc_fence_after();
                // strides 32, 64, 128 over columns 16 wh .. + 15 of each 32, as fragments of
                // 16 tokens; the low-rank term; the store (32-byte runs of a row)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t r[8][2][4];
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        tmem_ld_frag2(acc + ((uint32_t)(16 * h) << 16) + 32 * j + 16 * wh, r[j]);
                    tmem_wait_ld();
                    uint64_t v[8][2][2];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[j][i >> 1][i & 1] = f2_pack(__uint_as_float(r[j][i >> 1][2 * (i & 1)]),
                                                          __uint_as_float(r[j][i >> 1][2 * (i & 1) + 1]));
#pragma unroll
                    for (int x = 1; x <= 4; x <<= 1)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if ((j & x) == 0)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint64_t a = v[j][i >> 1][i & 1], b = v[j + x][i >> 1][i & 1];
                                    v[j][i >> 1][i & 1] = f2_add(a, b);
                                    v[j + x][i >> 1][i & 1] = f2_sub(a, b);
                                }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int col = 32 * j + 16 * wh;
                        float low[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
                        if (with_low) {                // B: 16 columns (two groups of 8) x 16 ranks
                            uint32_t b[4];
                            ldmatrix_x4<false>(smem_u32(col_low) +
                                                   (col + 8 * (lane >> 4) + (lane & 7)) * Cfg::kLowPitch +
                                                   16 * ((lane >> 3) & 1),
                                               b);
#pragma unroll
                            for (int p = kLowParts - 1; p >= 0; --p) {
                                mma_16816(low[0], ufrag[h][p], b[0], b[1]);
                                mma_16816(low[1], ufrag[h][p], b[2], b[3]);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {  // group i >> 1, fragment rows g + 8 (i & 1)
                            const int row = 16 * h + g + 8 * (i & 1);
                            float a, b;
                            f2_unpack(v[j][i >> 1][i & 1], a, b);
                            a = __fmaf_rn(a, 0.0625f, low[i >> 1][2 * (i & 1)]);
                            b = __fmaf_rn(b, 0.0625f, low[i >> 1][2 * (i & 1) + 1]);
                            const int64_t at = (base + row) * width + (int64_t)t.wt * NT + col + 8 * (i >> 1) + 2 * q;
                            if (lane0 + row < w.lanes && SQ_DCHECK(at + 2 <= args.M * width, args.status)) {
                                if (ybf)
                                    *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(args.y) + at) =
                                        f32x2_to_bf16x2_bits(a, b);
                                else
                                    *reinterpret_cast<float2 *>(reinterpret_cast<float *>(args.y) + at) =
                                        make_float2(a, b);
                            }
                        }
                    }
                }
            } else {
                // this warp's columns: 16 at a time, in turn with the other warp of its lanes
                constexpr int kStep = 16 * Cfg::kColHalves;
                const int c_begin = 16 * wh, c_end = t.rows;
                // the sums of 16 columns as fragments [16 channels][8 tokens][4]
                auto load_acc = [&](int c, uint32_t (&r)[2][2][4]) {
                    __syncwarp();
                    tmem_ld_frag2(acc + c, r[0]);
                    tmem_ld_frag2(acc + (16u << 16) + c, r[1]);
                };
                const bool live = lane0 < w.lanes;
                auto finish16 = [&](int c, const uint32_t (&r)[2][2][4]) {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {          // 8 tokens
                        float o[2][4];
                        const float2 sx = *reinterpret_cast<const float2 *>(col_scale + c + 8 * n + 2 * q);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {      // token 2 q + j, fragment rows g + 8 i
                            const float4 *src = reinterpret_cast<const float4 *>(
                                col_low + (c + 8 * n + 2 * q + j) * Cfg::kLowPitch);
                            uint64_t f[8];
                            pairs16(src[0], src[1], src[2], src[3], f);
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    o[h][2 * i + j] = __fmaf_rn(__int2float_rn((int32_t)r[h][n][2 * i + j]),
                                                                __fmul_rn(j ? sx.y : sx.x, fscale[h][i]),
                                                                with_low ? dot16(lane_low[h][i], f) : 0.0f);
                        }
                        // through the warp's patch, so that a token's 32 channels leave in one run
                        uint8_t *buf = patch + n * (8 * 36 * 4);
                        const int64_t y0 = ((int64_t)t.row0 + c + 8 * n) * width + base;
                        if (ybf) {                         // [8 tokens] rows of 80 bytes
                            const uint32_t pairs[4] = {f32x2_to_bf16x2_bits(o[0][0], o[0][1]),
                                                       f32x2_to_bf16x2_bits(o[0][2], o[0][3]),
                                                       f32x2_to_bf16x2_bits(o[1][0], o[1][1]),
                                                       f32x2_to_bf16x2_bits(o[1][2], o[1][3])};
                            stmatrix_x4_trans(smem_u32(buf) + (lane & 7) * 80 + (lane >> 3) * 16, pairs);
                            __syncwarp();
                            if (CG == 2) {                 // (whole 32 channels: N % 128 == 0)
                                const int tok = lane >> 2, piece = lane & 3;
                                const uint4 v = *reinterpret_cast<const uint4 *>(buf + tok * 80 + piece * 16);
                                const int64_t at = y0 + tok * width + 8 * piece;
                                if (c + 8 * n + tok < t.rows && SQ_DCHECK(at + 8 <= args.M * width, args.status))
                                    *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(args.y) + at) = v;
                            } else {
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const int tok = (lane >> 3) + 4 * k, piece = lane & 7;
                                    const uint2 v = *reinterpret_cast<const uint2 *>(buf + tok * 80 + piece * 8);
                                    const int64_t at = y0 + tok * width + 4 * piece;
                                    if (c + 8 * n + tok < t.rows && 4 * piece < min(span, w.lanes - lane0) &&
                                        SQ_DCHECK(at + 4 <= args.M * width, args.status))
                                        *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(args.y) + at) = v;
                                }
                            }
                        } else {                           // [8 tokens] rows of 36 floats
                            float *f = reinterpret_cast<float *>(buf);
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    f[(2 * q + (i & 1)) * 36 + 16 * h + g + 8 * (i >> 1)] = o[h][i];
                            __syncwarp();
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int tok = (lane >> 3) + 4 * k, piece = lane & 7;
                                const float4 v = *reinterpret_cast<const float4 *>(f + tok * 36 + 4 * piece);
                                const int64_t at = y0 + tok * width + 4 * piece;
                                if (c + 8 * n + tok < t.rows && 4 * piece < min(span, w.lanes - lane0) &&
                                    SQ_DCHECK(at + 4 <= args.M * width, args.status))
                                    *reinterpret_cast<float4 *>(reinterpret_cast<float *>(args.y) + at) = v;
                            }
                        }
                    }
                };
                if (live) {
                    uint32_t r[2][2][4];
                    if (c_begin < c_end) {
                        load_acc(c_begin, r);
                        tmem_wait_ld();
                    }
                    for (int c = c_begin; c < c_end; c += kStep) {
                        uint32_t now[2][2][4];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            now[i >> 3][(i >> 2) & 1][i & 3] = r[i >> 3][(i >> 2) & 1][i & 3];
                        if (c + kStep < c_end)
                            load_acc(c + kStep, r);           // on its way while these 16 are finished
                        finish16(c, now);
                        tmem_wait_ld();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2)
                    mbar_arrive_cluster(acc_empty_leader + 8 * slot);
                else
                    mbar_arrive(acc_empty_leader + 8 * slot);
            }
        }
    }

    tc_fence_before();
    if (CG == 2)
        cluster_meet();                               // no CTA leaves while its peer may still signal it
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

struct Shape {
    int nt, cg;
};

// Token tile by the rows of one product (experts: the mean over all, since the host does not see
// the offsets): up to 128 the narrowest tile of one CTA that takes them, above 256 x 256 tiles of a
// CTA pair.  The two sides of each border, us a call:
//   rows                     16 | 17      32 | 33      64 | 65      128 | 129
//   dense, 6144 x 6144       16.4 17.6    19.0 20.2    20.7 23.0    24.8 24.9
//   dense, 2816 x 2048       11.8 12.3    12.5 13.5    13.8 15.1    16.6 13.1
//   64 experts, 2816 x 2048  73.9 75.3    77.4 83.1    88.0 94.6    113  109
// Rows that lie far from their mean pay for it: 2048 rows on one of 128 experts (2816 x 2048) take
// 16-token tiles and 81 us, on the only one 38 us.
Shape pick_shape(bool bwd, int E, int64_t M)
{
    if (bwd)
        return {256, 2};
    const int64_t rows = E > 1 ? (M + E - 1) / E : M;
    if (rows <= 16)
        return {16, 1};
    if (rows <= 32)
        return {32, 1};
    if (rows <= 64)
        return {64, 1};
    if (rows <= 128)
        return {128, 1};
    return {256, 2};
}

// CTA pairs: tokens of a tile.  Dense: of 256, 192, 128 and 64 the size with the least time, rounds
// of tiles times a chunk's cycles: the larger of the MMAs (2 a column) and the copies (16 KB of
// weight and 64 bytes a token per CTA, at about 64 bytes a cycle).  Experts: 256 (a tile's cost
// follows its rows).
int pair_tokens(int E, int64_t M, int64_t N, int pairs)
{
    if (E > 0)
        return 256;
    int best = 256;
    int64_t best_cost = INT64_MAX;
    for (int tok = 256; tok >= 64; tok -= 64) {
        const int64_t tiles = (M + tok - 1) / tok * ((N + 255) / 256);
        const int64_t cost = (tiles + pairs - 1) / pairs * (2 * tok > 256 + tok ? 2 * tok : 256 + tok);
        if (cost < best_cost) {
            best_cost = cost;
            best = tok;
        }
    }
    return best;
}

template <int NT, int CG, bool BWD>
cudaError_t launch_shape(const I8GemmLaunch &g, int sms, cudaStream_t stream)
{
    using Cfg = I8Cfg<NT, CG, BWD>;
    constexpr int kMaxDev = 64;
    static unsigned long long ctx_seen[kMaxDev];
    static int resident_units[kMaxDev];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev)
        return cudaErrorInvalidDevice;
    const unsigned long long ctx = current_context_id();
    if (ctx == 0 || ctx_seen[dev] != ctx) {
        cudaError_t e = cudaFuncSetAttribute(sq_i8_kernel<NT, CG, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
            e = cudaOccupancyMaxActiveClusters(&resident, sq_i8_kernel<NT, CG, BWD>, &q);
            (void)cudaGetLastError();
            if (e == cudaSuccess && resident > 0 && resident < units)
                units = resident;
        }
        resident_units[dev] = units;
        ctx_seen[dev] = ctx;
    }
    const int64_t Em = g.E > 0 ? g.E : 1;
    const int tok = BWD || CG == 1 ? NT : pair_tokens(g.E, g.M, g.N, resident_units[dev]);
    bool one_box = true;
    const int box = CG == 1 ? i8_whole_box(g.E, g.M, g.N, resident_units[dev], NT, &one_box) : 128;
    // 128-byte wide boxes: weight codes [E N, K], row codes [M, K] (backward [M, N]) by whole tiles
    // and by kBox tokens; maps that this call cannot use are not encoded
    CUtensorMap tmW, tmX, tmBox, tmW64, tmW16;
    auto weight_map = [&](CUtensorMap *m, int rows) {
        return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.wcodes, (uint64_t)g.K, (uint64_t)(Em * g.N), 128, rows,
                         CU_TENSOR_MAP_SWIZZLE_128B);
    };
    auto row_map = [&](CUtensorMap *m, int rows) {
        return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.codes, (uint64_t)(BWD ? g.N : g.K), (uint64_t)g.M, 128,
                         rows, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    bool ok = weight_map(&tmW, box) && row_map(&tmX, BWD ? 128 : Cfg::kColsPerCta);
    tmBox = tmX;
    tmW64 = tmW16 = tmW;
    if (!BWD && (g.E > 0 || tok != NT || (g.M % NT != 0 && !(NT <= 32 && g.M <= NT))))
        ok = ok && row_map(&tmBox, Cfg::kBox);
    if (!one_box)
        ok = ok && weight_map(&tmW64, 64) && weight_map(&tmW16, 16);
    if (!ok)
        return cudaErrorInvalidValue;
    I8Args a;
    a.offsets = g.offsets;
    a.scales = g.scales;
    a.low = g.low;
    a.wscales = g.wscales;
    a.factor = g.factor;
    a.y = g.y;
    a.status = g.status;
    a.M = g.M;
    a.N = g.N;
    a.K = g.K;
    a.E = g.E;
    a.out_bf16 = g.out_bf16;
    a.box = box;
    a.tok = tok;
    // dependent launch: set-up and the first weight tiles overlap the quantisation in front
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(resident_units[dev] * CG));
    cfg.blockDim = dim3(Cfg::kThreads);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sq_i8_kernel<NT, CG, BWD>, BWD ? tmX : tmW, BWD ? tmW : tmX, tmBox, tmW64, tmW16, a);
}

}  // namespace

cudaError_t launch_i8_gemm(const I8GemmLaunch &g, int sms, cudaStream_t stream)
{
    const Shape sh = pick_shape(g.bwd, g.E, g.M);
    if (g.bwd)
        return launch_shape<256, 2, true>(g, sms, stream);
    switch (sh.nt) {
    case 16:
        return launch_shape<16, 1, false>(g, sms, stream);
    case 32:
        return launch_shape<32, 1, false>(g, sms, stream);
    case 64:
        return launch_shape<64, 1, false>(g, sms, stream);
    case 128:
        return launch_shape<128, 1, false>(g, sms, stream);
    default:
        return launch_shape<256, 2, false>(g, sms, stream);
    }
}

}  // namespace sq
