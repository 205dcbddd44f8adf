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
// CTA (CG = 1) or CTA pair (CG = 2, 256 x 256 tiles) per SM, persistent, 6 warps:
// 0-3 epilogue, 4 TMA producer, 5 MMA issuer and tensor-memory allocator.  Two
// accumulators in tensor memory: the next tile's MMAs run while one drains.
// Weight tiles of the first stages are fetched before the kernel waits for the
// quantisation kernel in front of it.
//
// Few tiles: each is split over the summed axis into as many items as there are
// idle CTAs; an item writes its 32-bit partial sums to its own slab and counts up,
// and the one that counts last adds them all and finishes the tile.  Integer sums
// do not depend on the order, so the result does not either.
#include <cuda.h>

#include "sq_device.cuh"
#include "sq_kernels.h"
#include "sq_ptx.cuh"

namespace sq {

constexpr int kI8Rank = 16;
constexpr int kChunk = 128;                       // summed values (bytes) per stage
constexpr int kI8Threads = 192;
constexpr int kMaxExperts = 1024;
constexpr int kMinSplitChunks = 4;                // a split sums at least 512 values

template <int NT, int CG, bool BWD>
struct I8Cfg {
    static constexpr int kLaneTile = 128 * CG;                       // A rows of the tile
    static constexpr int kColsPerCta = NT / CG;                      // B rows (or columns) each CTA loads
    static constexpr int kABytes = 128 * kChunk;
    static constexpr int kBBytes = kColsPerCta * kChunk;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = (192 * 1024) / kStageBytes < 10 ? (192 * 1024) / kStageBytes : 10;
    static constexpr int kLowOff = kStages * kStageBytes;            // column factors [NT][16] fp32
    static constexpr int kScaleOff = kLowOff + NT * kI8Rank * 4;     // column scales [NT] fp32 (forward)
    static constexpr int kPlanOff = kScaleOff + NT * 4;              // start and prefix of every expert
    static constexpr int kBarOff = kPlanOff + (2 * kMaxExperts + 4) * 4;
    static constexpr int kNumBars = 2 * kStages + 5;                 // full, empty, acc_full[2], acc_empty[2], drain
    static constexpr int kSmemBytes = kBarOff + 8 * kNumBars + 32 + 1024;
    static constexpr uint32_t kTmemCols = 2 * NT < 32 ? 32 : 2 * NT;
    static constexpr uint32_t kIdesc = (2u << 4) | (1u << 7) | (1u << 10) | (BWD ? 1u << 16 : 0u) |
                                       ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(kLaneTile >> 4) << 24);
    static constexpr uint32_t kBStep16 = BWD ? (32u * 128u) >> 4 : 2u;   // B descriptor step per MMA (32 values)
};

struct I8Args {
    const int32_t *offsets;
    const float *scales;      // per token
    const float *low;         // per token [M, 16] or NULL
    const float *wscales;     // per channel (forward)
    const uint16_t *factor;   // lane-side (forward: lora_up) or column-side (backward: lora_down) factor
    void *y;
    int32_t *slabs;
    uint32_t *counters;
    uint32_t *status;
    int64_t M, N, K;          // N, K of one expert
    int E;
    int out_bf16;
    int slab_items;           // slabs there is room for
};

// where an item's tile lies
struct I8Tile {
    int e;                    // expert
    int row0, rows;           // first token and tokens of the tile
    int wt;                   // tile along the weight: channels (forward) or input features (backward)
};

// The tiles of all experts in a row: expert e has ceil(rows / tok_tile) token tiles, each times
// `wts` weight tiles; the token tile changes fastest, so that the tiles which share a weight
// tile run together.  Offsets are clamped to [0, M] and to their running maximum, so that the
// experts' rows never overlap or leave the matrix, whatever the offsets hold.
struct I8Plan {
    int32_t *start;           // [E + 1] first row of each expert
    int32_t *prefix;          // [E + 1] token tiles before each expert
    int E, wts, tok_tile;

    __device__ __forceinline__ void build(const int32_t *__restrict__ offsets, int64_t M, int tid, int threads)
    {
        for (int i = tid; i <= E; i += threads) {
            const int64_t o = offsets ? (int64_t)__ldg(offsets + i) : i == 0 ? 0 : M;
            start[i] = (int32_t)(o < 0 ? 0 : o > M ? M : o);
        }
        __syncthreads();
        if (tid < 32) {
            int32_t top = 0, sum = 0;             // running maximum and token tiles up to here
            for (int base = 0; base <= E; base += 32) {
                const int i = base + tid;
                int32_t v = i <= E ? start[i] : 0;
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) {
                    const int32_t up = __shfl_up_sync(0xffffffffu, v, x);
                    v = tid >= x ? max(v, up) : v;
                }
                v = max(v, top);
                const int32_t left = __shfl_up_sync(0xffffffffu, v, 1);
                int32_t n = i == 0 || i > E ? 0 : (v - (tid == 0 ? top : left) + tok_tile - 1) / tok_tile;
                top = __shfl_sync(0xffffffffu, v, 31);
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) {
                    const int32_t up = __shfl_up_sync(0xffffffffu, n, x);
                    n += tid >= x ? up : 0;
                }
                n += sum;
                sum = __shfl_sync(0xffffffffu, n, 31);
                if (i <= E) {
                    start[i] = v;
                    prefix[i] = n;
                }
            }
        }
        __syncthreads();
    }

    __device__ __forceinline__ int tiles() const
    {
        return prefix[E] * wts;
    }

    // tile number `tile`, below tiles(); e: a role's own walk, starting at 0 (its tiles only grow)
    __device__ __forceinline__ I8Tile find(int tile, int &e) const
    {
        while (tile >= prefix[e + 1] * wts)
            ++e;
        const int tts = prefix[e + 1] - prefix[e];
        const int i = tile - prefix[e] * wts;
        I8Tile t;
        t.e = e;
        t.wt = i / tts;
        t.row0 = start[e] + (i % tts) * tok_tile;
        t.rows = min(start[e + 1] - t.row0, tok_tile);
        return t;
    }
};

// Items per tile: with at most half as many tiles as units (CTAs or CTA pairs), the summed
// axis is split so that every unit has one, into at least kMinSplitChunks chunks each.
__host__ __device__ __forceinline__ int i8_splits(int tiles, int units, int chunks, int slab_items)
{
    if (tiles <= 0)
        return 1;
    int s = units / tiles;
    s = s < chunks / kMinSplitChunks ? s : chunks / kMinSplitChunks;
    s = s < slab_items / tiles ? s : slab_items / tiles;
    return s < 1 ? 1 : s;
}

template <int CG>
__device__ __forceinline__ bool acc_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag,
                                         uint32_t *status)
{
    return CG == 2 ? mbar_wait_cluster(bar, parity, abort_flag, status) : mbar_wait(bar, parity, abort_flag, status);
}

// sum over r of low[r] f[r], pairs of neighbouring r in packed arithmetic
__device__ __forceinline__ float dot16(const uint64_t (&f)[8], const float *__restrict__ low)
{
    uint64_t s = f2_pack(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 v = *reinterpret_cast<const float4 *>(low + 4 * j);
        s = f2_fma(f2_pack(v.x, v.y), f[2 * j], s);
        s = f2_fma(f2_pack(v.z, v.w), f[2 * j + 1], s);
    }
    float a, b;
    f2_unpack(s, a, b);
    return __fadd_rn(a, b);
}

template <int NT, int CG, bool BWD>
__global__ void __cluster_dims__(CG, 1, 1) __launch_bounds__(kI8Threads, 1)
    sq_i8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const I8Args args)
{
    using Cfg = I8Cfg<NT, CG, BWD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *col_low = reinterpret_cast<float *>(smem + Cfg::kLowOff);
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
    volatile uint32_t *last_item = tmem_holder + 3;

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
            mbar_init(bar_acc_empty + 8 * i, 4 * CG);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 5) {
        if (CG == 2) {
            tmem_alloc2(smem_u32(tmem_holder), Cfg::kTmemCols);
            tmem_relinquish2();
        } else {
            tmem_alloc(smem_u32(tmem_holder), Cfg::kTmemCols);
            tmem_relinquish();
        }
    }
    if (warp == 4 && lane == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    // the offsets are an input of the call: they are there before the kernel in front starts
    I8Plan plan;
    plan.E = args.E > 0 ? args.E : 1;
    plan.start = plan_mem;
    plan.prefix = plan_mem + kMaxExperts + 1;
    plan.wts = BWD ? (int)(args.K / NT) : (int)((args.N + Cfg::kLaneTile - 1) / Cfg::kLaneTile);
    plan.tok_tile = BWD ? Cfg::kLaneTile : NT;
    plan.build(args.E > 0 ? args.offsets : nullptr, args.M, threadIdx.x, kI8Threads);
    tc_fence_before();
    if (CG == 2)
        cluster_sync();                           // barriers of both CTAs initialised, TMEM allocated
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;

    const int tiles = plan.tiles();
    const int units = (int)gridDim.x / CG;
    const int unit = (int)blockIdx.x / CG;
    const int chunks = (int)((BWD ? args.N : args.K) / kChunk);
    const int splits = i8_splits(tiles, units, chunks, args.slab_items);
    const int items = tiles * splits;

    if (warp == 4) {
        // ------------------------------------------------------------ producer (every CTA)
        if (lane == 0) {
            // weight operand of stage `stage`, chunk c of tile t, and the row operand
            auto load_w = [&](int stage, const I8Tile &t, int c) {
                const uint32_t sA = smem_u32(smem + stage * Cfg::kStageBytes), fb = bar_full + 8 * stage;
                const int n0 = t.e * (int)args.N;
                const uint32_t dst = BWD ? sA + Cfg::kABytes : sA;
                const void *tm = BWD ? &tmB : &tmA;
                const int x = BWD ? t.wt * NT + (int)rank * Cfg::kColsPerCta : c * kChunk;
                const int y = BWD ? n0 + c * kChunk : n0 + t.wt * Cfg::kLaneTile + (int)rank * 128;
                if (CG == 2)
                    tma_load_2d_pair(dst, tm, x, y, fb);
                else
                    tma_load_2d(dst, tm, x, y, fb);
            };
            auto load_x = [&](int stage, const I8Tile &t, int c) {
                const uint32_t sA = smem_u32(smem + stage * Cfg::kStageBytes), fb = bar_full + 8 * stage;
                const uint32_t dst = BWD ? sA : sA + Cfg::kABytes;
                const void *tm = BWD ? &tmA : &tmB;
                const int y = t.row0 + (int)rank * (BWD ? 128 : Cfg::kColsPerCta);
                if (CG == 2)
                    tma_load_2d_pair(dst, tm, c * kChunk, y, fb);
                else
                    tma_load_2d(dst, tm, c * kChunk, y, fb);
            };
            int e = 0;
            int early = 0;                        // stages whose weight operand is on its way
            if (unit < items) {
                const I8Tile t = plan.find(unit / splits, e);
                const int s = unit % splits;
                const int c0 = (int)((int64_t)chunks * s / splits), c1 = (int)((int64_t)chunks * (s + 1) / splits);
                early = min(c1 - c0, Cfg::kStages);
                for (int i = 0; i < early; ++i) {
                    if (leader)
                        mbar_arrive_expect_tx(bar_full + 8 * i, CG * Cfg::kStageBytes);
                    load_w(i, t, c0 + i);
                }
            }
            grid_dep_wait();                      // codes, scales and low-rank input of the rows
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int item = unit; item < items && ok; item += units) {
                const I8Tile t = plan.find(item / splits, e);
                const int s = item % splits;
                const int c0 = (int)((int64_t)chunks * s / splits), c1 = (int)((int64_t)chunks * (s + 1) / splits);
                for (int c = c0; c < c1; ++c) {
                    if (early > 0) {              // the first stages of the first item
                        --early;
                    } else {
                        if (!mbar_wait(bar_empty + 8 * stage, phase ^ 1u, abort_flag, args.status)) {
                            ok = false;
                            break;
                        }
                        if (leader)
                            mbar_arrive_expect_tx(bar_full + 8 * stage, CG * Cfg::kStageBytes);
                        load_w(stage, t, c);
                    }
                    load_x(stage, t, c);
                    if (++stage == Cfg::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // let every load that was issued land (and be consumed) before the CTA exits
            for (int st = 0; st < Cfg::kStages; ++st) {
                (void)mbar_wait(bar_empty + 8 * stage, phase ^ 1u, abort_flag, args.status);
                if (++stage == Cfg::kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        // ------------------------------------------------------------ MMA issuer (leader)
        if (leader && lane == 0) {
            const uint32_t s0 = smem_u32(smem);
            const uint64_t dA0 = sdesc_sw128(s0), dB0 = sdesc_sw128(s0 + Cfg::kABytes);
            constexpr uint32_t kStage16 = Cfg::kStageBytes >> 4;
            int stage = 0;
            uint32_t phase = 0;
            int count = 0;
            bool ok = true;
            for (int item = unit; item < items && ok; item += units, ++count) {
                const int s = item % splits;
                const int n = (int)((int64_t)chunks * (s + 1) / splits) - (int)((int64_t)chunks * s / splits);
                const uint32_t acc = tmem_base + ((count & 1) ? (uint32_t)NT : 0u);
                // the tile before last (same accumulator) has left tensor memory
                if (count >= 2 && !acc_wait<CG>(bar_acc_empty + 8 * (count & 1), (uint32_t)(((count >> 1) - 1) & 1),
                                                abort_flag, args.status))
                    break;
                tc_fence_after();
                for (int c = 0; c < n; ++c) {
                    if (!acc_wait<CG>(bar_full + 8 * stage, phase, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a = dA0 + stage * kStage16, b = dB0 + stage * kStage16;
#pragma unroll
                    for (int k = 0; k < kChunk / 32; ++k)
                        mma_i8<CG>(acc, a + 2 * k, b + Cfg::kBStep16 * k, Cfg::kIdesc, (c > 0 || k > 0) ? 1u : 0u);
                    if (CG == 2)
                        tc_commit2_both(bar_empty + 8 * stage);
                    else
                        tc_commit(bar_empty + 8 * stage);
                    if (++stage == Cfg::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) {
                    if (CG == 2)
                        tc_commit2_both(bar_acc_full + 8 * (count & 1));
                    else
                        tc_commit(bar_acc_full + 8 * (count & 1));
                }
            }
            // all issued MMAs must finish before tensor memory is released
            if (CG == 2)
                tc_commit2_local(bar_drain);
            else
                tc_commit(bar_drain);
            (void)mbar_wait(bar_drain, 0, abort_flag, args.status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue (every CTA)
        // Thread 0 alone waits (bounded); the 128 threads meet at named barrier 1, so that they
        // always take the same way out.
        const int et = threadIdx.x;
        const uint32_t acc_empty_leader = CG == 2 ? mapa_shared(bar_acc_empty, 0) : bar_acc_empty;
        const bool ybf = args.out_bf16 != 0;
        const bool with_low = args.low != nullptr;
        const int64_t width = BWD ? args.K : args.N;      // columns of y
        grid_dep_wait();
        int e = 0;
        int count = 0;
        for (int item = unit; item < items; item += units, ++count) {
            const int tile = item / splits, split = item % splits;
            const I8Tile t = plan.find(tile, e);
            const int slot = count & 1;
            named_barrier_sync(1, 128);                    // the previous tile's column factors are used up
            if (BWD) {
                if (with_low)
                    for (int c = et; c < NT; c += 128) {
                        const uint4 *src = reinterpret_cast<const uint4 *>(
                            args.factor + ((int64_t)t.e * args.K + t.wt * NT + c) * kI8Rank);
                        const uint4 p = __ldg(src), q = __ldg(src + 1);
                        const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float2 *>(col_low + c * kI8Rank + 2 * j) =
                                make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
                    }
            } else {
                for (int c = et; c < NT; c += 128)
                    col_scale[c] = c < t.rows ? args.scales[t.row0 + c] : 0.0f;
                if (with_low)
                    for (int i = et; i < NT * 4; i += 128)
                        if ((i >> 2) < t.rows)
                            reinterpret_cast<float4 *>(col_low)[i] =
                                reinterpret_cast<const float4 *>(args.low + (int64_t)t.row0 * kI8Rank)[i];
            }
            // this lane's channel (forward) or token (backward): scale and low-rank values
            const int in_tile = (int)rank * 128 + et;
            const int64_t at = BWD ? (int64_t)t.row0 + in_tile : (int64_t)t.wt * Cfg::kLaneTile + in_tile;
            const bool live = BWD ? in_tile < t.rows : at < args.N;
            float lane_scale = 0.0f;
            uint64_t lane_low[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                lane_low[j] = 0;
            if (live) {
                if (BWD) {
                    lane_scale = args.scales[at];
                    if (with_low)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 v = reinterpret_cast<const float4 *>(args.low + at * kI8Rank)[j];
                            lane_low[2 * j] = f2_pack(v.x, v.y);
                            lane_low[2 * j + 1] = f2_pack(v.z, v.w);
                        }
                } else {
                    lane_scale = __ldg(args.wscales + (int64_t)t.e * args.N + at);
                    if (with_low) {
                        const uint4 *src =
                            reinterpret_cast<const uint4 *>(args.factor + ((int64_t)t.e * args.N + at) * kI8Rank);
                        const uint4 p = __ldg(src), q = __ldg(src + 1);
                        const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            lane_low[j] = f2_pack(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
                    }
                }
            }
            if (et == 0)
                *verdict = acc_wait<CG>(bar_acc_full + 8 * slot, (uint32_t)((count >> 1) & 1), abort_flag, args.status)
                               ? 1u
                               : 0u;
            named_barrier_sync(1, 128);
            if (*verdict == 0u)
                break;
            tc_fence_after();
            const uint32_t acc = tmem_base + ((uint32_t)(32 * warp) << 16) + (slot ? (uint32_t)NT : 0u);
            constexpr int CH = NT < 32 ? NT : 32;
            const int live_cols = BWD ? NT : t.rows;

            // the raw sums of CH columns, column q * CH on
            auto load_acc = [&](int q, uint32_t (&r)[CH]) {
                __syncwarp();
                if constexpr (CH == 16)
                    tmem_ld_16cols(acc + CH * q, r);
                else
                    tmem_ld_32cols(acc + CH * q, r);
                tmem_wait_ld();
            };
            constexpr int64_t kSlab = (int64_t)NT * 128;
            int32_t *slab0 = args.slabs + ((int64_t)tile * splits * CG + rank) * kSlab + et;   // + split CG kSlab + 128 c
            bool finish = true;
            if (splits > 1) {
                int32_t *mine = slab0 + (int64_t)split * CG * kSlab;
                for (int q = 0; q * CH < live_cols; ++q) {
                    uint32_t r[CH];
                    load_acc(q, r);
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        mine[128 * (CH * q + i)] = (int32_t)r[i];
                }
                __threadfence();
                named_barrier_sync(1, 128);
                if (et == 0) {
                    *last_item = atomicAdd(args.counters + tile * CG + rank, 1u) == (uint32_t)(splits - 1) ? 1u : 0u;
                    __threadfence();
                }
                named_barrier_sync(1, 128);
                finish = *last_item != 0u;
            }
            // ... and with the other items' partial sums
            auto load_sum = [&](int q, uint32_t (&r)[CH]) {
                load_acc(q, r);
                if (splits > 1)
                    for (int s = 0; s < splits; ++s)
                        if (s != split) {
                            const int32_t *p = slab0 + (int64_t)s * CG * kSlab + 128 * CH * q;
#pragma unroll
                            for (int i = 0; i < CH; ++i)
                                r[i] += (uint32_t)__ldcg(p + 128 * i);
                        }
            };
            if constexpr (BWD) {
                if (finish) {
                    // strides 1 .. 16 inside each 32 columns, back into tensor memory
                    for (int q = 0; q < NT / 32; ++q) {
                        uint32_t r[32];
                        load_sum(q, r);
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = __fmul_rn(__int2float_rn((int32_t)r[i]), lane_scale);
#pragma unroll
                        for (int h = 1; h <= 16; h <<= 1)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if ((i & h) == 0) {
                                    const float a = v[i], b = v[i + h];
                                    v[i] = __fadd_rn(a, b);
                                    v[i + h] = __fsub_rn(a, b);
                                }
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            r[i] = __float_as_uint(v[i]);
                        tmem_st_32cols(acc + 32 * q, r);
                    }
                    tmem_wait_st();
                    // strides 32, 64, 128 over four columns of each 32, the low-rank term, the store
                    for (int c4 = 0; c4 < 32; c4 += 4) {
                        uint32_t r[8][4];
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            tmem_ld_4cols(acc + 32 * j + c4, r[j]);
                        tmem_wait_ld();
                        float v[8][4];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[j][i] = __uint_as_float(r[j][i]);
#pragma unroll
                        for (int h = 1; h <= 4; h <<= 1)
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if ((j & h) == 0)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const float a = v[j][i], b = v[j + h][i];
                                        v[j][i] = __fadd_rn(a, b);
                                        v[j + h][i] = __fsub_rn(a, b);
                                    }
                        if (!live)
                            continue;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float o[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                o[i] = __fmul_rn(v[j][i], 0.0625f);
                                if (with_low)
                                    o[i] = __fadd_rn(o[i], dot16(lane_low, col_low + (32 * j + c4 + i) * kI8Rank));
                            }
                            const int64_t col = (int64_t)t.wt * NT + 32 * j + c4;
                            if (!SQ_DCHECK(at < args.M && col + 4 <= width, args.status))
                                continue;
                            if (ybf)
                                *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(args.y) + at * width + col) =
                                    make_uint2(f32x2_to_bf16x2_bits(o[0], o[1]), f32x2_to_bf16x2_bits(o[2], o[3]));
                            else
                                *reinterpret_cast<float4 *>(reinterpret_cast<float *>(args.y) + at * width + col) =
                                    make_float4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
            } else {
                if (finish)
                    for (int q = 0; q * CH < live_cols; ++q) {
                        uint32_t r[CH];
                        load_sum(q, r);
                        if (!live)
                            continue;
#pragma unroll
                        for (int i = 0; i < CH; ++i) {
                            const int c = CH * q + i;
                            if (c >= t.rows)
                                break;
                            float o = __fmul_rn(__int2float_rn((int32_t)r[i]), __fmul_rn(col_scale[c], lane_scale));
                            if (with_low)
                                o = __fadd_rn(o, dot16(lane_low, col_low + c * kI8Rank));
                            const int64_t row = (int64_t)t.row0 + c;
                            if (!SQ_DCHECK(row < args.M && at < width, args.status))
                                continue;
                            if (ybf)
                                reinterpret_cast<uint16_t *>(args.y)[row * width + at] = (uint16_t)f32_to_bf16_bits(o);
                            else
                                reinterpret_cast<float *>(args.y)[row * width + at] = o;
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
        cluster_sync();                               // no CTA leaves while its peer may still signal it
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 5) {
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

// Token tile by the rows of one product (experts: their mean).  Up to 128 rows one tile takes
// them all, the narrowest that does; above, 256 x 256 tiles of a CTA pair.
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

constexpr int kSlabSms = 148;                     // CTAs the slabs are sized for (a B200's SMs)

int64_t slab_items(bool bwd, int E, int64_t M, int64_t N, int64_t K)
{
    const Shape sh = pick_shape(bwd, E, M);
    const int units = kSlabSms / sh.cg;
    if (E > 0)                                    // how the rows spread is known on the device only
        return units;
    const int64_t tok = bwd ? 128 * sh.cg : sh.nt, tts = (M + tok - 1) / tok;
    const int64_t wts = bwd ? K / sh.nt : (N + 128 * sh.cg - 1) / (128 * sh.cg);
    if (tts * wts > units)
        return 0;
    const int s = i8_splits((int)(tts * wts), units, (int)((bwd ? N : K) / kChunk), units);
    return s > 1 ? tts * wts * s : 0;
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
            q.blockDim = dim3(kI8Threads);
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
    // 128-byte wide boxes: weight codes [E N, K], row codes [M, K] (backward [M, N])
    CUtensorMap tmW, tmX;
    bool ok = make_tmap(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.wcodes, (uint64_t)g.K, (uint64_t)(Em * g.N), 128,
                        128, CU_TENSOR_MAP_SWIZZLE_128B);
    ok &= make_tmap(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.codes, (uint64_t)(BWD ? g.N : g.K), (uint64_t)g.M, 128,
                    BWD ? 128 : Cfg::kColsPerCta, CU_TENSOR_MAP_SWIZZLE_128B);
    if (!ok)
        return cudaErrorInvalidValue;
    I8Args a;
    a.offsets = g.offsets;
    a.scales = g.scales;
    a.low = g.low;
    a.wscales = g.wscales;
    a.factor = g.factor;
    a.y = g.y;
    a.slabs = g.slabs;
    a.counters = g.counters;
    a.status = g.status;
    a.M = g.M;
    a.N = g.N;
    a.K = g.K;
    a.E = g.E;
    a.out_bf16 = g.out_bf16;
    a.slab_items = (int)slab_items(BWD, g.E, g.M, g.N, g.K);
    // dependent launch: set-up and the first weight tiles overlap the quantisation in front
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(resident_units[dev] * CG));
    cfg.blockDim = dim3(kI8Threads);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sq_i8_kernel<NT, CG, BWD>, BWD ? tmX : tmW, BWD ? tmW : tmX, a);
}

}  // namespace

size_t i8_slab_bytes(bool bwd, int E, int64_t M, int64_t N, int64_t K)
{
    const Shape sh = pick_shape(bwd, E, M);
    return (size_t)slab_items(bwd, E, M, N, K) * sh.cg * 128 * sh.nt * 4;
}

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
