// sq_w8a8_quant.cu -- the 8-bit operands of the integer products (sq_w8a8.cu):
// one int8 code per value and one fp32 scale per row, plus the row's low-rank
// input.
//
//   forward   r = H256 x            low = x lora_down   [M, 16]
//   backward  r = RN(dy s_w)        low = dy lora_up    [M, 16]
//   s = RN(max|r| / 127),  code = rint(RN(r RN(1 / s)))
//
// A code never leaves [-127, 127]: |r| <= max|r| and the three roundings move
// 127 by less than 2^-16.  A scale below 2^-120 is stored as 0 with zero codes
// (1 / s would leave fp32's range); a row with a NaN or an infinity in r gets
// the scale NaN, so its outputs are NaN.  Each product is rounded once, in the
// order written, so the codes are the same bits in any kernel.
//
// One kernel for both directions and any number of rows.  A warp takes 8 rows x
// 256 columns in registers: lane 4 g + q holds of row g the 16-byte pieces q,
// q + 4, ..., q + 28 of the block, so that a load touches whole 64-byte runs,
// strides 1, 2, 4 and 32, 64, 128 of the transform stay in a lane and strides 8
// and 16 pair lanes q ^ 1 and q ^ 2.  The same words, as loaded, are the B
// operand of mma m16n8k16 (8 rows, 16 values of K in the lanes' own order); the
// A operand is the block's 256 x 16 low-rank factor from shared memory, its rows
// picked in that order by ldmatrix.  A cluster of up to 8 CTAs with 8 warps each
// covers K <= 16384, so a row group is read once, its maximum and low-rank sums
// meet over distributed shared memory, and the codes leave from registers.  The
// clusters are persistent: a warp keeps its block's factor in shared memory from
// row group to row group (of one expert) and loads the next group, and its expert's
// factor where that is another one, while it transforms this one.  Longer rows (backward, N > 16384) take their blocks in
// turns and read them a second time for the codes.
//
// Measured on B200: forward 4480 x 6144 38 us (2.2 TB/s; with the low-rank input 46), backward
// 4480 x 16384 78 us (2.8 TB/s; 90).  Latency is the bound: 64 values a lane leave room for 16
// warps an SM, which use 47 % (36 %) of the issue slots, and every 8 rows wait for one exchange of
// the maximum.  Three CTAs an SM (spills), four-warp CTAs and exchanges with all loads at once
// (registers) were slower.
#include <cuda.h>

#include "sq_device.cuh"
#include "sq_kernels.h"
#include "sq_ptx.cuh"
#include "sq_w8a8.cuh"

namespace sq {

constexpr uint32_t kInfBits = 0x7F800000u;
constexpr int kQRows = 8;                         // rows of a group
constexpr int kQWarps = 8;                        // warps of a CTA at most
constexpr int kQMaxCluster = 8;
constexpr int kQFactorBytes = kHad * kI8Rank * 2; // 8 KB: a block's factor

// (everything twice: for even and odd groups)
struct QShared {
    uint32_t warp_max[2][kQWarps][kQRows];
    float warp_low[2][kQWarps][kI8Rank * kQRows];
    uint32_t max[2][kQMaxCluster][kQRows];        // from every CTA of the cluster
    float low[2][kQMaxCluster][kI8Rank * kQRows]; // (first CTA) from the others
    uint64_t max_bar[2], low_bar[2];              // count the bytes that have come
    uint32_t abort_flag;
    int32_t start[kMaxExperts + 1], prefix[kMaxExperts + 1];
};

// scale and reciprocal of a row from the largest |r| (NaN and infinity on top)
__device__ __forceinline__ void row_scale(uint32_t amax_bits, float &s, float &inv)
{
    s = __fdiv_rn(__uint_as_float(amax_bits), 127.0f);
    if (amax_bits >= kInfBits) {
        s = __uint_as_float(0x7FFFFFFFu);
        inv = 0.0f;
    } else if (s < 7.52316385e-37f) {             // 2^-120
        s = 0.0f;
        inv = 0.0f;
    } else {
        inv = __frcp_rn(s);
    }
}

// max(a, |b|, |c|), NaN if any is
__device__ __forceinline__ float absmax3(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}

// 4 bytes into another CTA's shared memory, counted on its barrier
__device__ __forceinline__ void st_async(uint32_t addr, uint32_t v, uint32_t bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];"
                 ::"r"(addr), "r"(v), "r"(bar) : "memory");
}

// a 16-byte chunk (factor row k, half h) of a block sits at chunk 2 k + h with bits 0 and 2
// flipped by bits 3 and 4 of k: the eight rows an ldmatrix matrix takes (k = 8 q + b and
// the next, q = 0..3) then lie in eight different bank groups
__device__ __forceinline__ uint32_t factor_chunk(uint32_t c)
{
    const uint32_t q = c >> 4;                    // (k >> 3)
    return c ^ ((q & 1u) | ((q & 2u) << 1));
}

// the lane's pieces q + 4 j of its row, x at piece q; the first `pieces` of them (8, or 4 in a
// half block at the end of a row), the others 0
template <bool BWD>
__device__ __forceinline__ void load_block(const uint16_t *__restrict__ x, int pieces, uint4 (&w)[8])
{
    if (BWD && pieces == 8) {                     // no zeros to lay out first (86 -> 80 us at 4480 x 16384)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = __ldg(reinterpret_cast<const uint4 *>(x) + 4 * j);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        w[j] = j < pieces ? __ldg(reinterpret_cast<const uint4 *>(x) + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
}

// this lane's row address for the ldmatrix of step (j, h): matrix m = lane / 8 takes rows
// k = 8 ((s >> 1) + 4 j) + 4 h + (s & 1) + 2 (m >> 1), s = lane % 8, half m & 1; steps lie a
// constant 1024 j + 128 h apart (they leave the flipped bits alone)
__device__ __forceinline__ uint32_t factor_lane(uint32_t factor, int lane)
{
    const uint32_t m = lane >> 3, s = lane & 7;
    return factor + 16 * factor_chunk(16 * (s >> 1) + 2 * (s & 1) + 4 * (m >> 1) + (m & 1));
}

// acc[16 ranks x 8 rows] += factor^T x of the block (two chains of sums, added at the end)
__device__ __forceinline__ void low_block(const uint4 (&w)[8], uint32_t lane_addr, float (&acc)[4])
{
    float odd[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t a[4], b[4];
        ldmatrix_x4<true>(lane_addr + 1024 * j, a);
        ldmatrix_x4<true>(lane_addr + 1024 * j + 128, b);
        mma_16816(acc, a, w[j].x, w[j].y);
        mma_16816(odd, b, w[j].z, w[j].w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        acc[i] = __fadd_rn(acc[i], odd[i]);
}

// the lane's 64 values as pairs p[4 j + i], widened from bf16
__device__ __forceinline__ void widen(const uint4 (&w)[8], uint64_t (&p)[32])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t v[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[4 * j + i] = f2_pack(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xFFFF0000u));
    }
}

// H256 of them without the final 1/16, strides 1, 2, 4 | 8, 16 | 32, 64, 128; stride 1 is folded
// into the widening (mixed bf16 / fp32 arithmetic, one rounding each, the same bits)
__device__ __forceinline__ void fwht_rows8(const uint4 (&w)[8], uint64_t (&p)[32], int lane)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t v[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = __uint_as_float(v[i] << 16);
            float sum, diff;
            asm("{\n\t.reg .b16 h0, h1, m1;\n\tmov.b32 {h0, h1}, %2;\n\tmov.b16 m1, 0xBF80;\n\t"
                "add.rn.f32.bf16 %0, h1, %3;\n\t"
                "fma.rn.f32.bf16 %1, h1, m1, %3;\n\t}"
                : "=f"(sum), "=f"(diff) : "r"(v[i]), "f"(lo));
            p[4 * j + i] = f2_pack(sum, diff);
        }
    }
#pragma unroll
    for (int h = 1; h <= 2; h <<= 1)              // strides 2, 4
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if ((j & h) == 0) {
                const uint64_t a = p[j], b = p[j + h];
                p[j] = f2_add(a, b);
                p[j + h] = f2_sub(a, b);
            }
#pragma unroll
    for (int x = 1; x <= 2; x <<= 1) {            // strides 8, 16
        const float sg = (lane & x) == 0 ? 1.0f : -1.0f;
        const uint64_t sg2 = f2_pack(sg, sg);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            float lo, hi;
            f2_unpack(p[j], lo, hi);
            const uint64_t o = f2_pack(__shfl_xor_sync(0xffffffffu, lo, x), __shfl_xor_sync(0xffffffffu, hi, x));
            p[j] = f2_fma(sg2, p[j], o);          // lower lane own + partner, upper partner - own
        }
    }
#pragma unroll
    for (int h = 4; h <= 16; h <<= 1)             // strides 32, 64, 128
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if ((j & h) == 0) {
                const uint64_t a = p[j], b = p[j + h];
                p[j] = f2_add(a, b);
                p[j + h] = f2_sub(a, b);
            }
}

// p *= the block's channel scales (shared memory, 256 floats)
__device__ __forceinline__ void scale_rows8(uint64_t (&p)[32], const float *sw, int q)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 v = *reinterpret_cast<const float4 *>(sw + 8 * (q + 4 * j) + 4 * i);
            p[4 * j + 2 * i] = f2_mul(p[4 * j + 2 * i], f2_pack(v.x, v.y));
            p[4 * j + 2 * i + 1] = f2_mul(p[4 * j + 2 * i + 1], f2_pack(v.z, v.w));
        }
}

// the codes of the lane's values: RN(p inv) + 1.5 2^23 rounds to the integer, whose low byte
// is then the value's low byte (finite rows; |RN(p inv)| < 128).  The product is the scalar
// instruction: a packed product and sum in a row come out fused, rounded once instead of
// twice, which moves the values that RN puts on a tie.
__device__ __forceinline__ void store_codes(const uint64_t (&p)[32], float inv, int pieces, int8_t *dst)
{
    const uint64_t magic = f2_pack(12582912.0f, 12582912.0f);
    auto scaled = [&](uint64_t v, uint32_t &a, uint32_t &b) {
        float x, y;
        f2_unpack(v, x, y);
        f2_unpack(f2_add(f2_pack(__fmul_rn(x, inv), __fmul_rn(y, inv)), magic), x, y);
        a = __float_as_uint(x);
        b = __float_as_uint(y);
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t a, b, c, d;
            scaled(p[4 * j + 2 * i], a, b);
            scaled(p[4 * j + 2 * i + 1], c, d);
            w[i] = __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
        }
        if (j < pieces)
            *reinterpret_cast<uint2 *>(dst + 32 * j) = make_uint2(w[0], w[1]);
    }
}

// what the first block does for the whole call: the status word
__device__ __forceinline__ void begin_call(const I8QuantArgs &a)
{
    bool bad = false;
    if (a.E > 0) {
        for (int i = threadIdx.x; i <= a.E; i += blockDim.x) {
            const int32_t o = a.offsets[i];
            bad |= o < 0 || o > a.M || (i > 0 && o < a.offsets[i - 1]);
        }
        bad = __syncthreads_or(bad);
    }
    if (threadIdx.x == 0) {
        if (a.finite_check) {                     // (the word was cleared before the launch)
            if (bad)
                atomicOr(a.status, kStatusIndex);
        } else {
            *a.status = bad ? kStatusIndex : 0u;
        }
    }
}

// GROUPED: called with E > 0 only.  Dense calls have a kernel of their own (4480 x 16384 backward
// 78 us against 85); tests of a.E that are always true stay in the grouped one, since without them
// the compiler keeps fewer of the forward's values in registers (115 us a call against 108, 8192
// rows of 64 experts, 2816 x 2048).
template <bool BWD, bool TURNS, bool GROUPED>
__global__ void __launch_bounds__(32 * kQWarps, 2) i8_quant_kernel(const I8QuantArgs a, int cluster)
{
    extern __shared__ __align__(16) uint8_t q_smem[];
    __shared__ QShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int rank = cluster > 1 ? (int)cluster_ctarank() : 0;
    const int unit = (int)blockIdx.x / cluster, units = (int)gridDim.x / cluster;
    const int nb = (int)((a.K + kHad - 1) / kHad);
    const int lanes_of_k = cluster * warps;       // blocks a cluster holds at once
    const int block0 = rank * warps + warp;       // this warp's (first) block
    // the warp's factor and channel scales
    uint8_t *my_factor = q_smem + warp * kQFactorBytes;
    float *my_scale = reinterpret_cast<float *>(q_smem + warps * kQFactorBytes) + warp * kHad;
    const bool with_low = a.low != nullptr;
    const uint32_t max_bar = smem_u32(sh.max_bar), low_bar = smem_u32(sh.low_bar);
    if (cluster > 1 && tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(max_bar + 8 * i, 1);
            mbar_init(low_bar + 8 * i, 1);
        }
        sh.abort_flag = 0u;
        fence_mbar_init();
    }
    const uint32_t factor_at = factor_lane(smem_u32(my_factor), lane);

    if ((!GROUPED || a.E == 0) && with_low && block0 < nb && (int)blockIdx.x < cluster * 2) {
        // the factor on its way into L2 (a prefetch: whoever still writes it is not overtaken)
        const uint8_t *src = reinterpret_cast<const uint8_t *>(a.factor + (int64_t)block0 * kHad * kI8Rank);
        const int64_t bytes = (a.K - (int64_t)block0 * kHad) * kI8Rank * 2;
        for (int c = 128 * lane; c < kQFactorBytes && c < bytes; c += 128 * 32)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(src + c));
    }
    if (cluster > 1) {
        __syncwarp();
        cluster_meet();                               // every CTA has started and set up its barriers
    }
    grid_dep_wait();                                  // x, and the workspace of the call before
    grid_dep_launch();                                // the product may fetch its first weights
    I8Plan plan;
    plan.start = sh.start;
    plan.prefix = sh.prefix;
    plan.E = a.E;
    plan.wts = 1;
    plan.tok_tile = kQRows;
    if (GROUPED && a.E > 0)
        plan.build(a.offsets, a.M, tid, blockDim.x);
    const int tiles = GROUPED && a.E > 0 ? plan.tiles() : (int)((a.M + kQRows - 1) / kQRows);
    auto tile_at = [&](int i, int &e) {
        if (GROUPED && a.E > 0)
            return plan.find(i, e);
        const int64_t row0 = (int64_t)i * kQRows, left = a.M - row0;
        return I8Tile{0, (int)row0, left < kQRows ? (int)left : kQRows, 0};
    };

    // columns of block b: 256, 128 (the last one, backward), or 0 behind the row's end
    auto columns = [&](int b) {
        const int64_t left = a.K - (int64_t)b * kHad;
        return left <= 0 ? 0 : left < kHad ? (int)left : kHad;
    };
    // factor and scales of block b of expert e on their way into shared memory, 0 behind the end
    auto fetch = [&](int e, int b) {
        const int cols = columns(b);
        if (with_low) {
            const uint8_t *src =
                reinterpret_cast<const uint8_t *>(a.factor + ((int64_t)e * a.K + (int64_t)b * kHad) * kI8Rank);
#pragma unroll 4
            for (uint32_t c = lane; c < kQFactorBytes / 16; c += 32)
                cp_async16(smem_u32(my_factor) + 16 * factor_chunk(c), (int)c < 2 * cols ? src + 16 * c : (const void *)a.factor,
                           (int)c < 2 * cols);
        }
        if (BWD) {
            const float *src = a.col_scale + (int64_t)e * a.K + (int64_t)b * kHad;
            for (int c = lane; c < kHad / 4; c += 32)
                cp_async16(smem_u32(my_scale) + 16 * c, 4 * c < cols ? src + 4 * c : a.col_scale, 4 * c < cols);
        }
    };
    auto fetched = [&]() {
        cp_async_wait_all();
        __syncwarp();
    };
    // this lane's first piece of its row in block b, and how many it has
    auto pieces_of = [&](const I8Tile &t, int b) { return g < t.rows ? columns(b) / 32 : 0; };
    auto row_of = [&](const I8Tile &t, int b) {
        return a.x + (int64_t)(t.row0 + g) * a.K + (int64_t)b * kHad + 8 * q;
    };
    auto spread = [&](const uint4(&w)[8], uint64_t(&p)[32]) {
        if (BWD) {
            widen(w, p);
            scale_rows8(p, my_scale, q);
        } else {
            fwht_rows8(w, p, lane);
        }
    };

    // dense: the clusters side by side (what they read at a time lies close together; in shares of
    // neighbouring groups 4480 x 6144 takes 47 us instead of 38); grouped: neighbouring groups,
    // mostly of one expert, whose factor then stays in shared memory
    const int first = GROUPED && a.E > 0 ? (int)((int64_t)tiles * unit / units) : unit;
    const int end = GROUPED && a.E > 0 ? (int)((int64_t)tiles * (unit + 1) / units) : tiles;
    const int step = GROUPED && a.E > 0 ? 1 : units;
    int e = 0;                                        // expert walked to
    uint4 w[8];
    I8Tile t = {0, 0, 0, 0};
    if (first < end) {
        t = tile_at(first, e);
        if (!TURNS) {
            load_block<BWD>(row_of(t, block0), pieces_of(t, block0), w);
            fetch(t.e, block0);
        }
    }
    if (blockIdx.x == 0)                              // while the first loads are on their way
        begin_call(a);
    // rows of no expert: 0
    if (GROUPED && a.y_zero && a.E > 0) {
        const int64_t head = plan.start[0], tail = a.M - plan.start[a.E], n16 = a.y_row_bytes / 16;
        for (int64_t i = blockIdx.x; i < head + tail; i += gridDim.x) {
            const int64_t m = i < head ? i : plan.start[a.E] + (i - head);
            uint4 *row = reinterpret_cast<uint4 *>(a.y_zero + m * a.y_row_bytes);
            for (int64_t c = tid; c < n16; c += blockDim.x)
                if (SQ_DCHECK(m < a.M, a.status))
                    row[c] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    int round = 0;
    for (int tile = first; tile < end; tile += step, ++round) {
        const int parity = round & 1;
        const bool live = g < t.rows;
        float low[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        float amax = 0.0f;
        uint64_t p[32];
        I8Tile next = t;
        if (TURNS) {
            for (int b = block0; b < nb; b += lanes_of_k) {
                fetch(t.e, b);
                load_block<BWD>(row_of(t, b), pieces_of(t, b), w);
                fetched();
                if (with_low)
                    low_block(w, factor_at, low);
                spread(w, p);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float x0, x1;
                    f2_unpack(p[j], x0, x1);
                    amax = absmax3(amax, x0, x1);
                }
                __syncwarp();                         // the next block's factor takes this one's place
            }
        } else {
            fetched();
            if (with_low && block0 < nb)
                low_block(w, factor_at, low);
            spread(w, p);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                float x0, x1;
                f2_unpack(p[j], x0, x1);
                amax = absmax3(amax, x0, x1);
            }
            if (tile + step < end) {                  // the next group's values, while this one is finished
                next = tile_at(tile + step, e);
                load_block<BWD>(row_of(next, block0), pieces_of(next, block0), w);
                if (next.e != t.e) {
                    __syncwarp();
                    fetch(next.e, block0);
                }
            }
        }
        // the row's maximum: 4 lanes, the CTA's warps, the cluster's CTAs (max of bit patterns:
        // not below zero, NaN above infinity above all others); the low-rank sums in the same order
        // of warps and CTAs.  What the CTAs exchange is counted on barriers: a buffer is written
        // again two groups later, by a CTA that has this one's values of the group between, sent
        // after this one had read the buffer.
        const uint32_t bar_phase = (uint32_t)(round >> 1) & 1u;
        uint32_t m = __float_as_uint(amax);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (q == 0)
            sh.warp_max[parity][warp][g] = m;
        if (with_low) {                               // low[0..3]: ranks g, g + 8; rows 2 q, 2 q + 1
            float *wl = sh.warp_low[parity][warp];
            wl[(2 * q) * kI8Rank + g] = low[0];
            wl[(2 * q + 1) * kI8Rank + g] = low[1];
            wl[(2 * q) * kI8Rank + g + 8] = low[2];
            wl[(2 * q + 1) * kI8Rank + g + 8] = low[3];
        }
        if (cluster > 1 && tid == 0) {
            mbar_arrive_expect_tx(max_bar + 8 * parity, cluster * kQRows * 4);
            if (rank == 0 && with_low)
                mbar_arrive_expect_tx(low_bar + 8 * parity, (cluster - 1) * kI8Rank * kQRows * 4);
        }
        __syncthreads();
        uint32_t top = 0;
        if (cluster > 1) {
            for (int i = tid; i < kQRows * cluster; i += blockDim.x) {
                const int row = i % kQRows, to = i / kQRows;
                uint32_t v = 0;
                for (int k = 0; k < warps; ++k)
                    v = max(v, sh.warp_max[parity][k][row]);
                st_async(mapa_shared(smem_u32(&sh.max[parity][rank][row]), to), v,
                         mapa_shared(max_bar + 8 * parity, to));
            }
        }
        auto low_sum = [&](int i) {                   // of the CTA's warps
            float v = sh.warp_low[parity][0][i];
            for (int k = 1; k < warps; ++k)
                v = __fadd_rn(v, sh.warp_low[parity][k][i]);
            return v;
        };
        if (with_low && rank > 0)
            for (int i = tid; i < kI8Rank * kQRows; i += blockDim.x)
                st_async(mapa_shared(smem_u32(&sh.low[parity][rank][i]), 0), __float_as_uint(low_sum(i)),
                         mapa_shared(low_bar + 8 * parity, 0));
        if (cluster > 1) {
            (void)mbar_wait(max_bar + 8 * parity, bar_phase, &sh.abort_flag, a.status);
            for (int r = 0; r < cluster; ++r)
                top = max(top, sh.max[parity][r][g]);
        } else {
            for (int k = 0; k < warps; ++k)
                top = max(top, sh.warp_max[parity][k][g]);
        }
        if (!BWD && top < kInfBits)                   // the transform's 1/16 (exact where the scale is not 0)
            top = __float_as_uint(__fmul_rn(__uint_as_float(top), 0.0625f));
        float s, inv;
        row_scale(top, s, inv);
        if (!BWD)
            inv *= 0.0625f;                           // exact: 1 / s is above 2^-122
        if (rank == 0 && tid < 32 && q == 0 && live && SQ_DCHECK(t.row0 + g < a.M, a.status)) {
            a.scales[t.row0 + g] = s;
            if (a.finite_check && top >= kInfBits)
                atomicOr(a.status, kStatusNonfinite);
        }
        if (TURNS) {
            for (int b = block0; b < nb; b += lanes_of_k) {
                if (BWD)
                    fetch(t.e, b);
                load_block<BWD>(row_of(t, b), pieces_of(t, b), w);
                fetched();
                spread(w, p);
                if (live && SQ_DCHECK(t.row0 + g < a.M, a.status))
                    store_codes(p, inv, pieces_of(t, b),
                                a.codes + (int64_t)(t.row0 + g) * a.K + (int64_t)b * kHad + 8 * q);
                __syncwarp();
            }
        } else if (live && SQ_DCHECK(t.row0 + g < a.M, a.status)) {
            store_codes(p, inv, pieces_of(t, block0), a.codes + (int64_t)(t.row0 + g) * a.K + (int64_t)block0 * kHad + 8 * q);
        }
        if (with_low && rank == 0)                    // the low-rank input, once the codes are out
            for (int i = tid; i < kI8Rank * kQRows; i += blockDim.x) {
                float v = low_sum(i);
                if (cluster > 1) {
                    (void)mbar_wait(low_bar + 8 * parity, bar_phase, &sh.abort_flag, a.status);
                    for (int r = 1; r < cluster; ++r)
                        v = __fadd_rn(v, sh.low[parity][r][i]);
                }
                const int row = i / kI8Rank, k = i % kI8Rank;
                if (row < t.rows && SQ_DCHECK(t.row0 + row < a.M, a.status))
                    a.low[(int64_t)(t.row0 + row) * kI8Rank + k] = v;
            }
        t = TURNS && tile + step < end ? tile_at(tile + step, e) : next;
    }
    if (cluster > 1) {
        __syncwarp();
        cluster_meet();                               // nobody leaves while another CTA may still write to it
    }
}

template <bool BWD, bool TURNS, bool GROUPED>
static cudaError_t launch_quant_v(const I8QuantArgs &a, int cluster, int warps, int sms, cudaStream_t s)
{
    constexpr int kMaxDev = 64;
    static unsigned long long attr_ctx[kMaxDev];
    static unsigned long long room_ctx[kMaxDev][kQMaxCluster][kQWarps];
    static int room[kMaxDev][kQMaxCluster][kQWarps];
    constexpr int kMaxSmem = kQWarps * (kQFactorBytes + kHad * 4);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev)
        return cudaErrorInvalidDevice;
    const unsigned long long ctx = current_context_id();
    if (ctx == 0 || attr_ctx[dev] != ctx) {
        cudaError_t e = cudaFuncSetAttribute(i8_quant_kernel<BWD, TURNS, GROUPED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kMaxSmem);
        if (e != cudaSuccess)
            return e;
        attr_ctx[dev] = ctx;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = warps * (kQFactorBytes + (BWD ? kHad * 4 : 0));
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    // dependent launch of small grids: the CTAs are there when the kernel in front (the product of
    // the call before, perhaps) ends, which saves 2 us a call.  A grid that fills the device would
    // be placed piece by piece as that kernel's CTAs end, clusters no longer all fit, and some wait
    // for a second turn (4480x16384x6144, call after call: 427 instead of 408 us).
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    // persistent: as many clusters as are resident at once (clusters left over for a second
    // wave would double the time), but never more than row groups
    if (ctx == 0 || room_ctx[dev][cluster - 1][warps - 1] != ctx) {
        cfg.gridDim = dim3((unsigned)(2 * sms / cluster * cluster));
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, i8_quant_kernel<BWD, TURNS, GROUPED>, &cfg);
        (void)cudaGetLastError();
        room[dev][cluster - 1][warps - 1] = e == cudaSuccess && n > 0 ? n : 1;
        room_ctx[dev][cluster - 1][warps - 1] = ctx;
    }
    const int64_t groups = (a.M + kQRows - 1) / kQRows + a.E;
    const int64_t fit = room[dev][cluster - 1][warps - 1];
    cfg.gridDim = dim3((unsigned)((groups < fit ? groups : fit) * cluster));
    cfg.attrs = at;
    cfg.numAttrs = (int64_t)cfg.gridDim.x <= sms ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, i8_quant_kernel<BWD, TURNS, GROUPED>, a, cluster);
}

cudaError_t launch_i8_quant(const I8QuantArgs &a, bool bwd, int sms, cudaStream_t s)
{
    const int nb = (int)(a.K + kHad - 1) / kHad;
    int cluster = (nb + kQWarps - 1) / kQWarps;
    cluster = cluster < kQMaxCluster ? cluster : kQMaxCluster;
    // few row groups: more CTAs of fewer warps, while each still has an SM of its own
    const int64_t groups = (a.M + kQRows - 1) / kQRows + a.E;
    while (cluster < kQMaxCluster && cluster < nb && groups * (cluster + 1) <= sms)
        ++cluster;
    int warps = (nb + cluster - 1) / cluster;
    const bool turns = warps > kQWarps;
    warps = turns ? kQWarps : warps;
    if (a.E > 0) {
        if (bwd)
            return turns ? launch_quant_v<true, true, true>(a, cluster, warps, sms, s)
                         : launch_quant_v<true, false, true>(a, cluster, warps, sms, s);
        return launch_quant_v<false, false, true>(a, cluster, warps, sms, s);
    }
    if (bwd)
        return turns ? launch_quant_v<true, true, false>(a, cluster, warps, sms, s)
                     : launch_quant_v<true, false, false>(a, cluster, warps, sms, s);
    return launch_quant_v<false, false, false>(a, cluster, warps, sms, s);
}

}  // namespace sq
