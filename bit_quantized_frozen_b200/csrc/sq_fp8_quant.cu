// sq_fp8_quant.cu -- e4m3 codes with one power-of-two scale for each block of 128: of the rows
// that the block-scaled product (sq_fp8.cu) multiplies, and of a weight (128 x 128 blocks).
//
//   s = the least power of two >= 2^-127 with max|r| <= 448 s,   code = e4m3(r / s)
//
// max|r| = 2^E (1.m): s = 2^(E - 8), or the next one where 1.m > 1.75 (448 = 1.75 * 2^8), straight
// from the maximum's bits; r / s = r 2^-e is exact in fp32, so the code is one rounding of r.
//
// Rows: r = x, or the two gradients of a gated pair, formed here from dh, g and u:
//   dg = (dh u) act'(g),  du = dh act(g)            (fp32)
//
// A block with a NaN or an infinity gets NaN codes, so that the whole row's sums are NaN.
//
// One read of the rows, one write of the codes: bound by DRAM, and where they are formed from a gated pair by
// instructions too (two powers, two quotients, some 30 others for two values: packed arithmetic took the 2049 x
// 8192 pair from 30.1 us to 26 with gelu).  Alone: 4480 x 6144 15 us (5.5 TB/s), 4480 x 16384 30 us (7.3 TB/s, the
// codes staying in L2), gated pair of 2049 x 8192 24 us with silu, 26 to 27 with gelu (5 TB/s).
#include <cuda.h>

#include "sq_fp8.cuh"
#include "sq_kernels.h"
#include "sq_ptx.cuh"

namespace sq {

constexpr int kQuantThreads = 128;
// CTAs of an SM.  The grid is no larger, since what waits for a second turn would make the last CTAs of the
// first wait too.  Fewer CTAs have more registers each (92 instead of 56 hold a gated pair's operands without
// spills) and end closer together: a call of 2049 rows, gated gradient, 8192 x 4096, takes 133.8, 132.5, 132.0,
// 130.4, 131.3 us with 9, 7, 6, 5, 4 of them; 777 x 4240 x 2832, forward, 22.4, 21.0, 21.1, 21.1 us with 8, 6,
// 5, 4; 4480 x 16384 x 6144 334, 334, 336, 337.  (The product's CTAs take 46 to 64 K of an SM's 64 K registers, one of
// these 10 to 12 K: a product's CTA starts where at most one of them is left, a gated forward's where none is.)
constexpr int quant_ctas(int gated)
{
    return gated ? 5 : 6;
}

// GATED 0: rows of x; 1, 2: the gradients of a gated pair with silu, gelu.  A warp takes ROWS rows x
// 512 columns at a time, a lane 16 neighbouring values of each row.
template <int GATED, int ROWS>
__global__ void __launch_bounds__(kQuantThreads, quant_ctas(GATED)) fp8_quant_kernel(const Fp8QuantArgs a)
{
    const int lane = threadIdx.x & 31;
    grid_dep_wait();                              // x, and the workspace of the call before
    grid_dep_launch();                            // the product may fetch its first weights
    if (blockIdx.x == 0 && threadIdx.x < 32)
        fp8_begin_call(a.offsets, a.E, a.M, a.keep_status, a.status, lane);
    // rows of no expert are not looked at
    int64_t lo = 0, hi = a.M;
    if (a.E > 0) {
        const int64_t first = __ldg(a.offsets), last = __ldg(a.offsets + a.E);
        lo = first < 0 ? 0 : first > a.M ? a.M : first;
        hi = last < lo ? lo : last > a.M ? a.M : last;
    }
    // the warps take (rows, group) pairs in turn, the group changing fastest; the next pair is found without
    // a division (two of 64 bits cost more than a pair's values)
    const int groups = (int)fp8_groups(a.L);
    const unsigned warps = gridDim.x * (kQuantThreads / 32), me = blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5);
    const int step_grp = (int)(warps % (unsigned)groups);
    const int64_t step_row = (int64_t)(warps / (unsigned)groups) * ROWS;
    int grp = (int)(me % (unsigned)groups);
    int64_t row0 = lo + (int64_t)(me / (unsigned)groups) * ROWS;
    auto settle = [&]() {                         // past the last group: the next rows
        if (grp >= groups) {
            grp -= groups;
            row0 += ROWS;
        }
    };
    bool bad = false;
    while (row0 < hi) {
        const int64_t row = row0, col = (int64_t)grp * (kFp8Block * kFp8Group) + 16 * lane;
        const int g512 = grp;
        constexpr int OPS = GATED ? 3 : 1;
        uint4 w[OPS][ROWS][2];
#pragma unroll
        for (int o = 0; o < OPS; ++o) {
            const uint16_t *src = o == 0 ? a.x : o == 1 ? a.g : a.u;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const bool live = row + r < hi && col < a.L;
                const uint4 *p = reinterpret_cast<const uint4 *>(src + (row + r) * a.L + col);
                w[o][r][0] = live ? __ldg(p) : make_uint4(0u, 0u, 0u, 0u);
                w[o][r][1] = live ? __ldg(p + 1) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        row0 += step_row;
        grp += step_grp;
        settle();
        uint32_t words[GATED ? 2 : 1] = {};
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const bool live = row + r < hi && col < a.L;
            uint32_t byte;
            uint4 c;
            if constexpr (GATED == 0) {
                c = quantise16(w[0][r], byte, bad);
            } else {
                uint64_t v[8], second[8];
                pair_gradients<GATED - 1>(w[0][r], w[1][r], w[2][r], v, second);
                c = quantise16(second, byte, bad);
                const uint32_t word = scale_word(byte, lane);
                if (lane == r)
                    words[1] = word;
                if (live && SQ_DCHECK(row + r < a.M, a.status))
                    *reinterpret_cast<uint4 *>(a.codes + (a.M + row + r) * a.L + col) = c;
                c = quantise16(v, byte, bad);
            }
            const uint32_t word = scale_word(byte, lane);
            if (lane == r)
                words[0] = word;
            if (live && SQ_DCHECK(row + r < a.M, a.status))
                *reinterpret_cast<uint4 *>(a.codes + (row + r) * a.L + col) = c;
        }
        if (lane < ROWS && row + lane < hi) {
            a.words[(int64_t)g512 * a.M + row + lane] = words[0];
            if constexpr (GATED != 0)
                a.words[(int64_t)(groups + g512) * a.M + row + lane] = words[1];
        }
    }
    if (a.finite_check && bad)
        atomicOr(a.status, kStatusNonfinite);
    // rows of no expert: 0
    if (a.E > 0) {
        for (int k = 0; k < 3; ++k) {
            if (!a.zero[k])
                continue;
            const int64_t n16 = a.zero_row_bytes[k] / 16, rows = lo + a.M - hi;
            for (int64_t i = blockIdx.x; i < rows; i += gridDim.x) {
                const int64_t m = i < lo ? i : hi + (i - lo);
                uint4 *row = reinterpret_cast<uint4 *>(a.zero[k] + m * a.zero_row_bytes[k]);
                for (int64_t c = threadIdx.x; c < n16; c += kQuantThreads)
                    if (SQ_DCHECK(m < a.M, a.status))
                        row[c] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }
}

template <int GATED, int ROWS>
static cudaError_t launch_quant(const Fp8QuantArgs &a, int sms, cudaStream_t s)
{
    const int64_t units = (a.M + ROWS - 1) / ROWS * fp8_groups(a.L);
    const int64_t blocks = (units + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
    const int64_t most = (int64_t)sms * quant_ctas(GATED);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
    cfg.blockDim = dim3(kQuantThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp8_quant_kernel<GATED, ROWS>, a);
}

cudaError_t launch_fp8_quant(const Fp8QuantArgs &a, int sms, cudaStream_t s)
{
    if (!a.g)
        return launch_quant<0, 4>(a, sms, s);
    return a.act == 0 ? launch_quant<1, 1>(a, sms, s) : launch_quant<2, 1>(a, sms, s);
}

// ---------------------------------------------------------------------------
// the weight: a CTA a block of 128 x 128, 8 lanes a row of 128.  One read, one write: 16384 x 6144 from fp32
// takes 0.10 ms (5.0 to 5.2 TB/s, bound by DRAM)
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ void __launch_bounds__(256) fp8_build_kernel(const void *__restrict__ W, int64_t N, int64_t K,
                                                        uint8_t *__restrict__ codes, uint8_t *__restrict__ scales)
{
    __shared__ uint32_t warp_top[8];
    const int64_t kbs = (K + kFp8Block - 1) / kFp8Block;
    const int64_t kb = (int64_t)blockIdx.x % kbs, nb = (int64_t)blockIdx.x / kbs;
    const int64_t col = kb * kFp8Block + 16 * (threadIdx.x & 7);
    const int64_t row = nb * kFp8Block + (threadIdx.x >> 3);          // and 32, 64, 96 further
    float v[4][16];
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t n = row + 32 * r;
        if (n < N && col < K) {
            if (BF16) {
                const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(W) + n * K + col);
                widen8(__ldg(p), v[r], 0);
                widen8(__ldg(p + 1), v[r], 8);
            } else {
                const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(W) + n * K + col);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 f = __ldg(p + i);
                    v[r][4 * i] = f.x;
                    v[r][4 * i + 1] = f.y;
                    v[r][4 * i + 2] = f.z;
                    v[r][4 * i + 3] = f.w;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[r][i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t b = __float_as_uint(v[r][i]) & 0x7FFFFFFFu;
            top = max(top, b < kFp8Inf ? b : 0u);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0)
        warp_top[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = max(top, warp_top[i]);
    const uint32_t byte = fp8_scale_byte(top);
    const float inv = fp8_inverse(byte);
    if (threadIdx.x == 0)
        scales[nb * kbs + kb] = (uint8_t)byte;
    auto code = [&](float f) {                    // (the conversion would clamp an infinity)
        return (__float_as_uint(f) & 0x7FFFFFFFu) >= kFp8Inf ? __uint_as_float(0x7FFFFFFFu) : f * inv;
    };
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t n = row + 32 * r;
        if (n < N && col < K) {
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c[i] = to_e4m3x4(code(v[r][4 * i]), code(v[r][4 * i + 1]), code(v[r][4 * i + 2]),
                                 code(v[r][4 * i + 3]));
            *reinterpret_cast<uint4 *>(codes + n * K + col) = make_uint4(c[0], c[1], c[2], c[3]);
        }
    }
}

cudaError_t launch_fp8_build(const void *W, int bf16, int64_t N, int64_t K, uint8_t *codes, uint8_t *scales,
                             cudaStream_t s)
{
    const int64_t blocks = (N + kFp8Block - 1) / kFp8Block * ((K + kFp8Block - 1) / kFp8Block);
    if (bf16)
        fp8_build_kernel<true><<<(unsigned)blocks, 256, 0, s>>>(W, N, K, codes, scales);
    else
        fp8_build_kernel<false><<<(unsigned)blocks, 256, 0, s>>>(W, N, K, codes, scales);
    return cudaGetLastError();
}

}  // namespace sq
