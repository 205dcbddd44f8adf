// sq_w8a8_quant.cu -- the 8-bit operands of the integer products (sq_w8a8.cu):
// one int8 code per value and one fp32 scale per row, plus the row's low-rank
// input.
//
//   forward   r = H256 x            low = x lora_down   [M, 16]
//   backward  r = RN(dy s_w)        low = dy lora_up    [M, 16]
//   s = RN(max|r| / 127),  code = clamp(rint(RN(r RN(1 / s))), -127, 127)
//
// A scale below 2^-120 is stored as 0 with zero codes (1 / s would leave fp32's
// range); a row with a NaN or an infinity in r gets the scale NaN, so its
// outputs are NaN.  Each product is rounded once, in the order written, so the
// codes are the same bits whatever kernel forms them.  With experts (E > 0) the
// row's expert, found from the offsets, picks the lora and scale arrays.
#include <cuda.h>

#include "sq_device.cuh"
#include "sq_kernels.h"
#include "sq_ptx.cuh"

namespace sq {

constexpr int kLow = 16;                          // rank of the int8 layer's low-rank branch
constexpr uint32_t kInfBits = 0x7F800000u;

// expert of row m: the e with offsets[e] <= m < offsets[e + 1], -1 if there is none.  Every
// lane of the warp takes part; valid offsets do not decrease, and with others the answer is
// still in range.  E == 0: one layer, expert 0 for every row.
__device__ __forceinline__ int expert_of(const int32_t *__restrict__ offsets, int E, int64_t m, int lane)
{
    if (E == 0)
        return 0;
    int below = 0;
    for (int i = 0; i <= E; i += 32)
        below += __popc(__ballot_sync(0xffffffffu, i + lane <= E && (int64_t)__ldg(offsets + i + lane) <= m));
    return below == 0 || below == E + 1 ? -1 : below - 1;
}

// scale and reciprocal of a row from the largest |r| (bit pattern, NaN and infinity on top)
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

__device__ __forceinline__ uint32_t code8(float r, float inv)
{
    // (a NaN r comes with inv = 0: fminf and fmaxf drop the NaN, the code is some number)
    return (uint32_t)__float2int_rn(fminf(fmaxf(__fmul_rn(r, inv), -127.0f), 127.0f)) & 0xFFu;
}

__device__ __forceinline__ uint32_t abs_bits(float v)
{
    return __float_as_uint(v) & 0x7FFFFFFFu;
}

// sums a[0..15] over the 32 lanes; lane l returns the total of a[l / 2]
__device__ __forceinline__ float reduce16(float (&a)[16], int lane)
{
#pragma unroll
    for (int h = 8; h >= 1; h >>= 1) {            // lanes with bit 2h keep the upper half
        const bool up = lane & (2 * h);
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float mine = up ? a[i + h] : a[i];
            const float other = __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + h], 2 * h);
            a[i] = __fadd_rn(mine, other);
        }
    }
    return __fadd_rn(a[0], __shfl_xor_sync(0xffffffffu, a[0], 1));
}

// a[j] += x * (16 bf16 of one row of a low-rank factor)
__device__ __forceinline__ void low_fma(float x, const uint16_t *__restrict__ row, float (&a)[16])
{
    const uint4 p = __ldg(reinterpret_cast<const uint4 *>(row)), q = __ldg(reinterpret_cast<const uint4 *>(row) + 1);
    const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        a[2 * j] = __fmaf_rn(x, __uint_as_float(w[j] << 16), a[2 * j]);
        a[2 * j + 1] = __fmaf_rn(x, __uint_as_float(w[j] & 0xFFFF0000u), a[2 * j + 1]);
    }
}

// what the first block does for the whole call: the status word and the product's counters
__device__ __forceinline__ void begin_call(const I8QuantArgs &a)
{
    for (int i = threadIdx.x; i < a.n_counters; i += blockDim.x)
        a.counters[i] = 0u;
    bool bad = false;
    for (int i = threadIdx.x; i <= a.E && a.E > 0; i += blockDim.x) {
        const int32_t o = a.offsets[i];
        bad |= o < 0 || o > a.M || (i > 0 && o < a.offsets[i - 1]);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        if (a.finite_check) {                     // (the word was cleared before the launch)
            if (bad)
                atomicOr(a.status, kStatusIndex);
        } else {
            *a.status = bad ? kStatusIndex : 0u;
        }
    }
}

// rows of y that belong to no expert become 0
__device__ __forceinline__ void zero_row(const I8QuantArgs &a, int64_t m)
{
    if (!a.y_zero)
        return;
    uint4 *row = reinterpret_cast<uint4 *>(a.y_zero + m * a.y_row_bytes);
    for (int64_t i = threadIdx.x; i < a.y_row_bytes / 16; i += blockDim.x)
        row[i] = make_uint4(0u, 0u, 0u, 0u);
}

// the row's partial maxima and low-rank sums of the CTA's warps, combined in order
struct RowShared {
    uint32_t amax[32];
    float low[32][kLow];
};

__device__ __forceinline__ uint32_t combine_row(const I8QuantArgs &a, RowShared &sh, int64_t m, uint32_t amax,
                                                float (&low)[16], int warps)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    amax = __reduce_max_sync(0xffffffffu, amax);
    if (lane == 0)
        sh.amax[warp] = amax;
    if (a.low) {
        const float v = reduce16(low, lane);
        if ((lane & 1) == 0)
            sh.low[warp][lane >> 1] = v;
    }
    __syncthreads();
    amax = 0;
    for (int w = 0; w < warps; ++w)
        amax = max(amax, sh.amax[w]);
    if (a.low && threadIdx.x < kLow) {
        float v = sh.low[0][threadIdx.x];
        for (int w = 1; w < warps; ++w)
            v = __fadd_rn(v, sh.low[w][threadIdx.x]);
        if (SQ_DCHECK(m < a.M, a.status))
            a.low[m * kLow + threadIdx.x] = v;
    }
    if (threadIdx.x == 0 && a.finite_check && amax >= kInfBits)
        atomicOr(a.status, kStatusNonfinite);
    return amax;
}

// ---------------------------------------------------------------------------
// Forward, one row per CTA, UNITS 256-blocks per warp held in registers: x is
// read once.
// ---------------------------------------------------------------------------
template <int UNITS>
__global__ void __launch_bounds__(1024) i8_quant_row_kernel(const I8QuantArgs a)
{
    __shared__ RowShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t m = blockIdx.x;
    const int nb = (int)(a.K / kHad);
    grid_dep_launch();
    if (blockIdx.x == 0)
        begin_call(a);
    const int e = expert_of(a.offsets, a.E, m, lane);
    if (e < 0) {
        zero_row(a, m);
        return;
    }
    const uint16_t *factor = a.factor + (int64_t)e * a.K * kLow;
    float v[UNITS][8];
    float low[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        low[i] = 0.0f;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        const int b = warp + u * warps;
        uint2 p = make_uint2(0u, 0u), q = p;
        if (b < nb) {
            const uint2 *src = reinterpret_cast<const uint2 *>(a.x + m * a.K + (int64_t)b * kHad);
            p = __ldg(src + lane);
            q = __ldg(src + 32 + lane);
        }
        const uint32_t w[4] = {p.x, p.y, q.x, q.y};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[u][2 * j] = __uint_as_float(w[j] << 16);
            v[u][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
    uint32_t amax = 0;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        const int b = warp + u * warps;
        if (b >= nb)
            continue;
        if (a.low) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = b * kHad + 4 * lane + (j & 3) + 128 * (j >> 2);
                low_fma(v[u][j], factor + (int64_t)k * kLow, low);
            }
        }
        fwht256_warp(v[u], lane);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            amax = max(amax, abs_bits(v[u][j]));
    }
    amax = combine_row(a, sh, m, amax, low, warps);
    float s, inv;
    row_scale(amax, s, inv);
    if (threadIdx.x == 0 && SQ_DCHECK(m < a.M, a.status))
        a.scales[m] = s;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        const int b = warp + u * warps;
        if (b >= nb || !SQ_DCHECK(m < a.M, a.status))
            continue;
        uint32_t *dst = reinterpret_cast<uint32_t *>(a.codes + m * a.K + (int64_t)b * kHad);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            dst[lane + 32 * h] = code8(v[u][4 * h], inv) | code8(v[u][4 * h + 1], inv) << 8 |
                                 code8(v[u][4 * h + 2], inv) << 16 | code8(v[u][4 * h + 3], inv) << 24;
    }
}

// ---------------------------------------------------------------------------
// Backward, one row per CTA: a pass for the maximum and the low-rank input, a
// pass for the codes (the row comes from L1 or L2 the second time).
// ---------------------------------------------------------------------------
constexpr int kBwdThreads = 256;

__device__ __forceinline__ void scaled8(const uint16_t *__restrict__ x, const float *__restrict__ s, float (&raw)[8],
                                        float (&r)[8])
{
    const uint4 p = __ldg(reinterpret_cast<const uint4 *>(x));
    const float4 s0 = __ldg(reinterpret_cast<const float4 *>(s)), s1 = __ldg(reinterpret_cast<const float4 *>(s) + 1);
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
    const float sc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        raw[2 * j] = __uint_as_float(w[j] << 16);
        raw[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        r[j] = __fmul_rn(raw[j], sc[j]);
}

__global__ void __launch_bounds__(kBwdThreads) i8_quant_row_bwd_kernel(const I8QuantArgs a)
{
    __shared__ RowShared sh;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int64_t m = blockIdx.x;
    grid_dep_launch();
    if (blockIdx.x == 0)
        begin_call(a);
    const int e = expert_of(a.offsets, a.E, m, lane);
    if (e < 0) {
        zero_row(a, m);
        return;
    }
    const uint16_t *x = a.x + m * a.K;
    const float *sw = a.col_scale + (int64_t)e * a.K;
    const uint16_t *factor = a.factor + (int64_t)e * a.K * kLow;
    float low[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        low[i] = 0.0f;
    uint32_t amax = 0;
    for (int64_t k = 8 * threadIdx.x; k < a.K; k += 8 * kBwdThreads) {
        float raw[8], r[8];
        scaled8(x + k, sw + k, raw, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            amax = max(amax, abs_bits(r[j]));
            if (a.low)
                low_fma(raw[j], factor + (k + j) * kLow, low);
        }
    }
    amax = combine_row(a, sh, m, amax, low, warps);
    float s, inv;
    row_scale(amax, s, inv);
    if (threadIdx.x == 0 && SQ_DCHECK(m < a.M, a.status))
        a.scales[m] = s;
    for (int64_t k = 8 * threadIdx.x; k < a.K; k += 8 * kBwdThreads) {
        float raw[8], r[8];
        scaled8(x + k, sw + k, raw, r);
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j >> 2] |= code8(r[j], inv) << (8 * (j & 3));
        if (SQ_DCHECK(m < a.M, a.status))
            *reinterpret_cast<uint2 *>(a.codes + m * a.K + k) = make_uint2(w[0], w[1]);
    }
}

cudaError_t launch_i8_quant(const I8QuantArgs &a, bool bwd, int sms, cudaStream_t s)
{
    (void)sms;
    if (bwd) {
        i8_quant_row_bwd_kernel<<<(unsigned)a.M, kBwdThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
    const int nb = (int)(a.K / kHad);             // <= 64
    if (nb <= 32)
        i8_quant_row_kernel<1><<<(unsigned)a.M, 32 * nb, 0, s>>>(a);
    else
        i8_quant_row_kernel<2><<<(unsigned)a.M, 32 * ((nb + 1) / 2), 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace sq
