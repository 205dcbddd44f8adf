// sq_fp8.cuh -- what the row rounding (sq_fp8_quant.cu) and the block-scaled e4m3 product
// (sq_fp8.cu) share: the activations, the rounding to e4m3, and the tcgen05 and copy instructions of the
// product.
#pragma once

#include <cstdint>

#include "sq_device.cuh"
#include "sq_ptx.cuh"

namespace sq {

constexpr int kFp8Block = 128;                    // values of a scale
constexpr int kFp8Group = 4;                      // blocks whose scales share a 32-bit word

// 32-bit words of row scales along an axis of `len` values
__host__ __device__ __forceinline__ int64_t fp8_groups(int64_t len)
{
    return (len + kFp8Block * kFp8Group - 1) / (kFp8Block * kFp8Group);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu2C = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

__device__ __forceinline__ uint64_t f2_both(float v)
{
    return f2_pack(v, v);
}

// t = 2^x and 1 / (1 + t), two at a time (an infinite t gives 0)
__device__ __forceinline__ void power_and_share(uint64_t x, float (&t)[2], uint64_t &share)
{
    float v[2], d[2], s[2];
    f2_unpack(x, v[0], v[1]);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t[0]) : "f"(v[0]));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t[1]) : "f"(v[1]));
    f2_unpack(f2_add(f2_pack(t[0], t[1]), f2_both(1.0f)), d[0], d[1]);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s[0]) : "f"(d[0]));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s[1]) : "f"(d[1]));
    share = f2_pack(s[0], s[1]);
}

// g^2, kept finite, so that what it multiplies may be 0
__device__ __forceinline__ uint64_t finite_square(uint64_t g)
{
    float a, b;
    f2_unpack(f2_mul(g, g), a, b);
    return f2_pack(fminf(a, 1e30f), fminf(b, 1e30f));
}

// minus act's argument of the sigmoid, in units of ln 2; gelu: (1 + tanh z) / 2 = sigmoid(2 z)
template <int ACT>
__device__ __forceinline__ uint64_t act_arg(uint64_t g, uint64_t g2)
{
    return ACT == 0 ? f2_mul(g, f2_both(-kLog2e))
                    : f2_mul(g, f2_fma(g2, f2_both(-kLog2e * kGelu2C * kGeluCube), f2_both(-kLog2e * kGelu2C)));
}

// act(g) = g / (1 + 2^-x) of two: where the power leaves fp32's range, the quotient is 0
template <int ACT>
__device__ __forceinline__ uint64_t act_value(uint64_t g)
{
    float t[2];
    uint64_t s;
    power_and_share(act_arg<ACT>(g, ACT == 0 ? 0 : finite_square(g)), t, s);
    return f2_mul(g, s);
}

// act(g) and act'(g) of two.  1 - sigmoid = 2^-x sigmoid, without cancellation; a power out of range
// meets a sigmoid of 0, so that it may be cut to a finite one
template <int ACT>
__device__ __forceinline__ void act_grad(uint64_t g, uint64_t &a, uint64_t &slope)
{
    float t[2];
    uint64_t s;
    const uint64_t g2 = ACT == 0 ? 0 : finite_square(g);
    power_and_share(act_arg<ACT>(g, g2), t, s);
    const uint64_t o = f2_mul(f2_pack(fminf(t[0], 1e38f), fminf(t[1], 1e38f)), s);
    a = f2_mul(g, s);
    const uint64_t w = f2_mul(a, o);              // g sigmoid'
    slope = ACT == 0 ? f2_add(s, w)
                     : f2_fma(w, f2_fma(g2, f2_both(3.0f * kGelu2C * kGeluCube), f2_both(kGelu2C)), s);
}

// ---- rounding to e4m3 --------------------------------------------------------------
constexpr uint32_t kFp8Inf = 0x7F800000u;
constexpr uint32_t kFp8NanCodes = 0x7F7F7F7Fu;

// e8m0 byte of a block from the bits of its largest |r| (finite)
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t amax_bits)
{
    const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e < 0 ? 0u : (uint32_t)e;
}

// 2^-e as a float (the byte is at most 247)
__device__ __forceinline__ float fp8_inverse(uint32_t byte)
{
    return __uint_as_float((254u - byte) << 23);
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

__device__ __forceinline__ void widen8(const uint4 &w, float (&v)[16], int at)
{
    const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[at + 2 * i] = __uint_as_float(p[i] << 16);
        v[at + 2 * i + 1] = __uint_as_float(p[i] & 0xFFFF0000u);
    }
}

// max(a, |b|, |c|), NaN if any is
__device__ __forceinline__ float fp8_absmax3(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}

// the largest |r| of a block from its eight lanes' (bits: NaN above infinity above all others)
__device__ __forceinline__ uint32_t block_top(uint32_t top)
{
#pragma unroll
    for (int x = 1; x <= 4; x <<= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
    return top;
}

// the bf16 pair in a word as two fp32 values
__device__ __forceinline__ uint64_t widen2(uint32_t w)
{
    return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// A lane's 16 neighbouring values of a row (8 lanes a block), in pairs: their codes, and the block's byte.
__device__ __forceinline__ uint4 quantise16(const uint64_t (&v)[8], uint32_t &byte, bool &bad)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a, b;
        f2_unpack(v[i], a, b);
        m = fp8_absmax3(m, a, b);
    }
    const uint32_t top = block_top(__float_as_uint(m) & 0x7FFFFFFFu);
    if (top >= kFp8Inf) {
        bad = true;
        byte = 127u;
        return make_uint4(kFp8NanCodes, kFp8NanCodes, kFp8NanCodes, kFp8NanCodes);
    }
    byte = fp8_scale_byte(top);
    const uint64_t inv = f2_both(fp8_inverse(byte));
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float r[4];
        f2_unpack(f2_mul(v[2 * i], inv), r[0], r[1]);
        f2_unpack(f2_mul(v[2 * i + 1], inv), r[2], r[3]);
        c[i] = to_e4m3x4(r[0], r[1], r[2], r[3]);
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// Eight bf16 pairs of dh, g and u: the gradients dg = (dh u) act'(g) and du = dh act(g).
template <int ACT>
__device__ __forceinline__ void pair_gradients(const uint4 (&dh)[2], const uint4 (&g)[2], const uint4 (&u)[2],
                                               uint64_t (&dg)[8], uint64_t (&du)[8])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t d[4] = {dh[h].x, dh[h].y, dh[h].z, dh[h].w}, a[4] = {g[h].x, g[h].y, g[h].z, g[h].w},
                       b[4] = {u[h].x, u[h].y, u[h].z, u[h].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint64_t act, slope;
            act_grad<ACT>(widen2(a[i]), act, slope);
            const uint64_t v = widen2(d[i]);
            du[4 * h + i] = f2_mul(v, act);
            dg[4 * h + i] = f2_mul(f2_mul(v, widen2(b[i])), slope);
        }
    }
}

// The same of 16 bf16 values, two at a time as long as that is exact (the maximum, and the product with
// a power of two: what it loses below bf16's range rounds to 0 all the same).
__device__ __forceinline__ uint4 quantise16(const uint4 (&w)[2], uint32_t &byte, bool &bad)
{
    const uint32_t p[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(p[i] & 0x7FFF7FFFu));
    const uint32_t top = block_top(max(m << 16, m & 0xFFFF0000u) & 0x7FFFFFFFu);
    if (top >= kFp8Inf) {
        bad = true;
        byte = 127u;
        return make_uint4(kFp8NanCodes, kFp8NanCodes, kFp8NanCodes, kFp8NanCodes);
    }
    byte = fp8_scale_byte(top);
    const uint32_t inv = __float_as_uint(fp8_inverse(byte)), inv2 = inv | inv >> 16;
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a, b;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(p[2 * i]), "r"(inv2));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(p[2 * i + 1]), "r"(inv2));
        c[i] = to_e4m3x4(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u), __uint_as_float(b << 16),
                         __uint_as_float(b & 0xFFFF0000u));
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// a block's byte to the word of its four blocks: lanes 0, 8, 16, 24 hold them
__device__ __forceinline__ uint32_t scale_word(uint32_t byte, int lane)
{
    uint32_t w = byte << (8 * (lane >> 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 8);
    w |= __shfl_xor_sync(0xffffffffu, w, 16);
    return w;
}

// What one warp does for the whole call: the status word (with `keep` it is only added to).
__device__ __forceinline__ void fp8_begin_call(const int32_t *offsets, int E, int64_t M, int keep, uint32_t *status,
                                               int lane)
{
    bool bad = false;
    if (E > 0)
        for (int i = lane; i <= E; i += 32) {
            const int32_t o = offsets[i];
            bad |= o < 0 || o > M || (i > 0 && o < offsets[i - 1]);
        }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        if (!keep)
            *status = bad ? kStatusIndex : 0u;
        else if (bad)
            atomicOr(status, kStatusIndex);
    }
}

// ---- tcgen05, block-scaled e4m3 --------------------------------------------------
// D[tmem] (+)= (A SFA)(B SFB)^T, 32 values deep; one e8m0 scale for each row's 32 values, picked
// from the rows' words by the two scale numbers in idesc.  CG = 1: this CTA, 2: the CTA pair
// (a, b: the low words of the operands' descriptors, desc_hi: the high word of both)
template <int CG>
__device__ __forceinline__ void mma_fp8(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t desc_hi, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate)
{
    if (CG == 2)
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
                     "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %7};\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.block32 [%0], da, db, %3, [%5], [%6], p;\n\t}"
                     ::"r"(d_tmem), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(desc_hi)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
                     "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %7};\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.block32 [%0], da, db, %3, [%5], [%6], p;\n\t}"
                     ::"r"(d_tmem), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(desc_hi)
                     : "memory");
}

// ---- copies of the product ---------------------------------------------------------
// CG = 2: counted on the pair's leader (see tma_load_2d_pair)
template <int CG>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int32_t x, int32_t y, int32_t z,
                                            uint32_t bar)
{
    if (CG == 2)
        asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3, %4}], [%5];"
                     ::"r"(dst), "l"((uint64_t)tmap), "r"(x), "r"(y), "r"(z), "r"(bar & 0xFEFFFFFFu) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3, %4}], [%5];"
                     ::"r"(dst), "l"((uint64_t)tmap), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

// the same box on its way into L2 only
__device__ __forceinline__ void tma_prefetch_3d(const void *tmap, int32_t x, int32_t y, int32_t z)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
                 ::"l"((uint64_t)tmap), "r"(x), "r"(y), "r"(z) : "memory");
}

// each thread of the warp reads 16 consecutive 32-bit columns of its lane
__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
}

// 16 bytes into another CTA's shared memory, counted on its barrier
__device__ __forceinline__ void st_async_v4(uint32_t cluster_addr, const float *v, uint32_t cluster_bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(cluster_addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"(cluster_bar) : "memory");
}

}  // namespace sq
