// sq_fp8.cuh -- what the row rounding (sq_fp8_quant.cu) and the block-scaled e4m3 product
// (sq_fp8.cu) share: the launch arguments, the activations, and the tcgen05 instructions of
// kind::mxf8f6f4.
#pragma once

#include <cstdint>

#include "sq_device.cuh"

namespace sq {

constexpr int kFp8Block = 128;                    // values of a scale
constexpr int kFp8Group = 4;                      // blocks whose scales share a 32-bit word

// 32-bit words of row scales along an axis of `len` values (one tcgen05.cp brings a word of each row)
__host__ __device__ __forceinline__ int64_t fp8_groups(int64_t len)
{
    return (len + kFp8Block * kFp8Group - 1) / (kFp8Block * kFp8Group);
}

// sigmoid(v) and sigmoid(-v), both without cancellation: t = e^-|v| <= 1
__device__ __forceinline__ void sigmoid2(float v, float &s, float &other)
{
    const float t = __expf(-fabsf(v));
    const float big = __fdividef(1.0f, 1.0f + t), small = t * big;
    s = v < 0.0f ? small : big;
    other = v < 0.0f ? big : small;
    if (v != v)
        s = other = v;
}

constexpr float kGelu2C = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

// act(g); gelu: (1 + tanh z) / 2 = sigmoid(2 z)
template <int ACT>
__device__ __forceinline__ float act_value(float g)
{
    float s, o;
    sigmoid2(ACT == 0 ? g : kGelu2C * (g + kGeluCube * g * g * g), s, o);
    return g * s;
}

// act(g) and act'(g)
template <int ACT>
__device__ __forceinline__ void act_grad(float g, float &a, float &slope)
{
    float s, o;
    sigmoid2(ACT == 0 ? g : kGelu2C * (g + kGeluCube * g * g * g), s, o);
    a = g * s;
    const float w = s * o;                        // sigmoid'; where it is 0, so is its term, whatever g^2 comes to
    if (ACT == 0)
        slope = s + (w == 0.0f ? 0.0f : g * w);
    else
        slope = s + (w == 0.0f ? 0.0f : g * w * (kGelu2C + 3.0f * kGelu2C * kGeluCube * g * g));
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

// A lane's 16 neighbouring values of a row (8 lanes a block): their codes, and the block's byte.
__device__ __forceinline__ uint4 quantise16(const float (&v)[16], uint32_t &byte, bool &bad)
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int x = 1; x <= 4; x <<= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
    if (top >= kFp8Inf) {
        bad = true;
        byte = 127u;
        return make_uint4(kFp8NanCodes, kFp8NanCodes, kFp8NanCodes, kFp8NanCodes);
    }
    byte = fp8_scale_byte(top);
    const float inv = fp8_inverse(byte);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = to_e4m3x4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
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

// 16 bytes into another CTA's shared memory, counted on its barrier
__device__ __forceinline__ void st_async_v4(uint32_t cluster_addr, const float *v, uint32_t cluster_bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(cluster_addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"(cluster_bar) : "memory");
}

}  // namespace sq
