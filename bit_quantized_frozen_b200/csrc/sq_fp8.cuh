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

// ---- tcgen05, block-scaled e4m3 --------------------------------------------------
// D[tmem] (+)= (A SFA)(B SFB)^T, 32 values deep; one e8m0 scale for each row's 32 values, picked
// from the rows' words by the two scale numbers in idesc.  CG = 1: this CTA, 2: the CTA pair
template <int CG>
__device__ __forceinline__ void mma_fp8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate)
{
    if (CG == 2)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
                     ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
                     ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
                     : "memory");
}

// ---- mbarriers and copies of the product -----------------------------------------
// arrive on a barrier of any CTA of the cluster; shared memory written before (and handed to the
// async proxy by a fence) is seen by whoever waits with acquire at cluster scope
__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_acquire_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

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

}  // namespace sq
