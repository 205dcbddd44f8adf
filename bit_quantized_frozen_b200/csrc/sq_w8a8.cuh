// sq_w8a8.cuh -- what the row quantisation (sq_w8a8_quant.cu) and the integer
// product (sq_w8a8.cu) share: the plan of tiles over the experts' rows, the tensor
// memory accesses and the MMA of 8-bit integers, and small products of low-rank values.
#pragma once

#include <cstdint>

#include "sq_device.cuh"

namespace sq {

constexpr int kI8Rank = 16;                       // rank of the int8 layer's low-rank branch
constexpr int kMaxExperts = 1024;

// where a tile lies
struct I8Tile {
    int e;                    // expert
    int row0, rows;           // first token and tokens of the tile
    int wt;                   // tile along the weight (0 with wts = 1)
};

// The tiles of all experts in a row: expert e has ceil(rows / tok_tile) token tiles, each times
// `wts` weight tiles; the token tile changes fastest, so that the tiles which share a weight
// tile run together.  Offsets are clamped to [0, M] and to their running maximum, so that the
// experts' rows never overlap or leave the matrix, whatever the offsets hold.
struct I8Plan {
    int32_t *start;           // [E + 1] first row of each expert (shared memory)
    int32_t *prefix;          // [E + 1] token tiles before each expert
    int E, wts, tok_tile;

    // every thread of the CTA; offsets NULL: one expert with all M rows
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

// ---- tensor memory and tcgen05 of the integer product ---------------------------
// D[tmem] (+)= A[smem] * B[smem]^T, signed 8-bit integers, 32-bit integer accumulation
// (exact while |sum| < 2^31); CG = 1: this CTA, 2: the CTA pair
template <int CG>
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate)
{
    if (CG == 2)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
                     ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
                     ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

// 16 lanes x 16 columns as the fragments of mma's accumulator: per 8 columns, thread 4 g + q
// gets (lane g, columns 2 q and 2 q + 1) and (lane g + 8, the same columns)
__device__ __forceinline__ void tmem_ld_frag2(uint32_t taddr, uint32_t (&r)[2][4])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0][0]), "=r"(r[0][1]), "=r"(r[0][2]), "=r"(r[0][3]), "=r"(r[1][0]), "=r"(r[1][1]),
                   "=r"(r[1][2]), "=r"(r[1][3])
                 : "r"(taddr)
                 : "memory");
}

// each thread writes 32 consecutive 32-bit columns of its lane
__device__ __forceinline__ void tmem_st_32cols(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
                   "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
                   "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
                   "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
                   "r"(v[29]), "r"(v[30]), "r"(v[31])
                 : "memory");
}

// ---- clusters, small products ----------------------------------------------------
// Every thread of the cluster meets here; nothing written before is published by it (the release
// of cluster_sync() waits for every global store that the CTA has on its way).  For barriers set up
// before with fence_mbar_init(), and for CTAs that must not leave before their peers.
__device__ __forceinline__ void cluster_meet()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// four 8x8 matrices of 16-bit values from shared memory (each lane gives one row's address);
// with TRANS each is transposed on the way
template <bool TRANS>
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4])
{
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

// c[16 x 8] += a[16 x 16] b[16 x 8], bf16 inputs, fp32 sums (one warp; the rows' low-rank input and
// the gradient's low-rank term -- the large products run on tcgen05)
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes, or 16 zero bytes with live = false (src is then not read)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// 16 values as pairs of neighbours, from fp32 (64 bytes) or bf16 (32 bytes)
__device__ __forceinline__ void pairs16(const float4 &a, const float4 &b, const float4 &c, const float4 &d,
                                        uint64_t (&f)[8])
{
    f[0] = f2_pack(a.x, a.y);
    f[1] = f2_pack(a.z, a.w);
    f[2] = f2_pack(b.x, b.y);
    f[3] = f2_pack(b.z, b.w);
    f[4] = f2_pack(c.x, c.y);
    f[5] = f2_pack(c.z, c.w);
    f[6] = f2_pack(d.x, d.y);
    f[7] = f2_pack(d.z, d.w);
}

constexpr int kLowParts = 3;                      // bf16 terms of an fp32 low-rank value

// v as the sum of three bf16 terms, largest first (24 significant bits: exact but for
// subnormal remainders)
__device__ __forceinline__ void split3(float v, uint32_t (&p)[kLowParts])
{
#pragma unroll
    for (int i = 0; i < kLowParts; ++i) {
        p[i] = f32_to_bf16_bits(v);
        v = __fsub_rn(v, bf16_bits_to_f32(p[i]));
    }
}

__device__ __forceinline__ void pairs16(const uint4 &a, const uint4 &b, uint64_t (&f)[8])
{
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] = f2_pack(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
}

// sum over r = 0 .. 15 of a[r] b[r]: even and odd r apart, then their sum
__device__ __forceinline__ float dot16(const uint64_t (&a)[8], const uint64_t (&b)[8])
{
    uint64_t s = 0;                               // (0.0f, 0.0f)
#pragma unroll
    for (int j = 0; j < 8; ++j)
        s = f2_fma(a[j], b[j], s);
    float lo, hi;
    f2_unpack(s, lo, hi);
    return __fadd_rn(lo, hi);
}

}  // namespace sq
