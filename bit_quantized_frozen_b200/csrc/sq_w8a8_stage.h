// sq_w8a8_stage.h -- the integer product's channel shares and shared-memory stages of one-CTA
// tiles (sq_w8a8.cu, few tokens): which channels a CTA takes, which copies bring a tile's weight
// rows, and what a stage reserves for them.  Plain arithmetic, the same on the host and the
// device, so that a host program can walk every share and check that the copies stay in it.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SQ_HD __host__ __device__ __forceinline__
#else
#define SQ_HD inline
#endif

namespace sq {

constexpr int kI8Chunk = 128;                     // summed values (bytes) of a shared-memory row
constexpr int kI8MaxStages = 24;                  // of one-CTA tiles

// one-CTA tiles of NT tokens: bytes for stages, and producer warps (each with its own stages: one
// copy takes a thread about 60 ns to issue, so tiles that need little time per stage share it out)
constexpr int i8_ring_bytes(int nt)
{
    return (nt == 128 ? 176 : 184) * 1024;
}
constexpr int i8_producers(int nt)
{
    return nt <= 32 ? 4 : 2;
}

// a CTA's share of all (token tile, channel) pairs, in tiles of up to 128 channels
struct I8ChannelWalk {
    int64_t pos, end;         // in groups of 4 channels, token tile after token tile
    int per_tile;             // N / 4
    int tile, n0, channels;

    SQ_HD I8ChannelWalk(int tiles, int64_t N, int cta, int ctas) : per_tile((int)(N / 4)), tile(0), n0(0), channels(0)
    {
        const int64_t all = (int64_t)tiles * per_tile;
        pos = all * cta / ctas;
        end = all * (cta + 1) / ctas;
    }
    // channels of the largest tile, at most
    SQ_HD int largest() const
    {
        return 4 * (end - pos) < 128 ? (int)(4 * (end - pos)) : 128;
    }
    SQ_HD bool next()
    {
        if (pos >= end)
            return false;
        tile = (int)(pos / per_tile);
        const int first = (int)(pos - (int64_t)tile * per_tile);
        const int left = (int)(end - pos < per_tile - first ? end - pos : per_tile - first);
        const int tiles_left = (left + 31) / 32;
        const int now = (left + tiles_left - 1) / tiles_left;      // of equal size
        n0 = 4 * first;
        channels = 4 * now;
        pos += now;
        return true;
    }
};

// Rows of the box that takes a CTA's whole tile in one copy.  Dense: the shares are known and
// nearly equal; experts: 128.  `only`: every tile of the call is taken so.
inline int i8_whole_box(int E, int64_t M, int64_t N, int ctas, int nt, bool *only)
{
    *only = false;
    if (E > 0)
        return 128;
    const int64_t all = (M + nt - 1) / nt * (N / 4), share = (all + ctas - 1) / ctas;
    const int64_t tiles = (share + 31) / 32, groups = (share + tiles - 1) / tiles;
    const int64_t rows = (4 * groups + 7) / 8 * 8;
    *only = M <= nt && (all / ctas + 31) / 32 == tiles;            // (sizes then differ by 4 channels)
    return rows < 16 ? 16 : (int)rows;
}

// Weight rows that a tile of `channels` takes up in a stage: whole 8-row groups, or the whole box
// where that is not much more (one copy instead of several).
SQ_HD int i8_weight_rows(int channels, int box)
{
    const int rows = channels <= 16 ? 16 : (channels + 7) / 8 * 8;
    return rows <= box && rows + 16 >= box ? box : rows;
}

// The copies of those rows: copy(kind, first row), kind 0 the whole box, 1 a box of 64 rows, 2 of
// 16.  Two boxes may overlap (the same bytes to the same place).
template <class Copy>
SQ_HD void i8_weight_copies(int rows, int box, const Copy &copy)
{
    if (rows == box) {
        copy(0, 0);
    } else if (rows > 64) {                       // two boxes, the second one back from the end
        copy(1, 0);
        copy(1, rows - 64);
    } else {
        for (int r = 0; r < rows; r += 16)
            copy(2, r < rows - 16 ? r : rows - 16);
    }
}

// rows that they bring, overlaps twice
SQ_HD int i8_copied_rows(int rows, int box)
{
    return rows == box ? box : rows > 64 ? 128 : (rows + 15) / 16 * 16;
}

// Rows that a stage reserves for the weight of any of the CTA's tiles: what the largest (of
// `largest` channels at most) takes up.  A smaller tile that is promoted to the whole box has at
// least box - 16 rows, so the largest is promoted too or is larger than the box.
SQ_HD int i8_stage_rows(int largest, int box)
{
    return i8_weight_rows(largest, box);
}

// A stage: `per` chunks, each the weight rows and then the tokens' codes.  A stage costs the MMA
// issuer about 85 ns (wait, commit) beside 20 ns for each of a chunk's four narrow MMAs, so few
// tokens take several chunks, as long as every producer has a stage to fill (16 tokens,
// N = K = 6144: one, two, four chunks 24.5, 17.4, 16.4 us a call).  Chunks behind the end of the
// summed axis read as 0.
struct I8Stages {
    int a_bytes, chunk_bytes, per, stage_bytes, stages;
};
SQ_HD I8Stages i8_stages(int rows, int token_bytes, int ring, int producers)
{
    I8Stages s;
    s.a_bytes = rows * kI8Chunk;
    s.chunk_bytes = s.a_bytes + token_bytes;
    s.per = 1;
    while (s.per < 4 && 2 * s.per * s.chunk_bytes * (producers > 4 ? producers : 4) <= ring)
        s.per *= 2;
    s.stage_bytes = s.per * s.chunk_bytes;
    const int fit = ring / s.stage_bytes;
    s.stages = (fit < kI8MaxStages ? fit : kI8MaxStages) / producers * producers;
    return s;
}

}  // namespace sq
