"""The few-token forward's channel shares and shared-memory stages, walked on the host.

sq_w8a8_stage.h holds the arithmetic that the kernel and its launch use.  The program below compiles
it with the host compiler and walks every CTA's share of the channels, for every N of a dense call
and for many (token tiles, N) of grouped ones: no copy of weight rows may reach past the rows that
the stage reserves for them (the token codes lie behind), the bytes must be those the barrier
expects, the stages must fit, and the shares must cover every channel once.
"""
import os
import shutil
import subprocess

import pytest

from bit_quantized_frozen_b200 import build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "sq_w8a8_stage.h"
using namespace sq;

static long long walked, promoted;

static void fail(const char *what, int nt, int E, int tiles, long long N, int ctas, int cta, int channels)
{
    std::printf("%s: tile of %d tokens, E %d, %d token tiles, N %lld, CTA %d of %d, %d channels\n", what, nt, E, tiles, N,
                cta, ctas, channels);
    std::exit(1);
}

static void walk(int nt, int E, int tiles, long long N, int ctas)
{
    bool only = false;
    const int box = i8_whole_box(E, nt, N, ctas, nt, &only);
    long long covered = 0;
    for (int cta = 0; cta < ctas; ++cta) {
        I8ChannelWalk share(tiles, N, cta, ctas);
        auto bad = [&](const char *what) { fail(what, nt, E, tiles, N, ctas, cta, share.channels); };
        const int rows = i8_stage_rows(share.largest(), box);
        const int ring = i8_ring_bytes(nt), P = i8_producers(nt);
        const I8Stages s = i8_stages(rows, nt * kI8Chunk, ring, P);
        if (rows < 8 || rows > 128 || rows % 8)
            bad("reserved rows");
        if (s.stages < P || s.stages % P || s.stages > kI8MaxStages || s.stages * s.stage_bytes > ring)
            bad("stages do not fit");
        if (s.a_bytes % 1024 || s.chunk_bytes != s.a_bytes + nt * 128 || s.stage_bytes != s.per * s.chunk_bytes)
            bad("layout of a stage");
        for (; share.next(); ++walked) {
            if (share.channels < 4 || share.channels > 128 || share.n0 < 0 || share.n0 + share.channels > N ||
                share.tile >= tiles)
                bad("share");
            covered += share.channels;
            const int have = i8_weight_rows(share.channels, box);
            promoted += have == box && box > share.channels + 7;
            if (only && have != box)
                bad("a tile that the one box does not take");
            int end = 0, bytes = 0;
            i8_weight_copies(have, box, [&](int kind, int at) {
                const int size = kind == 0 ? box : kind == 1 ? 64 : 16;
                if (at < 0 || at > end || at % 8)
                    bad("a gap between copies");
                if (at + size > rows)
                    bad("a copy reaches past the reserved rows");
                end = at + size > end ? at + size : end;
                bytes += size;
            });
            if (end < share.channels)
                bad("channels that no copy brings");
            if (bytes != i8_copied_rows(have, box))
                bad("bytes that the barrier does not expect");
        }
    }
    if (covered != (long long)tiles * N)
        fail("channels left out or taken twice", nt, E, tiles, N, ctas, -1, 0);
}

int main()
{
    const int sizes[] = {16, 32, 64, 128};
    for (int nt : sizes) {
        for (int ctas : {148, 132, 1})
            for (long long N = 128; N <= (ctas == 148 ? 1 << 20 : 32768); N += N < 32768 ? 128 : 128 * 61)
                walk(nt, 0, 1, N, ctas);
        // (a CTA with several tiles' worth of channels reserves a whole box: the large sizes are sampled)
        for (int ctas : {148, 132})
            for (int tiles = 1; tiles <= 2300; tiles += tiles < 200 ? 1 : 131)
                for (long long N = 128; N <= 20480; N += tiles * N < 40000 ? 128 : 128 * 19)
                    walk(nt, 8, tiles, N, ctas);
    }
    std::printf("%lld tiles, %lld with a box larger than their rows\n", walked, promoted);
    return promoted > 0 ? 0 : 1;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_copies_stay_in_their_stage(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", build.CSRC, str(src), "-o", str(exe)],
                   check=True)
    p = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout


def test_the_kernel_uses_this_arithmetic():
    """The product's source takes shares, rows, copies and stages from the header the walk checks."""
    text = open(os.path.join(build.CSRC, "sq_w8a8.cu")).read()
    for name in ("I8ChannelWalk", "i8_whole_box(", "i8_weight_rows(", "i8_weight_copies(", "i8_copied_rows(",
                 "i8_stage_rows(", "i8_stages(", "i8_ring_bytes(", "i8_producers("):
        assert name in text, name
    assert "struct I8ChannelWalk" not in text
