"""The block-scaled products as programs call them: special values, a whole feed-forward block and its
gradient, streams, captured graphs, the ends of their ranges, the builder."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import bit_quantized_frozen_b200 as sq
import fp8ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def weight(q, s):
    c, e = dev(q).to(torch.float8_e4m3fn), dev(s).view(torch.float8_e8m0fnu)
    if q.ndim == 3:
        return sq.GroupedWeight(*q.shape, c, e, fmt=sq.SQ_FMT_FP8_BLOCK)
    return sq.Weight(sq.SQ_FMT_FP8_BLOCK, *q.shape, c, e)


def layer(rng, N, K, E=None):
    """Codes and scales of a layer whose sums over K are about 1."""
    q, s = ref.layer(rng, N, K, E)
    return q, (s.astype(int) - 113 + 127 - round(np.log2(np.sqrt(K) * 90))).astype(np.uint8)


def rand(rng, M, width, size=1.0):
    return ref.bf16((rng.standard_normal((M, width)) * size).astype(np.float32))


def f32(t):
    return t.float().cpu().numpy()


# ---- the builder ---------------------------------------------------------------------------------

@pytest.mark.parametrize("N,K", [(16, 16), (128, 128), (144, 400), (272, 2064)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_builder_bit_for_bit(N, K, dtype):
    """Codes and scales are the definition's, with blocks of zeros, of subnormal and of the largest values,
    NaN and infinities among them."""
    rng = np.random.default_rng(N + K)
    W = (rng.standard_normal((N, K)) * np.exp(rng.standard_normal((N, 1)) * 3)).astype(np.float32)
    W[:8, :8] = 0
    W[3, 5], W[N - 1, K - 1], W[N // 2, K // 2] = np.nan, np.inf, -np.inf
    if N > 128:
        W[128:, :128] = 0
        W[128, 0] = 1e-39
        W[128:, 128:256] = 3.3e38
    if K > 300:
        W[:128, 256:] *= 1e-38
    W = dev(W).to(dtype)
    w = sq.build_fp8(W)
    q, s = ref.build(f32(W))
    got = f32(w.codes)
    assert np.array_equal(np.isnan(got), np.isnan(q)) and np.array_equal(w.scales.view(torch.uint8).cpu().numpy(), s)
    full = np.repeat(np.repeat(s.astype(np.float64), 128, 0), 128, 1)[:N, :K]
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(q)), full
    E = sq.build_fp8_grouped(torch.stack([W, W.flip(0).contiguous()]))
    assert torch.equal(E.expert(0).codes.view(torch.uint8), w.codes.view(torch.uint8)) and E.expert(1).N == N


def test_built_weight_in_a_product():
    """y of a built weight lies within the roundings of W and x (half a step of e4m3 each, 2^-4 of the value)."""
    rng = np.random.default_rng(4)
    M, N, K = 70, 528, 912
    W, x = rng.standard_normal((N, K)).astype(np.float32) / 30, rand(rng, M, K)
    y = f32(sq.linear_fwd_fp8(sq.build_fp8(dev(W)), dev(x, BF)))
    want, mag = x.astype(np.float64) @ W.T.astype(np.float64), np.abs(x.astype(np.float64)) @ np.abs(W).T
    small = 2.0 ** -10 / 448 * 2       # below 2^-6 of the scale the step is 2^-9 of it, at most 2^-9 2 max / 448
    tops = np.abs(x).max() * np.abs(W).sum(axis=1)[None, :] + np.abs(x).sum(axis=1)[:, None] * np.abs(W).max()
    assert (np.abs(y - want) <= mag * (2 * 2.0 ** -4 + 2.0 ** -8) + small * tops).all()
    assert np.linalg.norm(y - want) <= 0.06 * np.linalg.norm(want)


# ---- special values ------------------------------------------------------------------------------

@pytest.mark.parametrize("M", [5, 40, 300])
def test_special_rows(M):
    """A NaN or an infinity makes its row NaN and is reported on demand; zeros, the smallest and the largest
    values come out as the definition has them; other rows are not affected."""
    rng = np.random.default_rng(M)
    N, K = 272, 400
    q, s = layer(rng, N, K)
    w, W = weight(q, s), ref.dequant(q, s)
    x, dy = rand(rng, M, K), rand(rng, M, N)
    for v in (x, dy):
        v[0] = 0
        v[1] = ref.bf16(np.float32(1e-39) * rng.standard_normal(v.shape[1]).astype(np.float32))
        v[2, ::7] = 3.3e38
    plain = [(sq.linear_fwd_fp8, x, ref.forward), (sq.linear_bwd_dx_fp8, dy, ref.backward)]
    for f, v, r in plain:
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        got = f(w, dev(v, BF), ws=ws, flags=sq.SQ_CHECK_FINITE)
        sq.sq_check_device_status(ws)
        want, bound = r(v, W)
        # products below fp32's normal range (row 1) may be cut to it.  Row 2: where the magnitudes of a sum
        # add up to more than fp32 holds (about 57 terms of 3.3e38 times a weight of 0.05: 9e38), a part of
        # it, in whatever order, may pass the end of the range, and says nothing
        most = bound / (2 * ref.U23) * 32 / (ref.nblocks(v.shape[1]) * 128)
        big = most > 3.4e38
        assert not big[[0, 1]].any() and not big[3:].any()
        ref.check(np.where(big, 0, f32(got)), np.where(big, 0, want), bound + 2.0 ** -126 * v.shape[1], False)
        assert not f32(got)[0].any()
        for bad in (np.nan, np.inf, -np.inf):
            u = v.copy()
            u[3, 200], u[4, 0] = bad, bad
            again = f(w, dev(u, BF), ws=ws, flags=sq.SQ_CHECK_FINITE)
            with pytest.raises(sq.SqError) as e:
                sq.sq_check_device_status(ws)
            assert e.value.status == 9
            assert torch.isnan(again[3:5]).all()
            keep = torch.arange(M, device="cuda") % M
            keep = keep[(keep != 3) & (keep != 4)]
            assert torch.equal(again[keep].view(torch.int32), got[keep].view(torch.int32))
            again = f(w, dev(u, BF), ws=ws)
            sq.sq_check_device_status(ws)                    # not asked for
            assert torch.isnan(again[3:5]).all()


@pytest.mark.parametrize("M", [3, 33, 257])
def test_nan_weights_stay_in_their_columns(M):
    """A NaN code or scale byte of one expert reaches the sums that it enters, not its neighbours."""
    rng = np.random.default_rng(M)
    E, N, K = 3, 144, 272
    q, s = layer(rng, N, K, E)
    x, dy = rand(rng, M, K), rand(rng, M, N)
    off = dev(np.array([0, M // 3, 2 * M // 3, M], np.int32))
    w = weight(q, s)
    y, dx = sq.grouped_fwd_fp8(w, dev(x, BF), off), sq.grouped_bwd_dx_fp8(w, dev(dy, BF), off)
    w.codes.view(torch.uint8)[1, 0, 5] = 0x7F                # first row of expert 1: next to expert 0's last rows
    y2, dx2 = sq.grouped_fwd_fp8(w, dev(x, BF), off), sq.grouped_bwd_dx_fp8(w, dev(dy, BF), off)
    mid = slice(M // 3, 2 * M // 3)
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[mid] = False
    assert torch.isnan(y2[mid, 0]).all() and torch.isnan(dx2[mid, 5]).all()
    assert torch.equal(y2[rest], y[rest]) and torch.equal(dx2[rest], dx[rest])
    assert torch.equal(y2[mid, 1:], y[mid, 1:])
    w.codes.view(torch.uint8)[1, 0, 5] = 0
    w.scales.view(torch.uint8)[1, 1, 2] = 255                # rows 128 .. 143, columns 256 .. 271
    y2, dx2 = sq.grouped_fwd_fp8(w, dev(x, BF), off), sq.grouped_bwd_dx_fp8(w, dev(dy, BF), off)
    assert torch.isnan(y2[mid, 128:]).all() and not torch.isnan(y2[mid, :128]).any()
    assert torch.isnan(dx2[mid, 256:]).all() and not torch.isnan(dx2[mid, :256]).any()
    assert torch.equal(y2[rest], y[rest]) and torch.equal(dx2[rest], dx[rest])


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("M", [4, 50])
def test_gated_at_the_ends_of_the_activation(kind, M):
    """Gates far out on both sides, zeros among dh, g and u: finite gradients as the definition has them."""
    rng = np.random.default_rng(M)
    N, K = 256, 144
    (qg, sg), (qu, su) = layer(rng, N, K), layer(rng, N, K)
    g = np.tile(ref.bf16(np.array([-3e38, -1e20, -100, -30, -5, -1e-30, 0, 1e-30, 5, 30, 100, 1e19, 0, -0.7517, -1.28, 1],
                                  np.float32)), (M, N // 16))
    dh, u = rand(rng, M, N, 1e-2), rand(rng, M, N)
    dh[:, ::11], u[:, 5::13] = 0, 0
    dh[0], u[1] = 0, 0
    g[2] = 0
    dx = sq.gated_bwd_dx_fp8(weight(qg, sg), weight(qu, su), dev(dh, BF), dev(g, BF), dev(u, BF), act=kind)
    ref.check(f32(dx), *ref.gated_backward(dh, g, u, ref.dequant(qg, sg), ref.dequant(qu, su), kind), False)
    assert torch.isfinite(dx).all() and not dx[0].any()


@pytest.mark.parametrize("off", [[-5, 3, 7, 9], [0, 8, 4, 9], [0, 2, 5, 99], [9, 6, 3, 0], [2 ** 31 - 1] * 4, [-2 ** 31] * 4])
@pytest.mark.parametrize("M", [9, 90])
def test_bad_offsets_are_clamped_and_reported(off, M):
    rng = np.random.default_rng(1)
    N, K = 144, 272
    w, v = weight(*layer(rng, N, K, 3)), weight(*layer(rng, N, K, 3))
    off = dev(np.array([o * (M // 9) if abs(o) < 100 else o for o in off], np.int32))
    x, dy = dev(rand(rng, M, K), BF), dev(rand(rng, M, N), BF)
    for call in (lambda ws: sq.grouped_fwd_fp8(w, x, off, ws=ws), lambda ws: sq.grouped_bwd_dx_fp8(w, dy, off, ws=ws),
                 lambda ws: sq.grouped_gated_fwd_fp8(w, v, x, off, save=True, ws=ws),
                 lambda ws: sq.grouped_gated_bwd_dx_fp8(w, v, dy, dy, dy, off, ws=ws)):
        buf = torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
        call(buf[: 1 << 19])
        with pytest.raises(sq.SqError) as e:
            sq.sq_check_device_status(buf)
        assert e.value.status == 10
        assert bool((buf[1 << 19:] == 0xFF).all())


def test_no_rows():
    rng = np.random.default_rng(2)
    w = weight(*layer(rng, 128, 128, 2))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    empty = torch.empty(0, 128, dtype=BF, device="cuda")
    assert sq.grouped_fwd_fp8(w, empty, off).shape == (0, 128)
    h, g, u = sq.grouped_gated_fwd_fp8(w, w, empty, off, save=True)
    assert h.shape == g.shape == u.shape == (0, 128)
    with pytest.raises(sq.SqError):
        sq.linear_fwd_fp8(w.expert(0), empty)
    for M in (3, 100):                                       # rows, but none of any expert
        y = sq.grouped_fwd_fp8(w, torch.full((M, 128), float("nan"), dtype=BF, device="cuda"), off)
        assert not y.any()


# ---- gradients -----------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("M", [6, 75])
def test_gradient_against_differences(kind, M):
    """sum(dh h) over a step of x along v changes as dx v says, but for the rounding of dg and du (half a
    step of e4m3, 2^-4 of each value, or 2^-10 of its block's scale)."""
    rng = np.random.default_rng(M)
    N, K = 272, 144
    (qg, sg), (qu, su) = layer(rng, N, K), layer(rng, N, K)
    Wg, Wu = ref.dequant(qg, sg), ref.dequant(qu, su)
    x, dh = rand(rng, M, K).astype(np.float64), rand(rng, M, N)
    g, u = x @ Wg.T, x @ Wu.T
    dx = f32(sq.gated_bwd_dx_fp8(weight(qg, sg), weight(qu, su), dev(dh, BF), dev(ref.bf16(g.astype(np.float32)), BF),
                                 dev(ref.bf16(u.astype(np.float32)), BF), act=kind)).astype(np.float64)
    v = rng.standard_normal((M, K))
    t = 1e-5
    f = lambda z: (dh * ref.act(z @ Wg.T, kind)[0] * (z @ Wu.T)).sum(axis=1)  # noqa: E731
    diff = (f(x + t * v) - f(x - t * v)) / (2 * t)
    a, slope, _, _ = ref.act(g, kind)
    dg, du = np.abs(dh * u * slope), np.abs(dh * a)
    # g and u as kept: half a step of bf16, 2^-8, which moves dg and du by what act'' <= 1.2 and act' <= 1.13 allow
    dg = dg * (2.0 ** -4 + 2 * 2.0 ** -8) + 1.2 * np.abs(dh * u * g) * 2.0 ** -8 + dg.max(axis=1, keepdims=True) / 224 * 2.0 ** -10
    du = du * (2.0 ** -4 + 2 * 2.0 ** -8) + 1.13 * np.abs(dh * g) * 2.0 ** -8 + du.max(axis=1, keepdims=True) / 224 * 2.0 ** -10
    bound = (dg * np.abs(v @ Wg.T) + du * np.abs(v @ Wu.T)).sum(axis=1)
    assert (np.abs((dx * v).sum(axis=1) - diff) <= bound + 1e-6).all()
    assert np.corrcoef((dx * v).sum(axis=1), diff)[0, 1] > 0.99


@pytest.mark.parametrize("M", [1, 14, 70, 400])
def test_feed_forward_block_and_its_gradient(M):
    """Gate, up, down and back, dense and by experts, each step from what the step before gave."""
    rng = np.random.default_rng(M)
    F, K, E = 528, 272, 3
    qs = [layer(rng, F, K, E), layer(rng, F, K, E), layer(rng, K, F, E)]
    gate, up, down = (weight(*q) for q in qs)
    off = np.array([0, M // 4, M // 4, M], np.int32)
    x, dy = rand(rng, M, K), rand(rng, M, K, 1e-2)
    offd, xd, dyd = dev(off), dev(x, BF), dev(dy, BF)
    for dense in (False, True):
        if dense:
            g_, u_, d_ = (w.expert(2) for w in (gate, up, down))
            h, g, u = sq.gated_fwd_fp8(g_, u_, xd, save=True, out_bf16=True)
            y = sq.linear_fwd_fp8(d_, h, out_bf16=True)
            dh = sq.linear_bwd_dx_fp8(d_, dyd, out_bf16=True)
            dx = sq.gated_bwd_dx_fp8(g_, u_, dh, g, u)
            spans = [(2, 0, M)]
        else:
            h, g, u = sq.grouped_gated_fwd_fp8(gate, up, xd, offd, save=True, out_bf16=True)
            y = sq.grouped_fwd_fp8(down, h, offd, out_bf16=True)
            dh = sq.grouped_bwd_dx_fp8(down, dyd, offd, out_bf16=True)
            dx = sq.grouped_gated_bwd_dx_fp8(gate, up, dh, g, u, offd)
            spans = [(e, off[e], off[e + 1]) for e in range(E) if off[e + 1] > off[e]]
        h, g, u, y, dh, dx = (f32(v) for v in (h, g, u, y, dh, dx))
        for e, a, b in spans:
            Wg, Wu, Wd = (ref.dequant(q[e], s[e]) for q, s in qs)
            for got, (v, bound) in zip((h, g, u), ref.gated_forward(x[a:b], Wg, Wu, "silu")):
                ref.check(got[a:b], v, bound, True)
            ref.check(y[a:b], *ref.forward(h[a:b], Wd), True)
            ref.check(dh[a:b], *ref.backward(dy[a:b], Wd), True)
            ref.check(dx[a:b], *ref.gated_backward(dh[a:b], g[a:b], u[a:b], Wg, Wu, "silu"), False)


# ---- streams, graphs, company --------------------------------------------------------------------

def jobs_of(rng, sizes, N=272, K=528, E=4):
    w, v = weight(*layer(rng, N, K, E)), weight(*layer(rng, N, K, E))
    jobs = []
    for M in sizes:
        x, dy, g, u = (dev(rand(rng, M, n), BF) for n in (K, N, N, N))
        off = dev(np.sort(rng.integers(0, M + 1, E + 1)).astype(np.int32))
        a, b = w.expert(2), v.expert(1)
        jobs += [lambda s=None, x=x: sq.linear_fwd_fp8(a, x, stream=s),
                 lambda s=None, dy=dy: sq.linear_bwd_dx_fp8(b, dy, out_bf16=True, stream=s),
                 lambda s=None, x=x: sq.gated_fwd_fp8(a, b, x, save=True, stream=s)[0],
                 lambda s=None, dy=dy, g=g, u=u: sq.gated_bwd_dx_fp8(a, b, dy, g, u, act="gelu", stream=s),
                 lambda s=None, x=x, off=off: sq.grouped_fwd_fp8(w, x, off, out_bf16=True, stream=s),
                 lambda s=None, dy=dy, off=off: sq.grouped_bwd_dx_fp8(w, dy, off, stream=s),
                 lambda s=None, x=x, off=off: sq.grouped_gated_fwd_fp8(w, v, x, off, stream=s),
                 lambda s=None, dy=dy, g=g, u=u, off=off: sq.grouped_gated_bwd_dx_fp8(w, v, dy, g, u, off, stream=s)]
    return jobs


def test_many_calls_at_once():
    """Calls of different sizes in flight on four streams: each gives the bits that it gives alone."""
    rng = np.random.default_rng(7)
    jobs = jobs_of(rng, (1, 12, 16, 17, 40, 140, 333))
    alone = [j() for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [(i, jobs[i](streams[(k + i) % 4])) for k in range(4) for i in rng.permutation(len(jobs))]
    torch.cuda.synchronize()
    for i, y in got:
        assert torch.equal(y, alone[i]), i


def test_call_after_call_without_waiting():
    """The same calls in a row, small ones between large ones: no call reads what another one still writes."""
    rng = np.random.default_rng(8)
    jobs = jobs_of(rng, (2, 300))
    alone = [j() for j in jobs]
    torch.cuda.synchronize()
    got = [(i, jobs[i]()) for i in rng.integers(0, len(jobs), 400)]
    torch.cuda.synchronize()
    for i, y in got:
        assert torch.equal(y, alone[i]), i


@pytest.mark.parametrize("M", [3, 90, 700])
def test_a_graph_that_forks_and_joins(M):
    rng = np.random.default_rng(M)
    N, K = 528, 784
    A, B = layer(rng, N, K), layer(rng, N, K)
    a, b = weight(*A), weight(*B)
    WA, WB = ref.dequant(*A), ref.dequant(*B)
    x = dev(rand(rng, M, K), BF)
    other = torch.cuda.Stream()
    sq.linear_fwd_fp8(a, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        other.wait_stream(main)
        h, g, u = sq.gated_fwd_fp8(a, b, x, save=True, out_bf16=True)
        with torch.cuda.stream(other):
            y = sq.linear_fwd_fp8(b, x, flags=sq.SQ_CHECK_FINITE, out_bf16=True)
            dy = sq.linear_bwd_dx_fp8(a, y)
        main.wait_stream(other)
        s = h + y
        dx = sq.gated_bwd_dx_fp8(a, b, s, g, u)
    for _ in range(3):
        v = rand(rng, M, K)
        x.copy_(dev(v, BF))
        graph.replay()
        torch.cuda.synchronize()
        for got, (w, bound) in zip((h, g, u), ref.gated_forward(v, WA, WB, "silu")):
            ref.check(f32(got), w, bound, True)
        ref.check(f32(y), *ref.forward(v, WB), True)
        ref.check(f32(dy), *ref.backward(f32(y), WA), False)
        ref.check(f32(dx), *ref.gated_backward(f32(s), f32(g), f32(u), WA, WB, "silu"), False)


@pytest.mark.parametrize("M", [20, 200])
def test_captured_grouped_calls_follow_the_offsets(M):
    rng = np.random.default_rng(M)
    E, N, K = 4, 144, 272
    q, s = layer(rng, N, K, E)
    w = weight(q, s)
    x = rand(rng, M, K)
    xd, off = dev(x, BF), torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    sq.grouped_fwd_fp8(w, xd, off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sq.grouped_fwd_fp8(w, xd, off)
    for _ in range(6):
        o = np.sort(rng.integers(0, M + 1, E + 1)).astype(np.int32)
        off.copy_(dev(o))
        graph.replay()
        torch.cuda.synchronize()
        got = f32(y)
        assert not got[:o[0]].any() and not got[o[-1]:].any()
        for e in range(E):
            if o[e + 1] > o[e]:
                ref.check(got[o[e]:o[e + 1]], *ref.forward(x[o[e]:o[e + 1]], ref.dequant(q[e], s[e])), False)


FIRST = r'''
import sys
sys.path.insert(0, sys.argv[1])
import torch
import bit_quantized_frozen_b200 as sq
M, op = int(sys.argv[2]), sys.argv[3]
N = K = 256
c = torch.ones(N, K, device="cuda").to(torch.float8_e4m3fn)
e = torch.full((2, 2), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
w = sq.Weight(sq.SQ_FMT_FP8_BLOCK, N, K, c, e)
x = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    y = sq.linear_fwd_fp8(w, x) if op == "fwd" else sq.linear_bwd_dx_fp8(w, x)
g.replay()
torch.cuda.synchronize()
assert bool((y == 256).all())
print("fine")
'''


@pytest.mark.parametrize("M", [4, 60, 600])
@pytest.mark.parametrize("op", ["fwd", "bwd"])
def test_first_call_inside_a_capture(M, op):
    r = subprocess.run([sys.executable, "-c", FIRST, ROOT, str(M), op], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


DEBUG = r'''
import sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import numpy as np, torch
import bit_quantized_frozen_b200 as sq
import test_fp8_calls_gpu as t
assert sq.sq_debug_checks() == int(sys.argv[2])
out = [j().float().cpu().numpy() for j in t.jobs_of(np.random.default_rng(5), (3, 50, 290))]
sq.sq_check_device_status(None)
np.savez(sys.argv[3], *out)
'''


def test_debug_library_gives_the_same_bits(tmp_path):
    from bit_quantized_frozen_b200 import build
    got = []
    for flag, lib in ((0, build.LIB), (1, build.LIB_DEBUG)):
        path = str(tmp_path / f"{flag}.npz")
        r = subprocess.run([sys.executable, "-c", DEBUG, ROOT, str(flag), path], capture_output=True, text=True, timeout=900,
                           env=dict(os.environ, SQ_LIBSQ_PATH=lib))
        assert r.returncode == 0, r.stderr[-2000:]
        got.append(np.load(path))
    assert got[0].files == got[1].files
    for k in got[0].files:
        assert np.array_equal(got[0][k], got[1][k])


def test_few_rows_need_no_workspace():
    """The bits of a call without a workspace, whose status is the library's own word, and with one."""
    rng = np.random.default_rng(3)
    w = weight(*layer(rng, 400, 272))
    x = dev(rand(rng, 16, 272), BF)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    y = torch.empty(16, 400, device="cuda")
    sq.sq_linear_fwd_fp8(w, x, y)
    assert torch.equal(y, sq.linear_fwd_fp8(w, x, ws=ws))
    sq.sq_check_device_status(ws)
    x[3, 7] = float("inf")
    sq.sq_linear_fwd_fp8(w, x, y, sq.SQ_CHECK_FINITE)
    x[3, 7] = 0
    sq.sq_linear_fwd_fp8(w, x, y, sq.SQ_CHECK_FINITE)        # (does not clear what the call before has found)
    with pytest.raises(sq.SqError) as e:
        sq.sq_check_device_status(None)
    assert e.value.status == 9
    sq.sq_check_device_status(None)
    with pytest.raises(sq.SqError):
        sq.sq_linear_fwd_fp8(w, torch.zeros(33, 272, dtype=BF, device="cuda"), torch.empty(33, 400, device="cuda"))


def test_views_and_streams():
    """Rows and experts that are views into larger tensors; a stream given by its handle."""
    rng = np.random.default_rng(9)
    q, s = layer(rng, 272, 144, 2)
    w = weight(q, s)
    x = rand(rng, 90, 144)
    big = dev(np.concatenate([x, x]), BF)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for M in (8, 90):
        y = sq.linear_fwd_fp8(w.expert(1), big[5:5 + M], stream=st.cuda_stream)
        st.synchronize()
        ref.check(f32(y), *ref.forward(np.concatenate([x, x])[5:5 + M], ref.dequant(q[1], s[1])), False)
    with pytest.raises(ValueError, match="contiguous"):
        sq.linear_fwd_fp8(w.expert(1), big.t().contiguous().t())


# ---- the ends of the ranges ----------------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", [(1, 1 << 20, 16), (40, 1 << 20, 16), (2, 16, 1 << 20), (40, 16, 1 << 20), (300, 16, 1 << 20),
                                   (1 << 21, 16, 32)])
def test_ends_of_the_ranges(M, N, K):
    """The widest layers, the longest sums, very many rows; both ends and the middle are compared."""
    rng = np.random.default_rng(M + K)
    q, s = ref.layer(rng, N, K)
    w = weight(q, s)
    part = lambda n, k: np.unique(np.r_[0:min(n, k), n // 2:min(n, n // 2 + k), max(0, n - k):n])  # noqa: E731
    m, n, k = part(M, 30), part(N, 150), part(K, 150)
    x, dy = rand(rng, M, K), rand(rng, M, N)
    W = ref.dequant(q, s)
    y = sq.linear_fwd_fp8(w, dev(x, BF))
    ref.check(f32(y[dev(m)][:, dev(n)]), *ref.forward(x[m], W[n]), False)
    del y
    dx = sq.linear_bwd_dx_fp8(w, dev(dy, BF))
    ref.check(f32(dx[dev(m)][:, dev(k)]), *ref.backward(dy[m], W[:, k]), False)


def test_offsets_past_32_bits():
    """More than 2^31 row values, codes and weight values; saved products past 2^31 values."""
    rng = np.random.default_rng(0)
    M, N, K = 140_000, 16, 16_384
    q, s = layer(rng, N, K)
    x = torch.randn(M, K, dtype=BF, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    m = np.r_[0:20, M // 2:M // 2 + 20, M - 20:M]
    ref.check(f32(sq.linear_fwd_fp8(weight(q, s), x)[dev(m)]), *ref.forward(f32(x[dev(m)]), ref.dequant(q, s)), False)
    q, s = layer(rng, K, N)
    dx = sq.linear_bwd_dx_fp8(weight(q, s), x)
    ref.check(f32(dx[dev(m)]), *ref.backward(f32(x[dev(m)]), ref.dequant(q, s)), False)
    del dx
    h, g, u = sq.gated_fwd_fp8(weight(q, s), weight(q, s), x[:, :N].contiguous(), save=True, out_bf16=True)
    W = ref.dequant(q, s)
    for got, (v, bound) in zip((h, g, u), ref.gated_forward(f32(x[dev(m)][:, :N]), W, W, "silu")):
        ref.check(f32(got[dev(m)]), v, bound, True)
    dx = sq.gated_bwd_dx_fp8(weight(q, s), weight(q, s), h, g, u)
    ref.check(f32(dx[dev(m)]), *ref.gated_backward(f32(h[dev(m)]), f32(g[dev(m)]), f32(u[dev(m)]), W, W, "silu"), False)
    del x, h, g, u, dx
    E, N, K = 130, 4096, 4112                                # experts
    c = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    e = torch.full((E, 32, 33), 120, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    q, s = ref.layer(rng, N, K)
    c[E - 1].copy_(dev(q).to(torch.float8_e4m3fn))
    e.view(torch.uint8)[E - 1] = dev(s)
    w = sq.GroupedWeight(E, N, K, c, e, fmt=sq.SQ_FMT_FP8_BLOCK)
    for M in (10, 50):
        x = rand(rng, M, K)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[E] = M
        y = sq.grouped_fwd_fp8(w, dev(x, BF), off)
        ref.check(f32(y), *ref.forward(x, ref.dequant(q, s)), False)
        dy = rand(rng, M, N)
        ref.check(f32(sq.grouped_bwd_dx_fp8(w, dev(dy, BF), off)), *ref.backward(dy, ref.dequant(q, s)), False)


@pytest.mark.parametrize("E,M", [(1024, 1), (1024, 30), (1024, 20000), (1, 1), (64, 9000)])
def test_few_and_many_rows_of_many_experts(E, M):
    N, K = 128, 144
    rng = np.random.default_rng(E + M)
    q, s = layer(rng, N, K, E)
    w = weight(q, s)
    counts = np.zeros(E, int)
    if M < 10:
        counts[-1] = M
    else:
        counts = rng.multinomial(M - 6, rng.dirichlet(np.full(E, 0.3)))
    before = (M - int(counts.sum())) // 2
    off = before + np.concatenate([[0], np.cumsum(counts)])
    x, dy = rand(rng, M, K), rand(rng, M, N)
    offd = dev(off.astype(np.int32))
    y, dx = f32(sq.grouped_fwd_fp8(w, dev(x, BF), offd)), f32(sq.grouped_bwd_dx_fp8(w, dev(dy, BF), offd))
    for v in (y, dx):
        assert not v[:off[0]].any() and not v[off[-1]:].any()
    for e in np.nonzero(counts)[0]:
        a = slice(int(off[e]), int(off[e + 1]))
        W = ref.dequant(q[e], s[e])
        ref.check(y[a], *ref.forward(x[a], W), False)
        ref.check(dx[a], *ref.backward(dy[a], W), False)


@pytest.mark.parametrize("off", [[0, 31], [0, 18, 32], [0, 0, 32], [2, 24, 24]])
@pytest.mark.parametrize("long", [2064, 16384])
def test_few_rows_of_few_experts_on_shared_tiles(off, long):
    # one or two experts with more than 16 rows, few columns and a long sum: a cluster shares each tile
    E, M, short = len(off) - 1, off[-1], 96
    rng = np.random.default_rng([M, E, long])
    offd = dev(np.array(off, np.int32))
    rows_of = [(e, slice(off[e], off[e + 1])) for e in range(E) if off[e + 1] > off[e]]
    q, s = layer(rng, short, long, E)
    q2, s2 = layer(rng, short, long, E)
    x = rand(rng, M, long)
    y = f32(sq.grouped_fwd_fp8(weight(q, s), dev(x, BF), offd))
    h = f32(sq.grouped_gated_fwd_fp8(weight(q, s), weight(q2, s2), dev(x, BF), offd))
    for e, a in rows_of:
        W, W2 = ref.dequant(q[e], s[e]), ref.dequant(q2[e], s2[e])
        ref.check(y[a], *ref.forward(x[a], W), False)
        ref.check(h[a], *ref.gated_forward(x[a], W, W2, "silu")[0], False)
    q, s = layer(rng, long, short, E)
    q2, s2 = layer(rng, long, short, E)
    dy, g, u = rand(rng, M, long), rand(rng, M, long), rand(rng, M, long)
    dx = f32(sq.grouped_bwd_dx_fp8(weight(q, s), dev(dy, BF), offd))
    dx2 = f32(sq.grouped_gated_bwd_dx_fp8(weight(q, s), weight(q2, s2), dev(dy, BF), dev(g, BF), dev(u, BF), offd))
    for e, a in rows_of:
        W, W2 = ref.dequant(q[e], s[e]), ref.dequant(q2[e], s2[e])
        ref.check(dx[a], *ref.backward(dy[a], W), False)
        ref.check(dx2[a], *ref.gated_backward(dy[a], g[a], u[a], W, W2, "silu"), False)


def test_device_checks(monkeypatch):
    w = weight(*layer(np.random.default_rng(0), 128, 256))
    W, x, dy = torch.zeros(128, 256, device="cuda"), torch.zeros(4, 256, dtype=BF, device="cuda"), torch.zeros(40, 128, dtype=BF, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: 1)
        for f in (lambda: sq.build_fp8(W), lambda: sq.linear_fwd_fp8(w, x), lambda: sq.linear_bwd_dx_fp8(w, dy, ws=ws),
                  lambda: sq.gated_fwd_fp8(w, w, x, save=True)):
            with pytest.raises(ValueError, match="current device"):
                f()
    with pytest.raises(ValueError, match="ws is on cpu"):
        sq.linear_bwd_dx_fp8(w, dy, ws=ws.cpu())
    w.scales = w.scales.cpu()
    with pytest.raises(ValueError, match="scales is on cpu"):
        sq.linear_fwd_fp8(w, x)


@pytest.mark.parametrize("M,off", [(5, None), (8, None), (9, None), (16, None), (17, None), (32, None), (33, None), (16, [0, 16]), (17, [0, 17]), (32, [0, 32]),
                                   (33, [1, 33]), (16, [0, 0, 16, 16]), (17, [0, 17, 17, 17]),
                                   (32, [0, 1, 31, 32]), (33, [0, 33, 33, 33])])
def test_rows_around_the_border_of_one_kernel(M, off):
    """The most rows that the product rounds itself and one more, all of one expert among them; tiles that end
    inside a block, a second weight."""
    E = None if off is None else len(off) - 1
    N, K = 336, 1168
    rng = np.random.default_rng([M, E or 0])
    p, r = layer(rng, N, K, E), layer(rng, N, K, E)
    w, w2 = weight(*p), weight(*r)
    x, dy, g, u = rand(rng, M, K), rand(rng, M, N), rand(rng, M, N), rand(rng, M, N)
    a = [dev(v, BF) for v in (x, dy, g, u)]
    if E is None:
        got = [sq.linear_fwd_fp8(w, a[0]), sq.linear_bwd_dx_fp8(w, a[1]), *sq.gated_fwd_fp8(w, w2, a[0], act="gelu", save=True),
               sq.gated_bwd_dx_fp8(w, w2, *a[1:], act="gelu")]
    else:
        o = dev(np.array(off, np.int32))
        got = [sq.grouped_fwd_fp8(w, a[0], o), sq.grouped_bwd_dx_fp8(w, a[1], o),
               *sq.grouped_gated_fwd_fp8(w, w2, a[0], o, act="gelu", save=True),
               sq.grouped_gated_bwd_dx_fp8(w, w2, *a[1:], o, act="gelu")]
    for e in range(E or 1):
        s = slice(None) if E is None else slice(off[e], off[e + 1])
        if E is not None and off[e] == off[e + 1]:
            continue
        W, W2 = (ref.dequant(*v) if E is None else ref.dequant(v[0][e], v[1][e]) for v in (p, r))
        want = [ref.forward(x[s], W), ref.backward(dy[s], W), *ref.gated_forward(x[s], W, W2, "gelu"),
                ref.gated_backward(dy[s], g[s], u[s], W, W2, "gelu")]
        for i, (y, v) in enumerate(zip(got, want)):
            ref.check(f32(y[s]), *v, i in (3, 4))
