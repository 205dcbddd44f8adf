"""Calls of the 8-bit products as programs make them: on streams of their own, several at once, in
captured graphs that fork and join, at the ends of the ranges."""
import numpy as np
import pytest
import torch

import bit_quantized_frozen_b200 as sq
import w8a8ref as ref

pytestmark = pytest.mark.gpu


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def weight(L):
    b = lambda a: None if a is None else dev(a, torch.bfloat16)  # noqa: E731
    Q, sw, up, down = L
    if Q.ndim == 3:
        return sq.GroupedWeight(*Q.shape, dev(Q), dev(sw), b(up), b(down))
    return sq.Weight(sq.SQ_FMT_INT8_ROW, *Q.shape, dev(Q), dev(sw), None, b(up), b(down))


def f32(t):
    return t.float().cpu().numpy()


def test_build_on_another_stream_owns_its_memory():
    """Memory that the current stream has freed with a write to it still queued is not taken for the
    experts' codes, which another stream writes at once."""
    R = torch.randn(2, 512, 1024, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 0.02
    want = sq.build_int8_grouped(R)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    junk = torch.empty(2, 512, 1024, dtype=torch.int8, device="cuda")
    torch.cuda._sleep(200_000_000)
    junk.fill_(99)
    del junk
    got = sq.build_int8_grouped(R, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)


@pytest.mark.parametrize("M", [3, 90, 700])
def test_a_graph_that_forks_and_joins(M):
    """Forward and gradient of two layers on two branches of one capture, with the check for finite
    values, joined and followed by a third call that reads both."""
    rng = np.random.default_rng(M)
    N, K = 512, 768
    A, B, C = (ref.layer(rng, N, K) for _ in range(3))
    a, b, c = weight(A), weight(B), weight(C)
    x = dev(ref.bf16(rng.standard_normal((M, K)).astype(np.float32)), torch.bfloat16)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        other.wait_stream(main)
        y = sq.linear_fwd_w8a8(a, x, flags=sq.SQ_CHECK_FINITE, out_bf16=True)
        with torch.cuda.stream(other):
            z = sq.linear_fwd_w8a8(b, x, out_bf16=True)
            dz = sq.linear_bwd_dx_w8a8(b, z, flags=sq.SQ_CHECK_FINITE)
        main.wait_stream(other)
        s = y + z
        ds = sq.linear_bwd_dx_w8a8(c, s)
    for k in range(3):
        v = ref.bf16(rng.standard_normal((M, K)).astype(np.float32))
        x.copy_(dev(v, torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        ref.check(f32(y), *ref.forward(v, *A, bf16_out=True), True)
        ref.check(f32(z), *ref.forward(v, *B, bf16_out=True), True)
        ref.check(f32(dz), *ref.backward(f32(z), *B), False)
        ref.check(f32(ds), *ref.backward(f32(s), *C), False)


def test_many_calls_at_once():
    """Dense and grouped calls of different sizes in flight on four streams: each gives the bits it
    gives alone."""
    rng = np.random.default_rng(7)
    E, N, K = 5, 640, 1024
    w = weight(ref.layer(rng, N, K, E=E))
    jobs = []
    for M in (1, 12, 40, 100, 333):
        x = dev(rng.standard_normal((M, K)).astype(np.float32), torch.bfloat16)
        dy = dev(rng.standard_normal((M, N)).astype(np.float32), torch.bfloat16)
        off = dev(np.sort(rng.integers(0, M + 1, E + 1)).astype(np.int32))
        jobs += [lambda s, x=x: sq.linear_fwd_w8a8(w.expert(3), x, stream=s),
                 lambda s, dy=dy: sq.linear_bwd_dx_w8a8(w.expert(2), dy, out_bf16=True, stream=s),
                 lambda s, x=x, off=off: sq.grouped_fwd_w8a8(w, x, off, out_bf16=True, stream=s),
                 lambda s, dy=dy, off=off: sq.grouped_bwd_dx_w8a8(w, dy, off, stream=s)]
    alone = [j(None) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [(i, jobs[i](streams[(k + i) % 4])) for k in range(4) for i in rng.permutation(len(jobs))]
    torch.cuda.synchronize()
    for i, y in got:
        assert torch.equal(y, alone[i]), i


@pytest.mark.parametrize("M,N,K", [(1, 1 << 20, 256), (2, 128, 16384), (70, 131072, 256), (1 << 19, 128, 256)])
def test_ends_of_the_ranges(M, N, K):
    """The widest layer, the longest rows, the longest sums of the gradient, very many rows; rows and
    channels at both ends and in between are compared."""
    rng = np.random.default_rng(M + K)
    Q, sw, up, down = ref.layer(rng, N, K)
    w = weight((Q, sw, up, down))
    x = ref.bf16(rng.standard_normal((M, K)).astype(np.float32))
    m = np.unique(np.r_[0:min(M, 40), M // 2:min(M, M // 2 + 40), max(0, M - 40):M])
    n = np.unique(np.r_[0:min(N, 300), N // 2:min(N, N // 2 + 300), max(0, N - 300):N])
    y = sq.linear_fwd_w8a8(w, dev(x, torch.bfloat16))
    ref.check(f32(y[dev(m)][:, dev(n)]), *ref.forward(x[m], Q[n], sw[n], up[n], down), False)
    if N <= 131072:
        dy = ref.bf16(rng.standard_normal((M, N)).astype(np.float32))
        dx = sq.linear_bwd_dx_w8a8(w, dev(dy, torch.bfloat16))
        ref.check(f32(dx[dev(m)]), *ref.backward(dy[m], Q, sw, up, down), False)


@pytest.mark.parametrize("E,M", [(1024, 1), (1024, 30000), (1, 1), (64, 9000)])
def test_few_and_many_rows_of_many_experts(E, M):
    """Rows on the last experts only, or spread unevenly, with rows of no expert at both ends."""
    N, K = 128, 256
    rng = np.random.default_rng(E + M)
    Q, sw, up, down = ref.layer(rng, N, K, E=E)
    w = weight((Q, sw, up, down))
    counts = np.zeros(E, int)
    if M < 10:
        counts[-1] = M
    else:
        counts = rng.multinomial(M - 20, rng.dirichlet(np.full(E, 0.3)))
    before = (M - int(counts.sum())) // 2
    off = before + np.concatenate([[0], np.cumsum(counts)])
    x, dy = (ref.bf16(rng.standard_normal((M, n)).astype(np.float32)) for n in (K, N))
    offd = dev(off.astype(np.int32))
    y, dx = f32(sq.grouped_fwd_w8a8(w, dev(x, torch.bfloat16), offd)), f32(sq.grouped_bwd_dx_w8a8(w, dev(dy, torch.bfloat16), offd))
    for v in (y, dx):
        assert not v[:off[0]].any() and not v[off[-1]:].any()
    for e in np.nonzero(counts)[0]:
        s = slice(int(off[e]), int(off[e + 1]))
        ref.check(y[s], *ref.forward(x[s], Q[e], sw[e], up[e], down[e]), False)
        ref.check(dx[s], *ref.backward(dy[s], Q[e], sw[e], up[e], down[e]), False)
