"""fp32 results of long sums keep fp32's precision: a CTA's accumulator takes at most 64 groups of 512 values at a
time, and the parts are joined in fp32.

Each tensor-core step of 32 products may cut 2^-22 of the magnitudes summed so far (fp8ref.py): for a part of 64 groups
64 * 16 * 2^-22 = 2^-12 of them.  The parts' join adds a rounding each, 2^-24.  Rows and weights are positive, so that the
magnitudes are the result and every cut goes the same way; in one accumulator 2^18 values lose four times the bound and
more (8192 steps)."""
import numpy as np
import pytest
import torch

import bit_quantized_frozen_b200 as sq

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def data(seed, M, L, other, n, transposed):
    """Positive rows [M, L] and a weight whose `other` channels repeat n columns of it; those columns [L, n] in float64."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.rand(M, L, generator=g, device="cuda") + 0.05).to(BF)
    q = (torch.rand(L, n, generator=g, device="cuda") * 400 + 40).to(torch.float8_e4m3fn)
    s = torch.randint(110, 113, (L // 128,), generator=g, device="cuda").to(torch.uint8)
    W = q.double() * torch.exp2(s.double() - 127).repeat_interleave(128)[:, None]
    b = q.view(torch.uint8).repeat(1, other // n)                             # [L, other]
    e = s[:, None].repeat(1, -(-other // 128))
    if not transposed:
        b, e = b.T.contiguous(), e.T.contiguous()
    return x, sq.Weight(sq.SQ_FMT_FP8_BLOCK, *b.shape, b.view(torch.float8_e4m3fn), e.view(torch.float8_e8m0fnu)), W


def rounded(x):
    b = x.double().view(x.shape[0], -1, 128)
    m, e = torch.frexp(b.amax(-1, keepdim=True))              # 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875)
    return (torch.ldexp(b, -e).float().to(torch.float8_e4m3fn).double() * torch.exp2(e.double())).view(x.shape)


def check(y, want, what):
    rel = ((y.double() - want) / want).abs().max().item()
    assert rel <= 2.0 ** -12 + 64 * 2.0 ** -24, (what, rel)


# few rows, one-CTA tiles, pairs; a cluster that shares the tiles (48 channels); over 4 parts and a few groups more
@pytest.mark.parametrize("M", [1, 5, 40, 300, 1100])
@pytest.mark.parametrize("L,other", [(1 << 18, 4096), (1 << 20, 48), ((1 << 18) + 1536, 1040)])
@pytest.mark.parametrize("back", [False, True])
def test_dense(M, L, other, back):
    x, w, W = data(M, M, L, other, 16, back)
    f = sq.linear_bwd_dx_fp8 if back else sq.linear_fwd_fp8
    y = f(w, x)
    for some in (slice(0, 64), slice(max(M - 64, 0), M)):
        want = rounded(x[some]) @ W
        for c in range(0, other, 16):
            check(y[some, c:c + 16], want, c)
    assert torch.isfinite(y).all() and (y > 0).all()
    assert torch.equal(y, f(w, x))                            # (nothing of a call is added to the next)
    # bf16 results: one rounding, 2^-8 of the value, and the sum's own error, of all steps at once
    h = f(w, x, out_bf16=True)[some, :16].double()
    assert (((h - want) / want).abs() <= 2.0 ** -8 + L / 32 * 2.0 ** -22).all()


@pytest.mark.parametrize("M", [3, 90, 1300])
@pytest.mark.parametrize("back", [False, True])
def test_grouped_and_rows_of_no_expert(M, back):
    L, other, E = 1 << 18, 144, 3
    off = [M // 3, M // 3, M // 2, M - 1]
    x, w, W = data(M + 7, M, L, other, 16, back)
    w = sq.GroupedWeight(E, w.N, w.K, w.codes.view(torch.uint8)[None].repeat(E, 1, 1).view(torch.float8_e4m3fn),
                         w.scales.view(torch.uint8)[None].repeat(E, 1, 1).view(torch.float8_e8m0fnu), fmt=sq.SQ_FMT_FP8_BLOCK)
    f = sq.grouped_bwd_dx_fp8 if back else sq.grouped_fwd_fp8
    y = f(w, x, torch.tensor(off, dtype=torch.int32, device="cuda"), flags=sq.SQ_CHECK_FINITE)
    sq.sq_check_device_status(None)
    assert not y[:off[0]].any() and not y[off[-1]:].any()
    want = rounded(x[off[0]:off[-1]]) @ W
    for c in range(0, other, 16):
        check(y[off[0]:off[-1], c:c + 16], want, c)
    # the first part's finding stays, the raw call leaves the other rows alone
    x[off[0], 5] = float("nan")
    ws = torch.zeros(max(256, sq.sq_grouped_workspace_bytes(sq.SQ_OP_GROUPED_BWD_DX_FP8 if back else sq.SQ_OP_GROUPED_FWD_FP8,
                                                            E, M, w.N, w.K)), dtype=torch.uint8, device="cuda")
    y.fill_(7.0)
    getattr(sq, "sq_" + f.__name__)(w, x, torch.tensor(off, dtype=torch.int32, device="cuda"), y, flags=sq.SQ_CHECK_FINITE, ws=ws)
    with pytest.raises(sq.SqError) as err:
        sq.sq_check_device_status(ws)
    assert err.value.status == 9
    assert (y[:off[0]] == 7).all() and (y[off[-1]:] == 7).all() and torch.isnan(y[off[0]]).all()


@pytest.mark.parametrize("M", [2, 8, 70, 600])
def test_gated_gradient(M):
    """dh act(g) and (dh u) act'(g) positive: the sum through both weights."""
    L, other = 1 << 18, 1040
    x, w, W = data(M + 3, M, L, other, 16, True)
    g, u = torch.full_like(x, 2.0), torch.full_like(x, 1.0)
    dx = sq.gated_bwd_dx_fp8(w, w, x, g, u)
    # silu(2) and silu'(2) in fp32, in the kernel's order of products
    s = torch.sigmoid(torch.tensor(2.0, dtype=torch.float64, device="cuda"))
    du, dg = x[:64].double() * (2 * s), x[:64].double() * (s + 2 * s * (1 - s))
    want = (rounded(du) + rounded(dg)) @ W
    # a value of dg or du next to a border may fall to its other side, 2^-3 of it: one in some 10^5
    rel = ((dx[:64, :16].double() - want) / want).abs().max().item()
    assert rel <= 2.0 ** -12 + 64 * 2.0 ** -24 + 2.0 ** -3 * 1e-4, rel


@pytest.mark.parametrize("M", [4, 130])
def test_in_a_graph(M):
    x, w, W = data(M, M, 1 << 18, 272, 16, False)
    sq.linear_fwd_fp8(w, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sq.linear_fwd_fp8(w, x)
    for i in range(3):
        x.mul_(2.0 if i else 1.0)
        graph.replay()
        torch.cuda.synchronize()
        check(y[:64, :16], rounded(x[:64]) @ W, i)
