"""The 8-bit integer products on the GPU against the float64 reference of w8a8ref.py."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import bit_quantized_frozen_b200 as sq
import w8a8ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GUARD = 4096


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def weight(Q, sw, up, down):
    b = lambda a: None if a is None else dev(a, torch.bfloat16)  # noqa: E731
    if Q.ndim == 3:
        return sq.GroupedWeight(Q.shape[0], Q.shape[1], Q.shape[2], dev(Q), dev(sw), b(up), b(down))
    return sq.Weight(sq.SQ_FMT_INT8_ROW, Q.shape[0], Q.shape[1], dev(Q), dev(sw), None, b(up), b(down))


def rows(rng, M, width, loud=True):
    x = rng.standard_normal((M, width)).astype(np.float32)
    if loud:
        x[:, :: 97] *= 15
    return ref.bf16(x)


def guarded(nbytes):
    """A byte buffer with GUARD bytes behind it, all 0xFF."""
    return torch.full((nbytes + GUARD,), 0xFF, dtype=torch.uint8, device="cuda")


def call(op, w, x, offsets=None, bf16=False, flags=0, fill=None):
    """One C call on poisoned, guarded buffers; returns y (fp32 or bf16 tensor)."""
    back = op.endswith("bwd")
    M, width = x.shape[0], w.K if back else w.N
    dt = torch.bfloat16 if bf16 else torch.float32
    nb = M * width * (2 if bf16 else 4)
    yb = guarded(nb)
    y = yb[:nb].view(dt).view(M, width)
    if fill is not None:
        y.copy_(fill)
    flags |= sq.SQ_OUT_BF16 if bf16 else 0
    if offsets is None:
        opn = sq.SQ_OP_LINEAR_BWD_DX_W8A8 if back else sq.SQ_OP_LINEAR_FWD_W8A8
        n = sq.sq_workspace_bytes(opn, M, w.N, w.K)
        ws = guarded(n)
        f = sq.sq_linear_bwd_dx_w8a8 if back else sq.sq_linear_fwd_w8a8
        f(w, x, y, flags=flags, ws=ws[:n])
    else:
        opn = sq.SQ_OP_GROUPED_BWD_DX_W8A8 if back else sq.SQ_OP_GROUPED_FWD_W8A8
        n = sq.sq_grouped_workspace_bytes(opn, w.E, M, w.N, w.K)
        ws = guarded(n)
        f = sq.sq_grouped_bwd_dx_w8a8 if back else sq.sq_grouped_fwd_w8a8
        f(w, x, offsets, y, flags=flags, ws=ws[:n])
    torch.cuda.synchronize()
    assert bool((yb[nb:] == 0xFF).all()), "written behind the output"
    assert bool((ws[n:] == 0xFF).all()), "written behind the workspace"
    call.ws = ws[:n]
    return y


def status():
    try:
        sq.sq_check_device_status(call.ws)
    except sq.SqError as e:
        return e.status
    return sq.SQ_OK


DENSE = [(1, 128, 256), (1, 256, 512), (2, 640, 4864), (15, 384, 1280), (16, 128, 16384), (17, 256, 768), (32, 128, 512),
         (33, 384, 2816), (64, 256, 1024), (65, 640, 256), (128, 128, 2304), (129, 384, 512), (255, 128, 1280),
         (256, 512, 256), (257, 1152, 1536), (600, 896, 3840)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lora", [True, False])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_forward(M, N, K, lora, bf16):
    rng = np.random.default_rng(M * 7 + N + K)
    L = ref.layer(rng, N, K, lora)
    x = rows(rng, M, K)
    y = call("fwd", weight(*L), dev(x, torch.bfloat16), bf16=bf16)
    ref.check(y.float().cpu().numpy(), *ref.forward(x, *L, bf16_out=bf16), bf16)
    assert status() == sq.SQ_OK


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lora", [True, False])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_backward(M, N, K, lora, bf16):
    rng = np.random.default_rng(M * 11 + N + K)
    L = ref.layer(rng, N, K, lora)
    dy = ref.bf16(rows(rng, M, N) * np.exp(rng.standard_normal((M, 1))).astype(np.float32) * 1e-3)
    dx = call("bwd", weight(*L), dev(dy, torch.bfloat16), bf16=bf16)
    ref.check(dx.float().cpu().numpy(), *ref.backward(dy, *L, bf16_out=bf16), bf16)
    assert status() == sq.SQ_OK


def test_backward_long_sum():
    """The longest sum the call takes: codes of +-127 on both sides stay exact in 32 bits."""
    M, N, K = 2, 131072, 256
    Q = np.full((N, K), 127, np.int8)
    Q[:, 1::2] = -127
    sw = np.full(N, 2.0 ** -10, np.float32)
    dy = np.full((M, N), 1.0, np.float32)
    dy[1] = -2.0
    dx = call("bwd", weight(Q, sw, None, None), dev(dy, torch.bfloat16))
    ref.check(dx.cpu().numpy(), *ref.backward(dy, Q, sw), False)


def test_codes_and_scales_bit_exact():
    """With Q the identity and s_w = 1 the forward returns s_x q_x: every code and scale is compared bit for bit."""
    K = 512
    rng = np.random.default_rng(0)
    w = weight(np.eye(K, dtype=np.int8), np.ones(K, np.float32), None, None)
    for M in (1, 20, 70, 300):
        x = ref.bf16(rows(rng, M, K) * np.exp(3 * rng.standard_normal((M, 1))).astype(np.float32))
        q, s = ref.codes(ref.rotate32(x))
        y = call("fwd", w, dev(x, torch.bfloat16)).cpu().numpy()
        assert np.array_equal(y, (q.astype(np.float32) * s[:, None]).astype(np.float32))
    # many values, so that some land next to a rounding border: 1.5 million of them
    x = rows(rng, 3000, K)
    q, s = ref.codes(ref.rotate32(x))
    y = call("fwd", w, dev(x, torch.bfloat16)).cpu().numpy()
    assert np.array_equal(y, (q.astype(np.float32) * s[:, None]).astype(np.float32))
    # backward: dx = H (s_g q_g) is compared through its exact rotation in 64 bits
    dy = rows(rng, 3000, K)
    q, s = ref.codes(dy * np.float32(1))
    dx = call("bwd", w, dev(dy, torch.bfloat16)).cpu().numpy()
    back = ref.blocks(dx.astype(np.float64), ref.hadamard()) / s.astype(np.float64)[:, None]
    assert np.array_equal(np.rint(back), q) and np.abs(back - q).max() < 1e-3


GROUPS = {
    "one_expert": ([5], 0, 0),
    "empty_first_and_last": ([0, 0, 7, 300, 0], 0, 0),
    "all_empty": ([0, 0, 0], 0, 9),
    "single_rows": ([1] * 40, 0, 0),
    "before_and_behind": ([3, 0, 20, 64], 5, 11),
    "tile_borders": ([16, 17, 15, 32, 33, 64, 128, 129, 256, 257], 1, 1),
    "one_takes_all": ([0] * 30 + [600] + [0] * 33, 0, 2),
    "many_experts": ([(7 * i) % 5 for i in range(1024)], 3, 4),
}


def groups(name):
    counts, before, behind = GROUPS[name]
    off = before + np.concatenate([[0], np.cumsum(counts)])
    return len(counts), off.astype(np.int32), int(off[-1]) + behind


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lora", [True, False])
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("op", ["fwd", "bwd"])
def test_grouped(op, name, lora, bf16):
    E, off, M = groups(name)
    N, K = (256, 512) if E < 200 else (128, 256)
    rng = np.random.default_rng(E + M)
    Q, sw, up, down = ref.layer(rng, N, K, lora, E=E)
    x = rows(rng, M, N if op == "bwd" else K)
    w = weight(Q, sw, up, down)
    f = ref.backward if op == "bwd" else ref.forward
    width = K if op == "bwd" else N
    left = torch.full((M, width), 123.0, device="cuda")
    for flags, rest in ((0, 123.0), (sq.SQ_ZERO_UNGROUPED, 0.0)):
        y = call(op, w, dev(x, torch.bfloat16), dev(off), bf16=bf16, flags=flags, fill=left)
        assert status() == sq.SQ_OK
        y = y.float().cpu().numpy()
        assert (y[:off[0]] == rest).all() and (y[off[-1]:] == rest).all()
        for e in range(E):
            a, b = off[e], off[e + 1]
            if a < b:
                r, bound = f(x[a:b], Q[e], sw[e], *((up[e], down[e]) if lora else (None, None)), bf16_out=bf16)
                ref.check(y[a:b], r, bound, bf16)


def test_no_rows():
    w = weight(*ref.layer(np.random.default_rng(0), 128, 256, E=3))
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert sq.grouped_fwd_w8a8(w, torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), off).shape == (0, 128)
    assert sq.grouped_bwd_dx_w8a8(w, torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), off).shape == (0, 256)


@pytest.mark.parametrize("op", ["fwd", "bwd"])
@pytest.mark.parametrize("off", [[0, 40, 20, 64], [-5, 10, 30, 64], [0, 10, 30, 4000], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0]])
def test_bad_offsets_are_clamped_and_reported(op, off):
    """Offsets that decrease or leave the matrix: nothing is written outside y, and the status says so."""
    rng = np.random.default_rng(3)
    w = weight(*ref.layer(rng, 256, 512, E=3))
    x = dev(rows(rng, 64, 256 if op == "bwd" else 512), torch.bfloat16)
    call(op, w, x, torch.tensor(off, dtype=torch.int32, device="cuda"))
    assert status() == 10
    call(op, w, x, torch.tensor([0, 10, 30, 64], dtype=torch.int32, device="cuda"))
    assert status() == sq.SQ_OK


@pytest.mark.parametrize("M", [6, 40, 300])
def test_special_rows(M):
    """Rows of zeros, of subnormal and of the largest values, with NaN and infinities: each its own result."""
    N, K = 256, 512
    rng = np.random.default_rng(M)
    L = ref.layer(rng, N, K)
    x = rows(rng, M, K)
    x[0] = 0
    x[1] = ref.bf16(x[1] * np.float32(2.0) ** -130)        # its scale counts as 0: only the low-rank term is left
    x[2, 7] = np.nan
    x[3, 300] = np.inf
    x[4] = ref.bf16(np.float32(3e38) * np.sign(x[4]))      # the rotation overflows fp32
    w = weight(*L)
    y = call("fwd", w, dev(x, torch.bfloat16), flags=sq.SQ_CHECK_FINITE)
    assert status() == 9
    y = y.cpu().numpy()
    assert (y[0] == 0).all() and np.isnan(y[2:5]).all()
    with np.errstate(all="ignore"):
        r, b = ref.forward(x, *L)
    # subnormal fp32 sums have an absolute error of half the smallest step (2^-149) each: K of t,
    # which sum_r |lora_up[n, r]| takes into y, and the 20 behind them
    off = 2.0 ** -149 * (K * np.abs(L[2].astype(np.float64)).sum(axis=1) + 20)
    ref.check(y[1:2], r[1:2], b[1:2] + off[None, :], False)
    ref.check(y[5:], r[5:], b[5:], False)
    call("fwd", w, dev(x[5:6], torch.bfloat16), flags=sq.SQ_CHECK_FINITE)
    assert status() == sq.SQ_OK

    dy = rows(rng, M, N)
    dy[0] = 0
    dy[2, 7] = np.nan
    dy[3, 200] = -np.inf
    dx = call("bwd", w, dev(dy, torch.bfloat16), flags=sq.SQ_CHECK_FINITE)
    assert status() == 9
    dx = dx.cpu().numpy()
    assert (dx[0] == 0).all() and np.isnan(dx[2:4]).all()
    with np.errstate(all="ignore"):
        r, b = ref.backward(dy, *L)
    keep = [i for i in range(M) if i not in (2, 3)]
    ref.check(dx[keep], r[keep], b[keep], False)


@pytest.mark.parametrize("op", ["fwd", "bwd"])
def test_same_bits_again_and_in_any_company(op):
    """Twice the same bits; a row's result without a low-rank branch is the same bits alone, among
    others and as a row of an expert (other tiles, split and unsplit sums)."""
    N, K = 384, 1280
    rng = np.random.default_rng(9)
    Q, sw, up, down = ref.layer(rng, N, K, True, E=2)
    x = dev(rows(rng, 700, N if op == "bwd" else K), torch.bfloat16)
    w2 = weight(Q, sw, up, down)
    w = w2.expert(1)
    a, b = call(op, w, x), call(op, w, x)
    assert torch.equal(a, b)
    off = torch.tensor([0, 100, 700], dtype=torch.int32, device="cuda")
    assert torch.equal(call(op, w2, x, off), call(op, w2, x, off))
    w.lora_up = w.lora_down = w2.lora_up = w2.lora_down = None
    full = call(op, w, x)
    for lo, hi in ((0, 1), (3, 19), (60, 100), (100, 164), (200, 328), (0, 300)):
        assert torch.equal(call(op, w, x[lo:hi].contiguous()), full[lo:hi])
    assert torch.equal(call(op, w2, x, off)[100:], full[100:])


def test_gradient_against_differences():
    """dx . delta against the change of <dy, x W^T> in float64, W the layer's exact weight.  The codes
    of dy are off by at most half a scale (and the clamp never acts: |r| <= 127 s (1 + 2^-22)), so
    |dx - dy W| <= (1/2 + 2^-16) s_g sum_n |(H Q)[n, k]| + the fp32 bound."""
    M, N, K = 9, 256, 512
    rng = np.random.default_rng(4)
    Q, sw, up, down = ref.layer(rng, N, K)
    H = ref.hadamard()
    HQ = ref.blocks(Q.astype(np.float64), H)
    W = up.astype(np.float64) @ down.astype(np.float64).T + sw[:, None].astype(np.float64) * HQ
    dy, x = rows(rng, M, N), rng.standard_normal((M, K))
    dx = call("bwd", weight(Q, sw, up, down), dev(dy, torch.bfloat16)).cpu().numpy().astype(np.float64)
    _, s = ref.codes(dy * sw[None, :])
    _, fp = ref.backward(dy, Q, sw, up, down)
    off = (0.5 + 2.0 ** -16) * s.astype(np.float64)[:, None] * np.abs(HQ).sum(axis=0)[None, :] + fp
    f = lambda v: (dy.astype(np.float64) * (v @ W.T)).sum()  # noqa: E731
    h = 2.0 ** -10
    for m in range(M):
        for k in (0, 1, 255, 256, 511):
            d = np.zeros((M, K))
            d[m, k] = h
            diff = (f(x + d) - f(x - d)) / (2 * h)
            assert abs(diff - dx[m, k]) <= off[m, k] * 1.0001, (m, k)


def test_streams_and_graph():
    """Two streams at once with a workspace each, and a captured call replayed on new inputs."""
    N, K, M = 640, 1024, 90
    rng = np.random.default_rng(5)
    Q, sw, up, down = ref.layer(rng, N, K)
    w = weight(Q, sw, up, down)
    xs = [rows(rng, M, K) for _ in range(2)]
    xd = [dev(x, torch.bfloat16) for x in xs]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    ys = [[], []]
    for _ in range(10):
        for i in range(2):
            ys[i].append(sq.linear_fwd_w8a8(w, xd[i], stream=st[i]))
    torch.cuda.synchronize()
    for i in range(2):
        r, b = ref.forward(xs[i], Q, sw, up, down)
        for y in ys[i]:
            assert torch.equal(y, ys[i][0])
        ref.check(ys[i][0].cpu().numpy(), r, b, False)
    # capture: forward and backward of it with their own workspaces
    x = xd[0].clone()
    fws = sq.workspace(sq.SQ_OP_LINEAR_FWD_W8A8, M, N, K)
    bws = sq.workspace(sq.SQ_OP_LINEAR_BWD_DX_W8A8, M, N, K)
    sq.linear_bwd_dx_w8a8(w, sq.linear_fwd_w8a8(w, x, ws=fws, out_bf16=True), ws=bws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = sq.linear_fwd_w8a8(w, x, ws=fws, out_bf16=True)
        dx = sq.linear_bwd_dx_w8a8(w, y, ws=bws)
    for v in (xs[1], xs[0]):
        x.copy_(dev(v, torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        r, b = ref.forward(v, Q, sw, up, down, bf16_out=True)
        ref.check(y.float().cpu().numpy(), r, b, True)
        r, b = ref.backward(y.float().cpu().numpy(), Q, sw, up, down)
        ref.check(dx.cpu().numpy(), r, b, False)


def test_experts_forward_and_back():
    """A feed-forward layer of experts as a training step uses it: two grouped products with a gate
    between, and the input gradient back through both; each product is checked on the inputs it had."""
    E, K, F = 6, 512, 768
    counts = [30, 0, 5, 100, 1, 64]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(off[-1]) + 6
    rng = np.random.default_rng(8)
    gate_up, down = ref.layer(rng, 2 * F, K, E=E), ref.layer(rng, K, F, E=E)
    w1, w2 = weight(*gate_up), weight(*down)
    offd = dev(off)
    x = dev(rows(rng, M, K), torch.bfloat16)
    h = sq.grouped_fwd_w8a8(w1, x, offd, out_bf16=True)
    hr = h.float().requires_grad_(True)
    act = torch.nn.functional.silu(hr[:, :F]) * hr[:, F:]
    a = act.detach().to(torch.bfloat16)
    y = sq.grouped_fwd_w8a8(w2, a, offd)
    dy = dev(rows(rng, M, K) * np.float32(1e-2), torch.bfloat16)
    da = sq.grouped_bwd_dx_w8a8(w2, dy, offd)
    act.backward(da)
    dh = hr.grad.to(torch.bfloat16)
    dx = sq.grouped_bwd_dx_w8a8(w1, dh, offd)
    torch.cuda.synchronize()
    f32 = lambda t: t.float().cpu().numpy()  # noqa: E731
    for t in (h, y, da, dx):
        assert (f32(t)[off[-1]:] == 0).all()
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        if s.start == s.stop:
            continue
        one = lambda L: tuple(v[e] for v in L)  # noqa: E731
        ref.check(f32(h)[s], *ref.forward(f32(x)[s], *one(gate_up), bf16_out=True), True)
        ref.check(f32(y)[s], *ref.forward(f32(a)[s], *one(down)), False)
        ref.check(f32(da)[s], *ref.backward(f32(dy)[s], *one(down)), False)
        ref.check(f32(dx)[s], *ref.backward(f32(dh)[s], *one(gate_up)), False)


def test_next_to_the_bf16_path():
    """On a built weight the integer product stays near sq_linear_fwd: the codes of x are off by at
    most half a scale, so |y8 - y| <= s_x/2 s_w sum_k |Q[n, k]| (1 + 2^-8) plus the bf16 path's own
    2e-3 of the largest |y|."""
    N, K, M = 256, 512, 50
    rng = np.random.default_rng(2)
    R = rng.standard_normal((N, K)).astype(np.float32) * 0.02
    up, down = ref.bf16(rng.standard_normal((N, 16)) * 0.1), ref.bf16(rng.standard_normal((K, 16)) * 0.1)
    w = sq.build_int8(dev(R), dev(up, torch.bfloat16), dev(down, torch.bfloat16))
    x = rows(rng, M, K)
    y = sq.linear_fwd(w, dev(x, torch.bfloat16)).cpu().numpy().astype(np.float64)
    y8 = sq.linear_fwd_w8a8(w, dev(x, torch.bfloat16)).cpu().numpy().astype(np.float64)
    _, s = ref.codes(ref.rotate32(x))
    Q, sw = w.codes.cpu().numpy().astype(np.float64), w.scales.cpu().numpy().astype(np.float64)
    off = 0.5 * s.astype(np.float64)[:, None] * (sw * np.abs(Q).sum(axis=1))[None, :] * (1 + 2.0 ** -8)
    assert (np.abs(y8 - y) <= off + 2 * 2e-3 * np.abs(y).max()).all()
    g = sq.build_int8_grouped(dev(np.stack([R, 2 * R])))
    assert torch.equal(g.expert(0).codes, w.codes) and torch.equal(g.expert(0).scales, w.scales)


CHILD = r"""
import sys, numpy as np, torch
sys.path.insert(0, sys.argv[1]); sys.path.insert(0, sys.argv[1] + "/tests")
import bit_quantized_frozen_b200 as sq, w8a8ref as ref
assert sq.sq_debug_checks() == int(sys.argv[2])
rng = np.random.default_rng(6)
out = []
Q, sw, up, down = ref.layer(rng, 384, 768, True, E=4)
d = lambda a, t=None: torch.from_numpy(a).cuda() if t is None else torch.from_numpy(a).cuda().to(t)
w = sq.GroupedWeight(4, 384, 768, d(Q), d(sw), d(up, torch.bfloat16), d(down, torch.bfloat16))
for M in (1, 30, 500):
    x = d(rng.standard_normal((M, 768)).astype(np.float32), torch.bfloat16)
    dy = d(rng.standard_normal((M, 384)).astype(np.float32), torch.bfloat16)
    off = torch.tensor([0, M // 3, M // 3, M // 2, M], dtype=torch.int32, device="cuda")
    for bf in (False, True):
        out += [sq.linear_fwd_w8a8(w.expert(2), x, out_bf16=bf), sq.linear_bwd_dx_w8a8(w.expert(2), dy, out_bf16=bf),
                sq.grouped_fwd_w8a8(w, x, off, out_bf16=bf), sq.grouped_bwd_dx_w8a8(w, dy, off, out_bf16=bf)]
torch.cuda.synchronize()
np.savez(sys.argv[3], *[t.float().cpu().numpy() for t in out])
"""


def test_debug_library_gives_the_same_bits(tmp_path):
    from bit_quantized_frozen_b200 import build
    got = []
    for i, lib in enumerate((build.LIB, build.LIB_DEBUG)):
        if not os.path.exists(lib):
            build.build(debug_checks=i == 1)
        out = str(tmp_path / f"{i}.npz")
        p = subprocess.run([sys.executable, "-c", CHILD, ROOT, str(i), out], env=dict(os.environ, SQ_LIBSQ_PATH=lib),
                           capture_output=True, text=True, timeout=600)
        assert p.returncode == 0, p.stderr
        got.append(np.load(out))
    for name in got[0].files:
        assert np.array_equal(got[0][name], got[1][name]), name


def test_offsets_past_32_bits():
    """Row codes and weight codes of more than 2^31 values: the last rows and the last expert are right."""
    N, K, M = 128, 8192, 270000
    rng = np.random.default_rng(12)
    L = ref.layer(rng, N, K)
    last = rows(rng, 70, K)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-70:] = dev(last, torch.bfloat16)
    y = sq.linear_fwd_w8a8(weight(*L), x)
    assert not y[:-70].any()
    ref.check(y[-70:].cpu().numpy(), *ref.forward(last, *L), False)
    del x, y
    E, N, K = 600, 1024, 3840
    Q, sw, up, down = ref.layer(rng, N, K)
    w = sq.GroupedWeight(E, N, K, torch.zeros(E, N, K, dtype=torch.int8, device="cuda"),
                         torch.zeros(E, N, device="cuda"),
                         torch.zeros(E, N, 16, dtype=torch.bfloat16, device="cuda"),
                         torch.zeros(E, K, 16, dtype=torch.bfloat16, device="cuda"))
    one = weight(Q, sw, up, down)
    for a, b in ((w.codes, one.codes), (w.scales, one.scales), (w.lora_up, one.lora_up), (w.lora_down, one.lora_down)):
        a[-1] = b
    off = torch.full((E + 1,), 3, dtype=torch.int32, device="cuda")
    off[0], off[-1] = 0, 13
    for f, r, width in ((sq.grouped_fwd_w8a8, ref.forward, K), (sq.grouped_bwd_dx_w8a8, ref.backward, N)):
        x = rows(rng, 13, width)
        y = f(w, dev(x, torch.bfloat16), off).cpu().numpy()
        assert not y[:3].any()
        ref.check(y[3:], *r(x[3:], Q, sw, up, down), False)


@pytest.mark.parametrize("N", [32768, 32768 + 128])
def test_backward_rows_longer_than_a_cluster(N):
    """Rows of more than 64 blocks are read twice; a half block at the end."""
    rng = np.random.default_rng(N)
    for M in (1, 37):
        L = ref.layer(rng, N, 256)
        dy = rows(rng, M, N)
        ref.check(call("bwd", weight(*L), dev(dy, torch.bfloat16)).cpu().numpy(), *ref.backward(dy, *L), False)


def test_row_views_and_one_expert():
    """x and offsets that are views into larger buffers; a grouped call with one expert is the dense call."""
    rng = np.random.default_rng(21)
    w = weight(*ref.layer(rng, 256, 768, lora=False, E=1))
    big = dev(rows(rng, 200, 768), torch.bfloat16)
    off = torch.tensor([7, 7, 0, 50], dtype=torch.int32, device="cuda")[2:]
    dense = sq.linear_fwd_w8a8(w.expert(0), big[13:63])
    assert torch.equal(sq.grouped_fwd_w8a8(w, big[13:63], off), dense)
    assert torch.equal(dense, sq.linear_fwd_w8a8(w.expert(0), big)[13:63])
    with pytest.raises(ValueError, match="contiguous"):
        sq.linear_fwd_w8a8(w.expert(0), big[::2])


def test_device_checks(monkeypatch):
    w = weight(*ref.layer(np.random.default_rng(0), 128, 256))
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="current device"):
        sq.linear_fwd_w8a8(w, x, ws=ws)
    w.codes = w.codes.cpu()
    with pytest.raises(ValueError, match="codes is on cpu"):
        sq.linear_fwd_w8a8(w, x)


FIRST = r"""
import sys, torch
sys.path.insert(0, sys.argv[1])
import bit_quantized_frozen_b200 as sq
w = sq.Weight(4, 256, 512, torch.ones(256, 512, dtype=torch.int8, device="cuda"), torch.ones(256, device="cuda"))
x = torch.ones(300, 512, dtype=torch.bfloat16, device="cuda")
dy = torch.ones(300, 256, dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y, z, dx = sq.linear_fwd_w8a8(w, x), sq.linear_fwd_w8a8(w, x[:5]), sq.linear_bwd_dx_w8a8(w, dy)
g.replay()
torch.cuda.synchronize()
assert torch.equal(y[:5], z) and torch.equal(y, sq.linear_fwd_w8a8(w, x)) and torch.equal(dx, sq.linear_bwd_dx_w8a8(w, dy))
print("ok")
"""


def test_first_call_inside_a_capture():
    """The library's first call of a process may be a captured one."""
    p = subprocess.run([sys.executable, "-c", FIRST, ROOT], capture_output=True, text=True, timeout=600)
    assert p.returncode == 0 and p.stdout.strip() == "ok", p.stderr


@pytest.mark.parametrize("op", ["fwd", "bwd"])
def test_expert_changes_between_row_groups(op):
    """More row groups than clusters: a cluster's next group is often of another expert, of one a few
    experts on, or of the same one; a last group of an expert holds 1 to 8 rows."""
    rng = np.random.default_rng(31)
    N, K, E = 640, 1024, 160
    counts = rng.integers(0, 90, E) * (rng.random(E) < 0.7)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(off[-1])
    assert sum((c + 7) // 8 for c in counts) > 2 * 148
    Q, sw, up, down = ref.layer(rng, N, K, E=E)
    x = rows(rng, M, N if op == "bwd" else K)
    y = call(op, weight(Q, sw, up, down), dev(x, torch.bfloat16), dev(off)).cpu().numpy()
    f = ref.backward if op == "bwd" else ref.forward
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a < b:
            ref.check(y[a:b], *f(x[a:b], Q[e], sw[e], up[e], down[e]), False)


def test_captured_grouped_calls_follow_the_offsets():
    """Two captured graphs that share a workspace, replayed in turn with offsets that change in between:
    what a replay computes depends on the values it finds, not on those of the capture."""
    rng = np.random.default_rng(32)
    M, N, K, E = 333, 256, 512, 6
    Q, sw, up, down = ref.layer(rng, N, K, E=E)
    w = weight(Q, sw, up, down)
    x, dy = rows(rng, M, K), rows(rng, M, N)
    xd, dyd = dev(x, torch.bfloat16), dev(dy, torch.bfloat16)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    n = max(sq.sq_grouped_workspace_bytes(o, E, M, N, K)
            for o in (sq.SQ_OP_GROUPED_FWD_W8A8, sq.SQ_OP_GROUPED_BWD_DX_W8A8))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    sq.grouped_fwd_w8a8(w, xd, offsets, ws=ws)
    sq.grouped_bwd_dx_w8a8(w, dyd, offsets, ws=ws)
    torch.cuda.synchronize()
    gf, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gf):
        y = sq.grouped_fwd_w8a8(w, xd, offsets, ws=ws)
    with torch.cuda.graph(gb):
        dx = sq.grouped_bwd_dx_w8a8(w, dyd, offsets, ws=ws)
    for off in ([0, 333, 333, 333, 333, 333, 333], [3, 3, 20, 170, 171, 300, 301], [0, 0, 0, 0, 0, 0, 1]):
        offsets.copy_(torch.tensor(off, dtype=torch.int32))
        gf.replay()
        gb.replay()
        torch.cuda.synchronize()
        for got, f, v in ((y.cpu().numpy(), ref.forward, x), (dx.cpu().numpy(), ref.backward, dy)):
            assert (got[:off[0]] == 0).all() and (got[off[-1]:] == 0).all()
            for e in range(E):
                a, b = off[e], off[e + 1]
                if a < b:
                    ref.check(got[a:b], *f(v[a:b], Q[e], sw[e], up[e], down[e]), False)
