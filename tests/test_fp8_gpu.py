"""The block-scaled e4m3 products and gated projections on the GPU against the float64 reference of fp8ref.py."""
import numpy as np
import pytest
import torch

import bit_quantized_frozen_b200 as sq
import fp8ref as ref

pytestmark = pytest.mark.gpu
GUARD = 4096


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def weight(q, s):
    """The library's handle of code values (fp32) and scale bytes."""
    c, e = dev(q).to(torch.float8_e4m3fn), dev(s).view(torch.float8_e8m0fnu)
    if q.ndim == 3:
        return sq.GroupedWeight(*q.shape, c, e, fmt=sq.SQ_FMT_FP8_BLOCK)
    return sq.Weight(sq.SQ_FMT_FP8_BLOCK, *q.shape, c, e)


def rows(rng, M, width, size=1.0):
    x = rng.standard_normal((M, width)) * size
    x[:, ::97] *= 15
    return ref.bf16(x.astype(np.float32))


def guarded(nbytes):
    """A byte buffer with GUARD bytes behind it, all 0xFF."""
    return torch.full((nbytes + GUARD,), 0xFF, dtype=torch.uint8, device="cuda")


class Out:
    def __init__(self, M, width, dtype, fill=None):
        self.n = M * width * dtype.itemsize
        self.buf = guarded(self.n)
        self.t = self.buf[:self.n].view(dtype).view(M, width)
        if fill is not None:
            self.t.fill_(fill)

    def check(self):
        assert bool((self.buf[self.n:] == 0xFF).all()), "written behind the output"


def call(fn, weights, operands, offsets=None, act="silu", bf16=False, flags=0, save=False, fill=None):
    """One raw call on poisoned, guarded buffers; the output, or (h, g, u)."""
    back, two, w, M = "bwd" in fn, "gated" in fn, weights[0], operands[0].shape[0]
    width = w.K if back else w.N
    outs = [Out(M, width, torch.bfloat16 if bf16 else torch.float32, fill)]
    if save:
        outs += [Out(M, width, torch.bfloat16, fill) for _ in range(2)]
    op = getattr(sq, "SQ_OP_" + fn[3:].upper())
    n = sq.sq_grouped_workspace_bytes(op, w.E, M, w.N, w.K) if offsets is not None else sq.sq_workspace_bytes(op, M, w.N, w.K)
    n = max(n, 256)
    ws = guarded(n)
    kw = dict(act=act) if two else {}
    getattr(sq, fn)(*weights, *operands, *(() if offsets is None else (offsets,)), *(o.t for o in outs),
                    flags=flags | (sq.SQ_OUT_BF16 if bf16 else 0), ws=ws[:n], **kw)
    torch.cuda.synchronize()
    for o in outs:
        o.check()
    assert bool((ws[n:] == 0xFF).all()), "written behind the workspace"
    call.ws = ws[:n]
    return tuple(o.t for o in outs) if save else outs[0].t


def status():
    try:
        sq.sq_check_device_status(call.ws)
    except sq.SqError as e:
        return e.status
    return sq.SQ_OK


def host(t):
    return t.float().cpu().numpy()


# one token, one block, widths that end inside a block and a scale word, tiles that end inside a pair
SHAPES = [(1, 128, 128), (1, 16, 16), (3, 48, 144), (17, 272, 528), (32, 640, 1280), (33, 2064, 400), (128, 128, 2048),
          (129, 256, 512), (200, 400, 1040), (257, 1296, 656), (300, 144, 4112), (600, 2832, 176)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("bf16", [False, True])
def test_forward(M, N, K, bf16):
    rng = np.random.default_rng([M, N, K])
    q, s = ref.layer(rng, N, K)
    x = rows(rng, M, K)
    y = call("sq_linear_fwd_fp8", (weight(q, s),), (dev(x, torch.bfloat16),), bf16=bf16)
    ref.check(host(y), *ref.forward(x, ref.dequant(q, s)), bf16)
    assert status() == sq.SQ_OK


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("bf16", [False, True])
def test_backward(M, N, K, bf16):
    rng = np.random.default_rng([M, N, K, 1])
    q, s = ref.layer(rng, N, K)
    dy = rows(rng, M, N, 1e-3)
    dx = call("sq_linear_bwd_dx_fp8", (weight(q, s),), (dev(dy, torch.bfloat16),), bf16=bf16)
    ref.check(host(dx), *ref.backward(dy, ref.dequant(q, s)), bf16)
    assert status() == sq.SQ_OK


def pair(rng, N, K, E=None):
    (qg, sg), (qu, su) = ref.layer(rng, N, K, E), ref.layer(rng, N, K, E)
    # sums of about 1, where the activations bend
    top = np.uint8(round(np.log2(np.sqrt(K) * 90)))
    return (qg, sg - 113 + 127 - top), (qu, su - 113 + 127 - top)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("bf16,save", [(False, True), (True, False)])
def test_gated_forward(M, N, K, kind, bf16, save):
    rng = np.random.default_rng([M, N, K, 2])
    (qg, sg), (qu, su) = pair(rng, N, K)
    x = rows(rng, M, K)
    out = call("sq_gated_fwd_fp8", (weight(qg, sg), weight(qu, su)), (dev(x, torch.bfloat16),), act=kind, bf16=bf16,
               save=save)
    want = ref.gated_forward(x, ref.dequant(qg, sg), ref.dequant(qu, su), kind)
    for got, (v, bound), half in zip(out if save else (out,), want, (bf16, True, True)):
        ref.check(host(got), v, bound, half)
    assert status() == sq.SQ_OK


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("bf16", [False, True])
def test_gated_backward(M, N, K, kind, bf16):
    rng = np.random.default_rng([M, N, K, 3])
    (qg, sg), (qu, su) = pair(rng, N, K)
    dh, g, u = rows(rng, M, N, 1e-2), ref.bf16(rng.standard_normal((M, N)).astype(np.float32) * 2), rows(rng, M, N)
    dx = call("sq_gated_bwd_dx_fp8", (weight(qg, sg), weight(qu, su)), [dev(v, torch.bfloat16) for v in (dh, g, u)],
              act=kind, bf16=bf16)
    ref.check(host(dx), *ref.gated_backward(dh, g, u, ref.dequant(qg, sg), ref.dequant(qu, su), kind), bf16)
    assert status() == sq.SQ_OK


# offsets: no rows, one row, more than a tile; rows of no expert before and behind; one expert
GROUPS = [([0, 0, 1, 1, 40, 75], 80, 272, 144), ([3, 7, 7, 140, 141], 150, 400, 528), ([0, 300], 300, 144, 640),
          ([5, 5, 5, 5], 9, 128, 128), ([0, 700, 1000, 1000, 1300], 1300, 528, 272),
          ([2, 130, 387, 388, 900], 903, 256, 400), (list(range(0, 65)), 64, 128, 256)]


def expert_rows(off):
    return [(e, off[e], off[e + 1]) for e in range(len(off) - 1) if off[e + 1] > off[e]]


@pytest.mark.parametrize("off,M,N,K", GROUPS)
@pytest.mark.parametrize("fn", ["sq_grouped_fwd_fp8", "sq_grouped_bwd_dx_fp8", "sq_grouped_gated_fwd_fp8",
                                "sq_grouped_gated_bwd_dx_fp8"])
@pytest.mark.parametrize("zero", [False, True])
def test_grouped(off, M, N, K, fn, zero):
    rng = np.random.default_rng([M, N, K, len(fn)])
    E, back, two = len(off) - 1, "bwd" in fn, "gated" in fn
    pairs = pair(rng, N, K, E)[: 2 if two else 1]
    ops = [rows(rng, M, N if back else K, 1e-2 if back else 1.0)]
    if two and back:
        ops += [rows(rng, M, N), rows(rng, M, N)]
    # rows of no expert hold what must not be looked at
    for o in ops:
        o[:off[0]] = np.nan
        o[off[-1]:] = np.inf
    outside = np.ones(M, bool)
    outside[off[0]:off[-1]] = False
    out = call(fn, [weight(*p) for p in pairs], [dev(o, torch.bfloat16) for o in ops],
               dev(np.array(off, np.int32)), bf16=two, save=two and not back, fill=7.0,
               flags=sq.SQ_CHECK_FINITE | (sq.SQ_ZERO_UNGROUPED if zero else 0))
    outs = [host(o) for o in (out if isinstance(out, tuple) else (out,))]
    for e, lo, hi in expert_rows(off):
        W = [ref.dequant(q[e], s[e]) for q, s in pairs]
        v = [o[lo:hi] for o in ops]
        if not two:
            want = [(ref.backward if back else ref.forward)(v[0], W[0])]
        else:
            want = [ref.gated_backward(*v, *W, "silu")] if back else ref.gated_forward(v[0], *W, "silu")
        for got, (y, bound) in zip(outs, want):
            ref.check(got[lo:hi], y, bound, two)
    for got in outs:
        assert (got[outside] == (0.0 if zero else 7.0)).all()
    assert status() == sq.SQ_OK
