"""The block-scaled e4m3 products on the host: refusals of the C calls and of the binding, workspace sizes,
and the reference that the GPU tests compare with (against torch's own conversions)."""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import bit_quantized_frozen_b200 as sq
import fp8ref as ref
from bit_quantized_frozen_b200 import build

NULL, SHAPE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 7
A = 0x7F0000000000            # never dereferenced: the checks come before any CUDA call
BIG = 1 << 40


def cw(fmt=sq.SQ_FMT_FP8_BLOCK, N=256, K=512, codes=A, scales=A, g_w=None, up=None, down=None):
    return ctypes.byref(sq.sq_weight(fmt, N, K, codes, scales, g_w, up, down))


def linear(fn, w=None, w2=None, x=A, M=40, y=A, flags=0, ws=A, nb=BIG, **_):
    return getattr(sq.lib(), fn)(w or cw(), x, M, y, flags, ws, nb, None)


def grouped(fn, w=None, w2=None, E=4, x=A, M=40, off=A, y=A, flags=0, ws=A, nb=BIG, **_):
    return getattr(sq.lib(), fn)(w or cw(), E, x, M, off, y, flags, ws, nb, None)


def gated(fn, w=None, w2=None, x=A, g=A, u=A, M=40, y=A, act=0, flags=0, ws=A, nb=BIG, **_):
    rows, outs = ((x, g, u), (y,)) if "bwd" in fn else ((x,), (y, g, u))
    return getattr(sq.lib(), fn)(w or cw(), w2 or w or cw(), *rows, M, act, *outs, flags, ws, nb, None)


def grouped_gated(fn, w=None, w2=None, E=4, x=A, g=A, u=A, M=40, off=A, y=A, act=0, flags=0, ws=A, nb=BIG, **_):
    rows, outs = ((x, g, u), (y,)) if "bwd" in fn else ((x,), (y, g, u))
    return getattr(sq.lib(), fn)(w or cw(), w2 or w or cw(), E, *rows, M, off, act, *outs, flags, ws, nb, None)


CALLS = [(linear, "sq_linear_fwd_fp8", sq.SQ_OP_LINEAR_FWD_FP8),
         (linear, "sq_linear_bwd_dx_fp8", sq.SQ_OP_LINEAR_BWD_DX_FP8),
         (gated, "sq_gated_fwd_fp8", sq.SQ_OP_GATED_FWD_FP8),
         (gated, "sq_gated_bwd_dx_fp8", sq.SQ_OP_GATED_BWD_DX_FP8),
         (grouped, "sq_grouped_fwd_fp8", sq.SQ_OP_GROUPED_FWD_FP8),
         (grouped, "sq_grouped_bwd_dx_fp8", sq.SQ_OP_GROUPED_BWD_DX_FP8),
         (grouped_gated, "sq_grouped_gated_fwd_fp8", sq.SQ_OP_GROUPED_GATED_FWD_FP8),
         (grouped_gated, "sq_grouped_gated_bwd_dx_fp8", sq.SQ_OP_GROUPED_GATED_BWD_DX_FP8)]


def size(fn, op, M, N, K, E=4):
    return sq.sq_grouped_workspace_bytes(op, E, M, N, K) if "grouped" in fn else sq.sq_workspace_bytes(op, M, N, K)


def few_rows(fn, e, n=256, k=512):
    """Rows that the product rounds itself: calls that need no workspace."""
    return (8 if "gated_bwd" in fn else 16) * (2 if "grouped" in fn and e > 1 or n * k <= 1 << 24 else 1)


@pytest.mark.parametrize("call,fn,op", CALLS)
def test_refusals(call, fn, op):
    two = "gated" in fn
    for name in ("x", "y", "ws"):
        assert call(fn, **{name: None}) == NULL
        assert call(fn, **{name: A + 8}) == ALIGN
    assert call(fn, ws=A + 128) == ALIGN
    for which in ("w", "w2") if two else ("w",):
        assert call(fn, **{which: cw(codes=None)}) == NULL
        assert call(fn, **{which: cw(scales=None)}) == NULL
        assert call(fn, **{which: cw(codes=A + 8)}) == ALIGN
        for fmt in (sq.SQ_FMT_INT4_G32, sq.SQ_FMT_INT4_G64, sq.SQ_FMT_NVFP4, sq.SQ_FMT_INT8_ROW, 0, 9):
            assert call(fn, **{which: cw(fmt=fmt)}) == ARG
        for extra in (dict(g_w=A), dict(up=A), dict(down=A)):
            assert call(fn, **{which: cw(**extra)}) == ARG
    for shape in (dict(N=100), dict(N=0), dict(K=300), dict(K=0), dict(K=-16), dict(N=1 << 21), dict(K=(1 << 20) + 16),
                  dict(N=1 << 20, K=1 << 20)):
        assert call(fn, w=cw(**shape)) == SHAPE
    assert call(fn, M=-1) == SHAPE and call(fn, M=(1 << 24) + 1) == SHAPE
    for flags in (sq.SQ_ACT_STATIC_SCALE, sq.SQ_RECON_RESIDUAL_ONLY, sq.SQ_RECON_TRANSPOSED, sq.SQ_IN_BF16, 0x80):
        assert call(fn, flags=flags) == ARG
    few = few_rows(fn, E)
    assert call(fn, M=few, nb=255) == WORKSPACE and call(fn, M=few + 1, ws=None) == NULL
    n = size(fn, op, 40, 256, 512)
    assert n > 40 * 256 and call(fn, nb=n - 1) == WORKSPACE and call(fn, nb=0) == WORKSPACE
    if two:
        assert call(fn, w=cw(), w2=cw(N=128)) == SHAPE and call(fn, w=cw(), w2=cw(K=256)) == SHAPE
        assert call(fn, act=2) == ARG and call(fn, act=-1) == ARG
        assert call(fn, g=None) == NULL and call(fn, u=None) == NULL       # both or neither; backward both
        if "bwd" in fn:
            assert call(fn, g=None, u=None) == NULL
        for name in ("g", "u"):
            assert call(fn, **{name: A + 8}) == ALIGN
    if "grouped" in fn:
        assert call(fn, E=0) == SHAPE and call(fn, E=1025) == SHAPE and call(fn, E=-1) == SHAPE
        assert call(fn, off=None) == NULL and call(fn, off=A + 2) == ALIGN
        assert call(fn, M=0, x=None, y=None, ws=None) == sq.SQ_OK           # nothing to do
    else:
        assert call(fn, M=0) == SHAPE and call(fn, flags=sq.SQ_ZERO_UNGROUPED) == ARG


def test_other_calls_refuse_the_format():
    L, w = sq.lib(), cw()
    assert L.sq_linear_fwd(w, A, 4, A, None, 0, A, BIG, None) == ARG
    assert L.sq_reconstruct_bf16(w, A, 0, None) == ARG
    assert L.sq_linear_bwd_dx(w, A, 4, A, A, BIG, None) == ARG
    assert L.sq_linear_fwd_w8a8(w, A, 4, A, 0, A, BIG, None) == ARG


def test_builder_refusals():
    f = sq.lib().sq_build_fp8
    assert f(None, 256, 512, 0, A, A, None) == NULL and f(A, 256, 512, 0, None, A, None) == NULL
    assert f(A, 256, 512, 0, A, None, None) == NULL
    for N, K in ((0, 512), (100, 512), (256, 300), (256, 0), (1 << 21, 512), (256, 1 << 21)):
        assert f(A, N, K, 0, A, A, None) == SHAPE
    assert f(A, 256, 512, sq.SQ_OUT_BF16, A, A, None) == ARG
    assert f(A + 8, 256, 512, 0, A, A, None) == ALIGN and f(A, 256, 512, 0, A + 8, A, None) == ALIGN
    W = torch.zeros(256, 512)
    for bad, says in ((lambda: sq.sq_build_fp8(W.double(), None, None), "float32 or bfloat16"),
                      (lambda: sq.sq_build_fp8(W, W[:10], None), "codes holds"),
                      (lambda: sq.sq_build_fp8(W, W, torch.zeros(7, dtype=torch.uint8)), "scales holds"),
                      (lambda: sq.build_fp8(W), "expected a CUDA tensor")):
        with pytest.raises(ValueError, match=says):
            bad()


def t(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def weight(E=None, N=256, K=512):
    lead = () if E is None else (E,)
    q, s = t(lead + (N, K), torch.float8_e4m3fn), t(lead + (ref.nblocks(N), ref.nblocks(K)), torch.uint8)
    s = s.view(torch.float8_e8m0fnu)
    return sq.Weight(sq.SQ_FMT_FP8_BLOCK, N, K, q, s) if E is None else sq.GroupedWeight(E, N, K, q, s,
                                                                                          fmt=sq.SQ_FMT_FP8_BLOCK)


M, N, K, E = 40, 256, 512, 3
OFF = t(E + 1, torch.int32)
WS = t(256, torch.uint8)


def raw(fn, w, x, y, flags=0, g=None, u=None, w2=None, off=OFF, **kw):
    f = getattr(sq, fn)
    ws = (w, w2 or w) if "gated" in fn else (w,)
    rows = (x, t(x.shape) if g is None else g, t(x.shape) if u is None else u) if "gated_bwd" in fn else (x,)
    return f(*ws, *rows, *((off,) if "grouped" in fn else ()), y, flags=flags, ws=WS, **kw)


@pytest.mark.parametrize("fn", [c[1] for c in CALLS])
def test_binding_refusals(fn):
    """Wrong types, shapes and short buffers are refused by name; the right ones get as far as the CUDA check."""
    e, back, two = E if "grouped" in fn else None, "bwd" in fn, "gated" in fn
    wide, out = (N, K) if back else (K, N)
    xn, yn = ("dh" if two else "dy", "dx") if back else ("x", "h" if two else "y")
    w, x, y = weight(e), t((M, wide)), t((M, out), torch.float32)
    cases = [(lambda: raw(fn, w, x, y), "expected a CUDA tensor"),
             (lambda: raw(fn, w, x.float(), y), f"{xn} must be bfloat16"),
             (lambda: raw(fn, w, t((M, wide + 256)), y), f"{xn} must be bfloat16"),
             (lambda: raw(fn, w, x.flatten(), y), f"{xn} must be bfloat16"),
             (lambda: raw(fn, w, t((wide, M)).t(), y), f"contiguous tensor for {xn}"),
             (lambda: raw(fn, w, x, y[:-1]), f"{yn} must be"),
             (lambda: raw(fn, w, x, None), f"{yn} must be a tensor"),
             (lambda: raw(fn, w, x, y, sq.SQ_OUT_BF16), f"{yn} must be torch.bfloat16"),
             (lambda: raw(fn, weight(None if e else E), x, y), "the weight is a")]
    if two:
        cases += [(lambda: raw(fn, w, x, y, w2=weight(e, N=128)), "differ in their sizes"),
                  (lambda: raw(fn, w, x, y, act="relu"), "act must be one of")]
        if back:
            cases += [(lambda: raw(fn, w, x, y, g=x.float()), "gate must be"), (lambda: raw(fn, w, x, y, u=x[1:]), "up must be")]
        else:
            f = getattr(sq, fn)
            o = (OFF,) if e else ()
            cases += [(lambda: f(w, w, x, *o, y, t((M, N - 1)), t((M, N)), ws=WS), "g must be"),
                      (lambda: f(w, w, x, *o, y, t((M, N)), t((M, N), torch.float32), ws=WS), "u must be")]
    if e:
        for o in (t(E, torch.int32), t(E + 1, torch.int64), t((1, E + 1), torch.int32)):
            cases.append((lambda o=o: raw(fn, w, x, y, off=o), "offsets must be torch.int32"))
        cases += [(lambda: raw(fn, w, x, y, off=None), "offsets must be an int32 tensor"),
                  (lambda: raw(fn, w, x, y, off=[0, 1, 2, 40]), "offsets must be an int32 tensor")]
    for bad, says in cases:
        with pytest.raises(ValueError, match=says):
            bad()
    for field, value in (("codes", t((e or 1, N, K), torch.int8)), ("codes", w.codes[..., :-1]),
                         ("scales", w.scales.view(torch.uint8)), ("scales", w.scales[..., :-1]),
                         ("fmt", sq.SQ_FMT_INT8_ROW), ("lora_up", t((N, 16)))):
        v = weight(e)
        setattr(v, field, value)
        with pytest.raises(ValueError, match="SQ_FMT_FP8_BLOCK" if field == "fmt" else "low-rank" if field == "lora_up" else field):
            raw(fn, v, x, y)


def test_workspace_covers_its_parts():
    """Header, row codes and scale words, and little more."""
    for _, fn, op in CALLS:
        back, halves = "bwd" in fn, 2 if "gated_bwd" in fn else 1
        for m, n, k in ((1, 6144, 6144), (4480, 16384, 6144), (333, 144, 16), (7, 16, 2064), (33, 256, 512), (17, 256, 512), (32, 4096, 4096), (17, 4096, 4112),
                        (16, 4096, 4112), (9, 4096, 4112), (8, 4096, 4112)):
            wide = n if back else k
            need = 256 + halves * m * (wide + 4 * ((wide + 511) // 512))
            for e in (1, 64, 1024):
                if m <= few_rows(fn, e, n, k):
                    assert size(fn, op, m, n, k, e) == 0
                else:
                    assert need <= size(fn, op, m, n, k, e) <= need + 4 * 1024
    for e in (0, 1025):
        assert sq.sq_grouped_workspace_bytes(sq.SQ_OP_GROUPED_FWD_FP8, e, 1, 256, 512) == 0
    assert sq.sq_grouped_workspace_bytes(sq.SQ_OP_LINEAR_FWD_FP8, 4, 1, 256, 512) == 0


def test_header_is_plain_c_and_exports():
    """include/sq_fp8.h compiles as strict C99, and both libraries export what it declares."""
    import re
    text = open(os.path.join(build.INCLUDE, "sq_fp8.h")).read()
    names = sorted(re.findall(r"SQ_API\s+\w+\s+(sq_\w+)\s*\(", text))
    assert names == sorted(sq.EXPORTED_FP8)
    for lib in (sq.LIB_PATH, build.build(debug_checks=True)):
        L = ctypes.CDLL(lib)
        for name in names:
            assert hasattr(L, name), name
    with tempfile.TemporaryDirectory() as d:
        src = os.path.join(d, "t.c")
        with open(src, "w") as f:
            f.write('#include "sq_fp8.h"\nint main(void) { return SQ_FMT_FP8_BLOCK == 0; }\n')
        subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I", build.INCLUDE, "-c", src, "-o",
                        os.path.join(d, "t.o")], check=True)


def test_reference_against_torch():
    """The reference's e4m3, its scales and activations against torch's conversions and autograd."""
    rng = np.random.default_rng(3)
    v = np.concatenate([np.linspace(-448, 448, 40001), rng.standard_normal(20000) * 0.02, 2.0 ** np.arange(-12, 9)])
    assert np.array_equal(ref.e4m3(v), torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy()) or \
        np.array_equal(ref.e4m3(v.astype(np.float32).astype(np.float64)),
                       torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy())
    top = np.array([0.0, 448.0, np.nextafter(448.0, 500), 447.9, 1.0, 1.75, 1.75 + 2 ** -20, 2.0 ** -130, 3e38])
    e = ref.exponent(top)
    assert list(e) == [-127, 0, 1, 0, -8, -8, -7, -127, 120]
    assert (top <= 448 * 2.0 ** e).all()
    g = torch.linspace(-12, 12, 4001, dtype=torch.float64, requires_grad=True)
    for kind, f in (("silu", torch.nn.functional.silu), ("gelu", lambda x: torch.nn.functional.gelu(x, approximate="tanh"))):
        y = f(g)
        d, = torch.autograd.grad(y.sum(), g)
        a, s, _, _ = ref.act(g.detach().numpy(), kind)
        assert np.abs(a - y.detach().numpy()).max() < 1e-12 and np.abs(s - d.numpy()).max() < 1e-12
        assert np.abs(s).max() <= 1.13
    # differences: the gated backward's gradient before its rounding
    h = 1e-6
    x = np.linspace(-5, 5, 101)
    for kind in ("silu", "gelu"):
        assert np.abs((ref.act(x + h, kind)[0] - ref.act(x - h, kind)[0]) / (2 * h) - ref.act(x, kind)[1]).max() < 1e-8


def test_reference_rounds_rows():
    r = np.zeros((4, 300))
    r[0, :3] = 448, 1, -449
    r[1, 299] = 1e-30
    r[2, 5] = np.inf
    r[3, :] = np.linspace(1, 2, 300)
    q = ref.rounded(r)
    assert q[0, 0] == 448 and q[0, 1] == 1 and q[0, 2] == -448 and (q[0, 3:] == 0).all()
    assert abs(q[1, 299] / 1e-30 - 1) < 2 ** -4 and np.isnan(q[2, :128]).all() and (q[2, 128:] == 0).all()
    assert (np.abs(q[3] / r[3] - 1) <= 2.0 ** -4).all()
    same, doubt = ref.doubtful(r, np.zeros_like(r))
    assert np.array_equal(same, q, equal_nan=True) and np.nanmax(doubt) == 0
