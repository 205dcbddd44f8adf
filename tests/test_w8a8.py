"""The 8-bit integer products on the host: refusals of the C calls and of the binding, the workspace
layout, and the reference the GPU tests compare with (against definitions it does not use)."""
import ctypes

import numpy as np
import pytest
import torch

import bit_quantized_frozen_b200 as sq
import w8a8ref as ref

NULL, SHAPE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 7
A = 0x7F0000000000            # never dereferenced: the checks come before any CUDA call
BIG = 1 << 40


def cw(fmt=sq.SQ_FMT_INT8_ROW, N=256, K=512, codes=A, scales=A, up=A, down=A):
    return ctypes.byref(sq.sq_weight(fmt, N, K, codes, scales, A, up, down))


def dense(fn, w=None, x=A, M=40, y=A, flags=0, ws=A, nb=BIG):
    return getattr(sq.lib(), fn)(cw() if w is None else w, x, M, y, flags, ws, nb, None)


def grouped(fn, w=None, E=4, x=A, M=40, off=A, y=A, flags=0, ws=A, nb=BIG):
    return getattr(sq.lib(), fn)(cw() if w is None else w, E, x, M, off, y, flags, ws, nb, None)


CALLS = [(dense, "sq_linear_fwd_w8a8"), (dense, "sq_linear_bwd_dx_w8a8"), (grouped, "sq_grouped_fwd_w8a8"),
         (grouped, "sq_grouped_bwd_dx_w8a8")]


@pytest.mark.parametrize("call,fn", CALLS)
def test_refusals(call, fn):
    for name in ("x", "y", "ws"):
        assert call(fn, **{name: None}) == NULL
        assert call(fn, **{name: A + 8}) == ALIGN
    assert call(fn, ws=A + 128) == ALIGN
    assert call(fn, w=cw(codes=None)) == NULL
    assert call(fn, w=cw(scales=None)) == NULL
    assert call(fn, w=cw(up=None)) == NULL and call(fn, w=cw(down=None)) == NULL      # both or neither
    for name in ("codes", "scales", "up", "down"):
        assert call(fn, w=cw(**{name: A + 8})) == ALIGN
    for fmt in (sq.SQ_FMT_INT4_G32, sq.SQ_FMT_INT4_G64, sq.SQ_FMT_NVFP4, 0, 9):
        assert call(fn, w=cw(fmt=fmt)) == ARG
    for shape in (dict(N=100), dict(N=0), dict(K=300), dict(K=0), dict(K=16384 + 256), dict(N=1 << 21)):
        assert call(fn, w=cw(**shape)) == SHAPE
    assert call(fn, M=-1) == SHAPE and call(fn, M=(1 << 24) + 1) == SHAPE
    for flags in (sq.SQ_ACT_STATIC_SCALE, sq.SQ_RECON_RESIDUAL_ONLY, sq.SQ_RECON_TRANSPOSED, 0x40):
        assert call(fn, flags=flags) == ARG
    assert call(fn, nb=0) == WORKSPACE
    n = (sq.sq_workspace_bytes(sq.SQ_OP_LINEAR_BWD_DX_W8A8 if "bwd" in fn else sq.SQ_OP_LINEAR_FWD_W8A8, 40, 256, 512)
         if call is dense else
         sq.sq_grouped_workspace_bytes(sq.SQ_OP_GROUPED_BWD_DX_W8A8 if "bwd" in fn else sq.SQ_OP_GROUPED_FWD_W8A8,
                                       4, 40, 256, 512))
    assert n > 40 * 256 and call(fn, nb=n - 1) == WORKSPACE


def test_refusals_of_each_kind():
    for fn in ("sq_linear_fwd_w8a8", "sq_linear_bwd_dx_w8a8"):
        assert dense(fn, M=0) == SHAPE
        assert dense(fn, flags=sq.SQ_ZERO_UNGROUPED) == ARG
    # the sums of the backward run over N
    assert dense("sq_linear_bwd_dx_w8a8", w=cw(N=131072 + 128)) == SHAPE
    assert grouped("sq_grouped_bwd_dx_w8a8", w=cw(N=131072 + 128)) == SHAPE
    for fn in ("sq_grouped_fwd_w8a8", "sq_grouped_bwd_dx_w8a8"):
        assert grouped(fn, E=0) == SHAPE and grouped(fn, E=1025) == SHAPE and grouped(fn, E=-1) == SHAPE
        assert grouped(fn, off=None) == NULL and grouped(fn, off=A + 2) == ALIGN
        assert grouped(fn, M=0, x=None, y=None, ws=None) == sq.SQ_OK                  # nothing to do
    assert sq.sq_grouped_workspace_bytes(sq.SQ_OP_GROUPED_FWD_W8A8, 0, 1, 256, 512) == 0
    assert sq.sq_grouped_workspace_bytes(sq.SQ_OP_GROUPED_FWD_W8A8, 1025, 1, 256, 512) == 0
    assert sq.sq_grouped_workspace_bytes(sq.SQ_OP_LINEAR_FWD_W8A8, 4, 1, 256, 512) == 0


def t(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def weights(E=None, N=256, K=512):
    lead = () if E is None else (E,)
    parts = (t(lead + (N, K), torch.int8), t(lead + (N,), torch.float32), t(lead + (N, 16)), t(lead + (K, 16)))
    if E is None:
        return sq.Weight(sq.SQ_FMT_INT8_ROW, N, K, parts[0], parts[1], None, parts[2], parts[3])
    return sq.GroupedWeight(E, N, K, *parts)


def test_binding_refusals():
    """Wrong types, shapes and short buffers are refused by name; the right ones get as far as the CUDA check."""
    M, N, K, E = 40, 256, 512, 3
    off = t(E + 1, torch.int32)
    ws = t(256, torch.uint8)
    cases = [(lambda w, x, y, f=0: sq.sq_linear_fwd_w8a8(w, x, y, f, ws), None, K, N, "x", "y"),
             (lambda w, x, y, f=0: sq.sq_linear_bwd_dx_w8a8(w, x, y, f, ws), None, N, K, "dy", "dx"),
             (lambda w, x, y, f=0: sq.sq_grouped_fwd_w8a8(w, x, off, y, f, ws), E, K, N, "x", "y"),
             (lambda w, x, y, f=0: sq.sq_grouped_bwd_dx_w8a8(w, x, off, y, f, ws), E, N, K, "dy", "dx")]
    for call, e, wide, out, xn, yn in cases:
        w, x, y = weights(e), t((M, wide)), t((M, out), torch.float32)
        for bad, says in ((lambda: call(w, x, y), "expected a CUDA tensor"),
                          (lambda: call(w, x.float(), y), f"{xn} must be bfloat16"),
                          (lambda: call(w, t((M, wide + 256)), y), f"{xn} must be bfloat16"),
                          (lambda: call(w, x.flatten(), y), f"{xn} must be bfloat16"),
                          (lambda: call(w, x, y.flatten()[:-1]), f"{yn} holds"),
                          (lambda: call(w, x, y.view(torch.int32)), f"{yn} is torch.int32"),
                          (lambda: call(w, x, y, sq.SQ_OUT_BF16), f"{yn} is torch.float32")):
            with pytest.raises(ValueError, match=says):
                bad()
        for field in ("codes", "scales", "lora_up", "lora_down"):
            w = weights(e)
            setattr(w, field, getattr(w, field).flatten()[:-1])
            with pytest.raises(ValueError, match=f"{field} holds"):
                call(w, x, y)
        w = weights(e)
        w.fmt = sq.SQ_FMT_INT4_G32
        with pytest.raises(ValueError, match="SQ_FMT_INT8_ROW"):
            call(w, x, y)
    w, x, y = weights(E), t((M, K)), t((M, N), torch.float32)
    for o in (t(E, torch.int32), t(E + 1, torch.int64), t((1, E + 1), torch.int32)):
        with pytest.raises(ValueError, match="offsets must be int32"):
            sq.sq_grouped_fwd_w8a8(w, x, o, y, 0, ws)


def test_binding_weight_kinds():
    """A grouped call wants a GroupedWeight and an offsets tensor, a dense call a Weight."""
    x, dy, off = t((40, 512)), t((40, 256)), t(4, torch.int32)
    one, many = weights(), weights(3)
    for bad, says in ((lambda: sq.linear_fwd_w8a8(many, x), "is a GroupedWeight"),
                      (lambda: sq.linear_bwd_dx_w8a8(many, dy), "is a GroupedWeight"),
                      (lambda: sq.grouped_fwd_w8a8(one, x, off), "is a Weight"),
                      (lambda: sq.grouped_bwd_dx_w8a8(one, dy, off), "is a Weight"),
                      (lambda: sq.grouped_fwd_w8a8(many, x, None), "offsets must be an int32 tensor"),
                      (lambda: sq.grouped_bwd_dx_w8a8(many, dy, [0, 7, 7, 40]), "offsets must be an int32 tensor")):
        with pytest.raises(ValueError, match=says):
            bad()


def test_workspace_covers_its_parts():
    """Header, row codes, scales and low-rank input, and little more."""
    for op, gop, back in ((sq.SQ_OP_LINEAR_FWD_W8A8, sq.SQ_OP_GROUPED_FWD_W8A8, False),
                          (sq.SQ_OP_LINEAR_BWD_DX_W8A8, sq.SQ_OP_GROUPED_BWD_DX_W8A8, True)):
        for M, N, K in ((1, 6144, 6144), (4480, 16384, 6144), (333, 128, 256)):
            need = 256 + M * ((N if back else K) + 4 + 64)
            assert need <= sq.sq_workspace_bytes(op, M, N, K) <= need + 5 * 1024
            for E in (1, 64, 1024):
                assert sq.sq_grouped_workspace_bytes(gop, E, M, N, K) == sq.sq_workspace_bytes(op, M, N, K)


def test_header_is_plain_c_and_exports():
    """include/sq_w8a8.h compiles as strict C99 beside sq.h, and both libraries export what it declares."""
    import os
    import re
    import shutil
    import subprocess
    from bit_quantized_frozen_b200 import build
    text = open(os.path.join(build.INCLUDE, "sq_w8a8.h")).read()
    names = sorted(set(re.findall(r"^SQ_API[^;(]*?\b(sq_\w+)\s*\(", text, re.M)))
    assert names == sorted(sq.EXPORTED_W8A8)
    for lib in (sq.LIB_PATH, build.build(debug_checks=True)):
        L = ctypes.CDLL(lib)
        for n in names:
            assert hasattr(L, n), n
    if shutil.which("gcc"):
        src = '#include "sq_w8a8.h"\nint main(void) { return SQ_ZERO_UNGROUPED == 0u; }\n'
        subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", build.INCLUDE, "-x", "c",
                        "-fsyntax-only", "-"], input=src, text=True, check=True)


# ---- the reference ------------------------------------------------------------------------------

def test_reference_rotation_and_rounding():
    rng = np.random.default_rng(0)
    v = rng.integers(-64, 64, (5, 512)).astype(np.float32)        # exact in fp32 all through
    H = ref.hadamard()
    assert np.array_equal(ref.rotate32(v).astype(np.float64), ref.blocks(v.astype(np.float64), H))
    assert np.allclose(H @ H, np.eye(256), atol=0, rtol=0)
    a = (rng.standard_normal(1000) * np.exp(rng.standard_normal(1000) * 5)).astype(np.float32)
    assert np.array_equal(ref.bf16(a), torch.from_numpy(a).to(torch.bfloat16).float().numpy())


def test_reference_codes():
    r = np.array([[127.0, -127.0, 63.5, 0.5, 1.5, 2.5, -0.5, 0.0]], np.float32)
    q, s = ref.codes(r)
    assert s[0] == 1 and q[0].tolist() == [127, -127, 64, 0, 2, 2, 0, 0]          # ties to even
    q, s = ref.codes(np.zeros((1, 8), np.float32))
    assert s[0] == 0 and not q.any()
    q, s = ref.codes(np.full((1, 8), 1e-37, np.float32))
    assert s[0] == 0 and not q.any()
    for bad in (np.nan, np.inf, -np.inf):
        r[0, 3] = bad
        q, s = ref.codes(r)
        assert np.isnan(s[0]) and not q.any()


@pytest.mark.parametrize("lora", [True, False])
def test_reference_products(lora):
    """Forward and backward against the layer's weight, the codes' error bounded by half a scale; and a
    planted mistake of one code step, one swapped scale or one wrong sign is outside the bound."""
    M, N, K = 6, 128, 512
    rng = np.random.default_rng(1)
    Q, sw, up, down = ref.layer(rng, N, K, lora)
    H = ref.hadamard()
    HQ = ref.blocks(Q.astype(np.float64), H)
    W = sw[:, None].astype(np.float64) * HQ
    if lora:
        W = W + up.astype(np.float64) @ down.astype(np.float64).T
    x, dy = ref.bf16(rng.standard_normal((M, K))), ref.bf16(rng.standard_normal((M, N)))
    y, b = ref.forward(x, Q, sw, up, down)
    _, s = ref.codes(ref.rotate32(x))
    assert (np.abs(y - x @ W.T) <= 0.51 * s[:, None] * (sw * np.abs(Q.astype(np.float64)).sum(1))[None, :]).all()
    dx, bd = ref.backward(dy, Q, sw, up, down)
    _, s = ref.codes(dy * sw[None, :])
    assert (np.abs(dx - dy @ W) <= 0.51 * s[:, None] * np.abs(HQ).sum(0)[None, :]).all()
    ref.check(y.astype(np.float32), y, b, False)
    ref.check(ref.bf16(y), y, b, True)
    Q2 = Q.copy()
    Q2[5, 7] += 1 if Q2[5, 7] < 0 else -1
    for wrong in (lambda: ref.forward(x, Q2, sw, up, down)[0], lambda: ref.forward(x, Q, np.roll(sw, 1), up, down)[0],
                  lambda: ref.forward(-x, Q, sw, up, down)[0]):
        with pytest.raises(AssertionError):
            ref.check(wrong(), y, b, False)
    with pytest.raises(AssertionError):
        ref.check(ref.backward(dy, Q2, sw, up, down)[0], dx, bd, False)
