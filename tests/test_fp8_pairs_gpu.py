"""The block-scaled products at the sizes that CTA pairs, tiles of 256 columns (whose two accumulators share some) and
several rounds of tiles are used for, dense and grouped, every element against the float64 reference of fp8ref.py.

The weights are made on the GPU and the reference's two products of each call are formed there (in float64 as well);
its roundings, activations and bounds are fp8ref.py's."""
import os
import re
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


@pytest.fixture(autouse=True)
def products_on_the_gpu(monkeypatch):
    def product(r, W, doubt=None):
        on = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        r, W = on(r), W.double()
        bound = ref.nblocks(r.shape[1]) * ref.B / 32 * 2 * ref.U23 * (r.abs() @ W.abs().T)
        if doubt is not None:
            bound += on(doubt) @ W.abs().T
        return (r @ W.T).cpu().numpy(), bound.cpu().numpy()

    monkeypatch.setattr(ref, "product", product)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def layer(seed, N, K, E=None):
    """A layer whose sums over K are about 1: its handle."""
    lead, g = (() if E is None else (E,)), gen(seed)
    q = torch.randn(*lead, N, K, generator=g, device="cuda").mul_(90).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s = torch.randint(-2, 3, (*lead, ref.nblocks(N), ref.nblocks(K)), generator=g, device="cuda")
    s = (s + (127 - round(np.log2(np.sqrt(K) * 90)))).to(torch.uint8).view(torch.float8_e8m0fnu)
    if E is None:
        return sq.Weight(sq.SQ_FMT_FP8_BLOCK, N, K, q, s)
    return sq.GroupedWeight(E, N, K, q, s, fmt=sq.SQ_FMT_FP8_BLOCK)


def values(w):
    """W in float64 (on the GPU)."""
    s = torch.exp2(w.scales.view(torch.uint8).double() - 127)
    s = s.repeat_interleave(128, 0)[:w.N].repeat_interleave(128, 1)[:, :w.K]
    return w.codes.double() * s


def rows(seed, M, width, size=1.0):
    x = torch.randn(M, width, generator=gen(seed), device="cuda") * size
    x[:, ::97] *= 15
    return x.to(BF)


def f32(t):
    return t.float().cpu().numpy()


def status(ws):
    try:
        sq.sq_check_device_status(ws)
    except sq.SqError as e:
        return e.status
    return sq.SQ_OK


def run(op, weights, ops, off=None, act="silu", bf16=False):
    """The outputs of a call on a workspace of its own, whose status is read; all rows of it written."""
    f = getattr(sq, ("grouped_" if off is not None else "" if op.startswith("gated") else "linear_") + op + "_fp8")
    w, M = weights[0], ops[0].shape[0]
    code = getattr(sq, "SQ_OP_" + f.__name__.upper())
    n = (sq.sq_workspace_bytes(code, M, w.N, w.K) if off is None
         else sq.sq_grouped_workspace_bytes(code, w.E, M, w.N, w.K))
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    kw = dict(act=act) if op.startswith("gated") else {}
    if op == "gated_fwd":
        kw["save"] = True
    out = f(*weights, *ops, *(() if off is None else (off,)), ws=ws, out_bf16=bf16, **kw)
    assert status(ws) == sq.SQ_OK
    return out if isinstance(out, tuple) else (out,)


def wanted(op, W, ops, act):
    """[(value, bound)] of the outputs."""
    v = [f32(o) for o in ops]
    if op == "fwd":
        return [ref.forward(v[0], W[0])]
    if op == "bwd":
        return [ref.backward(v[0], W[0])]
    return ref.gated_forward(v[0], *W, act) if op == "gated_fwd" else [ref.gated_backward(*v, *W, act)]


def operands(op, M, N, K):
    if not op.endswith("bwd_dx"):
        return [rows(M, M, K)]
    return [rows(M + i, M, N, size) for i, size in enumerate((1e-2, 1.5, 1.0)[:3 if op.startswith("gated") else 1])]


# Two to five rounds of tiles of pairs, or just less than one; sums that bring buffers of scales and stages round
# again; last row tiles of 1 to 128 rows (the second CTA of the pair has none) and of more; odd widths.  Then one row
# tile and many columns, more tiles than CTAs for few rows, and (the last line) one-CTA tiles wider than 128 columns.
DENSE = [("fwd", 2305, 8192, 4624), ("fwd", 2100, 4096, 2064), ("fwd", 777, 4240, 2832), ("fwd", 200, 9008, 2064),
         ("bwd_dx", 2305, 4624, 8192), ("bwd_dx", 2100, 2064, 8208), ("bwd_dx", 1300, 2064, 2832),
         ("bwd_dx", 140, 2064, 30000),
         ("gated_fwd", 1854, 3376, 4112), ("gated_fwd", 2100, 4096, 2064), ("gated_fwd", 250, 9232, 1040),
         ("gated_fwd", 8, 16384, 1552),
         ("gated_bwd_dx", 2100, 2064, 4096), ("gated_bwd_dx", 1290, 3600, 4112), ("gated_bwd_dx", 300, 1040, 25616),
         ("fwd", 353, 6384, 992), ("bwd_dx", 798, 3296, 4992), ("gated_fwd", 278, 8624, 2176), ("gated_bwd_dx", 318, 3168, 10784)]


@pytest.mark.parametrize("op,M,N,K", DENSE)
def test_dense(op, M, N, K):
    two, act, bf16 = op.startswith("gated"), "gelu" if N % 32 else "silu", M % 2 == 1
    ws = [layer(N + i, N, K) for i in range(2 if two else 1)]
    ops = operands(op, M, N, K)
    out = run(op, ws, ops, act=act, bf16=bf16)
    for i, (got, (v, bound)) in enumerate(zip(out, wanted(op.removesuffix("_dx"), [values(w) for w in ws], ops, act))):
        ref.check(f32(got), v, bound, bf16 or i > 0)
    again = run(op, ws, ops, act=act, bf16=bf16)
    for a, b in zip(out, again):
        assert torch.equal(a, b)


# Experts of 512 rows and more on average take pairs: tiles of 1, 97, 128, 129, 225 and 256 rows, none, rows of no
# expert in front and behind; one expert.  Then 20 experts on one-CTA tiles of up to 256 columns, two and a half rounds.
GROUPS = [([17, 18, 147, 1647], 1700, 3600, 2064), ([0, 97, 97, 322, 578, 2078, 2206, 4196], 4200, 2064, 2832),
          ([3, 690], 700, 2064, 5136), ([100 + 125 * e + (7 * e * e) % 61 for e in range(21)], 2700, 2064, 2832)]


@pytest.mark.parametrize("off,M,N,K", GROUPS)
@pytest.mark.parametrize("op", ["fwd", "bwd_dx", "gated_fwd", "gated_bwd_dx"])
def test_grouped(op, off, M, N, K):
    E, two, bf16 = len(off) - 1, op.startswith("gated"), op == "fwd"
    ws = [layer(N + i, N, K, E) for i in range(2 if two else 1)]
    ops = operands(op, M, N, K)
    for o in ops:                                            # what must not be looked at
        o[:off[0]] = float("nan")
        o[off[-1]:] = float("inf")
    out = run(op, ws, ops, torch.tensor(off, dtype=torch.int32, device="cuda"), bf16=bf16)
    for o in out:
        assert not o[:off[0]].any() and not o[off[-1]:].any()
    for e in range(E):
        s = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        want = wanted(op.removesuffix("_dx"), [values(w.expert(e)) for w in ws], [o[s] for o in ops], "silu")
        for i, (got, (v, bound)) in enumerate(zip(out, want)):
            ref.check(f32(got[s]), v, bound, bf16 or i > 0)


def test_these_sizes_run_on_pairs():
    """The kernels that the cases above are there for (the first template argument is the CTAs of a tile, the second
    forward, gated forward or gradient): what the host picks may change, and must not leave them untested."""
    jobs = []
    for op, M, N, K in DENSE:
        ws = [layer(1, N, K) for _ in range(2 if op.startswith("gated") else 1)]
        jobs.append(lambda op=op, ws=ws, ops=operands(op, M, N, K): run(op, ws, ops))
    for off, M, N, K in GROUPS[:2]:
        w = layer(1, N, K, len(off) - 1)
        jobs.append(lambda w=w, x=rows(1, M, K), o=torch.tensor(off, dtype=torch.int32, device="cuda"): run("fwd", [w], [x], o))
    jobs[0]()
    names = []
    for job in jobs:
        torch.cuda.synchronize()
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
            job()
            torch.cuda.synchronize()
        names.append({re.sub(r"\((int|bool)\)| ", "", e.name).replace("false", "0").replace("true", "1").split("(")[0]
                      for e in p.events() if "sq_fp8_kernel" in e.name})
    if not any(names):
        pytest.skip("the profiler records no kernels here")
    flat = [n for s in names for n in s]
    for want in ("<2,0,0", "<2,1,0", "<2,2,0"):
        assert sum(want in n for n in flat) >= 3, (want, flat)
    assert all("<2,0,0" in n for s in names[-2:] for n in s), names[-2:]


DEBUG = r'''
import sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import torch
import bit_quantized_frozen_b200 as sq
import test_fp8_pairs_gpu as t
assert sq.sq_debug_checks() == int(sys.argv[2])
out = []
for op in ("fwd", "bwd_dx", "gated_fwd", "gated_bwd_dx"):
    M, N, K = 1300, 2064, 2832
    ws = [t.layer(N + i, N, K) for i in range(2 if "gated" in op else 1)]
    out += t.run(op, ws, t.operands(op, M, N, K))
    off, M = t.GROUPS[0][:2]
    ws = [t.layer(N + i, N, K, len(off) - 1) for i in range(2 if "gated" in op else 1)]
    out += t.run(op, ws, t.operands(op, M, N, K), torch.tensor(off, dtype=torch.int32, device="cuda"))
torch.save([o.cpu() for o in out], sys.argv[3])
'''


def test_debug_library_gives_the_same_bits(tmp_path):
    """No index check of the debug library fails (run() reads each call's status), and its results are the same."""
    from bit_quantized_frozen_b200 import build
    got = []
    for flag, lib in ((0, build.LIB), (1, build.LIB_DEBUG)):
        path = str(tmp_path / f"{flag}.pt")
        r = subprocess.run([sys.executable, "-c", DEBUG, ROOT, str(flag), path], capture_output=True, text=True, timeout=900,
                           env=dict(os.environ, SQ_LIBSQ_PATH=lib))
        assert r.returncode == 0, r.stderr[-2000:]
        got.append(torch.load(path))
    assert len(got[0]) == len(got[1]) == 12
    for a, b in zip(*got):
        assert torch.equal(a, b)
