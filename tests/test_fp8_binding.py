"""The binding of the block-scaled products on the host, beside test_fp8.py."""
import os
import subprocess
import sys

import pytest
import torch

import bit_quantized_frozen_b200 as sq
from test_fp8 import OFF, E, K, M, N, raw, t, weight

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

OLD_TORCH = r'''
import sys
import torch
for name in sys.argv[2:]:
    delattr(torch, name)
sys.path.insert(0, sys.argv[1])
import bit_quantized_frozen_b200 as sq
assert sq.sq_workspace_bytes(sq.SQ_OP_LINEAR_FWD_INT4, 4, 256, 512) > 0
x, q = torch.zeros(4, 512, dtype=torch.bfloat16), torch.zeros(256, 512, dtype=torch.uint8)
w = sq.Weight(sq.SQ_FMT_FP8_BLOCK, 256, 512, q, q[:2, :4])
e = sq.GroupedWeight(1, 256, 512, q[None], q[None, :2, :4], fmt=sq.SQ_FMT_FP8_BLOCK)
off = torch.tensor([0, 4], dtype=torch.int32)
for f in (lambda: sq.build_fp8(x[:, :256].float()), lambda: sq.build_fp8_grouped(x[None].float()),
          lambda: sq.linear_fwd_fp8(w, x), lambda: sq.grouped_fwd_fp8(e, x, off), lambda: sq.gated_fwd_fp8(w, w, x, save=True)):
    try:
        f()
    except RuntimeError as err:
        assert "needs a PyTorch with" in str(err), err
    else:
        raise AssertionError("not refused")
v = sq.Weight(sq.SQ_FMT_INT8_ROW, 256, 512, q.view(torch.int8), torch.zeros(256))
try:
    sq.linear_fwd_w8a8(v, x)
except ValueError as err:
    assert "expected a CUDA tensor" in str(err), err
print("fine")
'''


def test_a_torch_without_the_8_bit_types():
    """The other formats work without them, the block-scaled calls say what they need."""
    for names in (["float8_e8m0fnu"], ["float8_e4m3fn", "float8_e8m0fnu"]):
        r = subprocess.run([sys.executable, "-c", OLD_TORCH, ROOT, *names], capture_output=True, text=True, timeout=600)
        assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("act", [None, 0, "relu", ["silu"]])
def test_activations_are_refused_by_name(act):
    w, e, x, dy = weight(), weight(E), t((M, K)), t((M, N))
    for f in (lambda: sq.gated_fwd_fp8(w, w, x, act=act), lambda: sq.gated_fwd_fp8(w, w, x, act=act, save=True),
              lambda: sq.gated_bwd_dx_fp8(w, w, dy, dy, dy, act=act),
              lambda: sq.grouped_gated_fwd_fp8(e, e, x, OFF, act=act, save=True),
              lambda: sq.grouped_gated_bwd_dx_fp8(e, e, dy, dy, dy, OFF, act=act),
              lambda: raw("sq_gated_fwd_fp8", w, x, t((M, N), torch.float32), act=act),
              lambda: raw("sq_grouped_gated_bwd_dx_fp8", e, dy, t((M, K), torch.float32), act=act)):
        with pytest.raises(ValueError, match="act must be one of"):
            f()
