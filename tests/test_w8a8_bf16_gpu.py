"""A bf16 result of the 8-bit products is the fp32 result rounded once: nothing else is computed in
fewer bits for it."""
import numpy as np
import pytest
import torch

import bit_quantized_frozen_b200 as sq
import w8a8ref as ref

pytestmark = pytest.mark.gpu


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


@pytest.mark.parametrize("op", ["fwd", "bwd"])
@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (20, 384, 1280), (100, 640, 768), (300, 1152, 1536)])
def test_bf16_is_the_fp32_result_rounded(op, M, N, K):
    rng = np.random.default_rng(M + N)
    E = 3
    Q, sw, up, down = ref.layer(rng, N, K, E=E)
    b = lambda a: dev(a, torch.bfloat16)  # noqa: E731
    w = sq.GroupedWeight(E, N, K, dev(Q), dev(sw), b(up), b(down))
    x = b(rng.standard_normal((M, N if op == "bwd" else K)).astype(np.float32))
    off = dev(np.array([0, M // 3, M // 3, M], np.int32))
    dense, grouped = ((sq.linear_bwd_dx_w8a8, sq.grouped_bwd_dx_w8a8) if op == "bwd" else
                      (sq.linear_fwd_w8a8, sq.grouped_fwd_w8a8))
    assert torch.equal(dense(w.expert(1), x, out_bf16=True), dense(w.expert(1), x).to(torch.bfloat16))
    assert torch.equal(grouped(w, x, off, out_bf16=True), grouped(w, x, off).to(torch.bfloat16))


@pytest.mark.parametrize("bf16", [False, True])
def test_low_rank_input_of_the_gradient_keeps_24_bits(bf16):
    """u = (1 + 2^-9 + 2^-18, -1, -2^-9) times a power of two, lora_down of ones and codes of zeros:
    dx is 2^-18 times that power.  Every product and every partial sum, in any order, is a multiple
    of 2^-18 below 4 (times the power), 20 bits, so fp32 holds each exactly and so does bf16 the
    result.  u[0] with its lowest bit dropped would give 0."""
    M, N, K = 5, 128, 256
    up, down = np.zeros((N, 16), np.float32), np.zeros((K, 16), np.float32)
    up[0, :2], up[1, 0], up[1, 2], up[2, 0] = (1, -1), 1, -1, 1
    down[:, :3] = 1
    power = 2.0 ** -np.arange(M, dtype=np.float32)[:, None]
    dy = np.zeros((M, N), np.float32)
    dy[:, 0], dy[:, 1], dy[:, 2] = 1, 2.0 ** -9, 2.0 ** -18
    b = lambda a: dev(a, torch.bfloat16)  # noqa: E731
    w = sq.Weight(sq.SQ_FMT_INT8_ROW, N, K, dev(np.zeros((N, K), np.int8)), dev(np.ones(N, np.float32)), None, b(up),
                  b(down))
    dx = sq.linear_bwd_dx_w8a8(w, b(dy * power), out_bf16=bf16).float().cpu().numpy()
    assert np.array_equal(dx, np.broadcast_to(power * np.float32(2.0) ** -18, (M, K)))
