"""The few-token forward at the channel shares of real layers: every CTA takes one to four tiles of
16 to 128 channels, the sums are long enough that every stage is used again, and the weights come
from DRAM (a copy that is late lands on top of what came before it)."""
import numpy as np
import pytest
import torch

import bit_quantized_frozen_b200 as sq
import w8a8ref as ref

pytestmark = pytest.mark.gpu
K = 2048


def layers(N, E, seed):
    """E layers [N, K] as tensors, made on the device."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(-127, 128, (E, N, K), dtype=torch.int8, device="cuda", generator=g)
    scales = (torch.rand(E, N, device="cuda", generator=g) + 0.5) * 1e-3
    up = (torch.randn(E, N, 16, device="cuda", generator=g) * 0.2).to(torch.bfloat16)
    down = (torch.randn(E, K, 16, device="cuda", generator=g) * 0.01).to(torch.bfloat16)
    return sq.GroupedWeight(E, N, K, codes, scales, up, down)


def rows(M, seed):
    x = np.random.default_rng(seed).standard_normal((M, K)).astype(np.float32)
    x[:, ::97] *= 15
    return ref.bf16(x)


def cold():
    """What was in L2 makes room."""
    torch.full((256 << 20,), 1, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()


def check(y, x, w, bf16):
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    r, b = ref.forward(x, w.codes.cpu().numpy(), f(w.scales), f(w.lora_up), f(w.lora_down), bf16_out=bf16)
    ref.check(f(y), r, b, bf16)


@pytest.mark.parametrize("N", [4736, 6144, 9472, 9600, 14208, 16384, 17792, 17920, 18304, 18944, 19200, 37888])
def test_dense_shares(N):
    """N = 17792 .. 18304 on 148 SMs: CTAs with 120 and with 124 channels beside a box of 128 rows."""
    w = layers(N, 1, N).expert(0)
    for M, bf16 in ((1, True), (16, False), (24, False), (64, True), (128, False)):
        x = rows(M, N + M)
        xd = torch.from_numpy(x).cuda().to(torch.bfloat16)
        cold()
        first = sq.linear_fwd_w8a8(w, xd, out_bf16=bf16)
        check(first, x, w, bf16)
        for _ in range(8):
            cold()
            assert torch.equal(sq.linear_fwd_w8a8(w, xd, out_bf16=bf16), first)


# (experts with rows, N): shares of 112 and 120 channels on 148 SMs, and sizes around them
SHARES = [(8, 2048), (4, 4096), (2, 8192), (1, 16384), (6, 2816), (5, 3584), (7, 2560), (11, 1536), (16, 1024), (17, 1024),
          (8, 1920), (8, 2304), (27, 2816), (3, 2944), (1, 6144)]


@pytest.mark.parametrize("used,N", SHARES)
def test_experts_shares(used, N):
    """One token through `used` of the experts (a row each), then a few rows for each."""
    E = used + 5
    w = layers(N, E, used * N)
    rng = np.random.default_rng(used + N)
    for per in (1, 3):
        counts = np.zeros(E, int)
        counts[rng.permutation(E)[:used]] = per
        off = np.concatenate([[0], np.cumsum(counts)])
        x = rows(int(off[-1]), N + per)
        xd = torch.from_numpy(x).cuda().to(torch.bfloat16)
        offd = torch.from_numpy(off.astype(np.int32)).cuda()
        cold()
        first = sq.grouped_fwd_w8a8(w, xd, offd)
        for e in np.nonzero(counts)[0]:
            check(first[off[e]:off[e + 1]], x[off[e]:off[e + 1]], w.expert(int(e)), False)
        for _ in range(8):
            cold()
            assert torch.equal(sq.grouped_fwd_w8a8(w, xd, offd), first)


@pytest.mark.parametrize("rows_each,used,N", [(24, 8, 2048), (60, 4, 4096), (60, 6, 2816), (100, 2, 8192), (128, 8, 2048)])
def test_experts_shares_of_wider_tiles(rows_each, used, N):
    """Tiles of 32, 64 and 128 tokens at the same shares."""
    w = layers(N, used, N + rows_each)
    off = np.arange(used + 1) * rows_each
    x = rows(int(off[-1]), rows_each)
    cold()
    y = sq.grouped_fwd_w8a8(w, torch.from_numpy(x).cuda().to(torch.bfloat16), torch.from_numpy(off.astype(np.int32)).cuda())
    for e in range(used):
        check(y[off[e]:off[e + 1]], x[off[e]:off[e + 1]], w.expert(e), False)
