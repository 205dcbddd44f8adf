"""Calls of the 8-bit products as programs make them: on streams of their own."""
import pytest
import torch

import bit_quantized_frozen_b200 as sq

pytestmark = pytest.mark.gpu


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
