"""The 8-bit products refuse weight tensors of another type or shape by name: they would be read
with the wrong stride or as other numbers."""
import pytest
import torch

import bit_quantized_frozen_b200 as sq

M, N, K = 40, 256, 512


def t(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def weight(E, **other):
    lead = () if E is None else (E,)
    parts = dict(codes=t(lead + (N, K), torch.int8), scales=t(lead + (N,), torch.float32), lora_up=t(lead + (N, 16)),
                 lora_down=t(lead + (K, 16)))
    parts.update(other)
    if E is None:
        return sq.Weight(sq.SQ_FMT_INT8_ROW, N, K, g_w=None, **parts)
    return sq.GroupedWeight(E, N, K, **parts)


def calls(E):
    x, dy, off = t((M, K)), t((M, N)), t((E or 0) + 1, torch.int32)
    if E is None:
        return [lambda w: sq.linear_fwd_w8a8(w, x), lambda w: sq.linear_bwd_dx_w8a8(w, dy)]
    return [lambda w: sq.grouped_fwd_w8a8(w, x, off), lambda w: sq.grouped_bwd_dx_w8a8(w, dy, off)]


@pytest.mark.parametrize("E", [None, 3])
def test_types_and_shapes(E):
    lead = () if E is None else (E,)
    wrong = dict(
        codes=[t(lead + (N, K), torch.uint8), t(lead + (N, K), torch.float16), t(lead + (K, N), torch.int8),
               t(lead + (N, 2 * K), torch.int8), t((4,) + (N, K), torch.int8)],
        scales=[t(lead + (N,), torch.float64), t(lead + (2 * N,), torch.bfloat16), t(lead + (N, 1), torch.float32)],
        # the rank-32 factors of the other modes, single-precision ones, the transposed layout
        lora_up=[t(lead + (N, 32)), t(lead + (N, 16), torch.float32), t(lead + (N, 16), torch.float16), t(lead + (16, N))],
        lora_down=[t(lead + (K, 32)), t(lead + (K, 16), torch.float32), t(lead + (K, 16), torch.float16), t(lead + (16, K))])
    for call in calls(E):
        with pytest.raises(ValueError, match="expected a CUDA tensor"):        # all right but for the device
            call(weight(E))
        with pytest.raises(ValueError, match="expected a CUDA tensor"):
            call(weight(E, lora_up=None, lora_down=None))
        for name, tensors in wrong.items():
            for bad in tensors:
                with pytest.raises(ValueError, match=f"{name} must be torch"):
                    call(weight(E, **{name: bad}))


def test_a_missing_output_is_the_librarys_to_refuse():
    """y = None (NULL) passes the binding's checks of types, as it does in the other entry points."""
    x, dy, off = t((M, K)), t((M, N)), t(4, torch.int32)
    for call in (lambda: sq.sq_linear_fwd_w8a8(weight(None), x, None), lambda: sq.sq_linear_bwd_dx_w8a8(weight(None), dy, None),
                 lambda: sq.sq_grouped_fwd_w8a8(weight(3), x, off, None),
                 lambda: sq.sq_grouped_bwd_dx_w8a8(weight(3), dy, off, None)):
        with pytest.raises(ValueError, match="expected a CUDA tensor"):
            call()


@pytest.mark.gpu
def test_a_missing_output_on_the_device():
    x = t((M, K)).cuda()
    w = weight(None)
    for name in ("codes", "scales", "lora_up", "lora_down"):
        setattr(w, name, getattr(w, name).cuda())
    with pytest.raises(sq.SqError) as e:
        sq.sq_linear_fwd_w8a8(w, x, None, ws=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 1
