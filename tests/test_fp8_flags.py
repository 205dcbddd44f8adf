"""The status flag of the block-scaled calls on the host: theirs, and no other call's."""
import pytest

import bit_quantized_frozen_b200 as sq
from test_fp8 import ALIGN, ARG, CALLS, cw, A, BIG


@pytest.mark.parametrize("call,fn,op", CALLS)
def test_status_flag(call, fn, op):
    # (accepted, and the refusal that comes behind the flags' own check)
    assert call(fn, flags=sq.SQ_STATUS_LIBRARY, x=A + 8) == ALIGN
    assert call(fn, flags=sq.SQ_STATUS_LIBRARY | sq.SQ_CHECK_FINITE | sq.SQ_OUT_BF16, x=A + 8) == ALIGN
    for flags in (0x200, 0x400, 1 << 31):
        assert call(fn, flags=flags, x=A + 8) == ARG


def test_other_calls_refuse_the_flag():
    L = sq.lib()
    w8 = cw(fmt=sq.SQ_FMT_INT8_ROW)
    assert L.sq_linear_fwd_w8a8(w8, A, 4, A, sq.SQ_STATUS_LIBRARY, A, BIG, None) == ARG
    assert L.sq_linear_bwd_dx_w8a8(w8, A, 4, A, sq.SQ_STATUS_LIBRARY, A, BIG, None) == ARG
    assert L.sq_build_fp8(A, 256, 512, sq.SQ_STATUS_LIBRARY, A, A, None) == ARG
