"""Where the block-scaled products report what they found on the device."""
import threading
import time

import numpy as np
import pytest
import torch

import bit_quantized_frozen_b200 as sq
from test_fp8_calls_gpu import BF, dev, layer, rand, weight

pytestmark = pytest.mark.gpu
N, K, E = 272, 400, 3
NONFINITE, INDEX = 9, 10


def status(ws=None):
    torch.cuda.synchronize()
    try:
        sq.sq_check_device_status(ws)
    except sq.SqError as e:
        return e.status
    return sq.SQ_OK


def calls(M, off=None):
    """{name: call(x's or dy's first value, further arguments)}"""
    rng = np.random.default_rng(M)
    ws = [weight(*layer(rng, N, K, None if off is None else E)) for _ in range(2)]
    x, dy, g, u = (dev(rand(rng, M, n), BF) for n in (K, N, N, N))
    o = () if off is None else (dev(np.array(off, np.int32)),)

    def first(t, v):
        t = t.clone()
        t[M // 2, 5] = v
        return t

    name = ("grouped_%s_fp8" if o else "%s_fp8") % "%s"
    linear = "" if o else "linear_"
    return {"fwd": lambda v, **kw: getattr(sq, name % (linear + "fwd"))(ws[0], first(x, v), *o, **kw),
            "bwd": lambda v, **kw: getattr(sq, name % (linear + "bwd_dx"))(ws[0], first(dy, v), *o, **kw),
            "gated_fwd": lambda v, **kw: getattr(sq, name % "gated_fwd")(*ws, first(x, v), *o, **kw),
            "gated_bwd": lambda v, **kw: getattr(sq, name % "gated_bwd_dx")(*ws, first(dy, v), g, u, *o, **kw)}


@pytest.mark.parametrize("M", [1, 8, 9, 32, 33, 300, 1500])
@pytest.mark.parametrize("grouped", [False, True])
def test_calls_without_a_workspace_report_to_the_library(M, grouped):
    """The same place on both sides of the border of one kernel: the library's word, which a call with its own
    workspace leaves alone."""
    assert status() == sq.SQ_OK
    for name, call in calls(M, [0, M // 3, M // 2, M] if grouped else None).items():
        call(1.0, flags=sq.SQ_CHECK_FINITE)
        assert status() == sq.SQ_OK, name
        for bad in (float("nan"), float("inf")):
            call(bad)
            assert status() == sq.SQ_OK, name                # not asked for
            call(bad, flags=sq.SQ_CHECK_FINITE)
            call(1.0, flags=sq.SQ_CHECK_FINITE)              # (does not clear what the call before has found)
            assert status() == NONFINITE, name
            assert status() == sq.SQ_OK, name
            ws = torch.full((1 << 23,), 0xFF, dtype=torch.uint8, device="cuda")
            call(bad, flags=sq.SQ_CHECK_FINITE, ws=ws)
            assert status() == sq.SQ_OK and status(ws) == NONFINITE, name
            call(1.0, flags=sq.SQ_CHECK_FINITE, ws=ws)
            assert status(ws) == sq.SQ_OK, name
            call(bad, flags=sq.SQ_CHECK_FINITE | sq.SQ_STATUS_LIBRARY, ws=ws.fill_(0))
            assert status(ws) == sq.SQ_OK and status() == NONFINITE, name


@pytest.mark.parametrize("M", [6, 90])
def test_clamped_offsets_are_reported_without_a_workspace(M):
    for off in ([0, M, M // 2, M], [0, 1, 2, M + 1], [-1, 0, 0, M]):
        for name, call in calls(M, off).items():
            call(1.0)
            assert status() == INDEX, name
            assert status() == sq.SQ_OK, name


def test_no_report_is_lost_between_streams():
    """One thread asks all the time and another one's calls find NaN all the time, each on a stream of its own: the
    offsets that a call on a third stream clamps are in a report all the same."""
    rng = np.random.default_rng(1)
    w, bad = weight(*layer(rng, N, K, E)), torch.full((4, K), float("nan"), dtype=BF, device="cuda")
    fine, off = torch.zeros_like(bad), dev(np.array([0, 1, 2, 4], np.int32))
    wrong = dev(np.array([0, 2, 1, 4], np.int32))
    assert status() == sq.SQ_OK
    done, asked, found = threading.Event(), [0], [0]

    def ask():
        stream = torch.cuda.Stream()
        while not done.is_set():
            try:
                sq.sq_check_device_status(None, stream=stream)
            except sq.SqError as e:
                found[0] += e.status == INDEX
            asked[0] += 1

    sq.grouped_fwd_fp8(w, bad, off, flags=sq.SQ_CHECK_FINITE)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(200):
            sq.grouped_fwd_fp8(w, bad, off, flags=sq.SQ_CHECK_FINITE)

    def find():
        with torch.cuda.stream(torch.cuda.Stream()):
            while not done.is_set():
                graph.replay()
                torch.cuda.current_stream().synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=f) for f in (ask, find)]
    for t in threads:
        t.start()
    lost = []
    stream = torch.cuda.Stream()
    try:
        for i in range(400):
            before, wait = found[0], time.perf_counter() + rng.uniform(0, 1e-4)
            while time.perf_counter() < wait:
                pass
            sq.grouped_fwd_fp8(w, fine, wrong, stream=stream)
            stream.synchronize()
            n, until = asked[0], time.monotonic() + 20
            while asked[0] < n + 2 and time.monotonic() < until:      # (one that began after the call)
                time.sleep(0)
            assert asked[0] >= n + 2, "nobody asks"
            # (two of the call's CTAs may find it, and a report lie between them)
            if found[0] == before:
                lost.append(i)
    finally:
        done.set()
        for t in threads:
            t.join()
    assert not lost, lost
    status()


def test_a_report_names_all_findings():
    rng = np.random.default_rng(2)
    w, bad = weight(*layer(rng, N, K, E)), torch.full((4, K), float("nan"), dtype=BF, device="cuda")
    off = torch.tensor([0, 2, 1, 4], dtype=torch.int32, device="cuda")
    for ws in (None, torch.zeros(256, dtype=torch.uint8, device="cuda")):
        sq.grouped_fwd_fp8(w, bad, off, ws=ws, flags=sq.SQ_CHECK_FINITE)
        with pytest.raises(sq.SqError, match="index non-finite") as e:
            sq.sq_check_device_status(ws)
        assert e.value.status == INDEX
        assert status(ws) == sq.SQ_OK
