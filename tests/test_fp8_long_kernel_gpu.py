"""Block-scaled products behind a kernel that runs for longer than their own waits may take (2 s) and lets the kernel
behind it start at once."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

import bit_quantized_frozen_b200 as sq
import fp8ref as ref
from bit_quantized_frozen_b200 import build
from test_fp8_calls_gpu import BF, dev, f32, layer, rand, weight

pytestmark = pytest.mark.gpu

SLOW = r'''
// runs for `ns` nanoseconds (at most 2^24 rounds of a microsecond's sleep), having let the next kernel start
__global__ void slow_kernel(unsigned long long ns, unsigned *done)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    unsigned long long t0, t = 0;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    t = t0;
    for (int i = 0; i < (1 << 24) && t - t0 < ns; ++i) {
        __nanosleep(1000);
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    }
    *done = 1;
}

extern "C" int slow(unsigned long long ns, unsigned *done, void *stream)
{
    slow_kernel<<<1, 1, 0, (cudaStream_t)stream>>>(ns, done);
    return (int)cudaGetLastError();
}
'''


@pytest.fixture(scope="module")
def slow(tmp_path_factory):
    d = tmp_path_factory.mktemp("slow")
    (d / "slow.cu").write_text(SLOW)
    subprocess.run([build.nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC", "-o",
                    str(d / "slow.so"), str(d / "slow.cu")], check=True)
    f = ctypes.CDLL(str(d / "slow.so")).slow
    f.argtypes = [ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p]
    return f


@pytest.mark.parametrize("M,grouped", [(4, False), (90, False), (4, True)])
def test_a_call_behind_a_long_kernel(slow, M, grouped):
    rng = np.random.default_rng(M)
    N, K = 272, 1168
    q, s = layer(rng, N, K)
    w = weight(q[None], s[None]) if grouped else weight(q, s)
    x, off = rand(rng, M, K), dev(np.array([0, M], np.int32))
    xd, done = dev(x, BF), torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: sq.grouped_fwd_fp8(w, xd, off) if grouped else sq.linear_fwd_fp8(w, xd)  # noqa: E731
    call()                                                   # (everything is loaded)
    torch.cuda.synchronize()
    assert slow(2_300_000_000, done.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    y = call()
    torch.cuda.synchronize()
    assert int(done) == 1
    sq.sq_check_device_status(None)
    ref.check(f32(y), *ref.forward(x, ref.dequant(q, s)), False)
