"""Bounded waits of the attention kernels: they end and say so, and their limit covers the
kernel's own progress, not the time of the kernel that it starts beside.  No GPU fault is caused."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import attention_util as au

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_memory_attention_b200 import build
    path = str(tmp_path_factory.mktemp("waits") / "attention_waits.so")
    subprocess.run([build.NVCC] + build.FLAGS + ["-I", os.path.join(build.ROOT, "include"), "-I", build.SRC_DIR, "-o", path,
                                                 os.path.join(HERE, "attention_waits.cu")], check=True, timeout=600)
    lib = ctypes.CDLL(path)
    lib.dkdv_behind.argtypes = ([ctypes.c_int] + [ctypes.c_void_p] * 9 + [ctypes.c_int] * 4 + [ctypes.c_float] +
                                [ctypes.c_uint] * 2)
    lib.run_out.argtypes = [ctypes.c_uint, ctypes.c_void_p]
    return lib


def test_a_wait_runs_out(waits):
    """A wait on a barrier that nothing arrives at ends after its limit with its fault bit, the
    block's later waits end at once, a complete phase is still seen, and the context lives on."""
    got = torch.full((5,), 7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert waits.run_out(50_000, got.data_ptr()) == 0x20 | 0x100  # the wait's own bit, the exit wait's
    done, us, again, us_again, complete = got.tolist()
    assert done == 0 and 50_000 <= us < 500_000
    assert again == 0 and us_again < 50_000
    assert complete == 1
    assert waits.run_out(1, got.data_ptr()) == 0x120
    assert (got + 1).tolist()[4] == 2


# More units of 64 rows than the ring has stages; one; two and a half.
@pytest.mark.parametrize("Hq,Hkv,n,m", [(4, 2, 600, 300), (1, 1, 20, 100), (2, 2, 160, 128)])
@pytest.mark.parametrize("d", [64, 128])
def test_key_gradients_wait_for_a_slow_kernel(waits, Hq, Hkv, n, m, d):
    """delta comes 60 ms after dK and dV's kernel may start, whose waits end after 20 ms: its
    first tiles take microseconds, so that only a wait for delta could run out."""
    tau = 1.0 / math.sqrt(d)
    q, do = (au.randn((1, Hq, n, d), torch.bfloat16, s) for s in (1, 2))
    k, v = (au.randn((1, Hkv, m, d), torch.bfloat16, s) for s in (3, 4))
    want = au.cross(q, k, v, tau, None, do)
    lse = want["lse"][0].float().cuda()
    ready = (au.f64(do) * want["out"][0]).sum(-1).float().cuda()
    delta = torch.full_like(ready, float("nan"))
    got = {"dk": torch.empty_like(k), "dv": torch.empty_like(v)}
    torch.cuda.synchronize()
    ptrs = [x.data_ptr() for x in (q, k, v, do, got["dk"], got["dv"], lse, ready, delta)]
    assert waits.dkdv_behind(d, *ptrs, Hq, Hkv, n, m, tau, 60_000, 20_000) == 0
    au.check(got, {x: want[x] for x in got})
