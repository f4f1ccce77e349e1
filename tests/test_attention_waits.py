"""Bounded waits of the attention kernels: a wait's limit covers the kernel's own progress,
not the time of the kernel that it starts beside."""
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
def behind(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_memory_attention_b200 import build
    lib = str(tmp_path_factory.mktemp("dkdv") / "dkdv_behind.so")
    subprocess.run([build.NVCC] + build.FLAGS + ["-I", os.path.join(build.ROOT, "include"), "-I", build.SRC_DIR, "-o", lib,
                                                 os.path.join(HERE, "dkdv_behind.cu")], check=True, timeout=600)
    f = ctypes.CDLL(lib).dkdv_behind
    f.restype = ctypes.c_int
    f.argtypes = ([ctypes.c_int] + [ctypes.c_void_p] * 9 + [ctypes.c_int] * 4 + [ctypes.c_float] + [ctypes.c_uint] * 2)
    return f


# More units of 64 rows than the ring has stages; one; two and a half.
@pytest.mark.parametrize("Hq,Hkv,n,m", [(4, 2, 600, 300), (1, 1, 20, 100), (2, 2, 160, 128)])
@pytest.mark.parametrize("d", [64, 128])
def test_key_gradients_wait_for_a_slow_kernel(behind, Hq, Hkv, n, m, d):
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
    assert behind(d, *ptrs, Hq, Hkv, n, m, tau, 60_000, 20_000) == 0
    au.check(got, {x: want[x] for x in got})
