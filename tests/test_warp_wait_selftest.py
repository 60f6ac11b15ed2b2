"""The warp's bounded wait of the channel recurrence: gives up on a phase that never
completes without a fault or a hang, returns at once on one that has."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gated_deltanet_linear_20_b200", "csrc")
SRC = os.path.join(HERE, "csrc", "warp_wait_selftest.cu")
LIB = os.path.join(HERE, "csrc", "libwarp_wait_selftest.so")


def build_warp_wait_selftest(force: bool = False) -> str:
    deps = [SRC, os.path.join(CSRC, "sm100.cuh")]
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(map(os.path.getmtime, deps)):
        from gated_deltanet_linear_20_b200.build import ARCH_FLAGS, nvcc
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([nvcc(), *ARCH_FLAGS, "-O2", "-std=c++17", "-Xcompiler", "-fPIC",
                               "-shared", "-cudart", "static", "-I" + CSRC, SRC, "-o", tmp])
        os.replace(tmp, LIB)
    return LIB


def test_warp_wait_selftest_library_builds():
    assert os.path.exists(build_warp_wait_selftest())


@pytest.mark.gpu
def test_a_warp_gives_up_together_and_waits_no_more():
    lib = ctypes.CDLL(build_warp_wait_selftest())
    lib.warp_wait_selftest.argtypes = [ctypes.c_ulonglong, ctypes.c_void_p, ctypes.c_void_p]
    out = torch.zeros(4, dtype=torch.int64, device="cuda:0")
    assert lib.warp_wait_selftest(1_000_000, out.data_ptr(),
                                  torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    late, other, first, second = out.tolist()
    assert late == 32 and other == 0
    assert 1_000_000 <= first < 1_000_000_000 and second < 1_000_000
