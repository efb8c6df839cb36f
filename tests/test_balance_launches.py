"""The launches of the balance loss when one of them fails, without a GPU: the
object of csrc/balance.cu is linked against fakes of the CUDA runtime."""
import ctypes
import os
import subprocess

import pytest

from conftest import ROOT
from reducescatter_reduction_gb300 import build as ccl_build
from test_logit_refusals import CUDA

pytestmark = pytest.mark.cpu

SCRATCH, STREAM = 4 << 44, 5 << 44
FORWARD, BACKWARD, BOTH = 1, 2, 3


@pytest.fixture(scope="module")
def fakes(tmp_path_factory):
    ccl_build.build()
    so = str(tmp_path_factory.mktemp("launches") / "launches.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-Wl,-Bsymbolic",
                    "-I", os.path.join(ROOT, "include"), "-I", CUDA, os.path.join(ROOT, "tests", "logit_checks", "launches.cpp"),
                    os.path.join(ccl_build.BUILD, "balance.cu.o"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    sz, i, u = ctypes.c_size_t, ctypes.c_int, ctypes.c_uint
    L.fake_balance.argtypes = [i, sz, u, u, i, sz, sz, i, i]
    L.fake_log.restype = ctypes.c_char_p
    L.fake_scratch_head.restype = L.fake_scratch_counters.restype = sz
    return L


def calls(fakes, rows=4096, experts=64, steps=BOTH, p=8, fail_launch=0, fail_attribute=0):
    """(status, the CUDA calls made)"""
    status = fakes.fake_balance(p, rows, experts, 4, steps, SCRATCH, STREAM, fail_launch, fail_attribute)
    return status, fakes.fake_log().decode().splitlines()


def cleared(fakes):
    return f"memset {SCRATCH + fakes.fake_scratch_head()} 0 {fakes.fake_scratch_counters()} {STREAM}"


@pytest.mark.parametrize("experts", [64, 61, 1500])
@pytest.mark.parametrize("steps", [FORWARD, BOTH])
def test_counters_are_cleared_if_the_second_launch_fails(fakes, experts, steps):
    status, log = calls(fakes, experts=experts, steps=steps)
    launches = [x for x in log if "launch" in x]
    assert status == 0 and launches == ["launch 1024", "launch 256"] and not [x for x in log if "memset" in x]
    status, log = calls(fakes, experts=experts, steps=steps, fail_launch=2)
    assert status != 0 and log[-3:] == ["launch 1024", "failed launch 256", cleared(fakes)]


def test_nothing_is_counted_before_the_kernel_is_ready(fakes):
    """Rows that are no aligned groups raise a kernel's shared-memory limit: if that fails, nothing has been launched."""
    for experts in (61, 700 + 1):
        status, log = calls(fakes, experts=experts, fail_attribute=1)
        assert status != 0 and log == ["failed attribute"]


def test_what_used_no_counters_clears_none(fakes):
    status, log = calls(fakes, rows=16, fail_launch=1)                       # counts in the pass itself
    assert status != 0 and log == ["failed launch 256"]
    status, log = calls(fakes, steps=BACKWARD, fail_launch=1)
    assert status != 0 and log == ["failed launch 256"]
    status, log = calls(fakes, experts=3000, fail_launch=2)                  # counts in the caller's own
    assert status != 0 and len(log) == 4 and [x.split()[0] for x in log] == ["memset", "memset", "launch", "failed"]
    status, log = calls(fakes, fail_launch=1)                                # the counting kernel itself
    assert status != 0 and log == ["failed launch 1024"]
