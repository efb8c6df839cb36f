"""Row counts beyond what one launch numbers, without a GPU: the front end and
the launch code of the logit operators against fakes of the CUDA runtime."""
import ctypes
import os
import subprocess

import pytest

import reducescatter_reduction_gb300 as ccl
from conftest import ROOT
from reducescatter_reduction_gb300 import build as ccl_build
from test_logit_refusals import CUDA

pytestmark = pytest.mark.cpu

ROWS = 2 ** 31 - 1
LIST = 1 << 60                     # far from the rank buffers


@pytest.fixture(scope="module")
def fakes(tmp_path_factory):
    ccl_build.build()
    so = str(tmp_path_factory.mktemp("sizes") / "sizes.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-Wl,-Bsymbolic",
                    "-I", os.path.join(ROOT, "include"), "-I", CUDA, os.path.join(ROOT, "tests", "logit_checks", "sizes.cpp")]
                   + [os.path.join(ccl_build.BUILD, f"{n}.cu.o") for n in ("logit_rules", "distill", "balance")] + ["-o", so], check=True)
    L = ctypes.CDLL(so)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.fake_comm.restype = vp
    L.fake_comm_free.argtypes = [vp]
    L.fake_message.restype = ctypes.c_char_p
    L.ccl_logit_rules.argtypes = [vp, i, sz, sz, sz, ctypes.POINTER(ccl.LogitRules), vp]
    L.ccl_distill_topk.argtypes = [vp, i, i, sz, sz, sz, sz, vp, vp, i, ctypes.c_float, vp, vp, vp, vp]
    return L


def outcome(L, p, call):
    c, before = L.fake_comm(p), L.fake_launches()
    st = call(c)
    L.fake_comm_free(c)
    return st, L.fake_launches() - before


@pytest.mark.parametrize("p,rows,vocab,fits", [(1, ROWS, 8, True), (2, ROWS, 8, False), (2, ROWS // 2, 8, True), (64, ROWS // 64 + 1, 64, False),
                                               (1, ROWS // 3, 50000, False)])
def test_rules(fakes, p, rows, vocab, fits):
    rules = ccl.LogitRules()
    got = outcome(fakes, p, lambda c: fakes.ccl_logit_rules(c, ccl.CCL_BF16, rows, vocab, 0, ctypes.byref(rules), None))
    assert got == ((ccl.CCL_OK, 1) if fits else (ccl.CCL_ERR_UNSUPPORTED, 0))
    if not fits:
        assert b"logit_rules" in fakes.fake_message() and str(rows).encode() in fakes.fake_message()


@pytest.mark.parametrize("steps", [ccl.CCL_PASS_FORWARD, ccl.CCL_PASS_BACKWARD, ccl.CCL_PASS_BOTH])
@pytest.mark.parametrize("p,rows,vocab,fits", [(1, ROWS, 8, True), (2, ROWS // 2, 60000, False), (16, ROWS, 300000, False), (16, ROWS // 32, 300000, True)])
def test_distillation(fakes, steps, p, rows, vocab, fits):
    got = outcome(fakes, p, lambda c: fakes.ccl_distill_topk(c, ccl.CCL_BF16, steps, rows, vocab, 0, 2, LIST, 2 * LIST, ccl.CCL_F32, 1.0, 0,
                                                             3 * LIST, 4 * LIST, None))
    assert got == ((ccl.CCL_OK, 1) if fits else (ccl.CCL_ERR_UNSUPPORTED, 0))
    if not fits:
        assert b"distill_topk" in fakes.fake_message() and str(rows).encode() in fakes.fake_message()
