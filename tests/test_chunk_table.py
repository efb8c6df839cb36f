"""The look-up of a unit's chunk in rows that are read element by element (csrc/chunks.h), on the host: every column's own
chunk, and a chunk of the table for lanes without columns, whatever lies in memory after it."""
import ctypes
import os
import subprocess

import pytest

import reducescatter_reduction_gb300 as ccl
from conftest import ROOT

pytestmark = pytest.mark.cpu


@pytest.fixture(scope="module")
def chunk_of(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("chunks") / "chunks.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC",
                    os.path.join(ROOT, "tests", "layer_checks", "chunks.cpp"), "-o", so], check=True)
    f = ctypes.CDLL(so).chunk_of
    f.argtypes = [ctypes.POINTER(ctypes.c_uint64), ctypes.c_int, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_uint32]
    return f


@pytest.mark.parametrize("p, rows, hidden", [(1, 1, 1), (2, 7, 3), (5, 3, 1), (16, 152, 1), (33, 152, 9), (64, 152, 3), (64, 160, 22), (64, 9, 7)])
def test_every_element(chunk_of, p, rows, hidden):
    n = rows * hidden
    bounds, _ = ccl.ccl_schedule_build(p, n, "ring")
    table = (ctypes.c_uint64 * (p + 1 + 64))(*bounds, *[0] * 64)        # zeros after the table: a walk past it goes on
    for row in range(rows):
        base = row * hidden
        first = max(c for c in range(p) if bounds[c] <= base)
        for column in range(-(-hidden // 32) * 32):
            c = chunk_of(table, first, base, column, hidden)
            assert 0 <= c < p
            assert bounds[c] <= base + min(column, hidden - 1) < bounds[c + 1]
