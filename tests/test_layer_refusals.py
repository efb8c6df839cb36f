"""What the operators around layers refuse, tested without a GPU: the host
front ends (csrc/layers.cpp, csrc/ccl.cpp) are compiled against fakes of the
CUDA runtime and of the kernel launchers.  Each case starts from arguments that
are accepted and changes one thing."""
import ctypes
import glob
import os
import subprocess

import pytest

import reducescatter_reduction_gb300 as ccl
from conftest import ROOT

pytestmark = pytest.mark.cpu

CUDA = next((d for d in ("/usr/local/cuda/include", *glob.glob("/usr/local/cuda*/include")) if os.path.isdir(d)), None)
OK, BAD, UNSUPPORTED = ccl.CCL_OK, ccl.CCL_ERR_INVALID_ARG, ccl.CCL_ERR_UNSUPPORTED
P, ROWS, HIDDEN, EXPERTS, K, CAPACITY = 2, 4, 24, 5, 3, 7
A = 1 << 20                        # distance between the buffers' made-up addresses
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def front(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("layer_checks") / "driver.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC",
                    "-Wl,-Bsymbolic",      # the driver's own fakes, whatever CUDA runtime the process has loaded
                    "-I", os.path.join(ROOT, "include"), "-I", CUDA,
                    os.path.join(ROOT, "tests", "layer_checks", "driver.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    vp, i, sz, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    pvp = ctypes.POINTER(vp)
    L.ccl_comm_create.argtypes = [pvp, i, pvp]
    L.ccl_comm_set_outputs.argtypes = [vp, pvp]
    L.ccl_comm_destroy.argtypes = [vp]
    L.ccl_last_error.restype = ctypes.c_char_p
    L.ccl_allreduce_residual_rmsnorm_e4m3.argtypes = [vp, i, sz, sz, vp, vp, vp, pvp, sz, f, i, vp]
    L.ccl_expert_sort.argtypes = [vp, sz, sz, sz, pvp, pvp, sz, pvp, vp, vp]
    L.ccl_expert_dispatch.argtypes = L.ccl_expert_combine.argtypes = [vp, i, sz, sz, sz, pvp, pvp, sz, vp]
    L.ccl_expert_combine_grad.argtypes = [vp, i, sz, sz, sz, pvp, pvp, pvp, sz, pvp, vp]
    L.ccl_grad_norm.argtypes = [vp, sz, ctypes.POINTER(ccl.Tensor), vp, vp]
    L.ccl_grad_clip.argtypes = [vp, sz, ctypes.POINTER(ccl.Tensor), f, vp, vp]
    return L


def pointers(values):
    return None if values is None else (ctypes.c_void_p * len(values))(*values)


def status(front, call, ins=(1 * A, 2 * A), outs=(3 * A, 4 * A)):
    """(status, kernels launched) of one call."""
    h = ctypes.c_void_p()
    assert front.ccl_comm_create(ctypes.byref(h), P, pointers(ins)) == OK
    assert front.ccl_comm_set_outputs(h, pointers(outs)) == OK
    before = front.fake_launches()
    try:
        return call(h), front.fake_launches() - before
    finally:
        front.ccl_comm_destroy(h)


def norm(front, dtype=ccl.CCL_BF16, rows=ROWS, hidden=HIDDEN, residual=10 * A, residual_out=11 * A, gamma=12 * A,
         scales=(13 * A, 14 * A), group=0, eps=1e-6, schedule=ccl.CCL_SCHED_RING):
    return lambda c: front.ccl_allreduce_residual_rmsnorm_e4m3(c, dtype, rows, hidden, residual, residual_out, gamma,
                                                               pointers(scales), group, eps, schedule, None)


def sort(front, rows=ROWS, experts=EXPERTS, k=K, ids=(10 * A, 11 * A), valid=(12 * A, 13 * A), capacity=CAPACITY,
         slots=(14 * A, 15 * A), offsets=16 * A):
    return lambda c: front.ccl_expert_sort(c, rows, experts, k, pointers(ids), pointers(valid), capacity, pointers(slots),
                                           offsets, None)


def move(front, name, dtype=ccl.CCL_BF16, rows=ROWS, hidden=HIDDEN, k=K, slots=(10 * A, 11 * A), weights=(12 * A, 13 * A),
         capacity=CAPACITY, experts=(14 * A, 15 * A), dweights=(16 * A, 17 * A)):
    if name == "grad":
        return lambda c: front.ccl_expert_combine_grad(c, dtype, rows, hidden, k, pointers(slots), pointers(weights),
                                                       pointers(experts), capacity, pointers(dweights), None)
    f = getattr(front, "ccl_expert_" + name)
    return lambda c: f(c, dtype, rows, hidden, k, pointers(slots), pointers(weights), capacity, None)


def tensor(at=10 * A, out=11 * A, n=100, dtype=ccl.CCL_BF16, copy=0):
    return ccl.Tensor(at, out, n, dtype, copy)


def grads(front, name, *tensors, count=None, max_norm=1.0, at=20 * A):
    arr = (ccl.Tensor * max(1, len(tensors)))(*tensors)
    n = len(tensors) if count is None else count
    given = arr if tensors else None
    if name == "norm":
        return lambda c: front.ccl_grad_norm(c, n, given, at, None)
    return lambda c: front.ccl_grad_clip(c, n, given, max_norm, at, None)


def check(front, call, want, said="", **buffers):
    got, launches = status(front, call, **buffers)
    assert got == want, front.ccl_last_error()
    assert launches == (1 if want == OK else 0)
    if said:
        assert said.encode() in front.ccl_last_error()


NORM_OUT = ROWS * HIDDEN            # bytes of an e4m3 output
IN_BYTES = 2 * NORM_OUT             # of a bf16 input


@pytest.mark.parametrize("change, want", [
    (dict(), OK), (dict(dtype=ccl.CCL_I32), UNSUPPORTED), (dict(dtype=9), BAD), (dict(dtype=-1), BAD),
    (dict(hidden=0), BAD), (dict(group=32), OK), (dict(group=64), OK), (dict(group=128), OK), (dict(group=16), BAD),
    (dict(group=256), BAD), (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD), (dict(eps=INF), BAD), (dict(eps=0.0), OK),
    (dict(schedule=9), BAD), (dict(schedule=ccl.CCL_SCHED_CUSTOM), BAD), (dict(rows=1 << 62), BAD),
    (dict(rows=1 << 28, hidden=1), UNSUPPORTED), (dict(hidden=1 << 31, rows=1), UNSUPPORTED), (dict(residual=0), BAD), (dict(residual_out=0), BAD),
    (dict(gamma=0), BAD), (dict(scales=None), BAD), (dict(scales=(13 * A, 0)), BAD), (dict(scales=(13 * A, 14 * A + 2)), BAD),
    (dict(residual=10 * A + 1), BAD), (dict(residual=10 * A + 2), OK), (dict(residual_out=10 * A), OK),
    (dict(residual_out=10 * A + 2), BAD), (dict(gamma=11 * A + 8), BAD), (dict(gamma=3 * A), BAD),
    (dict(scales=(13 * A, 13 * A + 4 * ROWS)), OK), (dict(scales=(13 * A, 13 * A + 4 * ROWS - 4)), BAD),
    (dict(scales=(13 * A, 1 * A)), BAD), (dict(residual=3 * A), BAD),
    (dict(residual_out=1 * A), BAD), (dict(dtype=ccl.CCL_F32), OK), (dict(dtype=ccl.CCL_F16), OK),
])
def test_norm(front, change, want):
    check(front, norm(front, **change), want)


def test_norm_buffers(front):
    call = norm(front)
    check(front, call, BAD, "overlaps", outs=(1 * A, 4 * A))                      # in place
    check(front, call, BAD, "overlaps", outs=(2 * A + IN_BYTES - 1, 4 * A))
    check(front, call, OK, outs=(2 * A + IN_BYTES, 4 * A))
    check(front, call, BAD, "overlaps", outs=(3 * A, 3 * A + NORM_OUT - 1))
    check(front, call, OK, outs=(3 * A, 3 * A + NORM_OUT))
    check(front, call, OK, ins=(1 * A, 1 * A))                                     # two ranks that read one buffer
    check(front, call, BAD, "aligned", ins=(1 * A + 1, 2 * A))
    assert status(front, norm(front, rows=0)) == (OK, 0)
    assert front.ccl_allreduce_residual_rmsnorm_e4m3(None, 2, 1, 8, A, A, A, None, 0, 0.0, 1, None) == BAD


@pytest.mark.parametrize("change, want", [
    (dict(), OK), (dict(experts=0), BAD), (dict(experts=4096), OK), (dict(experts=4097), UNSUPPORTED), (dict(k=0), BAD),
    (dict(k=4097), BAD), (dict(k=EXPERTS + 1), OK), (dict(rows=(1 << 30) // K + 1), BAD), (dict(capacity=0), OK),
    (dict(capacity=1 << 30), BAD), (dict(ids=None), BAD), (dict(ids=(10 * A, 0)), BAD), (dict(ids=(10 * A, 11 * A + 1)), BAD),
    (dict(valid=None), OK), (dict(valid=(0, 13 * A)), BAD), (dict(valid=(12 * A + 1, 13 * A)), OK), (dict(slots=None), BAD),
    (dict(slots=(14 * A, 14 * A)), BAD), (dict(slots=(10 * A, 15 * A)), BAD), (dict(slots=(14 * A + 2, 15 * A)), BAD),
    (dict(offsets=0), BAD), (dict(offsets=16 * A + 2), BAD), (dict(offsets=14 * A), BAD), (dict(offsets=12 * A), BAD),
    (dict(ids=(10 * A, 10 * A)), OK), (dict(slots=(14 * A, 14 * A + ROWS * K * 4 - 4)), BAD),
    (dict(slots=(14 * A, 14 * A + ROWS * K * 4)), OK), (dict(rows=0, ids=None, slots=None, valid=None), OK),
])
def test_sort(front, change, want):
    check(front, sort(front, **change), want)


@pytest.mark.parametrize("name", ["dispatch", "combine", "grad"])
@pytest.mark.parametrize("change, want", [
    (dict(), OK), (dict(dtype=7), BAD), (dict(hidden=0), BAD), (dict(hidden=1 << 61), UNSUPPORTED), (dict(hidden=(1 << 30) + 1), UNSUPPORTED), (dict(k=0), BAD),
    (dict(k=4097), BAD), (dict(rows=(1 << 30) // K + 1), BAD), (dict(capacity=1 << 30), BAD), (dict(capacity=0), OK),
    (dict(slots=None), BAD), (dict(slots=(10 * A, 0)), BAD), (dict(slots=(10 * A, 11 * A + 2)), BAD),
    (dict(weights=None), OK), (dict(weights=(12 * A, 0)), BAD), (dict(weights=(12 * A + 1, 13 * A)), BAD),
    (dict(slots=(10 * A, 10 * A)), OK), (dict(slots=(3 * A, 11 * A)), BAD), (dict(weights=(4 * A, 13 * A)), BAD),
    (dict(dtype=ccl.CCL_I32), UNSUPPORTED), (dict(dtype=ccl.CCL_F32), OK), (dict(hidden=23), OK),
])
def test_rows(front, name, change, want):
    check(front, move(front, name, **change), want)


def test_rows_more(front):
    check(front, move(front, "dispatch", dtype=ccl.CCL_I32, weights=None), OK)
    check(front, move(front, "combine", dtype=ccl.CCL_I32, weights=None), UNSUPPORTED)
    check(front, move(front, "grad", dtype=ccl.CCL_I32, weights=None), UNSUPPORTED)
    for change in (dict(experts=None), dict(experts=(14 * A, 0)), dict(experts=(14 * A + 1, 15 * A)), dict(experts=(3 * A, 15 * A)),
                   dict(dweights=None), dict(dweights=(16 * A, 0)), dict(dweights=(16 * A, 16 * A)),
                   dict(dweights=(16 * A, 12 * A)), dict(dweights=(16 * A, 1 * A)), dict(dweights=(16 * A + 2, 17 * A))):
        check(front, move(front, "grad", **change), BAD)
    tokens, experts = ROWS * HIDDEN * 2, CAPACITY * HIDDEN * 2
    for name, own_in, own_out in (("dispatch", tokens, experts), ("combine", experts, tokens), ("grad", tokens, experts)):
        call = move(front, name)
        check(front, call, BAD, "overlaps", outs=(1 * A, 4 * A))
        check(front, call, BAD, "overlaps", outs=(3 * A, 3 * A + own_out - 2))
        check(front, call, OK, outs=(3 * A, 3 * A + own_out))
        check(front, call, BAD, "overlaps", outs=(2 * A + own_in - 2, 4 * A))
        check(front, call, OK, outs=(2 * A + own_in, 4 * A))
        check(front, call, BAD, "aligned", ins=(1 * A + 1, 2 * A))
        check(front, call, BAD, "aligned", outs=(3 * A + 1, 4 * A))
        assert status(front, move(front, name, rows=0, slots=None)) == (OK, 0)


@pytest.mark.parametrize("name", ["norm", "clip"])
def test_grads(front, name):
    check(front, grads(front, name), OK)                                          # no tensor: the norm of nothing
    check(front, grads(front, name, tensor()), OK)
    check(front, grads(front, name, count=1), BAD, "NULL")
    check(front, grads(front, name, tensor(), at=0), BAD, "NULL")
    check(front, grads(front, name, tensor(), at=20 * A + 2), BAD, "aligned")
    check(front, grads(front, name, tensor(), count=1 << 40), BAD, "count")
    check(front, grads(front, name, tensor(at=0)), BAD, "tensor 0 is NULL")
    check(front, grads(front, name, tensor(at=0, out=0, n=0)), OK)
    check(front, grads(front, name, tensor(), tensor(at=12 * A + 1, out=13 * A)), BAD, "tensor 1 is not aligned")
    check(front, grads(front, name, tensor(dtype=ccl.CCL_I32)), UNSUPPORTED)
    check(front, grads(front, name, tensor(dtype=5)), BAD, "dtype")
    check(front, grads(front, name, tensor(n=(1 << 40) + 1)), BAD, "2^40")
    check(front, grads(front, name, tensor(at=1 << 48, n=1 << 39, out=1 << 50), tensor(at=1 << 51, out=1 << 52, n=(1 << 39) + 1)), BAD, "2^40")
    check(front, grads(front, name, tensor(), at=10 * A + 8), BAD, "norm overlaps")
    check(front, grads(front, name, tensor(n=100), at=10 * A + 200), OK)


def test_clip(front):
    for bad in (-1.0, NAN, INF):
        check(front, grads(front, "clip", tensor(), max_norm=bad), BAD, "max_norm")
    check(front, grads(front, "clip", tensor(), max_norm=0.0), OK)
    check(front, grads(front, "clip", tensor(out=0)), BAD, "NULL")
    check(front, grads(front, "clip", tensor(out=11 * A + 1)), BAD, "aligned")
    check(front, grads(front, "clip", tensor(), at=11 * A), BAD, "norm overlaps")
    check(front, grads(front, "clip", tensor(out=10 * A)), OK)                    # in place
    check(front, grads(front, "clip", tensor(out=10 * A + 2)), BAD, "overlaps")
    check(front, grads(front, "clip", tensor(out=10 * A + 198)), BAD, "overlaps")
    check(front, grads(front, "clip", tensor(out=10 * A + 200)), OK)
    a = tensor(out=10 * A)
    check(front, grads(front, "clip", a, a), BAD, "overlaps")                     # a tensor twice
    check(front, grads(front, "norm", a, a), OK)
    check(front, grads(front, "clip", a, tensor(at=10 * A + 200, out=10 * A + 200)), OK)
    check(front, grads(front, "clip", a, tensor(at=10 * A + 198, out=10 * A + 198)), BAD, "overlaps")
    check(front, grads(front, "clip", tensor(), tensor(at=12 * A, out=10 * A)), BAD, "overlaps")
    check(front, grads(front, "clip", tensor(), tensor(at=12 * A, out=11 * A)), BAD, "overlaps")
    check(front, grads(front, "clip", tensor(), tensor(at=10 * A, out=12 * A)), OK)   # one gradient read twice


@pytest.mark.parametrize("n", [3, 40, 100, 1000])
def test_clip_of_many(front, n):
    """Tensors in any order, next to each other or not."""
    import random
    for gap in (0, 2, 600):
        at = [(1 << 30) + i * (200 + gap) for i in range(n)]
        out = [(1 << 40) + i * (200 + gap) for i in range(n)]
        for seed in (0, 1):
            order = list(range(n))
            if seed:
                random.Random(n).shuffle(order)
            ts = [tensor(at=at[i], out=out[i]) for i in order]
            check(front, grads(front, "clip", *ts), OK)
            check(front, grads(front, "clip", *[tensor(at=at[i], out=at[i]) for i in order]), OK)
            j = n // 2
            ts[j] = tensor(at=at[order[j]], out=out[order[(j + 1) % n]] + 2)
            check(front, grads(front, "clip", *ts), BAD, "overlaps")
            ts[j] = tensor(at=at[order[j]], out=at[order[0]] + 198)
            check(front, grads(front, "clip", *ts), BAD, "overlaps")
