"""What the logit operators refuse, tested without a GPU: the library's host
front end (csrc/logits.cpp) is compiled against fakes of the CUDA runtime and
of the kernel launchers.  Each case starts from arguments that are accepted
and changes one thing."""
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
P, ROWS, VOCAB = 2, 4, 11          # shards of 6 and 5 columns
A = 1 << 20                        # distance between the buffers' made-up addresses


@pytest.fixture(scope="module")
def front(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("logit_checks") / "driver.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC",
                    "-Wl,-Bsymbolic",      # the driver's own fakes, whatever CUDA runtime the process has loaded
                    "-I", os.path.join(ROOT, "include"), "-I", CUDA,
                    os.path.join(ROOT, "tests", "logit_checks", "driver.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    real = ccl._lib
    ccl._lib = None
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    pvp = ctypes.POINTER(vp)
    L.fake_comm.restype, L.fake_comm.argtypes = vp, [i, pvp, pvp]
    L.fake_comm_free.argtypes = [vp]
    L.fake_message.restype = ctypes.c_char_p
    L.ccl_logit_rules.argtypes = [vp, i, sz, sz, sz, ctypes.POINTER(ccl.LogitRules), vp]
    L.ccl_distill_topk.argtypes = [vp, i, i, sz, sz, sz, sz, vp, vp, i, ctypes.c_float, vp, vp, vp, vp]
    L.ccl_balance_loss.argtypes = [vp, i, i, sz, sz, sz, pvp, pvp, ctypes.c_float, vp, vp, vp, vp, vp]
    ccl._lib = real
    return L


def pointers(values):
    return (ctypes.c_void_p * len(values))(*values)


def status(front, call, inputs=None, outputs=None):
    """(status, whether a kernel was launched) of one call."""
    c = front.fake_comm(P, pointers(inputs or [1 * A, 2 * A]), pointers(outputs or [3 * A, 4 * A]))
    before = front.fake_launches()
    try:
        return call(c), front.fake_launches() - before
    finally:
        front.fake_comm_free(c)


def rules_call(front, dtype=ccl.CCL_BF16, rows=ROWS, vocab=VOCAB, ld=0, rules=..., **change):
    r = ccl.LogitRules(repetition=10 * A, frequency=11 * A, presence=12 * A, history=13 * A, history_ld=7,
                       history_len=14 * A, prompt_len=15 * A, bias_offsets=16 * A, bias_tokens=17 * A,
                       bias_values=18 * A, bias_count=5, mask=19 * A, mask_rows=3, mask_ld=1, mask_index=20 * A)
    for k, v in change.items():
        setattr(r, k, v)
    return lambda c: front.ccl_logit_rules(c, dtype, rows, vocab, ld, ctypes.byref(r) if rules is ... else None, None)


def distill_call(front, dtype=ccl.CCL_BF16, steps=ccl.CCL_PASS_BOTH, rows=ROWS, vocab=VOCAB, ld=0, k=3, ids=10 * A,
                 teacher=11 * A, teacher_dtype=ccl.CCL_F32, temperature=1.0, weight=12 * A, loss=13 * A, stats=14 * A):
    return lambda c: front.ccl_distill_topk(c, dtype, steps, rows, vocab, ld, k, ids, teacher, teacher_dtype,
                                            temperature, weight, loss, stats, None)


def balance_call(front, dtype=ccl.CCL_BF16, steps=ccl.CCL_PASS_BOTH, rows=ROWS, experts=8, k=2, ids=(10 * A, 11 * A),
                 valid=(12 * A, 13 * A), coef=0.01, dloss=14 * A, counts=15 * A, tokens=16 * A, loss=17 * A):
    return lambda c: front.ccl_balance_loss(c, dtype, steps, rows, experts, k, None if ids is None else pointers(ids),
                                            None if valid is None else pointers(valid), coef, dloss, counts, tokens,
                                            loss, None)


CALLS = {"rules": rules_call, "distill": distill_call, "balance": balance_call}


@pytest.mark.parametrize("op", CALLS)
def test_accepted(front, op):
    assert status(front, CALLS[op](front)) == (OK, 1)
    assert not front.fake_alias()
    assert status(front, CALLS[op](front), outputs=[1 * A, 2 * A]) == (OK, 1)      # in place
    assert front.fake_alias()


@pytest.mark.parametrize("op", CALLS)
def test_shared_refusals(front, op):
    call = CALLS[op]
    assert call(front)(None) == BAD
    assert status(front, call(front, dtype=ccl.CCL_I32)) == (UNSUPPORTED, 0)
    for dtype in (-1, 4):
        assert status(front, call(front, dtype=dtype)) == (BAD, 0)
    assert status(front, call(front), inputs=[1 * A + 1, 2 * A]) == (BAD, 0)       # not aligned to bf16
    assert status(front, call(front), outputs=[3 * A, 4 * A + 1]) == (BAD, 0)
    assert status(front, call(front), outputs=[2 * A, 1 * A]) == (BAD, 0)          # another rank's input
    assert status(front, call(front), outputs=[1 * A + 4, 4 * A]) == (BAD, 0)      # partly its own input
    assert status(front, call(front), outputs=[3 * A, 3 * A + 8]) == (BAD, 0)      # two outputs
    assert status(front, call(front, rows=1 << 62)) == (BAD, 0)


@pytest.mark.parametrize("change,want", [
    (dict(rules=None), BAD), (dict(vocab=0), BAD), (dict(vocab=(1 << 30) + 1), BAD), (dict(ld=5), BAD),
    (dict(ld=6), OK), (dict(ld=1 << 62), BAD), (dict(rows=0), OK),
    (dict(history=0), BAD), (dict(history=0, history_ld=0), OK), (dict(history_ld=1 << 30), BAD),
    (dict(bias_tokens=0), BAD), (dict(bias_values=0), BAD), (dict(bias_offsets=0), BAD),
    (dict(bias_offsets=0, bias_tokens=0, bias_values=0, bias_count=0), OK),
    (dict(mask_ld=0), BAD), (dict(mask_index=0), BAD), (dict(mask_index=0, mask_rows=ROWS), OK),
    (dict(mask=0, mask_rows=0, mask_ld=0), OK), (dict(mask_rows=1 << 62), BAD), (dict(mask_rows=0), OK),
    (dict(frequency=11 * A + 2), BAD), (dict(history=13 * A + 1), BAD), (dict(mask=19 * A + 2), BAD),
    (dict(bias_count=1 << 31), BAD),
    (dict(repetition=3 * A), BAD), (dict(history=4 * A), BAD), (dict(mask=3 * A + 16), BAD),   # over an output
    (dict(history_len=1 * A), OK),                                                            # shares an input: both read
])
def test_rules(front, change, want):
    assert status(front, rules_call(front, **change)) == (want, int(want == OK and change != dict(rows=0)))


@pytest.mark.parametrize("change,want", [
    (dict(steps=0), BAD), (dict(steps=4), BAD), (dict(vocab=0), BAD), (dict(vocab=(1 << 30) + 1), BAD),
    (dict(ld=5), BAD), (dict(ld=6), OK), (dict(rows=0), OK), (dict(k=0), BAD), (dict(k=1024), OK),
    (dict(k=1025), UNSUPPORTED), (dict(teacher_dtype=ccl.CCL_I32), BAD), (dict(teacher_dtype=-1), BAD),
    (dict(temperature=0.0), BAD), (dict(temperature=-1.0), BAD), (dict(temperature=float("nan")), BAD),
    (dict(temperature=float("inf")), BAD), (dict(ids=0), BAD), (dict(teacher=0), BAD), (dict(loss=0), BAD),
    (dict(loss=0, steps=ccl.CCL_PASS_BACKWARD), OK), (dict(stats=0), OK), (dict(stats=0, steps=ccl.CCL_PASS_BACKWARD), BAD),
    (dict(weight=0), OK), (dict(ids=10 * A + 2), BAD), (dict(teacher=11 * A + 2), BAD),
    (dict(teacher=11 * A + 2, teacher_dtype=ccl.CCL_F16), OK), (dict(loss=13 * A + 2), BAD), (dict(stats=14 * A + 1), BAD),
    (dict(loss=14 * A), BAD), (dict(stats=10 * A), BAD), (dict(loss=1 * A), BAD), (dict(loss=3 * A), BAD),
    (dict(teacher=3 * A), BAD), (dict(teacher=3 * A, steps=ccl.CCL_PASS_FORWARD), OK),
    (dict(weight=3 * A, steps=ccl.CCL_PASS_FORWARD), OK), (dict(stats=3 * A, steps=ccl.CCL_PASS_BACKWARD), BAD),
])
def test_distill(front, change, want):
    assert status(front, distill_call(front, **change)) == (want, int(want == OK and change != dict(rows=0)))


@pytest.mark.parametrize("change,want", [
    (dict(steps=0), BAD), (dict(steps=4), BAD), (dict(experts=0), BAD), (dict(experts=4096), OK),
    (dict(experts=4097), UNSUPPORTED), (dict(k=0), BAD), (dict(k=8), OK), (dict(k=9), BAD),
    (dict(rows=1 << 30), BAD), (dict(coef=float("nan")), BAD), (dict(coef=float("inf")), BAD),
    (dict(ids=None), BAD), (dict(ids=(10 * A, 0)), BAD), (dict(ids=None, steps=ccl.CCL_PASS_BACKWARD), OK),
    (dict(valid=None), OK), (dict(valid=(0, 13 * A)), BAD), (dict(counts=0), BAD), (dict(tokens=0), BAD),
    (dict(loss=0), BAD), (dict(loss=0, steps=ccl.CCL_PASS_BACKWARD), OK), (dict(dloss=0), OK),
    (dict(counts=15 * A + 2), BAD), (dict(ids=(10 * A + 1, 11 * A)), BAD), (dict(valid=(12 * A + 1, 13 * A)), OK),
    (dict(counts=16 * A), BAD), (dict(loss=15 * A + 4), BAD), (dict(tokens=10 * A), BAD), (dict(counts=2 * A), BAD),
    (dict(counts=3 * A), BAD), (dict(valid=(3 * A, 13 * A)), BAD), (dict(valid=(3 * A, 13 * A), steps=ccl.CCL_PASS_FORWARD), OK),
    (dict(counts=3 * A, steps=ccl.CCL_PASS_BACKWARD), BAD), (dict(rows=0), OK),
])
def test_balance(front, change, want):
    assert status(front, balance_call(front, **change)) == (want, int(want == OK))


def test_no_rows_need_no_launch(front):
    assert status(front, balance_call(front, rows=0, steps=ccl.CCL_PASS_BACKWARD)) == (OK, 0)


def test_messages_name_the_argument(front):
    status(front, distill_call(front, k=1025))
    assert b"k=1025" in front.fake_message()
    status(front, balance_call(front, valid=(0, 13 * A)))
    assert b"valid[0]" in front.fake_message()
    status(front, rules_call(front, repetition=3 * A))
    assert b"repetition overlaps the output of rank 0" in front.fake_message()


def test_binding_refuses_lists_of_the_wrong_length(monkeypatch):
    class Lib:
        def ccl_comm_ranks(self, comm):
            return 3
    monkeypatch.setattr(ccl, "_lib", Lib())
    with pytest.raises(ccl.CclError, match="expert_ids has 2 pointers, p = 3"):
        ccl.ccl_balance_loss(1, "bf16", "both", 4, 8, 2, [16, 32], None, 0.01, 0, 16, 16, 16)
    with pytest.raises(ccl.CclError, match="valid has 4 pointers, p = 3"):
        ccl.ccl_balance_loss(1, "bf16", "both", 4, 8, 2, [16, 32, 48], [1, 2, 3, 4], 0.01, 0, 16, 16, 16)
