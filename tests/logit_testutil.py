"""Helpers for the tests of the logit operators: rank buffers with guard
bands, made from a [rows, columns] matrix, at any stride and offset."""
from __future__ import annotations

import numpy as np
import torch

import reducescatter_reduction_gb300 as ccl

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# the largest relative error of one rounding to the type
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
U32 = 2.0 ** -24
# half the spacing of the type's subnormal numbers: the absolute error of a rounding below the normal range (bf16 and
# fp32: 2^x is flushed to zero there, an error of up to the smallest normal number)
FLOOR = {"f32": 2.0 ** -125, "f16": 2.0 ** -25, "bf16": 2.0 ** -125}
GUARD = 512


def widths(n, p):
    return [n // p + (1 if r < n % p else 0) for r in range(p)]


class Buffer:
    """[rows, width] elements, row stride ld, `offset` elements past a 16-byte boundary, NaN around and between."""

    def __init__(self, rows, width, dtype, ld=0, offset=0, values=None):
        self.rows, self.width, self.ld = rows, width, ld or width
        size = max(0, (rows - 1) * self.ld + width) if rows else 0
        self.raw = torch.full((GUARD + offset + size + GUARD,), float("nan"), dtype=TORCH[dtype], device="cuda")
        self.start = GUARD + offset
        flat = self.raw[self.start:]
        self.view = flat.as_strided((rows, width), (self.ld, 1))
        if values is not None and values.numel():
            self.view.copy_(values)

    def ptr(self):
        return self.raw.data_ptr() + self.start * self.raw.element_size()

    def outside_untouched(self):
        seen = self.raw.clone()
        seen[self.start:].as_strided((self.rows, self.width), (self.ld, 1)).fill_(float("nan"))
        return bool(torch.isnan(seen).all())


class Ranks:
    """A communicator over p buffers and their outputs (or in place)."""

    def __init__(self, parts, dtype, ld=0, offset=0, out_offset=None, in_place=False):
        self.dtype = dtype
        offsets = offset if isinstance(offset, (list, tuple)) else [offset] * len(parts)
        self.ins = [Buffer(*t.shape, dtype, ld, o, t) for t, o in zip(parts, offsets)]
        if in_place:
            self.outs = self.ins
        else:
            outs = offsets if out_offset is None else [out_offset] * len(parts)
            self.outs = [Buffer(*t.shape, dtype, ld, o) for t, o in zip(parts, outs)]
        self.before = [b.raw.clone() for b in self.ins]
        self.comm = ccl.ccl_comm_create(len(parts), [b.ptr() for b in self.ins])
        ccl.ccl_comm_set_outputs(self.comm, [b.ptr() for b in self.outs])

    def output(self):
        return [b.view.double() for b in self.outs]

    def finish(self, wrote=True):
        """Synchronises; the guards are whole, the inputs unchanged, nothing recorded."""
        torch.cuda.synchronize()
        ccl.ccl_comm_check(self.comm)
        assert all(b.outside_untouched() for b in self.ins + self.outs)
        if self.outs is not self.ins:
            for b, old in zip(self.ins, self.before):
                bits = torch.int32 if b.raw.element_size() == 4 else torch.int16
                assert torch.equal(b.raw.view(bits), old.view(bits))
            if not wrote:
                assert all(bool(torch.isnan(b.raw).all()) for b in self.outs)
        ccl.ccl_comm_destroy(self.comm)


def shards(full, p):
    return list(full.split(widths(full.shape[1], p), dim=1))


def stream():
    return torch.cuda.current_stream().cuda_stream


def ptr(t):
    return 0 if t is None else t.data_ptr()


def assert_within(got, want, tol, what=""):
    """Infinities and NaN in the same places; finite values within tol."""
    got, want = got.double().cpu(), want.double().cpu()
    tol = torch.as_tensor(tol, dtype=torch.float64).cpu().expand_as(want)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: infinities"
    err = (got - want).abs()[fine]
    bad = err > tol[fine]
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst "
                                 f"{float((err / tol[fine]).max())} times the tolerance")


def rng(seed):
    return np.random.default_rng(seed)
