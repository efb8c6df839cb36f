"""Helpers for the tests of the operators around layers: device arrays with
guard bands, and the plain forms in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

import reducescatter_reduction_gb300 as ccl
from logit_testutil import FLOOR, HALF_STEP, TORCH, U32, assert_within, stream, widths  # noqa: F401

GUARD = 64


class Array:
    """A device array `offset` elements past a 16-byte boundary, between guards of a byte pattern."""

    def __init__(self, shape, dtype, offset=0, values=None, fill=0xA5):
        n = int(np.prod(shape))
        size = torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full(((GUARD + offset + n + GUARD) * size,), fill, dtype=torch.uint8, device="cuda")
        self.fill, self.lo, self.hi = fill, (GUARD + offset) * size, (GUARD + offset + n) * size
        self.t = self.raw[self.lo:self.hi].view(dtype).view(shape)
        if values is not None and n:
            self.t.copy_(values)

    def ptr(self):
        return self.raw.data_ptr() + self.lo

    def guarded(self):
        return bool((self.raw[:self.lo] == self.fill).all()) and bool((self.raw[self.hi:] == self.fill).all())


def ptrs(arrays):
    return None if arrays is None else [a.ptr() for a in arrays]


class Comm:
    """A communicator for a test; checks it at the end."""

    def __init__(self, ins, outs=None):
        self.arrays = list(ins) + list(outs or [])
        self.h = ccl.ccl_comm_create(len(ins), ptrs(ins))
        if outs is not None:
            ccl.ccl_comm_set_outputs(self.h, ptrs(outs))

    def __enter__(self):
        return self.h

    def __exit__(self, kind, value, trace):
        torch.cuda.synchronize()
        if kind is None:
            ccl.ccl_comm_check(self.h)
            assert all(a.guarded() for a in self.arrays)
        ccl.ccl_comm_destroy(self.h)


def sort_by_expert(ids, valid, experts, capacity):
    """(slots [p, rows, k], offsets [experts + p]) of numpy ids [p, rows, k], choice by choice."""
    p, rows, k = ids.shape
    owner = np.repeat(np.arange(p), widths(experts, p))
    fill = np.zeros(p, dtype=np.int64)
    slots = np.full((p, rows, k), -1, dtype=np.int32)
    offsets = []
    by_expert = [[] for _ in range(experts)]
    for r in range(p):
        for t in range(rows):
            if valid is not None and not valid[r, t]:
                continue
            for j in range(k):
                if 0 <= ids[r, t, j] < experts:
                    by_expert[ids[r, t, j]].append((r, t, j))
    e = 0
    for r in range(p):
        for _ in range(widths(experts, p)[r]):
            offsets.append(min(fill[r], capacity))
            for at in by_expert[e]:
                assert owner[e] == r
                if fill[r] < capacity:
                    slots[at] = r * capacity + fill[r]
                fill[r] += 1
            e += 1
        offsets.append(min(fill[r], capacity))
    return slots, np.array(offsets, dtype=np.int32)
