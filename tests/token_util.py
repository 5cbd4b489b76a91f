"""Device buffers for the token operators' GPU tests: tensors at chosen element
offsets inside a frame of sentinels, and their values as float64."""
from __future__ import annotations

import numpy as np
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODE = {"f32": 0, "bf16": 1, "f16": 2}
_BITS = {4: torch.int32, 2: torch.int16, 8: torch.int64}
_PAD = 64


class Framed:
    """A [rows][d] tensor with row stride ld, `offset` elements into its frame;
    what lies outside the rows has to keep its bits."""

    def __init__(self, rows, d, dtype, ld=None, offset=0, fill=None):
        self.ld = d if ld is None else ld
        n = (rows - 1) * self.ld + d if rows else 0
        size = torch.empty(0, dtype=dtype).element_size()
        self.bits = torch.full((n + 2 * _PAD + offset,), 0x55 if size == 2 else 0x5EADBEEF,
                               dtype=_BITS[size], device="cuda")
        flat = self.bits.view(dtype)
        self.view = flat[_PAD + offset:].as_strided((rows, d), (self.ld, 1))
        self.inside = torch.zeros_like(self.bits, dtype=torch.bool)
        self.inside[_PAD + offset:].as_strided((rows, d), (self.ld, 1)).fill_(True)
        if fill is not None:
            self.view.copy_(fill)
        self.before = self.bits.clone()

    def check(self, what="frame"):
        same = (self.bits == self.before) | self.inside
        assert bool(same.all()), f"{what}: written outside its rows"

    def f64(self):
        return self.view.double().cpu().numpy()


def f64(t):
    return t.detach().double().cpu().numpy()


def rounded(rng, shape, dtype, std=1.0):
    """Normal values as a CUDA tensor of the storage type."""
    a = torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32))
    return a.to(DT[dtype]).cuda()
