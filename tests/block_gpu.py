"""Inputs and comparisons of the GPU tests of a sequence block's operators."""
from __future__ import annotations

import numpy as np
import torch

import block_util as K

DT = {"f64": torch.float64, "f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def unit_of(dtype):
    return K.U64 if dtype == "f64" else K.U32


def own_of(dtype):
    return torch.float64 if dtype == "f64" else torch.float32


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


class make:
    """Normal tensors of a type: r(*shape) of the sequences', r.own(*shape) of the
    parameters'."""

    def __init__(self, seed, dtype):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype = dtype

    def _randn(self, *shape):
        return torch.randn(*shape, device="cuda", generator=self.g, dtype=torch.float64)

    def __call__(self, *shape, strided=False):
        if strided:  # a slice of a wider tensor, 24 elements further in each row
            wide = self._randn(*shape[:-1], shape[-1] + 24).to(DT[self.dtype])
            return wide[..., 8:8 + shape[-1]]
        return self._randn(*shape).to(DT[self.dtype])

    def own(self, *shape):
        return self._randn(*shape).to(own_of(self.dtype))


def offsets_of(lengths, lead):
    if lengths is None:
        return None, lead[0]
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    return torch.from_numpy(off).cuda(), len(lengths)


def check(got, want):
    for name, t in got.items():
        if t is None:
            continue
        v, bound = want[name]
        g = np64(t)
        assert g.shape == v.shape, (name, g.shape, v.shape)
        off = np.abs(g - v) > bound
        assert np.isfinite(g).all() and not off.any(), \
            (name, int(off.sum()), g.size, float((np.abs(g - v) / bound).max()))
