"""Helpers of the block operators' GPU tests: device copies, guarded output
buffers, and error bounds.

U = 2^-24 is half a step of fp32 relative to the value; HALF[t] that of each
output type."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}  # half a subnormal step, or less


def dev(a, dtype=None):
    """Host array on the device (fp32 unless a type is named; uint8 stays)."""
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a))
    if dtype is not None:
        return t.to("cuda", TORCH[dtype]).contiguous()
    return (t if t.dtype == torch.uint8 else t.float()).cuda()


def host(t) -> np.ndarray:
    """Exact float64 (codes: uint8) copy."""
    if t is None:
        return None
    t = t.detach().cpu()
    return t.numpy() if t.dtype == torch.uint8 else t.double().numpy()


class Guarded:
    """An output inside a larger buffer of a sentinel byte; `untouched()` says
    whether the bytes around it are still the sentinel."""

    def __init__(self, shape, dtype, pad=4096):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((n + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
        self.n, self.pad = n, pad
        self.t = self.raw[pad:pad + n].view(dtype).view(shape)

    def untouched(self) -> bool:
        return bool((self.raw[:self.pad] == 0xA5).all()) and bool((self.raw[self.pad + self.n:] == 0xA5).all())


def assert_within(got, ref, bound, dtype="f32", what=""):
    """|got - ref| <= bound + one rounding of the result to `dtype`, element by element."""
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    tol = bound + HALF[dtype] * (np.abs(ref) + bound) + TINY[dtype]
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / tol, 0)), got.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; at {i} got "
                             f"{got[i]!r}, expected {ref[i]!r}, bound {float(np.broadcast_to(tol, got.shape)[i])!r}")
