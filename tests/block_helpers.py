"""Shared by the GPU tests of the rest of the block: inputs, and bounds that follow
from the roundings.

HALF[dtype] is the most that one rounding of an output may be off, relative to
the value: half of torch.finfo(dtype).eps."""
import numpy as np
import torch

import test_weight_mlp_amd as ip

BF16, F32 = ip.IPTTT_BF16, ip.IPTTT_F32
TDT = {BF16: torch.bfloat16, F32: torch.float32}
HALF = {d: torch.finfo(t).eps / 2 for d, t in TDT.items()}
E32 = 2.0 ** -24   # one fp32 rounding


def np64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, dt, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(TDT[dt])


def wide(dt, rows, cols, extra, fill=7.0):
    """A [rows, cols] slice of a tensor with `extra` more columns, half before and
    half after (multiples of 8), and a check that those still hold `fill`."""
    left = extra // 16 * 8
    t = torch.full((rows, cols + extra), fill, dtype=TDT[dt], device="cuda")

    def untouched():
        return bool((t[:, :left] == fill).all()) and bool((t[:, left + cols:] == fill).all())

    return t[:, left:left + cols], untouched


def within(got, want, bound):
    """Every element of `got` within `bound` (array or number) of `want`."""
    got, want = np64(got) if isinstance(got, torch.Tensor) else got, np.asarray(want)
    assert got.shape == want.shape and np.isfinite(got).all()
    over = np.abs(got - want) - bound
    assert over.max(initial=-1.0) <= 0, f"{(over > 0).sum()} of {over.size} are off by up to {np.abs(got - want).max()}"
