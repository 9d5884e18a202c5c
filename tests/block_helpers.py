"""Shared pieces of the training-block operators' GPU tests: inputs, types and
the error bounds, which follow from the arithmetic alone."""
import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# Unit roundoff of each type, and half the spacing of its subnormals.
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def f64(t):
    return t.detach().double().cpu().numpy()


def assert_close(got, exact, magnitude, adds, what):
    """|got - exact| <= adds fp32 roundings of the summed magnitudes (each at most
    2^-23 of them: half a unit, or a whole one for a truncating adder) + the
    rounding to got's type. Values beyond the type's range are infinities."""
    g = f64(got)
    assert not np.isnan(g).any(), what
    bound = adds * 2.0 ** -23 * magnitude
    bound = bound + ROUND[got.dtype] * (np.abs(exact) + bound) + TINY[got.dtype]
    top = torch.finfo(got.dtype).max
    inf = np.isinf(g)
    assert np.all(np.abs(exact[inf]) + bound[inf] > top) and np.all(np.sign(g[inf]) == np.sign(exact[inf])), what
    worst = np.max(np.abs(g - exact)[~inf] - bound[~inf], initial=-1.0)
    assert worst <= 0, f"{what}: {worst:.3g} over the bound"


def strided(rows, cols, pad, dtype, rng, scale=1.0):
    """A [rows, cols] view with `pad` columns between its rows; the gaps hold NaN."""
    full = torch.full((rows, cols + pad), float("nan"), dtype=dtype)
    full[:, :cols] = torch.from_numpy(rng.normal(size=(rows, cols)) * scale).to(dtype)
    return full.cuda()[:, :cols]
