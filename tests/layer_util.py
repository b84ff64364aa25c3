"""Shared by the tests of the operators around the recurrence."""
import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}     # the output's own rounding


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def near(name, got, ref, err, dtype, top=1.0):
    """Element by element: the error of the evaluation, then one rounding to the output's type."""
    got = f64(got)
    assert got.shape == ref.shape, name
    assert np.isfinite(got).all(), name
    u = ROUND[dtype]
    tol = err * (1 + u) + u * np.abs(ref) + 2.0 ** -126
    off = np.abs(got - ref) / tol
    assert off.size == 0 or off.max() <= top, "%s: %.3g of its tolerance at %s" % (
        name, off.max(), np.unravel_index(off.argmax(), off.shape))


def spread(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu
