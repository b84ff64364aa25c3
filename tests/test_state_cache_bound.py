"""How far a value that went through the 8-bit cache may be off: what include/gdr.h states, held
against rows whose values lie next to the ties between two codes.

With e = 2^-24 the relative error of one float32 operation: the code is rounded from x (1 + 3 e) in
steps of the row's a / 127 (1 / a, times 127, times x), or x (1 + 6 e) where a > 2^126 and 1 / a is
subnormal, held to 2^-150; the scale is a / 127 (1 + 1.07 e), and the product brings one e more.  A
value of up to 127 steps is then off by half a step and 127 (6 + 1.07 + 1) e = 1026 e at most, and
2^-13 steps are 2048 e."""
import os
import re

import numpy as np
import pytest
import torch

from oracle import speculation

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gdr.h")
TOPS = {"ordinary": 2.0 ** np.linspace(-3, 3, 601), "large": 2.0 ** np.linspace(126, 127.99, 601),
        "small": 2.0 ** np.linspace(-99.6, -90, 601)}


def rows(tops):
    """One row per top: itself, and the floats around the ties below it; [1, n, dk 32, dv 128]."""
    out = []
    for top in np.float32(tops):
        ties = ((np.arange(1, 127) + 0.5) * float(top) / 127).astype(np.float32)
        for off in (-4, -2, -1, 0, 1, 2, 4, 6):
            near = np.minimum((ties.view(np.int32) + off).view(np.float32), top)
            out.append(np.r_[top, -near, np.float32(0)])
    out += [out[-1]] * (-len(out) % 32)
    return np.array(out, np.float32).reshape(1, -1, 32, 128)


def stated():
    """The header's bound: half a step and 2^-n of one, and rows that come back as zeros."""
    text = re.sub(r"\s*\n \* *", " ", open(HEADER).read())
    m = re.search(r"at most \(1/2 \+ 2\^-(\d+)\) times its row's scale, of a row with a <= (1e-\d+) "
                  r"its magnitude", text)
    assert m, "include/gdr.h does not state the cache's error"
    return 0.5 + 2.0 ** -int(m.group(1)), float(m.group(2))


@pytest.mark.parametrize("which", sorted(TOPS))
def test_the_stated_bound_holds_at_the_ties(which):
    x = rows(TOPS[which])
    codes, scale = speculation.quantise(x)
    err = np.abs(speculation.dequantise(codes, scale).astype(np.float64) - x)
    steps = err / scale[..., None].astype(np.float64)
    assert steps.max() <= stated()[0]
    assert steps.max() > 0.5          # half a step alone would not do


def test_rows_stored_as_zeros_are_off_by_their_magnitude():
    limit = np.float32(stated()[1])
    x = np.full((1, 1, 32, 32), limit, np.float32)
    codes, scale = speculation.quantise(x)
    assert not codes.any() and not scale.any()
    assert speculation.quantise(np.nextafter(x, np.float32(1)))[0].all()


@pytest.mark.gpu
@pytest.mark.parametrize("which", sorted(TOPS))
def test_the_kernels_round_these_rows_as_the_oracle_does(which):
    from channelwise_gated_delta_gb300 import gdr_state_cache, gdr_state_load, gdr_state_store
    x = rows(TOPS[which])
    cache, scale = gdr_state_cache(1, *x.shape[1:])
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdr_state_store(torch.from_numpy(x).cuda(), slot, cache, scale)
    codes, sc = speculation.quantise(x)
    assert np.array_equal(cache.cpu().numpy(), codes)
    assert np.array_equal(scale.cpu().numpy(), sc)
    back = gdr_state_load(cache, scale, slot).cpu().numpy()
    assert np.array_equal(back, speculation.dequantise(codes, sc))
