"""gdr_short_conv against its definition in float64."""
import numpy as np
import pytest
import torch

from channelwise_gated_delta_gb300 import gdr_short_conv
from oracle import layer_ops
from tests.layer_util import DT, f64, near, spread

pytestmark = pytest.mark.gpu


def draw(lens, D, W, dtype, wide=0, seed=0, state=True, bias=True):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    dt = DT[dtype]
    x = n(sum(lens), D + wide).to(dt).cuda()[:, wide // 2:wide // 2 + D]
    return dict(x=x, weight=(0.5 * n(D, W)).cuda(), bias=n(D).cuda() if bias else None,
                s0=n(len(lens), W - 1, D).to(dt).cuda() if state else None)


def check(d, lens, out, st, dtype, silu):
    cu = spread(lens)
    out = out.reshape(-1, out.shape[-1])
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        s0 = None if d["s0"] is None else f64(d["s0"][i])
        ref, state, err = layer_ops.short_conv(f64(d["x"][a:b]), f64(d["weight"]), f64(d["bias"]),
                                               s0, silu)
        near("out[%d]" % i, out[a:b], ref, err, dtype)
        if st is not None:
            assert np.array_equal(f64(st[i]), state), "state[%d]" % i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D,wide", [(1, 0), (8, 0), (64, 64), (257, 0), (520, 3), (1032, 8)])
def test_packed(dtype, W, D, wide):
    lens = [0, 1, 2, 3, 4, 0, 5, 64, 65, 150, 0]
    d = draw(lens, D, W, dtype, wide, seed=D + W)
    for silu in (True, False):
        out, st = gdr_short_conv(**d, cu_seqlens=spread(lens), silu=silu)
        check(d, lens, out, st, dtype, silu)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 8192), (3, 1, 40), (300, 1, 64), (2, 2, 33), (2, 700, 96),
                                   (1, 5, 4096), (2, 0, 16), (0, 3, 16)])
def test_dense(dtype, B, T, D):
    for state, bias in ((True, False), (False, True)):
        d = draw([T] * B, D, 4, dtype, wide=16, seed=T, state=state, bias=bias)
        x = torch.empty(B, T, D + 16, dtype=DT[dtype], device="cuda")[..., :D]
        x.copy_(d["x"].reshape(B, T, D))
        out, st = gdr_short_conv(x, d["weight"], d["bias"], s0=d["s0"])
        check(d, [T] * B, out, st, dtype, True)


def test_many_sequences():
    """More sequences than a launch's table holds."""
    lens = [(7 * i) % 5 for i in range(700)]
    d = draw(lens, 24, 3, "bf16")
    out, st = gdr_short_conv(**d, cu_seqlens=spread(lens))
    check(d, lens, out, st, "bf16", True)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f32", 37)])
@pytest.mark.parametrize("W", [2, 4])
def test_pieces_equal_the_whole(dtype, D, W):
    """A sequence in pieces, the state handed on in place, bit for bit."""
    d = draw([300], D, W, dtype)
    whole, end = gdr_short_conv(d["x"][None], d["weight"], d["bias"], s0=d["s0"])
    state, at, parts = d["s0"].clone(), 0, []
    for n in (1, 1, 1, 2, 1, 3, 64, 70, 157):
        out, st = gdr_short_conv(d["x"][None, at:at + n], d["weight"], d["bias"], s0=state, st=state)
        assert st is state
        parts.append(out)
        at += n
    assert at == 300 and torch.equal(torch.cat(parts, 1), whole) and torch.equal(state, end)


def test_given_outputs_and_rows_behind():
    """Outputs that are parts of a wider tensor, in front of which and behind which nothing changes."""
    d = draw([9, 0, 40], 64, 4, "bf16")
    wide = torch.full((49 + 3, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    out, st = gdr_short_conv(**d, cu_seqlens=[0, 9, 9, 49], out=wide[:49, 16:80], store_st=False)
    assert st is None
    check(d, [9, 0, 40], out, None, "bf16", True)
    assert (wide[:, :16] == 7).all() and (wide[:, 80:] == 7).all() and (wide[49:] == 7).all()


def test_extreme_values():
    """Infinities and NaN reach the W rows that look at them, and no others."""
    d = draw([40], 16, 4, "f32", state=False, bias=False)
    x = d["x"].clone()
    x[10, 3], x[20, 5], x[30, 7] = float("nan"), float("inf"), -1e30
    out, _ = gdr_short_conv(x[None], d["weight"].abs() + 0.1)
    plain, _ = gdr_short_conv(d["x"][None], d["weight"].abs() + 0.1)
    bad = torch.zeros(40, 16, dtype=torch.bool, device="cuda")
    bad[10:14, 3] = bad[20:24, 5] = bad[30:34, 7] = True
    assert torch.equal(out[0][~bad], plain[0][~bad])
    assert out[0, 10:14, 3].isnan().all() and (out[0, 20:24, 5] == float("inf")).all()
    assert (out[0, 30:34, 7] == 0).all()
