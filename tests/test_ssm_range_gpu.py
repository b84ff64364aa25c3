"""The range of values of gdr_ssm_forward by chunks: at decays just within the reference's range, where
a chunk's outputs are held times 2^80 and its state times 2^-80 for a while, and just beyond."""
import pytest
import torch

from channelwise_gated_delta_gb300 import (GDR_FLAG_FORCE_GENERIC, gdr_device_check, gdr_flag_segments,
                                           gdr_ssm_forward)
from oracle import layer_ops
from tests.layer_util import ROUND, f64, near
from tests.test_ssm_gpu import CHUNKS, READ, WALK

pytestmark = pytest.mark.gpu

T, D = 160, 128                       # two chunks and a half
WITHIN, BEYOND = 158.0, 164.0         # a chunk's decay in powers of two


def draw(decay, x=1.0, h0=1.0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    bf = lambda t: t.bfloat16().cuda()
    step = 0.01
    a = -decay / 64 * 0.6931471805599453 / step
    return dict(x=bf(x * n(T, 2, D).clamp(-4, 4)), b=bf(n(T, 1, D).clamp(-2, 2)), c=bf(n(T, 1, D).clamp(-2, 2)),
                dt=torch.full((T, 2), step).cuda(), a=torch.full((2,), a).cuda(), d=torch.ones(2).cuda(), z=None,
                dt_bias=None, h0=(h0 * n(1, 2, D, D)).cuda())


def reference(d, unit, read):
    r = {k: None if v is None else f64(v[0] if k == "h0" else v) for k, v in d.items()}
    return layer_ops.ssm(**r, softplus=False, unit=unit, read=read)


def run(d, flags=0):
    out, ht = gdr_ssm_forward(**d, softplus=False, cu_seqlens=[0, T], flags=flags)
    gdr_device_check()
    return out, ht[0]


@pytest.mark.parametrize("decay", [1.0, 100.0, WITHIN, BEYOND])
@pytest.mark.parametrize("x,h0", [(2.0 ** 44, 1.0), (1.0, 2.0 ** -40), (2.0 ** -40, 2.0 ** -40),
                                  (2.0 ** 44, 2.0 ** 44)])
@pytest.mark.parametrize("flags", [0, gdr_flag_segments(2)])
def test_values_within_the_range(decay, x, h0, flags):
    """|x| up to 2^46 and (|c . b| step + |D|) up to 1 + 0.01 * 128 * 4 / 8: sums below 2^47."""
    d = draw(decay, x, h0)
    out, ht = run(d, flags)
    ref, S, err, E = reference(d, CHUNKS, READ["bf16"])
    near("out", out, ref, err, "bf16")
    near("ht", ht, S, E, "f32")


@pytest.mark.parametrize("x", [2.0 ** 49, 2.0 ** 70, 2.0 ** 110])
def test_large_values(x):
    """Beyond the range an output is right or not finite; the state and what runs token by token, or
    beyond the decays of the reference, are right.  (The last half chunk decays by half of BEYOND:
    2^-82, within the reference's range, which ends at values of 2^86 there.)"""
    d = draw(WITHIN, x)
    out, ht = run(d)
    ref, S, err, E = reference(d, CHUNKS, READ["bf16"])
    near("ht", ht, S, E, "f32")
    fine = torch.isfinite(out)
    keep = f64(fine) > 0
    near("finite outputs", out[fine], ref[keep], err[keep], "bf16")
    out, ht = run(d, GDR_FLAG_FORCE_GENERIC)
    ref, S, err, E = reference(d, WALK, 0.0)
    near("out token by token", out, ref, err, "bf16")
    near("ht token by token", ht, S, E, "f32")
    d = draw(BEYOND, x)
    out, ht = run(d)
    ref, S, err, E = reference(d, CHUNKS, READ["bf16"])
    near("out beyond", out[:128], ref[:128], err[:128], "bf16")
    fine = torch.isfinite(out)
    keep = f64(fine) > 0
    assert keep[:128].all()
    near("finite outputs of the last half", out[fine], ref[keep], err[keep], "bf16")
    near("ht beyond", ht, S, E, "f32")


def test_small_states():
    """Elements below 2^-46 may count as zeros in the outputs; the state keeps them."""
    d = draw(WITHIN, 2.0 ** -50, 2.0 ** -50)
    out, ht = run(d)
    ref, S, err, E = reference(d, CHUNKS, READ["bf16"])
    near("ht", ht, S, E, "f32")
    lost = 2.0 ** -46 * abs(f64(d["c"])).sum(-1)[..., None]
    off = abs(f64(out) - ref)
    assert (off <= err + ROUND["bf16"] * abs(ref) + lost).all()
