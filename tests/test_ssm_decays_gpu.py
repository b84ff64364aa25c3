"""gdr_ssm_forward by chunks where single tokens decay by far more than those around them: a state that
is dropped within a chunk, and what the slow tokens behind make of it."""
import pytest
import torch

from channelwise_gated_delta_gb300 import gdr_device_check, gdr_flag_segments, gdr_ssm_forward
from tests.test_ssm_gpu import CHUNKS, check

pytestmark = pytest.mark.gpu

T, HK, HV = 190, 1, 4
# tokens of a head that drop the state: first and last of a half, some in between, two in one half
DROPS = [(5,), (31, 96), (32, 63, 127), (0, 10, 45, 50, 150)]


def dropping(nats, dk, dv, x_there, a=1.0, seed=0):
    """Decays of some 0.05 nats a token but for those of DROPS.  Those add x_there times what stands in x."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    dt = 0.05 * (0.5 + torch.rand(T, HV, generator=gen))
    x = n(T, HV, dv)
    for h, tokens in enumerate(DROPS):
        for t in tokens:
            dt[t, h] = nats
            x[t, h] *= x_there
    bf = lambda t: t.bfloat16().cuda()
    return dict(x=bf(x), b=bf(n(T, HK, dk)), c=bf(n(T, HK, dk)), dt=(dt / a).cuda(), a=torch.full((HV,), -a).cuda(),
                d=None, z=None, dt_bias=None, h0=n(1, HV, dk, dv).cuda())


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 32)])
@pytest.mark.parametrize("nats", [100.0, 1e3, 1e4, 1e5, 1e6, 1e8, 3e38])
@pytest.mark.parametrize("flags", [0, gdr_flag_segments(2)])
def test_tokens_that_drop_the_state(dk, dv, nats, flags):
    """The pairs of tokens behind such a one keep their own decay, which is none of its digits: the
    tolerance is that of every other chunk.  (3e38 nats are infinite in log2 units.)"""
    d = dropping(nats, dk, dv, 0.0 if nats > 1e4 else 1.0 / nats, a=1e20 if nats > 1e30 else 1.0)
    out, ht = gdr_ssm_forward(**d, softplus=False, cu_seqlens=[0, T], flags=flags)
    gdr_device_check()
    check(d, [T], out, ht, "bf16", CHUNKS, softplus=False)


def test_drops_in_every_place_of_a_chunk():
    """One head a place: the outputs behind the drop are those of the sequence that starts there."""
    n, D = 64, 64
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()
    x, b, c = r(n, 1, D).expand(n, 64, D).contiguous(), r(n, 1, D), r(n, 1, D)
    dt = torch.full((n, 64), 0.03).cuda()
    places = torch.arange(64, device="cuda")
    dt[places, places] = 1e7
    x[places, places] = 0
    out, ht = gdr_ssm_forward(x, b, c, dt, -torch.ones(64).cuda(), softplus=False, cu_seqlens=[0, n])
    plain = torch.full((n, 64), 0.03).cuda()
    for p in (0, 1, 15, 16, 30, 31, 32, 33, 47, 48, 62):
        rest = slice(p + 1, n)
        want, end = gdr_ssm_forward(x[rest, p:p + 1].contiguous(), b[rest], c[rest], plain[rest, :1].contiguous(),
                                    -torch.ones(1).cuda(), softplus=False, cu_seqlens=[0, n - p - 1])
        # both are the same sums but for their order, and rounded once
        scale = want.float().abs().amax(0)
        assert ((out[rest, p] - want[:, 0]).float().abs() <= 2.0 ** -7 * scale).all(), p
        assert (ht[0, p] - end[0, 0]).abs().max() <= 2.0 ** -15 * end.abs().max(), p


@pytest.mark.parametrize("flags", [0, gdr_flag_segments(2)])
def test_steps_of_both_signs(flags):
    """Without softplus a step may be negative: a token that grows the state and takes from it."""
    d = dropping(3.0, 128, 64, 0.5, seed=3)
    gen = torch.Generator().manual_seed(4)
    d["dt"] *= torch.where(torch.rand(T, HV, generator=gen) < 0.4, -1.0, 1.0).cuda()
    out, ht = gdr_ssm_forward(**d, softplus=False, cu_seqlens=[0, T], flags=flags)
    gdr_device_check()
    check(d, [T], out, ht, "bf16", CHUNKS, softplus=False)
    # decays and growths of some 1.5 nats, 0.3 a token on the whole: chunks near the reference's range
    # and beyond.  (The tokens of DROPS decay: 90 nats of growth would be no float32 number.)
    d["dt"] = torch.where(d["dt"].abs() < 1, 30 * d["dt"], d["dt"].abs())
    out, ht = gdr_ssm_forward(**d, softplus=False, cu_seqlens=[0, T], flags=flags)
    gdr_device_check()
    check(d, [T], out, ht, "bf16", CHUNKS, softplus=False)
