"""gdr_short_conv over as many rows as an int counts: the last rows of such a sequence."""
import pytest
import torch

from channelwise_gated_delta_gb300 import gdr_short_conv

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def rows():
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(MOST, 1, dtype=torch.bfloat16, device="cuda")
    for part in x.split(2 ** 28):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
    yield x, torch.empty_like(x)
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [MOST - 64, MOST - 63, MOST - 1, MOST])
@pytest.mark.parametrize("packed", [False, True])
def test_the_last_rows(rows, T, packed):
    x, out = rows[0][:T], rows[1][:T]
    w = torch.tensor([[0.5, -0.25, 1.0, 0.75]], device="cuda")
    out.fill_(float("nan"))
    if packed:
        _, st = gdr_short_conv(x, w, cu_seqlens=[0, 3, T], out=out)
    else:
        _, st = gdr_short_conv(x[None], w, out=out[None])
    for part in out.split(2 ** 28):
        assert torch.isfinite(part).all()
    for a, b in ((T - 300, T), (2 ** 30 - 100, 2 ** 30 + 100)):
        want, _ = gdr_short_conv(x[None, a:b], w, s0=x[None, a - 3:a].contiguous())
        assert torch.equal(out[a:b], want[0]), (a, b)
    assert torch.equal(st[-1], x[T - 3:])
