"""Sizes that no int holds are refused by the Python entries around the recurrence, before the library
sees their low 32 bits (CPU only)."""
import pytest
import torch

from channelwise_gated_delta_gb300 import _binding
from tests.binding_fakes import Host, OnGpu

FAR = 2 ** 32 + 64      # 64 in 32 bits
f32, bf16 = torch.float32, torch.bfloat16


def big(*s, dt=bf16):
    return OnGpu(torch.empty(*s, dtype=dt, device="meta"))


conv, norm, ssm = _binding.gdr_short_conv, _binding.gdr_qk_norm, _binding.gdr_ssm_forward
w = big(1, 4, dt=f32)
CALLS = {
    "conv rows": (conv, [big(1, FAR, 1), w], {}),
    "conv sequences": (conv, [big(FAR, 1, 1), w], {}),
    "conv channels": (conv, [big(1, 1, FAR), big(FAR, 4, dt=f32)], {}),
    "conv packed": (conv, [big(FAR, 1), w], dict(cu_seqlens=[0, FAR])),
    "conv offsets": (conv, [big(64, 1), w], dict(cu_seqlens=[0, 2 ** 32, 64])),
    "conv negative offsets": (conv, [big(64, 1), w], dict(cu_seqlens=[0, -2 ** 32, 64])),
    "norm channels": (norm, [big(1, 1, 1, FAR), big(1, 1, 1, FAR)], {}),
    "norm heads": (norm, [big(1, 1, FAR, 32), big(1, 1, 1, 32)], {}),
    "ssm rows": (ssm, [big(1, FAR, 1, 32), big(1, FAR, 1, 32), big(1, FAR, 1, 32), big(1, FAR, 1, dt=f32),
                       big(1, dt=f32)], {}),
    "ssm columns": (ssm, [big(1, 1, 1, FAR), big(1, 1, 1, 32), big(1, 1, 1, 32), big(1, 1, 1, dt=f32),
                          big(1, dt=f32)], dict(store_ht=False)),
}
MOST = [big(1, 2 ** 31 - 1, 1), w, big(1, 2 ** 31 - 1, 1)]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_sizes_beyond_an_int(name, monkeypatch):
    host = Host(monkeypatch)
    call, args, kw = CALLS[name]
    with pytest.raises(ValueError, match="2.31"):
        call(*args, **kw)
    assert not host.calls and not host.allocations


def test_the_largest_ints_pass(monkeypatch):
    host = Host(monkeypatch)
    conv(*MOST[:2], out=MOST[2], store_st=False)
    assert host.calls[-1][0] == "gdr_short_conv"


def test_a_workspace_that_is_less_than_it_counts(monkeypatch):
    """One element expanded counts as many, and is no memory to write to."""
    z = lambda *s, dt=bf16: OnGpu(torch.zeros(*s, dtype=dt))
    args = [z(1, 3, 1, 32), z(1, 3, 1, 32), z(1, 3, 1, 32), z(1, 3, 1, dt=f32), z(1, dt=f32)]
    host = Host(monkeypatch)
    with pytest.raises(ValueError, match="contiguous"):
        ssm(*args, workspace=OnGpu(torch.zeros(1, dtype=torch.uint8).expand(256)))
    assert "gdr_ssm_forward" not in [c[0] for c in host.calls]
    ssm(*args, workspace=OnGpu(torch.zeros(256, dtype=torch.uint8)))
    assert host.calls[-1][0] == "gdr_ssm_forward"
