"""The scalar-gate flag beside gates that are channelwise (CPU: stand-ins for the library and the
tensors): the flag's layout of g is [.., HV], and read so, [.., HV, dk] gives other tokens' gates."""
import pytest
import torch

from channelwise_gated_delta_gb300 import GDR_FLAG_SCALAR_GATE
from tests.binding_fakes import Host, OnGpu, arguments

ENTRIES = {"gdr_forward_ex": 3, "gdr_forward_varlen": 3, "gdr_forward_tree": 3, "gdr_commit_path": 2}


@pytest.mark.parametrize("entry", sorted(ENTRIES))
def test_flag_and_shape_have_to_agree(entry, monkeypatch):
    call, args, kw = arguments()[entry]
    host = Host(monkeypatch)
    with pytest.raises(ValueError):
        call(*args, flags=GDR_FLAG_SCALAR_GATE, **kw)
    assert entry not in [c[0] for c in host.calls]
    g = args[ENTRIES[entry]]
    args = list(args)
    args[ENTRIES[entry]] = OnGpu(torch.zeros(*g.shape[:-1]))
    call(*args, **kw)                                  # the shape says it
    call(*args, flags=GDR_FLAG_SCALAR_GATE, **kw)      # and so may the flag
    assert [c[2][-1] for c in host.calls if c[0] == entry] == [GDR_FLAG_SCALAR_GATE] * 2
