"""Tensors of another device than the current one (CPU: stand-ins for the library and the tensors).
The C entries look up SMs, the error word and their launches' target on the current device, so it has
to be the tensors' own while one runs."""
import pytest

from channelwise_gated_delta_gb300 import _binding
from tests.binding_fakes import Host, Stream, arguments

ENTRIES = sorted(arguments())


@pytest.mark.parametrize("current,tensors", [(0, 1), (1, 0), (0, 0), (2, 2)])
@pytest.mark.parametrize("entry", ENTRIES)
def test_the_library_runs_on_the_tensors_device(entry, current, tensors, monkeypatch):
    call, args, kw = arguments(tensors)[entry]
    if entry == "gdr_forward_host":
        kw = dict(device="cuda:%d" % tensors)
    host = Host(monkeypatch, device=current)
    call(*args, **kw)
    assert entry in [c[0] for c in host.calls]
    assert {device for _, device, _ in host.calls} == {tensors}
    given = [getattr(a, "value", a) for name, _, x in host.calls if name == entry for a in x]
    assert 1000 + tensors in given           # that device's current stream
    assert host.device == current            # and the caller's is current again


@pytest.mark.parametrize("entry", ENTRIES)
def test_a_stream_of_another_device_is_refused(entry, monkeypatch):
    call, args, kw = arguments(0)[entry]
    host = Host(monkeypatch)
    with pytest.raises(ValueError):
        call(*args, stream=Stream(77, index=1), **kw)
    assert entry not in [c[0] for c in host.calls]


def test_device_check_reads_the_streams_device(monkeypatch):
    host = Host(monkeypatch)
    _binding.gdr_device_check(Stream(77, index=1))
    _binding.gdr_device_check()
    assert [c[1] for c in host.calls] == [1, 0]
