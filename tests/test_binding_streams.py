"""What the Python entries allocate for a call on a given stream (CPU: stand-ins for the library
and the tensors).  The caching allocator hands out a freed block at once to the stream that it was
freed on, where work on it may still be queued: memory that a kernel on another stream writes has to
come from that stream's blocks, and goes back to them when it is dropped."""
import pytest

from tests.binding_fakes import Host, Stream, arguments

ENTRIES = sorted(arguments())


@pytest.mark.parametrize("entry", ENTRIES)
def test_outputs_and_workspaces_are_memory_of_the_given_stream(entry, monkeypatch):
    call, args, kw = arguments()[entry]
    host = Host(monkeypatch)
    stream = Stream(77)
    call(*args, stream=stream, **kw)
    handles = [getattr(a, "value", a) for n, _, given in host.calls if n == entry for a in given]
    assert 77 in handles
    assert host.allocations == [(0, stream)] * len(host.allocations)
    assert bool(host.allocations) == (entry != "gdr_state_store")


@pytest.mark.parametrize("entry", ENTRIES)
def test_without_a_stream_the_current_one_is_used(entry, monkeypatch):
    call, args, kw = arguments()[entry]
    host = Host(monkeypatch)
    call(*args, **kw)
    handles = [getattr(a, "value", a) for n, _, given in host.calls if n == entry for a in given]
    assert 1000 in handles
    assert host.allocations == [(0, None)] * len(host.allocations)
