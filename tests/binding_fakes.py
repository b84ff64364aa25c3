"""Stand-ins for CUDA tensors, streams and the C library, for tests of what the Python entries do
on the host: which device and stream is current at each allocation and each call of the library."""
import contextlib

import torch

from channelwise_gated_delta_gb300 import _binding


class OnGpu:
    """A CPU tensor that says it is on CUDA device ``index``."""

    def __init__(self, t, index=0):
        self.t, self.index = t, index

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.index

    @property
    def device(self):
        return torch.device("cuda", self.index)


class Stream:
    def __init__(self, handle, index=0):
        self.cuda_stream, self.device, self.device_index = handle, torch.device("cuda", index), index


class Host:
    """Patches torch and the binding.  ``allocations`` and ``calls`` say what was current:
    (device, the stream or None for the device's current one) and (entry, device, arguments)."""

    def __init__(self, monkeypatch, device=0):
        self.device, self.stream = device, None
        self.allocations, self.calls = [], []
        host = self

        @contextlib.contextmanager
        def use(name, value):
            before = getattr(host, name)
            setattr(host, name, value)
            yield
            setattr(host, name, before)

        def index_of(device):
            device = torch.device("cuda", device) if isinstance(device, int) else \
                torch.device(device)
            return host.device if device.index is None else device.index

        def fresh(make, like=None):
            def call(*args, device=None, **kw):
                if like:
                    args = (args[0].t,) + args[1:]
                host.allocations.append((host.device, host.stream))
                return OnGpu(make(*args, **kw), host.device if device is None else index_of(device))
            return call

        class Library:
            def __getattr__(self, name):
                if name.endswith("_bytes"):
                    return lambda *a: host.calls.append((name, host.device, a)) or 64
                return lambda *a: host.calls.append((name, host.device, a)) or 0

        p = monkeypatch.setattr
        p(_binding, "load_library", lambda: Library())
        p(torch, "empty", fresh(torch.empty))
        p(torch, "empty_strided", fresh(torch.empty_strided))
        p(torch, "empty_like", fresh(torch.empty_like, like=True))
        p(torch.cuda, "stream", lambda s: use("stream", s))
        p(torch.cuda, "device", lambda d: use("device", index_of(d)))
        p(torch.cuda, "current_device", lambda: host.device)
        p(torch._C, "_cuda_getDevice", lambda: host.device)
        p(torch.cuda, "current_stream", lambda d=None: Stream(1000 + index_of(
            host.device if d is None else d), index_of(host.device if d is None else d)))
        p(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i)


def arguments(index=0):
    """One call of every Python entry that launches: name -> (function, args, keywords)."""
    B, T, HK, HV, d, V = 2, 3, 1, 2, 32, 10
    z = lambda *s, dt=torch.float32: OnGpu(torch.zeros(*s, dtype=dt), index)
    i32 = lambda *s: z(*s, dt=torch.int32)
    five = lambda *lead: [z(*lead, HK, d), z(*lead, HK, d), z(*lead, HV, d), z(*lead, HV, d),
                          z(*lead, HV)]
    host = [torch.zeros(*x.shape) for x in five(B, T)]
    b = _binding
    return {
        "gdr_forward_ex": (b.gdr_forward, five(B, T), {}),
        "gdr_forward_varlen": (b.gdr_forward_varlen, five(T), dict(cu_seqlens=[0, 1, 3])),
        "gdr_forward_tree": (b.gdr_forward_tree, five(B, T), dict(parent=[[-1, 0, 1]] * B)),
        "gdr_forward_host": (b.gdr_forward_host,
                             host + [None, torch.zeros(B, T, HV, d), torch.zeros(B, HV, d, d)], {}),
        "gdr_verify_drafts": (b.gdr_verify_drafts, [z(B, T, V), i32(B, T), i32(B, T), z(B, T), z(B)],
                              dict(max_path=2)),
        "gdr_commit_path": (b.gdr_commit_path, five(B, T)[1:] + [i32(B, 2), i32(B)], {}),
        "gdr_state_store": (b.gdr_state_store, [z(B, HV, d, d), i32(B),
                                                z(4, HV, d, d, dt=torch.int8), z(4, HV, d)], {}),
        "gdr_state_load": (b.gdr_state_load, [z(4, HV, d, d, dt=torch.int8), z(4, HV, d), i32(B)],
                           {}),
    }
