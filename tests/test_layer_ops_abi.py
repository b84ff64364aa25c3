"""What gdr_short_conv, gdr_qk_norm and gdr_ssm_forward refuse: on the host, before anything is
enqueued (CPU only: fake pointers, no compute call); and what the Python entries check."""
import ctypes
import math

import pytest
import torch

from channelwise_gated_delta_gb300 import _binding
from tests.binding_fakes import Host, OnGpu, Stream

FAKE, STEP = 1 << 40, 1 << 36


@pytest.fixture(scope="module")
def lib():
    from channelwise_gated_delta_gb300 import build as cbuild
    cbuild.build()
    return _binding.load_library()


def pointers(names, ptrs):
    p = {n: FAKE + i * STEP for i, n in enumerate(names)}
    p.update(ptrs or {})
    return [None if p[n] is None else ctypes.c_void_p(p[n]) for n in names]


def cu_array(vals):
    return None if vals is None else (ctypes.c_int * len(vals))(*vals)


CONV = ("x", "w", "bias", "s0", "out", "st")


def conv(lib, ptrs=None, cu=None, N=2, T=5, D=64, W=4, ldx=64, ldo=64, dtype=1, flags=0):
    return lib.gdr_short_conv(*pointers(CONV, ptrs), cu_array(cu), N, T, D, W, ldx, ldo, None,
                              dtype, flags)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 2), (dict(T=-1), 2), (dict(D=0), 2), (dict(ldx=63), 2), (dict(ldo=63), 2),
    (dict(ldx=1 << 60), 2), (dict(D=1 << 23, ldx=1 << 24, ldo=(1 << 24) + 1), 2),
    (dict(cu=[1, 2, 3]), 2), (dict(cu=[0, 3, 2]), 2),
    (dict(W=1), 3), (dict(W=5), 3), (dict(dtype=2), 3), (dict(flags=4), 3),
    (dict(ptrs=dict(x=None)), 1), (dict(ptrs=dict(w=None)), 1), (dict(ptrs=dict(out=None)), 1),
    (dict(ptrs=dict(x=FAKE + 1)), 4), (dict(ptrs=dict(st=FAKE + 5 * STEP + 1)), 4),
    (dict(ptrs=dict(w=FAKE + STEP + 2)), 4), (dict(ptrs=dict(bias=FAKE + 2 * STEP + 2)), 4),
    (dict(ptrs=dict(out=FAKE + 128)), 8),                       # the rows of x, one on
    (dict(ptrs=dict(out=FAKE)), 8),                             # a window needs its neighbours
    (dict(ptrs=dict(out=FAKE + 64), ldx=128, ldo=128), 8),      # half of each row
    (dict(ptrs=dict(st=FAKE + 4 * STEP)), 8), (dict(ptrs=dict(st=FAKE)), 8),
    (dict(ptrs=dict(st=FAKE + 3 * STEP + 128)), 8),             # s0, one row on
    (dict(ptrs=dict(s0=FAKE + 4 * STEP)), 8),
    (dict(N=0, ptrs=dict(x=None, w=None, out=None)), 0),        # nothing to do
    (dict(T=0, ptrs=dict(x=None, out=None, st=None)), 0),
])
def test_conv_refusals(lib, kw, status):
    assert conv(lib, **kw) == status


NORM = ("q", "k", "weight_q", "weight_k", "positions", "freqs", "out_q", "out_k")


def norm(lib, ptrs=None, rows=5, HQ=4, HK=2, d=64, d_rot=32, ldq=256, ldk=128, ldoq=256,
         ldok=128, eps=0.0, dtype=1, flags=0):
    return lib.gdr_qk_norm(*pointers(NORM, ptrs), rows, HQ, HK, d, d_rot, ldq, ldk, ldoq, ldok,
                           eps, 1.0, None, dtype, flags)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 2), (dict(HQ=0), 2), (dict(HK=0), 2), (dict(eps=-1.0), 2),
    (dict(eps=float("nan")), 2), (dict(ldq=255), 2), (dict(ldok=64), 2), (dict(ldk=1 << 60), 2),
    (dict(d=48), 3), (dict(d=512), 3), (dict(d_rot=8), 3), (dict(d_rot=80), 3), (dict(d_rot=-16), 3),
    (dict(dtype=2), 3), (dict(flags=1), 3),
    (dict(ptrs=dict(q=None)), 1), (dict(ptrs=dict(out_k=None)), 1),
    (dict(ptrs=dict(positions=None)), 1), (dict(ptrs=dict(freqs=None)), 1),
    (dict(ptrs=dict(q=FAKE + 8)), 4), (dict(ptrs=dict(freqs=FAKE + 5 * STEP + 4)), 4),
    (dict(ldq=260), 4), (dict(ptrs=dict(positions=FAKE + 4 * STEP + 2)), 4),
    (dict(ptrs=dict(out_q=FAKE + 16)), 8), (dict(ptrs=dict(out_q=FAKE + STEP)), 8),
    (dict(ptrs=dict(out_k=FAKE + 6 * STEP)), 8), (dict(ptrs=dict(out_k=FAKE + 2 * STEP)), 8),
    (dict(ptrs=dict(out_q=FAKE), ldq=512), 8),                  # in place at another distance
    (dict(rows=0, ptrs=dict(q=None)), 0),
])
def test_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status


SSM = ("x", "b", "c", "dt", "A", "D", "z", "dt_bias", "h0", "out", "ht")


def ssm(lib, ptrs=None, cu=None, N=2, T=5, HK=1, HV=2, dk=32, dv=64, ldx=128, ldb=32, ldc=32,
        ldz=128, dtype=1, ws=None, ws_bytes=0, flags=0):
    return lib.gdr_ssm_forward(*pointers(SSM, ptrs), cu_array(cu), N, T, HK, HV, dk, dv, ldx, ldb,
                               ldc, ldz, None, dtype, ws, ws_bytes, flags)


SEG = 4 << 8


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 2), (dict(T=-1), 2), (dict(HK=2, HV=3), 2), (dict(HK=0), 2), (dict(ldx=127), 2),
    (dict(ldb=31), 2), (dict(ldc=31), 2), (dict(ldz=127), 2), (dict(ldz=1 << 60), 2),
    (dict(cu=[1, 2, 3]), 2), (dict(cu=[0, 3, 2]), 2),
    (dict(dk=48), 3), (dict(dv=256), 3), (dict(dtype=2), 3), (dict(flags=4), 3),
    (dict(ptrs=dict(x=None)), 1), (dict(ptrs=dict(A=None)), 1), (dict(ptrs=dict(dt=None)), 1),
    (dict(ptrs=dict(out=None)), 1), (dict(ptrs=dict(x=FAKE + 1)), 4),
    (dict(ptrs=dict(z=FAKE + 6 * STEP + 1)), 4), (dict(ptrs=dict(ht=FAKE + 10 * STEP + 8)), 4),
    (dict(ptrs=dict(dt=FAKE + 3 * STEP + 2)), 4),
    (dict(ptrs=dict(out=FAKE)), 8), (dict(ptrs=dict(out=FAKE + 6 * STEP)), 8),
    (dict(ptrs=dict(ht=FAKE + 9 * STEP)), 8), (dict(ptrs=dict(ht=FAKE + 8 * STEP + 16)), 8),
    (dict(ptrs=dict(ht=FAKE + 3 * STEP)), 8), (dict(ptrs=dict(out=FAKE + 4 * STEP)), 8),
    (dict(T=1000, flags=SEG), 5), (dict(T=1000, flags=SEG, ws=FAKE + 20 * STEP, ws_bytes=64), 5),
    (dict(T=1000, flags=SEG, ws=FAKE + 20 * STEP + 16, ws_bytes=1 << 30), 4),
    (dict(N=0, ptrs=dict(x=None, A=None)), 0),
    (dict(T=0, ptrs=dict(x=None, ht=None)), 0),
])
def test_ssm_refusals(lib, kw, status):
    assert ssm(lib, **kw) == status


def test_ssm_workspace(lib):
    """Forced segments: a state and a number per segment and head, and room for the first states."""
    ws = lambda cu, n, T, f: lib.gdr_ssm_workspace_bytes(cu_array(cu), n, T, 1, 2, 32, 64, 1, f)
    state = 2 * 32 * 64 * 4
    assert ws(None, 3, 64, SEG) == 0 and ws(None, 3, 1000, SEG | 8) == 0
    assert ws(None, 0, 1000, SEG) == 0 and ws(None, 3, 1000, 1 << 30) == 0
    need = ws(None, 3, 1000, SEG)                      # segments of 256 rows
    assert 15 * state <= need < 15 * state + 1024
    need = ws([0, 1000, 1000, 1300], 3, 0, SEG)        # 4, 1 and 2 of them
    assert 10 * state <= need < 10 * state + 1024


# ------------------------------------------------------------------ the Python entries
def z(*s, dt=torch.bfloat16, index=0):
    return OnGpu(torch.zeros(*s, dtype=dt), index)


def calls(index=0):
    f = torch.float32
    t = lambda *s, dt=torch.bfloat16: z(*s, dt=dt, index=index)
    b = _binding
    return {
        "gdr_short_conv": (b.gdr_short_conv, [t(2, 3, 64), t(64, 4, dt=f)], {}),
        "gdr_qk_norm": (b.gdr_qk_norm, [t(2, 3, 4, 32), t(2, 3, 2, 32)], {}),
        "gdr_ssm_forward": (b.gdr_ssm_forward, [t(2, 3, 2, 32), t(2, 3, 1, 64), t(2, 3, 1, 64),
                                                t(2, 3, 2, dt=f), t(2, dt=f)], {}),
    }


@pytest.mark.parametrize("entry", sorted(calls()))
@pytest.mark.parametrize("current,tensors", [(0, 1), (1, 0), (0, 0)])
def test_device_and_stream(entry, current, tensors, monkeypatch):
    call, args, kw = calls(tensors)[entry]
    host = Host(monkeypatch, device=current)
    call(*args, **kw)
    assert {device for _, device, _ in host.calls} == {tensors} and host.device == current
    given = [a for n, _, x in host.calls if n == entry for a in x]
    assert 1000 + tensors in given
    stream = Stream(77, index=tensors)
    host.allocations.clear()
    call(*args, stream=stream, **kw)
    assert 77 in [a for n, _, x in host.calls if n == entry for a in x]
    assert host.allocations and {s for _, s in host.allocations} == {stream}
    with pytest.raises(ValueError):
        call(*args, stream=Stream(77, index=tensors + 1), **kw)


def test_distances_of_rows():
    rows = _binding._rows_of
    wide = torch.zeros(3, 5, 100)
    bf = torch.float32
    at = lambda t, *inner: rows("t", OnGpu(t), t.shape, t.dim() - len(inner), math.prod(inner), bf, 0)
    assert at(wide, 100) == 100 and at(wide[..., :64], 64) == 100
    assert at(wide[..., 4:68].unflatten(-1, (2, 32)), 2, 32) == 100
    assert at(wide[:, :1, :64], 64) == 500 and at(wide[:1, :, :64], 64) == 100
    assert at(wide[:, 0, :64], 64) == 500 and at(wide[0, :1, :64], 64) == 64
    for bad, inner in ((wide[:, :4, :64], (64,)), (wide[..., ::2], (50,)),
                       (torch.zeros(1, 1, 64).expand(3, 5, 64), (64,)),
                       (torch.zeros(3, 5, 32, 2).transpose(2, 3), (2, 32)),
                       (wide.transpose(0, 1)[..., :64], (64,))):
        with pytest.raises(ValueError):
            at(bad, *inner)


@pytest.mark.parametrize("change", [
    dict(x=z(2, 3, 64, dt=torch.float16)), dict(weight=z(64, 4)), dict(weight=z(63, 4, dt=torch.float32)),
    dict(bias=z(64)), dict(s0=z(2, 4, 64)), dict(s0=z(2, 3, 64, dt=torch.float32)),
    dict(out=z(2, 3, 65)), dict(st=z(1, 3, 64)), dict(x=z(64)), dict(cu_seqlens=[0, 3]),
    dict(x=z(6, 64)), dict(x=z(6, 64), cu_seqlens=[0, 5]), dict(weight=z(64, 4, dt=torch.float32, index=1)),
])
def test_conv_arguments(change, monkeypatch):
    host = Host(monkeypatch)
    kw = dict(dict(x=z(2, 3, 64), weight=z(64, 4, dt=torch.float32)), **change)
    with pytest.raises((ValueError, TypeError)):
        _binding.gdr_short_conv(**kw)
    assert not host.calls


@pytest.mark.parametrize("change", [
    dict(norm="layer"), dict(k=z(2, 4, 2, 32)), dict(k=z(2, 3, 2, 64)), dict(k=z(6, 2, 32)),
    dict(positions=z(2, 3, dt=torch.int32)), dict(freqs=z(16, dt=torch.int64)),
    dict(positions=z(2, 3, dt=torch.int64), freqs=z(16, dt=torch.int64)),
    dict(positions=z(2, 3, dt=torch.int32), freqs=z(16, dt=torch.float32)),
    dict(weight_q=z(32)), dict(weight_k=z(31, dt=torch.float32)), dict(out_q=z(2, 3, 2, 32)),
])
def test_norm_arguments(change, monkeypatch):
    host = Host(monkeypatch)
    with pytest.raises((ValueError, TypeError)):
        _binding.gdr_qk_norm(**dict(dict(q=z(2, 3, 4, 32), k=z(2, 3, 2, 32)), **change))
    assert not host.calls


@pytest.mark.parametrize("change", [
    dict(b=z(2, 3, 1, 32)), dict(c=z(2, 3, 1, 64, dt=torch.float32)), dict(dt=z(2, 3, 2)),
    dict(a=z(1, dt=torch.float32)), dict(d=z(2)), dict(z=z(2, 3, 2, 64)), dict(h0=z(2, 2, 64, 32)),
    dict(ht=z(2, 2, 32, 64, dt=torch.float32)), dict(out=z(2, 3, 2, 32, dt=torch.float32)),
    dict(dt_bias=z(3, dt=torch.float32)), dict(x=z(2, 32)), dict(cu_seqlens=[0, 6]),
])
def test_ssm_arguments(change, monkeypatch):
    host = Host(monkeypatch)
    f = torch.float32
    kw = dict(x=z(2, 3, 2, 32), b=z(2, 3, 1, 64), c=z(2, 3, 1, 64), dt=z(2, 3, 2, dt=f), a=z(2, dt=f))
    with pytest.raises((ValueError, TypeError)):
        _binding.gdr_ssm_forward(**dict(kw, **change))
    assert "gdr_ssm_forward" not in [c[0] for c in host.calls]


def test_rope_freqs():
    """Turns of a position in 2^-64, negative numbers for the upper half."""
    f = _binding.gdr_rope_freqs(8, base=100.0, device="cpu")
    want = [100.0 ** (-2 * i / 8) / (2 * 3.141592653589793) * 2.0 ** 64 for i in range(4)]
    assert f.dtype == torch.int64 and all(abs(int(a) - b) < 2 ** 12 for a, b in zip(f, want))
    f = _binding.gdr_rope_freqs(4, inv_freq=[5.0, -0.5], device="cpu")
    assert all(abs(int(a) % 2 ** 64 - b % 2 ** 64) < 2 ** 12 for a, b in zip(
        f, [5.0 / (2 * 3.141592653589793) * 2.0 ** 64, -0.5 / (2 * 3.141592653589793) * 2.0 ** 64]))
    with pytest.raises(ValueError):
        _binding.gdr_rope_freqs(8, inv_freq=[1.0])
