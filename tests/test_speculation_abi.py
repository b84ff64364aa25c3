"""What gdr_verify_drafts, gdr_commit_path and the state cache refuse: on the
host, before anything is enqueued (CPU only: fake pointers, no compute call)."""
import ctypes

import pytest
import torch

FAKE, STEP = 1 << 40, 1 << 34


@pytest.fixture(scope="module")
def lib():
    from channelwise_gated_delta_gb300 import _binding
    from channelwise_gated_delta_gb300 import build as cbuild
    cbuild.build()
    return _binding.load_library()


def pointers(names, ptrs):
    p = {n: FAKE + i * STEP for i, n in enumerate(names)}
    p.update(ptrs or {})
    return [None if p[n] is None else ctypes.c_void_p(p[n]) for n in names]


VERIFY = ("p", "q", "tokens", "parent", "coins", "u", "path", "n_path", "next_token")


def verify(lib, ptrs=None, B=2, T=4, V=100, ldp=100, ldq=100, sb=4, st=1, max_path=3,
           dtype=0):
    return lib.gdr_verify_drafts(*pointers(VERIFY, ptrs), B, T, V, ldp, ldq, sb, st, max_path,
                                 None, dtype)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 2), (dict(T=0), 2), (dict(V=0), 2), (dict(max_path=0), 2), (dict(max_path=5), 2),
    (dict(ldp=99), 2), (dict(ldq=99), 2), (dict(ldp=1 << 60), 2),
    (dict(sb=-1), 2), (dict(st=-1), 2), (dict(st=1 << 60), 2),
    (dict(T=513), 3), (dict(V=(1 << 22) + 1, ldp=1 << 23, ldq=1 << 23), 3), (dict(dtype=2), 3),
    (dict(ptrs=dict(p=None)), 1), (dict(ptrs=dict(parent=None)), 1),
    (dict(ptrs=dict(next_token=None)), 1), (dict(ptrs=dict(u=None)), 1),
    (dict(ptrs=dict(p=FAKE + 8)), 4), (dict(ptrs=dict(q=FAKE + STEP + 4)), 4),
    (dict(ptrs=dict(coins=FAKE + 4 * STEP + 2)), 4),
    (dict(ptrs=dict(path=FAKE + 16)), 8),                 # inside p
    (dict(ptrs=dict(n_path=FAKE + 6 * STEP + 4)), 8),     # inside path
    (dict(ptrs=dict(next_token=FAKE + 2 * STEP + 28)), 8),  # the last token
    (dict(B=0, ptrs=dict(p=None, tokens=None)), 0),       # nothing to do
])
def test_verify_refusals(lib, kw, status):
    assert verify(lib, **kw) == status


COMMIT = ("k", "v", "g", "beta", "h0", "ht", "path", "n_path")


def commit(lib, ptrs=None, B=2, T=4, HK=1, HV=2, dk=32, dv=32, max_path=3, dtype=0, flags=0):
    return lib.gdr_commit_path(*pointers(COMMIT, ptrs), B, T, HK, HV, dk, dv, max_path, None,
                               dtype, flags)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 2), (dict(T=0), 2), (dict(max_path=-1), 2), (dict(HK=0), 2),
    (dict(HK=2, HV=3), 2), (dict(B=1 << 28, HV=8), 2),
    (dict(dk=48), 3), (dict(dv=256), 3), (dict(dtype=9), 3), (dict(flags=1), 3),
    (dict(flags=8), 3),
    (dict(ptrs=dict(k=None)), 1), (dict(ptrs=dict(ht=None)), 1), (dict(ptrs=dict(path=None)), 1),
    (dict(ptrs=dict(n_path=None)), 1),
    (dict(ptrs=dict(v=FAKE + STEP + 8)), 4), (dict(ptrs=dict(h0=FAKE + 4 * STEP + 4)), 4),
    (dict(ptrs=dict(path=FAKE + 6 * STEP + 2)), 4),
    (dict(ptrs=dict(ht=FAKE + 4 * STEP + 16)), 8),        # part of h0
    (dict(ptrs=dict(ht=FAKE)), 8),                        # k
    (dict(ptrs=dict(n_path=FAKE + 5 * STEP + 64)), 8),    # inside ht
    (dict(B=0, ptrs=dict(k=None)), 0),
])
def test_commit_refusals(lib, kw, status):
    assert commit(lib, **kw) == status


@pytest.mark.parametrize("store", [True, False])
@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 2), (dict(n_slots=-1), 2), (dict(HV=0), 2), (dict(N=1 << 28, HV=8), 2),
    (dict(dk=16), 3), (dict(dv=100), 3),
    (dict(ptrs=dict(state=None)), 1), (dict(ptrs=dict(slots=None)), 1),
    (dict(ptrs=dict(cache=None)), 1), (dict(ptrs=dict(scale=None)), 1),
    (dict(ptrs=dict(state=FAKE + 4)), 4), (dict(ptrs=dict(cache=FAKE + 2 * STEP + 8)), 4),
    (dict(ptrs=dict(scale=FAKE + 3 * STEP + 1)), 4), (dict(ptrs=dict(slots=FAKE + STEP + 2)), 4),
    (dict(ptrs=dict(cache=FAKE + 64)), 8), (dict(ptrs=dict(scale=FAKE + 64)), 8),
    (dict(N=0, ptrs=dict(state=None, cache=None)), 0),
])
def test_state_cache_refusals(lib, kw, status, store):
    kw = dict(kw)
    a = dict(N=2, n_slots=3, HV=2, dk=32, dv=32)
    a.update({n: kw[n] for n in a if n in kw})
    state, slots, cache, scale = pointers(("state", "slots", "cache", "scale"), kw.get("ptrs"))
    sizes = (a["N"], a["n_slots"], a["HV"], a["dk"], a["dv"], None)
    got = (lib.gdr_state_store(state, slots, cache, scale, *sizes) if store
           else lib.gdr_state_load(cache, scale, slots, state, *sizes))
    assert got == status


def test_python_entries_refuse_host_tensors(lib):
    import channelwise_gated_delta_gb300 as gdr
    i32, f32 = dict(dtype=torch.int32), dict(dtype=torch.float32)
    with pytest.raises(ValueError):
        gdr.gdr_verify_drafts(torch.zeros(1, 2, 8), torch.zeros(1, 2, **i32),
                              torch.zeros(1, 2, **i32), torch.zeros(1, 2), torch.zeros(1))
    with pytest.raises(TypeError):
        gdr.gdr_verify_drafts(torch.zeros(1, 2, 8, dtype=torch.float16), torch.zeros(1, 2, **i32),
                              torch.zeros(1, 2, **i32), torch.zeros(1, 2), torch.zeros(1))
    with pytest.raises(ValueError):
        gdr.gdr_commit_path(torch.zeros(1, 2, 1, 32), torch.zeros(1, 2, 1, 32),
                            torch.zeros(1, 2, 1, 32), torch.zeros(1, 2, 1),
                            torch.zeros(1, 2, **i32), torch.zeros(1, **i32))
    cache, scale = gdr.gdr_state_cache(2, 1, 32, 32, device="cpu")
    with pytest.raises(ValueError):
        gdr.gdr_state_load(cache, scale, torch.zeros(1, **i32))
    with pytest.raises(ValueError):
        gdr.gdr_state_store(torch.zeros(1, 1, 32, 32, **f32), torch.zeros(1, **i32), cache, scale)


@pytest.mark.parametrize("shape,strides,ld", [
    ((2, 3, 8), (24, 8, 1), 8), ((2, 3, 7), (24, 8, 1), 8), ((1, 1, 5), (99, 77, 1), 5),
    ((2, 1, 5), (9, 1, 1), 9), ((1, 3, 1), (1, 4, 9), 4),
    ((2, 3, 8), (24, 8, 2), None), ((2, 3, 8), (32, 8, 1), None), ((2, 3, 8), (0, 0, 1), None),
])
def test_row_distance(shape, strides, ld):
    from channelwise_gated_delta_gb300._binding import _prob_rows
    t = torch.zeros(300).as_strided(shape, strides)
    if ld is None:
        with pytest.raises(ValueError):
            _prob_rows("p", t)
    else:
        assert _prob_rows("p", t) == ld
