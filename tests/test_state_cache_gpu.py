"""gdr_state_store / gdr_state_load on the GPU: codes, scales and values equal the oracle's to the
bit (each is one float32 operation after the other), and are within half a step of the state."""
import numpy as np
import pytest
import torch

from channelwise_gated_delta_gb300 import gdr_state_cache, gdr_state_load, gdr_state_store
from oracle import speculation

pytestmark = pytest.mark.gpu


def states(N, HV, dk, dv, seed=0):
    gen = torch.Generator()
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    return r(N, HV, dk, dv) * torch.exp(3 * r(N, HV, dk, 1))


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def check(x, slots, n_slots):
    """Stores and loads; every other slot keeps what it held."""
    N, HV, dk, dv = x.shape
    cache, scale = gdr_state_cache(n_slots, HV, dk, dv)
    cache.fill_(5)
    scale.fill_(2.0)
    gdr_state_store(x.cuda(), i32(slots), cache, scale)
    codes, sc = speculation.quantise(x.numpy())
    want_c, want_s = np.full(cache.shape, 5, np.int8), np.full(scale.shape, 2.0, np.float32)
    for n, s in enumerate(slots):
        if 0 <= s < n_slots:
            want_c[s], want_s[s] = codes[n], sc[n]
    assert np.array_equal(cache.cpu().numpy(), want_c)
    assert np.array_equal(scale.cpu().numpy(), want_s, equal_nan=True)
    back = gdr_state_load(cache, scale, i32(slots)).cpu().numpy()
    for n, s in enumerate(slots):
        with np.errstate(invalid="ignore"):
            want = (speculation.dequantise(codes[n], sc[n]) if 0 <= s < n_slots
                    else np.zeros_like(back[n]))
        assert np.array_equal(back[n], want, equal_nan=True)
        if 0 <= s < n_slots and np.isfinite(x[n].numpy()).all():
            # half a step, and the roundings of the product and the scale (127 * 3 2^-24 steps)
            step = sc[n][..., None].astype(np.float64)
            err = np.abs(back[n].astype(np.float64) - x[n].numpy())
            assert (err <= step * (0.5 + 127 * 3 * 2.0 ** -24) + 1e-30).all()


@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("N,HV", [(1, 1), (3, 5), (2, 32)])
def test_shapes(N, HV, dk, dv):
    check(states(N, HV, dk, dv, seed=dk + dv), np.random.RandomState(N).permutation(N + 2)[:N],
          N + 2)


def test_slots_outside_are_neither_stored_nor_known():
    check(states(6, 2, 64, 64, seed=1), [3, -1, 4, 0, -2 ** 31, 2 ** 31 - 1], 4)


def test_rows_at_their_ends():
    x = states(4, 2, 32, 64, seed=2)
    x[0, 0, 0] = 0.0                      # a row of zeros
    x[0, 0, 1] = 1e-38                    # as good as zero
    x[0, 0, 2] = 1e-30                    # the largest that counts as zero
    x[0, 0, 3] = 1.0000001e-30
    x[0, 0, 4] = torch.linspace(-3e38, 3e38, 64)
    x[0, 0, 5] = -1.0                     # one magnitude
    x[0, 0, 6, :] = 0.0
    x[0, 0, 6, 63] = -7.0                 # the largest magnitude last and negative
    x[0, 0, 7] = torch.arange(-32, 32) * 0.5   # halves: ties to even
    x[0, 0, 7, 0] = 127.0
    x[1, 1, 3, 7] = float("nan")
    x[1, 1, 4, 63] = float("inf")
    x[2, 0, 31, 0] = float("-inf")
    x[2, 0, 30] = float("nan")
    check(x, [0, 3, 2, 1], 4)


def test_a_slot_serves_several_sequences():
    x = states(2, 3, 128, 64, seed=3)
    cache, scale = gdr_state_cache(2, 3, 128, 64)
    gdr_state_store(x.cuda(), i32([1, 0]), cache, scale)
    a = gdr_state_load(cache, scale, i32([1, 1, -1, 0, 1]))
    assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[4]) and not a[2].any()
    assert not torch.equal(a[0], a[3])


def test_stored_again_it_is_the_same():
    """What came out of the cache goes in and out again without a change beyond its scale's
    rounding: the codes are those of the first time."""
    x = states(2, 4, 64, 128, seed=4).cuda()
    c1, s1 = gdr_state_cache(2, 4, 64, 128)
    gdr_state_store(x, i32([0, 1]), c1, s1)
    c2, s2 = gdr_state_cache(2, 4, 64, 128)
    gdr_state_store(gdr_state_load(c1, s1, i32([0, 1])), i32([0, 1]), c2, s2)
    assert torch.equal(c1, c2)


def test_offsets_past_32_bits():
    HV, dk, dv, n_slots = 32, 128, 128, 8200          # 4.3 GB of codes
    x = states(3, HV, dk, dv, seed=5)
    cache = torch.empty(n_slots, HV, dk, dv, dtype=torch.int8, device="cuda")
    scale = torch.empty(n_slots, HV, dk, device="cuda")
    slots = i32([n_slots - 1, 0, 4097])
    gdr_state_store(x.cuda(), slots, cache, scale)
    codes, sc = speculation.quantise(x.numpy())
    for n, s in enumerate([n_slots - 1, 0, 4097]):
        assert np.array_equal(cache[s].cpu().numpy(), codes[n])
    back = gdr_state_load(cache, scale, slots).cpu().numpy()
    assert np.array_equal(back, speculation.dequantise(codes, sc))


def test_given_output_and_another_stream():
    x = states(2, 2, 32, 32, seed=6).cuda()
    cache, scale = gdr_state_cache(2, 2, 32, 32)
    out, slots = torch.full_like(x, 9.0), i32([1, 0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gdr_state_store(x, slots, cache, scale, stream=s)
    assert gdr_state_load(cache, scale, slots, out=out, stream=s) is out
    s.synchronize()
    codes, sc = speculation.quantise(x.cpu().numpy())
    assert np.array_equal(out.cpu().numpy(), speculation.dequantise(codes, sc))


def test_nothing_to_do():
    cache, scale = gdr_state_cache(0, 2, 32, 32)
    assert gdr_state_load(cache, scale, i32([])).shape == (0, 2, 32, 32)
    assert not gdr_state_load(cache, scale, i32([0, -1])).any()        # no slots: all new
    gdr_state_store(torch.ones(2, 2, 32, 32, device="cuda"), i32([0, 1]), cache, scale)
