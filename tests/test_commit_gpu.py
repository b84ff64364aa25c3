"""gdr_commit_path on the GPU against the fp64 recurrence run along each sequence's path.

Tolerance: a step's column sum has dk products, whose roundings add up like a random walk
(sqrt(dk) 2^-24 of the largest term), and a few more operations (decay with expf within 2 ulp,
beta, update: 8 2^-24); k has norm 1 and no step makes an error larger, so n steps are off by at
most (n + 1) (sqrt(dk) + 8) 2^-24 M, M the largest magnitude of h0, v and the result."""
import numpy as np
import pytest
import torch

from channelwise_gated_delta_gb300 import gdr_commit_path, gdr_forward
from channelwise_gated_delta_gb300.inputs import draw, to_f64
from oracle import speculation
from tests.parity_util import to_cuda

pytestmark = pytest.mark.gpu


def paths(B, T, P, seed=0, lengths=None):
    """Increasing nodes from 0 on; -1 behind each path."""
    rng = np.random.default_rng(seed)
    path, n = np.full((B, P), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n[b] = min(P, T, lengths[b % len(lengths)]) if lengths else rng.integers(0, min(P, T) + 1)
        if n[b]:
            path[b, :n[b]] = np.r_[0, np.sort(1 + rng.permutation(T - 1)[:n[b] - 1])]
    return torch.from_numpy(path), torch.from_numpy(n)


def check(d, path, n_path, in_place=False):
    c = to_cuda(d)
    h0 = c["h0"]
    keep = None if h0 is None else h0.clone()
    ht = gdr_commit_path(c["k"], c["v"], c["g"], c["beta"], path.cuda(), n_path.cuda(), h0=h0,
                         ht=h0 if in_place else None)
    ref = speculation.commit_path(*(to_f64(d[x]) for x in ("k", "v", "g", "beta", "h0")),
                                  path.numpy(), n_path.numpy())
    if h0 is not None and not in_place:
        assert torch.equal(h0, keep)
    got = to_f64(ht)
    assert got.shape == ref.shape and np.isfinite(got).all()
    dk = d["k"].shape[-1]
    for b in range(ref.shape[0]):
        n = max(0, min(int(n_path[b]), path.shape[1]))
        start = 0.0 if d["h0"] is None else float(d["h0"][b].abs().max())
        big = max(start, float(d["v"][b].float().abs().max()), float(np.abs(ref[b]).max()))
        tol = (n + 1) * (dk ** 0.5 + 8) * 2.0 ** -24 * big
        err = np.abs(got[b] - ref[b]).max()
        assert err <= tol, (b, n, err, tol)
        if n == 0:
            assert np.array_equal(got[b], ref[b])
    return ht


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scalar", [False, True])
@pytest.mark.parametrize("dk,dv", [(32, 32), (32, 128), (64, 64), (64, 32), (128, 32), (128, 64),
                                   (128, 128)])
def test_shapes(dk, dv, scalar, dtype):
    d = draw(3, 11, 2, 6, dk, dv, dtype=dtype, seed=dk + dv, scalar_gate=scalar)
    check(d, *paths(3, 11, 7, seed=dk))


@pytest.mark.parametrize("lengths", [[0], [1], [2], [0, 1, 5, 16], [15, 16, 17], [31, 33, 47, 64]])
@pytest.mark.parametrize("dims", [(128, 128), (64, 32)])
def test_lengths(lengths, dims):
    d = draw(4, 64, 2, 4, *dims, dtype=torch.bfloat16, seed=3)
    check(d, *paths(4, 64, 64, lengths=lengths))


@pytest.mark.parametrize("B,HK,HV", [(1, 1, 1), (1, 16, 32), (2, 5, 15), (7, 16, 32), (33, 8, 16)])
def test_numbers_of_heads(B, HK, HV):
    """Every split of a state over CTAs, which goes by the number of heads."""
    d = draw(B, 6, HK, HV, 128, 128, dtype=torch.bfloat16, seed=B)
    check(d, *paths(B, 6, 6, seed=B))


@pytest.mark.parametrize("h0", [True, False])
@pytest.mark.parametrize("scalar", [False, True])
def test_many_heads_of_all_lengths(scalar, h0):
    """More heads than the device holds at once, several times over; lengths that differ from
    head to head, so that no two of them take the same time."""
    d = draw(60, 40, 8, 32, 128, 128, dtype=torch.bfloat16, h0=h0, seed=20, scalar_gate=scalar)
    p = paths(60, 40, 40, lengths=[1, 4, 0, 9, 2, 37, 5, 1, 8, 3, 40, 1, 1, 12])
    ht = check(d, *p)
    for _ in range(3):
        assert torch.equal(ht, check(d, *p, in_place=h0))


def test_long_path_of_512():
    d = draw(1, 512, 1, 2, 128, 128, dtype=torch.float32, seed=4)
    check(d, *paths(1, 512, 512, lengths=[512]))


@pytest.mark.parametrize("mu", [-6.0, 3.0, 60.0])
def test_decay_from_slow_to_everything(mu):
    """|g| from 2e-3 to 60 per token: exp(g) down to the smallest numbers."""
    check(draw(2, 9, 2, 4, 128, 128, dtype=torch.bfloat16, seed=5, g_mu=mu), *paths(2, 9, 9, 1))


@pytest.mark.parametrize("dims", [(128, 128), (64, 32)])
def test_channels_that_forget_everything(dims):
    """g = -inf: exp(g) = 0 and the row starts again; beta = 0: the node only decays."""
    d = draw(2, 8, 1, 2, *dims, seed=13)
    d["g"][:, 2, :, ::3] = float("-inf")
    d["g"][1, 4] = float("-inf")
    d["beta"][:, 5] = 0.0
    check(d, *paths(2, 8, 8, lengths=[8]))


def test_state_grows_where_the_gate_lets_it():
    d = draw(2, 5, 1, 2, 64, 64, seed=6)
    d["g"] = d["g"].abs() * 0.1
    check(d, *paths(2, 5, 5, lengths=[5]))


def test_no_initial_state():
    check(draw(3, 8, 2, 4, 128, 128, dtype=torch.bfloat16, h0=False, seed=7), *paths(3, 8, 8, 2))
    check(draw(3, 8, 2, 4, 32, 64, h0=False, seed=7), *paths(3, 8, 8, 2))


@pytest.mark.parametrize("dims", [(128, 128), (32, 64)])
def test_in_place_is_the_same_to_the_bit(dims):
    d = draw(6, 12, 2, 4, *dims, dtype=torch.bfloat16, seed=8)
    p = paths(6, 12, 8, lengths=[0, 3, 8])
    assert torch.equal(check(d, *p), check(d, *p, in_place=True))


def test_entries_that_end_a_path():
    d = draw(5, 6, 1, 2, 64, 64, seed=9)
    path = torch.tensor([[0, 2, 6, 3], [0, -1, 2, 3], [-1, 0, 1, 2], [0, 1, 2, 3], [0, 5, 4, 0]],
                        dtype=torch.int32)
    n = torch.tensor([4, 4, 4, 99, 4], dtype=torch.int32)   # 99: as many as there is room for
    check(d, path, n)
    check(d, path, torch.tensor([-3, 0, -2 ** 31, 2 ** 31 - 1, 2], dtype=torch.int32))
    check(d, path[:, :0].contiguous(), n)                    # no room at all


def test_equals_the_forward_pass_along_the_path():
    """A chain that is accepted whole leaves the state of gdr_forward over its tokens."""
    d = to_cuda(draw(2, 7, 2, 4, 128, 128, dtype=torch.bfloat16, seed=10))
    n = torch.full((2,), 7, dtype=torch.int32, device="cuda")
    path = torch.arange(7, dtype=torch.int32, device="cuda").expand(2, 7).contiguous()
    ht = gdr_commit_path(d["k"], d["v"], d["g"], d["beta"], path, n, h0=d["h0"])
    ref = gdr_forward(d["q"], d["k"], d["v"], d["g"], d["beta"], d["h0"])[1]
    assert (ht - ref).abs().max() <= 2e-2 * ref.abs().max()   # the forward pass's bf16 products


def test_nothing_leaks_between_sequences():
    """NaN and infinities in one sequence, and in rows that no path visits, stay there."""
    d = draw(3, 6, 1, 2, 128, 128, dtype=torch.bfloat16, seed=11)
    path, n = paths(3, 6, 4, lengths=[4])
    path[:, 1:] = torch.tensor([1, 3, 5])
    clean = gdr_commit_path(*(to_cuda(d)[x] for x in ("k", "v", "g", "beta")), path.cuda(),
                            n.cuda(), h0=d["h0"].cuda())
    for x in ("k", "v", "g", "beta"):
        d[x][1] = float("nan")
        d[x][:, 2] = float("inf")
        d[x][:, 4] = float("nan")
    c = to_cuda(d)
    ht = gdr_commit_path(c["k"], c["v"], c["g"], c["beta"], path.cuda(), n.cuda(), h0=c["h0"])
    assert torch.equal(ht[0], clean[0]) and torch.equal(ht[2], clean[2])
    assert torch.isnan(ht[1]).all()


def test_empty_batch():
    d = to_cuda(draw(1, 4, 1, 2, 64, 64, seed=12))
    z = {x: d[x][:0].contiguous() for x in ("k", "v", "g", "beta", "h0")}
    i32 = dict(dtype=torch.int32, device="cuda")
    assert gdr_commit_path(z["k"], z["v"], z["g"], z["beta"], torch.empty(0, 3, **i32),
                           torch.empty(0, **i32), h0=z["h0"]).shape == (0, 2, 64, 64)
