"""gdr_commit_path on float32 nodes with more heads of 128 x 128 than SMs: both groups of the
persistent kernel, its three state buffers in turn and the hand-over from head to head, with the four
producer warps a group that float32 nodes take.  Tolerance as in test_commit_gpu.py."""
import pytest
import torch

from channelwise_gated_delta_gb300.inputs import draw
from tests.test_commit_gpu import check, paths

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h0", [True, False])
@pytest.mark.parametrize("scalar", [False, True])
def test_many_heads_of_all_lengths(scalar, h0):
    d = draw(60, 40, 8, 32, 128, 128, dtype=torch.float32, h0=h0, seed=21, scalar_gate=scalar)
    p = paths(60, 40, 40, lengths=[1, 4, 0, 9, 2, 37, 5, 1, 8, 3, 40, 1, 1, 12])
    ht = check(d, *p)
    for _ in range(3):
        assert torch.equal(ht, check(d, *p, in_place=h0))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,HK,HV", [(7, 16, 32), (19, 16, 16), (39, 4, 8), (33, 8, 16), (61, 5, 15)])
def test_from_one_to_seven_heads_an_sm(B, HK, HV, dtype):
    """Also odd numbers, where one group has a head more than the other, or the only one."""
    d = draw(B, 9, HK, HV, 128, 128, dtype=dtype, seed=B)
    check(d, *paths(B, 9, 9, seed=B))


@pytest.mark.parametrize("lengths", [[0], [1], [4], [5], [0, 33], [8, 1]])
def test_equal_and_alternating_lengths(lengths):
    d = draw(24, 36, 16, 32, 128, 128, dtype=torch.float32, seed=22)
    check(d, *paths(24, 36, 36, lengths=lengths))
