"""Calls on a given stream whose outputs and workspaces nobody gave, while the current stream still
has work queued on blocks of their sizes that it has already given back."""
import pytest
import torch

from channelwise_gated_delta_gb300 import (gdr_commit_path, gdr_forward, gdr_forward_tree,
                                           gdr_state_cache, gdr_state_load, gdr_verify_drafts)
from channelwise_gated_delta_gb300.inputs import draw
from tests.parity_util import to_cuda

pytestmark = pytest.mark.gpu

B, T, HK, HV, D, V = 3, 40, 2, 4, 128, 1000


def calls():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rand = lambda *s: torch.rand(*s, device="cuda", generator=gen)
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
    x = to_cuda(draw(B, T, HK, HV, D, D, dtype=torch.bfloat16, seed=2))
    y = to_cuda(draw(B, T, HK, HV, D, D, dtype=torch.float32, seed=3))
    parent = torch.arange(T, dtype=torch.int32).expand(B, T) - 1
    p = torch.softmax(3 * rand(B, T, V), -1)
    tokens, coins, u = p.argmax(-1).int(), 0.01 * rand(B, T), rand(B)
    on_gpu, path, n = parent.contiguous().cuda(), i32([[0, 2, 5, 9]] * B), i32([4, 0, 2])
    cache, scale = gdr_state_cache(4, HV, D, D)
    cache.random_(-127, 128, generator=gen)
    scale.copy_(rand(4, HV, D))
    slots = i32([2, 0, 3])
    inputs = lambda d: [d[k] for k in ("q", "k", "v", "g", "beta")]
    return {
        "forward": lambda **kw: gdr_forward(*inputs(x), h0=x["h0"], **kw),
        "forward f32, a workspace": lambda **kw: gdr_forward(*inputs(y), h0=y["h0"], **kw),
        "tree": lambda **kw: (gdr_forward_tree(*inputs(y), parent, h0=y["h0"], **kw),),
        "verify": lambda **kw: gdr_verify_drafts(p, tokens, on_gpu, coins, u, **kw),
        "commit": lambda **kw: (gdr_commit_path(x["k"], x["v"], x["g"], x["beta"], path, n,
                                                h0=x["h0"], **kw),),
        "load": lambda **kw: (gdr_state_load(cache, scale, slots, **kw),),
    }


@pytest.mark.parametrize("name", ["forward", "forward f32, a workspace", "tree", "verify", "commit",
                                  "load"])
def test_outputs_are_not_written_by_work_of_the_current_stream(name):
    call = calls()[name]
    want = call()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)               # some 50 ms, in front of what fills the blocks
    sizes = [t.numel() * t.element_size() for t in want] + [1 << k for k in range(9, 26)]
    for size in sizes * 2:
        block = torch.empty(size, dtype=torch.uint8, device="cuda")
        block.fill_(0x7f)
        del block
    got = call(stream=other)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
