"""The operators around the recurrence at their edges: rows beyond 32-bit offsets, the smallest
shapes, calls on two streams at once, and a process whose first calls are captured."""
import os
import subprocess
import sys

import pytest
import torch

from channelwise_gated_delta_gb300 import (GDR_FLAG_FORCE_GENERIC, gdr_device_check, gdr_flag_segments,
                                           gdr_qk_norm, gdr_rope_freqs, gdr_short_conv,
                                           gdr_ssm_forward)
from tests.test_ssm_gpu import CHUNKS, WALK, check, draw

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def far_rows():
    """70 rows, 2^26 elements of bf16 apart: the last ones lie beyond 2^32 elements."""
    rows = torch.empty(70, 2 ** 26, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(3)
    rows[:, :2048] = torch.randn(70, 2048, generator=gen).to(torch.bfloat16).cuda()
    yield rows
    del rows
    torch.cuda.empty_cache()


def test_rows_beyond_32_bit_offsets(far_rows):
    x, near = far_rows[:, :2048], far_rows[:, :2048].contiguous()
    w = torch.randn(1024, 4, device="cuda")
    for got, want in zip(gdr_short_conv(x[:, :1024], w, cu_seqlens=[0, 70]),
                         gdr_short_conv(near[:, :1024], w, cu_seqlens=[0, 70])):
        assert torch.equal(got, want)
    out = far_rows[:, 4096:4096 + 1024]
    gdr_short_conv(near[:, :1024], w, cu_seqlens=[0, 70], out=out, store_st=False)
    assert torch.equal(out, gdr_short_conv(near[:, :1024], w, cu_seqlens=[0, 70])[0])
    positions = torch.arange(70, dtype=torch.int32, device="cuda")
    heads = lambda t, a, b: t[:, a:b].unflatten(-1, (-1, 128))
    args = dict(positions=positions, freqs=gdr_rope_freqs(64))
    for got, want in zip(gdr_qk_norm(heads(x, 0, 1024), heads(x, 1024, 1536), **args),
                         gdr_qk_norm(heads(near, 0, 1024), heads(near, 1024, 1536), **args)):
        assert torch.equal(got, want)
    dt, a = torch.rand(70, 4, device="cuda"), -torch.rand(4, device="cuda")
    for flags in (0, GDR_FLAG_FORCE_GENERIC):
        runs = [gdr_ssm_forward(heads(t, 0, 512), heads(t, 512, 768), heads(t, 768, 1024), dt, a,
                                z=heads(t, 1024, 1536), cu_seqlens=[0, 70], flags=flags)
                for t in (x, near)]
        assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    gdr_device_check()


@pytest.mark.parametrize("T", [1, 2, 130, 1025])
@pytest.mark.parametrize("flags", [0, gdr_flag_segments(5)])
def test_one_head_of_32(T, flags):
    for dtype, unit in (("bf16", CHUNKS), ("f32", WALK)):
        d = draw([T], 1, 1, 32, 32, dtype, seed=T, apart=False)
        check(d, [T], *gdr_ssm_forward(**d, cu_seqlens=[0, T], flags=flags), dtype, unit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_streams_at_once(dtype):
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets = [draw([1500, 70], 2, 4, 128, 64, dtype, seed=i) for i in range(2)]
    call = lambda d, **k: gdr_ssm_forward(**d, cu_seqlens=[0, 1500, 1570], **k)
    want = [call(d) for d in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for d, side in zip(sets, sides):
            got.append(call(d, stream=side))
    torch.cuda.synchronize()
    for i, pair in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(pair, want[i % 2])), i
    gdr_device_check()


def test_graphs_share_nothing():
    """Two captured packed calls of different offsets, replayed on two streams at once."""
    sets = [(draw(lens, 1, 2, 128, 128, "bf16", seed=9), [0, lens[0], sum(lens)])
            for lens in ([3000, 40], [700, 2500])]
    want, graphs, got = [], [], []
    for d, cu in sets:
        want.append(gdr_ssm_forward(**d, cu_seqlens=cu))
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(gdr_ssm_forward(**d, cu_seqlens=cu))
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for graph, side in zip(graphs, sides):
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])


@pytest.mark.parametrize("segments", [0, 4])
@pytest.mark.parametrize("steps", [(0.001, 0.1), (0.05, 0.5)])
def test_the_state_of_chunks_is_near_float32(segments, steps):
    """A weighted value enters the state as three bf16 numbers of which the last one's rounding
    stays: at most 2^-18 of the value, 1.6e-6 rms where all weights lie worst between powers of
    two, 8e-7 over weights of any size; float32 sums add 2e-7.  (A pair would leave 4e-6.)"""
    d = draw([1200], 2, 4, 128, 128, "bf16", seed=11, z=False, h0=False, steps=steps)
    _, ht = gdr_ssm_forward(**d, cu_seqlens=[0, 1200], flags=gdr_flag_segments(segments) if segments else 0)
    x, b, dt, a, bias = (d[k].double() for k in ("x", "b", "dt", "a", "dt_bias"))
    step = torch.nn.functional.softplus(dt + bias)
    left = (step * a).flip(0).cumsum(0).flip(0) - step * a      # log of the decay behind each token
    S = torch.einsum("thk,thv->hkv", b.repeat_interleave(2, 1), x * (step * left.exp())[..., None])
    assert (ht[0].double() - S).norm() <= 2.0 ** -19 * S.norm()


FIRST = """
import torch
from channelwise_gated_delta_gb300 import gdr_qk_norm, gdr_rope_freqs, gdr_short_conv, gdr_ssm_forward
gen = torch.Generator().manual_seed(0)
n = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()
x, w, dt = n(2, 300, 1024), n(1024, 4).float(), torch.rand(2, 300, 4, generator=gen).cuda()
positions = torch.arange(300, dtype=torch.int32).repeat(2, 1).cuda()
freqs, a = gdr_rope_freqs(128), -torch.ones(4).cuda()
def run():
    y, st = gdr_short_conv(x, w)
    heads = y.unflatten(-1, (-1, 128))
    q, k = gdr_qk_norm(heads[:, :, :2], heads[:, :, 2:4], positions=positions, freqs=freqs)
    out, ht = gdr_ssm_forward(heads[:, :, 4:], k, q, dt, a)
    return st, q, out, ht
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(got, run()))
print("the same")
"""


def test_first_calls_captured():
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "the same" in r.stdout, r.stderr[-2000:]
