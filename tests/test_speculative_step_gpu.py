"""The calls of a speculative step together: the example, and the same step in a CUDA graph."""
import pytest
import torch

from channelwise_gated_delta_gb300 import (gdr_commit_path, gdr_state_cache, gdr_state_load,
                                           gdr_state_store, gdr_trace_enable, gdr_trace_read,
                                           gdr_verify_drafts)
from examples import speculative_step

pytestmark = pytest.mark.gpu


def test_example():
    """Accepted tokens leave the states of one forward pass over them, within the 2e-2 of that
    pass's bf16 products; a row of the cache is off by at most 1/254 of its largest value."""
    r = speculative_step.run(batch=3, steps=6)
    assert r["counts"].shape == (3, 6) and int(r["counts"].min()) >= 1
    assert int(r["counts"].max()) > 1            # some drafts stand
    assert r["error"] <= 2e-2
    assert r["cache_error"] <= 1 / 254 * 1.001


def problem(seed, B=3, T=7, V=1000, HK=2, HV=4, d=128, slots=5):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    uni = lambda *s: torch.rand(*s, device="cuda", generator=gen)
    logits = 2 * rnd(B, T, V)
    parent = (torch.arange(T, device="cuda", dtype=torch.int32) - 1).expand(B, T)
    return dict(p=torch.softmax(logits, -1), q=torch.softmax(logits + 0.5 * rnd(B, T, V), -1),
                tokens=logits.argmax(-1).roll(1, 1).int(), parent=parent, coins=uni(B, T), u=uni(B),
                k=torch.nn.functional.normalize(rnd(B, T, HK, d), dim=-1).bfloat16(),
                v=rnd(B, T, HV, d).bfloat16(), g=-uni(B, T, HV, d), beta=uni(B, T, HV),
                state=rnd(B, HV, d, d),
                slots=torch.randperm(slots, device="cuda", generator=gen)[:B].int())


def step(x, cache, scale):
    path, n, token = gdr_verify_drafts(x["p"], x["tokens"], x["parent"], x["coins"], x["u"],
                                       q=x["q"], max_path=5)
    gdr_commit_path(x["k"], x["v"], x["g"], x["beta"], path, n, h0=x["state"], ht=x["state"])
    gdr_state_store(x["state"], x["slots"], cache, scale)
    return path, n, token, gdr_state_load(cache, scale, x["slots"])


def test_in_a_cuda_graph():
    """One graph, replayed on other inputs, gives what the calls give."""
    x = problem(1)
    cache, scale = gdr_state_cache(5, 4, 128, 128)
    held = {n: t.clone() if n != "parent" else t for n, t in x.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held, cache, scale)      # the first call of each looks things up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(held, cache, scale)
    for seed in (2, 3):
        y = problem(seed)
        for n in held:
            if n != "parent":
                held[n].copy_(y[n])
        graph.replay()
        want = step(y, *gdr_state_cache(5, 4, 128, 128))
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        assert torch.equal(held["state"], y["state"])


def test_trace_names_the_kernels():
    x = problem(4)
    cache, scale = gdr_state_cache(5, 4, 128, 128)
    gdr_trace_enable()
    try:
        step(x, cache, scale)
        torch.cuda.synchronize()
        got = gdr_trace_read()
    finally:
        gdr_trace_enable(False)
    for name in ("gdr_verify_kernel", "gdr_commit_kernel", "gdr_state_store_kernel",
                 "gdr_state_load_kernel"):
        assert got[name][0] == 1, got


def test_results_do_not_change_from_run_to_run():
    x = problem(5, B=40)
    x["slots"] = torch.arange(40, device="cuda").int()
    first = None
    for _ in range(5):
        y = {n: t.clone() if n != "parent" else t for n, t in x.items()}
        got = step(y, *gdr_state_cache(40, 4, 128, 128)) + (y["state"],)
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
