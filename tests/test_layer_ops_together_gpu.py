"""The operators around the recurrence together with it, as a layer runs them."""
import numpy as np
import pytest
import torch

import oracle
from channelwise_gated_delta_gb300 import (gdr_device_check, gdr_forward, gdr_forward_varlen,
                                           gdr_qk_norm, gdr_rope_freqs, gdr_short_conv,
                                           gdr_ssm_forward, gdr_state_cache, gdr_state_load,
                                           gdr_state_store)
from oracle import layer_ops
from tests.layer_util import f64, spread

pytestmark = pytest.mark.gpu

HK, HV, D = 1, 2, 128


def delta_layer(x, w, s0, h0, g, beta, cu, positions, freqs, st=None, ht=None):
    """Convolution of q, k and v, norms and rotation of q and k, the delta rule."""
    mixed, st = gdr_short_conv(x, w, cu_seqlens=cu, s0=s0, st=st)
    q, k, v = mixed.split([HK * D, HK * D, HV * D], -1)
    q, k = gdr_qk_norm(q.unflatten(-1, (HK, D)), k.unflatten(-1, (HK, D)), positions=positions,
                       freqs=freqs, q_scale=D ** -0.5)
    out, ht = gdr_forward_varlen(q, k, v.unflatten(-1, (HV, D)).contiguous(), g, beta, cu, h0=h0, ht=ht)
    return out, st, ht


def draw(rows, n, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    wide = (2 * HK + HV) * D
    return dict(x=r(rows, wide).bfloat16().cuda(), w=(0.5 * r(wide, 4)).cuda(),
                s0=r(n, 3, wide).bfloat16().cuda(), h0=(0.3 * r(n, HV, D, D)).cuda(),
                g=-torch.nn.functional.softplus(r(rows, HV, D)).cuda(),
                beta=torch.sigmoid(r(rows, HV)).cuda())


def test_delta_layer():
    lens = [70, 1, 40]
    cu = spread(lens)
    d = draw(sum(lens), 3)
    pos = torch.cat([100000 + torch.arange(n) for n in lens]).int().cuda()
    out, st, ht = delta_layer(**d, cu=cu, positions=pos, freqs=gdr_rope_freqs(64))
    gdr_device_check()
    inv = [10000.0 ** (-2 * i / 64) for i in range(32)]
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        y, state, _ = layer_ops.short_conv(f64(d["x"][a:b]), f64(d["w"]), None, f64(d["s0"][i]))
        q, k, v = (t.reshape(b - a, -1, D) for t in np.split(y, [HK * D, 2 * HK * D], -1))
        q, _ = layer_ops.qk_norm(q, scale=D ** -0.5, positions=f64(pos[a:b]), inv_freq=inv)
        k, _ = layer_ops.qk_norm(k, positions=f64(pos[a:b]), inv_freq=inv)
        ro, rh = oracle.recurrence(*(np.ascontiguousarray(t[None]) for t in
                                     (q, k, v, f64(d["g"][a:b]), f64(d["beta"][a:b]))),
                                   f64(d["h0"][i:i + 1]))
        assert np.array_equal(f64(st[i]), state)
        # gdr_forward's tolerance, and as much again for the roundings of q, k and v to bf16
        for got, ref in ((out[a:b], ro[0]), (ht[i], rh[0])):
            assert np.abs(f64(got) - ref).max() <= 4e-2 * np.abs(ref).max()


def test_prompt_then_tokens_in_a_graph():
    """A prompt, then a captured step of both kinds of layer, replayed token by token on states
    that it updates in place, is the whole sequence; the states pass through the 8-bit cache."""
    T, P = 48, 40
    d = draw(T, 1, seed=3)
    freqs = gdr_rope_freqs(D)
    pos = torch.arange(T, dtype=torch.int32).cuda()
    whole, st_end, ht_end = delta_layer(**d, cu=[0, T], positions=pos, freqs=freqs)
    rows = lambda a, b: {k: v[a:b] if k in ("x", "g", "beta") else v for k, v in d.items()}
    head, st, ht = delta_layer(**rows(0, P), cu=[0, P], positions=pos[:P], freqs=freqs)

    dt = torch.randn(T, HV).cuda()
    A = -torch.rand(HV).cuda()

    def scan(out, a, b, h0, ht=None):
        bc = d["x"][a:b, :2 * HK * D].unflatten(-1, (2 * HK, D))
        return gdr_ssm_forward(out[None], bc[None, :, :HK], bc[None, :, HK:], dt[None, a:b], A, h0=h0,
                               ht=ht, z=out[None])

    both, end = scan(whole, 0, T, None)
    first, state = scan(head, 0, P, None)

    step = {k: v.clone() for k, v in rows(P, P + 1).items()}
    spos, sdt = pos[P:P + 1].clone(), dt[None, P:P + 1].clone()

    def one():
        # gdr_forward_varlen copies tables from the host, so a captured step takes the dense call
        mixed, _ = gdr_short_conv(step["x"][None], step["w"], s0=st, st=st)
        q, k, v = mixed.split([HK * D, HK * D, HV * D], -1)
        q, k = gdr_qk_norm(q.unflatten(-1, (HK, D)), k.unflatten(-1, (HK, D)), positions=spos[None],
                           freqs=freqs, q_scale=D ** -0.5)
        o, _ = gdr_forward(q, k, v.unflatten(-1, (HV, D)).contiguous(), step["g"][None],
                           step["beta"][None], ht, ht=ht)
        bc = step["x"][None, :, :2 * HK * D].unflatten(-1, (2 * HK, D))
        y, _ = gdr_ssm_forward(o, bc[:, :, :HK], bc[:, :, HK:], sdt, A, h0=state, ht=state, z=o)
        return o[0], y[0]

    keep = [t.clone() for t in (st, ht, state)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, y = one()
    for t, k in zip((st, ht, state), keep):
        t.copy_(k)
    for t in range(P, T):
        for k in ("x", "g", "beta"):
            step[k].copy_(d[k][t:t + 1])
        spos.copy_(pos[t:t + 1])
        sdt.copy_(dt[None, t:t + 1])
        graph.replay()
        for got, ref in ((o, whole[t:t + 1]), (y, both[:, t])):
            assert (got.float() - ref.float()).abs().max() <= 4e-2 * ref.float().abs().max()
    gdr_device_check()
    assert torch.equal(st, st_end)
    for got, ref in ((ht, ht_end), (state, end)):
        assert (got - ref).abs().max() <= 2e-2 * ref.abs().max()
    cache, scale = gdr_state_cache(2, HV, D, D)
    slot = torch.tensor([1], dtype=torch.int32, device="cuda")
    gdr_state_store(state, slot, cache, scale)
    back = gdr_state_load(cache, scale, slot)
    assert ((back - state).abs() <= 0.501 * scale[1][None, ..., None]).all()


def test_on_another_stream():
    """On a given stream, whose inputs are made there; outputs are that stream's memory."""
    d = draw(300, 1, seed=5)
    want = delta_layer(**d, cu=[0, 300], positions=None, freqs=None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        busy = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            busy = busy @ busy * 1e-2
        x = d["x"].clone()
    mixed, st = gdr_short_conv(x, d["w"], cu_seqlens=[0, 300], s0=d["s0"], stream=side)
    heads = mixed.unflatten(-1, (-1, D))
    q, k = gdr_qk_norm(heads[:, :HK], heads[:, HK:2 * HK], q_scale=D ** -0.5, stream=side)
    y, _ = gdr_ssm_forward(heads[:, 2 * HK:], k, q, d["g"][..., 0].contiguous(),
                           -torch.ones(HV).cuda(), cu_seqlens=[0, 300], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(st, want[1])
    mixed2, _ = gdr_short_conv(d["x"], d["w"], cu_seqlens=[0, 300], s0=d["s0"])
    heads = mixed2.unflatten(-1, (-1, D))
    q2, k2 = gdr_qk_norm(heads[:, :HK], heads[:, HK:2 * HK], q_scale=D ** -0.5)
    y2, _ = gdr_ssm_forward(heads[:, 2 * HK:], k2, q2, d["g"][..., 0].contiguous(),
                            -torch.ones(HV).cuda(), cu_seqlens=[0, 300])
    assert torch.equal(mixed, mixed2) and torch.equal(q, q2) and torch.equal(k, k2)
    assert torch.equal(y, y2)
