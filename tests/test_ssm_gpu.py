"""gdr_ssm_forward against its recurrence in float64."""
import pytest
import torch

from channelwise_gated_delta_gb300 import (GDR_FLAG_FORCE_GENERIC, GDR_FLAG_NO_SEGMENTS,
                                           gdr_device_check, gdr_flag_segments, gdr_ssm_forward,
                                           gdr_ssm_workspace_bytes)
from oracle import layer_ops
from tests.layer_util import DT, f64, near, spread

pytestmark = pytest.mark.gpu

# the relative error of an update: token by token eight float32 roundings; on the tensor cores
# each product's one operand is a pair of bf16 numbers that is off by 2^-16, the decays of a chunk
# are differences of sums, and up to 64 terms meet in a float32 sum
WALK, CHUNKS = 2.0 ** -21, 2.0 ** -15
# with bf16 inputs the outputs of a chunk read a copy of the state rounded to bf16: each product
# with c is off by 2^-8 of its size, and so is their sum by 2^-8 of the sum of the sizes
READ = {"bf16": 2.0 ** -8, "f32": 0.0}


def draw(lens, HK, HV, dk, dv, dtype, seed=0, z=True, h0=True, apart=True, steps=(0.001, 0.1), A=16.0,
         wide=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    dt, rows = DT[dtype], sum(lens)
    mixed = n(rows, HV * dv + 2 * HK * dk + wide).to(dt).cuda()
    at = HV * dv
    start = torch.empty(HV).uniform_(*steps, generator=gen)
    d = dict(x=mixed[:, :at].unflatten(-1, (HV, dv)),
             b=mixed[:, at:at + HK * dk].unflatten(-1, (HK, dk)),
             c=mixed[:, at + HK * dk:at + 2 * HK * dk].unflatten(-1, (HK, dk)),
             dt=(0.5 * n(rows, HV)).cuda(), a=-(1 + (A - 1) * torch.rand(HV, generator=gen)).cuda(),
             d=(1 + n(HV)).cuda(), z=n(rows, HV, dv).to(dt).cuda() if z else None,
             dt_bias=torch.log(torch.expm1(start)).cuda(),
             h0=n(len(lens), HV, dk, dv).cuda() if h0 else None)
    if not apart:
        d = {k: None if v is None else v.contiguous() for k, v in d.items()}
    return d


def check(d, lens, out, ht, dtype, unit, softplus=True):
    cu = spread(lens)
    for i, (p, q) in enumerate(zip(cu, cu[1:])):
        r = {k: None if v is None else f64(v[p:q] if k in ("x", "b", "c", "dt", "z") else
                                           v[i] if k == "h0" else v) for k, v in d.items()}
        ref, S, err, E = layer_ops.ssm(**r, softplus=softplus, unit=unit,
                                       read=READ[dtype] if unit == CHUNKS else 0.0)
        near("out[%d]" % i, out[p:q], ref, err, dtype)
        if ht is not None:
            near("ht[%d]" % i, ht[i], S, E, "f32")


LENS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 0, 129, 200]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_packed(dtype, dk, dv):
    d = draw(LENS, 2, 6, dk, dv, dtype, seed=dk + dv)
    out, ht = gdr_ssm_forward(**d, cu_seqlens=spread(LENS))
    gdr_device_check()
    check(d, LENS, out, ht, dtype, CHUNKS)
    out, ht = gdr_ssm_forward(**d, cu_seqlens=spread(LENS), flags=GDR_FLAG_FORCE_GENERIC)
    check(d, LENS, out, ht, dtype, WALK)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("HK,HV,dk,dv", [(1, 1, 128, 128), (2, 4, 128, 128), (3, 9, 64, 32),
                                         (16, 32, 128, 128), (1, 7, 32, 64), (1, 2, 64, 128)])
@pytest.mark.parametrize("B", [1, 3, 40])
def test_single_tokens(dtype, HK, HV, dk, dv, B):
    d = draw([1] * B, HK, HV, dk, dv, dtype, seed=B)
    lead = {k: v[:, None] for k, v in d.items() if k in ("x", "b", "c", "dt", "z")}
    out, ht = gdr_ssm_forward(**dict(d, **lead))
    gdr_device_check()
    check(d, [1] * B, out[:, 0], ht, dtype, WALK)
    h0 = d["h0"].clone()
    again, end = gdr_ssm_forward(**dict(d, **lead, h0=h0), ht=h0)
    assert end is h0 and torch.equal(again, out) and torch.equal(h0, ht)
    lead["z"] = None
    out, none = gdr_ssm_forward(**dict(d, **lead, h0=None, d=None, dt_bias=None), softplus=False,
                                store_ht=False)
    assert none is None
    check(dict(d, z=None, h0=None, d=None, dt_bias=None), [1] * B, out[:, 0], None, dtype, WALK, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,HK,HV,dk,dv", [(2, 150, 1, 2, 128, 128), (1, 64, 2, 2, 64, 64),
                                             (3, 257, 1, 3, 128, 64), (1, 1000, 1, 1, 32, 32)])
def test_dense(dtype, B, T, HK, HV, dk, dv):
    lens = [T] * B
    d = draw(lens, HK, HV, dk, dv, dtype, seed=T, apart=False)
    dense = {k: v.unflatten(0, (B, T)) if k in ("x", "b", "c", "dt", "z") else v for k, v in d.items()}
    out, ht = gdr_ssm_forward(**dense)
    gdr_device_check()
    check(d, lens, out.flatten(0, 1), ht, dtype, CHUNKS)


@pytest.mark.parametrize("dtype,flags", [("bf16", 0), ("f32", 0), ("bf16", GDR_FLAG_FORCE_GENERIC)])
@pytest.mark.parametrize("n", [2, 3, 7])
def test_segments(dtype, flags, n):
    """Walks cut into segments, with states handed over in place."""
    lens = [600, 0, 1, 300, 64]
    d = draw(lens, 1, 2, 128, 128, dtype, seed=n)
    flags |= gdr_flag_segments(n)
    h0 = d["h0"].clone()
    out, ht = gdr_ssm_forward(**dict(d, h0=h0), ht=h0, cu_seqlens=spread(lens), flags=flags)
    gdr_device_check()
    assert gdr_ssm_workspace_bytes(5, 0, 1, 2, 128, 128, DT[dtype], spread(lens), flags) > 0
    check(d, lens, out, ht, dtype, CHUNKS)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_fast_and_slow_decays(dtype):
    """Steps and decays of every size: states that are gone within a token, and ones that stay."""
    lens = [200, 130]
    for steps, A in (((1.0, 5.0), 16.0), ((1e-6, 1e-5), 1.5), ((0.5, 20.0), 100.0)):
        d = draw(lens, 1, 2, 128, 128, dtype, steps=steps, A=A)
        out, ht = gdr_ssm_forward(**d, cu_seqlens=spread(lens))
        check(d, lens, out, ht, dtype, CHUNKS)


@pytest.mark.parametrize("wide", [0, 1, 3, 8])
def test_rows_at_any_distance(wide):
    """Parts of a projection whose rows are a whole number of 16 bytes apart, or not."""
    d = draw([70, 3, 100], 1, 2, 128, 128, "bf16", wide=wide)
    out, ht = gdr_ssm_forward(**d, cu_seqlens=[0, 70, 73, 173])
    check(d, [70, 3, 100], out, ht, "bf16", CHUNKS)


def test_the_neighbours_values_do_not_matter():
    """What stands in the rows of other sequences, NaN or infinite, reaches no output of one."""
    lens = [70, 30, 100, 1, 64]
    d = draw(lens, 1, 2, 128, 128, "bf16", wide=8)
    cu = spread(lens)
    clean, end = gdr_ssm_forward(**d, cu_seqlens=cu)
    for i in (0, 2, 4):
        for n in ("x", "b", "c", "dt", "z"):
            d[n][cu[i]:cu[i + 1]] = float("nan") if i != 2 else float("inf")
    out, ht = gdr_ssm_forward(**d, cu_seqlens=cu)
    for i in (1, 3):
        assert torch.equal(out[cu[i]:cu[i + 1]], clean[cu[i]:cu[i + 1]]) and torch.equal(ht[i], end[i])


def test_many_sequences():
    """More sequences than a launch's table holds."""
    lens = [(3 * i) % 4 for i in range(600)]
    d = draw(lens, 1, 1, 32, 32, "f32")
    out, ht = gdr_ssm_forward(**d, cu_seqlens=spread(lens))
    check(d, lens, out, ht, "f32", WALK)
    d = draw(lens, 1, 1, 64, 64, "bf16")
    out, ht = gdr_ssm_forward(**d, cu_seqlens=spread(lens), flags=gdr_flag_segments(2))
    check(d, lens, out, ht, "bf16", CHUNKS)


def test_pieces_agree_with_the_whole():
    """A prompt, then single tokens: the states are those of the whole."""
    d = draw([140], 1, 2, 128, 128, "bf16")
    out, ht = gdr_ssm_forward(**d, cu_seqlens=[0, 140])
    state, at, parts = d["h0"].clone(), 0, []
    for n in (100, 1, 1, 38):
        part = {k: v[at:at + n] if k in ("x", "b", "c", "dt", "z") else v for k, v in d.items()}
        o, _ = gdr_ssm_forward(**dict(part, h0=state), ht=state, cu_seqlens=[0, n])
        parts.append(o)
        at += n
    check(d, [140], torch.cat(parts), state, "bf16", CHUNKS)


def test_runs_are_alike():
    """The same call twice gives the same bits, segments or not."""
    d = draw([2000], 2, 4, 128, 128, "bf16")
    for flags in (0, GDR_FLAG_NO_SEGMENTS, gdr_flag_segments(5)):
        a = gdr_ssm_forward(**d, cu_seqlens=[0, 2000], flags=flags)
        b = gdr_ssm_forward(**d, cu_seqlens=[0, 2000], flags=flags)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype,flags", [("bf16", 0), ("f32", 0), ("bf16", gdr_flag_segments(3))])
@pytest.mark.parametrize("name", ["x", "b", "c", "dt", "z"])
def test_values_that_are_not_finite_stay_behind_their_token(dtype, flags, name):
    """What is not finite reaches no output of a token before it, wherever it stands in a chunk, and
    none of another column (x, z) or head."""
    T, HK, HV, D = 200, 1, 3, 128
    d = draw([T], HK, HV, D, D, dtype, seed=9)
    clean, _ = gdr_ssm_forward(**d, cu_seqlens=[0, T], flags=flags)
    for t, v in ((0, "nan"), (5, "inf"), (37, "-inf"), (63, "nan"), (64, "nan"), (100, "inf"), (199, "nan")):
        e = dict(d, **{name: d[name].clone()})
        if name == "dt":
            e["dt"][t, 1] = float(v)
        else:
            e[name][t, 0 if name in "bc" else 1, 70] = float(v)
        out, _ = gdr_ssm_forward(**e, cu_seqlens=[0, T], flags=flags)
        gdr_device_check()
        # nothing else than a chunk's own reference may differ: compare by the tolerance of a rounding
        tol = 4e-2 * clean.float().abs().amax()
        same = torch.ones(T, HV, D, dtype=torch.bool, device="cuda")
        if name in "bc":
            same[t:] = False
        elif name == "dt":
            same[t:, 1] = False
        else:
            same[t:, 1, 70] = False
        assert torch.isfinite(out[same].float()).all(), (name, t)
        assert ((out - clean).float()[same].abs() <= tol).all(), (name, t)
        if name != "dt" and v == "nan":
            hit = out[t, :, :] if name in "bc" else out[t, 1, 70]
            assert not torch.isfinite(hit.float()).any(), (name, t)
