"""Routes of gdr_ssm_forward that need their own inputs: batches of more than a launch's table of
sequences, cut into segments, and a z that TMA cannot read."""
import pytest
import torch

from channelwise_gated_delta_gb300 import (GDR_FLAG_FORCE_GENERIC, gdr_device_check, gdr_flag_segments,
                                           gdr_ssm_forward, gdr_ssm_workspace_bytes)
from tests.layer_util import DT, spread
from tests.test_ssm_gpu import CHUNKS, WALK, check, draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,flags", [("bf16", 0), ("f32", 0), ("bf16", GDR_FLAG_FORCE_GENERIC)])
@pytest.mark.parametrize("segments", [0, 3])
def test_long_sequences_on_both_sides_of_a_table(dtype, flags, segments):
    """More than 256 sequences, long ones first, last, and around the places where a launch ends, states
    updated in place."""
    lens = [(5 * i) % 7 for i in range(530)]
    for i in (0, 100, 255, 256, 257, 400, 511, 512, 529):
        lens[i] = 65 + 26 * (i % 10)
    d = draw(lens, 1, 2, 64, 64, dtype, seed=7)
    cu = spread(lens)
    if segments:
        flags |= gdr_flag_segments(segments)
        # a state a segment: the long sequences have two or three
        states = 2 * 64 * 64 * 4 * (len(lens) + sum((n + 127) // 128 - 1 for n in lens))
        assert gdr_ssm_workspace_bytes(len(lens), 0, 1, 2, 64, 64, DT[dtype], cu, flags) > states
    h0 = d["h0"].clone()
    out, ht = gdr_ssm_forward(**dict(d, h0=h0), ht=h0, cu_seqlens=cu, flags=flags)
    gdr_device_check()
    assert ht is h0
    check(d, lens, out, ht, dtype, CHUNKS)


def test_chunks_on_both_sides_of_a_table():
    """As many long sequences, which the chunk kernel takes without segments too."""
    lens = [65 + (11 * i) % 70 for i in range(300)]
    d = draw(lens, 1, 1, 128, 128, "bf16", seed=8)
    for flags in (0, gdr_flag_segments(2)):
        out, ht = gdr_ssm_forward(**d, cu_seqlens=spread(lens), flags=flags)
        gdr_device_check()
        check(d, lens, out, ht, "bf16", CHUNKS)


@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("flags", [0, gdr_flag_segments(2), GDR_FLAG_FORCE_GENERIC])
@pytest.mark.parametrize("first,apart", [(1, 8), (0, 3), (5, 11)])
def test_a_z_that_tma_cannot_read(dv, flags, first, apart):
    """z not on 16 bytes, or its rows not a whole number of 16 bytes apart, beside x, b and c that are."""
    lens = [330, 70, 200]
    HV = 2
    d = draw(lens, 1, HV, 128, dv, "bf16", seed=dv, apart=False)
    wide = torch.zeros(sum(lens), HV * dv + apart, dtype=torch.bfloat16, device="cuda")
    z = wide[:, first:first + HV * dv]
    z.copy_(d["z"].flatten(1))
    z = z.unflatten(-1, (HV, dv))
    assert z.data_ptr() % 16 or z.stride(0) % 8
    out, ht = gdr_ssm_forward(**dict(d, z=z), cu_seqlens=spread(lens), flags=flags)
    gdr_device_check()
    generic = bool(flags & GDR_FLAG_FORCE_GENERIC)
    check(d, lens, out, ht, "bf16", WALK if generic else CHUNKS)
    if not generic:   # the same bits as with a z that it can read
        same, end = gdr_ssm_forward(**d, cu_seqlens=spread(lens), flags=flags)
        assert torch.equal(out, same) and torch.equal(ht, end)


def test_long_runs_are_alike():
    """Many CTAs over many chunks, other work between: the same bits each time."""
    N, T, HK, HV, D = 4, 4096, 16, 32, 128
    sets = []
    for seed in range(2):
        d = draw([T] * N, HK, HV, D, D, "bf16", seed=seed, z=seed == 1)
        sets.append({k: v.unflatten(0, (N, T)) if k in ("x", "b", "c", "dt", "z") and v is not None else v
                     for k, v in d.items()})
    want = [[t.clone() for t in gdr_ssm_forward(**d)] for d in sets]
    for _ in range(5):
        for d, w in zip(sets, want):
            assert all(torch.equal(p, q) for p, q in zip(gdr_ssm_forward(**d), w))
    gdr_device_check()
