"""gdr_qk_norm against its definition in float64."""
import pytest
import torch

from channelwise_gated_delta_gb300 import gdr_qk_norm, gdr_rope_freqs
from oracle import layer_ops
from tests.layer_util import DT, f64, near

pytestmark = pytest.mark.gpu


def draw(rows, HQ, HK, d, dtype, seed=0, wide=0, weights=True, far=1000):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    both = n(rows, (HQ + HK) * d + wide).to(DT[dtype]).cuda()
    return dict(q=both[:, :HQ * d].unflatten(-1, (HQ, d)),
                k=both[:, HQ * d:(HQ + HK) * d].unflatten(-1, (HK, d)),
                weight_q=(1 + 0.3 * n(d)).cuda() if weights else None,
                weight_k=(1 + 0.3 * n(d)).cuda() if weights else None), torch.randint(
                    -far, far, (rows,), generator=gen, dtype=torch.int32).cuda()


def check(a, outs, dtype, norm, scale, eps=1e-6, positions=None, inv_freq=None, interleaved=False):
    for n, out, f in (("q", outs[0], scale), ("k", outs[1], 1.0)):
        ref, err = layer_ops.qk_norm(f64(a[n]), f64(a["weight_" + n]), f, norm == "rms", eps,
                                     f64(positions), inv_freq, interleaved)
        near(n, out, ref, err, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("rows,HQ,HK", [(1, 1, 1), (1, 33, 5), (7, 4, 3), (130, 9, 2), (3000, 2, 2)])
def test_norms(dtype, d, rows, HQ, HK):
    a, _ = draw(rows, HQ, HK, d, dtype, seed=rows + d)
    for norm, scale in (("l2", d ** -0.5), ("rms", 1.0)):
        check(a, gdr_qk_norm(**a, norm=norm, q_scale=scale), dtype, norm, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,d_rot", [(32, 16), (32, 32), (64, 32), (64, 48), (128, 128), (128, 80),
                                     (256, 16), (256, 256)])
def test_rotation(dtype, interleaved, d, d_rot):
    inv = [10000.0 ** (-2.0 * i / d_rot) for i in range(d_rot // 2)]
    freqs = gdr_rope_freqs(d_rot)
    for rows, HQ, HK, far in ((1, 5, 2, 10), (33, 3, 3, 10 ** 6), (600, 2, 1, 2 ** 31 - 1)):
        a, pos = draw(rows, HQ, HK, d, dtype, seed=rows, weights=rows == 33, far=far)
        outs = gdr_qk_norm(**a, norm="rms", positions=pos, freqs=freqs, interleaved=interleaved)
        if far < 10 ** 7:
            check(a, outs, dtype, "rms", 1.0, positions=pos, inv_freq=inv, interleaved=interleaved)
        else:
            # in float64 an angle of 2^31 is off by 2^-22: whole turns are taken out in whole numbers
            turns = [int(f) % 2 ** 64 for f in freqs]
            for n, out in (("q", outs[0]), ("k", outs[1])):
                for r in range(0, rows, 37):
                    small = [(int(pos[r]) * t % 2 ** 64) / 2.0 ** 64 * 2 * 3.141592653589793238
                             for t in turns]
                    ref, err = layer_ops.qk_norm(f64(a[n][r:r + 1]), None, 1.0, True, 1e-6, [1.0],
                                                 small, interleaved)
                    near(n, out[r:r + 1], ref, err, dtype)


def test_in_place_in_a_projection():
    """q and k replaced where they stand, between each other's rows and beside others."""
    a, pos = draw(50, 4, 2, 64, "bf16", wide=72)
    freqs = gdr_rope_freqs(32)
    want = gdr_qk_norm(**a, positions=pos, freqs=freqs)
    base = a["q"]._base if a["q"]._base is not None else None
    rest = base[:, 6 * 64:].clone()
    got = gdr_qk_norm(**a, positions=pos, freqs=freqs, out_q=a["q"], out_k=a["k"])
    assert got[0] is a["q"] and torch.equal(a["q"], want[0]) and torch.equal(a["k"], want[1])
    assert torch.equal(base[:, 6 * 64:], rest)


def test_dense_batches_and_given_outputs():
    a, pos = draw(24, 3, 1, 128, "f32")
    want = gdr_qk_norm(**a, positions=pos, freqs=gdr_rope_freqs(128))
    q, k = a["q"].reshape(2, 12, 3, 128), a["k"].reshape(2, 12, 1, 128)
    room = torch.zeros(2, 12, 5, 128, device="cuda")
    got = gdr_qk_norm(q, k, a["weight_q"], a["weight_k"], positions=pos.reshape(2, 12),
                      freqs=gdr_rope_freqs(128), out_q=room[:, :, 1:4], out_k=room[:, :, 4:])
    assert torch.equal(got[0].reshape(24, 3, 128), want[0])
    assert torch.equal(got[1].reshape(24, 1, 128), want[1]) and (room[:, :, 0] == 0).all()
    empty = gdr_qk_norm(q[:0], k[:0])
    assert empty[0].shape == (0, 12, 3, 128)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zeros_and_extremes(dtype):
    """A head of zeros stays zeros, with and without eps; a NaN stays in its head; large and small
    heads come out at their size."""
    q = torch.randn(4, 6, 64).to(DT[dtype]).cuda()
    q[0, 0] = 0
    q[1, 1, 5] = float("nan")
    q[2, 2] *= 1e15
    q[3, 3] *= 1e-15
    for eps in (0.0, 1e-6):
        out, _ = gdr_qk_norm(q, q.clone(), eps=eps)
        assert (out[0, 0] == 0).all() and out[1, 1].isnan().all()
        ok = torch.ones(4, 6, dtype=torch.bool)
        ok[1, 1] = False
        assert torch.isfinite(out.float().cpu()[ok]).all()
        ref, err = layer_ops.qk_norm(f64(q[2:3]), eps=eps)
        near("large", out[2:3], ref, err, dtype)
        if eps == 0:
            ref, err = layer_ops.qk_norm(f64(q[3:4]), eps=eps)
            near("small", out[3:4], ref, err, dtype)
