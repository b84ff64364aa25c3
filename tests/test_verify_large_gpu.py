"""gdr_verify_drafts over the longest rows it takes, against the oracle's rule (equality).  A warp of
the streamed form sums its part of a row in batches of 1024 elements and keeps one sum a lane: above
32 batches (2,097,152 elements for one tree, 262,144 where a tree has one CTA) a lane holds several,
and refusals, the search and the ends of the row go by groups of batches."""
import numpy as np
import pytest
import torch

from tests.test_verify_gpu import check

pytestmark = pytest.mark.gpu

LONGEST = 1 << 22
NEAR_ONE = 1.0 - 2.0 ** -24


def rows(T, V, seed, dtype=torch.float32, B=1):
    gen = torch.Generator().manual_seed(seed)
    x = torch.rand(B, T, V, generator=gen)
    x[..., 5::1009] *= 3000.0                      # a few likely tokens all over the row
    x /= x.sum(-1, keepdim=True)
    return x.to(dtype)


def tree(p, q, tokens, parent, coin, u):
    B, T, _ = p.shape
    d = dict(p=p, q=q, tokens=torch.as_tensor(tokens).expand(B, T).to(torch.int32).contiguous(),
             parent=torch.as_tensor(parent).expand(B, T).to(torch.int32).contiguous(),
             coins=torch.full((B, T), coin), u=torch.as_tensor(u).expand(B).float().contiguous())
    return d


@pytest.mark.parametrize("u", [0.0, 2.0 ** -24, 0.37, 0.99, NEAR_ONE])
@pytest.mark.parametrize("V", [LONGEST, LONGEST - 5, 2097152 + 1027])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_refused_tokens_in_late_groups(V, dtype, u):
    """Proposals at both ends of the row, of its CTAs' parts and of its batches, all refused."""
    likely = 5 + 1009 * ((V - 6) // 1009)
    tokens = [0, 0, V - 1, V // 2, likely, 5, V // 8 - 1, V // 8, 1023, 1024, likely - 1009]
    d = tree(rows(len(tokens), V, 3, dtype), None, tokens, [-1] + [0] * 10, 1.0, u)
    _, n, _ = check(d)
    assert int(n[0]) == 1


@pytest.mark.parametrize("u", [0.0, 0.61, NEAR_ONE])
@pytest.mark.parametrize("V", [LONGEST, 2097152 + 1027])
def test_residuals_of_long_rows(V, u):
    """Siblings refused one after the other against rows of q."""
    p, q = rows(4, V, 4), rows(4, V, 5)
    tokens = [0] + [int(x) for x in q[0, 0].topk(3).indices]
    d = tree(p, q, tokens, [-1, 0, 0, 0], 1.0, u)
    check(d)
    d["coins"][0, 3] = 0.0
    check(d)


@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("u", [0.0, 0.5, NEAR_ONE])
def test_every_weight_as_large_as_it_counts(u, with_q):
    """2^22 probabilities of 1: sums of 2^62, the largest there are."""
    p = torch.ones(1, 3, LONGEST)
    d = tree(p, torch.zeros_like(p) if with_q else None, [0, 7, LONGEST - 1], [-1, 0, 0], 1.0, u)
    path, n, token = check(d)
    if with_q:        # c q(x) = 0 is below any weight
        d["q"][0, 0, 7] = d["q"][0, 0, LONGEST - 1] = 1.0
        check(d)
    one = tree(p[:, :1].contiguous(), None, [0], [-1], 1.0, u)
    _, _, token = check(one)
    assert int(token[0]) == int(u * 2 ** 24) * LONGEST // 2 ** 24


@pytest.mark.parametrize("with_q", [True, False])
def test_one_cta_a_tree(with_q):
    B, V = 160, 300001
    p = rows(3, V, 6, B=B)
    q = p.roll(1, 0) if with_q else None
    gen = torch.Generator().manual_seed(7)
    d = tree(p, q, [0, V - 1, 5], [-1, 0, 0], 1.0, 0.0)
    d["u"] = torch.rand(B, generator=gen)
    d["tokens"][:, 1] = torch.randint(0, V, (B,), generator=gen).int()
    d["tokens"][:, 2] = 5 + 1009 * torch.randint(0, V // 1009, (B,), generator=gen).int()
    path, n, _ = check(d)
    assert np.array_equal(n.cpu().numpy(), (path >= 0).sum(1).cpu().numpy())
