"""gdr_verify_drafts on the GPU against the oracle's rule.  Every output is a whole number that the
rule fixes to the last bit, so the comparison is equality."""
import numpy as np
import pytest
import torch

from channelwise_gated_delta_gb300 import gdr_verify_drafts
from channelwise_gated_delta_gb300.inputs import draw_parents
from oracle import speculation

pytestmark = pytest.mark.gpu


def problem(B, T, V, tree="beam", with_q=True, dtype=torch.float32, seed=0, branching=3, heat=2.0):
    """Rows near each other, drafts from q (or likely tokens of p where there is no q)."""
    gen = torch.Generator()
    gen.manual_seed(seed)
    logits = heat * torch.randn(B, T, V, generator=gen)
    p = torch.softmax(logits, -1).to(dtype)
    ql = logits + 0.7 * torch.randn(B, T, V, generator=gen)
    q = torch.softmax(ql, -1).to(dtype)
    parent = draw_parents(B, T, tree, seed=seed, branching=branching)
    if tree == "star":  # every node a child of the root
        parent = parent.clamp(min=0)
    parent[:, 0] = -1
    up = parent.clamp(min=0).long()
    rows = torch.arange(B)[:, None]
    if with_q:
        tokens = torch.multinomial(q.float()[rows, up].reshape(B * T, V), 1,
                                   generator=gen).reshape(B, T)
    else:
        top = ql.topk(min(V, 5), -1).indices[rows, up]
        tokens = top.gather(2, torch.randint(0, top.shape[2], (B, T, 1), generator=gen))[..., 0]
    d = dict(p=p, q=q if with_q else None, tokens=tokens.to(torch.int32), parent=parent,
             coins=torch.rand(B, T, generator=gen), u=torch.rand(B, generator=gen))
    return d


def expect(d, max_path):
    n = lambda x: None if x is None else x.float().numpy() if x.is_floating_point() else x.numpy()
    return speculation.verify_drafts(*(n(d[k]) for k in ("p", "q", "tokens", "parent", "coins",
                                                         "u")), max_path)[:3]


def on_gpu(d, max_path, **kw):
    c = {k: None if x is None else x.cuda() for k, x in d.items()}
    return gdr_verify_drafts(c["p"], c["tokens"], c["parent"], c["coins"], c["u"], q=c["q"],
                             max_path=max_path, **kw)


def check(d, max_path=None):
    max_path = d["p"].shape[1] if max_path is None else max_path
    got = on_gpu(d, max_path)
    for name, x, y in zip(("path", "n_path", "next_token"), got, expect(d, max_path)):
        assert x.dtype == torch.int32
        assert np.array_equal(x.cpu().numpy(), y), (name, x.cpu().numpy(), y)
    return got


@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 128, 129, 1000, 4099, 70001])
def test_vocabularies(V, dtype, with_q):
    check(problem(3, 6, V, "beam", with_q, dtype, seed=V))


@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("tree", ["chain", "beam", "star", "random"])
@pytest.mark.parametrize("T", [1, 2, 5, 32, 33, 65])
def test_trees(T, tree, with_q):
    for seed in range(3):
        check(problem(4, T, 601, tree, with_q, seed=10 * T + seed))


@pytest.mark.parametrize("tree", ["chain", "beam", "star"])
def test_longest_trees(tree):
    """512 nodes; near-equal rows so that paths get long, and flat ones with many refusals."""
    for heat in (0.0, 6.0):
        d = problem(2, 512, 97, tree, True, seed=5, heat=heat)
        check(d)
        d["q"] = None
        check(d)


@pytest.mark.parametrize("max_path", [1, 2, 3, 9])
def test_paths_end_at_max_path(max_path):
    d = problem(5, 9, 200, "chain", True, seed=3)
    d["q"] = d["p"].clone()
    d["coins"].zero_()   # everything is accepted
    path, n, _ = check(d, max_path)
    assert (n == max_path).all()


@pytest.mark.parametrize("B", [1, 2, 5, 19, 40, 150, 333])
def test_batches(B):
    """Every split of a row over CTAs, which goes by the batch and the vocabulary."""
    check(problem(B, 3, 20011 if B < 100 else 3001, "random", True, seed=B))
    check(problem(B, 3, 20011 if B < 100 else 3001, "star", False, torch.bfloat16, seed=B))


def test_refusal_of_everything():
    d = problem(4, 40, 300, "star", True, seed=7)
    d["coins"].fill_(1.0 - 2.0 ** -24)
    gen = torch.Generator().manual_seed(1)
    d["q"] = torch.softmax(3.0 * torch.randn(4, 40, 300, generator=gen), -1)
    d["tokens"][:] = d["q"][:, 0].argmax(-1)[:, None].to(torch.int32)
    check(d)
    d["q"] = None   # the same token proposed again and again: refused once, then without mass
    check(d)


def test_rows_without_mass_and_strange_values():
    d = problem(8, 4, 129, "chain", True, seed=8)
    p, q = d["p"], d["q"]
    p[0] = 0.0                                   # no mass at all
    p[1, :, ::2] = float("nan")
    p[2, :, 1::3] = -0.25                        # counts as nothing
    p[3, :, 5] = float("inf")                    # counts as one
    p[4] = 0.0
    p[4, :, 128] = 1.0                           # one token, the last
    q[5] = p[5]                                  # nothing is left after a refusal
    q[6, :, :] = float("nan")
    q[7] = 0.0
    for coin in (0.0, 0.5, 1.0, float("nan"), -1.0, 2.0):
        d["coins"].fill_(coin)
        check(d)
    d["q"] = None
    for coin in (0.0, 0.5, 1.0, float("nan")):
        d["coins"].fill_(coin)
        check(d)


@pytest.mark.parametrize("u", [0.0, 2.0 ** -24, 0.5, 1.0 - 2.0 ** -24, 1.0, 7.0, -1.0,
                               float("nan")])
def test_random_numbers_at_their_ends(u):
    d = problem(3, 3, 1030, "chain", True, seed=9)
    d["u"].fill_(u)
    check(d)
    d["p"][:, :, :3] = 0.0        # the lowest token with mass is 3, the highest 1019
    d["p"][:, :, 1020:] = 0.0
    check(d)


def test_nodes_that_cannot_stand():
    d = problem(4, 10, 64, "beam", True, seed=11)
    d["coins"].zero_()
    d["tokens"][0, 1], d["tokens"][0, 2] = -1, 64          # not in the vocabulary
    d["tokens"][0, 3] = -2 ** 31
    d["parent"][1, 1:] = torch.arange(1, 10)               # their own parents
    d["parent"][2, 1:4] = torch.tensor([-1, -7, 9])        # no parent, or a later one
    d["parent"][3, 4:] = 2 ** 31 - 1
    d["tokens"][:, 0], d["parent"][:, 0] = 12345, 77       # the root's are not read
    check(d)
    d["q"] = None
    check(d)


def test_node_zero_is_not_read():
    d = problem(2, 4, 50, "chain", True, seed=12)
    a = check(d)
    d["coins"][:, 0] = float("nan")
    d["tokens"][:, 0] = -5
    assert all(torch.equal(x, y) for x, y in zip(a, check(d)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad_p,pad_q", [(0, 5), (3, 0), (7, 7), (8, 16), (1, 2)])
def test_padded_rows(pad_p, pad_q, dtype):
    """p and q as slices of wider tensors whose padding is not to be read as mass."""
    V = 1001
    d = problem(3, 7, V, "random", True, dtype, seed=13)
    want = expect(d, 7)
    c = {k: x.cuda() for k, x in d.items()}
    wide = {}
    for name, pad in (("p", pad_p), ("q", pad_q)):
        wide[name] = torch.full((3, 7, V + pad), 1.0, dtype=dtype, device="cuda")
        wide[name][:, :, :V] = c[name]
    got = gdr_verify_drafts(wide["p"][:, :, :V], c["tokens"], c["parent"], c["coins"], c["u"],
                            q=wide["q"][:, :, :V])
    for x, y in zip(got, want):
        assert np.array_equal(x.cpu().numpy(), y)


def test_strides_of_the_parents():
    """One tree for the whole batch, and node-major parents."""
    d = problem(5, 9, 300, "beam", True, seed=17)
    want = expect(d, 9)
    c = {k: x.cuda() for k, x in d.items()}
    for parent in (c["parent"][0].expand(5, 9), c["parent"].t().contiguous().t(),
                   torch.stack([c["parent"], c["parent"]], -1)[..., 0]):
        got = gdr_verify_drafts(c["p"], c["tokens"], parent, c["coins"], c["u"], q=c["q"])
        for x, y in zip(got, want):
            assert np.array_equal(x.cpu().numpy(), y)


def test_rows_past_32_bit_offsets():
    """The last row starts past 2^32 bytes and past 2^31 elements."""
    V, ld = 1000, 2 ** 30 + 8
    flat = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    p = flat.as_strided((1, 3, V), (3 * ld, ld, 1))
    d = problem(1, 3, V, "chain", False, torch.bfloat16, seed=14)
    d["coins"].fill_(-1.0)
    for t in range(3):
        p[0, t] = d["p"][0, t].cuda()
    c = {k: x.cuda() for k, x in d.items() if x is not None}
    got = gdr_verify_drafts(p, c["tokens"], c["parent"], c["coins"], c["u"])
    assert int(got[1][0]) == 3
    for x, y in zip(got, expect(d, 3)):
        assert np.array_equal(x.cpu().numpy(), y)


def test_given_outputs_and_another_stream():
    d = problem(6, 5, 5000, "beam", True, seed=15)
    want = expect(d, 4)
    c = {k: x.cuda() for k, x in d.items()}
    outs = [torch.full((6, 4), 99, dtype=torch.int32, device="cuda"),
            torch.full((6,), 99, dtype=torch.int32, device="cuda"),
            torch.full((6,), 99, dtype=torch.int32, device="cuda")]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kw = dict(q=c["q"], path=outs[0], n_path=outs[1], next_token=outs[2])
    got = gdr_verify_drafts(c["p"], c["tokens"], c["parent"], c["coins"], c["u"], stream=s, **kw)
    s.synchronize()
    for x, o, y in zip(got, outs, want):
        assert x is o and np.array_equal(x.cpu().numpy(), y)


def test_the_first_token_follows_the_target():
    """40000 trees at once: the token after the root has the frequencies of p, to 5 sigma."""
    N, V = 40000, 6
    gen = torch.Generator(device="cuda")
    gen.manual_seed(16)
    rnd = lambda *s: torch.rand(*s, device="cuda", generator=gen)
    P = torch.softmax(1.5 * torch.randn(V, device="cuda", generator=gen), 0)
    Q = torch.softmax(1.5 * torch.randn(V, device="cuda", generator=gen), 0)
    p = P.expand(N, 3, V).contiguous()
    q = Q.expand(N, 3, V).contiguous()
    tok = torch.multinomial(Q, 3 * N, replacement=True, generator=gen).reshape(N, 3).int()
    parent = torch.tensor([-1, 0, 0], dtype=torch.int32, device="cuda").expand(N, 3).contiguous()
    path, n, nxt = gdr_verify_drafts(p, tok, parent, rnd(N, 3), rnd(N), q=q)
    took = tok.gather(1, path[:, 1:2].clamp(min=0).long())[:, 0]
    first = torch.where(n > 1, took, nxt).cpu().numpy()
    P = P.cpu().double().numpy()
    assert (np.abs(np.bincount(first, minlength=V) / N - P)
            <= 5 * np.sqrt(P * (1 - P) / N)).all()


def test_empty_batch():
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")
    path, n, nxt = gdr_verify_drafts(e(0, 3, 10), e(0, 3, dt=torch.int32), e(0, 3, dt=torch.int32),
                                     e(0, 3), e(0), q=e(0, 3, 10))
    assert path.shape == (0, 3) and n.numel() == 0 and nxt.numel() == 0
