"""Speculative decoding with trees of drafted tokens, on recurrent states only.

A toy decoder of ``layers`` gated delta rule layers: every token has its keys, values, gates and
queries in a table, and the target's logits are a bigram table's plus a reading of the last
layer's output.  The draft model is the bigram table alone.  One step of it, on one stream and
without the host learning anything:

    tree of drafted tokens -> gdr_forward_tree (each layer) -> gdr_verify_drafts
        -> gdr_commit_path (each layer, states in place)

The prompt's states are kept in an 8-bit cache; a second batch starts from them.  At the end the
states are compared with those of gdr_forward over the tokens that were accepted.

    python examples/speculative_step.py [--steps 8] [--batch 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from channelwise_gated_delta_gb300 import (gdr_commit_path, gdr_forward,  # noqa: E402
                                           gdr_forward_tree, gdr_state_cache, gdr_state_load,
                                           gdr_state_store, gdr_verify_drafts)
from channelwise_gated_delta_gb300.inputs import draw_parents  # noqa: E402


class Toy:
    """The tables of a vocabulary of V tokens."""

    def __init__(self, V, layers, HK, HV, d, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)
        unit = lambda x: torch.nn.functional.normalize(x, dim=-1).bfloat16()
        self.V, self.layers, self.shape = V, layers, (HK, HV, d)
        self.bigram = 2.0 * rnd(V, V)
        self.read = rnd(HV * d, V)
        self.table = [dict(q=unit(rnd(V, HK, d)), k=unit(rnd(V, HK, d)), v=rnd(V, HV, d).bfloat16(),
                           g=-torch.nn.functional.softplus(rnd(V, HV, d) - 3.0),
                           beta=torch.sigmoid(rnd(V, HV))) for _ in range(layers)]

    def inputs(self, layer, tokens):
        """What layer ``layer`` sees of tokens [B, T]."""
        return {n: t[tokens.long()] for n, t in self.table[layer].items()}

    def draft(self, tokens):
        return torch.softmax(self.bigram[tokens.long()], -1)

    def target(self, tokens, out):
        logits = self.bigram[tokens.long()] + 0.3 * out.flatten(2).float() @ self.read
        return torch.softmax(logits, -1)


def draft_tree(toy, root, parent, gen):
    """Tokens of a tree below ``root`` [B], each drawn from the draft's distribution after its
    parent, and those distributions after every node."""
    B, T = root.shape[0], len(parent)
    tokens = torch.empty(B, T, dtype=torch.int32, device="cuda")
    tokens[:, 0] = root
    for t in range(1, T):
        tokens[:, t] = torch.multinomial(toy.draft(tokens[:, parent[t]]), 1, generator=gen)[:, 0]
    return tokens, toy.draft(tokens)


def run(batch=4, steps=8, T=12, branching=2, max_path=4, V=512, layers=2, HK=2, HV=4, d=128,
        seed=1):
    toy = Toy(V, layers, HK, HV, d)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.rand(*s, device="cuda", generator=gen)

    # the prompt, the same for all sequences: its states go into the 8-bit cache, one slot a layer
    prompt = torch.randint(0, V, (1, 40), device="cuda", generator=gen)
    slots = torch.arange(layers, dtype=torch.int32, device="cuda")
    cache, scale = gdr_state_cache(layers, HV, d, d)
    after = torch.cat([gdr_forward(**toy.inputs(i, prompt))[1] for i in range(layers)])
    gdr_state_store(after, slots, cache, scale)

    # every sequence starts from it
    states = [gdr_state_load(cache, scale, slots[i:i + 1].expand(batch).contiguous())
              for i in range(layers)]
    start = [s.clone() for s in states]
    parent = draw_parents(1, T, "beam", branching=branching)[0]
    parents_host = parent.expand(batch, T)
    parents = parent.cuda().expand(batch, T)           # one tree for the batch
    root = torch.randint(0, V, (batch,), device="cuda", generator=gen).int()
    accepted, counts = [], []
    for _ in range(steps):
        tokens, q = draft_tree(toy, root, parent.tolist(), gen)
        seen = [toy.inputs(i, tokens) for i in range(layers)]
        for i in range(layers):
            out = gdr_forward_tree(parent=parents_host, h0=states[i], **seen[i])
        path, n_path, root = gdr_verify_drafts(toy.target(tokens, out), tokens, parents,
                                               rand(batch, T), rand(batch), q=q,
                                               max_path=max_path)
        for i in range(layers):
            x = seen[i]
            gdr_commit_path(x["k"], x["v"], x["g"], x["beta"], path, n_path, h0=states[i],
                            ht=states[i])
        accepted.append(torch.where(path >= 0, tokens.gather(1, path.clamp(min=0).long()), -1))
        counts.append(n_path)
    accepted, counts = torch.cat(accepted, 1), torch.stack(counts, 1)

    # the same tokens in one piece
    worst = 0.0
    for b in range(batch):
        line = accepted[b][accepted[b] >= 0][None]
        for i in range(layers):
            _, want = gdr_forward(h0=start[i][b:b + 1].contiguous(), **toy.inputs(i, line))
            worst = max(worst, float((states[i][b] - want[0]).abs().max() / want.abs().max()))
    lost = max(float((start[i][0] - after[i]).abs().max() / after[i].abs().max())
               for i in range(layers))
    return dict(counts=counts.cpu(), error=worst, cache_error=lost)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--batch", type=int, default=4)
    a = ap.parse_args()
    r = run(batch=a.batch, steps=a.steps)
    print("tokens accepted per step (the root included), one line a sequence:")
    print("\n".join(" ".join(map(str, row)) for row in r["counts"].tolist()))
    print("states against one forward pass over the accepted tokens: %.1e of their largest value"
          % r["error"])
    print("prompt's states after the 8-bit cache: %.1e" % r["cache_error"])
