"""Cases of the operators that close a step of speculative decoding on a recurrent state.

Three operators, in two forms each: a plain one (elementary torch operations) and, where ``own`` is
true, the calls that a user makes of this package.

verify    Draft trees against the target's probabilities.  Node 0 of a tree is the token already
          decided, node t > 0 a drafted token whose parent is parent[t] < t; row t of p is the
          target's distribution after node t, row t of q the one its children were drawn from (no q:
          each child was proposed as it is).  From the root on, a node's children are tried in order
          of their index.  With q, child x with coin c is accepted if R(x) > 0 and c q(x) < R(x),
          where R = p at first; a refusal turns R into max(R - q, 0), brought back to a sum of one
          (or leaves it, if nothing would be left).  Without q it is accepted if p(x) > 0 and
          c M < p(x), M being the mass that the refused children have left; a refused token has no
          mass any more.  Where no child is accepted the next token is drawn from what is left of the
          row by the given u: the first token at which the running sum, in units of 2^-40, is above
          floor(u total).  Outputs: the accepted nodes (-1 behind them), how many, the next token
          (-1 for a row without mass).

commit    The state after the accepted nodes: for each node on the path S <- exp(g) S (per key
          channel), S <- S + beta k (v - S^T k)^T.

snapshot  States into the slots of an 8-bit cache (a row of S has one scale, its largest magnitude
          over 127), and back.  restore: only back; a sequence without a slot starts from zero.
"""
import math

import numpy as np
import torch

own = False

UNIT = 2.0 ** 40       # probabilities are summed as integers in units of 2^-40
BITS = 24              # a random number counts as a multiple of 2^-24


def listed():
    """The listed cases."""
    d128 = {"HK": 16, "HV": 32, "dk": 128, "dv": 128}
    return [
        # one user: four drafted tokens in a chain, latency is all
        {"name": "verify one chain", "op": "verify", "B": 1, "T": 5, "V": 32768, "tree": "chain",
         "width": 1, "D": 5, "dtype": "f32", "q": True},
        # a full batch, seven drafted tokens each, a large vocabulary
        {"name": "verify batch of chains", "op": "verify", "B": 64, "T": 8, "V": 131072,
         "tree": "chain", "width": 1, "D": 8, "dtype": "f32", "q": True},
        # trees of proposals without draft probabilities, bf16, a vocabulary of odd size
        {"name": "verify proposed trees", "op": "verify", "B": 8, "T": 64, "V": 100003,
         "tree": "beam", "width": 4, "D": 8, "dtype": "bf16", "q": False},
        # trees whose siblings were drawn from q, each tree of another shape
        {"name": "verify drawn trees", "op": "verify", "B": 16, "T": 32, "V": 50001,
         "tree": "random", "width": 3, "D": 6, "dtype": "f32", "q": True},
        # the same user's states after the accepted tokens
        dict({"name": "commit one sequence", "op": "commit", "B": 1, "T": 5, "D": 5,
              "dtype": "bf16", "gate": "channel"}, **d128),
        # a full batch, paths through trees of 64 tokens
        dict({"name": "commit batch", "op": "commit", "B": 64, "T": 64, "D": 8,
              "dtype": "bf16", "gate": "channel"}, **d128),
        # small heads, f32, one decay per head, odd counts
        {"name": "commit small heads", "op": "commit", "B": 5, "T": 17, "D": 9, "HK": 3, "HV": 9,
         "dk": 64, "dv": 32, "dtype": "f32", "gate": "scalar"},
        # long drafts: up to 48 accepted tokens in a row
        dict({"name": "commit long paths", "op": "commit", "B": 8, "T": 48, "D": 48,
              "dtype": "bf16", "gate": "channel"}, **d128),
        # one sequence's states put away and taken up again
        dict({"name": "snapshot one sequence", "op": "snapshot", "N": 1, "slots": 8}, **d128),
        # a batch is put away and taken up again
        dict({"name": "snapshot batch", "op": "snapshot", "N": 64, "slots": 80}, **d128),
        # small heads, an odd number of sequences, some of them new
        {"name": "restore small heads", "op": "restore", "N": 7, "slots": 9, "HK": 2, "HV": 6,
         "dk": 64, "dv": 32},
        # many sequences that begin with a known prefix
        dict({"name": "restore batch", "op": "restore", "N": 128, "slots": 100}, **d128),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 10)


def draw(rng):
    """One more case, no dearer than the largest listed one of its operator."""
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        op = rng.choice(["verify", "verify", "commit", "commit", "snapshot", "restore"])
        if op == "verify":
            tree = rng.choice(["chain", "beam", "random"])
            T = _log_uniform(rng, 1, 64)
            case = {"op": op, "B": _log_uniform(rng, 1, 64), "T": T,
                    "V": _log_uniform(rng, 500, 131072), "tree": tree,
                    "width": 1 if tree == "chain" else rng.randint(2, 5),
                    "D": rng.randint(1, min(T, 12)), "dtype": rng.choice(["f32", "bf16"]),
                    "q": rng.random() < 0.6}
            if case["B"] * T * case["V"] > 64 * 8 * 131072:
                continue
        else:
            G = rng.choice([1, 2, 3, 4])
            HK = _log_uniform(rng, 1, 16)
            case = {"op": op, "HK": HK, "HV": HK * G, "dk": rng.choice([32, 64, 128, 128]),
                    "dv": rng.choice([32, 64, 128, 128])}
            if op == "commit":
                D = _log_uniform(rng, 1, 48)
                case.update({"B": _log_uniform(rng, 1, 64), "D": D, "T": rng.randint(D, 64),
                             "dtype": rng.choice(["f32", "bf16"]),
                             "gate": rng.choice(["channel", "channel", "scalar"])})
            else:
                N = _log_uniform(rng, 1, 128)
                case.update({"N": N, "slots": rng.randint(N, 2 * N)})
        if _cost(case) <= most[op]:
            return case


def work(case):
    """Bytes and operations that one pass cannot do without."""
    if case["op"] == "verify":
        # the row of p of the last node, that of q where a child of it was refused (nearly always),
        # and each node's token, parent, coin and two probabilities
        rows = case["B"] * case["V"] * (2 if case["q"] else 1)
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * es + case["B"] * (case["T"] * 20 + case["D"] * 4 + 12),
                "flops": 3 * rows}
    heads = case.get("B", case.get("N")) * case["HV"]
    state = case["dk"] * case["dv"]
    if case["op"] == "commit":
        # the state in and out; paths are of 1 to D nodes, each as likely: k, v, g and beta of those
        n = (case["D"] + 1) / 2
        es = 2 if case["dtype"] == "bf16" else 4
        token = (case["HK"] * case["dk"] * es + case["HV"] * (case["dv"] * es + 4)
                 + case["HV"] * 4 * (1 if case["gate"] == "scalar" else case["dk"]))
        return {"bytes": heads * state * 8 + case["B"] * n * token,
                "flops": heads * n * 6 * state}
    # a state element is 4 bytes outside and 1 in the cache, a row's scale 4
    if case["op"] == "snapshot":
        return {"bytes": heads * (state * 10 + case["dk"] * 8), "flops": heads * state * 4}
    fresh = _fresh(case["N"])
    return {"bytes": heads * state * 4 + (case["N"] - fresh) * case["HV"] * (state + case["dk"] * 4),
            "flops": heads * state}


def _fresh(N):
    """How many of N sequences have no slot."""
    return N // 8 + (1 if N > 4 else 0)


def _parents(case, seed):
    """parent[b, t]: -1 for the root."""
    B, T, w = case["B"], case["T"], case["width"]
    t = np.arange(T)
    if case["tree"] == "chain":
        par = np.broadcast_to(t - 1, (B, T))
    elif case["tree"] == "beam":
        par = np.broadcast_to(np.where(t > 0, (t - 1) // w, -1), (B, T))
    else:  # a random earlier node that has fewer than w children
        r = np.random.RandomState(seed % (1 << 31))
        par = np.full((B, T), -1)
        for b in range(B):
            room = [w]
            for n in range(1, T):
                free = [i for i, x in enumerate(room) if x]
                par[b, n] = free[r.randint(len(free))]
                room[par[b, n]] -= 1
                room.append(w)
    return torch.from_numpy(np.array(par, dtype=np.int32)).cuda()


def _siblings(parent):
    """The place of each node among its parent's children."""
    same = parent[:, :, None] == parent[:, None, :]
    return torch.tril(same, diagonal=-1).sum(2)


def prepare(case, seed):
    """What a user's program holds before the call."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    s = {"case": case}
    dt = torch.bfloat16 if case.get("dtype") == "bf16" else torch.float32
    if case["op"] == "verify":
        B, T, V = case["B"], case["T"], case["V"]
        s["parent"] = _parents(case, seed)
        up = s["parent"].clamp(min=0).long()
        logits = 4.0 * normal(B, T, V)                      # a few likely tokens, a long tail
        s["p"] = torch.softmax(logits, dim=-1).to(dt)
        logits += 0.7 * normal(B, T, V)                     # the draft model: near the target
        s["q"] = torch.softmax(logits, dim=-1).to(dt) if case["q"] else None
        tokens = torch.empty(B, T, dtype=torch.int64, device="cuda")
        place = _siblings(s["parent"])
        for b in range(B):                                  # a batch element at a time: memory
            if case["q"]:                                   # drawn from q
                noise = -torch.log(-torch.log(uniform(T, V).clamp(1e-20, 1 - 1e-7)))
                tokens[b] = (logits[b, up[b]] + noise).argmax(-1)
            else:                                           # the draft's likeliest
                top = logits[b].topk(min(V, max(1, case["width"])), dim=-1).indices
                tokens[b] = top[up[b], place[b].clamp(max=top.shape[1] - 1)]
        s["tokens"] = tokens.to(torch.int32)
        s["coins"], s["u"] = uniform(B, T), uniform(B)
        return s
    HK, HV, dk, dv = case["HK"], case["HV"], case["dk"], case["dv"]
    if case["op"] == "commit":
        B, T, D = case["B"], case["T"], case["D"]
        s["k"] = torch.nn.functional.normalize(normal(B, T, HK, dk), dim=-1).to(dt)
        s["v"] = normal(B, T, HV, dv).to(dt)
        g = normal(B, T, HV) if case["gate"] == "scalar" else normal(B, T, HV, dk)
        s["g"] = -torch.nn.functional.softplus(g - 2.0)
        s["beta"] = torch.sigmoid(normal(B, T, HV))
        s["h0"] = 0.3 * normal(B, HV, dk, dv)
        n = 1 + (uniform(B) * D).long().clamp(max=D - 1)
        nodes = uniform(B, T)
        nodes[:, 0] = -1.0                                  # the root is on every path
        pick = nodes.argsort(1)[:, :D]
        at = torch.arange(D, device="cuda")[None, :]
        pick = torch.where(at < n[:, None], pick, T).sort(1).values
        s["path"] = torch.where(at < n[:, None], pick, -1).to(torch.int32)
        s["n_path"] = n.to(torch.int32)
        s["ht"] = torch.empty_like(s["h0"])
        return s
    N, slots = case["N"], case["slots"]
    # rows of very different size: a channel that forgets fast holds little
    state = normal(N, HV, dk, dv) * torch.exp(1.5 * normal(N, HV, dk, 1))
    s["cache"] = torch.zeros(slots, HV, dk, dv, dtype=torch.int8, device="cuda")
    s["scale"] = torch.zeros(slots, HV, dk, device="cuda")
    s["out"] = torch.empty_like(state)
    order = torch.rand(max(N, slots), device="cuda", generator=gen).argsort()
    if case["op"] == "snapshot":
        s["state"] = state
        s["slots"] = order[:N].to(torch.int32)
        return s
    s["cache"] = torch.randint(-127, 128, s["cache"].shape, device="cuda", generator=gen,
                               dtype=torch.int8)
    s["scale"] = torch.exp(1.5 * normal(slots, HV, dk)) / 127
    at = order[:N] % slots                                  # a prefix may serve several sequences
    fresh = _fresh(N)
    at[:fresh] = -1
    s["slots"] = at[torch.rand(N, device="cuda", generator=gen).argsort()].to(torch.int32)
    return s


def run(state):
    """One pass."""
    op = state["case"]["op"]
    if own:
        import channelwise_gated_delta_gb300 as gdr

        if op == "verify":
            return gdr.gdr_verify_drafts(state["p"], state["tokens"], state["parent"],
                                         state["coins"], state["u"], q=state["q"],
                                         max_path=state["case"]["D"])
        if op == "commit":
            return gdr.gdr_commit_path(state["k"], state["v"], state["g"], state["beta"],
                                       state["path"], state["n_path"], h0=state["h0"],
                                       ht=state["ht"])
        if op == "snapshot":
            gdr.gdr_state_store(state["state"], state["slots"], state["cache"], state["scale"])
        return gdr.gdr_state_load(state["cache"], state["scale"], state["slots"],
                                  out=state["out"])
    if op == "verify":
        return _verify(state)
    if op == "commit":
        return _commit(state, torch.float32)
    if op == "snapshot":
        _store(state)
    return _load(state, torch.float32)


# ------------------------------------------------------------------ plain forms
def _probs(x):
    return torch.nan_to_num(x.float(), nan=0.0, posinf=1.0, neginf=0.0).clamp(0.0, 1.0)


def _fixed(x):
    return (x * UNIT).to(torch.int64)


def _verify(s):
    p, q, case = s["p"], s["q"], s["case"]
    B, T, V = p.shape
    D, S = case["D"], case["width"]
    dev = p.device
    rows = torch.arange(B, device=dev)
    tokens, parent = s["tokens"].long(), s["parent"].long()
    # children[b, c, i]: the i-th child of node c, T where there is none
    children = torch.full((B, T + 1, T), T, dtype=torch.int64, device=dev)
    children[rows[:, None], parent % (T + 1), _siblings(parent)] = torch.arange(T, device=dev)
    tok = torch.cat([tokens, tokens.new_zeros(B, 1)], 1)
    coin = torch.cat([s["coins"], s["coins"].new_zeros(B, 1)], 1)

    here = torch.zeros(B, dtype=torch.int64, device=dev)          # the last accepted node
    path = torch.full((B, D), -1, dtype=torch.int64, device=dev)
    path[:, 0] = 0
    n = torch.ones(B, dtype=torch.int64, device=dev)
    walking = torch.ones(B, dtype=torch.bool, device=dev)
    w = _probs(p[rows, here])                                     # what the next token is drawn from
    for d in range(1, D):
        step = torch.full_like(here, -1)                          # the child that is accepted
        left = w
        mass = torch.full((B,), int(UNIT), dtype=torch.int64, device=dev)
        Q = _probs(q[rows, here]) if q is not None else None
        for i in range(S):
            t = children[rows, here, i]
            x = tok[rows, t]
            tried = walking & (step < 0) & (t < T)
            a = left[rows, x]
            b = Q[rows, x] if q is not None else mass.float() / UNIT
            yes = tried & (a > 0) & (coin[rows, t] * b < a)
            no = tried & ~yes
            step = torch.where(yes, t, step)
            if q is not None:
                r = (left - Q).clamp(min=0.0)
                total = _fixed(r).sum(1)
                no = no & (total > 0)
                w = torch.where(no[:, None], r, w)
                left = torch.where(no[:, None], r / (total.float() / UNIT)[:, None], left)
            else:
                mass = torch.where(no, (mass - _fixed(a)).clamp(min=0), mass)
                w = left = left.scatter(1, x[:, None], torch.where(no, 0.0, a)[:, None])
        walking = walking & (step >= 0)
        here = torch.where(walking, step, here)
        n = n + walking
        path[:, d] = torch.where(walking, step, -1)
        w = torch.where(walking[:, None], _probs(p[rows, here]), w)
    full = _probs(p[rows, here])
    w = torch.where((_fixed(w).sum(1) == 0)[:, None], full, w)
    run_sum = _fixed(w).cumsum(1)
    total = run_sum[:, -1]
    m = (torch.nan_to_num(s["u"], nan=0.0).clamp(0.0, 1.0 - 2.0 ** -BITS) * 2.0 ** BITS).long()
    low = (1 << BITS) - 1
    goal = (total >> BITS) * m + (((total & low) * m) >> BITS)    # floor(total m / 2^24)
    token = torch.where(total > 0, (run_sum <= goal[:, None]).sum(1), -1)
    return path.to(torch.int32), n.to(torch.int32), token.to(torch.int32)


def _commit(s, real):
    case = s["case"]
    B, T, HK, dk = s["k"].shape
    G = case["HV"] // HK
    S = s["h0"].to(real)
    rows = torch.arange(B, device=S.device)
    for d in range(case["D"]):
        t = s["path"][:, d].long().clamp(min=0)
        k = s["k"][rows, t].to(real).repeat_interleave(G, dim=1)              # [B, HV, dk]
        v = s["v"][rows, t].to(real)
        g = s["g"][rows, t].to(real).exp()
        beta = s["beta"][rows, t].to(real)
        decayed = S * (g[..., None] if g.dim() == 3 else g[..., None, None])
        seen = (decayed * k[..., None]).sum(2)                                # S^T k
        new = decayed + k[..., None] * (beta[..., None] * (v - seen))[:, :, None, :]
        S = torch.where((d < s["n_path"])[:, None, None, None], new, S)
    return S


def _store(s):
    x = s["state"]
    top = x.abs().amax(-1)
    held = top > 1e-30
    codes = torch.round(x * torch.where(held, 127.0 / top, 0.0)[..., None]).to(torch.int8)
    at = s["slots"].long()
    s["cache"][at] = codes
    s["scale"][at] = torch.where(held, top / 127.0, 0.0)


def _load(s, real):
    at = s["slots"].long()
    known = (at >= 0)[:, None, None, None]
    at = at.clamp(min=0)
    x = s["cache"][at].to(real) * s["scale"][at].to(real)[..., None]
    return torch.where(known, x, torch.zeros((), dtype=real, device=x.device))


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The outputs from the definitions in 64 bits; None for nodes and tokens, which are equal or wrong."""
    if case["op"] == "verify":
        return None
    s = prepare(case, seed)
    if case["op"] == "commit":
        # each sequence alone, its path node by node, as matrix products
        out = s["h0"].double()
        for b in range(case["B"]):
            for t in s["path"][b, :int(s["n_path"][b])].tolist():
                k = s["k"][b, t].double().repeat_interleave(case["HV"] // case["HK"], dim=0)
                a = torch.exp(s["g"][b, t].double()).reshape(case["HV"], -1, 1)
                S = a * out[b]
                u = s["v"][b, t].double() - torch.bmm(k[:, None, :], S)[:, 0]
                out[b] = S + torch.bmm(k[:, :, None],
                                       (s["beta"][b, t].double()[:, None] * u)[:, None, :])
        return out
    if case["op"] == "snapshot":
        x = s["state"].double()
        scale = x.abs().amax(-1, keepdim=True) / 127
        return torch.round(x / scale) * scale
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for n, at in enumerate(s["slots"].tolist()):
        if at >= 0:
            out[n] = s["cache"][at].double() * s["scale"][at].double()[..., None]
    return out
