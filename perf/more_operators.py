"""Cases of the operators around a recurrent layer: short convolution, norms of q and k, state space scan.

Three operators, in two forms each: a plain one (elementary torch operations) and, where ``own`` is
true, the calls that a user makes of this package.

conv   A causal convolution of each channel with W taps, over sequences of rows:
       out[t] = act(bias + sum_j w[:, j] x[t - W + 1 + j]), the rows before a sequence's first taken
       from its state [W - 1, D] (zeros without one), act = silu or none.  The new state holds the
       sequence's last W - 1 rows, older ones from the old state.

norm   Each head of q and k by itself: x / sqrt(sum x^2 + eps) ("l2") or x / sqrt(mean x^2 + eps)
       ("rms"), times a weight per channel if there is one, q times q_scale; then the first d_rot
       channels are rotated by the token's position: pair i by the angle position base^(-2 i / d_rot),
       the pair's channels being (i, i + d_rot / 2), or (2 i, 2 i + 1) interleaved.

ssm    The selective state space recurrence: per value head a state S [dk, dv], per token
       step = softplus(dt + dt_bias), S <- exp(step a) S + step b x^T, out = S^T c + d x, times silu(z)
       if there is z.  HK heads of b and c serve HV heads of x in contiguous groups.
"""
import math

import torch

own = False

RAGGED = "1 33 49 64 97 128 256 512"


def listed():
    """The listed cases."""
    d128 = {"HK": 16, "HV": 32, "dk": 128, "dv": 128}
    return [
        # one user's next token: q, k and v of 16 + 16 key heads and 32 value heads of 128
        {"name": "conv one token", "op": "conv", "N": 1, "T": 1, "lens": "", "D": 8192, "W": 4,
         "dtype": "bf16", "bias": False, "silu": True, "state": True, "wide": 0},
        # a full batch's next tokens
        {"name": "conv batch of tokens", "op": "conv", "N": 64, "T": 1, "lens": "", "D": 8192, "W": 4,
         "dtype": "bf16", "bias": False, "silu": True, "state": True, "wide": 0},
        # long prompts, read out of a wider projection
        {"name": "conv prompts", "op": "conv", "N": 4, "T": 16384, "lens": "", "D": 8192, "W": 4,
         "dtype": "bf16", "bias": False, "silu": True, "state": False, "wide": 4096},
        # packed continuations of different lengths, f32, an odd number of channels
        {"name": "conv ragged odd channels", "op": "conv", "N": 8, "T": 0, "lens": RAGGED, "D": 1157,
         "W": 3, "dtype": "f32", "bias": True, "silu": True, "state": True, "wide": 0},
        # one token of an attention layer far into a long text
        {"name": "norm one token", "op": "norm", "rows": 1, "HQ": 32, "HK": 16, "d": 128, "d_rot": 128,
         "kind": "rms", "weights": True, "interleaved": False, "far": 1000000, "dtype": "bf16"},
        # long prompts in front of the delta rule, q and k parts of one projection
        {"name": "norm prompts", "op": "norm", "rows": 65536, "HQ": 16, "HK": 16, "d": 128, "d_rot": 128,
         "kind": "l2", "weights": False, "interleaved": False, "far": 16384, "dtype": "bf16"},
        # f32, odd numbers of small heads and rows, half of the channels rotated pair by pair
        {"name": "norm small heads", "op": "norm", "rows": 1141, "HQ": 9, "HK": 3, "d": 64, "d_rot": 32,
         "kind": "rms", "weights": True, "interleaved": True, "far": 100000, "dtype": "f32"},
        # one user's next token
        dict({"name": "ssm one token", "op": "ssm", "N": 1, "T": 1, "lens": "", "dtype": "bf16",
              "z": True, "state": True}, **d128),
        # a full batch's next tokens
        dict({"name": "ssm batch of tokens", "op": "ssm", "N": 64, "T": 1, "lens": "", "dtype": "bf16",
              "z": True, "state": True}, **d128),
        # long prompts
        dict({"name": "ssm prompts", "op": "ssm", "N": 4, "T": 16384, "lens": "", "dtype": "bf16",
              "z": False, "state": False}, **d128),
        # one prompt: few heads, a long walk
        dict({"name": "ssm one prompt", "op": "ssm", "N": 1, "T": 4096, "lens": "", "dtype": "bf16",
              "z": True, "state": False}, **d128),
        # packed continuations of different lengths, f32, odd numbers of small heads
        {"name": "ssm ragged small heads", "op": "ssm", "N": 8, "T": 0, "lens": RAGGED, "HK": 3, "HV": 9,
         "dk": 64, "dv": 32, "dtype": "f32", "z": True, "state": True},
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
        op = rng.choice(["conv", "norm", "ssm", "ssm"])
        case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
        if op == "norm":
            d = rng.choice([32, 64, 128, 128, 256])
            case.update({"rows": _log_uniform(rng, 1, 65536), "HQ": _log_uniform(rng, 1, 64),
                         "HK": _log_uniform(rng, 1, 32), "d": d,
                         "d_rot": rng.choice([0, 16 * rng.randint(1, d // 16), d]),
                         "kind": rng.choice(["l2", "rms"]), "weights": rng.random() < 0.5,
                         "interleaved": rng.random() < 0.4,
                         "far": _log_uniform(rng, 100, 1 << 24)})
        else:
            shape = rng.choice(["tokens", "prompts", "packed"])
            case.update({"N": _log_uniform(rng, 1, 128 if shape == "tokens" else 16), "lens": "",
                         "T": 1 if shape == "tokens" else _log_uniform(rng, 2, 16384),
                         "state": rng.random() < 0.6})
            if shape == "packed":
                longest = case["T"]
                case["lens"] = " ".join(str(_log_uniform(rng, 1, longest)) for _ in range(case["N"]))
                case["T"] = 0
            if op == "conv":
                case.update({"D": _log_uniform(rng, 32, 12288), "W": rng.choice([2, 3, 4, 4]),
                             "bias": rng.random() < 0.5, "silu": rng.random() < 0.8,
                             "wide": rng.choice([0, 0, 64, _log_uniform(rng, 1, 4096)])})
                if rng.random() < 0.5:
                    case["D"] = max(32, case["D"] // 64 * 64)
            else:
                HK = _log_uniform(rng, 1, 16)
                case.update({"HK": HK, "HV": HK * rng.choice([1, 2, 3, 4, 8]),
                             "dk": rng.choice([32, 64, 128, 128]), "dv": rng.choice([32, 64, 128, 128]),
                             "z": rng.random() < 0.5})
        if _cost(case) <= most[op]:
            return case


def _lengths(case):
    return [int(n) for n in case["lens"].split()] if case["lens"] else [case["T"]] * case["N"]


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def work(case):
    """Bytes and operations that one pass cannot do without."""
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        values = case["rows"] * (case["HQ"] + case["HK"]) * case["d"]
        return {"bytes": 2 * values * es + case["rows"] * 4, "flops": 6 * values}
    rows = sum(_lengths(case))
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        states = (2 if case["state"] else 1) * case["N"] * (W - 1) * D
        return {"bytes": (2 * rows * D + states) * es + D * W * 4, "flops": rows * D * (2 * W + 4)}
    HK, HV, dk, dv = case["HK"], case["HV"], case["dk"], case["dv"]
    token = (2 * HK * dk + (3 if case["z"] else 2) * HV * dv) * es + HV * 4
    states = (2 if case["state"] else 1) * case["N"] * HV * dk * dv * 4
    # the recurrence: decay, update and output, each element of the state once a token
    return {"bytes": rows * token + states, "flops": rows * HV * 5 * dk * dv}


def prepare(case, seed):
    """What a user's program holds before the call."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    s = {"case": case}
    if case["op"] == "norm":
        rows, HQ, HK, d = case["rows"], case["HQ"], case["HK"], case["d"]
        # q and k beside each other in one projection; heads of different size
        both = (normal(rows, HQ + HK, d) * torch.exp(0.5 * normal(1, HQ + HK, 1))).to(dt)
        s["q"], s["k"] = both[:, :HQ], both[:, HQ:]
        s["wq"] = 1 + 0.2 * normal(d) if case["weights"] else None
        s["wk"] = 1 + 0.2 * normal(d) if case["weights"] else None
        s["q_scale"] = d ** -0.5
        s["eps"], s["base"] = 1e-6, 10000.0
        first = torch.randint(0, max(1, case["far"] - rows), (1,), device="cuda", generator=gen)
        s["positions"] = (first + torch.arange(rows, device="cuda")).to(torch.int32)
        if own and case["d_rot"]:
            import channelwise_gated_delta_gb300 as gdr

            s["freqs"] = gdr.gdr_rope_freqs(case["d_rot"], base=s["base"], device="cuda")
        return s
    lens = _lengths(case)
    rows, N = sum(lens), case["N"]
    s["cu"] = _offsets(lens) if case["lens"] else None
    lead = (rows,) if case["lens"] else (N, case["T"])
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        s["x"] = normal(*lead, D + case["wide"]).to(dt)[..., :D]
        s["w"] = normal(D, W) * W ** -0.5
        s["bias"] = 0.1 * normal(D) if case["bias"] else None
        s["s0"] = normal(N, W - 1, D).to(dt) if case["state"] else None
        return s
    HK, HV, dk, dv = case["HK"], case["HV"], case["dk"], case["dv"]
    # x, b and c as the convolution in front leaves them: parts of one tensor
    mixed = torch.nn.functional.silu(normal(*lead, HV * dv + 2 * HK * dk)).to(dt)
    s["x"] = mixed[..., :HV * dv].unflatten(-1, (HV, dv))
    s["b"] = mixed[..., HV * dv:HV * dv + HK * dk].unflatten(-1, (HK, dk))
    s["c"] = mixed[..., HV * dv + HK * dk:].unflatten(-1, (HK, dk))
    s["z"] = normal(*lead, HV, dv).to(dt) if case["z"] else None
    s["dt"] = 0.5 * normal(*lead, HV)
    start = torch.exp(uniform(HV) * math.log(100.0)) * 1e-3      # steps from 0.001 to 0.1
    s["dt_bias"] = start + torch.log(-torch.expm1(-start))       # softplus backwards
    s["a"] = -(1 + 15 * uniform(HV))
    s["d"] = 1 + 0.1 * normal(HV)
    s["h0"] = 0.3 * normal(N, HV, dk, dv) if case["state"] else None
    return s


def run(state):
    """One pass."""
    s, case = state, state["case"]
    if own:
        import channelwise_gated_delta_gb300 as gdr

        if case["op"] == "conv":
            return gdr.gdr_short_conv(s["x"], s["w"], bias=s["bias"], cu_seqlens=s["cu"], s0=s["s0"],
                                      silu=case["silu"])
        if case["op"] == "norm":
            turn = {"positions": s["positions"], "freqs": s["freqs"],
                    "interleaved": case["interleaved"]} if case["d_rot"] else {}
            return gdr.gdr_qk_norm(s["q"], s["k"], weight_q=s["wq"], weight_k=s["wk"],
                                   norm=case["kind"], eps=s["eps"], q_scale=s["q_scale"], **turn)
        return gdr.gdr_ssm_forward(s["x"], s["b"], s["c"], s["dt"], s["a"], d=s["d"], z=s["z"],
                                   dt_bias=s["dt_bias"], cu_seqlens=s["cu"], h0=s["h0"])
    if case["op"] == "conv":
        return _conv(s)
    if case["op"] == "norm":
        return (_norm(s["q"], s["wq"], s["q_scale"], s), _norm(s["k"], s["wk"], 1.0, s))
    return _ssm(s)


# ------------------------------------------------------------------ plain forms
def _conv(s):
    case, x = s["case"], s["x"]
    N, D, W = case["N"], case["D"], case["W"]
    old = s["s0"].float() if case["state"] else torch.zeros(N, W - 1, D, device=x.device)

    def part(rows, before):             # rows [n, T, D] behind their states [n, W - 1, D]
        T = rows.shape[1]
        y = torch.zeros_like(rows) if s["bias"] is None else s["bias"].expand_as(rows)
        full = torch.cat([before, rows], 1)
        for j in range(W):
            y = y + full[:, j:j + T] * s["w"][:, j]
        if case["silu"]:
            y = y / (1 + torch.exp(-y))
        return y.to(x.dtype), full[:, T:].to(x.dtype)

    if s["cu"] is None:
        return part(x.float(), old)
    parts = [part(x[None, a:b].float(), old[n:n + 1])
             for n, (a, b) in enumerate(zip(s["cu"], s["cu"][1:]))]
    return torch.cat([y[0] for y, _ in parts]), torch.cat([st for _, st in parts])


def _angles(s):
    """cos and sin of every pair's angle: formed in 64 bits, far positions have large angles."""
    d_rot = s["case"]["d_rot"]
    i = torch.arange(d_rot // 2, device="cuda", dtype=torch.float64)
    angle = s["positions"].double()[:, None] * s["base"] ** (-2 * i / d_rot)
    return angle.cos()[:, None], angle.sin()[:, None]


def _norm(x, weight, scale, s):
    case = s["case"]
    d, d_rot = case["d"], case["d_rot"]
    f = x.float()
    size = (f * f).sum(-1, keepdim=True)
    if case["kind"] == "rms":
        size = size / d
    y = f / torch.sqrt(size + s["eps"]) * scale
    if weight is not None:
        y = y * weight
    if d_rot:
        cos, sin = (t.float() for t in _angles(s))
        if case["interleaved"]:
            a, b = y[..., 0:d_rot:2], y[..., 1:d_rot:2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = y[..., :d_rot // 2], y[..., d_rot // 2:d_rot]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        y = torch.cat([turned, y[..., d_rot:]], -1)
    return y.to(x.dtype)


CHUNK = 64


def _ssm_chunks(x, b, c, la, step, S):
    """Sequences [n, T] by chunks: products within a chunk, the state from chunk to chunk."""
    n, T, HV, dv = x.shape
    HK, dk = b.shape[2:]
    C, G = min(T, CHUNK), HV // HK
    pad = -T % C
    if pad:                              # tokens that change nothing
        x, b, c, la, step = (torch.nn.functional.pad(t, (0, 0) * (t.dim() - 2) + (0, pad))
                             for t in (x, b, c, la, step))
    nc = (T + pad) // C
    x = x.view(n, nc, C, HV, dv).transpose(2, 3)                        # [n, nc, HV, C, dv]
    b = b.view(n, nc, C, HK, dk).transpose(2, 3)
    c = c.view(n, nc, C, HK, dk).transpose(2, 3)
    step = step.view(n, nc, C, HV).transpose(2, 3)                      # [n, nc, HV, C]
    log = la.view(n, nc, C, HV).transpose(2, 3).double().cumsum(-1)
    ones = torch.ones(C, C, dtype=torch.bool, device=x.device).tril()
    scores = (c @ b.transpose(-1, -2)).repeat_interleave(G, 2)          # [n, nc, HV, C, C]
    away = torch.where(ones, (log[..., :, None] - log[..., None, :]).float(), -math.inf)
    y = (scores * torch.exp(away) * step[..., None, :]) @ x
    del scores, away
    b, c = b.repeat_interleave(G, 2), c.repeat_interleave(G, 2)
    total = log[..., -1:]
    kept = torch.exp((total - log).float()) * step
    adds = b.transpose(-1, -2) @ (kept[..., None] * x)                  # [n, nc, HV, dk, dv]
    decay = torch.exp(total.float())[..., None]
    starts = torch.empty_like(adds)
    for i in range(nc):
        starts[:, i] = S
        S = decay[:, i] * S + adds[:, i]
    y = y + torch.exp(log.float())[..., None] * (c @ starts)
    return y.transpose(2, 3).reshape(n, nc * C, HV, dv)[:, :T], S


def _ssm(s):
    case = s["case"]
    N, HV, dk, dv = case["N"], case["HV"], case["dk"], case["dv"]
    raw = s["dt"] + s["dt_bias"]
    step = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    la = step * s["a"]
    x, b, c = s["x"].float(), s["b"].float(), s["c"].float()
    S = s["h0"] if case["state"] else torch.zeros(N, HV, dk, dv, device=x.device)
    if s["cu"] is None:
        y, S = _ssm_chunks(x, b, c, la, step, S)
    else:
        parts = [_ssm_chunks(*(t[None, p:q] for t in (x, b, c, la, step)), S[i:i + 1])
                 for i, (p, q) in enumerate(zip(s["cu"], s["cu"][1:]))]
        y = torch.cat([y[0] for y, _ in parts])
        S = torch.cat([e for _, e in parts])
    y = y + s["d"][:, None] * x
    if case["z"]:
        z = s["z"].float()
        y = y * z / (1 + torch.exp(-z))
    return y.to(s["x"].dtype), S


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The outputs from the definitions in 64 bits, without the plain forms' steps."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        return tuple(_exact_norm(s[n].double(), s["w" + n], f, s)
                     for n, f in (("q", s["q_scale"]), ("k", 1.0)))
    lens = _lengths(case)
    at = _offsets(lens)
    flat = {n: s[n].reshape(at[-1], *s[n].shape[1 if case["lens"] else 2:])
            for n in ("x", "b", "c", "dt", "z") if s.get(n) is not None}
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        w = s["w"].double()[:, None]
        outs, states = [], []
        for n, T in enumerate(lens):
            before = s["s0"][n].double() if case["state"] else torch.zeros(
                W - 1, D, dtype=torch.float64, device="cuda")
            full = torch.cat([before, flat["x"][at[n]:at[n + 1]].double()])
            y = full.unfold(0, W, 1)                                     # [T, D, W]: each row's window
            y = torch.cat([(y[a:a + 2048] * w[:, 0]).sum(-1) for a in range(0, T, 2048)])
            if s["bias"] is not None:
                y = y + s["bias"].double()
            outs.append(y * torch.sigmoid(y) if case["silu"] else y)
            states.append(full[T:])
        return torch.cat(outs).reshape(s["x"].shape), torch.stack(states)
    # token by token, all sequences of a length's step at once
    HK, HV, dk, dv = case["HK"], case["HV"], case["dk"], case["dv"]
    S = s["h0"].double() if case["state"] else torch.zeros(case["N"], HV, dk, dv, dtype=torch.float64,
                                                           device="cuda")
    S = S.clone()
    step = torch.nn.functional.softplus(flat["dt"].double() + s["dt_bias"].double(), threshold=1e9)
    decay = torch.exp(step * s["a"].double())
    y = torch.empty(at[-1], HV, dv, dtype=torch.float64, device="cuda")
    order = sorted(range(len(lens)), key=lambda n: -lens[n])
    S = S[order]
    first = torch.tensor([at[n] for n in order], device="cuda")
    for t in range(max(lens)):
        n = sum(1 for i in order if lens[i] > t)                         # the sequences that go on
        rows = first[:n] + t
        xt = flat["x"][rows].double()
        bt = flat["b"][rows].double().repeat_interleave(HV // HK, 1)
        ct = flat["c"][rows].double().repeat_interleave(HV // HK, 1)
        now = S[:n]
        now *= decay[rows][..., None, None]
        now += bt[..., None] * (step[rows][..., None] * xt)[..., None, :]
        y[rows] = torch.einsum("nhij,nhi->nhj", now, ct)
    y += s["d"].double()[:, None] * flat["x"].double()
    if case["z"]:
        y *= flat["z"].double() * torch.sigmoid(flat["z"].double())
    back = torch.empty_like(S)
    back[order] = S
    return y.reshape(s["x"].shape), back


def _exact_norm(x, weight, scale, s):
    case = s["case"]
    d, d_rot = case["d"], case["d_rot"]
    size = x.square().mean(-1, keepdim=True) if case["kind"] == "rms" else x.square().sum(-1, keepdim=True)
    y = x * (size + s["eps"]).rsqrt() * scale
    if weight is not None:
        y = y * weight.double()
    if d_rot:
        # a pair of channels as one complex number, turned by e^(i angle)
        part = y[..., :d_rot].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
        if not case["interleaved"]:
            part = part.transpose(-1, -2)
        i = torch.arange(d_rot // 2, device="cuda", dtype=torch.float64)
        angle = s["positions"].double()[:, None] * torch.exp(-2 * i / d_rot * math.log(s["base"]))
        turned = torch.view_as_real(torch.view_as_complex(part.contiguous())
                                    * torch.polar(torch.ones_like(angle), angle)[:, None])
        if not case["interleaved"]:
            turned = turned.transpose(-1, -2)
        y = torch.cat([turned.flatten(-2), y[..., d_rot:]], -1)
    return y
