"""Oracle of a speculative step's closing operators (CPU, numpy).

``verify_drafts`` follows the rule in include/gdr.h, one tree after another.
With ``real=np.float32`` every single operation is the float32 one that the
rule names, so that the library has to give the same whole numbers; with
``real=np.float64`` it is the mathematics of the rule (masses are real sums,
nothing is rounded), and ``margin`` says how near the closest of a tree's
decisions was to going the other way.

``commit_path`` gathers each sequence's path and runs the package's recurrence
over it.  ``quantise`` / ``dequantise`` are the 8-bit rows in float32.
"""
import numpy as np

UNIT = 2.0 ** 40


def _clean(x, real):
    x = np.where(np.isnan(x), 0.0, x)
    return np.clip(x, 0.0, 1.0).astype(real)


def _mass(w, real):
    """Sum of weights: whole units of 2^-40 as an int (float32), or the real sum."""
    if real == np.float64:
        return float(w.sum())
    return int((w * np.float32(UNIT)).astype(np.int64).sum())


def _as_real(mass, real):
    return real(mass) if real == np.float64 else np.float32(mass) / np.float32(UNIT)


def _draw(w, u, real):
    """(token, margin): the first running sum above the goal."""
    u = 0.0 if np.isnan(u) else min(max(float(u), 0.0), 1.0 - 2.0 ** -24)
    m = int(u * 2 ** 24)
    if real == np.float64:
        run = np.cumsum(w)
        if run[-1] <= 0:
            return -1, np.inf
        goal = run[-1] * m / 2 ** 24
        token = int(np.searchsorted(run, goal, side="right"))
        near = np.abs(run[max(0, token - 1):token + 2] - goal).min()
        return min(token, len(w) - 1), near / run[-1]
    run = np.cumsum((w * np.float32(UNIT)).astype(np.int64))
    total = int(run[-1])
    if total == 0:
        return -1, np.inf
    return int(np.searchsorted(run, (total * m) >> 24, side="right")), np.inf


def verify_drafts(p, q, tokens, parent, coins, u, max_path, real=np.float32):
    """p, q [B, T, V] (q may be None), tokens, parent, coins [B, T], u [B] as numpy arrays.
    Returns (path [B, max_path], n_path [B], next_token [B], margin [B])."""
    B, T, V = p.shape
    path = np.full((B, max_path), -1, np.int32)
    n_path, token = np.ones(B, np.int32), np.empty(B, np.int32)
    margin = np.full(B, np.inf)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        for b in range(B):
            here, n = 0, 1
            path[b, 0] = 0
            while True:
                P = _clean(p[b, here], real)
                Q = None if q is None else _clean(q[b, here], real)
                R = w = P
                left = 1.0 if real == np.float64 else int(UNIT)
                took = -1
                kids = [t for t in range(1, T) if parent[b, t] == here and parent[b, t] < t
                        and 0 <= tokens[b, t] < V] if n < max_path else []
                for t in kids:
                    x, c = tokens[b, t], real(coins[b, t])
                    a = R[x]
                    bar = c * (_as_real(left, real) if q is None else Q[x])
                    margin[b] = min(margin[b], abs(float(bar) - float(a)) if a > 0 else np.inf)
                    if a > 0 and bar < a:
                        took = t
                        break
                    if q is None:
                        left = max(left - _mass(R[x:x + 1], real), 0)
                        R = w = R.copy()
                        R[x] = 0
                    else:
                        r = np.maximum(R - Q, real(0))
                        mass = _mass(r, real)
                        if mass > 0:
                            w, R = r, r / _as_real(mass, real)
                if took < 0:
                    break
                here = took
                path[b, n] = took
                n += 1
            if _mass(w, real) == 0:
                w = P
            token[b], near = _draw(w, u[b], real)
            margin[b] = min(margin[b], near)
            n_path[b] = n
    return path, n_path, token, margin


def commit_path(k, v, g, beta, h0, path, n_path):
    """float64 arrays as in oracle.recurrence (g [B, T, HV, dk] or [B, T, HV]); returns ht."""
    from . import recurrence
    B, T, HK, dk = k.shape
    HV, dv = v.shape[2], v.shape[3]
    if g.ndim == 3:
        g = np.repeat(g[..., None], dk, axis=-1)
    ht = np.zeros((B, HV, dk, dv)) if h0 is None else h0.copy()
    for b in range(B):
        nodes = []
        for t in path[b, :max(0, min(int(n_path[b]), path.shape[1]))]:
            if not 0 <= t < T:
                break
            nodes.append(int(t))
        if nodes:
            pick = lambda x: np.ascontiguousarray(x[b:b + 1, nodes])  # noqa: E731
            ht[b:b + 1] = recurrence(pick(k), pick(k), pick(v), pick(g), pick(beta),
                                     np.ascontiguousarray(ht[b:b + 1]))[1]
    return ht


def quantise(state):
    """(codes int8, scale f32) of f32 rows."""
    state = state.astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        top = np.abs(state).max(-1)
        finite = np.isfinite(state).all(-1)
        held = finite & (top > np.float32(1e-30))
        inv = np.where(held, np.float32(127) * (np.float32(1) / top), np.float32(0))
        codes = np.where(held[..., None], np.rint(state * inv[..., None]), 0).astype(np.int8)
        scale = np.where(held, top * (np.float32(1) / np.float32(127)), np.float32(0))
    return codes, np.where(finite, scale, np.float32(np.nan)).astype(np.float32)


def dequantise(codes, scale):
    return codes.astype(np.float32) * scale[..., None]
