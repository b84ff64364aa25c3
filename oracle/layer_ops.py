"""What stands around the recurrence in a layer, in float64 and straight from the definitions
(include/gdr.h): the short convolution, the norms and rotation of q and k, and the state space scan.
Each also returns how far a float32 evaluation may be off, element by element, from the roundings
that it makes (u = 2^-24 each)."""
import numpy as np

U = 2.0 ** -24


def short_conv(x, w, bias=None, s0=None, silu=True):
    """x [T, D], w [D, W], s0 [W - 1, D] -> (out [T, D], state [W - 1, D], error of out)."""
    T, D = x.shape
    W = w.shape[1]
    full = np.concatenate([np.zeros((W - 1, D)) if s0 is None else s0, x])
    out, size = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        for j in range(W):
            out[t] += w[:, j] * full[t + j]
            size[t] += np.abs(w[:, j] * full[t + j])
    if bias is not None:
        out += bias
        size += np.abs(bias)
    err = (W + 1) * U * size                    # a product and sum a tap
    if silu:
        y = out
        with np.errstate(over="ignore"):
            out = y / (1 + np.exp(-y))
        # |silu'| < 1.1; an exponential off by 2^-22 and by its argument's rounding, one division
        err = 1.1 * err + np.abs(out) * (np.abs(y) * 4 + 8) * U
    return out, full[T:], err


def qk_norm(x, weight=None, scale=1.0, rms=False, eps=1e-6, positions=None, inv_freq=None,
            interleaved=False):
    """x [rows, H, d] -> (y, error).  inv_freq: radians a position, one per pair."""
    d = x.shape[-1]
    size = (x * x).sum(-1, keepdims=True) / (d if rms else 1) + eps
    y = np.where(size > 0, x * scale / np.sqrt(np.where(size > 0, size, 1.0)), 0.0)
    if weight is not None:
        y = y * weight
    err = np.abs(y) * (d / 2 + 8) * U           # the sum of d squares under a root, five roundings
    if inv_freq is not None and len(inv_freq):
        n = len(inv_freq)
        angle = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq)
        cos, sin = np.cos(angle)[:, None], np.sin(angle)[:, None]
        first = np.arange(n) * 2 if interleaved else np.arange(n)
        second = first + 1 if interleaved else first + n
        a, b = y[..., first], y[..., second]
        ea, eb = err[..., first], err[..., second]
        y, err = y.copy(), err.copy()
        y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
        # sine and cosine of an angle that is a float32: pi u for the angle, two units for each
        e = ea + eb + (np.abs(a) + np.abs(b)) * 8 * U
        err[..., first] = err[..., second] = e
    return y, err


def ssm(x, b, c, dt, a, d=None, z=None, dt_bias=None, h0=None, softplus=True, unit=8 * U, read=0.0):
    """x, z [T, HV, dv], b, c [T, HK, dk], dt [T, HV] -> (out, S, error of out, error of S).

    ``unit``: the relative error of a state's update, of its decay (beside that of the exponent,
    which grows with its size) and of what is read out of it; ``read``: how far the copy of the
    state that an output is read from is off, relative to each element."""
    T, HV, dv = x.shape
    HK, dk = b.shape[1:]
    S = np.zeros((HV, dk, dv)) if h0 is None else h0.copy()
    size, E = np.abs(S), np.zeros_like(S)
    out, err = np.zeros((T, HV, dv)), np.zeros((T, HV, dv))
    for t in range(T):
        raw = dt[t] + (0 if dt_bias is None else dt_bias)
        step = np.logaddexp(0, raw) if softplus else raw
        keep = np.exp(step * a)[:, None, None]
        bt = np.repeat(b[t], HV // HK, 0)[:, :, None]
        ct = np.repeat(c[t], HV // HK, 0)[:, :, None]
        new = bt * (step[:, None] * x[t])[:, None, :]
        rel = unit * (1 + np.abs(step * a))[:, None, None]
        E = keep * E + rel * (keep * size + np.abs(new))
        S = keep * S + new
        size = keep * size + np.abs(new)
        out[t] = (ct * S).sum(1)
        err[t] = (np.abs(ct) * E).sum(1) + (dk * U + unit + read) * (np.abs(ct) * size).sum(1)
        if d is not None:
            out[t] += d[:, None] * x[t]
            err[t] += 2 * U * np.abs(out[t]) + 2 * U * np.abs(d[:, None] * x[t])
    if z is not None:
        with np.errstate(over="ignore"):
            gate = z / (1 + np.exp(-z))
        out, err = out * gate, np.abs(gate) * err + np.abs(out * gate) * (np.abs(z) * 4 + 10) * U
    return out, S, err, E
