"""A state space layer's operators on the CPU in float64: the selective scan, the short causal
convolution and the gated norm, by their formulas.  Used only by the tests and the smoke run."""
import numpy as np


def softplus(x):
    with np.errstate(invalid="ignore"):
        return np.logaddexp(x, 0.0)


def scan_run(S, x, dt, A, B, C, D=None, dt_bias=None, dt_softplus=False, keep=False):
    """Tokens x [T, h, p], dt [T, h], B and C [T, g, n] from S [h, p, n].  Returns (o [T, h, p], S,
    the states before the first and after every token, or None)."""
    S = np.array(S, dtype=np.float64)
    T, h, _ = x.shape
    share = h // B.shape[1]
    o = np.zeros(x.shape)
    states = [S.copy()] if keep else None
    for t in range(T):
        step = np.asarray(dt[t], dtype=np.float64) + (0.0 if dt_bias is None else dt_bias)
        step = softplus(step) if dt_softplus else step
        b, c = np.repeat(B[t], share, 0), np.repeat(C[t], share, 0)
        with np.errstate(invalid="ignore", over="ignore"):
            S = S * np.exp(step * A)[:, None, None] + (step[:, None] * x[t])[:, :, None] * b[:, None, :]
            o[t] = (S * c[:, None, :]).sum(-1)
            if D is not None:
                o[t] += D[:, None] * x[t]
        if keep:
            states.append(S.copy())
    return o, S, states


def conv_run(tail, u, weight, bias=None, activation="silu"):
    """Inputs u [T, ch] after tail [w - 1, ch], filters [ch, w].  Returns (o [T, ch], the new tail)."""
    w = weight.shape[1]
    line = np.concatenate([tail, u])
    T = len(u)
    o = np.zeros(u.shape) if bias is None else np.tile(np.asarray(bias, dtype=np.float64), (T, 1))
    for j in range(w):
        o = o + line[j:j + T] * weight[:, j]
    if activation == "silu":
        with np.errstate(over="ignore"):
            o = o / (1 + np.exp(-o))
    return o, line[T:]


def gate(z, activation):
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-z))
    return z * s if activation == "silu" else s if activation == "sigmoid" else z


def gated_norm(x, z=None, weight=None, bias=None, group=None, eps=1e-5, kind="rms", activation="silu", gate_first=False):
    rows, width = x.shape
    group = width if group is None else group
    u = x * gate(z, activation) if z is not None and gate_first else x
    u = u.reshape(rows, width // group, group)
    if kind == "layer":
        u = u - u.mean(-1, keepdims=True)
    y = (u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)).reshape(rows, width)
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y * gate(z, activation) if z is not None and not gate_first else y
