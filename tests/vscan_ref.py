"""The vector-state scan in fp64 numpy, token by token from its definition
(test infrastructure): x_t = f_t x_{t-1} + i_t h_t, y_t = x_t SiLU(z_t) with
f = sigmoid(a), i = sigmoid(b) (b absent: 1 - f), and its reverse-mode
gradients."""
from __future__ import annotations

import numpy as np


def f64(t):
    if t is None:
        return None
    return t.detach().double().cpu().numpy() if hasattr(t, "detach") else np.asarray(t, np.float64)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def fwd(h, a, b=None, z=None, x0=None):
    """Returns (y, x_final, xs) with xs [batch, seqlen + 1, d], xs[:, 0] = x0."""
    h, a, b, z, x0 = map(f64, (h, a, b, z, x0))
    Bt, L, d = h.shape
    f = sigmoid(a)
    i = sigmoid(-a) if b is None else sigmoid(b)
    xs = np.zeros((Bt, L + 1, d))
    if x0 is not None:
        xs[:, 0] = x0
    for t in range(L):
        xs[:, t + 1] = f[:, t] * xs[:, t] + i[:, t] * h[:, t]
    y = xs[:, 1:] if z is None else xs[:, 1:] * z * sigmoid(z)
    return y, xs[:, -1], xs


def bwd(dy, h, a, b=None, z=None, x0=None, dx_final=None):
    """Gradients as a dict: dh, da, db, dz, dx0."""
    _, _, xs = fwd(h, a, b, z, x0)
    dy, h, a, b, z, dx_final = map(f64, (dy, h, a, b, z, dx_final))
    Bt, L, d = h.shape
    f, fc = sigmoid(a), sigmoid(-a)
    i = fc if b is None else sigmoid(b)
    out = {"db": None, "dz": None}
    dx = dy
    if z is not None:
        s = sigmoid(z)
        out["dz"] = dy * xs[:, 1:] * (s + z * s * (1 - s))
        dx = dy * z * s
    g = np.zeros_like(h)
    r = np.zeros((Bt, d)) if dx_final is None else dx_final
    for t in range(L - 1, -1, -1):
        g[:, t] = dx[:, t] + r
        r = f[:, t] * g[:, t]
    out["dx0"] = r
    out["dh"] = g * i
    df = g * xs[:, :-1]
    if b is None:
        df = df - g * h
    else:
        out["db"] = g * h * i * sigmoid(-b)  # 1 - i without cancellation
    out["da"] = df * f * fc
    return out
