"""Layer / RMS norm and the SwiGLU gate with their gradients, in fp64 (plain
numpy).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``). The SII open-source-week
post on Metis trains LLaMA-style layers; these are the parts between their FP4
projections:

    mean = sum(x) / n (0 for RMS), rstd = (sum((x - mean)^2) / n + eps)^(-1/2)
    y = (x - mean) rstd w + b
    dx = rstd (g - [layer: sum(g) / n] - xh sum(g xh) / n),  g = dy w
    dw = sum over rows of dy xh,  db = sum over rows of dy,  xh = (x - mean) rstd

    h = silu(a) b, silu(a) = a s, s = 1 / (1 + exp(-a))
    da = dh b s (1 + a (1 - s)),  db = dh a s

Pins (tests/test_oracle_ffn.py): gradients against central differences of the
forward functions; normalized rows have mean 0 and the stated second moment;
invariance under shifts and scalings of the input; silu against its limits.
"""
import numpy as np


def norm_stats(x, kind, eps):
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1) if kind == "layer" else np.zeros(x.shape[0])
    var = ((x - mean[:, None]) ** 2).mean(axis=1)
    return mean, 1.0 / np.sqrt(var + eps)


def norm_fwd(x, w, b, kind, eps):
    mean, rstd = norm_stats(x, kind, eps)
    xh = (np.asarray(x, dtype=np.float64) - mean[:, None]) * rstd[:, None]
    return xh * (1.0 if w is None else w) + (0.0 if b is None else b)


def norm_bwd(dy, x, w, mean, rstd, kind):
    """Gradients (dx, dw, db) at the given row statistics (mean is not read
    for RMS)."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    n = x.shape[1]
    m = np.asarray(mean, dtype=np.float64)[:, None] if kind == "layer" else 0.0
    r = np.asarray(rstd, dtype=np.float64)[:, None]
    xh = (x - m) * r
    g = dy * (1.0 if w is None else w)
    level = g.sum(axis=1, keepdims=True) / n if kind == "layer" else 0.0
    dx = r * (g - level - xh * ((g * xh).sum(axis=1, keepdims=True) / n))
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def sigmoid(a):
    """1 / (1 + exp(-a)) without overflow."""
    a = np.asarray(a, dtype=np.float64)
    z = np.exp(-np.abs(a))
    return np.where(a >= 0, 1.0 / (1.0 + z), z / (1.0 + z))


def swiglu_fwd(a, b):
    return a * sigmoid(a) * b


def swiglu_bwd(dh, a, b):
    """(da, db, h)."""
    s = sigmoid(a)
    return dh * b * s * (1.0 + a * sigmoid(-np.asarray(a))), dh * a * s, a * s * b
