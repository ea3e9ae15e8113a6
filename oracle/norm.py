"""Float64 oracle for the group norm with an activation, channels last -- TEST INFRASTRUCTURE ONLY.

Only tests/ may import this module.  It shares no code with the CUDA path.  x (n, S, C), statistics over the S
positions and C / G channels of each (n, group):
    v = x | x silu(z),  n = w (v - mean) / sqrt(var + eps) + b,  y = n | silu(n) | n silu(z)
"""
import numpy as np


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def silu(v):
    return v * sigmoid(v)


def dsilu(v):
    s = sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


def _by_group(v, G):
    n, S, C = v.shape
    return v.reshape(n, S, G, C // G)


def _spread(m, S, C):
    """(n, G) -> (n, 1, C)."""
    return np.repeat(m, C // m.shape[1], axis=1)[:, None, :]


def forward(x, w=None, b=None, G=1, z=None, eps=1e-5, act="none", rms=False):
    """Dict with y, mean, rstd and the intermediates v, xhat, n."""
    x = np.asarray(x, np.float64)
    n, S, C = x.shape
    z = None if z is None else np.asarray(z, np.float64)
    w = np.ones(C) if w is None else np.asarray(w, np.float64)
    b = np.zeros(C) if b is None else np.asarray(b, np.float64)
    v = x * silu(z) if act == "gate_first" else x
    mean = np.zeros((n, G)) if rms else _by_group(v, G).mean((1, 3))
    rstd = 1.0 / np.sqrt(np.square(_by_group(v, G) - mean[:, None, :, None]).mean((1, 3)) + eps)
    xhat = (v - _spread(mean, S, C)) * _spread(rstd, S, C)
    p = w * xhat + b
    y = silu(p) if act == "silu" else p * silu(z) if act == "gate" else p
    return dict(y=y, mean=mean, rstd=rstd, v=v, xhat=xhat, n=p)


def backward(x, dy, w=None, b=None, G=1, z=None, eps=1e-5, act="none", rms=False):
    """Dict with dx, dz, dweight, dbias, and dn (the gradient of n)."""
    f = forward(x, w, b, G, z, eps, act, rms)
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    n, S, C = x.shape
    z = None if z is None else np.asarray(z, np.float64)
    w = np.ones(C) if w is None else np.asarray(w, np.float64)
    xhat, rstd = f["xhat"], _spread(f["rstd"], S, C)
    dn = dy * (dsilu(f["n"]) if act == "silu" else silu(z) if act == "gate" else 1.0)
    q = dn * w
    m1 = 0.0 if rms else _spread(_by_group(q, G).mean((1, 3)), S, C)
    m2 = _spread(_by_group(q * xhat, G).mean((1, 3)), S, C)
    dv = rstd * (q - m1 - xhat * m2)
    dx, dz = dv, None
    if act == "gate":
        dz = dy * f["n"] * dsilu(z)
    elif act == "gate_first":
        dx, dz = dv * silu(z), dv * x * dsilu(z)
    return dict(dx=dx, dz=dz, dweight=(dn * xhat).sum((0, 1)), dbias=dn.sum((0, 1)), dn=dn, f=f)
