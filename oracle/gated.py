"""Float64 oracle for the gated linear recurrence -- TEST INFRASTRUCTURE ONLY.

Only tests/ may import this module.  It shares no code with the CUDA path.  Per (batch, channel):
    h_t = a_t h_{t-1} + u_t,  a_t = g_t | exp(g_t) | 1 / (1 + exp(-g_t)),  u_t = x_t | (1 - a_t) x_t
written token by token, and the gradients by the chain rule through each token's update.
"""
import numpy as np


def decay(g, kind):
    """(a, 1 - a) in float64."""
    g = np.asarray(g, np.float64)
    if kind == "decay":
        return g, 1.0 - g
    with np.errstate(over="ignore"):
        if kind == "log":
            return np.exp(g), -np.expm1(g)
        return 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))


def scan(x, g, init=None, kind="logit", complement=False):
    """(h, was): the states (b, L, D) and the state that each token starts from."""
    x = np.asarray(x, np.float64)
    a, s = decay(g, kind)
    u = s * x if complement else x
    h, was = np.empty_like(x), np.empty_like(x)
    last = np.zeros_like(x[:, 0]) if init is None else np.asarray(init, np.float64)
    for t in range(x.shape[1]):
        was[:, t] = last
        last = a[:, t] * last + u[:, t]
        h[:, t] = last
    return h, was


def scan_bwd(x, g, init, dy, dfinal=None, kind="logit", complement=False):
    """dx, dgate, dinit, and G (the gradient of each state)."""
    x = np.asarray(x, np.float64)
    a, s = decay(g, kind)
    _, was = scan(x, g, init, kind, complement)
    c = np.zeros_like(x[:, 0]) if dfinal is None else np.asarray(dfinal, np.float64)
    G = np.empty_like(x)
    for t in reversed(range(x.shape[1])):
        G[:, t] = dy[:, t] + c
        c = a[:, t] * G[:, t]
    da = G * (was - x if complement else was)
    slope = {"decay": 1.0, "log": a, "logit": a * s}[kind]
    return dict(dx=G * s if complement else G, dgate=da * slope, dinit=c, G=G)


def reach(g, kind, flip=False):
    """E_t = 1 + |a_t| E_{t-1} (or from the right): how many tokens' errors add up in a state."""
    a = np.abs(decay(g, kind)[0])
    if flip:  # the adjoint multiplies by the next token's decay
        a = np.concatenate([a[:, 1:], np.ones_like(a[:, :1])], 1)[:, ::-1]
    E = np.empty_like(a)
    last = np.ones_like(a[:, 0])
    for t in range(a.shape[1]):
        last = 1.0 + a[:, t] * last
        E[:, t] = last
    return E[:, ::-1] if flip else E
