"""The float64 oracles of the gated linear recurrence and the group norm against closed forms and differences."""
import numpy as np
import pytest

from oracle import gated, norm


def rng(seed=0):
    return np.random.default_rng(seed)


def gate_of(r, shape, kind):
    g = r.normal(size=shape)
    return {"decay": 1 / (1 + np.exp(-g)), "log": -np.exp(g), "logit": g}[kind]


@pytest.mark.parametrize("kind", ["decay", "log", "logit"])
@pytest.mark.parametrize("complement", [False, True])
def test_scan_is_the_weighted_sum(kind, complement):
    r = rng(1)
    x, g, init = r.normal(size=(2, 9, 3)), gate_of(r, (2, 9, 3), kind), r.normal(size=(2, 3))
    a = {"decay": g, "log": np.exp(g), "logit": 1 / (1 + np.exp(-g))}[kind]
    h, was = gated.scan(x, g, init, kind, complement)
    for t in range(9):
        want = np.prod(a[:, :t + 1], axis=1) * init
        for s in range(t + 1):
            want = want + np.prod(a[:, s + 1:t + 1], axis=1) * ((1 - a[:, s]) if complement else 1.0) * x[:, s]
        np.testing.assert_allclose(h[:, t], want, rtol=1e-12, atol=1e-13)
    np.testing.assert_array_equal(was[:, 1:], h[:, :-1])
    np.testing.assert_array_equal(was[:, 0], init)


def test_scan_with_constant_decay_is_geometric():
    x, g = np.ones((1, 50, 1)), np.full((1, 50, 1), np.log(0.9))
    h, _ = gated.scan(x, g, None, "log")
    np.testing.assert_allclose(h[0, :, 0], (1 - 0.9 ** np.arange(1, 51)) / 0.1, rtol=1e-12)
    np.testing.assert_allclose(gated.scan(x, g, None, "log", True)[0][0, :, 0], 1 - 0.9 ** np.arange(1, 51), rtol=1e-12)


def test_a_zero_decay_starts_anew():
    r = rng(2)
    x, g = r.normal(size=(1, 12, 4)), r.normal(size=(1, 12, 4))
    g[:, 5] = -np.inf
    h, _ = gated.scan(x, g, r.normal(size=(1, 4)), "logit")
    np.testing.assert_array_equal(h[:, 5:], gated.scan(x[:, 5:], g[:, 5:], None, "logit")[0])


@pytest.mark.parametrize("kind", ["decay", "log", "logit"])
@pytest.mark.parametrize("complement", [False, True])
def test_scan_gradients_by_differences(kind, complement):
    r = rng(3)
    x, g, init = r.normal(size=(2, 7, 3)), gate_of(r, (2, 7, 3), kind), r.normal(size=(2, 3))
    dy, dfinal = r.normal(size=(2, 7, 3)), r.normal(size=(2, 3))

    def loss(x, g, init):
        h, _ = gated.scan(x, g, init, kind, complement)
        return (h * dy).sum() + (h[:, -1] * dfinal).sum()

    d = gated.scan_bwd(x, g, init, dy, dfinal, kind, complement)
    for i, name in enumerate(("dx", "dgate", "dinit")):
        for _ in range(4):
            step = [np.zeros_like(x), np.zeros_like(g), np.zeros_like(init)]
            step[i] = r.normal(size=step[i].shape)
            e = 1e-6
            num = (loss(*(v + e * s for v, s in zip((x, g, init), step)))
                   - loss(*(v - e * s for v, s in zip((x, g, init), step)))) / (2 * e)
            assert abs(num - (d[name] * step[i]).sum()) <= 1e-7 * (1 + np.abs(d[name] * step[i]).sum())


def test_norm_closed_forms():
    r = rng(4)
    x = r.normal(size=(2, 5, 6)) * 3 + 1
    f = norm.forward(x, None, None, 3, eps=0.0)
    by = f["y"].reshape(2, 5, 3, 2)
    np.testing.assert_allclose(by.mean((1, 3)), 0, atol=1e-13)
    np.testing.assert_allclose(by.var((1, 3)), 1, rtol=1e-12)
    f = norm.forward(x, None, None, 3, eps=0.0, rms=True)
    np.testing.assert_allclose(np.square(f["y"].reshape(2, 5, 3, 2)).mean((1, 3)), 1, rtol=1e-12)
    # one position, one group: the norm of a row; the scale drops out
    row = norm.forward(x[:, :1], None, None, 1, eps=0.0)["y"]
    np.testing.assert_allclose(norm.forward(7 * x[:, :1], None, None, 1, eps=0.0)["y"], row, rtol=1e-12)


@pytest.mark.parametrize("act", ["none", "silu", "gate", "gate_first"])
@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradients_by_differences(act, rms):
    r = rng(5)
    shape, G = (2, 3, 8), 2
    v = dict(x=r.normal(size=shape) + 0.3, w=r.normal(size=8), b=r.normal(size=8))
    if act.startswith("gate"):
        v["z"] = r.normal(size=shape)
    dy = r.normal(size=shape)

    def loss(v):
        return (norm.forward(v["x"], v["w"], v["b"], G, v.get("z"), act=act, rms=rms)["y"] * dy).sum()

    d = norm.backward(v["x"], dy, v["w"], v["b"], G, v.get("z"), act=act, rms=rms)
    for k, name in dict(x="dx", z="dz", w="dweight", b="dbias").items():
        if k not in v:
            assert d[name] is None
            continue
        step, e = r.normal(size=v[k].shape), 1e-6
        num = (loss(dict(v, **{k: v[k] + e * step})) - loss(dict(v, **{k: v[k] - e * step}))) / (2 * e)
        assert abs(num - (d[name] * step).sum()) <= 1e-7 * (1 + np.abs(d[name] * step).sum())
