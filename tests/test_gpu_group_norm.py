"""The group norm with an activation (ssd_group_norm, _bwd) against the float64 oracle.

Tolerances, with e = 2^-24 (half a unit of float32): the statistics are sums of values up to V = max |v| of the
group, xhat is off by at most 64 e (|xhat| + rstd V), and every later step carries that on through its derivative
and adds a few roundings of its own; the sums of the backward pass are off by 64 e of the sum of their terms'
magnitudes and by what their terms are off.  bf16 results are rounded once more, by at most 2^-9 of the value; 2^-8 is
allowed.  Below 2^-126, float32's smallest normal number, values lose their bits or are zero.
"""
import numpy as np
import pytest

from oracle import norm
from state_space_model_02_gb300 import ssd

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E = 2.0 ** -24
TINY = 2.0 ** -126
ACTS = ["none", "silu", "gate", "gate_first"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_model_02_gb300 import build as cuda_build

    cuda_build.build()
    ssd.load_library()


def inputs(n, S, C, dtype, act, seed, shift=0.3):
    g = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    t = dict(x=(torch.randn(n, S, C, generator=g) + shift * torch.randn(C, generator=g)).to(dt),
             w=1 + 0.2 * torch.randn(C, generator=g), b=0.2 * torch.randn(C, generator=g),
             dy=torch.randn(n, S, C, generator=g).to(dt))
    t["z"] = torch.randn(n, S, C, generator=g).to(dt) if act.startswith("gate") else None
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, want, tol, dtype, name=""):
    got = host(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= TINY + tol + np.abs(want) * (2.0 ** -8 if dtype == "bf16" else 16 * E))
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:3], np.abs(got - want)[bad][:3])


def per_group(v, G, how):
    n, S, C = v.shape
    return np.repeat(how(v.reshape(n, S, G, C // G), axis=(1, 3)), C // G, axis=1)[:, None, :]


def check(t, G, dtype, act, rms, eps=1e-5, backward=True, affine=True):
    x, w, b, z, dy = (host(t[k]) for k in ("x", "w", "b", "z", "dy"))
    n, S, C = x.shape
    if not affine:
        w, b = np.ones(C), np.zeros(C)
    f = norm.forward(x, w, b, G, z, eps, act, rms)
    rstd = np.repeat(f["rstd"], C // G, axis=1)[:, None, :]
    tx = 64 * E * (np.abs(f["xhat"]) + rstd * per_group(np.abs(f["v"]), G, np.max))
    tp = np.abs(w) * tx + 4 * E * (np.abs(w * f["xhat"]) + np.abs(b))
    ty = 1.2 * tp if act == "silu" else np.abs(norm.silu(z)) * tp if act == "gate" else tp
    pw, pb = (t["w"], t["b"]) if affine else (None, None)
    y, mean, rs = ssd.group_norm(t["x"], pw, pb, groups=G, z=t["z"], eps=eps, act=act, rms=rms, want_stats=True)
    torch.cuda.synchronize()
    close(y, f["y"], ty + 16 * E * np.abs(f["y"]), dtype, "y")
    close(mean, f["mean"], 64 * E * per_group(np.abs(f["v"]), G, np.max)[:, 0, ::C // G], "f32", "mean")
    close(rs, f["rstd"], 64 * E * f["rstd"] * (1 + f["rstd"] * per_group(np.abs(f["v"]), G, np.max)[:, 0, ::C // G]),
          "f32", "rstd")
    if not backward:
        return
    r = norm.backward(x, dy, w, b, G, z, eps, act, rms)
    slope = np.abs(norm.dsilu(f["n"]) if act == "silu" else norm.silu(z) if act == "gate" else np.ones_like(x))
    tdn = np.abs(dy) * ((0.6 * tp if act == "silu" else 0) + 16 * E * (1 + slope))
    dn, q, xh = r["dn"], r["dn"] * w, f["xhat"]
    tq = tdn * np.abs(w) + 4 * E * np.abs(q)
    mean_of = lambda v: per_group(v, G, np.mean)
    m1, m2 = (0 if rms else np.abs(mean_of(q))), np.abs(mean_of(q * xh))
    t1 = 0 if rms else mean_of(tq) + 64 * E * mean_of(np.abs(q))
    t2 = mean_of(tq * np.abs(xh) + np.abs(q) * tx) + 64 * E * mean_of(np.abs(q * xh))
    tv = rstd * (tq + t1 + np.abs(xh) * t2 + tx * m2) + 64 * E * rstd * (np.abs(q) + m1 + np.abs(xh) * m2)
    tv = tv * (1 + 0 * x)
    d = ssd.group_norm_bwd(t["x"], t["dy"], mean, rs, pw, pb, groups=G, z=t["z"], act=act, rms=rms)
    torch.cuda.synchronize()
    if act == "gate_first":
        tdz = np.abs(x) * np.abs(norm.dsilu(z)) * tv + 16 * E * np.abs(x) * np.abs(r["dx"] * 0 + tv * 0 + 1) * np.abs(
            rstd * (np.abs(q) + m1 + np.abs(xh) * m2))
        close(d["dz"], r["dz"], tdz, dtype, "dz")
        tv = tv * np.abs(norm.silu(z))
    elif act == "gate":
        close(d["dz"], r["dz"], np.abs(dy) * (np.abs(norm.dsilu(z)) * tp + 16 * E * (1 + np.abs(f["n"]))), dtype, "dz")
    else:
        assert d["dz"] is None
    close(d["dx"], r["dx"], tv, dtype, "dx")
    close(d["dweight"], r["dweight"], (tdn * np.abs(xh) + np.abs(dn) * tx).sum((0, 1))
          + 64 * E * np.abs(dn * xh).sum((0, 1)), "f32", "dweight")
    close(d["dbias"], r["dbias"], tdn.sum((0, 1)) + 64 * E * np.abs(dn).sum((0, 1)), "f32", "dbias")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("n,S,C,G", [(37, 1, 256, 4), (3, 50, 96, 6)])
def test_forms(dtype, act, rms, n, S, C, G):
    check(inputs(n, S, C, dtype, act, 1), G, dtype, act, rms)


# one row a statistic: every width of a group from one channel to rows that fill a CTA and more
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,C,G", [(1, 1, 1), (5, 7, 7), (3, 30, 5), (130, 64, 1), (9, 1536, 24), (7, 1000, 1),
                                   (33, 520, 2), (300, 24, 3), (6, 5120, 8), (4, 5120, 1), (2, 6144, 1), (3, 8200, 1),
                                   (2, 20000, 1), (2, 40960, 2), (1, 100003, 1)])
def test_tokens(dtype, n, C, G):
    check(inputs(n, 1, C, dtype, "gate", 2 + C), G, dtype, "gate", False)
    check(inputs(n, 1, C, dtype, "gate_first", 3 + C), G, dtype, "gate_first", True)


# wide groups whose rows take packs of one or two channels, with more samples than CTAs and with fewer
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,C,G", [(401, 1337, 1), (200, 2050, 2), (160, 2091, 1), (3, 2047, 1), (3, 2049, 1), (2, 4095, 1),
                                   (2, 4097, 1), (161, 4098, 1), (2, 8190, 1), (2, 8191, 1), (2, 8193, 1)])
def test_wide_odd_rows(dtype, n, C, G):
    check(inputs(n, 1, C, dtype, "gate_first", 30 + C), G, dtype, "gate_first", False)
    check(inputs(n, 1, C, dtype, "none", 31 + C), G, dtype, "none", True)


# rows of single bf16 values at both offsets in a word; what lies around them is never taken in
@pytest.mark.parametrize("n,C,G", [(1, 3, 3), (700, 72, 24), (33, 299, 1), (200, 416, 32), (5, 2051, 1), (3, 16382, 2),
                                   (2, 16385, 1)])
@pytest.mark.parametrize("at,more", [(0, 1), (1, 2), (3, 8)])
def test_odd_rows(n, C, G, at, more):
    for act in ("gate", "none"):
        t = inputs(n, 1, C, "bf16", act, 40 + C + at)
        for k in ("x", "z"):
            if t[k] is not None:
                wide = torch.full((n, 1, C + more), float("nan"), dtype=torch.bfloat16, device="cuda")
                wide[:, :, at:at + C] = t[k]
                t[k] = wide[:, :, at:at + C]
        check(t, G, "bf16", act, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,S,C,G", [(1, 2, 1, 1), (2, 3, 5, 5), (2, 64, 64, 2), (3, 65, 64, 64), (2, 1000, 66, 11),
                                     (1, 4096, 64, 4), (5, 333, 320, 32), (2, 17, 2048, 1), (1, 20000, 48, 3),
                                     (1, 30000, 256, 8), (2, 5001, 130, 2), (40, 2, 64, 8), (1, 40000, 9, 3)])
def test_positions(dtype, n, S, C, G):
    check(inputs(n, S, C, dtype, "silu", 4 + S), G, dtype, "silu", False)


@pytest.mark.parametrize("act", ["none", "gate_first", "gate"])
@pytest.mark.parametrize("n,S,C,G", [(2, 2500, 128, 2), (1, 26000, 64, 4)])
def test_positions_with_other_forms(act, n, S, C, G):
    for rms in (False, True):
        check(inputs(n, S, C, "bf16", act, 5), G, "bf16", act, rms)


def test_no_affine_map():
    check(inputs(20, 1, 128, "f32", "silu", 6), 2, "f32", "silu", False, affine=False)
    check(inputs(2, 300, 64, "bf16", "gate", 6), 2, "bf16", "gate", False, affine=False)


def test_a_mean_far_from_zero():
    # a mean of 1000 deviations: sums of squares without the mean taken out would have lost the variance
    for n, S, C, G in ((16, 1, 256, 1), (2, 500, 64, 2), (1, 30000, 64, 1)):
        t = inputs(n, S, C, "f32", "none", 7)
        t["x"] += 1000.0
        check(t, G, "f32", "none", False)


def test_constant_and_zero_rows():
    for S in (1, 40, 6000):
        t = inputs(2, S, 64, "f32", "silu", 8)
        t["x"][0] = 0.0
        t["x"][1] = 5.0
        y, mean, rstd = ssd.group_norm(t["x"], t["w"], t["b"], groups=2, act="silu", want_stats=True)
        want = torch.nn.functional.silu(t["b"]).expand_as(y)
        torch.testing.assert_close(y, want, rtol=1e-6, atol=1e-6)
        assert torch.equal(mean[0], torch.zeros_like(mean[0])) and torch.isfinite(rstd).all()
        d = ssd.group_norm_bwd(t["x"], t["dy"], mean, rstd, t["w"], t["b"], groups=2, act="silu")
        assert all(torch.isfinite(d[k]).all() for k in ("dx", "dweight", "dbias"))


def test_infinities_and_nan_stay_in_their_group():
    for S in (1, 30, 9000):
        t = inputs(3, S, 64, "f32", "gate", 9)
        want = ssd.group_norm(t["x"], t["w"], t["b"], groups=4, z=t["z"], act="gate")
        bad = t["x"].clone()
        bad[1, S // 2, 20] = float("nan")
        bad[2, 0, 40] = float("inf")
        y = ssd.group_norm(bad, t["w"], t["b"], groups=4, z=t["z"], act="gate")
        keep = torch.ones(3, 4, dtype=torch.bool)
        keep[1, 1] = keep[2, 2] = False
        by, wt = y.view(3, S, 4, 16), want.view(3, S, 4, 16)
        for i in range(3):
            for g in range(4):
                if keep[i, g]:
                    assert torch.equal(by[i, :, g], wt[i, :, g])
                else:
                    assert torch.isnan(by[i, :, g]).any()


def test_gates_of_any_size():
    t = inputs(10, 1, 64, "f32", "gate", 10)
    t["z"][0, 0, :8] = torch.tensor([-200.0, 200.0, -88.0, 88.0, -1e30, 1e30, 0.0, -0.0])
    check(t, 2, "f32", "gate", False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [1, 70])
@pytest.mark.parametrize("at", [0, 1, 8, 64])
def test_slices_of_wider_rows(dtype, S, at):
    t = inputs(6, S, 64, dtype, "gate_first", 11)
    wide = torch.full((6, S, 192), float("nan"), dtype=t["x"].dtype, device="cuda")
    wide[..., at:at + 64], wide[..., 128:] = t["x"], t["z"]
    check(dict(t, x=wide[..., at:at + 64], z=wide[..., 128:]), 4, dtype, "gate_first", True)


def test_offsets_beyond_32_bits():
    S, C, W = 150000, 32, 16384
    t = inputs(1, S, C, "bf16", "silu", 12)
    wide = torch.empty((1, S, W), dtype=torch.bfloat16, device="cuda")
    x = wide[..., W - C:]
    x.copy_(t["x"])
    want = ssd.group_norm(t["x"], t["w"], t["b"], groups=2, act="silu", want_stats=True)
    got = ssd.group_norm(x, t["w"], t["b"], groups=2, act="silu", want_stats=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    want = ssd.group_norm_bwd(t["x"], t["dy"], want[1], want[2], t["w"], t["b"], groups=2, act="silu")
    got = ssd.group_norm_bwd(x, t["dy"], got[1], got[2], t["w"], t["b"], groups=2, act="silu")
    assert all(torch.equal(want[k], got[k]) for k in ("dx", "dweight", "dbias"))


def test_many_rows():
    # more rows than a grid has in its y direction
    t = inputs(70001, 1, 8, "bf16", "silu", 13)
    check(t, 1, "bf16", "silu", False)
    check(inputs(70001, 2, 4, "bf16", "silu", 14), 2, "bf16", "silu", False)


def test_the_same_call_gives_the_same_bits():
    for n, S, C, G in ((5000, 1, 1536, 24), (4, 4096, 256, 8), (1, 30000, 128, 4)):
        t = inputs(n, S, C, "bf16", "silu", 15)
        run = lambda: ssd.group_norm(t["x"], t["w"], t["b"], groups=G, act="silu", want_stats=True)
        one = run()
        back = lambda s: ssd.group_norm_bwd(t["x"], t["dy"], s[1], s[2], t["w"], t["b"], groups=G, act="silu")
        g1 = back(one)
        for _ in range(3):
            two = run()
            assert all(torch.equal(a, b) for a, b in zip(one, two))
            g2 = back(two)
            assert all(torch.equal(g1[k], g2[k]) for k in ("dx", "dweight", "dbias"))


def test_another_stream():
    t = inputs(2, 30000, 64, "bf16", "silu", 16)
    want = ssd.group_norm(t["x"], t["w"], t["b"], groups=2, act="silu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = ssd.group_norm(t["x"], t["w"], t["b"], groups=2, act="silu", stream=s)
    s.synchronize()
    assert torch.equal(want, got)


def test_gradient_by_differences():
    t = inputs(2, 40, 24, "f32", "gate_first", 17)
    _, mean, rstd = ssd.group_norm(t["x"], t["w"], t["b"], groups=3, z=t["z"], act="gate_first", want_stats=True)
    d = ssd.group_norm_bwd(t["x"], t["dy"], mean, rstd, t["w"], t["b"], groups=3, z=t["z"], act="gate_first")
    x, z, w, b, dy = (host(t[k]) for k in ("x", "z", "w", "b", "dy"))
    r = np.random.default_rng(0)
    sx, sz, sw, sb = (r.normal(size=v.shape) for v in (x, z, w, b))

    def loss(e):
        return (norm.forward(x + e * sx, w + e * sw, b + e * sb, 3, z + e * sz, act="gate_first")["y"] * dy).sum()

    num = (loss(1e-5) - loss(-1e-5)) / 2e-5
    terms = [host(d["dx"]) * sx, host(d["dz"]) * sz, host(d["dweight"]) * sw, host(d["dbias"]) * sb]
    scale = sum(np.abs(v).sum() for v in terms)
    assert abs(num - sum(v.sum() for v in terms)) <= scale * (256 * E + 1e-8)


def test_refusals():
    t = inputs(2, 10, 32, "bf16", "gate", 18)
    x, z = t["x"], t["z"]
    with pytest.raises(ValueError):
        ssd.group_norm(x, act="relu")
    with pytest.raises(ValueError):
        ssd.group_norm(x, act="gate")
    with pytest.raises(ValueError):
        ssd.group_norm(x, act="silu", z=z)
    with pytest.raises(ValueError):
        ssd.group_norm(x, act="gate", z=z[:1])
    with pytest.raises(ValueError):
        ssd.group_norm(x[0])
    with pytest.raises(TypeError):
        ssd.group_norm(x.half())
    with pytest.raises(TypeError):
        ssd.group_norm(x, t["w"].bfloat16())
    with pytest.raises(ValueError):
        ssd.group_norm(x.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ssd.SSDError):
        ssd.group_norm(x, groups=5)
    with pytest.raises(ssd.SSDError):
        ssd.group_norm(x, groups=0)
    with pytest.raises(ssd.SSDError):
        ssd.group_norm(x, eps=-1.0)
    with pytest.raises(ssd.SSDError):
        ssd.group_norm(x, eps=float("nan"))
