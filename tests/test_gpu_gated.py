"""The gated linear recurrence (ssd_gated_scan, _bwd, ssd_gated_decode) against the float64 oracle.

Tolerances, with e = 2^-24 (half a unit of float32): a step of the recurrence adds a handful of roundings of
values up to M = max |h| of the channel, and an error of token s reaches token t times the decays between them,
so |h - h_ref| <= 16 e M E_t with E_t = 1 + |a_t| E_{t-1} (oracle.gated.reach); likewise for the adjoint from the
right.  bf16 results are rounded once more, by at most 2^-9 of the value; 2^-8 is allowed.  Below 2^-126, float32's
smallest normal number, values lose their bits or are zero.
"""
import numpy as np
import pytest

from oracle import gated
from state_space_model_02_gb300 import ssd

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E = 2.0 ** -24
TINY = 2.0 ** -126
KINDS = ["decay", "log", "logit"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_model_02_gb300 import build as cuda_build

    cuda_build.build()
    ssd.load_library()


def inputs(b, L, D, dtype, kind, seed, resets=0, init=True):
    g = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    logit = torch.randn(b, L, D, generator=g) * 1.5 + 4 * torch.rand(D, generator=g) - 1
    gate = {"logit": logit, "log": -torch.exp(-logit), "decay": torch.sigmoid(logit)}[kind].clone()
    if kind == "decay":
        gate[:, 1::7] *= -1.0
    for k in range(resets):
        gate[k % b, (k * 37 + 5) % L] = 0.0 if kind == "decay" else -np.inf
    t = dict(x=torch.randn(b, L, D, generator=g).to(dt), gate=gate.to(dt),
             init=torch.randn(b, D, generator=g) if init else None,
             dy=torch.randn(b, L, D, generator=g).to(dt), dfinal=torch.randn(b, D, generator=g))
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, want, tol, dtype):
    got = host(got)
    bad = np.abs(got - want) > TINY + tol + np.abs(want) * (2.0 ** -8 if dtype == "bf16" else 4 * E)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], np.abs(got - want)[bad][:3])


def reference(t, kind, complement):
    x, gate, init = host(t["x"]), host(t["gate"]), host(t["init"])
    h, was = gated.scan(x, gate, init, kind, complement)
    M = np.maximum(np.abs(h).max(1), np.abs(was).max(1))[:, None]
    return h, was, 16 * E * M * gated.reach(gate, kind)


def check_forward(t, dtype, kind, complement, **kw):
    h, was, tol = reference(t, kind, complement)
    y, fin, states = ssd.gated_scan(t["x"], t["gate"], t["init"], kind=kind, complement=complement, want_states=True,
                                    **kw)
    torch.cuda.synchronize()
    close(y, h, tol, dtype)
    close(fin, h[:, -1], tol[:, -1], "f32")
    B = ssd.GATED_BLOCK
    tol_in = np.concatenate([np.zeros_like(tol[:, :1]), tol[:, :-1]], 1)
    close(states, was[:, ::B], tol_in[:, ::B], "f32")
    return states


def check_backward(t, states, dtype, kind, complement, dfinal=True):
    x, gate, init, dy = (host(t[k]) for k in ("x", "gate", "init", "dy"))
    df = host(t["dfinal"]) if dfinal else None
    h, was, tol_h = reference(t, kind, complement)
    r = gated.scan_bwd(x, gate, init, dy, df, kind, complement)
    tol_G = 16 * E * np.maximum(np.abs(r["G"]).max(1), 0 if df is None else np.abs(df))[:, None] * gated.reach(
        gate, kind, flip=True)
    tol_was = np.concatenate([np.zeros_like(tol_h[:, :1]), tol_h[:, :-1]], 1)
    d = ssd.gated_scan_bwd(t["x"], t["gate"], t["dy"], states, t["dfinal"] if dfinal else None, kind=kind,
                           complement=complement)
    torch.cuda.synchronize()
    a, s = gated.decay(gate, kind)
    close(d["dx"], r["dx"], tol_G * (np.abs(s) if complement else 1) + 8 * E * np.abs(r["dx"]), dtype)
    w = was - x if complement else was
    slope = {"decay": 1.0, "log": a, "logit": a * s}[kind]
    close(d["dgate"], r["dgate"], slope * (tol_G * np.abs(w) + np.abs(r["G"]) * (tol_was + 4 * E * np.abs(w)))
          + 16 * E * np.abs(r["dgate"]), dtype)
    close(d["dinit"], r["dinit"], np.abs(a[:, 0]) * tol_G[:, 0], "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("complement", [False, True])
def test_kinds_forward_and_backward(dtype, kind, complement):
    t = inputs(2, 333, 70, dtype, kind, 1, resets=5)
    states = check_forward(t, dtype, kind, complement)
    check_backward(t, states, dtype, kind, complement)


@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513, 1025, 2049])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths(L, dtype):
    t = inputs(2, L, 66, dtype, "logit", 100 + L, resets=1)
    check_backward(t, check_forward(t, dtype, "logit", True), dtype, "logit", True)


@pytest.mark.parametrize("D", [1, 2, 3, 31, 32, 33, 63, 64, 65, 127, 129, 258])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_channel_counts(D, dtype):
    t = inputs(3, 300, D, dtype, "log", 200 + D)
    check_backward(t, check_forward(t, dtype, "log", False), dtype, "log", False)


@pytest.mark.parametrize("b,L,D,dtype", [(1, 9000, 64, "bf16"), (1, 5003, 192, "f32"), (2, 3000, 1026, "bf16"),
                                         (4, 2048, 1536, "bf16"), (64, 40, 320, "bf16"), (9, 700, 2048, "f32"),
                                         (1, 20000, 33, "bf16")])
def test_larger(b, L, D, dtype):
    t = inputs(b, L, D, dtype, "logit", b + L, resets=9)
    check_backward(t, check_forward(t, dtype, "logit", True), dtype, "logit", True)


@pytest.mark.parametrize("b,L,D,dtype", [(1, 8, 130, "bf16"), (1, 9, 130, "bf16"), (1, 4, 130, "f32"), (1, 5, 130, "f32"),
                                         (64, 130, 2050, "bf16"), (64, 132, 2048, "bf16"), (64, 65, 2048, "f32"),
                                         (80, 63, 1001, "f32"), (2, 20, 9216, "bf16"), (2, 19, 9216, "bf16")])
def test_short_sequences(b, L, D, dtype):
    """On both sides of what single threads walk: few tokens, or many columns with blocks of 64 tokens to save."""
    t = inputs(b, L, D, dtype, "logit", seed=b + L + D)
    check_backward(t, check_forward(t, dtype, "logit", True), dtype, "logit", True)


@pytest.mark.parametrize("L,D,dtype", [(8192, 1600, "bf16"), (8193, 3008, "bf16"), (8191, 1601, "f32"), (8200, 1601, "f32"),
                                       (2048, 1536, "bf16"), (8192, 3009, "f32")])
def test_columns_in_segments_and_clusters(L, D, dtype):
    """On both sides of the columns and lengths that the backward pass cuts into segments."""
    t = inputs(1, L, D, dtype, "log", seed=L + D)
    check_backward(t, check_forward(t, dtype, "log", False), dtype, "log", False)


@pytest.mark.parametrize("b,L,D", [(1, 6000, 123), (2, 2600, 1001), (11, 257, 1001), (1, 40, 1), (3, 70, 65), (5, 200, 4097)])
@pytest.mark.parametrize("at,more", [(0, 0), (1, 2), (33, 40), (7, 9)])
def test_odd_rows(b, L, D, at, more):
    """bf16 rows at every offset from a multiple of 16 bytes, in each kernel; what lies around them is never taken in."""
    t = inputs(b, L, D, "bf16", "logit", seed=L + D + at)
    for k in ("x", "gate"):
        wide = torch.full((b, L, D + more), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :, at:at + D] = t[k]
        t[k] = wide[:, :, at:at + D]
    check_backward(t, check_forward(t, "bf16", "logit", True), "bf16", "logit", True)


def test_no_initial_state_and_no_dfinal():
    t = inputs(2, 200, 48, "f32", "logit", 7, init=False)
    check_backward(t, check_forward(t, "f32", "logit", False), "f32", "logit", False, dfinal=False)


def test_long_memory():
    # decays of 1 - 2^-12: a state is the sum over thousands of tokens and a tile's product stays near one
    t = inputs(1, 12000, 64, "f32", "decay", 8)
    t["gate"].fill_(1 - 2.0 ** -12)
    check_backward(t, check_forward(t, "f32", "decay", True), "f32", "decay", True)


def test_extreme_gates():
    for kind, values in (("logit", [-np.inf, -200.0, -30.0, 0.0, 30.0, 200.0, np.inf]), ("log", [-np.inf, -100.0, -1e-6, 0.0])):
        t = inputs(1, 7 * 30, 64, "f32", kind, 9)
        t["gate"][:] = torch.tensor(np.resize(values, 7 * 30), dtype=torch.float32, device="cuda")[None, :, None]
        for complement in (False, True):
            check_backward(t, check_forward(t, "f32", kind, complement), "f32", kind, complement)


@pytest.mark.parametrize("kind", KINDS)
def test_all_tokens_forgotten(kind):
    t = inputs(2, 150, 34, "f32", kind, 10)
    t["gate"].fill_(0.0 if kind == "decay" else -np.inf)
    y, fin = ssd.gated_scan(t["x"], t["gate"], t["init"], kind=kind)
    assert torch.equal(y, t["x"]) and torch.equal(fin, t["x"][:, -1])


def test_what_a_reset_follows_does_not_matter():
    # the tokens behind a reset, and their gradients, are those of a sequence that starts there: bit for bit where
    # the reset is the first token of a tile of every variant
    t = inputs(1, 8192 + 300, 64, "bf16", "logit", 11)
    t["gate"][:, 8192] = -np.inf
    y, fin = ssd.gated_scan(t["x"], t["gate"], t["init"])
    other = t["x"].clone()
    other[:, :8192] = 1e30
    y2, fin2 = ssd.gated_scan(other, t["gate"], None)
    assert torch.equal(y[:, 8192:], y2[:, 8192:]) and torch.equal(fin, fin2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at,width", [(0, 70), (1, 71), (33, 200), (64, 256)])
def test_slices_of_wider_rows(dtype, at, width):
    t = inputs(2, 130, 64 if at == 64 else 37, dtype, "logit", 12)
    D = t["x"].shape[2]
    want = ssd.gated_scan(t["x"], t["gate"], t["init"], complement=True, want_states=True)
    both = torch.full((2, 130, width + D), float("nan"), dtype=t["x"].dtype, device="cuda")
    both[..., at:at + D] = t["x"]
    wide = torch.full((2, 130, width), float("nan"), dtype=t["x"].dtype, device="cuda")
    wide[..., width - D:] = t["gate"]
    s = dict(t, x=both[..., at:at + D], gate=wide[..., width - D:])
    states = check_forward(s, dtype, "logit", True)
    check_backward(s, states, dtype, "logit", True)
    got = ssd.gated_scan(s["x"], s["gate"], t["init"], complement=True, want_states=True)
    close(got[2], host(want[2]), 1e-6, "f32")


def test_every_other_row():
    # a batch is 65 rows of 74 values on: what a row stride can say
    t = inputs(2, 130, 37, "f32", "logit", 21)
    s = dict(t, x=t["x"][:, ::2], gate=t["gate"][:, 1::2], dy=t["dy"][:, ::2].contiguous())
    assert not s["x"].is_contiguous()
    check_backward(s, check_forward(s, "f32", "logit", True), "f32", "logit", True)


def test_offsets_beyond_32_bits():
    # rows of 16384 elements, 150000 of them: the last rows start beyond 2^31 elements
    D, L, W = 40, 150000, 16384
    wide = torch.empty((1, L, W), dtype=torch.bfloat16, device="cuda")
    gate = wide[..., W - D:]
    t = inputs(1, L, D, "bf16", "log", 13)
    gate.copy_(t["gate"])
    want = ssd.gated_scan(t["x"], t["gate"], t["init"], kind="log", want_states=True)
    got = ssd.gated_scan(t["x"], gate, t["init"], kind="log", want_states=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    want = ssd.gated_scan_bwd(t["x"], t["gate"], t["dy"], want[2], kind="log")
    got = ssd.gated_scan_bwd(t["x"], gate, t["dy"], got[2], kind="log")
    assert all(torch.equal(want[k], got[k]) for k in want)


def test_split_and_resume():
    t = inputs(2, 700, 96, "f32", "logit", 14)
    h, _, tol = reference(t, "logit", True)
    k = 301
    y1, f1 = ssd.gated_scan(t["x"][:, :k].contiguous(), t["gate"][:, :k].contiguous(), t["init"], complement=True)
    y2, f2 = ssd.gated_scan(t["x"][:, k:].contiguous(), t["gate"][:, k:].contiguous(), f1, complement=True)
    close(torch.cat([y1, y2], 1), h, tol, "f32")
    close(f2, h[:, -1], tol[:, -1], "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,L,D", [(1, 1, 1), (1, 1, 1536), (64, 1, 5120), (3, 5, 33), (2, 70, 130)])
def test_decode(dtype, b, L, D):
    t = inputs(b, L, D, dtype, "logit", 15 + D)
    h, _, tol = reference(t, "logit", True)
    new = torch.empty_like(t["init"])
    was = t["init"].clone()
    y = ssd.gated_decode(t["x"], t["gate"], t["init"], complement=True, new_state=new)
    torch.cuda.synchronize()
    close(y, h, tol, dtype)
    close(new, h[:, -1], tol[:, -1], "f32")
    assert torch.equal(was, t["init"])
    y2 = ssd.gated_decode(t["x"], t["gate"], t["init"], complement=True)   # in place
    assert torch.equal(y, y2) and torch.equal(new, t["init"])


def test_the_same_call_gives_the_same_bits():
    t = inputs(3, 4000, 200, "bf16", "log", 16)
    one = ssd.gated_scan(t["x"], t["gate"], t["init"], kind="log", want_states=True)
    g1 = ssd.gated_scan_bwd(t["x"], t["gate"], t["dy"], one[2], t["dfinal"], kind="log")
    for _ in range(3):
        two = ssd.gated_scan(t["x"], t["gate"], t["init"], kind="log", want_states=True)
        g2 = ssd.gated_scan_bwd(t["x"], t["gate"], t["dy"], two[2], t["dfinal"], kind="log")
        assert all(torch.equal(a, b) for a, b in zip(one, two)) and all(torch.equal(g1[k], g2[k]) for k in g1)


def test_another_stream():
    t = inputs(2, 600, 128, "bf16", "logit", 17)
    want = ssd.gated_scan(t["x"], t["gate"], t["init"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = ssd.gated_scan(t["x"], t["gate"], t["init"], stream=s)
    s.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_captured_in_a_graph():
    t = inputs(8, 1, 256, "bf16", "logit", 18)
    state = t["init"].clone()
    y = torch.empty_like(t["x"])
    ssd.gated_decode(t["x"], t["gate"], state.clone(), y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.gated_decode(t["x"], t["gate"], state, y=y)
    want = t["init"].clone()
    for _ in range(3):
        graph.replay()
        ssd.gated_decode(t["x"], t["gate"], want)
    assert torch.equal(state, want)


def test_gradient_by_differences():
    # the directional derivative of the float64 forward pass, by central differences, against the kernel's gradients
    t = inputs(2, 150, 34, "f32", "logit", 19)
    _, _, states = ssd.gated_scan(t["x"], t["gate"], t["init"], complement=True, want_states=True)
    d = ssd.gated_scan_bwd(t["x"], t["gate"], t["dy"], states, t["dfinal"], complement=True)
    x, gate, init, dy, df = (host(t[k]) for k in ("x", "gate", "init", "dy", "dfinal"))
    r = np.random.default_rng(0)
    sx, sg, si = (r.normal(size=v.shape) for v in (x, gate, init))

    def loss(e):
        h, _ = gated.scan(x + e * sx, gate + e * sg, init + e * si, "logit", True)
        return (h * dy).sum() + (h[:, -1] * df).sum()

    num = (loss(1e-5) - loss(-1e-5)) / 2e-5
    terms = [host(d["dx"]) * sx, host(d["dgate"]) * sg, host(d["dinit"]) * si]
    scale = sum(np.abs(v).sum() for v in terms)
    assert abs(num - sum(v.sum() for v in terms)) <= scale * (64 * E + 1e-8)


def test_refusals():
    t = inputs(2, 10, 32, "bf16", "logit", 20)
    x, gate, init = t["x"], t["gate"], t["init"]
    with pytest.raises(ValueError):
        ssd.gated_scan(x, gate, init, kind="tanh")
    with pytest.raises(TypeError):
        ssd.gated_scan(x.half(), gate.half())
    with pytest.raises(TypeError):
        ssd.gated_scan(x, gate.float())
    with pytest.raises(ValueError):
        ssd.gated_scan(x, gate[:, :9])
    with pytest.raises(ValueError):
        ssd.gated_scan(x.transpose(1, 2).contiguous().transpose(1, 2), gate)
    with pytest.raises(ValueError):
        ssd.gated_scan(x[:, :6:2], gate[:, :3].contiguous())     # a batch is not its rows on
    with pytest.raises(ValueError):
        ssd.gated_scan(x, gate, init[:1])
    with pytest.raises(ValueError):
        ssd.gated_scan(x.cpu(), gate)
    with pytest.raises(ValueError):
        ssd.gated_scan_bwd(x, gate, t["dy"], torch.empty(2, 2, 32, device="cuda"))
    with pytest.raises(ssd.SSDError):
        ssd.gated_scan(x[:, :0].contiguous(), gate[:, :0].contiguous())
