"""The gated mixer of examples/: the recurrence and the norm together, trained and served."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_model_02_gb300 import build as cuda_build

    cuda_build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import gated_mixer

    return gated_mixer


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_trains_and_serves(example, dtype):
    # one batch over and over: its loss has to fall (of different ones each has a variance of its own)
    mixer, losses = example.train(steps=40, dim=32, heads=2, length=150, size=8, dtype=dtype, batches=1)
    assert losses[-1] < losses[0]
    tokens, _ = example.batch(3, 97, dtype, 5)
    with torch.no_grad():
        whole, final = mixer(tokens)
    served, state = example.serve(mixer, tokens)
    # the matrix products of a whole sequence and of one token may round their bf16 results differently: a unit of the
    # projection's last place (2^-8), carried through the recurrence and the norm
    tol = 2.0 ** -4 if dtype == torch.bfloat16 else 1e-4
    scale = float(whole.abs().max())
    assert float((whole - served).abs().max()) <= tol * scale
    assert float((final - state).abs().max()) <= tol * float(final.abs().max())


def test_gradients_against_the_plain_form(example):
    torch.manual_seed(3)
    mixer = example.GatedMixer(3, 24, 3, torch.float32)
    tokens, want = example.batch(2, 45, torch.float32, 11)
    got, _ = mixer(tokens)
    (got - want).square().mean().backward()
    kernel = {n: p.grad.clone() for n, p in mixer.named_parameters()}

    mixer.zero_grad()
    p = mixer.in_proj(tokens).double()
    x, gate, z = p.split(mixer.dim, 2)
    a, h, hs = torch.sigmoid(gate), torch.zeros(2, mixer.dim, device="cuda", dtype=torch.float64), []
    for t in range(45):
        h = a[:, t] * h + (1 - a[:, t]) * x[:, t]
        hs.append(h)
    v = torch.stack(hs, 1).view(2, 45, mixer.heads, -1)
    v = (v - v.mean(3, keepdim=True)) / (v.var(3, unbiased=False, keepdim=True) + 1e-5).sqrt()
    y = (v.reshape(2, 45, mixer.dim) * mixer.weight + mixer.bias) * z * torch.sigmoid(z)
    plain = (y.float() @ mixer.out_proj.weight.t() + mixer.out_proj.bias)[..., 0]
    (plain - want).square().mean().backward()
    for n, q in mixer.named_parameters():
        scale = float(q.grad.abs().max())
        assert float((kernel[n] - q.grad).abs().max()) <= 2e-4 * scale, n
