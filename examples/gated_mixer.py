"""A gated recurrent mixer: the gated linear recurrence and the group norm, in training and in serving.

    in_proj -> (x, gate, z)     h = gated_scan(x, gate)     y = group_norm(h) * silu(z)     -> out_proj

The mixer is trained on a toy task (report the sum of the marked tokens so far, forgetting at each reset token), with the
gradients of the library's backward passes, and then serves the same sequence token by token from the recurrent
state; both must say the same.  Needs a GB300 and the built library.

    python examples/gated_mixer.py [--steps 60] [--dim 64] [--heads 4] [--length 256] [--dtype bf16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from state_space_model_02_gb300 import ssd  # noqa: E402


class Scan(torch.autograd.Function):
    """ssd.gated_scan with its gradient; x and gate may be slices of one projection."""

    @staticmethod
    def forward(ctx, x, gate, init):
        y, final, states = ssd.gated_scan(x, gate, init, kind="logit", complement=True, want_states=True)
        ctx.save_for_backward(x, gate, states)
        return y, final

    @staticmethod
    def backward(ctx, dy, dfinal):
        x, gate, states = ctx.saved_tensors
        d = ssd.gated_scan_bwd(x, gate, dy.contiguous(), states, dfinal.contiguous(), kind="logit", complement=True)
        return d["dx"], d["dgate"], d["dinit"]


class Norm(torch.autograd.Function):
    """ssd.group_norm of single tokens, gated behind the norm, with its gradient."""

    @staticmethod
    def forward(ctx, x, z, weight, bias, groups):
        y, mean, rstd = ssd.group_norm(x, weight, bias, groups=groups, z=z, act="gate", want_stats=True)
        ctx.save_for_backward(x, z, weight, bias, mean, rstd)
        ctx.groups = groups
        return y

    @staticmethod
    def backward(ctx, dy):
        x, z, weight, bias, mean, rstd = ctx.saved_tensors
        d = ssd.group_norm_bwd(x, dy.contiguous(), mean, rstd, weight, bias, groups=ctx.groups, z=z, act="gate")
        return d["dx"], d["dz"], d["dweight"], d["dbias"], None


class GatedMixer(torch.nn.Module):
    def __init__(self, features, dim, heads, dtype):
        super().__init__()
        self.dim, self.heads = dim, heads
        self.in_proj = torch.nn.Linear(features, 3 * dim, device="cuda", dtype=dtype)
        self.out_proj = torch.nn.Linear(dim, 1, device="cuda", dtype=dtype)
        self.weight = torch.nn.Parameter(torch.ones(dim, device="cuda"))
        self.bias = torch.nn.Parameter(torch.zeros(dim, device="cuda"))
        with torch.no_grad():  # half lives from a few tokens to some hundreds
            self.in_proj.bias[dim:2 * dim] = torch.linspace(1.0, 6.0, dim)

    def split(self, tokens):
        b, L, _ = tokens.shape
        p = self.in_proj(tokens)
        return p[..., :self.dim], p[..., self.dim:2 * self.dim], p[..., 2 * self.dim:].reshape(b * L, 1, self.dim)

    def forward(self, tokens):
        """(b, L, features) -> (b, L), and the state after the last token (b, dim)."""
        b, L, _ = tokens.shape
        x, gate, z = self.split(tokens)
        h, final = Scan.apply(x, gate, torch.zeros(b, self.dim, device="cuda"))
        y = Norm.apply(h.view(b * L, 1, self.dim), z, self.weight, self.bias, self.heads)
        return self.out_proj(y.view(b, L, self.dim))[..., 0], final

    @torch.no_grad()
    def step(self, token, state):
        """One token (b, 1, features) of each sequence; advances the state (b, dim) in place."""
        x, gate, z = self.split(token)
        h = ssd.gated_decode(x, gate, state, kind="logit", complement=True)
        y = ssd.group_norm(h.view(-1, 1, self.dim), self.weight, self.bias, groups=self.heads, z=z, act="gate")
        return self.out_proj(y.view(-1, 1, self.dim))[:, 0, 0]


def batch(b, L, dtype, seed):
    """Tokens (b, L, 3): a value, whether it counts, whether the sum starts anew; and the sums."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    value = torch.randn(b, L, generator=g, device="cuda")
    counts = (torch.rand(b, L, generator=g, device="cuda") < 0.3).float()
    reset = (torch.rand(b, L, generator=g, device="cuda") < 0.05).float()
    keep = torch.arange(L, device="cuda")
    start = torch.where(reset > 0, keep, 0).cummax(1).values
    sums = (value * counts).cumsum(1)
    before = (sums - value * counts).gather(1, start)
    return torch.stack([value, counts, reset], 2).to(dtype), sums - before


def train(steps=60, dim=64, heads=4, length=256, size=32, dtype=torch.bfloat16, seed=0, batches=None, log=None):
    """Returns the trained mixer and its losses; `batches`: how many different ones to take in turn (None: all new)."""
    torch.manual_seed(seed)
    mixer = GatedMixer(3, dim, heads, dtype)
    opt = torch.optim.Adam(mixer.parameters(), lr=2e-2)
    losses = []
    for i in range(steps):
        tokens, want = batch(size, length, dtype, 1000 + (i if batches is None else i % batches))
        got, _ = mixer(tokens)
        loss = (got.float() - want).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        if log and (i % 10 == 0 or i + 1 == steps):
            log("step %3d  loss %.4f" % (i, losses[-1]))
    return mixer, losses


@torch.no_grad()
def serve(mixer, tokens):
    """The outputs (b, L) of a sequence taken token by token, and the last state."""
    state = torch.zeros(tokens.shape[0], mixer.dim, device="cuda")
    return torch.stack([mixer.step(tokens[:, i:i + 1], state) for i in range(tokens.shape[1])], 1), state


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dim", type=int, default=64)
    ap.add_argument("--heads", type=int, default=4)
    ap.add_argument("--length", type=int, default=256)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args()
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[a.dtype]
    mixer, losses = train(a.steps, a.dim, a.heads, a.length, dtype=dtype, log=print)
    tokens, _ = batch(4, a.length, dtype, 7)
    with torch.no_grad():
        whole, final = mixer(tokens)
    served, state = serve(mixer, tokens)
    print("loss %.4f -> %.4f; whole sequence against token by token: outputs differ by %.2g of %.2g, states by %.2g" % (
        losses[0], losses[-1], float((whole - served).abs().max()), float(whole.abs().max()),
        float((final - state).abs().max())))


if __name__ == "__main__":
    main()
