"""Trains a small stack of gated MLP blocks whose linear layers run in 8 bits
(`linear`) and whose matrices the optimizer step updates (`okls`, Muon mode):

    python examples/train_8bit_mlp.py [steps]

Each block norms the residual stream into 8 bits, multiplies by [gate; up] in one
product, and brings the gated values back through `down`; the stream's addition
is the next block's norm's first half.  Inputs and targets are synthetic: the
targets come from a fixed random stack of the same form.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from kronecker_factored_second_amd import linear, okls  # noqa: E402


def make(blocks, d, f, gen, device):
    """[(norm weight, [gate; up], down)] with fp32 master weights."""
    def w(rows, cols):
        return torch.randn(rows, cols, generator=gen, device=device) / cols ** 0.5
    return [(torch.ones(d, device=device), w(2 * f, d), w(d, f)) for _ in range(blocks)]


def forward(stack, x):
    """The stream after the last block, for x (tokens, d) in bf16."""
    stream, delta = x, torch.zeros_like(x)
    for norm, gate_up, down in stack:
        y, stream = linear.rms_norm_linear(delta, norm, gate_up, residual=stream, grad_dtype=torch.float8_e5m2)
        gate, up = y.chunk(2, dim=1)
        delta = linear.scaled_linear(torch.nn.functional.silu(gate) * up, down, grad_dtype=torch.float8_e5m2)
    return stream + delta


def train(steps=30, blocks=2, d=256, f=512, tokens=512, seed=0, lr=0.1, device="cuda"):
    """The loss of every step."""
    gen = torch.Generator(device=device).manual_seed(seed)
    teacher, stack = make(blocks, d, f, gen, device), make(blocks, d, f, gen, device)
    matrices = [m.requires_grad_() for _, gate_up, down in stack for m in (gate_up, down)]
    norms = [norm.requires_grad_() for norm, _, _ in stack]
    muon, sgd = okls.OKLS(matrices, lr=lr, mode="muon"), torch.optim.SGD(norms, lr=1e-2)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, d, generator=gen, device=device).bfloat16()
        with torch.no_grad():
            target = forward(teacher, x).float()
        loss = (forward(stack, x).float() - target).square().mean()
        loss.backward()
        with torch.no_grad():
            muon.step()
        sgd.step()
        muon.zero_grad()
        sgd.zero_grad()
        losses.append(loss.item())
    return losses


if __name__ == "__main__":
    for step, loss in enumerate(train(int(sys.argv[1]) if len(sys.argv) > 1 else 30)):
        print(f"step {step:3d}  loss {loss:.5f}")
