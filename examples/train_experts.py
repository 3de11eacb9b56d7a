"""Trains a small stack of blocks of experts whose products run in 8 bits (`experts`):
the stacks of matrices by the matrix step (`okls`, Muon mode), routers and norm
weights by AdamW with 8-bit moments (`optim`), clipped by one norm of all gradients:

    python examples/train_experts.py [steps]

Each block norms the residual stream, lets a router choose each token's best
experts, sorts the tokens by them, multiplies by [gate; up] and down of each expert's
own, and adds the weighted rows back into the stream.  Inputs and targets are
synthetic: the targets come from a fixed random stack of the same form.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from kronecker_factored_second_amd import experts, okls, optim  # noqa: E402


def make(blocks, n_experts, d, f, gen, device):
    """[(norm weight, router, [gate; up] stack, down stack)] with fp32 master weights."""
    def w(*shape):
        return torch.randn(*shape, generator=gen, device=device) / shape[-1] ** 0.5
    return [(torch.ones(d, device=device), w(n_experts, d), w(n_experts, 2 * f, d), w(n_experts, d, f)) for _ in range(blocks)]


def forward(stack, x, each):
    """The stream after the last block, for x (tokens, d) in fp32."""
    for norm, router, gate_up, down in stack:
        h = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * norm
        best, choice = (h @ router.T).topk(each)
        order = experts.plan(choice, router.shape[0])
        gate, up = experts.token_linear(h.bfloat16(), gate_up, order, grad_dtype=torch.float8_e5m2).chunk(2, dim=1)
        y = experts.linear(torch.nn.functional.silu(gate) * up, down, order, grad_dtype=torch.float8_e5m2)
        x = x + experts.combine(y, best.softmax(1), order).float()
    return x


def train(steps=30, blocks=2, n_experts=8, each=2, d=256, f=256, tokens=1024, seed=0, lr=0.05, device="cuda"):
    """The loss of every step."""
    gen = torch.Generator(device=device).manual_seed(seed)
    teacher, stack = make(blocks, n_experts, d, f, gen, device), make(blocks, n_experts, d, f, gen, device)
    every = [[t.requires_grad_() for t in block] for block in stack]
    matrices = okls.OKLS([t for block in every for t in block[2:]], lr=lr, mode="muon")
    rest = optim.AdamW([t for block in every for t in block[:2]], lr=1e-2, weight_decay=0.0, moments="8bit")
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, d, generator=gen, device=device)
        with torch.no_grad():
            target = forward(teacher, x, each)
        loss = (forward(stack, x, each) - target).square().mean()
        loss.backward()
        norm = optim.grad_norm([t.grad for block in every for t in block])
        with torch.no_grad():
            matrices.step()
        rest.step(norm=norm, max_norm=1.0)
        matrices.zero_grad()
        rest.zero_grad()
        losses.append(loss.item())
    return losses


if __name__ == "__main__":
    for step, loss in enumerate(train(int(sys.argv[1]) if len(sys.argv) > 1 else 30)):
        print(f"step {step:3d}  loss {loss:.5f}")
