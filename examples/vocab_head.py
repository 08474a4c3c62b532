"""Train a small language-model head with the library's own products: hidden states are a GEMM of the
inputs, the head's loss is cross entropy plus distillation from a teacher's top logits, and the gradient
goes back through the head into the GEMM's weights.  The T x V logits are not kept.

    python examples/vocab_head.py [--steps 30] [--dtype f32|bf16] [--tokens 512] [--vocab 4000] [--hidden 256]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp32_gemm_05_amd as sg  # noqa: E402


def train(steps=30, dtype="f32", tokens=512, vocab=4000, hidden=256, features=128, entries=8, rate=4.0, seed=0, say=print):
    """Returns the mean loss of each step."""
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)
    inputs = torch.randn(tokens, features, generator=g, device="cuda")
    target = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    target[::7] = -100  # every seventh token does not count
    # a teacher that gives its top entries, the target first
    index = torch.randint(0, vocab, (tokens, entries), generator=g, device="cuda")
    index[:, 0] = target.clamp(min=0)
    index[target < 0] = -1
    teacher = torch.randn(tokens, entries, generator=g, device="cuda")
    teacher[:, 0] += 3
    A = (torch.randn(features, hidden, generator=g, device="cuda") / features ** 0.5)
    W = (torch.randn(vocab, hidden, generator=g, device="cuda") / hidden ** 0.5).to(t).requires_grad_()
    weight = torch.full((tokens,), 1.0 / int((target >= 0).sum()), device="cuda")
    losses = []
    for step in range(steps):
        X = sg.gemm(inputs, A, torch.empty(tokens, hidden, device="cuda"))
        head_in = X.to(t).requires_grad_()
        loss = (0.7 * sg.vocab_cross_entropy(head_in, W, target)
                + 0.3 * sg.vocab_distillation(head_in, W, index, teacher, alpha=0.5, teacher_alpha=0.5))
        total = (loss * weight).sum()
        total.backward()
        dA = sg.gemm(inputs, head_in.grad.float(), torch.empty_like(A), trans_a=True)
        with torch.no_grad():
            A -= rate * dA
            W -= rate * W.grad
            W.grad = None
        losses.append(total.detach())
    losses = [float(x) for x in losses]
    for step in range(0, steps, max(1, steps // 10)):
        say(f"step {step:4d}  loss {losses[step]:.4f}")
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=30)
    p.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--vocab", type=int, default=4000)
    p.add_argument("--hidden", type=int, default=256)
    a = p.parse_args()
    train(a.steps, a.dtype, a.tokens, a.vocab, a.hidden)
