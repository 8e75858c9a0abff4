"""A training step at both ends of a model with a tied quantized table.

    python examples/tied_distill.py [--rows 2048] [--vocab 32768] [--hidden 1024] [--steps 20]

Tokens are looked up in the packed 4-bit table, a small trainable block stands
for the model's body, the final norm makes the head's hidden states, and the
same table scores them against a teacher's top logits.  The backward runs the
distillation's gradient into h (the table as a head is frozen: that loss has no
gradient into it), the norm's and the lookup's, whose table gradient is added
into a float32 [V, H] buffer.  Synthetic data; prints the loss as the body learns.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from verify_vocab_blocked_gb300 import qhead, synth  # noqa: E402
from verify_vocab_blocked_gb300.autograd import embed, head_distill, layer_norm  # noqa: E402


def make_teacher(M, V, K, seed, device):
    """Top logits a text might have: each row a peak and a fall-off."""
    g = torch.Generator(device=device).manual_seed(seed)
    stride = V // K
    ids = torch.arange(K, device=device) * stride + torch.randint(0, stride, (M, K), device=device,
                                                                  generator=g)
    t = 12.0 - 1.2 * torch.log1p(torch.arange(K, device=device)) \
        + 0.3 * torch.randn(M, K, device=device, generator=g)
    return ids.int(), t


class Step:
    """What a training loop keeps: table, body, norm parameters, buffers."""

    def __init__(self, M, V, H, K, seed=0, device="cuda"):
        hd = synth.make_head(V, H, 4, softcap=30.0, seed=seed)
        self.head = qhead.Head.from_numpy(hd.wq, hd.scales, hd.biases, 4, softcap=30.0,
                                          device=device)
        g = torch.Generator(device=device).manual_seed(seed)
        self.tokens = torch.randint(0, V, (M,), device=device, generator=g).int()
        self.mask = torch.rand(M, device=device, generator=g) < 0.9
        self.ids, self.teacher = make_teacher(M, V, K, seed + 1, device)
        w = torch.randn(H, H, device=device, generator=g) / H ** 0.5
        self.body = w.to(torch.bfloat16).requires_grad_(True)
        self.gain = torch.ones(H, device=device, requires_grad=True)
        self.shift = torch.zeros(H, device=device, requires_grad=True)
        self.dw = torch.zeros(V, H, device=device)
        self.scale = H ** 0.5

    def __call__(self):
        """The mean loss; gradients in body, gain, shift (.grad) and dw."""
        self.dw.zero_()
        x = embed(self.head, self.tokens, self.scale, self.mask, dw=self.dw)
        h = layer_norm(x + x @ self.body, self.gain, self.shift)
        loss = head_distill(h, self.head, self.ids, self.teacher, 1.0, self.mask)
        mean = loss.sum() / self.mask.sum()
        mean.backward()
        return mean.detach()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=2048)
    ap.add_argument("--vocab", type=int, default=32768)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--top", type=int, default=32)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    step = Step(a.rows, a.vocab, a.hidden, a.top)
    opt = torch.optim.Adam([step.body, step.gain, step.shift], lr=2e-3)
    for i in range(a.steps):
        opt.zero_grad(set_to_none=True)
        loss = step()
        opt.step()
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i:3d}  loss {loss.item():.4f}  |dW| {step.dw.norm().item():.4e}")


if __name__ == "__main__":
    main()
