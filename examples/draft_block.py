"""A draft block for the verify step: trained in 16 bits, served in 8.

    python examples/draft_block.py [--rows 1024] [--vocab 32768] [--hidden 1024] [--steps 30]

From the model's last hidden state and the embedding of the token it emitted, one
residual block proposes the hidden state of the next position, h' = g + W2 silu(W1
norm(x + h) + b1), and the frozen 4-bit head turns it into the draft's token.  The
block is trained by distillation against a teacher's top logits with its gradients
clipped; then it drafts for a batch of verify windows with e4m3 weights and
activations, and the target's verify step accepts what matches.  Synthetic data;
prints the loss, and how far the 8-bit block's hidden states are from the 16-bit one's.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tied_distill import make_teacher  # noqa: E402
from verify_vocab_blocked_gb300 import qhead, synth  # noqa: E402
from verify_vocab_blocked_gb300.autograd import add_norm, head_distill, linear  # noqa: E402


def quantize_rows(w):
    """(codes float8_e4m3fn, scale float32) of a weight's rows, laid out once."""
    scale = w.float().abs().amax(1).clamp_min(1e-30) / 448.0
    return (w.float() / scale[:, None]).to(torch.float8_e4m3fn), scale


class Block:
    def __init__(self, H, inner, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        w = lambda n, k: (torch.randn(n, k, device=device, generator=g) / k ** 0.5).to(torch.bfloat16)  # noqa: E731
        self.up = w(inner, H).requires_grad_(True)
        self.up_bias = torch.zeros(inner, device=device, requires_grad=True)
        self.down = (0.1 * w(H, inner)).requires_grad_(True)
        self.gain = torch.ones(H, device=device, requires_grad=True)

    def parameters(self):
        return [self.up, self.up_bias, self.down, self.gain]

    def __call__(self, x, h):
        """The next position's hidden state, from the token's embedding x and the last h."""
        y, total = add_norm(x, h, self.gain, center=False)
        return linear(linear(y, self.up, self.up_bias, "silu"), self.down, residual=total)

    def quantize(self):
        """Call after training: the weights that serve()d rows go through."""
        self.up8, self.up_scale = quantize_rows(self.up.detach())
        self.down8, self.down_scale = quantize_rows(self.down.detach())

    def serve(self, x, h):
        """The same with 8-bit operands (the inner activations requantized by rows)."""
        codes, scale, total = qhead.norm_8bit(x, self.gain.detach(), residual=h, center=False)
        inner = qhead.linear(codes, self.up8, self.up_bias.detach(), "silu", x_scale=scale, w_scale=self.up_scale)
        codes, scale = quantize_rows(inner)
        return qhead.linear(codes, self.down8, None, "none", total, x_scale=scale, w_scale=self.down_scale)


def make_data(M, V, H, K, seed=0, device="cuda"):
    hd = synth.make_head(V, H, 4, softcap=30.0, seed=seed)
    head = qhead.Head.from_numpy(hd.wq, hd.scales, hd.biases, 4, softcap=30.0, device=device)
    g = torch.Generator(device=device).manual_seed(seed)
    x = qhead.embed(head, torch.randint(0, V, (M,), device=device, generator=g).int(), H ** 0.5)
    h = torch.randn(M, H, device=device, generator=g).to(torch.bfloat16)
    return head, x, h, *make_teacher(M, V, K, seed + 1, device)


def train_step(block, head, x, h, ids, teacher, max_norm=1.0):
    """The mean loss and the gradient norm; clipped gradients in the parameters' .grad."""
    loss = head_distill(block(x, h), head, ids, teacher).mean()
    loss.backward()
    norm = qhead.clip_grads([p.grad for p in block.parameters()], max_norm)
    return loss.detach(), norm


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32768)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--top", type=int, default=32)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    block = Block(a.hidden, 4 * a.hidden)
    head, x, h, ids, teacher = make_data(a.rows, a.vocab, a.hidden, a.top)
    opt = torch.optim.Adam(block.parameters(), lr=2e-3)
    for i in range(a.steps):
        opt.zero_grad(set_to_none=True)
        loss, norm = train_step(block, head, x, h, ids, teacher)
        opt.step()
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i:3d}  loss {loss.item():.4f}  gradient norm {norm.item():.4e}")
    block.quantize()
    with torch.no_grad():
        exact, served = block(x, h), block.serve(x, h)
        far = ((served - exact).float().norm() / exact.float().norm()).item()
        # windows of 4 drafted tokens and one more row each, the 16-bit block as the target
        B, W = a.rows // 5, 5
        draft = qhead.fwd(head, served[:B * W], want_lse=False)[2].view(B, W)[:, :W - 1].contiguous()
        accepted = qhead.verify(head, exact[:B * W], W, draft)[0]
    print(f"8-bit hidden states off by {far:.3%}; {accepted.float().mean().item():.2f} of {W - 1} drafted tokens accepted")


if __name__ == "__main__":
    main()
