"""A small network with a tropical layer, trained with the package's operators.

Next-token prediction on a synthetic chain: token embeddings (float32) go
through a max-plus layer (``TropicalGemm``: h[i, j] = max_k e[i, k] + A[k, j],
its gradient routed through the argmax), a layer norm that hands bfloat16 on,
and a linear head whose cross entropy never forms the logits.  Two AdamW
optimisers step the parameters, one for the float32 gradients and one for the
head's bfloat16 ones; the head's float32 master weights leave their bfloat16
copy, which the next forward pass reads, in the same pass.

    python -m einsum_device_side_gb300.tropical_net
"""

from __future__ import annotations

import torch

import einsum_device_side_gb300 as trop


class TropicalNet:
    def __init__(self, vocab: int = 512, dim: int = 64, hidden: int = 128, device="cuda", seed: int = 0,
                 state_bits: int = 8, lr: float = 3e-3):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        normal = lambda *shape: torch.randn(*shape, generator=gen, device=device)  # noqa: E731
        self.embed, self.layer = normal(vocab, dim), 0.5 * normal(dim, hidden)
        self.weight, self.bias = torch.ones(hidden, device=device), torch.zeros(hidden, device=device)
        self.head = 0.1 * normal(vocab, hidden)
        self.head16 = self.head.to(torch.bfloat16)
        # float32 parameters with float32 gradients; the head's gradient comes in bfloat16
        wide = [self.embed, self.layer, self.weight, self.bias]
        self.grads = [torch.zeros_like(p) for p in wide]
        self.head_grad = torch.zeros_like(self.head16)
        self.optimizers = [trop.AdamW(wide, self.grads, lr=lr, state_bits=state_bits),
                           trop.AdamW([self.head], [self.head_grad], lr=lr, state_bits=state_bits, copies=[self.head16])]

    def loss(self, tokens, targets):
        """The mean loss, and what the backward pass reads."""
        e = self.embed[tokens]
        h, route = trop.gemm(e, self.layer)
        y, mean, rstd = trop.layer_norm(h[0], self.weight, self.bias, out_dtype=torch.bfloat16)
        loss, lse, kept = trop.linear_cross_entropy(y, self.head16, targets)
        return loss, (tokens, targets, e, h, route, y, mean, rstd, lse, kept)

    def step(self, tokens, targets):
        """One training step; returns the loss (on the device)."""
        loss, (tokens, targets, e, h, route, y, mean, rstd, lse, kept) = self.loss(tokens, targets)
        one = torch.ones((), device=loss.device)
        dy, dhead = trop.linear_cross_entropy_backward(one, y, self.head16, targets, lse, kept)
        dh, dw, db = trop.layer_norm_backward(dy, h[0], mean, rstd, self.weight)
        de, da = trop.gemm_backward(e, self.layer, dh[None], route)
        self.grads[0].zero_().index_add_(0, tokens, de[0])
        for to, g in zip(self.grads[1:] + [self.head_grad], (da[0], dw, db, dhead)):
            to.copy_(g)
        for o in self.optimizers:
            o.step()
        return loss


def batch(gen, n: int, vocab: int, device="cuda"):
    """Tokens and their successors: i -> (5 i + 3) mod vocab, one in ten of them left out."""
    tokens = torch.randint(0, vocab, (n,), generator=gen, device=device)
    targets = (5 * tokens + 3) % vocab
    targets[torch.rand(n, generator=gen, device=device) < 0.1] = -100
    return tokens, targets


def train(steps: int = 100, tokens: int = 2048, vocab: int = 512, seed: int = 0, state_bits: int = 8):
    """Trains a net and returns the losses of its steps."""
    net = TropicalNet(vocab, seed=seed, state_bits=state_bits)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)
    return torch.stack([net.step(*batch(gen, tokens, vocab)) for _ in range(steps)]).tolist()


if __name__ == "__main__":
    for bits in (32, 8):
        losses = train(state_bits=bits)
        print(f"{bits}-bit states: loss {losses[0]:.3f} -> {losses[-1]:.3f} over {len(losses)} steps")
