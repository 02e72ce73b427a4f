"""Policy-gradient steps of a small token model, with the library's operators at the
vocabulary-sized ends of the step.

    python examples/policy_step.py [--steps 40] [--vocab 2003] [--width 256]

The model is the smallest that has those ends: a token's embedding row, scaled,
times an output matrix gives the logits of the next token.  A step samples next
tokens, rewards those that follow a hidden rule, and then

    embedding            rows of the table for the tokens (and, in the backward pass,
                         the table's gradient by sorted tokens)
    token_stats          log-probabilities of the sampled tokens and entropies, with
                         their gradient with respect to the logits
    lse_grad_clip        the global norm of both gradients, clipped in place

At the end one token is decoded with its top alternatives (lse_token_stats), and a few more
are drawn with the output matrix held in 4 bits (lse_linear4, lse_sample).
"""
from __future__ import annotations

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import log_sum_exp_gb300 as L  # noqa: E402


class TokenModel:
    """logits = (sqrt(D) * table[ids]) @ out^T, in bfloat16 with float32 masters."""

    def __init__(self, vocab: int, width: int, seed: int = 0, device: str = "cuda",
                 dtype: torch.dtype = torch.bfloat16):
        g = torch.Generator(device=device).manual_seed(seed)
        self.master = [torch.randn((vocab, width), generator=g, device=device) * 0.02
                       for _ in range(2)]
        self.params = [m.to(dtype).requires_grad_() for m in self.master]
        self.scale = math.sqrt(width)
        for p in self.params:
            p.grad = torch.zeros_like(p)
        # The gradients keep their memory, so their list is laid out once.
        self.grads = L.GradList([p.grad for p in self.params])

    def logits(self, ids: torch.Tensor) -> torch.Tensor:
        table, out = self.params
        return L.embedding(ids, table, scale=self.scale) @ out.t()

    def update(self, lr: float, max_norm: float) -> torch.Tensor:
        """Clips the gradients, takes a step, zeroes them; returns the norm."""
        norm = L.lse_grad_clip(self.grads, max_norm)
        with torch.no_grad():
            for m, p in zip(self.master, self.params):
                m.add_(p.grad.float(), alpha=-lr)
                p.copy_(m)
                p.grad.zero_()
        return norm


def policy_loss(logits: torch.Tensor, actions: torch.Tensor, advantage: torch.Tensor,
                entropy_weight: float):
    """-mean(advantage * log p(action)) - entropy_weight * mean(entropy)."""
    s = L.token_stats(logits, actions)
    return -(advantage * s.logprob).mean() - entropy_weight * s.entropy.mean(), s


def train(steps: int = 40, vocab: int = 2003, width: int = 256, batch: int = 4096, lr: float = 3.0,
          max_norm: float = 1.0, entropy_weight: float = 0.002, seed: int = 0, quiet: bool = False):
    """Rewards next = (7 * token + 3) % 16 (half of the choices are the model's own, half
    are drawn from the 16); returns the mean reward of the model's own at every step."""
    model = TokenModel(vocab, width, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    rewards = []
    for step in range(steps):
        ids = torch.randint(0, 64, (batch,), generator=g, device="cuda")
        logits = model.logits(ids)
        with torch.no_grad():
            noise = torch.rand(logits.shape, generator=g, device="cuda").clamp_(1e-9).log_().neg_().log_()
            explore = torch.randint(0, 16, (batch,), generator=g, device="cuda")
            actions = torch.where(torch.arange(batch, device="cuda") % 2 == 0,
                                  (logits.float() - noise).argmax(1), explore)
            reward = (actions == (7 * ids + 3) % 16).float()
            advantage = reward * 16
        loss, s = policy_loss(logits, actions, advantage, entropy_weight)
        loss.backward()
        norm = model.update(lr, max_norm)
        rewards.append(float(reward[::2].mean()))  # of the model's own choices
        if not quiet and step % 4 == 0:
            print(f"step {step:3d}  reward {rewards[-1]:.3f}  loss {float(loss.detach()):+.4f}  "
                  f"entropy {float(s.entropy.detach().mean()):.3f}  gradient norm {float(norm):.4f}")
    return model, rewards


def decode(model: TokenModel, token: int, steps: int, seed: int = 0):
    """Tokens drawn one after the other, the output matrix held in 4 bits (lse_quantize4,
    lse_linear4, lse_sample)."""
    head = L.lse_quantize4(model.params[1].detach(), group=64)
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids, out = torch.tensor([token], device="cuda"), []
    for _ in range(steps):
        rows = L.lse_embedding(model.params[0].detach(), ids, scale=model.scale)
        logits = L.lse_linear4(rows, head, out_dtype=torch.float32)
        ids = L.lse_sample(logits, torch.rand(1, generator=g, device="cuda"), temperature=0.7, top_k=20).token
        out.append(int(ids))
    return out


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--vocab", type=int, default=2003)
    ap.add_argument("--width", type=int, default=256)
    a = ap.parse_args()
    model, rewards = train(a.steps, a.vocab, a.width)
    token = torch.tensor([5], device="cuda")
    with torch.no_grad():
        s = L.lse_token_stats(model.logits(token), top_k=3)
    top = ", ".join(f"{int(i)} ({math.exp(float(lp)):.2f})"
                    for i, lp in zip(s.top_index[0], s.top_logprob[0]))
    print(f"after token 5 (rule: {(7 * 5 + 3) % 16}): {top}")
    print("drawn from there with a 4-bit output matrix:", decode(model, 5, 8))


if __name__ == "__main__":
    main()
