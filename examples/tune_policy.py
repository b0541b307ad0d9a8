"""Tunes a small token policy, first by reward, then by preferences, with the
library's operators around its optimizer step.

The model reads one token and predicts the next: embedding -> layer norm ->
output matrix.  Each update runs

    loss.logps                       scores of the sampling and the reference policy
    norm.forward, matmul             logits
    loss.policy / loss.preference    loss and the logits' gradient
    matmul, norm.backward            gradients, written into the plan's grad buffers
    opt.grad_norm                    global norm, the scale that clips it, found-inf
    opt.step                         clipped AdamW step (skipped if a grad is not finite)

    python examples/tune_policy.py
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from adamw_optimizer_step_tensor_gb300 import FusedAdamW, FusedLayerNorm, FusedTokenLoss  # noqa: E402

VOCAB, WIDTH = 509, 64


class Policy:
    """Parameters, their grads and the optimizer's plan over both."""

    def __init__(self, seed: int, max_rows: int, max_pairs: int):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g) * 0.3  # noqa: E731
        self.emb, self.out = rand(VOCAB, WIDTH), rand(VOCAB, WIDTH)
        self.weight, self.bias = torch.ones(WIDTH, device="cuda"), torch.zeros(WIDTH, device="cuda")
        params = [self.emb, self.out, self.weight, self.bias]
        self.grads = [torch.zeros_like(p) for p in params]
        zeros = lambda: [torch.zeros_like(p) for p in params]  # noqa: E731
        self.opt = FusedAdamW(params, self.grads, zeros(), zeros(), [0.01, 0.01, 0.0, 0.0])
        self.lr = torch.tensor([0.01], device="cuda")
        self.steps = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.norm = FusedLayerNorm(WIDTH)
        self.loss = FusedTokenLoss(max_rows, max_pairs)
        self.grad_norm, self.clip_scale, self.found_inf = (torch.zeros(1, device="cuda") for _ in range(3))

    def logits(self, tokens):
        hidden = self.emb[tokens]
        y, mean, rstd = self.norm.forward(hidden, self.weight, self.bias)
        return y @ self.out.t(), (tokens, hidden, y, mean, rstd)

    def update(self, dlogits, saved, max_norm=1.0):
        tokens, hidden, y, mean, rstd = saved
        g_emb, g_out, g_weight, g_bias = self.grads
        torch.mm(dlogits.t(), y, out=g_out)
        dy = dlogits @ self.out
        dhidden, _, _ = self.norm.backward(dy, hidden, self.weight, mean, rstd, dx=dy, dweight=g_weight,
                                           dbias=g_bias)
        g_emb.zero_().index_add_(0, tokens, dhidden)
        self.opt.grad_norm(self.grad_norm, max_norm=max_norm, clip_scale=self.clip_scale,
                           found_inf=self.found_inf)
        self.opt.step(self.lr, self.steps, grad_scale=self.clip_scale, found_inf=self.found_inf)


def successor(tokens):
    """The token the reward asks for."""
    return (tokens * 7 + 3) % VOCAB


def tune_by_reward(policy, reference, rounds=40, rows=2048, epochs=2, seed=1):
    """Mean reward per round: 1 where the sampled token is one of 16 wanted ones."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    weights = torch.full((rows,), 1.0 / rows, device="cuda")
    history = []
    for _ in range(rounds):
        tokens = torch.randint(0, VOCAB, (rows,), device="cuda", generator=g)
        logits, _ = policy.logits(tokens)
        taken = torch.multinomial(torch.softmax(logits, 1), 1, generator=g)[:, 0]
        reward = ((taken - successor(tokens)) % VOCAB < 16).float()
        history.append(reward.mean())
        advantages = (reward - reward.mean()) / (reward.std() + 1e-4)
        old, _ = policy.loss.logps(logits, taken)
        ref, _ = policy.loss.logps(reference.logits(tokens)[0], taken)
        for _ in range(epochs):
            logits, saved = policy.logits(tokens)
            _, _, dlogits = policy.loss.policy(logits, taken, weights, advantages, old, ref, kl_coef=0.01,
                                               dlogits=logits)
            policy.update(dlogits, saved)
    return [float(r) for r in history]


def tune_by_preference(policy, reference, rounds=40, pairs=32, length=16, seed=2):
    """Share of pairs ahead per round: the chosen continuation follows `successor`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = 2 * pairs * length
    starts = torch.arange(0, rows + 1, length, dtype=torch.int32, device="cuda")
    history = []
    for _ in range(rounds):
        tokens = torch.randint(0, VOCAB, (rows,), device="cuda", generator=g)
        taken = successor(tokens)
        taken[rows // 2:] = torch.randint(0, VOCAB, (rows // 2,), device="cuda", generator=g)
        taken[::length] = -100                     # a sequence's first row is its prompt
        ref, _ = policy.loss.logps(reference.logits(tokens)[0], taken)
        logits, saved = policy.logits(tokens)
        stats, _, _, dlogits = policy.loss.preference(logits, taken, None, ref, starts, beta=0.1, dlogits=logits)
        policy.update(dlogits, saved)
        history.append(stats.clone())
    return [float(s[1]) for s in history], [float(s[0]) for s in history]


def main():
    make = lambda: Policy(0, 2048, 32)  # noqa: E731
    reference = make()
    policy = make()
    reward = tune_by_reward(policy, reference)
    print(f"reward      first rounds {sum(reward[:5]) / 5:.3f}  last rounds {sum(reward[-5:]) / 5:.3f}")
    policy = make()
    ahead, loss = tune_by_preference(policy, reference)
    print(f"preference  loss {loss[0]:.3f} -> {loss[-1]:.3f}  chosen ahead {ahead[1]:.2f} -> {ahead[-1]:.2f}")
    print(f"steps {int(policy.steps)}, last gradient norm {float(policy.grad_norm):.3f}, "
          f"clip scale {float(policy.clip_scale):.3f}")
    return reward, ahead, loss, policy


if __name__ == "__main__":
    main()
