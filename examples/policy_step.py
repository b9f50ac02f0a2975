"""Training steps of a small policy model on the library's operators.

A decoder (embedding, blocks of causal attention and a two-layer FFN, a head)
whose forward and backward passes are the framework's own: layer norm with the
residual sum and dropout in the same pass, attention with grouped heads, the
clipped policy loss on the logits, and bf16 products (opt_gemm_bf16) between
them. The weight gradients land in the G tensors of a RotatedAdamGroup, which
updates the matrices; norm weights and biases take plain gradient steps.

The task: at every position the model acts with one token and is rewarded for
naming the one that follows the token it sees, modulo the vocabulary.

    python -m examples.policy_step --steps 100
"""

from __future__ import annotations

import argparse
import sys

import torch

import matrix_optimizer_step_02_amd as mo
from matrix_optimizer_step_02_amd import train


def product(a, b, out=None, dtype=torch.bfloat16):
    """a (M x K) times b^T for b (N x K), both bf16 and contiguous, K a multiple of 8."""
    m, k = a.shape
    n = b.shape[0]
    c = torch.empty(m, n, device=a.device, dtype=dtype) if out is None else out
    mo.native.opt_gemm_bf16(m, n, k, 1.0, a.data_ptr(), k, b.data_ptr(), k, 0.0, c.data_ptr(),
                            int(c.dtype == torch.bfloat16), n, mo.stream_ptr())
    return c


def transposed(x):
    return x.t().contiguous()


class Norm:
    """Layer norm of residual + dropout(x); the residual stream is fp32."""

    def __init__(self, cols, device):
        self.weight, self.bias = torch.ones(cols, device=device), torch.zeros(cols, device=device)

    def forward(self, x, residual, p, rng):
        self.p, self.rng = p, rng
        y, self.h, self.mean, self.rstd = train.layer_norm_forward(x, self.weight, self.bias, residual=residual, p=p,
                                                                   rng=rng)
        return y, self.h

    def backward(self, dy, dh):
        """(gradient of x, gradient of the residual)."""
        dx, dres, self.dweight, self.dbias = train.layer_norm_backward(
            dy, self.h, self.weight, self.mean, self.rstd, dh=dh, p=self.p, rng=self.rng)
        return dx, dres

    def update(self, lr):
        self.weight.add_(self.dweight, alpha=-lr)
        self.bias.add_(self.dbias, alpha=-lr)


class Policy:
    def __init__(self, vocab=64, hidden=128, heads=4, kv_heads=2, ffn=256, layers=2, dropout=0.05, device="cuda",
                 seed=0):
        self.heads, self.kv, self.dim, self.p, self.seed = heads, kv_heads, hidden // heads, dropout, seed
        g = torch.Generator(device=device).manual_seed(seed)
        wide = (heads + 2 * kv_heads) * self.dim
        shapes = {"embed": (vocab, hidden), "head": (hidden, vocab)}
        for n in range(layers):
            shapes |= {f"qkv{n}": (hidden, wide), f"o{n}": (hidden, hidden), f"up{n}": (hidden, ffn),
                       f"down{n}": (ffn, hidden)}
        self.state = {}
        for name, (m, n) in shapes.items():
            w = torch.randn(m, n, generator=g, device=device) * (1.0 if name == "embed" else m ** -0.5)
            self.state[name] = mo.new_state(m, n, device=device, W0=w)
        self.norms = [(Norm(hidden, device), Norm(hidden, device)) for _ in range(layers)]
        self.last = Norm(hidden, device)
        self.passes = 0

    def matrices(self):
        return list(self.state.values())

    def rng(self, layer, site):
        """One offset per pass and place, so that no two masks agree."""
        return train.Rng(self.seed, (self.passes << 16) + 2 * layer + site)

    def weight(self, name):
        return self.state[name]["W"].bfloat16()

    def linear(self, name, x):
        self.saved[name] = x
        return product(x, transposed(self.weight(name)))

    def linear_backward(self, name, dy):
        product(transposed(self.saved[name]), transposed(dy), out=self.state[name]["G"])
        return product(dy, self.weight(name))

    def forward(self, tokens, p=None):
        """Logits (batch * length, vocab) of int64 tokens (batch, length)."""
        p = self.p if p is None else p
        self.passes += 1
        self.saved, self.tokens = {}, tokens
        b, t = tokens.shape
        h = self.state["embed"]["W"][tokens.reshape(-1)]
        x = torch.zeros_like(h, dtype=torch.bfloat16)   # nothing to add to the embedding yet
        for n, (before_attn, before_ffn) in enumerate(self.norms):
            y, h = before_attn.forward(x, h, p, self.rng(n, 0))
            q, k, v = self.linear(f"qkv{n}", y).view(b, t, -1, self.dim).split([self.heads, self.kv, self.kv], dim=2)
            out, lse = train.attention_forward(q, k, v, causal=True)
            self.saved[f"attn{n}"] = q, k, v, out, lse
            y, h = before_ffn.forward(self.linear(f"o{n}", out.view(b * t, -1)), h, p, self.rng(n, 1))
            x = self.linear(f"down{n}", self.linear(f"up{n}", y).relu_())
        y, _ = self.last.forward(x, h, p, self.rng(len(self.norms), 0))
        return self.linear("head", y)

    def backward(self, dlogits):
        """Writes every matrix's G and the norms' gradients."""
        dx, dh = self.last.backward(self.linear_backward("head", dlogits), None)
        for n in range(len(self.norms) - 1, -1, -1):
            before_attn, before_ffn = self.norms[n]
            d = self.linear_backward(f"down{n}", dx)
            d = d.masked_fill_(self.saved[f"down{n}"] <= 0, 0.0)
            dx, dh = before_ffn.backward(self.linear_backward(f"up{n}", d), dh)
            q, k, v, out, lse = self.saved[f"attn{n}"]
            dout = self.linear_backward(f"o{n}", dx).view(out.shape)
            dqkv = torch.empty(*q.shape[:2], self.heads + 2 * self.kv, self.dim, dtype=q.dtype, device=q.device)
            dq, dk, dv = dqkv.split([self.heads, self.kv, self.kv], dim=2)
            train.attention_backward(dout, q, k, v, out, lse, causal=True, dq=dq, dk=dk, dv=dv)
            dx, dh = before_attn.backward(self.linear_backward(f"qkv{n}", dqkv.view(dx.shape[0], -1)), dh)
        self.state["embed"]["G"].zero_().index_add_(0, self.tokens.reshape(-1), dh)

    def update_norms(self, lr):
        for norm in [n for pair in self.norms for n in pair] + [self.last]:
            norm.update(lr)


def train_policy(steps=100, batch=32, length=32, lr=1e-3, seed=0, log=print, **sizes):
    """Mean reward of each step."""
    torch.manual_seed(seed)
    model = Policy(seed=seed, **sizes)
    vocab = model.state["embed"]["W"].shape[0]
    group = mo.RotatedAdamGroup(model.matrices(), mo.Hyper(lr=lr, K=10, eps=1e-6))
    rewards = []
    for step in range(steps):
        tokens = torch.randint(0, vocab, (batch, length), device="cuda")
        with torch.no_grad():   # the sampling policy acts, without dropout
            logits = model.forward(tokens, p=0.0)
            action = torch.multinomial(logits.float().softmax(-1), 1).view(-1)
        reward = (action.view(batch, length) == (tokens + 1) % vocab).float()
        weight = (tokens > 0).float()   # token 0 is padding: its positions take no part in the loss
        weight /= weight.sum()
        rewards.append(float((reward * weight).sum()))
        advantage = (reward - rewards[-1]).view(-1) / max(rewards[-1] * (1 - rewards[-1]), 1e-2) ** 0.5
        scored = train.policy_loss_forward(logits, action, torch.zeros_like(advantage), advantage, weight.view(-1))
        logits = model.forward(tokens)
        loss, logp, dlogits = train.policy_loss_step(logits, action, scored.logp, advantage, weight.view(-1),
                                                     ref_logp=scored.logp, kl_coef=0.01, out=logits)
        model.backward(dlogits)
        group.step()
        model.update_norms(lr)
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:4d}  loss {float(loss):+.4f}  reward {rewards[-1]:.3f}")
    torch.cuda.synchronize()
    group.close()
    return rewards


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--length", type=int, default=32)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args(argv)
    rewards = train_policy(a.steps, a.batch, a.length, seed=a.seed, vocab=16)
    print(f"mean reward: first step {rewards[0]:.3f}, last 10 steps {sum(rewards[-10:]) / 10:.3f}")
    return 0


if __name__ == "__main__":
    sys.exit(main())
