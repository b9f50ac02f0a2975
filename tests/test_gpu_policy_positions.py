"""GPU tests of examples/policy_step.py with norms of queries and keys, position
rotation, a window with sinks, and AdamW: a run of these operators as a training
program makes it. The whole model's gradients are compared with automatic
differentiation of the same model in float64 on the CPU, from the same weights
rounded to bfloat16, with the units that the device's ReLU left open: one whose sum
lies within its rounding of zero opens in one and not in the other, and n of N such
units are sqrt(n / N) of a gradient's norm, 3 % at one in a thousand. Activations
are rounded 9 times a block (y, qkv, q and k turned, P, out, o, y, up, down), their
gradients as often, each by at most 2^-8 of what is rounded: 36 times in two
blocks, 2.3 % in norm if they are independent and 14 % if all added up: 5 %."""

import math

import pytest

from oracle import train_ops as T

pytestmark = pytest.mark.gpu


def reference(model, tokens, target, old, ref, adv, w, kl):
    """Loss and gradients in float64."""
    import torch
    W = {n: (s["W"] if n == "embed" else s["W"].bfloat16()).double().cpu().requires_grad_() for n, s in model.state.items()}
    nw = [n.weight.double().cpu().requires_grad_() for n in model.all_norms()]
    nb = [n.bias.double().cpu().requires_grad_() for n in model.all_norms()]
    qk = [[x.double().cpu().requires_grad_() for x in pair] for pair in model.qk]
    ln = lambda h, i: torch.nn.functional.layer_norm(h, h.shape[-1:], nw[i], nb[i], 1e-5)  # noqa: E731
    b, t = tokens.shape
    h = W["embed"][tokens.cpu()]
    see = torch.from_numpy(T.visible(t, t, True, model.mask["window"], model.mask["sinks"]))
    f = torch.tensor([10000.0 ** (-2 * i / model.dim) for i in range(model.dim // 2)], dtype=torch.float64)
    e = torch.polar(torch.ones(t, len(f), dtype=torch.float64), torch.arange(t)[:, None] * f)[None, :, None]

    def turned(x, weight):
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * weight
        z = torch.complex(*x.chunk(2, -1)) * e
        return torch.cat((z.real, z.imag), -1)

    for n in range(len(model.norms)):
        q, k, v = (ln(h, 2 * n) @ W[f"qkv{n}"]).view(b, t, -1, model.dim).split([model.heads, model.kv, model.kv], 2)
        q, k = turned(q, qk[n][0]), turned(k, qk[n][1])
        k, v = (x.repeat_interleave(model.heads // model.kv, 2) for x in (k, v))
        s = torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(model.dim)
        p = s.masked_fill(~see, -math.inf).softmax(-1)
        h = h + torch.einsum("bhij,bjhd->bihd", p, v).reshape(b, t, -1) @ W[f"o{n}"]
        open_ = (model.saved[f"down{n}"] > 0).double().cpu().view(b, t, -1)
        h = h + (ln(h, 2 * n + 1) @ W[f"up{n}"]) * open_ @ W[f"down{n}"]
    z = (ln(h, len(nw) - 1) @ W["head"]).view(b * t, -1)
    logp = z.log_softmax(-1).gather(1, target.cpu()[:, None])[:, 0]
    old, ref, adv, w = (x.double().cpu() for x in (old, ref, adv, w))
    r, d = (logp - old).exp(), ref - logp
    loss = (w * (torch.maximum(-adv * r, -adv * r.clip(0.8, 1.2)) + kl * (d.exp() - d - 1))).sum()
    loss.backward()
    vectors = [g.grad for pair in zip(nw, nb) for g in pair] + [x.grad for pair in qk for x in pair]
    return loss, {n: x.grad for n, x in W.items()}, vectors


def gradients():
    """A model after a forward and a backward pass, and what the pass was of."""
    import torch
    from examples import policy_step
    from matrix_optimizer_step_02_amd import train
    torch.manual_seed(0)
    model = policy_step.Policy(vocab=40, hidden=96, heads=6, kv_heads=2, ffn=200, layers=2, dropout=0.0, rotary=True,
                               window=11, sinks=3)
    for pair in model.qk:
        for w in pair:
            w.add_(0.2 * torch.randn(w.shape, device="cuda"))
    tokens = torch.randint(0, 40, (4, 30), device="cuda")
    n = tokens.numel()
    target = torch.randint(0, 40, (n,), device="cuda")
    logits = model.forward(tokens)
    logp = logits.double().log_softmax(-1).gather(1, target[:, None])[:, 0].float()
    # ratios away from the clip's borders by more than the activations' rounding
    old = logp - torch.tensor([0.0, 0.5, -0.5, 0.05], device="cuda").repeat(n // 4)
    ref, adv, w = logp + 0.2, torch.randn(n, device="cuda"), torch.rand(n, device="cuda") / n
    loss, _, dlogits = train.policy_loss_step(logits, target, old, adv, w, ref_logp=ref, kl_coef=0.1)
    model.backward(dlogits)
    torch.cuda.synchronize()
    return model, loss, (tokens, target, old, ref, adv, w, 0.1)


def test_gradients_of_the_whole_model():
    print("policy model with positions, gradients", flush=True)
    model, loss, given = gradients()
    want, grads, vectors = reference(model, *given)
    assert abs(float(loss) - want.item()) <= 0.05 * float(given[5].sum())
    near = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    off = {x: near(model.state[x]["G"], g) for x, g in grads.items()}
    off |= {f"vector{i}": near(a, b) for i, (a, b) in enumerate(zip(model.vector_grads(), vectors))}
    print({k: round(v, 4) for k, v in off.items()}, flush=True)
    assert max(off.values()) <= 0.05, off


def test_wrong_models_are_told_apart():
    """The reference without the rotation, the norms' weights, the window or its sinks is further off than the bound."""
    from examples import policy_step  # noqa: F401
    model, _, given = gradients()
    got = {n: s["G"].double().cpu() for n, s in model.state.items()}

    def off():
        _, grads, _ = reference(model, *given)
        return max(float((got[n] - g).norm() / g.norm()) for n, g in grads.items())

    assert off() <= 0.05
    for change in (dict(window=12), dict(sinks=2), dict(window=0, sinks=0)):
        was, model.mask = model.mask, model.mask | change
        assert off() > 0.05, change
        model.mask = was
    qk, model.qk = model.qk, [[w.flip(0) for w in pair] for pair in model.qk]
    assert off() > 0.05
    model.qk = qk


@pytest.mark.parametrize("bits", [32, 8])
def test_vectors_take_the_clipped_step(bits):
    """From zero moments the first step of AdamW is lr g / (|g| + eps') an element, whatever the clipping; eps' = 1e-8 over
    the clipping factor stays far below the gradients that are checked."""
    import torch
    from examples import policy_step
    model, _, _ = gradients()
    before = [v.clone() for v in model.vectors()]
    step = policy_step.Vectors(model, lr=0.01, max_norm=1e-3, bits=bits)
    step.step()
    torch.cuda.synchronize()
    norm = torch.stack([g.double().square().sum() for g in model.vector_grads()]).sum().sqrt()
    assert abs(float(step.group.grad_norm(1e-3).norm) / float(norm) - 1) < 1e-6
    scale = min(1.0, 1e-3 / (float(norm) + 1e-6))
    for v, b, g in zip(model.vectors(), before, model.vector_grads()):
        want = b.double() - 0.01 * g.double() / (g.double().abs() + 1e-8 / scale)
        assert float((v.double() - want).abs().max()) < 1e-5


@pytest.mark.parametrize("more", [dict(rotary=True), dict(rotary=True, window=8, sinks=2, adamw=True), dict(adamw=True)])
def test_the_example_runs(more):
    from examples import policy_step
    print("policy training", more, flush=True)
    rewards = policy_step.train_policy(steps=4, vocab=16, log=lambda s: print(s, flush=True), **more)
    assert len(rewards) == 4 and all(0 <= r <= 1 for r in rewards)
