"""Rollout and update of a policy head: final norm, LM head, sampling, scoring, loss.

Rollout: the hidden state of each sequence's last token goes through the final norm and the LM
head, and a token is drawn from its logits; one such step is captured in a CUDA graph and
replayed.  Update: the drawn tokens are scored again from the hidden states with the fused
log-prob, compared with the logp of the draw (the consistency audit), and the clipped-ratio
loss goes back through the head and the norm.

    python examples/policy_step.py [--norm layer] [--steps 4] [--rows 256] ...
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))

import rl_post_linear_gb300 as rlk                                            # noqa: E402


class PolicyHead:
    """The end of a language model: final norm and LM head, on hidden states [N, H]."""

    def __init__(self, hidden, vocab, norm="rms", eps=1e-6, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        w = torch.randn(vocab, hidden, generator=g) * hidden ** -0.5
        self.head = w.to(device=device, dtype=torch.bfloat16).requires_grad_()
        self.scale = torch.ones(hidden, device=device, requires_grad=True)
        self.shift = None
        if norm == "layer":
            self.shift = torch.zeros(hidden, device=device, requires_grad=True)
        self.eps = eps

    def parameters(self):
        return [p for p in (self.head, self.scale, self.shift) if p is not None]

    def norm(self, x, active_mask=None):
        if self.shift is not None:
            return rlk.layer_norm(x, self.scale, self.shift, self.eps, active_mask)
        return rlk.rms_norm(x, self.scale, self.eps, active_mask)

    @torch.no_grad()
    def sample(self, x, uniforms, active_mask=None, **settings):
        """(tokens, logp, kept_logp) of the next token of each row."""
        logits = torch.mm(self.norm(x, active_mask).float(), self.head.float().t())
        return rlk.sample_logits(logits, uniforms, active_mask=active_mask, **settings)

    def logp(self, x, tokens, active_mask=None, temperature=1.0):
        return rlk.linear_logp(self.norm(x, active_mask), self.head, tokens, active_mask,
                               temperature)


class Decoder:
    """One decoding step in a CUDA graph, on buffers of its own."""

    def __init__(self, policy, rows, hidden, active_mask, **settings):
        device = policy.head.device
        self.x = torch.zeros(rows, hidden, dtype=torch.bfloat16, device=device)
        self.uniforms = torch.zeros(rows, device=device)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            policy.sample(self.x, self.uniforms, active_mask, **settings)     # warm-up
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = policy.sample(self.x, self.uniforms, active_mask, **settings)

    def __call__(self, x, uniforms):
        self.x.copy_(x)
        self.uniforms.copy_(uniforms)
        self.graph.replay()
        return tuple(t.clone() for t in self.out)


def update(policy, x, tokens, logp_old, advantages, active_mask, temperature, lr, eps_clip=0.2):
    """One policy-gradient step.  Returns the audit's and the loss's results, and dx."""
    x = x.detach().requires_grad_()
    logp = policy.logp(x, tokens, active_mask, temperature)
    audit = rlk.dlogp_audit(logp.detach(), logp_old, active_mask)
    scale = 1.0 / max(1, audit["active_count"])
    grad, loss = rlk.grpo_clip_loss(logp.detach(), logp_old, advantages, active_mask, eps_clip,
                                    eps_clip, scale)
    logp.backward(grad)
    with torch.no_grad():
        for p in policy.parameters():
            p.sub_(lr * p.grad)
            p.grad = None
    return audit, loss, x.grad


def run(norm="rms", rows=256, hidden=512, vocab=1000, steps=4, temperature=0.8, top_k=0,
        top_p=0.95, min_p=0.0, lr=4.0, seed=0, log=print):
    """Teaches the policy to draw even tokens.  One dict a step: its share of even tokens, the
    audit's largest |logp - logp_old| and the loss."""
    policy = PolicyHead(hidden, vocab, norm, seed=seed)
    device = policy.head.device
    g = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(rows, hidden, generator=g).to(device=device, dtype=torch.bfloat16)
    mask = (torch.arange(rows) % 7 != 3).to(device=device, dtype=torch.uint8)  # others: padding
    decode = Decoder(policy, rows, hidden, mask, temperature=temperature, top_k=top_k,
                     top_p=top_p, min_p=min_p)
    on = mask.bool()
    history = []
    for step in range(steps):
        tokens, logp_old, _ = decode(x, torch.rand(rows, generator=g).to(device))
        even = (tokens % 2 == 0).float()
        audit, loss, _ = update(policy, x, tokens, logp_old, 2.0 * even - 1.0, mask, temperature,
                                lr)
        history.append({"even": float(even[on].mean()), "max_dlogp": audit["max_abs_dlogp"],
                        "active": audit["active_count"], "loss": loss["loss"]})
        if log is not None:
            log(f"step {step}: even tokens {history[-1]['even']:.3f}, "
                f"max |dlogp| {history[-1]['max_dlogp']:.2e}, loss {history[-1]['loss']:+.4f}")
    return history


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--norm", choices=("rms", "layer"), default="rms")
    for name, default in (("rows", 256), ("hidden", 512), ("vocab", 1000), ("steps", 4),
                          ("top-k", 0), ("seed", 0)):
        p.add_argument("--" + name, type=int, default=default)
    for name, default in (("temperature", 0.8), ("top-p", 0.95), ("min-p", 0.0), ("lr", 4.0)):
        p.add_argument("--" + name, type=float, default=default)
    run(**vars(p.parse_args(argv)))


if __name__ == "__main__":
    main()
