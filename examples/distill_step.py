"""On-policy distillation of a policy head from a teacher's top tokens.

Rollout: the student's hidden states go through the final norm and the LM head; penalties for the
tokens each sequence has drawn already and a mask of allowed tokens change the logits, and a token
is drawn from them (one step, captured in a CUDA graph and replayed).  Teacher: the K largest
log-probs of its own head's logits for the same states.  Update: the KL of those against the
student's head, without storing its logits, goes back through head and norm.

    python examples/distill_step.py [--steps 8] [--rows 256] [--top-k 32] ...
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import rl_post_linear_gb300 as rlk                                            # noqa: E402
from policy_step import PolicyHead                                            # noqa: E402


def pack_allowed(allow):
    """int32 words [N, ceil(V / 32)] of a boolean [N, V]: bit v % 32 of word v // 32."""
    n, v = allow.shape
    wide = torch.zeros(n, (v + 31) // 32 * 32, dtype=torch.int64, device=allow.device)
    wide[:, :v] = allow
    words = (wide.view(n, -1, 32) << torch.arange(32, device=allow.device)).sum(2)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).int()


class Rollout:
    """Sequences that are decoded together: their tokens, and one decoding step in a CUDA graph."""

    def __init__(self, student, prompts, room, hidden, allowed=None, active_mask=None,
                 repetition=1.1, frequency=0.1, presence=0.0, temperature=0.8, top_p=0.95):
        if room < 1:
            raise ValueError("room must be 1 or more, got %d" % room)
        self.left = room                          # tokens that may still be drawn
        device = student.head.device
        n, p = prompts.shape
        self.tokens = torch.full((n, p + room), -1, dtype=torch.int64, device=device)
        self.tokens[:, :p] = prompts
        self.prompt_lengths = torch.full((n,), p, dtype=torch.int64, device=device)
        self.lengths = self.prompt_lengths.clone()
        self.x = torch.zeros(n, hidden, dtype=torch.bfloat16, device=device)
        self.uniforms = torch.zeros(n, device=device)

        @torch.no_grad()
        def step():
            logits = torch.mm(student.norm(self.x, active_mask).float(), student.head.float().t())
            rlk.process_logits(logits, self.tokens, self.lengths, self.prompt_lengths, repetition,
                               frequency, presence, allowed=allowed, active_mask=active_mask,
                               out=logits)
            drawn, logp, _ = rlk.sample_logits(logits, self.uniforms, temperature, top_p=top_p,
                                               active_mask=active_mask)
            self.tokens.scatter_(1, self.lengths[:, None], drawn[:, None])
            return drawn, logp

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                                            # warm-up
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = step()

    def __call__(self, x, uniforms):
        """One token of each sequence from its state: (tokens, logp)."""
        if self.left < 1:
            raise RuntimeError("the sequences' buffer is full")
        self.left -= 1
        self.x.copy_(x)
        self.uniforms.copy_(uniforms)
        self.graph.replay()
        self.lengths += 1
        return tuple(t.clone() for t in self.out)


@torch.no_grad()
def teach(teacher, x, k, temperature, active_mask=None):
    """(ids, logp) [N, k]: what a teacher sends."""
    logits = torch.mm(teacher.norm(x, active_mask).float(), teacher.head.float().t())
    ids, logp, _ = rlk.topk_logp(logits, k, temperature, active_mask)
    return ids, logp


def update(student, x, ids, logp, temperature, active_mask=None, lr=1.0, renormalize=True):
    """One step on the mean KL.  Returns it and dx."""
    x = x.detach().requires_grad_()
    kl = rlk.linear_topk_kl(student.norm(x, active_mask), student.head, ids, logp, active_mask,
                            temperature, renormalize)
    count = x.shape[0] if active_mask is None else active_mask.sum().clamp(min=1)
    loss = kl.sum() / count
    loss.backward()
    with torch.no_grad():
        for p in student.parameters():
            p.sub_(lr * p.grad)
            p.grad = None
    return float(loss.detach()), x.grad


def run(rows=256, hidden=512, vocab=1000, prompt=16, steps=8, top_k=32, temperature=1.0, lr=10.0,
        seed=0, log=print):
    """One dict a step: the mean KL and the share of draws that the sequence had drawn before."""
    if steps < 1:
        raise ValueError("steps must be 1 or more, got %d" % steps)
    student = PolicyHead(hidden, vocab, seed=seed)
    teacher = PolicyHead(hidden, vocab, seed=seed + 1)
    with torch.no_grad():
        teacher.head.mul_(3.0)
    device = student.head.device
    g = torch.Generator().manual_seed(seed + 2)
    mask = (torch.arange(rows) % 7 != 3).to(device=device, dtype=torch.uint8)  # others: padding
    prompts = torch.randint(0, vocab, (rows, prompt), generator=g).to(device)
    allowed = pack_allowed((torch.rand(rows, vocab, generator=g) < 0.8).to(device))
    rollout = Rollout(student, prompts, steps, hidden, allowed, mask, temperature=temperature)
    on = mask.bool()
    states = torch.randn(rows, hidden, generator=g).to(device=device, dtype=torch.bfloat16)
    history = []
    for step in range(steps):
        tokens, _ = rollout(states, torch.rand(rows, generator=g).to(device))
        before = rollout.tokens[:, prompt:prompt + step]
        again = float((before[on] == tokens[on, None]).any(1).float().mean()) if step else 0.0
        ids, logp = teach(teacher, states, top_k, temperature, mask)
        loss, _ = update(student, states, ids, logp, temperature, mask, lr)
        history.append({"kl": loss, "again": again, "tokens": tokens})
        if log is not None:
            log(f"step {step}: KL {loss:.4f}, drawn again {again:.3f}")
    return history


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("rows", 256), ("hidden", 512), ("vocab", 1000), ("prompt", 16),
                          ("steps", 8), ("top-k", 32), ("seed", 0)):
        p.add_argument("--" + name, type=int, default=default)
    for name, default in (("temperature", 1.0), ("lr", 10.0)):
        p.add_argument("--" + name, type=float, default=default)
    run(**vars(p.parse_args(argv)))


if __name__ == "__main__":
    main()
