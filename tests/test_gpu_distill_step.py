"""The example of distillation: processing, draw, teacher's top tokens, KL and backward together."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

from helpers import GRAD_REL_L2, LOGP_ATOL, dev, rel_l2

pytestmark = pytest.mark.gpu

_DIR = os.path.join(os.path.dirname(__file__), os.pardir, "examples")
sys.path.insert(0, _DIR)
_SPEC = importlib.util.spec_from_file_location("distill_step", os.path.join(_DIR, "distill_step.py"))
example = importlib.util.module_from_spec(_SPEC)
_SPEC.loader.exec_module(example)


def test_runs():
    rows = 256
    history = example.run(rows=rows, steps=4, log=None)
    on = (torch.arange(rows) % 7 != 3).to(dev())
    for h in history:
        assert np.isfinite(h["kl"]) and h["kl"] >= -LOGP_ATOL
        assert bool((h["tokens"][on] >= 0).all()) and bool((h["tokens"][~on] == -1).all())


def test_pack_allowed():
    allow = torch.rand(5, 77, generator=torch.Generator().manual_seed(1)) < 0.5
    words = example.pack_allowed(allow.to(dev())).cpu().numpy()
    bits = np.unpackbits(words.view(np.uint8), axis=1, bitorder="little")[:, :77]
    assert np.array_equal(bits.astype(bool), allow.numpy())


def test_rollout_draws_only_what_is_allowed_and_counts_what_it_drew():
    n, h, v, p, room = 40, 128, 600, 5, 6
    student = example.PolicyHead(h, v, seed=5)
    g = torch.Generator().manual_seed(6)
    prompts = torch.randint(0, v, (n, p), generator=g).to(dev())
    allow = (torch.rand(n, v, generator=g) < 0.1).to(dev())
    rollout = example.Rollout(student, prompts, room, h, example.pack_allowed(allow),
                              presence=50.0, repetition=1.0, frequency=0.0)
    x = torch.randn(n, h, generator=g).to(device=dev(), dtype=torch.bfloat16)
    seen = torch.zeros(n, v, dtype=torch.bool, device=dev())
    for _ in range(room):
        tokens, _ = rollout(x, torch.rand(n, generator=g).to(dev()))
        assert bool(allow.gather(1, tokens[:, None]).all())
        # 50 below all others: drawn again only where nothing else is left
        left = (allow & ~seen).any(1)
        assert not bool((seen.gather(1, tokens[:, None])[:, 0] & left).any())
        seen.scatter_(1, tokens[:, None], True)
    assert torch.equal(rollout.tokens[:, :p], prompts)
    assert bool((rollout.tokens[:, p:p + room] >= 0).all())


def test_update_against_float64():
    # The normed rows y (bf16) and the teacher's tokens are given to the reference.  dh of the head
    # meets the contract of its backward; the norm's backward takes out one of 256 directions (below
    # a factor of 2) and rounds dx to bf16.
    n, h, v, k, t = 96, 256, 9000, 24, 1.2
    student, teacher = example.PolicyHead(h, v, seed=3), example.PolicyHead(h, v, seed=4)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(n, h, generator=g).to(device=dev(), dtype=torch.bfloat16)
    mask = (torch.arange(n) % 5 != 1).to(device=dev(), dtype=torch.uint8)
    on = mask.bool()
    ids, a = example.teach(teacher, x, k, t, mask)
    z = torch.mm(teacher.norm(x, mask).double(), teacher.head.double().t()) / t
    want = torch.log_softmax(z, 1).sort(dim=1, descending=True, stable=True)
    assert bool((ids[~on] == -1).all())
    # the logits are an fp32 product here: the order may differ where two are within its error
    assert float((a[on] - want.values[on, :k]).abs().max()) <= LOGP_ATOL
    head = student.head.detach().clone()
    y = student.norm(x, mask).detach()
    loss, dx = example.update(student, x, ids, a, t, mask, lr=0.0)
    yd = y.double().requires_grad_()
    lp = torch.log_softmax(yd @ head.double().t() / t, 1).gather(1, ids.clamp(min=0))
    la = torch.log_softmax(a.double(), 1)
    kl = ((la.exp() * (la - lp)).sum(1) * on).sum() / int(on.sum())
    kl.backward()
    assert abs(loss - float(kl)) <= LOGP_ATOL
    xd = x.double().requires_grad_()
    (xd * torch.rsqrt((xd * xd).mean(1, keepdim=True) + student.eps) * on[:, None]).backward(yd.grad)
    assert rel_l2(dx, xd.grad.cpu().numpy()) <= 2 * GRAD_REL_L2 + 2.0 ** -8
    assert bool((dx[~on] == 0).all())
