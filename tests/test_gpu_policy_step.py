"""The example of a policy head: norm, sampling, scoring, loss and backward in one step."""
import importlib.util
import os

import pytest
import torch

from helpers import GRAD_REL_L2, LOGP_ATOL, dev, rel_l2

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(__file__), os.pardir, "examples", "policy_step.py")
_SPEC = importlib.util.spec_from_file_location("policy_step", _PATH)
example = importlib.util.module_from_spec(_SPEC)
_SPEC.loader.exec_module(example)


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_learns_and_stays_consistent(norm):
    rows = 256
    history = example.run(norm=norm, rows=rows, steps=8, log=None)
    for h in history:
        assert h["active"] == int((torch.arange(rows) % 7 != 3).sum())
        assert h["max_dlogp"] <= 2 * LOGP_ATOL          # each side within the contract's 1e-3
    assert sum(h["even"] for h in history[-2:]) > sum(h["even"] for h in history[:2])


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_update_against_float64(norm):
    # The normed rows y (bf16) are given to the reference.  dh of the head meets the contract of
    # its backward, to which the ratio's error adds that of logp; the norm's backward takes out
    # one or two of 256 directions (below a factor of 2) and rounds dx to bf16.
    n, h, v, t = 96, 256, 2000, 0.7
    p = example.PolicyHead(h, v, norm, seed=3)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(n, h, generator=g).to(device=dev(), dtype=torch.bfloat16)
    mask = (torch.arange(n) % 5 != 1).to(device=dev(), dtype=torch.uint8)
    u = torch.rand(n, generator=g).to(dev())
    tokens, old, kept = p.sample(x, u, mask, temperature=t, top_p=0.9)
    on = mask.bool()
    assert bool((tokens[~on] == -1).all()) and bool((tokens[on] >= 0).all())
    assert bool((kept >= old).all())
    head = p.head.detach().clone()
    y = p.norm(x, mask).detach()
    adv = torch.randn(n, generator=g).to(dev())
    audit, loss, dx = example.update(p, x, tokens, old, adv, mask, t, lr=0.0)
    assert audit["active_count"] == int(on.sum()) and audit["max_abs_dlogp"] <= 2 * LOGP_ATOL
    # the head's gradient for these y, then the norm's backward, in float64
    yd = y.double().requires_grad_()
    lp = torch.log_softmax(yd @ head.double().t() / t, 1)[torch.arange(n, device=dev()),
                                                        tokens.clamp(min=0)]
    ratio = torch.exp(lp - old.double())
    a = adv.double()
    inner = torch.minimum(ratio * a, ratio.clamp(0.8, 1.2) * a)
    (-(inner * on).sum() / int(on.sum())).backward()
    xd = x.double().requires_grad_()
    c = xd - xd.mean(1, keepdim=True) if norm == "layer" else xd
    (c * torch.rsqrt((c * c).mean(1, keepdim=True) + p.eps) * on[:, None]).backward(yd.grad)
    assert rel_l2(dx, xd.grad.cpu().numpy()) <= 2 * GRAD_REL_L2 + LOGP_ATOL + 2.0 ** -8
    assert bool((dx[~on] == 0).all())
