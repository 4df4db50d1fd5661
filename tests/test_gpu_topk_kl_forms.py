"""KL against a teacher's top tokens where a gradient's weight is not at the teacher's tokens, and
where dh takes a vocabulary's sub-chunks one after the other: against float64.

dhidden and dweight: the contract for gradients (GRAD_REL_L2).
"""
import numpy as np
import pytest
import torch

import rl_post_linear_gb300 as rlk
from helpers import GRAD_REL_L2, LOGP_ATOL, dev, same_bits

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def oracle(hid, w, ids, a, grad, block=2048):
    """float64 (kl, lse, dh, dw) at T = 1 by the formulas, on the device, some rows at a time."""
    w64 = w.double()
    dw = torch.zeros_like(w64)
    kl, lse, dh = [], [], []
    for h, i, b, g in zip(*(x.split(block) for x in (hid, ids, a, grad))):
        h, b, g = h.double(), b.double(), g.double()
        s = h @ w64.t()
        at = torch.logsumexp(s, 1, keepdim=True)
        q = b.exp()
        kl.append((q * (b - s.gather(1, i) + at)).sum(1))
        lse.append(at[:, 0])
        ds = s.sub_(at).exp_().mul_(q.sum(1, keepdim=True)).scatter_add_(1, i, -q).mul_(g[:, None])
        dh.append(ds @ w64)
        dw += ds.t() @ h
    return torch.cat(kl), torch.cat(lse), torch.cat(dh), dw


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def step(hid, w, ids, a, grad):
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    kl, lse, lp = rlk.linear_topk_kl_fwd(hid, w, ids, a, error_word=err)
    dh, dw = rlk.linear_topk_kl_bwd(hid, w, ids, a, None, grad, lse, lp, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return kl, lse, lp, dh, dw


def check(hid, w, ids, a, grad):
    kl, lse, lp, dh, dw = step(hid, w, ids, a, grad)
    kl64, lse64, dh64, dw64 = oracle(hid, w, ids, a, grad)
    assert float((lse - lse64).abs().max()) <= LOGP_ATOL
    q = a.double().exp()
    size = q.sum(1) * LOGP_ATOL + 2.0 ** -20 * (q * a.double().abs()).sum(1)
    assert bool(((kl - kl64).abs() <= size).all())
    assert rel(dh, dh64) <= GRAD_REL_L2 and rel(dw, dw64) <= GRAD_REL_L2
    return kl, lse, lp, dh, dw


def head(h, v, seed):
    return (torch.randn(v, h, generator=gen(seed)) * h ** -0.5).to(torch.bfloat16).to(dev())


def listed(n, v, k, seed):
    """k tokens a row of nearly equal weight, distinct, from the lower half of the vocabulary."""
    g = gen(seed)
    ids = torch.randint(0, v // 2, (n, k), generator=g) // k * k + torch.arange(k)
    return ids.to(dev()), torch.log_softmax(0.5 * torch.randn(n, k, generator=g), 1).to(dev())


@pytest.mark.parametrize("others", [2, 5, 8])
@pytest.mark.parametrize("n,h,v", [(300, 512, 7000), (300, 512, 20000), (1024, 1024, 40000)])
def test_a_student_that_prefers_what_the_teacher_does_not_list(n, h, v, others):
    w = head(h, v, others)
    ids, a = listed(n, v, 64, others + 1)
    own = torch.randint(v // 2, v, (n, others), generator=gen(others + 2)).to(dev())
    hid = (14.0 * w[own].float()).sum(1).to(torch.bfloat16)
    check(hid, w, ids, a, torch.ones(n, device=dev()) / n)


@pytest.mark.parametrize("n,v", [(64, 7000), (64, 9000), (300, 9000), (64, 40000), (300, 40000),
                                 (2048, 33000)])
def test_entries_that_bf16_holds_worst(n, v):
    # Four equal rows of W, p = 1/4 each, and g for which g Q p is halfway between two numbers of
    # bf16, (1 + 2^-8 - 2^-12) 2^-7: one bf16 is off by 2^-8 of nearly the whole gradient.
    h, k = 256, 64
    w = head(h, v, 7)
    w[v - 4:] = w[v - 1].clone()
    ids, a = listed(n, v, k, 8)
    base = w[v - 1].float() * 40.0
    hid = (base + 0.1 * torch.randn(n, h, generator=gen(9)).to(dev())).to(torch.bfloat16)
    p = torch.softmax(hid.double() @ w.double().t(), 1)[:, v - 1]
    assert float(p.min()) > 0.2 and float(p.max()) <= 0.25
    grad = ((1 + 2.0 ** -8 - 2.0 ** -12) * 2.0 ** -7 / (p * a.double().exp().sum(1))).float()
    check(hid, w, ids, a, grad)


def test_a_student_that_agrees_with_its_teacher():
    # the listed entries nearly cancel, and the classes that are not listed weigh as much
    n, h, v, k = 256, 256, 50000, 16
    w = head(h, v, 10)
    hid = (3.0 * torch.randn(n, h, generator=gen(11))).to(torch.bfloat16).to(dev())
    lp, ids = torch.log_softmax(hid.double() @ w.double().t(), 1).topk(k, 1)
    a = (lp + 0.01 * torch.randn(n, k, generator=gen(12)).to(dev())).float()
    check(hid, w, ids, a, torch.randn(n, generator=gen(13)).to(dev()))


def in_parts(n, h, v, k):
    """Whether dh's sub-chunks are taken side by side: their sums need workspace then."""
    query = rlk.rlk_linear_topk_kl_bwd_workspace_bytes
    return query(n, h, v, k) > query(n, h, 1000, k)


@pytest.mark.parametrize("v", [5000, 8192, 20000, 33003, 45000])
def test_sub_chunks_one_after_the_other(v):
    # many tiles; some rows with a class near p = 1 that no slot names
    n, h, k = 15000, 64, 5
    assert not in_parts(n, h, v, k)
    w = head(h, v, 14)
    ids, a = listed(n, v, k, 15)
    hid = torch.randn(n, h, generator=gen(16)).to(dev()) + 2.0 * w[ids[:, 0]].float()
    own = torch.randint(v // 2, v, (n,), generator=gen(17)).to(dev())
    lean = (torch.arange(n, device=dev()) % 5 == 3).float() * 16.0
    hid = (hid + lean[:, None] * w[own].float()).to(torch.bfloat16)
    grad = torch.randn(n, generator=gen(18)).to(dev()) / n
    whole = check(hid, w, ids, a, grad)
    # the same bits for a part of the rows, whose sub-chunks are taken side by side
    rows = slice(4321, 4821)
    assert in_parts(500, h, v, k)
    part = step(hid[rows].contiguous(), w, ids[rows].contiguous(), a[rows].contiguous(), grad[rows])
    for got, want in zip(part[:4], whole[:4]):
        assert same_bits(got, want[rows].contiguous())


@pytest.mark.parametrize("n,h,v,k", [(4096, 512, 65537, 8), (2048, 1024, 33003, 8)])
def test_many_rows_that_share_tokens(n, h, v, k):
    # tokens that a row or two list, and some that very many do; masked rows, empty slots
    w = head(h, v, 19)
    ids, a = listed(n, v, k, 20)
    ids[:, 0] = v - 1
    ids[::3, 1] = v - 2
    hid = (torch.randn(n, h, generator=gen(21)).to(dev()) + w[ids[:, 2]].float()).to(torch.bfloat16)
    grad = torch.randn(n, generator=gen(22)).to(dev()) / n
    check(hid, w, ids, a, grad)
    mask = (torch.arange(n, device=dev()) % 7 != 2).to(torch.uint8)
    holes = torch.rand(n, k, generator=gen(23)).to(dev()) < 0.3
    some = torch.where(holes, -1, ids)
    kl, lse, lp = rlk.linear_topk_kl_fwd(hid, w, some, a, mask)
    dh, dw = rlk.linear_topk_kl_bwd(hid, w, some, a, mask, grad, lse, lp)
    b = torch.where(holes | (mask == 0)[:, None], -np.inf, a)      # a weight of 0
    kl64, _, dh64, dw64 = oracle(hid, w, ids, torch.where(b > -np.inf, b, -1e4), grad)
    assert float(((kl - kl64) * mask).abs().max()) <= 2 * LOGP_ATOL
    assert rel(dh, dh64) <= GRAD_REL_L2 and rel(dw, dw64) <= GRAD_REL_L2
