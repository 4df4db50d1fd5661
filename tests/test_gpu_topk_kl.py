"""KL of the head against a teacher's top tokens, forward and backward, against float64.

lse and logp are within the framework's contract for logp (LOGP_ATOL); kl is a sum of them with
weights q, so |error| <= LOGP_ATOL sum q + 2^-20 sum q |log q| (the exponential, the sum).  dhidden
and dweight: the contract for gradients (GRAD_REL_L2).
"""
import numpy as np
import pytest
import torch

import rl_post_linear_gb300 as rlk
from helpers import GRAD_REL_L2, LOGP_ATOL, dev, f64, rel_l2, same_bits

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def problem(n, h, v, k, seed, lean=3.0, empty=0.0):
    """A student that gives the teacher's tokens more weight than others, on the CPU."""
    g = gen(seed)
    w = (torch.randn(v, h, generator=g) * h ** -0.5).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(v, generator=g)[:k] for _ in range(n)]) if k <= v else \
        torch.randint(0, v, (n, k), generator=g)
    a = torch.log_softmax(2.0 * torch.randn(n, k, generator=g), 1)
    a += torch.log(0.4 + 0.6 * torch.rand(n, 1, generator=g))
    hid = torch.randn(n, h, generator=g)
    for j in range(min(k, 8)):
        hid += lean * torch.rand(n, 1, generator=g) * w[ids[:, j]].float()
    ids[torch.rand(n, k, generator=g) < empty] = -1
    return hid.to(torch.bfloat16), w, ids, a


def oracle(hid, w, ids, a, mask, t, renorm, grad=None):
    """float64 results by the formulas, numpy arrays; rows that cannot be are the caller's."""
    h64, w64 = f64(hid), f64(w)
    ids, a = ids.cpu().numpy(), a.cpu().double().numpy()
    n, k = ids.shape
    s = h64 @ w64.T / t
    m = s.max(1, keepdims=True)
    lse = (m + np.log(np.exp(s - m).sum(1, keepdims=True)))[:, 0]
    live = np.ones(n, bool) if mask is None else mask.cpu().numpy() != 0
    on = (ids >= 0) & live[:, None]
    a = np.where(on, a, -np.inf)
    if renorm:
        with np.errstate(divide="ignore", invalid="ignore"):
            top = a.max(1, keepdims=True)
            norm = top + np.log(np.exp(a - top).sum(1, keepdims=True))
        a = np.where(np.isfinite(norm), a - norm, -np.inf)
    q = np.exp(a)
    lp = np.where(on, np.take_along_axis(s, np.maximum(ids, 0), 1) - lse[:, None], 0.0)
    with np.errstate(invalid="ignore"):
        kl = np.where(q > 0, q * (a - lp), 0.0).sum(1)
        size = q.sum(1) * LOGP_ATOL + 2.0 ** -20 * np.where(q > 0, q * np.abs(a), 0.0).sum(1)
    out = [kl, np.where(live, lse, 0.0), lp, size]
    if grad is not None:
        g = np.where(live, grad.cpu().double().numpy(), 0.0) / t
        ds = g[:, None] * q.sum(1, keepdims=True) * np.exp(s - lse[:, None])
        for i in range(n):
            np.add.at(ds[i], ids[i][on[i]], -g[i] * q[i][on[i]])
        out += [ds @ w64, ds.T @ h64]
    return out


def check(hid, w, ids, a, mask=None, t=1.0, renorm=False, grad=None):
    d = [x if x is None else x.to(dev()) for x in (hid, w, ids, a, mask)]
    n = hid.shape[0]
    if grad is None:
        grad = torch.randn(n, generator=gen(99)) / n
    g = grad.to(dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    kl, lse, lp = rlk.linear_topk_kl_fwd(*d, t, renorm, err)
    dh, dw = rlk.linear_topk_kl_bwd(*d, g, lse, lp, t, renorm, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    kl64, lse64, lp64, size, dh64, dw64 = oracle(hid, w, ids, a, mask, t, renorm, grad)
    assert np.all(np.abs(f64(kl) - kl64) <= size + 1e-30)
    assert np.max(np.abs(f64(lse) - lse64)) <= LOGP_ATOL
    assert np.max(np.abs(f64(lp) - lp64)) <= LOGP_ATOL
    for got, want in ((dh, dh64), (dw, dw64)):
        if np.any(want):
            assert rel_l2(got, want) <= GRAD_REL_L2
        else:
            assert not bool(got.any())
    return kl, lse, lp, dh, dw


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("n,h,v,k", [(1, 64, 1, 1), (1, 64, 5, 1), (3, 64, 70, 5), (5, 128, 300, 20),
                                     (130, 192, 1000, 64), (257, 256, 4099, 33),
                                     (64, 512, 33000, 128), (300, 64, 70000, 7),
                                     (20, 64, 2000, 1024)])
def test_shapes(n, h, v, k, renorm):
    check(*problem(n, h, v, k, n + v), t=1.3, renorm=renorm)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("t", [0.3, 1.0, 2.0])
def test_temperatures_and_empty_slots(t, renorm):
    check(*problem(96, 256, 5000, 50, 1, empty=0.5), t=t, renorm=renorm)


def test_lse_is_that_of_the_log_prob():
    # but for the accumulators' loss, 1.04e-9 H of a logit, and the rounding of lse
    hid, w, ids, a = (x.to(dev()) for x in problem(77, 256, 9000, 5, 2))
    mask = (torch.arange(77) % 3 != 0).to(torch.uint8).to(dev())
    for m in (None, mask):
        lse = rlk.linear_topk_kl_fwd(hid, w, ids, a, m, 0.8)[1]
        want = rlk.linear_logp_fwd(hid, w, ids[:, 0].contiguous(), m, 0.8)[1]
        top = float((hid.float() @ w.float().t()).abs().max()) / 0.8
        assert float((lse - want).abs().max()) <= 1.04e-9 * 256 * top + 2.0 ** -21 * (1 + top)


@pytest.mark.parametrize("h", [1024, 4096, 7168])
def test_logits_keep_their_digits(h):
    # Large logits that build up evenly over H.  The accumulators cut off 1.04e-9 H of a logit,
    # which is given back; what is left is the scatter of H/16 truncations of at most an ulp of
    # the logit, s 2^-23 each: sqrt(H/16 / 12) of them as standard deviation, six of those.
    g = gen(h)
    n, v, k = 64, 8000, 32
    w = (torch.randn(v, h, generator=g) * h ** -0.5).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(v, generator=g)[:k] for _ in range(n)])
    hid = torch.randn(n, h, generator=g)
    for j in range(k):
        hid += (12.0 - 0.3 * j) * w[ids[:, j]].float()
    hid = hid.to(torch.bfloat16)
    _, lse, lp = rlk.linear_topk_kl_fwd(hid.to(dev()), w.to(dev()), ids.to(dev()),
                                        torch.zeros(n, k, device=dev()))
    s = f64(hid) @ f64(w).T
    at = np.take_along_axis(s, ids.numpy(), 1)
    got = f64(lp) + f64(lse)[:, None]
    tol = 6 * np.sqrt(h / 192) * 2.0 ** -23 * np.abs(at) + 2.0 ** -21 * (1 + np.abs(at).max())
    assert np.all(np.abs(got - at) <= tol)
    assert abs(np.mean((got - at)[at > 4] / at[at > 4])) <= 0.25 * 1.04e-9 * h + 2.0 ** -23


@pytest.mark.parametrize("share", [0.0, 0.3, 0.9, 1.0])
def test_masks(share):
    hid, w, ids, a = problem(150, 128, 3000, 16, 3)
    mask = (torch.rand(150, generator=gen(4)) < share).to(torch.uint8)
    hid[mask == 0] = float("nan")                       # never read
    ids[mask == 0] = 1 << 40
    clean = hid.clone().nan_to_num()
    cids = torch.where(mask[:, None] != 0, ids, -1)
    grad = torch.randn(150, generator=gen(5))
    d = [x.to(dev()) for x in (hid, w, ids, a, mask)]
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    kl, lse, lp = rlk.linear_topk_kl_fwd(*d, 1.0, False, err)
    dh, dw = rlk.linear_topk_kl_bwd(*d, grad.to(dev()), lse, lp, 1.0, False, err)
    assert int(err.item()) == 0
    want = check(clean, w, cids, a, mask, grad=grad)
    for got, ref in zip((kl, lse, lp, dh, dw), want):
        assert same_bits(got, ref)
    off = (mask == 0).to(dev())
    assert not bool(dh[off].any()) and not bool(kl[off].any()) and not bool(lp[off].any())


def test_an_agreeing_student_and_a_confident_one():
    # the listed entries Q p - q are differences of near numbers, or nearly a whole row
    for lean in (0.0, 40.0):
        hid, w, ids, a = problem(100, 256, 4000, 30, 6, lean=lean)
        lp = torch.from_numpy(oracle(hid, w, ids, a, None, 1.0, False)[2]).float()
        check(hid, w, ids, lp + 0.01 * torch.randn(lp.shape, generator=gen(7)))
        check(hid, w, ids, a, renorm=True)


def test_repeated_tokens_add_up():
    hid, w, ids, a = problem(40, 128, 900, 12, 8)
    ids[:, 5] = ids[:, 0]
    ids[:, 11] = ids[:, 0]
    ids[:, 7] = ids[:, 6]
    kl, _, _, dh, _ = check(hid, w, ids, a)
    # a slot split in two weighs the same
    b = torch.cat((a, a[:, :1] - np.log(2.0)), 1)
    b[:, 0] -= np.log(2.0)
    check(hid, w, torch.cat((ids, ids[:, :1]), 1), b)
    hard = problem(64, 128, 700, 1, 9)                  # a hard label is a slot of weight 1
    zero = torch.zeros(64, 1)
    kl = check(hard[0], hard[1], hard[2], zero)[0]
    want = rlk.linear_logp_fwd(hard[0].to(dev()), hard[1].to(dev()), hard[2][:, 0].to(dev()))[0]
    assert float((kl + want).abs().max()) <= LOGP_ATOL


def test_weights_of_zero_and_rows_without_any():
    hid, w, ids, a = problem(33, 64, 500, 6, 10)
    a[:, 2] = -np.inf
    ids[3], a[4] = -1, -np.inf
    a[7, 1], ids[7, 1] = float("nan"), -1               # an empty slot's value is not used
    for renorm in (False, True):
        kl, _, _, dh, _ = check(hid, w, ids, torch.where(ids < 0, 0.0, a), renorm=renorm)
        again = rlk.linear_topk_kl_fwd(*(x.to(dev()) for x in (hid, w, ids, a)), None, 1.0, renorm)[0]
        assert same_bits(again, kl)
        assert kl[3] == 0 and kl[4] == 0 and not bool(dh[3].any()) and not bool(dh[4].any())


@pytest.mark.parametrize("kind", ["id", "nan", "inf"])
def test_rows_that_cannot_be(kind):
    hid, w, ids, a = problem(20, 64, 500, 6, 11)
    flag = rlk.RLK_DEVERR_LOGITS
    if kind == "id":
        ids[5, 2], flag = 500, rlk.RLK_DEVERR_TARGET_RANGE
    else:
        a[5, 2] = float(kind)
    d = [x.to(dev()) for x in (hid, w, ids, a)] + [None]
    g = torch.ones(20, device=dev())
    err = torch.zeros(2, dtype=torch.int32, device=dev())
    kl, lse, lp = rlk.linear_topk_kl_fwd(*d, 1.0, False, err[:1])
    dh, dw = rlk.linear_topk_kl_bwd(*d, g, lse, lp, 1.0, False, err[1:])
    assert err.tolist() == [flag, flag]
    assert bool(torch.isnan(kl[5])) and bool(torch.isnan(lp[5]).all())
    ids[5], a[5] = -1, 0.0
    kl2, _, _, dh2, dw2 = check(hid, w, ids, a, grad=torch.ones(20))
    keep = torch.arange(20, device=dev()) != 5
    assert same_bits(kl[keep], kl2[keep]) and same_bits(dh, dh2) and same_bits(dw, dw2)


def test_a_row_does_not_depend_on_its_batch_and_dweight_is_reproducible():
    hid, w, ids, a = (x.to(dev()) for x in problem(300, 128, 40000, 24, 12))
    g = torch.randn(300, generator=gen(13)).to(dev())

    def both(rows):
        kl, lse, lp = rlk.linear_topk_kl_fwd(hid[rows], w, ids[rows], a[rows])
        dh, dw = rlk.linear_topk_kl_bwd(hid[rows], w, ids[rows], a[rows], None, g[rows], lse, lp)
        return kl, lse, lp, dh, dw

    whole = both(slice(0, 300))
    for got, want in zip(both(slice(0, 300)), whole):
        assert same_bits(got, want)
    part = both(slice(131, 260))
    for got, want in zip(part[:4], whole[:4]):
        assert same_bits(got, want[131:260])


def test_few_tiles_and_many_give_the_same_bits():
    # dh of few rows takes a vocabulary chunk's parts side by side, of many one after the other
    n, h, v, k = 10000, 64, 45000, 3
    hid, w, ids, a = (x.to(dev()) for x in problem(500, h, v, k, 22))
    reps = n // 500
    g = torch.randn(500, generator=gen(23)).to(dev())

    def both(hid, ids, a, g):
        kl, lse, lp = rlk.linear_topk_kl_fwd(hid, w, ids, a)
        return kl, lp, rlk.linear_topk_kl_bwd(hid, w, ids, a, None, g, lse, lp)[0]

    few = both(hid, ids, a, g)
    many = both(hid.repeat(reps, 1), ids.repeat(reps, 1), a.repeat(reps, 1), g.repeat(reps))
    for x, y in zip(few, many):
        for part in y.split(500):
            assert same_bits(x, part.contiguous())


@pytest.mark.parametrize("n,h,v,k", [(700, 128, 70000, 16), (1200, 64, 40000, 40),
                                     (3000, 64, 9000, 8)])
def test_tokens_that_many_rows_list(n, h, v, k):
    # dweight's sums over many entries of a vocabulary row, some of them in every row
    hid, w, ids, a = problem(n, h, v, k, 24)
    ids = (ids.double() / v).pow(6).mul(v).long()
    for j in range(k):                                  # distinct in a row
        ids[:, j] = (ids[:, j] // k) * k + j
    ids.clamp_(max=v - 1)
    ids[:, 0] = v - 1
    mask = (torch.arange(n) % 7 != 2).to(torch.uint8)
    check(hid, w, ids, a, mask, t=1.1)


def test_a_confident_student_that_the_teacher_does_not_follow():
    # a class with p near 1 that no slot names
    n, h, v, k = 200, 128, 20000, 6
    hid, w, ids, a = problem(n, h, v, k, 25)
    other = torch.randint(0, v, (n,), generator=gen(26))
    hid = (hid.float() + 14.0 * w[other].float()).to(torch.bfloat16)
    check(hid, w, ids, a)


def test_gradient_by_differences():
    # kl(h + d) - kl(h - d) = 2 dkl.d + R, |R| <= sum g Q max|ds|^3 / 3 (a third derivative of
    # logsumexp is a third central moment, at most max|ds|^3), with steps that bf16 holds exactly
    hid, w, ids, a = problem(50, 128, 600, 10, 14)
    g = torch.rand(50, generator=gen(15)) + 0.5
    d = [x.to(dev()) for x in (hid, w, ids, a)]
    _, lse, lp = rlk.linear_topk_kl_fwd(*d)
    dh, dw = rlk.linear_topk_kl_bwd(*d, None, g.to(dev()), lse, lp)
    q = a.double().exp().sum(1).numpy()
    for which in ("hidden", "weight"):
        base = hid if which == "hidden" else w
        u = torch.randn(base.shape, generator=gen(16)) * base.float().std() * 0.05
        up, down = (base.float() + u).to(torch.bfloat16), (base.float() - u).to(torch.bfloat16)
        step = (f64(up) - f64(down)) / 2                # about the midpoint, which rounds too
        mid = (f64(up) + f64(down)) / 2 - f64(base)
        kls = []
        for other in (up, down):
            x = [other.to(dev()) if which == "hidden" else d[0],
                 other.to(dev()) if which == "weight" else d[1], *d[2:]]
            kls.append(f64(rlk.linear_topk_kl_fwd(*x)[0]))
        diff = float(np.sum(g.double().numpy() * (kls[0] - kls[1])))
        grad = f64(dh if which == "hidden" else dw)
        want = 2 * float(np.sum(grad * step))
        ds = step @ f64(w).T if which == "hidden" else f64(hid) @ step.T
        off = mid @ f64(w).T if which == "hidden" else f64(hid) @ mid.T
        big, far = np.abs(ds).max(1), np.abs(off).max(1)
        gq = g.double().numpy() * q
        # the gradient moves by at most g Q far between the midpoint and the base; its own
        # rounding is GRAD_REL_L2 of its norm along the step; each kl has an error in fp32
        bound = float(np.sum(gq * (big ** 3 / 3 + 4 * big * far + 4e-6)))
        bound += 2 * GRAD_REL_L2 * np.linalg.norm(grad) * np.linalg.norm(step)
        assert abs(diff - want) <= bound
        assert bound < 0.5 * abs(want) + 0.5 * np.linalg.norm(grad) * np.linalg.norm(step)


def test_autograd_and_its_refusals():
    hid, w, ids, a = (x.to(dev()) for x in problem(40, 64, 900, 8, 17))
    hid.requires_grad_()
    w.requires_grad_()
    weight = torch.rand(40, generator=gen(18)).to(dev())
    kl = rlk.linear_topk_kl(hid, w, ids, a, None, 1.2, True)
    (kl * weight).sum().backward()
    _, lse, lp = rlk.linear_topk_kl_fwd(hid.detach(), w.detach(), ids, a, None, 1.2, True)
    dh, dw = rlk.linear_topk_kl_bwd(hid.detach(), w.detach(), ids, a, None, weight, lse, lp, 1.2,
                                    True)
    assert same_bits(hid.grad, dh) and same_bits(w.grad, dw)
    gh, = torch.autograd.grad(rlk.linear_topk_kl(hid, w, ids, a).sum(), hid, create_graph=True)
    with pytest.raises(RuntimeError):
        gh.square().sum().backward()


def test_captured_step():
    hid, w, ids, a = (x.to(dev()) for x in problem(64, 128, 5000, 16, 19))
    g = torch.rand(64, generator=gen(20)).to(dev())

    def step():
        kl, lse, lp = rlk.linear_topk_kl_fwd(hid, w, ids, a)
        return (kl, *rlk.linear_topk_kl_bwd(hid, w, ids, a, None, g, lse, lp))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    other = problem(64, 128, 5000, 16, 21)
    for to, x in zip((hid, w, ids, a), other):
        to.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    for got, want in zip(out, step()):
        assert same_bits(got, want)


def test_no_rows():
    hid, w, ids, a = (x.to(dev()) for x in problem(3, 64, 300, 4, 22))
    hid = hid[:0].clone().requires_grad_()
    w.requires_grad_()
    kl = rlk.linear_topk_kl(hid, w, ids[:0], a[:0])
    kl.sum().backward()
    assert kl.shape == (0,) and hid.grad.shape == (0, 64) and not bool(w.grad.any())


def test_temperatures_at_the_ends_of_their_range():
    hid, w, ids, a = (x.to(dev()) for x in problem(5, 64, 300, 4, 23))
    kl, lse, lp = rlk.linear_topk_kl_fwd(hid, w, ids, a, None, 1e30)
    # every logit is 0: p = 1/300, and the columns that fill the last tile up do not count
    assert torch.all((lse - np.log(300)).abs() <= LOGP_ATOL)
    assert torch.all((lp + np.log(300)).abs() <= LOGP_ATOL)
    g = torch.rand(5, generator=gen(24)).to(dev())
    for t in (1e30, 1e-4):         # below, 1e-30 too, is refused
        kl, lse, lp = rlk.linear_topk_kl_fwd(hid, w, ids, a, None, t)
        dh, dw = rlk.linear_topk_kl_bwd(hid, w, ids, a, None, g, lse, lp, t)
        for x in (kl, lse, lp, dh, dw):
            assert bool(torch.isfinite(x.float()).all())


def test_two_streams():
    # odd sizes and a mask, each on a stream of its own, against the same calls by themselves
    many = []
    for n, v, seed in ((130, 9001, 25), (70, 20000, 26)):
        hid, w, ids, a = (x.to(dev()) for x in problem(n, 128, v, 9, seed))
        g = torch.rand(n, generator=gen(seed)).to(dev())
        mask = (torch.rand(n, generator=gen(seed + 2)) < 0.7).to(torch.uint8).to(dev())
        many.append((hid, w, ids, a, mask, g))

    def step(hid, w, ids, a, mask, g):
        kl, lse, lp = rlk.linear_topk_kl_fwd(hid, w, ids, a, mask)
        return (kl, *rlk.linear_topk_kl_bwd(hid, w, ids, a, mask, g, lse, lp))

    want = [step(*x) for x in many]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in many]
    got = []
    for _ in range(5):
        for x, s in zip(many, streams):
            with torch.cuda.stream(s):
                got.append(step(*x))
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert all(same_bits(p, q) for p, q in zip(out, want[i % 2]))


def test_offsets_past_32_bits():
    check(*problem(70000, 64, 300, 2, 27))       # dS alone: 70000 rows of 2^16 entries


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("n,v", [(1, 700), (3, 9001), (15, 40000), (16, 700), (17, 9001)])
def test_whatever_the_workspace_holds(n, v, masked):
    # NaN everywhere on entry: nothing of it reaches the results (rows of maps past N, planes of dS)
    hid, w, ids, a = problem(n, 128, v, 6, 28)
    mask = (torch.arange(n) % 3 != 1).to(torch.uint8) if masked else None
    g = torch.randn(n, generator=gen(29)) / n
    kl, lse, lp, dh, dw = check(hid, w, ids, a, mask, 1.1, False, g)
    d = [x if x is None else x.to(dev()) for x in (hid, w, ids, a, mask)]
    for fill in (255, 0):
        out = [torch.full_like(x, float("nan")) for x in (kl, lse, lp, dh, dw)]
        ws = [torch.full((max(q(n, 128, v, 6), 256),), fill, dtype=torch.uint8, device=dev())
              for q in (rlk.rlk_linear_topk_kl_fwd_workspace_bytes,
                        rlk.rlk_linear_topk_kl_bwd_workspace_bytes)]
        rlk.rlk_linear_topk_kl_fwd(*d, 1.1, False, *out[:3], ws[0])
        rlk.rlk_linear_topk_kl_bwd(*d, g.to(dev()), out[1], out[2], 1.1, False, *out[3:], ws[1])
        for got, want in zip(out, (kl, lse, lp, dh, dw)):
            assert same_bits(got, want)
