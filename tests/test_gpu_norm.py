"""Layer norm and RMS norm against the definition in float64.

Tolerances count roundings.  fp32 sums: no value passes more than 128 additions on its way
into a row's mean or variance (32 to 40 in a thread, 5 in the shuffle tree, up to 31 across
warps), nor more than 256 into dweight (rows of a block, then the partial rows), so a sum of
terms a_i is off by at most 128 (256) x 2^-24 x sum |a_i|; the few multiplications beside it
are in the slack of that bound.  The output's own rounding adds half a step of its type.
"""
import numpy as np
import pytest
import torch

import rl_post_linear_gb300 as rlk
from helpers import dev, same_bits

pytestmark = pytest.mark.gpu

EPS = 1e-6
U32 = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BF16, F32 = torch.bfloat16, torch.float32


def make(n, h, dtype, seed, wdtype=None, pad=0, offset=0):
    """x, dy as [n, h] views (row stride h + pad, starting `offset` elements into the buffer)."""
    g = torch.Generator().manual_seed(seed)
    wide = h + pad

    def rows(scale, shift):
        flat = torch.randn(n * wide + offset, generator=g) * scale + shift
        flat = flat.to(dtype).to(dev())
        return flat[offset:].view(n, wide)[:, :h]

    x, dy = rows(1.5, 2.0), rows(0.01, 0.0)
    wdtype = wdtype or dtype
    w = (1 + 0.3 * torch.randn(h, generator=g)).to(wdtype).to(dev())
    b = (0.2 * torch.randn(h, generator=g)).to(wdtype).to(dev())
    return x, dy, w, b


def d64(t):
    return t.detach().double().cpu()


def ref_fwd(x, w, b, layer):
    x, w = d64(x), d64(w)
    mean = x.mean(1, keepdim=True) if layer else torch.zeros(x.shape[0], 1, dtype=torch.float64)
    rstd = ((x - mean) ** 2).mean(1, keepdim=True).add(EPS).rsqrt()
    y = (x - mean) * rstd * w
    return (y + d64(b) if b is not None else y), mean, rstd


def check_fwd(x, w, b, mask, y, mean, rstd, layer):
    yr, mr, rr = ref_fwd(x, w, b, layer)
    on = torch.ones(x.shape[0], dtype=torch.bool) if mask is None else mask.cpu() > 0
    base = yr - d64(b) if b is not None else yr
    size = d64(x).abs().mean(1, keepdim=True)
    tol = HALF_STEP[x.dtype] * yr.abs() + 128 * U32 * (
        base.abs() + yr.abs() + rr * d64(w).abs() * size)
    assert bool(((d64(y) - yr).abs() <= tol)[on].all())
    assert bool((d64(y)[~on] == 0).all())
    assert bool(((d64(rstd) - rr[:, 0]).abs() <= 128 * U32 * rr[:, 0])[on].all())
    assert bool((d64(rstd)[~on] == 0).all())
    if layer:
        assert bool(((d64(mean) - mr[:, 0]).abs() <= 128 * U32 * size[:, 0])[on].all())
        assert bool((d64(mean)[~on] == 0).all())


def check_bwd(x, w, dy, mean, rstd, mask, dx, dw, db, layer):
    on = torch.ones(x.shape[0], dtype=torch.bool) if mask is None else mask.cpu() > 0
    xs, g = d64(x)[on], d64(dy)[on]
    m = d64(mean)[on][:, None] if layer else 0.0
    r = d64(rstd)[on][:, None]
    xh = (xs - m) * r
    gw = g * d64(w)
    h = x.shape[1]
    m1 = gw.sum(1, keepdim=True) / h if layer else torch.zeros_like(r)
    m2 = (gw * xh).sum(1, keepdim=True) / h
    dxr = r * (gw - m1 - xh * m2)
    slack = r * (gw.abs() + gw.abs().mean(1, keepdim=True)
                 + xh.abs() * (gw * xh).abs().mean(1, keepdim=True))
    tol = HALF_STEP[x.dtype] * dxr.abs() + 128 * U32 * slack
    assert bool(((d64(dx)[on] - dxr).abs() <= tol).all())
    assert bool((d64(dx)[~on] == 0).all())
    for got, terms in ((dw, g * xh), (db, g)):
        if got is None:
            continue
        ref = terms.sum(0)
        # xh itself is off by (x - mean)'s rounding, in units of |mean| where that is larger
        tol = HALF_STEP[w.dtype] * ref.abs() + 256 * U32 * terms.abs().sum(0)
        assert bool(((d64(got) - ref).abs() <= tol).all())


def run_all(n, h, dtype, layer, seed, wdtype=None, pad=0, offset=0, mask=None, bias=True):
    x, dy, w, b = make(n, h, dtype, seed, wdtype, pad, offset)
    if mask is not None:                 # what a masked row holds must not matter
        x[mask == 0] = float("nan")
        dy[mask == 0] = float("nan")
    if layer:
        b = b if bias else None
        y, mean, rstd = rlk.layer_norm_fwd(x, w, b, EPS, mask)
        dx, dw, db = rlk.layer_norm_bwd(x, w, dy, mean, rstd, mask, with_bias=bias)
    else:
        b = mean = db = None
        y, rstd = rlk.rms_norm_fwd(x, w, EPS, mask)
        dx, dw = rlk.rms_norm_bwd(x, w, dy, rstd, mask)
    torch.cuda.synchronize()
    check_fwd(x, w, b, mask, y, mean, rstd, layer)
    check_bwd(x, w, dy, mean, rstd, mask, dx, dw, db, layer)
    return y, mean, rstd, dx, dw, db


WIDTHS = [1, 2, 7, 8, 9, 63, 64, 256, 257, 512, 513, 1000, 1024, 1025, 2048, 2049, 4096, 4097,
          7168, 8192, 8193, 16384, 16385, 20001]


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("h", WIDTHS)
def test_widths(h, dtype, layer):
    run_all(5, h, dtype, layer, h)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("n,h", [(1, 4096), (3, 300), (700, 256), (2500, 1000), (1300, 2048),
                                 (1500, 4096), (640, 7168), (330, 9000), (310, 16400)])
def test_row_counts(n, h, layer):
    # around and beyond the backward's number of blocks
    run_all(n, h, BF16, layer, n + h)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("dtype,wdtype", [(BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("h", [96, 1537, 4096, 16388])
def test_parameter_type_differs(h, dtype, wdtype, layer):
    run_all(9, h, dtype, layer, h, wdtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("h,pad,offset", [(256, 8, 0), (1000, 3, 0), (4096, 0, 1), (4096, 5, 3),
                                          (7168, 16, 2), (16392, 1, 0)])
def test_strides_and_offsets(h, pad, offset, dtype):
    run_all(6, h, dtype, True, h + pad, pad=pad, offset=offset)
    run_all(6, h, dtype, False, h + offset, pad=pad, offset=offset, bias=False)


@pytest.mark.parametrize("h", [40, 1024, 4096, 8192, 17000])
@pytest.mark.parametrize("kind", ["some", "none", "one"])
def test_masks(kind, h):
    n = 37
    mask = torch.zeros(n, dtype=torch.uint8)
    if kind == "some":
        mask = (torch.rand(n, generator=torch.Generator().manual_seed(3)) < 0.6).to(torch.uint8) * 7
    elif kind == "one":
        mask[20] = 1
    for layer in (True, False):
        out = run_all(n, h, BF16, layer, 11, mask=mask.to(dev()))
        if kind == "none":
            assert float(out[4].float().abs().max()) == 0.0


def test_no_rows():
    x = torch.empty(0, 128, dtype=BF16, device=dev())
    w = torch.ones(128, dtype=BF16, device=dev())
    y, mean, rstd = rlk.layer_norm_fwd(x, w)
    dx, dw, db = rlk.layer_norm_bwd(x, w, x, mean, rstd)
    assert y.shape == (0, 128) and float(dw.abs().max()) == 0 and float(db.abs().max()) == 0
    dx, dw = rlk.rms_norm_bwd(x, w, x, rstd)
    assert dx.shape == (0, 128) and float(dw.abs().max()) == 0


def test_constant_rows_and_large_mean():
    # zero variance: y = b and finite gradients; a mean of 1000 costs no digits of the variance
    w = torch.full((513,), 1.5, device=dev())
    b = torch.linspace(-1, 1, 513, device=dev())
    x = torch.full((3, 513), 7.0, device=dev())
    y, mean, rstd = rlk.layer_norm_fwd(x, w, b, EPS)
    assert torch.allclose(y, b.expand(3, -1), rtol=0, atol=1e-3)
    dx, dw, db = rlk.layer_norm_bwd(x, w, torch.ones_like(x), mean, rstd)
    assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())
    z = 1000.0 + torch.randn(4, 513, device=dev(), generator=torch.Generator("cuda").manual_seed(1))
    y, mean, rstd = rlk.layer_norm_fwd(z, w, b, EPS)
    check_fwd(z, w, b, None, y, mean, rstd, True)
    zero = torch.zeros(2, 4096, device=dev(), dtype=BF16)
    y, rstd = rlk.rms_norm_fwd(zero, torch.ones(4096, device=dev(), dtype=BF16), EPS)
    assert float(y.abs().max()) == 0.0 and float((rstd - 1e3).abs().max()) < 1e-2


def test_nan_stays_in_its_row():
    x, dy, w, b = make(6, 1000, BF16, 5)
    good = rlk.layer_norm_fwd(x, w, b, EPS)[0].clone()
    x[2, 17] = float("nan")
    y = rlk.layer_norm_fwd(x, w, b, EPS)[0]
    keep = [0, 1, 3, 4, 5]
    assert same_bits(y[keep].cpu(), good[keep].cpu()) and bool(torch.isnan(y[2]).all())


@pytest.mark.parametrize("h", [300, 4096, 7168, 16500])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_do_not_depend_on_batch_or_alignment(h, dtype):
    x, dy, w, b = make(700, h, dtype, 9)
    y, mean, rstd = rlk.layer_norm_fwd(x, w, b, EPS)
    dx, dw, db = rlk.layer_norm_bwd(x, w, dy, mean, rstd)
    again = rlk.layer_norm_bwd(x, w, dy, mean, rstd)
    for p, q in zip((dx, dw, db), again):
        assert same_bits(p.cpu(), q.cpu())

    def shifted(t):
        buf = torch.empty(41 * h + 1, dtype=dtype, device=dev())
        v = buf[1:].view(41, h)
        v.copy_(t[600:641])
        return v

    xs, gs = shifted(x), shifted(dy)
    ys, ms, rs = rlk.layer_norm_fwd(xs, w, b, EPS)
    ds, _, _ = rlk.layer_norm_bwd(xs, w, gs, ms, rs)
    for p, q in ((ys, y), (ms, mean), (rs, rstd), (ds, dx)):
        assert same_bits(p.cpu(), q[600:641].cpu())


def test_mask_equals_dropping_the_rows():
    x, dy, w, b = make(90, 4096, BF16, 21)
    mask = (torch.arange(90) % 3 != 0).to(torch.uint8).to(dev())
    y, rstd = rlk.rms_norm_fwd(x, w, EPS, mask)
    dx, _ = rlk.rms_norm_bwd(x, w, dy, rstd, mask)
    on = mask > 0
    y2, rstd2 = rlk.rms_norm_fwd(x[on].contiguous(), w, EPS)
    dx2, _ = rlk.rms_norm_bwd(x[on].contiguous(), w, dy[on].contiguous(), rstd2)
    assert same_bits(y[on].cpu(), y2.cpu()) and same_bits(dx[on].cpu(), dx2.cpu())


@pytest.mark.parametrize("layer", [True, False])
def test_gradient_against_differences(layer):
    # (L(p + s v) - L(p - s v)) / 2s of the float64 forward, along random directions v
    n, h, s = 6, 257, 1e-5
    x, dy, w, b = make(n, h, F32, 31)
    if layer:
        _, mean, rstd = rlk.layer_norm_fwd(x, w, b, EPS)
        dx, dw, db = rlk.layer_norm_bwd(x, w, dy, mean, rstd)
    else:
        _, rstd = rlk.rms_norm_fwd(x, w, EPS)
        dx, dw = rlk.rms_norm_bwd(x, w, dy, rstd)
    g = torch.Generator().manual_seed(2)

    def loss(xd, wd, bd):
        return float((ref_fwd(xd, wd, bd if layer else None, layer)[0] * d64(dy)).sum())

    for which, grad in (("x", dx), ("w", dw)) + ((("b", db),) if layer else ()):
        p = {"x": d64(x), "w": d64(w), "b": d64(b)}
        v = torch.randn(p[which].shape, generator=g, dtype=torch.float64)
        hi, lo = dict(p), dict(p)
        hi[which], lo[which] = p[which] + s * v, p[which] - s * v
        diff = (loss(hi["x"], hi["w"], hi["b"]) - loss(lo["x"], lo["w"], lo["b"])) / (2 * s)
        along = float((d64(grad) * v).sum())
        # differences: O(s^2) of third derivatives and 2^-52 / s of cancellation, both < 1e-8
        # of the gradient's size; the gradient itself 256 x 2^-24
        size = float(d64(grad).norm() * v.norm())
        assert abs(along - diff) <= (256 * U32 + 1e-6) * size


def test_autograd_of_leading_axes_and_expanded_gradients():
    x, _, w, b = make(24, 640, BF16, 41)
    x3 = x.reshape(4, 6, 640).detach().requires_grad_()
    w.requires_grad_(), b.requires_grad_()
    y = rlk.layer_norm(x3, w, b, EPS)
    assert y.shape == x3.shape
    y.sum().backward()                     # an expanded gradient of stride 0
    ones = torch.ones(24, 640, dtype=BF16, device=dev())
    _, mean, rstd = rlk.layer_norm_fwd(x, w.detach(), b.detach(), EPS)
    dx, dw, db = rlk.layer_norm_bwd(x, w.detach(), ones, mean, rstd)
    assert same_bits(x3.grad.reshape(24, 640).cpu(), dx.cpu())
    assert same_bits(w.grad.cpu(), dw.cpu()) and same_bits(b.grad.cpu(), db.cpu())
    xt = x.detach().reshape(4, 6, 640).transpose(0, 1).requires_grad_()
    w2 = w.detach().clone().requires_grad_()
    rlk.rms_norm(xt, w2, EPS).float().square().sum().backward()
    assert xt.grad.shape == xt.shape and bool(torch.isfinite(w2.grad).all())
    frozen = rlk.rms_norm(x3.detach().requires_grad_(), w.detach(), EPS)
    frozen.sum().backward()                # the weight asks for no gradient


def test_captured_training_step_beside_a_live_eager_graph():
    # autograd keeps a leaf's accumulation on the stream of the first live graph that used it,
    # for every operator alike: the eager graph is made on the stream that is captured
    x, dy, w, b = make(200, 1024, BF16, 51)
    xl, wl_, bl = (t.detach().clone().requires_grad_() for t in (x, w, b))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        alive = rlk.layer_norm(xl, wl_, bl, EPS)      # an eager graph of the same leaves
        torch.autograd.grad(rlk.layer_norm(xl, wl_, bl, EPS), (xl, wl_, bl), dy)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        grads = torch.autograd.grad(rlk.layer_norm(xl, wl_, bl, EPS), (xl, wl_, bl), dy)
    other = x.flip(0).contiguous()
    with torch.no_grad():
        xl.data.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    _, mean, rstd = rlk.layer_norm_fwd(other, w, b, EPS)
    want = rlk.layer_norm_bwd(other, w, dy, mean, rstd)
    for p, q in zip(grads, want):
        assert same_bits(p.cpu(), q.cpu())
    assert alive.requires_grad


def test_another_stream():
    x, dy, w, b = make(300, 4096, BF16, 61)
    want = rlk.layer_norm_fwd(x, w, b, EPS)
    side = torch.cuda.Stream()
    y = torch.empty_like(want[0])
    mean, rstd = torch.empty_like(want[1]), torch.empty_like(want[2])
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(rlk.rlk_layer_norm_bwd_workspace_bytes(300, 4096), dtype=torch.uint8,
                     device=dev())
    side.wait_stream(torch.cuda.current_stream())
    rlk.rlk_layer_norm_fwd(x, w, b, None, EPS, y, mean, rstd, stream=side)
    rlk.rlk_layer_norm_bwd(x, w, dy, mean, rstd, None, dx, dw, db, ws, stream=side)
    side.synchronize()
    assert same_bits(y.cpu(), want[0].cpu())
    check_bwd(x, w, dy, mean, rstd, None, dx, dw, db, True)


def test_workspace_size_is_enough_at_its_edge():
    # the byte count asked for, in a buffer with a guard behind it
    for n, h in ((5, 8), (700, 1000), (1000, 4096), (400, 7168), (200, 16384), (160, 16390)):
        x, dy, w, b = make(n, h, BF16, n)
        _, mean, rstd = rlk.layer_norm_fwd(x, w, b, EPS)
        need = rlk.rlk_layer_norm_bwd_workspace_bytes(n, h)
        buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=dev())
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
        rlk.rlk_layer_norm_bwd(x, w, dy, mean, rstd, None, dx, dw, db, buf[:need])
        assert bool((buf[need:] == 0xA5).all())
        check_bwd(x, w, dy, mean, rstd, None, dx, dw, db, True)
