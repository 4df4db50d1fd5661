"""Refusals of the norm and sampling entry points: argument errors are returned before
anything is enqueued, so these run without a GPU (explicit failure, no fallback)."""
import ctypes
import math

import pytest
import torch

import rl_post_linear_gb300 as rlk
from rl_post_linear_gb300 import build as rlk_build

FAKE = 1 << 20          # aligned, not null; validation never dereferences
F32, BF16 = rlk.RLK_DTYPE_F32, rlk.RLK_DTYPE_BF16
OK, INVALID, UNSUPPORTED, WORKSPACE = (rlk.RLK_OK, rlk.RLK_ERR_INVALID_VALUE,
                                       rlk.RLK_ERR_UNSUPPORTED, rlk.RLK_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    rlk_build.build()
    return rlk.load()


FWD = [("x", FAKE), ("x_dtype", BF16), ("x_stride", 96), ("weight", FAKE), ("bias", None),
       ("w_dtype", BF16), ("mask", None), ("N", 4), ("H", 96), ("eps", 1e-6), ("y", FAKE),
       ("y_stride", 96), ("mean", None), ("rstd", None), ("stream", None)]
BWD = [("x", FAKE), ("x_dtype", BF16), ("x_stride", 96), ("weight", FAKE), ("w_dtype", BF16),
       ("dy", FAKE), ("dy_stride", 96), ("mean", FAKE), ("rstd", FAKE), ("mask", None), ("N", 4),
       ("H", 96), ("dx", FAKE), ("dx_stride", 96), ("dw", FAKE), ("db", None), ("ws", FAKE),
       ("ws_bytes", 1 << 30), ("stream", None)]


def call(fn, spec, drop=(), **kw):
    a = dict(spec)
    assert set(kw) <= set(a)
    a.update(kw)
    return fn(*[a[k] for k, _ in spec if k not in drop])


NORM_BAD = [({"x_dtype": 2}, UNSUPPORTED), ({"w_dtype": -1}, UNSUPPORTED), ({"H": 0}, INVALID),
            ({"N": -1}, INVALID), ({"N": 1 << 31}, INVALID), ({"x_stride": 95}, INVALID),
            ({"x": None}, INVALID), ({"weight": None}, INVALID), ({"x": FAKE + 1}, INVALID),
            ({"weight": FAKE + 1}, INVALID),
            ({"x_dtype": F32, "x": FAKE + 2}, INVALID)]


@pytest.mark.parametrize("kw,status", NORM_BAD + [
    ({"y_stride": 10}, INVALID), ({"y": None}, INVALID), ({"eps": -1.0}, INVALID),
    ({"eps": math.nan}, INVALID), ({"eps": math.inf}, INVALID), ({"N": 0, "x": None}, OK)])
def test_forward_refusals(lib, kw, status):
    assert call(lib.rlk_layer_norm_fwd, FWD, **kw) == status
    assert call(lib.rlk_rms_norm_fwd, FWD, ("bias", "mean"), **kw) == status


def test_layer_norm_bias_alignment(lib):
    assert call(lib.rlk_layer_norm_fwd, FWD, bias=FAKE + 1) == INVALID
    wide = {"H": (1 << 24) + 1, "x_stride": 1 << 25, "y_stride": 1 << 25}
    assert call(lib.rlk_layer_norm_fwd, FWD, **wide) == UNSUPPORTED


@pytest.mark.parametrize("kw,status", NORM_BAD + [
    ({"dy": None}, INVALID), ({"dx": None}, INVALID), ({"rstd": None}, INVALID),
    ({"dy_stride": 1}, INVALID), ({"dx_stride": 95}, INVALID), ({"dy": FAKE + 1}, INVALID),
    ({"dx": FAKE + 1}, INVALID), ({"dw": FAKE + 1}, INVALID), ({"ws": None}, WORKSPACE),
    ({"ws": FAKE + 8}, WORKSPACE), ({"ws_bytes": 256}, WORKSPACE)])
def test_backward_refusals(lib, kw, status):
    assert call(lib.rlk_layer_norm_bwd, BWD, **kw) == status
    assert call(lib.rlk_rms_norm_bwd, BWD, ("mean", "db"), **kw) == status


def test_backward_only_layer_norm(lib):
    assert call(lib.rlk_layer_norm_bwd, BWD, mean=None) == INVALID
    assert call(lib.rlk_layer_norm_bwd, BWD, db=FAKE + 1) == INVALID
    assert call(lib.rlk_layer_norm_bwd, BWD, N=0, dw=None, x=None) == OK
    need = rlk.rlk_layer_norm_bwd_workspace_bytes(4, 96)
    assert call(lib.rlk_layer_norm_bwd, BWD, ws_bytes=need - 1) == WORKSPACE


def test_workspace_queries(lib):
    # fp32 planes (two for layer norm) of at most 304 partial rows at this width, a row padded
    # to the 16 columns of each of its threads
    assert rlk.rlk_layer_norm_bwd_workspace_bytes(8192, 4096) == 2 * 304 * 4096 * 4 + 256
    assert rlk.rlk_rms_norm_bwd_workspace_bytes(8192, 4096) == 304 * 4096 * 4 + 256
    assert rlk.rlk_rms_norm_bwd_workspace_bytes(3, 4096) == 3 * 4096 * 4 + 256
    assert rlk.rlk_rms_norm_bwd_workspace_bytes(2, 4097) >= 2 * 4097 * 4
    assert rlk.rlk_layer_norm_bwd_workspace_bytes(-1, 8) == 0
    assert rlk.rlk_layer_norm_bwd_workspace_bytes(8, 0) == 0
    assert rlk.rlk_sample_logits_workspace_bytes(-1, 8) == 0
    assert rlk.rlk_sample_logits_workspace_bytes(4, 0) == 0
    assert ctypes.sizeof(rlk.SampleParams) == 64


def sample(lib, params=None, **kw):
    a = dict(logits=FAKE, dtype=F32, N=4, V=1000, stride=1000, u=FAKE, mask=None, tokens=FAKE,
             logp=FAKE, kept=FAKE, ws=FAKE, ws_bytes=1 << 40, err=None, stream=None)
    a.update(kw)
    s = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    s.update(params or {})
    p = rlk.SampleParams(None, None, None, None, s["temperature"], s["top_k"], s["top_p"],
                         s["min_p"])
    ref = None if params is False else ctypes.byref(p)
    return lib.rlk_sample_logits(a["logits"], a["dtype"], a["N"], a["V"], a["stride"], a["u"],
                                 a["mask"], ref, a["tokens"], a["logp"], a["kept"], a["ws"],
                                 a["ws_bytes"], a["err"], a["stream"])


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 2}, UNSUPPORTED), ({"N": -1}, INVALID), ({"N": 1 << 31}, INVALID),
    ({"V": 0}, INVALID), ({"stride": 999}, INVALID), ({"logits": None}, INVALID),
    ({"u": None}, INVALID), ({"tokens": None}, INVALID), ({"logits": FAKE + 2}, INVALID),
    ({"V": (1 << 22) + 1, "stride": 1 << 23}, UNSUPPORTED), ({"params": False}, INVALID),
    ({"N": 0, "logits": None}, OK)])
def test_sampling_refusals(lib, kw, status):
    assert sample(lib, **kw) == status


@pytest.mark.parametrize("params", [
    {"temperature": 0.0}, {"temperature": -1.0}, {"temperature": math.nan},
    {"temperature": math.inf}, {"temperature": 1e-7}, {"temperature": 2e6}, {"top_k": -1},
    {"top_p": 0.0}, {"top_p": -0.5}, {"top_p": math.nan}, {"min_p": -0.1}, {"min_p": 1.1},
    {"min_p": math.nan}])
def test_sampling_settings_out_of_range(lib, params):
    assert sample(lib, params) == INVALID
    assert sample(lib, params, N=0) == INVALID


def test_binding_refuses_what_it_cannot_pass_on(lib):
    x = torch.zeros(4, 64)
    w = torch.ones(64)
    with pytest.raises(ValueError):
        rlk.layer_norm_fwd(x, w)                                # not on a GPU
    with pytest.raises(ValueError):
        rlk.sample_logits(x, torch.zeros(4))
    with pytest.raises(ValueError):
        rlk.rms_norm_fwd(x, w)


@pytest.mark.parametrize("wrt", ["x", "weight", "grad"])
@pytest.mark.parametrize("norm", ["layer_norm", "rms_norm"])
def test_second_derivatives_are_refused(monkeypatch, lib, norm, wrt):
    # the launches stood in for; a gradient of the gradient has no kernel, so it must not read as 0
    def forward(x, weight, *_):
        return (x * weight,) + (torch.ones(x.shape[0]),) * (2 if norm == "layer_norm" else 1)

    def backward(*args):
        args[6 if norm == "layer_norm" else 5].fill_(1.0)           # dx

    monkeypatch.setattr(rlk, norm + "_fwd", forward)
    monkeypatch.setattr(rlk, "rlk_%s_bwd" % norm, backward)
    t = {"x": torch.randn(2, 3, 8), "weight": torch.ones(8), "grad": torch.randn(2, 3, 8)}
    t["x"].requires_grad_()
    t[wrt].requires_grad_()
    y = getattr(rlk, norm)(t["x"], t["weight"])
    dx, = torch.autograd.grad(y, t["x"], t["grad"], retain_graph=True)
    assert bool((dx == 1.0).all()) and not dx.requires_grad
    dx, = torch.autograd.grad(y, t["x"], t["grad"], create_graph=True)
    assert bool((dx == 1.0).all())
    loss = dx.square().sum() + (t[wrt] ** 3).sum()
    with pytest.raises(RuntimeError, match="differentiated once"):
        torch.autograd.grad(loss, t[wrt])


def test_arrays_have_to_be_aligned_to_their_elements(lib):
    # a kernel that reads or writes them would fault
    for name in ("mean", "rstd"):
        for at in (1, 2, 3):
            assert call(lib.rlk_layer_norm_fwd, FWD, **{name: FAKE + at}) == INVALID
            assert call(lib.rlk_layer_norm_bwd, BWD, **{name: FAKE + at}) == INVALID
    assert call(lib.rlk_rms_norm_fwd, FWD, ("bias", "mean"), rstd=FAKE + 2) == INVALID
    assert call(lib.rlk_rms_norm_bwd, BWD, ("mean", "db"), rstd=FAKE + 2) == INVALID
    for name in ("u", "tokens", "logp", "kept", "err"):
        assert sample(lib, **{name: FAKE + 2}) == INVALID
    assert sample(lib, tokens=FAKE + 4) == INVALID
    for i in range(4):
        rows = [None] * 4
        rows[i] = FAKE + 2
        p = rlk.SampleParams(*rows, 1.0, 0, 1.0, 0.0)
        assert lib.rlk_sample_logits(FAKE, F32, 4, 1000, 1000, FAKE, None, ctypes.byref(p), FAKE,
                                     FAKE, FAKE, FAKE, 1 << 40, None, None) == INVALID


def test_scalar_top_k_reaches_the_kernel_as_it_is():
    def passed(top_k):
        return rlk._sample_params(4, 1.0, top_k, 1.0, 0.0).top_k

    assert passed(50) == passed(50.0) == passed(torch.tensor([50])[0].item()) == 50
    assert passed(1 << 64) >= 1 << 22 and passed((1 << 64) + 5) >= 1 << 22       # off
    assert passed(-(1 << 64) + 5) < 0                                           # refused
    for bad in (2.7, math.nan, math.inf):
        with pytest.raises((ValueError, OverflowError)):
            passed(bad)
