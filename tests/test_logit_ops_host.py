"""Refusals of the logit processing, top-k and top-k KL entry points: argument errors are returned
before anything is enqueued, so these run without a GPU."""
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


def process(lib, params=(), **kw):
    a = dict(logits=FAKE, dtype=F32, N=4, V=1000, stride=1000, mask=None, out=FAKE + (1 << 16),
             out_stride=1000, err=None, stream=None)
    assert set(kw) <= set(a) | {"params_ref"}
    p = dict(repetition=1.1, tokens=FAKE, tokens_width=8, tokens_stride=8)
    p.update(params)
    ref = kw.pop("params_ref", ctypes.byref(rlk.ProcessParams(**p)))
    a.update(kw)
    return lib.rlk_process_logits(a["logits"], a["dtype"], a["N"], a["V"], a["stride"], a["mask"],
                                  ref, a["out"], a["out_stride"], a["err"], a["stream"])


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 2}, UNSUPPORTED), ({"N": -1}, INVALID), ({"N": 1 << 31}, INVALID),
    ({"V": 0}, INVALID), ({"stride": 999}, INVALID), ({"out_stride": 999}, INVALID),
    ({"logits": None}, INVALID), ({"out": None}, INVALID), ({"logits": FAKE + 2}, INVALID),
    ({"out": FAKE + 1}, INVALID), ({"err": FAKE + 2}, INVALID), ({"params_ref": None}, INVALID),
    ({"out": FAKE, "out_stride": 1001}, INVALID),
    ({"V": (1 << 22) + 1, "stride": 1 << 23, "out_stride": 1 << 23}, UNSUPPORTED),
    ({"N": 0, "logits": None}, OK)])
def test_processing_refusals(lib, kw, status):
    assert process(lib, **kw) == status


@pytest.mark.parametrize("params,status", [
    ({"repetition": 0.0}, INVALID), ({"repetition": -1.0}, INVALID),
    ({"repetition": math.nan}, INVALID), ({"repetition": math.inf}, INVALID),
    ({"repetition": 1e-60}, INVALID), ({"repetition": 1e60}, INVALID),
    ({"frequency": math.nan}, INVALID), ({"frequency": math.inf}, INVALID),
    ({"presence": math.nan}, INVALID), ({"presence": -1e60}, INVALID),
    ({"tokens_width": -1}, INVALID), ({"tokens_stride": 7}, INVALID),
    ({"tokens_width": (1 << 29) + 1, "tokens_stride": 1 << 30}, UNSUPPORTED),
    ({"tokens": None}, INVALID), ({"tokens": None, "lengths": FAKE}, INVALID),
    ({"bias_count": -1}, INVALID),
    ({"bias_count": 4097, "bias_ids": FAKE, "bias_values": FAKE}, UNSUPPORTED),
    ({"bias_count": 1, "bias_ids": FAKE}, INVALID),
    ({"bias_count": 1, "bias_values": FAKE}, INVALID),
    ({"allowed": FAKE, "allowed_stride": 31}, INVALID), ({"tokens": FAKE + 4}, INVALID),
    ({"lengths": FAKE + 4}, INVALID), ({"prompt_lengths": FAKE + 4}, INVALID),
    ({"repetition_rows": FAKE + 2}, INVALID), ({"frequency_rows": FAKE + 2}, INVALID),
    ({"presence_rows": FAKE + 2}, INVALID), ({"allowed": FAKE + 2, "allowed_stride": 32}, INVALID),
    ({"bias_count": 1, "bias_ids": FAKE + 4, "bias_values": FAKE}, INVALID),
    ({"bias_count": 1, "bias_ids": FAKE, "bias_values": FAKE + 2}, INVALID)])
def test_processing_settings(lib, params, status):
    assert process(lib, params) == status


TOPK = [("logits", FAKE), ("dtype", F32), ("N", 4), ("V", 1000), ("stride", 1000), ("mask", None),
        ("K", 20), ("T", 1.0), ("ids", FAKE), ("logp", FAKE), ("lse", FAKE), ("err", None),
        ("stream", None)]
FWD = [("hidden", FAKE), ("weight", FAKE), ("ids", FAKE), ("teacher", FAKE), ("mask", None),
       ("N", 4), ("H", 64), ("V", 1000), ("K", 20), ("T", 1.0), ("renorm", 0), ("kl", FAKE),
       ("lse", FAKE), ("logp", FAKE), ("ws", FAKE), ("ws_bytes", 1 << 40), ("err", None),
       ("stream", None)]
BWD = [("hidden", FAKE), ("weight", FAKE), ("ids", FAKE), ("teacher", FAKE), ("mask", None),
       ("grad", FAKE), ("lse", FAKE), ("logp", FAKE), ("N", 4), ("H", 64), ("V", 1000), ("K", 20),
       ("T", 1.0), ("renorm", 0), ("dh", FAKE), ("dw", FAKE), ("ws", FAKE), ("ws_bytes", 1 << 40),
       ("err", None), ("stream", None)]


def call(fn, spec, **kw):
    a = dict(spec)
    assert set(kw) <= set(a)
    a.update(kw)
    return fn(*[a[k] for k, _ in spec])


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 5}, UNSUPPORTED), ({"N": -1}, INVALID), ({"N": 1 << 31}, INVALID),
    ({"V": 0}, INVALID), ({"stride": 999}, INVALID), ({"K": 0}, INVALID), ({"K": -3}, INVALID),
    ({"K": 1025}, UNSUPPORTED), ({"V": (1 << 22) + 1, "stride": 1 << 23}, UNSUPPORTED),
    ({"T": 0.0}, INVALID), ({"T": -1.0}, INVALID), ({"T": math.nan}, INVALID),
    ({"T": math.inf}, INVALID), ({"T": 1e-45}, INVALID), ({"logits": None}, INVALID),
    ({"ids": None}, INVALID), ({"logp": None}, INVALID), ({"logits": FAKE + 2}, INVALID),
    ({"ids": FAKE + 4}, INVALID), ({"logp": FAKE + 2}, INVALID), ({"lse": FAKE + 1}, INVALID),
    ({"err": FAKE + 2}, INVALID), ({"N": 0, "logits": None}, OK)])
def test_topk_refusals(lib, kw, status):
    assert call(lib.rlk_topk_logp, TOPK, **kw) == status


BOTH = [({"H": 100}, UNSUPPORTED), ({"H": 0}, INVALID), ({"N": -1}, INVALID), ({"V": 0}, INVALID),
        ({"K": 0}, INVALID), ({"K": 1025}, UNSUPPORTED), ({"N": 1 << 21, "K": 1024}, UNSUPPORTED),
        ({"T": 0.0}, INVALID), ({"T": 9e-5}, INVALID), ({"T": 1e-30}, INVALID), ({"T": 1e31}, INVALID),
        ({"T": math.nan}, INVALID), ({"hidden": None}, INVALID), ({"weight": None}, INVALID),
        ({"ids": None}, INVALID), ({"teacher": None}, INVALID), ({"lse": None}, INVALID),
        ({"logp": None}, INVALID), ({"hidden": FAKE + 8}, INVALID),
        ({"weight": FAKE + 2}, INVALID), ({"ids": FAKE + 4}, INVALID),
        ({"teacher": FAKE + 2}, INVALID), ({"lse": FAKE + 2}, INVALID),
        ({"logp": FAKE + 2}, INVALID), ({"err": FAKE + 2}, INVALID), ({"ws": None}, WORKSPACE),
        ({"ws": FAKE + 16}, WORKSPACE), ({"ws_bytes": 256}, WORKSPACE),
        ({"N": 0, "hidden": None}, OK)]


@pytest.mark.parametrize("kw,status", BOTH + [({"kl": None}, INVALID), ({"kl": FAKE + 2}, INVALID)])
def test_topk_kl_forward_refusals(lib, kw, status):
    assert call(lib.rlk_linear_topk_kl_fwd, FWD, **kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    ({"grad": None}, INVALID), ({"grad": FAKE + 2}, INVALID), ({"dh": None}, INVALID),
    ({"dw": None}, INVALID), ({"dh": FAKE + 8}, INVALID), ({"dw": FAKE + 8}, INVALID)])
def test_topk_kl_backward_refusals(lib, kw, status):
    assert call(lib.rlk_linear_topk_kl_bwd, BWD, **kw) == status


def test_workspace_queries(lib):
    need = rlk.rlk_linear_topk_kl_fwd_workspace_bytes(4, 64, 1000, 20)
    assert call(lib.rlk_linear_topk_kl_fwd, FWD, ws_bytes=need - 1) == WORKSPACE
    need = rlk.rlk_linear_topk_kl_bwd_workspace_bytes(4, 64, 1000, 20)
    assert need >= 4 * 20 * 8
    assert call(lib.rlk_linear_topk_kl_bwd, BWD, ws_bytes=need - 1) == WORKSPACE
    for fn in (rlk.rlk_linear_topk_kl_fwd_workspace_bytes,
               rlk.rlk_linear_topk_kl_bwd_workspace_bytes):
        assert fn(-1, 64, 10, 2) == fn(4, 64, 0, 2) == fn(4, 64, 10, 0) == 0
    assert ctypes.sizeof(rlk.ProcessParams) == 128


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    class On:
        def __init__(self, device):
            self.at, self.device = device, "cuda:%d" % device

        def get_device(self):
            return self.at

    monkeypatch.setattr(rlk, "_device", lambda: 1)
    rlk._here(On(1), None, On(1))
    for bad in ((On(0),), (On(1), On(2)), (On(1), None, On(0))):
        with pytest.raises(ValueError, match="current device"):
            rlk._here(*bad)


def test_binding_refuses_what_it_cannot_pass_on(lib):
    x, ids = torch.zeros(4, 64), torch.zeros(4, 3, dtype=torch.int64)
    with pytest.raises(ValueError):
        rlk.process_logits(x)                                   # not on a GPU
    with pytest.raises(ValueError):
        rlk.topk_logp(x, 3)
    with pytest.raises((TypeError, ValueError)):
        rlk.linear_topk_kl(x.bfloat16(), x.bfloat16(), ids, torch.zeros(4, 3))
    h = x.bfloat16()
    for bad in ((h, h, ids[0], torch.zeros(3)), (h[0], h, ids, torch.zeros(4, 3)),
                (h, h[0], ids, torch.zeros(4, 3))):
        with pytest.raises(ValueError, match=r"hidden must be \[N, H\]"):
            rlk.linear_topk_kl(*bad)
    with pytest.raises(ValueError):
        rlk.topk_logp(x[0], 3)
