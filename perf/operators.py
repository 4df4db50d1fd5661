"""The operators next to the LM head, as cases that can be measured.

What a training or rollout program runs around the fused linear log-prob: the
final norm that makes the hidden states (layer norm and RMS norm, forward and
backward with the weight's gradient) and the sampler that draws the next token
from the head's logits.  ``run`` computes a case in its plain form (elementary
torch operations) or, where ``own`` is true, with this package's kernels.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------- cases

def _norm(op, n, h, dtype, name=None, bias=False, masked=False, pad=0):
    c = {"op": op, "n": n, "h": h, "dtype": dtype, "bias": bias, "masked": masked, "pad": pad}
    return dict(c, name=name) if name else c


def _sample(n, v, dtype, name=None, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, per_row=False,
            banned=0.0):
    c = {"op": "sample", "n": n, "v": v, "dtype": dtype, "temperature": temperature,
         "top_k": top_k, "top_p": top_p, "min_p": min_p, "per_row": per_row, "banned": banned}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the final norm of one decoding step, one sequence: latency alone
        _norm("layer_norm_fwd", 1, 4096, "bf16", "layer_norm_fwd_token", bias=True),
        # the final norm of a packed training batch at the benchmark's N and H
        _norm("layer_norm_fwd", 8192, 4096, "bf16", "layer_norm_fwd_batch", bias=True),
        # the same batch's backward, with the reduction of both parameter gradients over all tokens
        _norm("layer_norm_bwd", 8192, 4096, "bf16", "layer_norm_bwd_batch", bias=True),
        # an fp32 reference model with an odd width, rows cut out of a wider buffer
        _norm("layer_norm_bwd", 1031, 1537, "f32", "layer_norm_bwd_f32_odd", bias=True, pad=7),
        # the norm of a decoding batch
        _norm("rms_norm_fwd", 64, 4096, "bf16", "rms_norm_fwd_decode"),
        # a masked training batch at the large head's N and H, a fifth of it padding
        _norm("rms_norm_fwd", 16384, 7168, "bf16", "rms_norm_fwd_masked", masked=True),
        _norm("rms_norm_bwd", 16384, 7168, "bf16", "rms_norm_bwd_masked", masked=True),
        # a short micro-batch: the gradient's reduction has few rows to spread
        _norm("rms_norm_bwd", 200, 2048, "bf16", "rms_norm_bwd_micro"),
        # decoding one sequence at the rollout temperature, the whole vocabulary: latency
        _sample(1, 151936, "f32", "sample_token", temperature=0.7),
        # a rollout batch from the whole distribution, as on-policy training wants it
        _sample(256, 151936, "f32", "sample_rollout", temperature=1.0),
        # a serving batch with the usual truncations
        _sample(64, 151936, "f32", "sample_topk_topp", temperature=0.8, top_k=50, top_p=0.95),
        # requests that each bring their own settings, bf16 logits, part of the vocabulary banned
        _sample(129, 129280, "bf16", "sample_per_row", per_row=True, banned=0.3),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm_fwd", "layer_norm_bwd", "rms_norm_fwd", "rms_norm_bwd", "sample",
                     "sample"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op != "sample":
        h = rng.choice([_log_int(rng, 64, 8192), 64 * _log_int(rng, 2, 112), 4096])
        n = _log_int(rng, 1, 16384)
        return _norm(op, n, h, dtype, bias=op.startswith("layer") and rng.random() < 0.7,
                     masked=rng.random() < 0.4, pad=rng.choice([0, 0, 8, 5]))
    v = rng.choice([151936, 129280, _log_int(rng, 1000, 152000)])
    n = _log_int(rng, 1, 256)
    kind = rng.choice(["all", "temperature", "top_k", "top_p", "min_p", "both", "per_row"])
    t = round(rng.uniform(0.5, 1.3), 2)
    return _sample(n, v, dtype, temperature=1.0 if kind == "all" else t,
                   top_k=_log_int(rng, 1, 2000) if kind in ("top_k", "both") else 0,
                   top_p=round(rng.uniform(0.5, 0.99), 3) if kind in ("top_p", "both") else 1.0,
                   min_p=round(rng.uniform(0.01, 0.2), 3) if kind == "min_p" else 0.0,
                   per_row=kind == "per_row", banned=rng.choice([0.0, 0.0, 0.5, 0.99]))


# ----------------------------------------------------------------------------- inputs

def _rows(n, h, pad, dtype, gen):
    """[n, h] hidden rows: unit noise on a per-channel mean, a few channels far larger."""
    wide = h + pad
    x = torch.randn(n, wide, device="cuda", generator=gen)
    scale = torch.where(torch.rand(wide, device="cuda", generator=gen) < 0.002, 30.0, 1.0)
    x = x * scale + 0.5 * torch.randn(wide, device="cuda", generator=gen)
    return x.to(dtype)[:, :h]


def _prepare_norm(c, gen):
    dt, n, h = DTYPES[c["dtype"]], c["n"], c["h"]
    layer, back = c["op"].startswith("layer"), c["op"].endswith("bwd")
    s = {"op": c["op"], "layer": layer, "mask": None, "bias": None}
    s["x"] = _rows(n, h, c["pad"], dt, gen)
    s["weight"] = (1.0 + 0.2 * torch.randn(h, device="cuda", generator=gen)).to(dt)
    if c["bias"]:
        s["bias"] = (0.1 * torch.randn(h, device="cuda", generator=gen)).to(dt)
    if c["masked"]:
        s["mask"] = (torch.rand(n, device="cuda", generator=gen) >= 0.2).to(torch.uint8)
    f32 = {"dtype": torch.float32, "device": "cuda"}
    if not back:
        s["y"] = torch.empty(n, h, dtype=dt, device="cuda")
        s["mean"] = torch.empty(n, **f32) if layer else None
        s["rstd"] = torch.empty(n, **f32)
        return s
    # what the forward saved, and the gradient that the head's backward hands over
    xd = s["x"].double()
    mean = xd.mean(1) if layer else torch.zeros(n, dtype=torch.float64, device="cuda")
    s["mean"] = mean.float() if layer else None
    s["rstd"] = ((xd - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
    s["dy"] = (1e-3 * torch.randn(n, h, device="cuda", generator=gen)).to(dt)
    if s["mask"] is not None:
        s["dy"] *= s["mask"][:, None].to(dt)
    s["dx"] = torch.empty(n, h, dtype=dt, device="cuda")
    s["dweight"] = torch.empty(h, dtype=dt, device="cuda")
    s["dbias"] = torch.empty(h, dtype=dt, device="cuda") if c["bias"] else None
    return s


def _pick(values, n, dtype, gen):
    at = torch.randint(len(values), (n,), device="cuda", generator=gen)
    return torch.tensor(values, dtype=dtype, device="cuda")[at]


def _prepare_sample(c, gen):
    n, v = c["n"], c["v"]
    # token probabilities that fall with a power of their rank, another power in each row
    a = 0.9 + 0.7 * torch.rand(n, 1, device="cuda", generator=gen)
    z = -a * torch.rand(n, v, device="cuda", generator=gen).clamp_(min=1e-9).log()
    z += 0.3 * torch.randn(n, v, device="cuda", generator=gen) - 4.0
    if c["banned"]:
        z.masked_fill_(torch.rand(n, v, device="cuda", generator=gen) < c["banned"], -math.inf)
        z[:, 0] = 1.0
    s = {"op": "sample", "logits": z.to(DTYPES[c["dtype"]])}
    s["uniforms"] = torch.rand(n, device="cuda", generator=gen)
    if c["per_row"]:
        s["temperature"] = 0.5 + 0.8 * torch.rand(n, device="cuda", generator=gen)
        s["top_k"] = _pick([0, 0, 20, 50, 100, 1000], n, torch.int32, gen)
        s["top_p"] = _pick([1.0, 1.0, 0.8, 0.9, 0.95], n, torch.float32, gen)
        s["min_p"] = _pick([0.0, 0.0, 0.02, 0.05, 0.1], n, torch.float32, gen)
    else:
        for k in ("temperature", "top_k", "top_p", "min_p"):
            s[k] = c[k]
    s["tokens"] = torch.empty(n, dtype=torch.int64, device="cuda")
    s["logp"] = torch.empty(n, dtype=torch.float32, device="cuda")
    s["kept_logp"] = torch.empty(n, dtype=torch.float32, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return _prepare_sample(case, gen) if case["op"] == "sample" else _prepare_norm(case, gen)


# ----------------------------------------------------------------------------- plain forms

def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1) if s["layer"] else None
    xc = x - mean[:, None] if s["layer"] else x
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + EPS)
    y = xc * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if s["mask"] is not None:
        keep = s["mask"] != 0
        y = torch.where(keep[:, None], y, 0.0)
        rstd = torch.where(keep, rstd, 0.0)
        mean = torch.where(keep, mean, 0.0) if s["layer"] else None
    out = {"y": y.to(s["x"].dtype), "rstd": rstd}
    if s["layer"]:
        out["mean"] = mean
    return out


def _plain_norm_bwd(s):
    x, dy, w, rstd = s["x"].float(), s["dy"].float(), s["weight"].float(), s["rstd"][:, None]
    if s["mask"] is not None:
        dy = torch.where((s["mask"] != 0)[:, None], dy, 0.0)
    xh = (x - s["mean"][:, None] if s["layer"] else x) * rstd
    g = dy * w
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if s["layer"]:
        dx = dx - g.mean(1, keepdim=True)
    out = {"dx": (dx * rstd).to(s["x"].dtype), "dweight": (dy * xh).sum(0).to(s["weight"].dtype)}
    if s["dbias"] is not None:
        out["dbias"] = dy.sum(0).to(s["weight"].dtype)
    return out


def _column(v, like):
    return v.double()[:, None] if isinstance(v, torch.Tensor) else torch.full_like(like, float(v))


def _asks(v, off):
    return isinstance(v, torch.Tensor) or v != off


def _plain_sample(s):
    x = s["logits"].float() + 0.0
    n, v = x.shape
    top = x.double().amax(1, keepdim=True)
    temp = _column(s["temperature"], top)
    z = (x.double() - top) / temp
    w = z.exp()
    keep = torch.ones_like(w, dtype=torch.bool)
    if _asks(s["min_p"], 0.0):
        keep &= z >= _column(s["min_p"], top).log()
    if _asks(s["top_k"], 0) or _asks(s["top_p"], 1.0):
        order = x.sort(dim=1, descending=True, stable=True).indices
        ws = w.gather(1, order)
        c = ws.cumsum(1)
        k = _column(s["top_k"], top)
        k = torch.where((k <= 0) | (k > v), float(v), k).long()
        p = _column(s["top_p"], top)
        p = torch.where(p >= 1.0, math.inf, p)
        first = torch.arange(v, device=x.device)[None, :] < k
        first &= c - ws < p * c.gather(1, k - 1)
        keep &= torch.zeros_like(keep).scatter_(1, order, first)
    c = torch.where(keep, w, 0.0).cumsum(1)
    total = c[:, -1:]
    token = torch.searchsorted(c, s["uniforms"].double()[:, None] * total, right=True)
    token = token.clamp_(max=v - 1)
    zt = z.gather(1, token)
    return {"tokens": token[:, 0], "logp": (zt - w.sum(1, keepdim=True).log())[:, 0].float(),
            "kept_logp": (zt - total.log())[:, 0].float()}


# ----------------------------------------------------------------------------- one pass

def _workspace(s, nbytes):
    """The call's scratch, which a program allocates once and keeps."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own(s):
    import rl_post_linear_gb300 as rlk
    op = s["op"]
    if op == "layer_norm_fwd":
        rlk.rlk_layer_norm_fwd(s["x"], s["weight"], s["bias"], s["mask"], EPS, s["y"], s["mean"],
                               s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "rms_norm_fwd":
        rlk.rlk_rms_norm_fwd(s["x"], s["weight"], s["mask"], EPS, s["y"], s["rstd"])
        return {"y": s["y"], "rstd": s["rstd"]}
    if op == "layer_norm_bwd":
        ws = _workspace(s, rlk.rlk_layer_norm_bwd_workspace_bytes(*s["x"].shape))
        rlk.rlk_layer_norm_bwd(s["x"], s["weight"], s["dy"], s["mean"], s["rstd"], s["mask"],
                               s["dx"], s["dweight"], s["dbias"], ws)
        out = {"dx": s["dx"], "dweight": s["dweight"]}
        return dict(out, dbias=s["dbias"]) if s["dbias"] is not None else out
    if op == "rms_norm_bwd":
        ws = _workspace(s, rlk.rlk_rms_norm_bwd_workspace_bytes(*s["x"].shape))
        rlk.rlk_rms_norm_bwd(s["x"], s["weight"], s["dy"], s["rstd"], s["mask"], s["dx"],
                             s["dweight"], ws)
        return {"dx": s["dx"], "dweight": s["dweight"]}
    ws = _workspace(s, rlk.rlk_sample_logits_workspace_bytes(*s["logits"].shape))
    rlk.rlk_sample_logits(s["logits"], s["uniforms"], None, s["temperature"], s["top_k"],
                          s["top_p"], s["min_p"], s["tokens"], s["logp"], s["kept_logp"],
                          ws)
    return {"tokens": s["tokens"], "logp": s["logp"], "kept_logp": s["kept_logp"]}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "sample":
        return _plain_sample(state)
    return _plain_norm_bwd(state) if state["op"].endswith("bwd") else _plain_norm_fwd(state)


def work(case):
    n = case["n"]
    if case["op"] == "sample":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = n * (4 + 8 + 4 + 4) + (n * 16 if case["per_row"] else 0)
        return {"bytes": n * case["v"] * e + rows, "flops": 4 * n * case["v"]}
    h, e = case["h"], 2 if case["dtype"] == "bf16" else 4
    read = 0.8 if case["masked"] else 1.0
    stats = (2 if case["op"].startswith("layer") else 1) * 4 * n + (n if case["masked"] else 0)
    vectors = (2 if case["bias"] else 1) * h * e
    if case["op"].endswith("fwd"):
        return {"bytes": (1 + read) * n * h * e + stats + vectors, "flops": 8 * read * n * h}
    return {"bytes": (1 + 2 * read) * n * h * e + stats + vectors + h * e,
            "flops": 14 * read * n * h}


# ----------------------------------------------------------------------------- 64 bits

def _exact_norm(c, s):
    """Row blocks in float64, each value from the definition."""
    n, h = s["x"].shape
    w = s["weight"].double()
    b = s["bias"].double() if s["bias"] is not None else torch.zeros_like(w)
    live = torch.ones(n, dtype=torch.bool, device=w.device) if s["mask"] is None else s["mask"] > 0
    big = {k: [] for k in ("y", "mean", "rstd", "dx")}
    dw, db = torch.zeros_like(w), torch.zeros_like(w)
    for a in range(0, n, 4096):
        rows = slice(a, min(n, a + 4096))
        x, on = s["x"][rows].double(), live[rows][:, None].double()
        if c["op"].endswith("fwd"):
            mu = x.sum(1, keepdim=True) / h if s["layer"] else torch.zeros_like(x[:, :1])
            r = ((x - mu).pow(2).sum(1, keepdim=True) / h + EPS).pow(-0.5)
            big["y"].append(on * ((x - mu) / r.reciprocal() * w + b))
            big["mean"].append((on * mu)[:, 0])
            big["rstd"].append((on * r)[:, 0])
            continue
        r = s["rstd"][rows].double()[:, None]
        xh = r * (x - s["mean"][rows].double()[:, None]) if s["layer"] else r * x
        g = on * s["dy"][rows].double()
        dw += torch.einsum("th,th->h", g, xh)
        db += torch.einsum("th->h", g)
        gw = g * w
        along = torch.einsum("th,th->t", gw, xh)[:, None] / h
        centre = gw.sum(1, keepdim=True) / h if s["layer"] else 0.0
        big["dx"].append(r * gw - r * centre - r * xh * along)
    got = {k: torch.cat(v) for k, v in big.items() if v}
    if c["op"].endswith("fwd"):
        return got if s["layer"] else {"y": got["y"], "rstd": got["rstd"]}
    got["dweight"] = dw
    return dict(got, dbias=db) if s["dbias"] is not None else got


def _exact_sample(s):
    """One row after another in numpy's float64."""
    x = s["logits"].float().cpu().numpy().astype(np.float64)
    n, v = x.shape

    def per_row(name):
        p = s[name]
        return p.cpu().numpy() if isinstance(p, torch.Tensor) else np.full(n, p)

    t, k, p, m = (per_row(q) for q in ("temperature", "top_k", "top_p", "min_p"))
    u = s["uniforms"].cpu().numpy().astype(np.float64)
    out = {"tokens": np.zeros(n, np.int64), "logp": np.zeros(n), "kept_logp": np.zeros(n)}
    for i in range(n):
        z = (x[i] - x[i].max()) / float(t[i])
        e = np.exp(z)
        kept = e.copy()
        kk = int(k[i]) if 0 < k[i] < v else v
        if kk < v or p[i] < 1.0:
            order = np.argsort(-x[i], kind="stable")[:kk]
            run_sum = np.cumsum(e[order])
            if p[i] < 1.0:
                order = order[: 1 + int(np.searchsorted(run_sum, float(p[i]) * run_sum[-1]))]
            kept = np.zeros(v)
            kept[order] = e[order]
        if m[i] > 0.0:
            kept[z < math.log(float(m[i]))] = 0.0
        c = np.cumsum(kept)
        tok = int(np.argmax(c > u[i] * c[-1]))
        out["tokens"][i] = tok
        out["logp"][i] = z[tok] - math.log(math.fsum(e))
        out["kept_logp"][i] = z[tok] - math.log(c[-1])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_sample(s) if case["op"] == "sample" else _exact_norm(case, s)
