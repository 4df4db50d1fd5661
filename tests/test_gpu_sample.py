"""Sampling from logits against the definition in float64, one row at a time.

Tokens have to be equal wherever u times the kept weight is more than 1e-11 of it away from a
border of the running sums, and top_p's boundary as far from one (nearer, float64's own order
of summation decides); the few rows nearer than that are left out by that rule alone.
logp and kept_logp: the sums' weights may be off by 2^-20 of themselves (a base-2 exponential
good to 2^-22 of an argument of up to 32 rounded to fp32), the logarithm and the difference
round in fp32: |error| <= 2^-19 + 2^-22 |logp|.
"""
import math

import numpy as np
import pytest
import torch

import rl_post_linear_gb300 as rlk
from helpers import dev, same_bits

pytestmark = pytest.mark.gpu

NEAR = 1e-11


def ref_row(x, t, k, p, m, u):
    """(token, logp, kept_logp, margin) of one float64 row."""
    v = x.size
    z = (x - x.max()) / t
    w = np.exp(z)
    margin = 1.0
    n = k if 0 < k < v else v
    order = np.argsort(-x, kind="stable")[:n]
    if p < 1.0:
        run = np.cumsum(w[order])
        need = p * run[-1]
        margin = min(margin, float(np.min(np.abs(run - need)) / run[-1]))
        if np.all(w[order] == 1.0):                 # whole numbers: float64 is exact
            margin = 1.0
        order = order[:1 + int(np.searchsorted(run, need))]
    kept = np.zeros(v)
    kept[order] = w[order]
    if m > 0.0:
        kept[z < math.log(m)] = 0.0
    c = np.cumsum(kept)
    at = u * c[-1]
    token = int(np.argmax(c > at))
    if not np.all((kept == 0.0) | (kept == 1.0)):
        margin = min(margin, float(np.min(np.abs(c - at)) / c[-1]) if u > 0 else 1.0)
    return token, z[token] - math.log(math.fsum(w)), z[token] - math.log(c[-1]), margin


def column(v, n):
    return v.cpu().double().numpy() if isinstance(v, torch.Tensor) else np.full(n, float(v))


def check(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, mask=None, most_near=0.02):
    n, v = logits.shape
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    tok, logp, kept = rlk.sample_logits(logits, u, temperature, top_k, top_p, min_p, mask, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    x = logits.float().cpu().double().numpy()
    uu, t, k, p, m = (column(q, n) for q in (u, temperature, top_k, top_p, min_p))
    tok, logp, kept = tok.cpu().numpy(), logp.cpu().double().numpy(), kept.cpu().double().numpy()
    near = 0
    for i in range(n):
        if mask is not None and int(mask[i]) == 0:
            assert tok[i] == -1 and logp[i] == 0 and kept[i] == 0
            continue
        want, lp, kl, margin = ref_row(x[i], t[i], int(k[i]), p[i], m[i], uu[i])
        if margin <= NEAR:
            near += 1
            continue
        assert tok[i] == want, (i, tok[i], want, margin)
        assert abs(logp[i] - lp) <= 2.0 ** -19 + 2.0 ** -22 * abs(lp)
        assert abs(kept[i] - kl) <= 2.0 ** -19 + 2.0 ** -22 * abs(kl)
    assert near <= max(1, most_near * n)
    return tok


def zipf(n, v, seed, dtype=torch.float32, power=(0.9, 1.6)):
    g = torch.Generator().manual_seed(seed)
    a = power[0] + (power[1] - power[0]) * torch.rand(n, 1, generator=g)
    z = -a * torch.rand(n, v, generator=g).clamp_(min=1e-9).log()
    return (z + 0.3 * torch.randn(n, v, generator=g) - 4.0).to(dtype).to(dev())


def normal(n, v, seed, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(n, v, generator=g)).to(dtype).to(dev())


def uniforms(n, seed):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed)).to(dev())


SETTINGS = [{}, {"temperature": 0.6}, {"temperature": 1.7}, {"top_k": 1}, {"top_k": 50},
            {"top_k": 700}, {"top_p": 0.3}, {"top_p": 0.95}, {"top_p": 0.9999}, {"min_p": 0.05},
            {"min_p": 1.0}, {"top_k": 40, "top_p": 0.9, "temperature": 0.8},
            {"top_k": 3000, "top_p": 0.8, "min_p": 0.001},
            {"temperature": 0.9, "top_p": 0.97, "min_p": 0.02}]


@pytest.mark.parametrize("setting", SETTINGS, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_settings(setting, dtype):
    check(zipf(24, 5003, 1, dtype), uniforms(24, 2), **setting)


@pytest.mark.parametrize("setting", SETTINGS, ids=str)
def test_flat_rows(setting):
    # a nucleus of most of the vocabulary
    check(normal(12, 20011, 3, 0.5), uniforms(12, 4), **setting)
    check(normal(12, 20011, 5, 1.0, torch.bfloat16), uniforms(12, 6), **setting)


@pytest.mark.parametrize("v", [1, 2, 3, 5, 31, 32, 33, 127, 255, 257, 511, 513, 1023, 1024, 1025,
                               2047, 4096, 4097, 8191, 16385, 32003, 65537])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_vocabulary_sizes(v, dtype):
    for i, setting in enumerate(({}, {"top_k": 20}, {"top_p": 0.9, "temperature": 0.7},
                                 {"min_p": 0.1}, {"top_k": 5, "top_p": 0.5})):
        check(zipf(7, v, v + i, dtype), uniforms(7, v + i + 1), **setting)


@pytest.mark.parametrize("setting", [{}, {"temperature": 0.7}, {"top_k": 50, "top_p": 0.95},
                                     {"top_p": 0.9}, {"min_p": 0.02}, {"top_k": 20000}], ids=str)
@pytest.mark.parametrize("v,dtype", [(151936, torch.float32), (129280, torch.bfloat16)])
def test_large_vocabularies(v, dtype, setting):
    check(zipf(6, v, 8, dtype), uniforms(6, 9), **setting)
    check(normal(3, v, 10, 2.0, dtype), uniforms(3, 11), **setting)


def test_beyond_the_usual_vocabularies():
    v = (1 << 20) + 77
    check(zipf(2, v, 12), uniforms(2, 13), top_p=0.9)
    check(zipf(2, v, 14, torch.bfloat16), uniforms(2, 15))


@pytest.mark.parametrize("n", [1, 2, 3, 37, 151, 153, 400])
def test_row_counts(n):
    check(zipf(n, 3001, n), uniforms(n, n), top_p=0.9, temperature=0.8)
    check(zipf(n, 3001, n + 1), uniforms(n, n + 1))


def test_settings_of_each_row():
    n = 90
    g = torch.Generator().manual_seed(6)

    def pick(values, dtype):
        return torch.tensor(values, dtype=dtype)[torch.randint(len(values), (n,), generator=g)].to(dev())

    check(zipf(n, 8001, 7), uniforms(n, 8), pick([0.3, 0.7, 1.0, 2.0], torch.float32),
          pick([0, 1, 5, 50, 2000, 8001, 100000], torch.int32),
          pick([0.2, 0.9, 0.99, 1.0, 3.0], torch.float32),
          pick([0.0, 0.0, 0.01, 0.3], torch.float32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties(dtype):
    # whole-number logits: every boundary falls inside a group of equal tokens
    g = torch.Generator().manual_seed(17)
    z = torch.randint(-3, 4, (16, 6001), generator=g).to(dtype).to(dev())
    for setting in ({"top_k": 100}, {"top_k": 3000}, {"top_p": 0.5}, {"top_p": 0.93},
                    {"top_k": 900, "top_p": 0.7}, {"min_p": 0.2}, {"top_k": 1}):
        check(z, uniforms(16, 18), **setting)
    same = torch.zeros(9, 4096, dtype=dtype, device=dev())
    u = torch.arange(9, device=dev()) / 9.0
    for setting in ({}, {"top_k": 7}, {"top_p": 0.5}, {"top_p": 0.25, "top_k": 64},
                    {"min_p": 1.0}):
        check(same, u.float(), **setting)
    zeros = torch.zeros(2, 50, dtype=dtype, device=dev())
    zeros[:, ::2] = -0.0                       # -0 and +0 are one value: lowest index first
    assert check(zeros, torch.full((2,), 0.99, device=dev()), top_k=3).tolist() == [2, 2]


def test_greedy_is_the_lowest_index_of_the_maximum():
    z = normal(40, 3000, 19).round_()
    tok = check(z, uniforms(40, 20), top_k=1)
    want = np.array([int(np.argmax(r)) for r in z.cpu().numpy()])
    assert np.array_equal(tok, want)


@pytest.mark.parametrize("setting", [{}, {"top_k": 10}, {"top_p": 0.9}, {"min_p": 0.1},
                                     {"top_k": 900, "top_p": 0.999}], ids=str)
def test_banned_tokens(setting):
    z = zipf(12, 4001, 21)
    z[0, 1:] = -math.inf                        # one token left
    z[1, :4000] = -math.inf
    z[2, 5:] = -math.inf                        # fewer left than top_k asks for
    z[3:6] = z[3:6].masked_fill(torch.rand(3, 4001, device=dev()) < 0.99, -math.inf)
    z[3:6, 77] = 0.0
    z[6:9, 100:] = torch.finfo(torch.float32).min     # masks of the lowest value
    z[9] = torch.finfo(torch.float32).min             # all of them: uniform
    tok = check(z, uniforms(12, 22), **setting)
    assert tok[0] == 0 and tok[1] == 4000 and tok[2] < 5 and (tok[6:9] < 100).all()
    zb = zipf(4, 4001, 23, torch.bfloat16)
    zb[:, 9:] = torch.finfo(torch.bfloat16).min
    assert (check(zb, uniforms(4, 24), **setting) < 9).all()


def test_uniforms_at_their_ends():
    z = zipf(6, 2500, 25)
    u = torch.tensor([0.0, 2.0 ** -149, 1e-30, 2.0 ** -24, 1 - 2.0 ** -24, 0.5], device=dev())
    for setting in ({}, {"top_k": 30}, {"top_p": 0.9}):
        tok = check(z, u, **setting, most_near=0.6)
    z[:, 0] = -math.inf
    z[:, 2499] = -math.inf
    tok, _, _ = rlk.sample_logits(z, u)
    # u = 0 gives the first token that can be drawn, the largest u below 1 never the banned last
    assert int(tok[0]) == 1 and int(tok[4]) < 2499


def test_extreme_temperatures():
    z = zipf(8, 3000, 27)
    check(z, uniforms(8, 28), temperature=1e-6)
    check(z, uniforms(8, 28), temperature=0.01, top_p=0.9)
    check(z, uniforms(8, 28), temperature=1e6, top_k=500)
    check(z, uniforms(8, 28), temperature=1e4)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v,pad,offset", [(3000, 8, 0), (3001, 0, 0), (2999, 3, 1), (4096, 0, 3)])
def test_strides_and_offsets(v, pad, offset, dtype):
    n = 9
    flat = zipf(1, n * (v + pad) + offset, 29, dtype)[0]
    z = flat[offset:].view(n, v + pad)[:, :v]
    for setting in ({}, {"top_k": 30, "top_p": 0.9}, {"top_p": 0.95}):
        check(z, uniforms(n, 30), **setting)


def test_rows_do_not_depend_on_batch_or_alignment():
    v = 30011
    z, u = zipf(160, v, 31), uniforms(160, 32)
    for setting in ({"temperature": 0.8}, {"top_k": 60}, {"top_p": 0.95}, {"min_p": 0.01}):
        a = rlk.sample_logits(z, u, **setting)
        one = torch.empty(v + 1, device=dev())
        for i in (0, 3, 77, 159):
            row = one[1:].view(1, v)
            row.copy_(z[i:i + 1])
            b = rlk.sample_logits(row, u[i:i + 1], **setting)
            c = rlk.sample_logits(z[i:i + 2], u[i:i + 2], **setting)
            for p, q, r in zip(a, b, c):
                assert p[i].item() == q[0].item() == r[0].item()
        again = rlk.sample_logits(z, u, **setting)
        assert all(torch.equal(p, q) for p, q in zip(a, again))


def test_inactive_rows_are_not_read():
    z, u = zipf(10, 1500, 33), uniforms(10, 34)
    mask = torch.tensor([1, 0, 1, 1, 0, 0, 1, 9, 1, 0], dtype=torch.uint8, device=dev())
    z[mask == 0] = float("nan")
    u[mask == 0] = float("nan")
    check(z, u, top_p=0.9, mask=mask)
    check(z, u, mask=torch.zeros_like(mask))


def test_rows_without_a_distribution_are_flagged():
    z, u = zipf(6, 900, 35), uniforms(6, 36)
    good = rlk.sample_logits(z, u, top_k=40)[0].clone()
    z[1, 50] = float("nan")
    z[2, 60] = math.inf
    z[4] = -math.inf
    for setting in ({}, {"top_k": 40}, {"top_p": 0.9}):
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        tok, logp, kept = rlk.sample_logits(z, u, error_word=err, **setting)
        assert int(err.item()) == rlk.RLK_DEVERR_LOGITS
        for i in (1, 2, 4):
            assert int(tok[i]) == -1 and math.isnan(logp[i]) and math.isnan(kept[i])
        if setting == {"top_k": 40}:
            assert torch.equal(tok[[0, 3, 5]], good[[0, 3, 5]])


def test_settings_out_of_range_in_a_row_are_flagged():
    n = 8
    z = zipf(n, 700, 37)
    u = uniforms(n, 38)
    t = torch.ones(n, device=dev())
    p = torch.ones(n, device=dev())
    m = torch.zeros(n, device=dev())
    k = torch.zeros(n, dtype=torch.int32, device=dev())
    u[0], u[1], t[2], t[3], p[4], m[5], k[6] = 1.0, -0.1, 0.0, float("nan"), 0.0, 1.5, -1
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    tok, logp, kept = rlk.sample_logits(z, u, t, k, p, m, error_word=err)
    assert int(err.item()) == rlk.RLK_DEVERR_SAMPLE_PARAM
    assert tok[:7].tolist() == [-1] * 7 and bool(torch.isnan(logp[:7]).all())
    assert int(tok[7]) >= 0 and not math.isnan(kept[7])


def test_optional_outputs_and_another_stream():
    z, u = zipf(5, 1200, 39), uniforms(5, 40)
    want, lp, _ = rlk.sample_logits(z, u, 0.9, 30)
    tok = torch.empty_like(want)
    ws = torch.empty(max(256, rlk.rlk_sample_logits_workspace_bytes(5, 1200)), dtype=torch.uint8,
                     device=dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rlk.rlk_sample_logits(z, u, None, 0.9, 30, 1.0, 0.0, tok, None, None, ws, stream=side)
    side.synchronize()
    assert torch.equal(tok, want)
    empty = rlk.sample_logits(z[:0], u[:0])
    assert empty[0].shape == (0,)


def test_captured_in_a_graph():
    z, u = zipf(20, 5000, 41), uniforms(20, 42)
    rlk.sample_logits(z, u, 0.8, 0, 0.9)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rlk.sample_logits(z, u, 0.8, 0, 0.9)
    for seed in (43, 44):
        z.copy_(zipf(20, 5000, seed))
        u.copy_(uniforms(20, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, rlk.sample_logits(z, u, 0.8, 0, 0.9)))


def test_logp_is_what_scoring_the_token_gives():
    z, u = zipf(64, 20000, 45), uniforms(64, 46)
    tok, logp, kept = rlk.sample_logits(z, u, 0.7, 0, 0.95)
    scored, _ = rlk.logp_from_logits(z, tok, None, 0.7)
    # both are fp32 with 2^-19 + 2^-22 |logp| each
    assert bool(((logp - scored).abs() <= 2.0 ** -18 + 2.0 ** -21 * logp.abs()).all())
    assert bool((kept >= logp).all())
    audit = rlk.dlogp_audit(scored, logp)
    assert audit["active_count"] == 64 and audit["max_abs_dlogp"] < 1e-4


def test_frequencies():
    # evenly spaced uniforms: a token is drawn as often as its probability says, within one
    n, v = 4096, 400
    row = zipf(1, v, 47)
    z = row.expand(n, v).contiguous()
    u = ((torch.arange(n, dtype=torch.float64) + 0.5) / n).float().to(dev())
    tok, _, _ = rlk.sample_logits(z, u)
    p = torch.softmax(row[0].double(), 0).cpu().numpy()
    got = np.bincount(tok.cpu().numpy(), minlength=v)
    assert np.abs(got - n * p).max() <= 1.0 + 1e-3
    assert bool((tok[1:] >= tok[:-1]).all())


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("setting", [{"top_k": 50}, {"top_p": 0.9}, {"top_k": 900, "top_p": 0.9},
                                     {"min_p": 0.001}, {"top_k": 50, "min_p": 0.3}, {}], ids=str)
def test_rows_in_order_of_the_tokens(setting, order):
    # the largest elements side by side: they fill a few segments, so a value that as many
    # segment maxima reach is reached by far more elements than the short list holds
    z = normal(8, 40000, 48, 1.5).sort(dim=1, descending=order < 0).values
    check(z.contiguous(), uniforms(8, 49), **setting)
    check(z.bfloat16(), uniforms(8, 50), **setting)


@pytest.mark.parametrize("setting", [{"top_p": 0.95}, {"top_k": 1500}], ids=str)
def test_many_rows_to_search(setting):
    # every row has a wide nucleus, and there are more of them than blocks, or than a batch
    check(normal(1400, 2050, 51, 0.4, torch.bfloat16), uniforms(1400, 52), **setting)


def test_many_rows_on_a_border():
    # equal tokens and uniforms on the borders between them: u V is a whole number, exactly
    n, v = 2100, 2048
    z = torch.full((n, v), -3.25, device=dev())
    z[::3] = 11.0
    u = (torch.arange(n) % v).float().div(v).to(dev())
    tok = check(z, u)
    assert np.array_equal(tok, np.arange(n) % v)
    mask = (torch.arange(n) % 4 != 2).to(device=dev(), dtype=torch.uint8)
    check(z, u, mask=mask)


def test_few_rows_to_search_among_many():
    # the searched rows lie far apart, the others are done by the first pass
    n, v = 1300, 3000
    z = zipf(n, v, 53, power=(1.5, 1.6))
    z[[3, 511, 512, 513, 1023, 1024, 1299]] = normal(7, v, 54, 0.3)
    check(z, uniforms(n, 55), top_p=0.9)


def test_workspace_size_is_enough_at_its_edge():
    # the byte count asked for, in a buffer with a guard behind it
    for n, v in ((1, 1), (3, 700), (40, 5003), (600, 1030), (2, 151936)):
        for dtype in (torch.float32, torch.bfloat16):
            z, u = normal(n, v, n, 0.7, dtype), uniforms(n, v)
            need = rlk.rlk_sample_logits_workspace_bytes(n, v)
            buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=dev())
            for p in (1.0, 0.9):
                want = rlk.sample_logits(z, u, 0.8, 0, p)
                out = tuple(torch.empty_like(t) for t in want)
                rlk.rlk_sample_logits(z, u, None, 0.8, 0, p, 0.0, *out, buf[:need])
                assert bool((buf[need:] == 0xA5).all())
                assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("v,dtype", [(32660, torch.bfloat16), (70001, torch.float32),
                                     (151936, torch.float32), (151936, torch.bfloat16)])
@pytest.mark.parametrize("k", [150, 300, 450, 600, 700, 701])
def test_top_k_of_hundreds(k, v, dtype):
    # lists of a few hundred to a thousand elements, from segments of every width
    check(zipf(5, v, k), uniforms(5, k + 1), top_k=k, temperature=0.8)
    check(normal(4, v, k + 2, 2.0, dtype), uniforms(4, k + 3), top_k=k, top_p=0.97)
    z = normal(4, v, k + 4, 1.0, dtype)
    z[:, ::3] = -math.inf
    check(z, uniforms(4, k + 5), top_k=k, min_p=1e-4)
