"""Sampling near its borders: gaps in the logits at top_p's boundary, rows with one dominant token,
the largest vocabularies, and batches that divide a row differently.

Compared with the definition in float64, one row at a time.  The kernel's weights carry a relative
error of 2^-40 and a rounding to whole units of 2^-bits of the largest, V 2^bits < 2^64: sums are
within 2^-39 + V 2^-(bits + 1) / S of themselves (S: the sum in units of the largest weight), and a
row whose target or top_p boundary is nearer than that to a border is left out.
logp and kept_logp: 2^-19 + 2^-22 |logp|, as the fp32 exponentials, logarithm and difference give.
"""
import numpy as np
import pytest
import torch

import rl_post_linear_gb300 as rlk
from helpers import dev
from test_gpu_sample import ref_row, uniforms, zipf

pytestmark = pytest.mark.gpu


def weight_bits(v):
    bits = 46
    while 1 << (64 - bits) <= v:
        bits -= 1
    return bits


def check(logits, u, temperature=1.0, top_k=0, top_p=1.0):
    """Compares each row; returns how many were far enough from a border to be compared."""
    n, v = logits.shape
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    out = rlk.sample_logits(logits, u, temperature, top_k, top_p, error_word=err)
    assert int(err.item()) == 0
    tok, logp, kept = (t.cpu().double().numpy() for t in out)
    x, uu = logits.float().cpu().double().numpy(), u.cpu().double().numpy()
    done = 0
    for i in range(n):
        s = np.exp((x[i] - x[i].max()) / temperature).sum()
        want, lp, kl, margin = ref_row(x[i], temperature, top_k, top_p, 0.0, uu[i])
        if margin <= 2.0 ** -39 + v * 2.0 ** -(weight_bits(v) + 1) / s:
            continue
        done += 1
        assert tok[i] == want, (i, tok[i], want, margin)
        assert abs(logp[i] - lp) <= 2.0 ** -19 + 2.0 ** -22 * abs(lp)
        assert abs(kept[i] - kl) <= 2.0 ** -19 + 2.0 ** -22 * abs(kl)
    return done


def two_levels(n, v, heavy, gap, spread_top, spread_tail, dtype, seed):
    """Rows with `heavy` logits in [-spread_top, 0], in the last columns, and the others in
    [-gap - spread_tail, -gap]."""
    g = torch.Generator().manual_seed(seed)
    z = -gap - spread_tail * torch.rand(n, v, generator=g)
    z[:, v - heavy:] = -spread_top * torch.rand(n, heavy, generator=g)
    z[:, v - 1] = 0.0
    return z.to(dtype).to(dev())


def check_nuclei(z, heavy, where, **setting):
    """Nuclei that end at `where` of the tail's weight, drawn from over the tail's part of them."""
    n, v = z.shape
    w = torch.exp(z[:1].double().cpu())[0]
    tail, top = float(w[:v - heavy].sum()), float(w[v - heavy:].sum())
    p = (top + where * tail) / (top + tail)
    u = (torch.arange(n, dtype=torch.float64) + 0.5) / n * (where * tail / (top + where * tail))
    return check(z, u.float().to(dev()), top_p=p, **setting)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heavy,spread_top,gaps", [(1, 0.0, (2, 5, 8, 10, 12, 14, 17, 20)),
                                                   (300, 0.0, (1, 3, 6, 9, 10, 12, 15)),
                                                   (300, 2.0, (1, 4, 7, 9, 11, 11.5, 13, 15)),
                                                   (2500, 3.0, (1, 6, 9, 11, 13))])
def test_nuclei_that_end_behind_a_gap(heavy, spread_top, gaps, dtype):
    done = 0
    for i, gap in enumerate(gaps):
        for spread_tail in (0.0, 0.05, 1.0):
            z = two_levels(6, 8003, heavy, gap, spread_top, spread_tail, dtype, 100 * i + heavy)
            for where in (0.003, 0.17, 0.5, 0.93):
                done += check_nuclei(z, heavy, where)
    assert done >= 6 * len(gaps)


@pytest.mark.parametrize("top_p", [0.99915, 0.9992, 0.9993, 0.99945, 0.9995, 0.99953, 0.9997])
def test_nuclei_of_a_flat_top_and_a_far_tail(top_p):
    for v, gap, spread in ((5003, 10.0, 0.0), (8003, 11.5, 2.0)):
        for k in (0, 4000):
            z = two_levels(16, v, 300, gap, spread, 0.05, torch.float32, 5)
            u = (torch.arange(16) + 0.5) / 16 * (3e-4 if k == 0 else 1e-4)
            assert check(z, u.to(dev()), top_p=top_p, top_k=k) >= 8


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nuclei_of_a_staircase(dtype):
    # steps of 200 tokens, each 2 to 5 nats below the one before: a gap inside every window
    g = torch.Generator().manual_seed(3)
    for step in (2.0, 3.5, 5.0):
        z = -step * (torch.arange(8001) // 200).clamp(max=9) - 0.01 * torch.rand(8, 8001, generator=g)
        z = z.flip(1).contiguous().to(dtype).to(dev())
        for p in (0.5, 0.9, 0.99, 0.9999, 1 - 1e-6, 1 - 1e-8):
            u = 10.0 ** -torch.arange(8, dtype=torch.float32)
            assert check(z, u.clamp(max=0.9999).to(dev()), top_p=p) >= 4


@pytest.mark.parametrize("v,n,gap", [(8003, 128, gap) for gap in (8.0, 14.0, 18.0003, 20.0, 21.5)] +
                         [(151936, 48, gap) for gap in (8.0, 14.0, 16.5, 18.0003, 19.0)])
def test_draws_from_the_tail_of_a_peaked_row(v, n, gap):
    # one token holds nearly all weight, in the last column; u over the others' part
    z = torch.full((1, v), -gap)
    z[0, v - 1] = 0.0
    tail = (v - 1) * float(np.exp(-np.float64(np.float32(gap))))
    u = (torch.arange(n, dtype=torch.float64) + 0.37) / n * (tail / (1 + tail))
    z = z.expand(n, v).contiguous()
    assert check(z.to(dev()), u.float().to(dev())) >= n // 2
    z += 0.3 * torch.randn(n, v, generator=torch.Generator().manual_seed(1)) * (z < 0)
    assert check(z.to(dev()), u.float().to(dev())) >= n // 2


def test_draws_next_to_a_long_light_tail():
    # 2^20 columns of 127 units, between a token of weight 1 and one of weight 1/2: uniforms on both
    # sides of the last one's border.  In the tail a token may be off by what the sums may.
    v, n = 1 << 20, 64
    z = torch.full((1, v), -float(np.log(2.0 ** weight_bits(v) / 127.0)))
    z[0, 0], z[0, v - 1] = 0.0, -float(np.log(2.0))
    w = np.exp(z[0].double().numpy())
    c = np.cumsum(w)
    u = np.float32(c[-2] / c[-1]) + np.arange(-n // 2, n // 2, dtype=np.float32) * np.float32(2.0 ** -24)
    want = np.searchsorted(c, u.astype(np.float64) * c[-1], side="right")
    units = (2.0 ** -39 * c[-1] + v * 2.0 ** -(weight_bits(v) + 1)) / w[1]
    z, u = z.expand(8, v).contiguous().to(dev()), torch.from_numpy(u).to(dev())
    tok = torch.cat([rlk.sample_logits(z, u[a:a + 8])[0] for a in range(0, n, 8)]).cpu().numpy()
    assert (want[:n // 2 - 2] < v - 1).all() and (want[n // 2 + 2:] == v - 1).all()
    far = np.abs(np.arange(n) - n // 2) > 2
    assert (np.abs(tok - want)[far] <= units).all()
    assert ((tok == v - 1) == (want == v - 1))[far].all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_below_half_a_unit_are_not_drawn(dtype):
    # weights of 2^-57.7 in front, one of 2^-45 behind them, the largest last: u = 0 draws the second
    for v in (700, 30011):
        z = torch.full((3, v), -40.0)
        z[:, v - 2], z[:, v - 1] = -45.0 * float(np.log(2.0)), 0.0
        u = torch.tensor([0.0, 2.0 ** -60, 2.0 ** -24], device=dev())
        for setting in ({}, {"top_p": 1 - 2.0 ** -20}, {"top_k": 5}):
            tok, logp, kept = rlk.sample_logits(z.to(dtype).to(dev()), u, **setting)
            last = v - 1 if "top_p" in setting else v - 2        # all but the largest is cut
            assert tok.tolist() == [last, last, v - 1]
            assert bool((kept >= logp).all())


@pytest.mark.parametrize("v,n", [(1 << 21, 78), (1 << 22, 40)])
def test_flat_rows_of_the_largest_vocabularies(v, n):
    # All tokens alike but one, which takes 5e-7 of a weight out of the total: a quarter of V is
    # kept, and u times that gives the token exactly.
    z = torch.full((n, v), -2.5, dtype=torch.bfloat16, device=dev())
    z[:, v // 2] = -3.0
    u = torch.arange(n, dtype=torch.float32, device=dev()) / n
    tok, _, kept = rlk.sample_logits(z, u, 1e6, 0, 0.25)
    assert torch.equal(tok, torch.floor(u.double() * (v // 4)).long())
    want = -float(np.log(v // 4))
    assert bool(((kept.double() - want).abs() <= 2.0 ** -19 - 2.0 ** -22 * want).all())


@pytest.mark.parametrize("setting", [{}, {"temperature": 0.7}, {"top_k": 50}, {"top_p": 0.9},
                                     {"top_k": 2000, "top_p": 0.95}, {"min_p": 0.01}], ids=str)
@pytest.mark.parametrize("v,dtype", [(151936, torch.float32), (151936, torch.bfloat16),
                                     (70001, torch.float32)])
def test_values_do_not_depend_on_the_batch(v, dtype, setting):
    # 1, 64, 100, 256 and 700 rows: 8, 8, 4, 2 and 1 blocks a row at the larger size
    g = torch.Generator().manual_seed(9)
    base = torch.cat([zipf(48, v, 7, dtype), (2 * torch.randn(16, v, generator=g)).to(dtype).to(dev())])
    u = uniforms(64, 8)
    want = rlk.sample_logits(base, u, **setting)
    for n in (100, 256, 700):
        at = torch.arange(n, device=dev()) % 64
        got = rlk.sample_logits(base[at], u[at], **setting)
        for a, b in zip(want, got):
            assert torch.equal(a[at], b)
    for i in (0, 17, 63):
        one = rlk.sample_logits(base[i:i + 1], u[i:i + 1], **setting)
        for a, b in zip(want, one):
            assert torch.equal(a[i:i + 1], b)
